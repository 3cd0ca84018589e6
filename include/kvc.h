/*
 * kvc.h -- C ABI of libkvc, the GB300 (sm_103a) budgeted-KV decode step and
 * LaProx prefill scorer.
 *
 * Method sources (web pages), cited per entry point:
 *   MomentKV  "MOMENTKV: Closing the Directional Gap in KV Cache Eviction for
 *             Long-Context Inference" (arXiv 2606.01563)
 *   InertiaKV "Key factors of KV cache eviction in aggressive decoding:
 *             temporal aggregation and rank preservation" (arXiv 2609.03515)
 *   KeepKV    "KeepKV: lossless KV cache compression with electoral votes and
 *             zero-perturbation merging" (reading notes, arXiv 2504.09936)
 *   LaProx    "Reformulating KV Cache Eviction Problem for Long-Context LLM
 *             Inference" (arXiv 2605.07234)
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - A unit is one (sequence, layer, KV head); units are independent.  The
 *   unit index of sequence b, layer l, KV head g is u = (b*NL + l)*Hkv + g.
 *   G = query heads per KV head (GQA group); query head h of the unit is the
 *   group's h-th head.
 * - bf16 values are passed as uint16_t bit patterns.  Every pointer is a
 *   DEVICE pointer owned by the caller unless stated otherwise; the library
 *   allocates no device memory.  Scratch lives in a caller-allocated
 *   workspace whose size the *_workspace_size functions return.
 * - Every call is asynchronous on the CUDA stream passed as `stream`
 *   (a cudaStream_t; NULL = legacy default stream).  Only
 *   kvc_get_device_status blocks.
 * - Arguments are validated on the host before any launch; a failed check
 *   returns an error code, launches nothing and sets kvc_last_error().
 *   Conditions that only the device can see (a unit whose length does not
 *   fit the caller's bounds) set a status word in the workspace and leave
 *   that unit untouched; kvc_get_device_status reads and clears it.
 * - Errors never trap or abort on the device.
 * - Layouts (row-major, innermost last):
 *     q        [U][G][d]   bf16     query of the current step
 *     k_new    [U][d]      bf16     key of the token appended this step
 *     v_new    [U][d]      bf16
 *     K, V     [U][cap][d] bf16     slot i of unit u at (u*cap + i)*d
 *     votes    [U][cap]    int32    integer vote p_i >= 1, or NULL = all 1
 *     pos      [U][cap]    int32    token position of each slot
 *     util     [U][cap]    fp64     aggregated utility m(i); +inf = never
 *                                   scored (protected from eviction).  fp64
 *                                   keeps the order of utilities far below
 *                                   fp32's range (sharp attention)
 *     len      [U]         int32    slots in use (slots [0, len) are live)
 *     moments  n [U], mu_k [U][d], mu_v [U][d], C [U][d][d]   fp32
 *              C[a][b] = cov(v_a, k_b) over the evicted set (population)
 * - Supported shapes: d = 128, G in {1, 2, 4, 8}.
 */
#ifndef KVC_H
#define KVC_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define KVC_VERSION 10400  /* major*10000 + minor*100 + patch */

/* Exported symbols (the library is built with hidden default visibility). */
#if defined(__GNUC__)
#define KVC_API __attribute__((visibility("default")))
#else
#define KVC_API
#endif

typedef enum {
    KVC_OK = 0,
    KVC_ERR_INVALID_ARG = 1,  /* a null pointer or a value out of range      */
    KVC_ERR_SHAPE = 2,        /* sizes inconsistent (e.g. len + 1 > cap)     */
    KVC_ERR_CUDA = 3,         /* a CUDA runtime call failed                  */
    KVC_ERR_TIMEOUT = 4,      /* a bounded device wait ran out               */
    KVC_ERR_UNSUPPORTED = 5,  /* shape outside the supported set             */
    KVC_ERR_WORKSPACE = 6     /* workspace missing, misaligned or too small  */
} kvc_status;

enum {
    KVC_RULE_SINGLE = 0,
    KVC_RULE_CUMULATIVE = 1,
    KVC_RULE_EMA = 2,
    KVC_RULE_MI = 3,
    KVC_RULE_EMA_CHAINED = 4   /* InertiaKV's layer-chained EMA: see
                                  kvc_params.chain_layers */
};
enum { KVC_CORR_OFF = 0, KVC_CORR_ZERO_ORDER = 1, KVC_CORR_FIRST_ORDER = 2 };
enum { KVC_ALLOC_GLOBAL = 0, KVC_ALLOC_LAYER = 1, KVC_ALLOC_HEAD = 2 };

/* Method parameters of a decode stream. */
typedef struct {
    int32_t U;               /* units                                        */
    int32_t G;               /* query heads per KV head (1, 2, 4, 8)         */
    int32_t d;               /* head dimension (128)                         */
    int32_t cap;             /* slot capacity per unit (row stride of K, V)  */
    int32_t L;               /* budget: slots kept per unit after a step     */
    int32_t rule;            /* KVC_RULE_*  (InertiaKV sec 3.1 eqs 2-4;
                                KVC_RULE_EMA_CHAINED: see chain_layers;
                                KVC_RULE_MI: MomentKV's moment-informed
                                score, every step, needs T = 1 and
                                merge = 0; see kvc_mi_scores and
                                kvc_mi_evict)                                */
    float alpha;             /* EMA coefficient, 0 <= alpha < 1              */
    int32_t refresh_period;  /* 0 <= T <= L: utilities refresh on step
                                t = 1 and whenever (t - 1) mod T == 0
                                (InertiaKV-Lazy; T = 1 is full refresh);
                                T = 0 refreshes on step 1 only (InertiaKV
                                Score-Free: the step-1 ranking is frozen)    */
    int32_t correction;      /* KVC_CORR_* (MomentKV sec 4.2 eq 12; the zero-
                                order variant of MomentKV Table 4)           */
    int32_t merge;           /* 0: victims are evicted; 1: a unit removing
                                one slot ZIP-merges its victim instead
                                (KeepKV; see kvc_zip_merge); needs votes     */
    int32_t merge_recent;    /* R >= 0: merge partners exclude the last R
                                token positions (KeepKV candidate choice)    */
    const int32_t *budget;   /* NULL, or a DEVICE array [U]: the budget of
                                each unit (1 <= budget[u] <= L; L is then
                                the largest), e.g. the variable per-head
                                budgets a prefill selection hands over
                                (LaProx key design 3, MomentKV's adaptive
                                per-head allocation; kvc_prefill_handoff).
                                A unit outside [1, L] records KVC_ERR_SHAPE
                                and is left untouched.  Wherever the other
                                entry points say L of a unit, they mean
                                budget[u].  The fused steady state runs when
                                max_len == L + 1 and every unit enters at
                                its own budget.                              */
    int32_t chain_layers;    /* KVC_RULE_EMA_CHAINED (InertiaKV sec 1 and sec
                                3.1, the evaluated implementation: one EMA
                                state updated after each layer): units are
                                grouped by sequence, NL = chain_layers layers
                                of Hkv = chain_heads KV heads (u = (b NL + l)
                                Hkv + g; U a multiple of NL Hkv), every unit
                                of a sequence holding the same positions in
                                the same slots.  On a refresh step each
                                slot's utility passes the layers in order,
                                m = alpha m + (1 - alpha) s_l (m = s_l at the
                                first observation), s_l the layer's mean
                                over its Hkv units' probabilities (all H
                                heads), and is stored in every unit; every
                                unit of the sequence evicts the same slots
                                (budget: the sequence's first unit's).  The
                                call sequence runs (no fused kernel).  Other
                                rules ignore both fields.                    */
    int32_t chain_heads;
} kvc_params;

/* Guard of the ZIP-merge key formula: below this |weighted mean logit| the
 * merged key is the plain mean of the two keys (KeepKV reading notes,
 * "numerical stability" item 2, which gives no value). */
#define KVC_ZIP_EPS 1e-3

/* The budgeted cache of every unit (device pointers, caller-owned). */
typedef struct {
    uint16_t *K;
    uint16_t *V;
    int32_t *votes;   /* NULL = every vote is 1 (no vote weighting)        */
    int32_t *pos;
    double *util;
    int32_t *len;
} kvc_cache;

/* Eviction-set moment statistics (device pointers, caller-owned; zero at the
 * start of each generation, MomentKV sec A4 setup). */
typedef struct {
    float *n;      /* [U]       vote-weighted count n_e                    */
    float *mu_k;   /* [U][d]    key mean k_bar                             */
    float *mu_v;   /* [U][d]    value mean v_bar                           */
    float *C;      /* [U][d][d] S_tilde / n_e, C[a][b] = cov(v_a, k_b)     */
} kvc_moments;

/* ------------------------------------------------------------------ */
/* library                                                             */
/* ------------------------------------------------------------------ */

/* KVC_VERSION of the loaded library. */
KVC_API int32_t kvc_version(void);

/* Message of the last failed call on this host thread ("" if none).  The
 * string is owned by the library and valid until the next call on the same
 * thread. */
KVC_API const char *kvc_last_error(void);

/* Static name of a status code. */
KVC_API const char *kvc_status_string(int32_t status);

/* ------------------------------------------------------------------ */
/* decode step                                                          */
/* ------------------------------------------------------------------ */

/* Bytes of workspace the decode entry points need for these parameters
 * (covers every decode call, including a step-1 pass over cap slots).  The
 * same workspace (device memory, 256-byte aligned) must be passed to every
 * call of one decode stream and left untouched between calls: it carries
 * per-step scratch and per-stream state. */
KVC_API size_t kvc_decode_workspace_size(const kvc_params *p);

/* Zero the workspace's persistent state and status word (enqueued on
 * `stream`).  Call once before the first step of a decode stream. */
KVC_API kvc_status kvc_decode_workspace_init(const kvc_params *p, void *ws,
                                     size_t ws_bytes, void *stream);

/* Read and clear the device status word of a workspace (blocks on `stream`).
 * *device_status receives KVC_OK or the first error a kernel recorded. */
KVC_API kvc_status kvc_get_device_status(void *ws, size_t ws_bytes, void *stream,
                                 int32_t *device_status);

/*
 * kvc_decode_attend -- append the step's token, then vote-weighted
 * single-query GQA attention over every slot of every unit.
 *
 * Defined by: MomentKV sec 2 (s_i = q^T k_i / sqrt(d), Z, alpha_i, f) and
 * Algorithm 1 (append before eviction); KeepKV eq 6 / eq 23 (votes, applied as the
 * logit bias ln p_i, KeepKV "integration" item 2); InertiaKV sec 3.1 eq 1
 * (head-mean probability s_t(i), averaged over the G query heads sharing the
 * KV head).
 *
 * For each unit u (n = len[u] on entry):
 *   slot n receives k_new[u], v_new[u], vote 1, position new_pos, utility
 *   +inf (unscored); len[u] becomes n + 1;
 *   x_hi = q_h . k_i / sqrt(d) + ln p_i, i in [0, n];
 *   lse[u][h]  = log sum_i exp(x_hi);
 *   f_all[u][h][:] = sum_i exp(x_hi - lse) v_i;
 *   probs[u][i] = (1/G) sum_h exp(x_hi - lse_h)   (only if probs != NULL).
 * t is the 1-based decode step (only recorded; it does not change the
 * arithmetic).  max_len >= n + 1 for every unit bounds the launch; a unit
 * with n + 1 > max_len or n + 1 > cap is skipped and sets the device status
 * KVC_ERR_SHAPE.
 * Outputs lse [U][G], f_all [U][G][d] fp32 (required), probs [U][cap] fp64
 * (optional; entries past len untouched).  Logits are fp32; the
 * probabilities are formed in fp64 so that values below fp32's range keep
 * their order.
 */
KVC_API kvc_status kvc_decode_attend(const kvc_params *p, int32_t t, int32_t new_pos,
                             int32_t max_len, const uint16_t *q,
                             const uint16_t *k_new, const uint16_t *v_new,
                             const kvc_cache *cache, float *lse, float *f_all,
                             double *probs, void *ws, size_t ws_bytes,
                             void *stream);

/*
 * kvc_aggregate_evict -- temporal utility update and lowest-utility victim
 * selection.
 *
 * Defined by: InertiaKV sec 3.1 eqs 2-4 (single m = s, cumulative
 * m = m + s, EMA m = alpha m + (1 - alpha) s) and "evict the lowest m_t(i)
 * while the cache exceeds the budget"; InertiaKV-Lazy periodic refresh;
 * MomentKV Algorithm 1 phase 1 (argmin loop).
 *
 * On a refresh step (t = 1, or (t - 1) mod T == 0 when T >= 1) every live
 * slot's utility is updated from probs (required then): an unscored slot
 * takes m = s, a scored one the rule.  On other steps utilities are left as they are.
 * Then k = len[u] - L victims (0 if len <= L) are chosen among scored slots:
 * the k smallest (m, pos) pairs, utility ascending, ties to the smaller
 * token position.  evict_idx[u][0..k) receives their slot indices in
 * ascending slot order, evict_pos (optional) their positions in the same
 * order, n_evict[u] = k.  A unit needing more than kmax victims, or with
 * fewer than k scored slots, gets n_evict = 0 and sets the device status
 * (KVC_ERR_SHAPE / KVC_ERR_INVALID_ARG).  Nothing is removed here.
 */
KVC_API kvc_status kvc_aggregate_evict(const kvc_params *p, int32_t t,
                               const double *probs, const kvc_cache *cache,
                               int32_t kmax, int32_t *evict_idx,
                               int32_t *evict_pos, int32_t *n_evict, void *ws,
                               size_t ws_bytes, void *stream);

/*
 * kvc_moment_update -- fold the evicted tokens into the eviction-set
 * moments, each weighted by its vote.
 *
 * Defined by: MomentKV sec 4.1 "efficient statistics update", Algorithm 1
 * eviction phase and App. A.1 (n_e, s_k, s_v, S updated by addition;
 * S_tilde = S - s_v s_k^T / n_e).  The library keeps the equivalent mean /
 * covariance form (n, mu_k, mu_v, C = S_tilde / n) and updates it with the
 * weighted pairwise merge of Chan, Golub and LeVeque (1979), the one-token
 * case being West's (1979) weighted incremental update.  A vote p counts as
 * p identical tokens (KeepKV eq 6).
 * Reads K, V, votes at evict_idx[u][0..n_evict[u]) (before compaction).
 */
KVC_API kvc_status kvc_moment_update(const kvc_params *p, const kvc_cache *cache,
                             int32_t kmax, const int32_t *evict_idx,
                             const int32_t *n_evict, const kvc_moments *mom,
                             void *ws, size_t ws_bytes, void *stream);

/*
 * kvc_correct -- retained-only attention and the moment-based normalization
 * correction.
 *
 * Defined by: MomentKV Algorithm 1 inference phase, sec 4.1 eq 9
 * (fhat_E = v_bar + S_tilde q / (n_e sqrt d)), sec 4.2 eqs 10-12 (Jensen
 * bound Zhat_E = n_e exp(q . k_bar / sqrt d), w_R = Z_R / (Z_R + Zhat_E)),
 * App. C.2 (log-domain weight); KeepKV eq 3 (o' = (o - A_e v_e)/(1 - A_e)),
 * used to obtain the retained-only output from the full pass.
 *
 * Call after kvc_moment_update and before kvc_compact, with lse / f_all from
 * kvc_decode_attend of the same step.  Per unit and head:
 *   f_R, log Z_R over the live slots not in evict_idx: by the eviction-error
 *     identity when at most 16 slots go and their attention mass is <= 0.5,
 *     otherwise by a direct pass over the retained slots;
 *   n = 0 or correction off: o = f_R;
 *   else log Zhat_E = ln n + q . mu_k / sqrt(d),
 *        fhat_E = mu_v + C q / sqrt(d)   (first order) or mu_v (zero order),
 *        w_R = 1 / (1 + exp(log Zhat_E - log Z_R)),
 *        o = w_R f_R + (1 - w_R) fhat_E.
 * Outputs o [U][G][d] fp32 (required), f_R [U][G][d] and logZ_R [U][G]
 * (optional).
 */
KVC_API kvc_status kvc_correct(const kvc_params *p, const uint16_t *q,
                       const kvc_cache *cache, int32_t kmax,
                       const int32_t *evict_idx, const int32_t *n_evict,
                       const float *lse, const float *f_all,
                       const kvc_moments *mom, float *o, float *f_R,
                       float *logZ_R, void *ws, size_t ws_bytes, void *stream);

/*
 * kvc_mi_scores -- MomentKV moment-informed eviction scores.
 *
 * Defined by: MomentKV sec 4.2 ("moment residual", "moment-aware eviction
 * score") and Algorithm 1, phase 1.  For every live slot i < len[u]:
 *   r_i = v_i - mu_v - C (k_i - mu_k) / sqrt(d)   (the moments as they are:
 *         all zero before the first eviction, so r_i = v_i),
 *   scores[u][i] = probs[u][i] * ||r_i||_2,
 * probs being the head-mean probabilities kvc_decode_attend wrote for this
 * step (the slot's attention weight).  scores may alias probs.  With rule
 * KVC_RULE_MI, kvc_aggregate_evict takes these scores as the utilities of
 * every slot (refreshed every step) and evicts the lowest, for steps that
 * remove one slot; a unit removing more (which MomentKV Algorithm 1 does
 * one fold at a time, re-scoring in between) is refused there with device
 * status KVC_ERR_UNSUPPORTED: use kvc_mi_evict.  fp32 residuals (CUDA
 * cores), fp64 scores.  max_len bounds len[u] (<= cap).
 */
KVC_API kvc_status kvc_mi_scores(const kvc_params *p, const kvc_cache *cache,
                                 const kvc_moments *mom, int32_t max_len,
                                 const double *probs, double *scores, void *stream);

/*
 * kvc_mi_evict -- MomentKV's moment-aware eviction phase for a step that
 * removes several slots.
 *
 * Defined by: MomentKV Algorithm 1, phase 1 (while |R| > L: re-form the
 * means and S_tilde from the running statistics, alpha = softmax over R,
 * score(j) = alpha_j ||r_j||, evict the argmin, fold it, remove it), sec 4.2
 * ("moment residual", "moment-aware eviction score"), sec 4.1 "efficient
 * statistics update".
 *
 * Call right after kvc_decode_attend of the same step, with probs requested
 * there: it reads the logits that call left in the workspace, and lse is
 * that call's output.  For each unit with k = len[u] - L > 0, k rounds:
 * alpha_i = (1/G) sum_h exp(x_hi - lse_h) / Z_h with Z_h summed over the
 * slots still present (fp64), r_i = v_i - mu_v - C (k_i - mu_k) / sqrt(d)
 * with the moments as they stand, the lowest alpha_i ||r_i|| goes (ties to
 * the smaller position) and is folded into the moments (weighted by its
 * vote, KeepKV eq 6).  evict_idx / evict_pos (optional) [U][kmax] receive
 * the victims in eviction order, n_evict[u] = k, util[i] the last score of
 * each slot still present.  Nothing is compacted: kvc_correct (whose
 * moments are then already folded: do not call kvc_moment_update) and
 * kvc_compact follow.  Each round re-scores the whole unit (O(len d^2)):
 * max_len <= 8192 and (max_len - L) * max_len <= 2^22, else
 * KVC_ERR_UNSUPPORTED (compress a long prompt first).  kmax >=
 * max_len - L.  fp32 residuals, fp64 weights and scores.
 */
KVC_API kvc_status kvc_mi_evict(const kvc_params *p, int32_t max_len, const kvc_cache *cache,
                                const kvc_moments *mom, const float *lse, int32_t kmax,
                                int32_t *evict_idx, int32_t *evict_pos, int32_t *n_evict,
                                void *ws, size_t ws_bytes, void *stream);

/*
 * kvc_zip_merge -- merge each unit's single victim into its most similar
 * slot instead of evicting it.
 *
 * Defined by: KeepKV reading notes, "ZIP-Merging" (eq 7 votes p_r = p_e +
 * p_c, eq 8 score condition, eq 10 value, eq 12 key, Thm 3 single-step
 * lossless), "why cosine similarity" (partner = most similar key, the most
 * recent R tokens excluded) and "numerical stability" item 2 (guard).
 *
 * Call after kvc_aggregate_evict and before kvc_moment_update, with q and
 * new_pos of the same step; needs cache->votes.  For each unit with
 * n_evict[u] == 1 and victim slot e = evict_idx[u][0]:
 *   candidates c: live slots other than e with pos <= new_pos - R
 *     (R = p->merge_recent); partner = the largest cos(k_e, k_c) (0 when a
 *     key is zero), ties to the smaller position.  No candidate: nothing
 *     happens (the victim is evicted by the calls that follow).
 *   xbar_j = (1/G) sum_h q_h . k_j / sqrt(d) (the group's mean query;
 *     G = 1 is the page's single-head score), w_j = p_j exp(xbar_j),
 *     lambda_j = w_j / (w_e + w_c), xt = lambda_e xbar_e + lambda_c xbar_c,
 *     ell = ln((w_e + w_c) / (p_e + p_c));
 *   v_c := lambda_e v_e + lambda_c v_c;
 *   k_c := (lambda_e k_e + lambda_c k_c) ell / xt, or (k_e + k_c) / 2 when
 *     |xt| < KVC_ZIP_EPS (both rounded to bf16, nearest even);
 *   votes[c] := p_e + p_c; util[c] := util[c] + util[e]; pos[c] kept;
 *   slot e is refilled from slot len - 1 (all fields), len[u] -= 1 and
 *   n_evict[u] := 0, so the moment fold, the correction (which then returns
 *   the output over every slot of the step, as KeepKV attends before it
 *   compresses) and the compaction leave the unit alone.
 * partner_pos [U] (optional) receives the partner's position or -1.
 * Scores and weights are fp32; cosine near-ties (|difference| ~ 1e-6) may
 * resolve either way.
 */
KVC_API kvc_status kvc_zip_merge(const kvc_params *p, int32_t new_pos, const uint16_t *q,
                                 const kvc_cache *cache, int32_t kmax,
                                 const int32_t *evict_idx, int32_t *n_evict,
                                 int32_t *partner_pos, void *ws, size_t ws_bytes,
                                 void *stream);

/*
 * kvc_compact -- remove the evicted slots (MomentKV Algorithm 1, end of the
 * eviction phase).
 * Live slots keep their contents; the slot order is not significant (slots
 * are identified by position).  With n = len - k, every evicted slot below
 * n is filled by a live slot at or above n (both taken in ascending order);
 * K, V, votes, pos and util move together; len[u] = n.
 */
KVC_API kvc_status kvc_compact(const kvc_params *p, const kvc_cache *cache,
                       int32_t kmax, const int32_t *evict_idx,
                       const int32_t *n_evict, void *ws, size_t ws_bytes,
                       void *stream);

/*
 * kvc_decode_step -- the whole decode step, fused: the same results as
 * kvc_decode_attend, kvc_aggregate_evict, kvc_moment_update, kvc_correct and
 * kvc_compact called in that order (same sets; outputs within fp32
 * rounding); with p->merge = 1, kvc_zip_merge runs between
 * kvc_aggregate_evict and kvc_moment_update; with rule KVC_RULE_MI,
 * kvc_mi_scores runs between kvc_decode_attend and kvc_aggregate_evict when
 * one slot goes, and kvc_mi_evict replaces kvc_mi_scores,
 * kvc_aggregate_evict and kvc_moment_update when several go (the call
 * sequence; no fused kernel; evict_idx / evict_pos then in eviction order,
 * and the bounds of kvc_mi_evict apply).
 *
 * In the steady state (max_len == L + 1: every unit enters with len = L and
 * evicts exactly one slot) one cluster kernel per step does everything: the
 * new token is written straight into the victim's slot.  Otherwise (e.g.
 * step 1 over the prefill cache) the five-call sequence runs.
 * probs (optional [U][cap] fp64) receives the head-mean probabilities on refresh
 * steps in the slot order of the step's input (the new token at index
 * len); evict_pos / evict_idx (optional [U][kmax]) the evicted positions /
 * slot indices; n_evict [U] (required) the victim counts; o [U][G][d] the
 * corrected output.
 */
KVC_API kvc_status kvc_decode_step(const kvc_params *p, int32_t t, int32_t new_pos,
                           int32_t max_len, const uint16_t *q,
                           const uint16_t *k_new, const uint16_t *v_new,
                           const kvc_cache *cache, const kvc_moments *mom,
                           float *o, double *probs, int32_t kmax,
                           int32_t *evict_idx, int32_t *evict_pos,
                           int32_t *n_evict, void *ws, size_t ws_bytes,
                           void *stream);

/*
 * kvc_decode_attend_noalloc -- kvc_decode_attend for callers that cannot
 * allocate device memory.  The pages have no counterpart to this entry
 * point; it exists for hosts that own every device allocation (a serving
 * runtime that reserves its memory pool at start-up and allows no cudaMalloc
 * afterwards, a plugin interface that passes tensors but no workspace).
 *
 * Same arguments, arithmetic, outputs and argument checks (with the same
 * status codes) as kvc_decode_attend, without the workspace: the scratch
 * (status word, logits, split partials, lengths) lives in a static device
 * array of 32 MiB inside the library, which every GPU that loads the library
 * holds until the process exits.  The call allocates nothing (no cudaMalloc,
 * cudaFree or allocating library routine).
 * - Sizes whose scratch exceeds 32 MiB are rejected with KVC_ERR_WORKSPACE
 *   and a message.  The scratch is about U*ceil(cap/1024)*G*520 bytes, plus
 *   U*G*cap*4 bytes of logits when probs != NULL (the logits are only kept
 *   to form the probabilities).
 * - Each call looks up the array's device address in the calling thread's
 *   current device context (cudaGetSymbolAddress), so a device reset or a
 *   change of context needs nothing from the caller.  The first call on a
 *   device also loads the library's device code there, the 32 MiB array
 *   with it: make that first call before any stream capture, and while
 *   32 MiB of device memory are free (a host that reserves the whole device
 *   for its pool calls once before reserving it, or loads modules eagerly,
 *   CUDA_MODULE_LOADING=EAGER); a load that finds no room returns
 *   KVC_ERR_CUDA.
 * - Every call on a device shares the one array and it keeps the previous
 *   call's contents: calls whose kernels overlap on the GPU race and must be
 *   ordered by the caller (one stream, or events).
 * - device_status (optional device pointer to one int32) receives the device
 *   status of this call (KVC_OK or the KVC_ERR_* a kernel recorded, e.g.
 *   KVC_ERR_SHAPE for a unit with len + 1 > max_len, which is left
 *   untouched).  With device_status = NULL such device-side errors are
 *   discarded: there is no workspace to read them from later.
 */
KVC_API kvc_status kvc_decode_attend_noalloc(const kvc_params *p, int32_t t,
                                             int32_t new_pos, int32_t max_len,
                                             const uint16_t *q, const uint16_t *k_new,
                                             const uint16_t *v_new,
                                             const kvc_cache *cache, float *lse,
                                             float *f_all, double *probs,
                                             int32_t *device_status, void *stream);

/* ------------------------------------------------------------------ */
/* drafted tokens (speculative decoding over the budgeted cache)        */
/* ------------------------------------------------------------------ */

/*
 * One verification of a tree of drafted tokens takes three calls:
 *   kvc_tree_attend   every drafted token attends over the cache and the
 *                     drafted tokens its mask shows; the cache does not
 *                     change;
 *   (the caller samples and accepts a path of the tree)
 *   kvc_tree_weights  the attention weight the accepted tokens gave to every
 *                     slot (from the lse of the first call);
 *   kvc_tree_commit   appends the accepted tokens, updates the utilities with
 *                     those weights and evicts down to the budget.
 * The pages decode one token per step; a verification step of several tokens
 * is this library's own extension of their definitions, cited per call.
 * A tree belongs to a sequence: `units` consecutive units (NL * Hkv of one
 * call, Hkv when the layers are called one by one) share its mask and path.
 * The calls may alternate with kvc_decode_step on the same cache.  Outputs do
 * not overlap inputs.
 */
typedef struct {
    int32_t T;              /* drafted tokens per tree, 1..64: the row stride of
                               q, k_tree, v_tree, o, lse and mask            */
    int32_t units;          /* units per tree; unit u belongs to tree
                               u / units; U is a multiple of units           */
    const uint64_t *mask;   /* DEVICE [U/units][T]: bit j of token i's word is
                               set when i attends drafted token j (its
                               ancestors and itself; any mask is allowed)    */
    const int32_t *n;       /* DEVICE [U/units] live tokens of each tree, 0..T,
                               or NULL = T.  Tokens at or behind it do not
                               exist: their rows of the inputs are not used
                               (they may hold anything, NaN included), their
                               rows of the outputs are left as they were     */
} kvc_tree;

typedef struct {
    int32_t A;              /* row stride of token and row_weight, 1..T      */
    const int32_t *token;   /* DEVICE [U/units][A] the accepted tokens, in the
                               order they are appended (root first); any
                               live tokens (one that is named twice counts
                               and is appended twice)                        */
    const int32_t *n;       /* DEVICE [U/units] accepted tokens, 0..A        */
    const int32_t *pos;     /* DEVICE [U/units] position of the first of them;
                               the j-th has pos + j                          */
} kvc_path;

/* Bytes of workspace kvc_tree_attend and kvc_tree_weights need for trees of
 * T tokens (0: invalid parameters).  Its first 256 bytes hold the status word
 * kvc_get_device_status reads: zero them once before the first call.  The
 * rest is scratch of one call; calls that overlap on the GPU need a workspace
 * each. */
KVC_API size_t kvc_tree_workspace_size(const kvc_params *p, int32_t T);

/*
 * kvc_tree_attend -- attention of drafted tokens over the cache and their
 * tree, with the normalization correction.
 *
 * Defined by: MomentKV sec 2 and KeepKV eq 6 as in kvc_decode_attend;
 * MomentKV sec 4.1 eq 9, sec 4.2 eqs 10-12, App. C.2 as in kvc_correct.
 * For unit u (n = len[u]), live drafted token t and query head h:
 *   x_i = q_th . k_i / sqrt(d) + ln p_i      cache slots i in [0, n)
 *   y_j = q_th . k_tree_j / sqrt(d)          live j with bit j of mask[t]
 *   lse = log(sum_i exp(x_i) + sum_j exp(y_j)),
 *   f   = (sum_i exp(x_i) v_i + sum_j exp(y_j) v_tree_j) / exp(lse)
 *   o   = f without moments (mom NULL, p->correction = KVC_CORR_OFF, or
 *         n_e[u] = 0); otherwise w f + (1 - w) fhat, with
 *         fhat = mu_v + C q / sqrt(d)  (KVC_CORR_ZERO_ORDER: mu_v),
 *         w = 1 / (1 + exp(ln n_e + q . mu_k / sqrt(d) - lse)).
 *   A row that sees nothing (empty cache, no bit) has lse = -inf, f = 0 (and
 *   o = fhat with moments).
 * What a row does not see does not reach it, NaN and infinities included.
 * q [U][T][G][d], k_tree, v_tree [U][T][d] bf16; o [U][T][G][d] bf16 (the
 * type the output projection reads; fp32 until that one rounding, but the
 * softmax weights are rounded to bf16 for the tensor cores and C enters as two
 * bf16 terms, 2^-16 of each product), lse [U][T][G] fp32.  A count n_e that is
 * NaN gives that unit NaN, as in kvc_correct.
 * Reads K, V, votes and len of the cache.  max_len >= len[u] bounds the
 * launch.  Device-side errors, which leave the unit's outputs untouched:
 * KVC_ERR_SHAPE (len[u] outside [0, max_len]), KVC_ERR_INVALID_ARG (live
 * tokens outside [0, T]).
 */
KVC_API kvc_status kvc_tree_attend(const kvc_params *p, int32_t max_len, const kvc_tree *tree,
                                   const uint16_t *q, const uint16_t *k_tree,
                                   const uint16_t *v_tree, const kvc_cache *cache,
                                   const kvc_moments *mom, uint16_t *o, float *lse, void *ws,
                                   size_t ws_bytes, void *stream);

/*
 * kvc_tree_weights -- accumulated attention weight of the accepted tokens.
 *
 * Defined by: InertiaKV sec 3.1 eq 1 (head-mean probability), summed over the
 * accepted tokens with weights w_j = row_weight[j] (KeepKV reading notes eq
 * 15 has such a windowed sum; NULL = 1, the plain accumulation).
 * With the accepted tokens c_0 .. c_{a-1} of unit u's tree and lse from
 * kvc_tree_attend of the same tree:
 *   S[u][i]     = sum_j w_j (1/G) sum_h exp(x_{c_j h i} - lse_{c_j h}),
 *                 i in [0, n) with x as above;
 *   S[u][n + r] = sum over the j whose mask shows c_r of
 *                 w_j (1/G) sum_h exp(q_{c_j h} . k_tree_{c_r} / sqrt(d)
 *                 - lse_{c_j h}),  r in [0, a)
 * (where kvc_tree_commit appends c_r).  Entries from n + a on are left as
 * they were; a = 0 gives S = 0 on [0, n).  Rows with lse = -inf give nothing.
 * row_weight: DEVICE [U/units][A] fp32, >= 0 (a negative weight gives NaN).
 * S [U][cap] fp32: a weight below fp32's range is 0, so over sharp attention
 * (logits further apart than about 87) slots tie that the method orders.  With
 * S in fp64 (kvc_tree_weights_f64) they do not: a weight has the one-token
 * calls' range and is held to fp32's precision.  The logits are formed again
 * from the keys (256 bytes per slot): which rows count is known only after the
 * verification, and keeping all T G logits per slot would move more.
 * max_len >= len[u].  Device-side errors, which leave the unit's
 * entries untouched: KVC_ERR_SHAPE (len[u] outside [0, max_len], or len[u] +
 * a > cap), KVC_ERR_INVALID_ARG (a outside [0, A], an accepted token that is
 * not live, live tokens outside [0, T]).
 */
KVC_API kvc_status kvc_tree_weights(const kvc_params *p, int32_t max_len, const kvc_tree *tree,
                                    const kvc_path *path, const float *row_weight,
                                    const uint16_t *q, const uint16_t *k_tree, const float *lse,
                                    const kvc_cache *cache, float *S, void *ws, size_t ws_bytes,
                                    void *stream);
/* The same with S in fp64 (8-byte aligned), read by kvc_tree_commit_f64. */
KVC_API kvc_status kvc_tree_weights_f64(const kvc_params *p, int32_t max_len,
                                        const kvc_tree *tree, const kvc_path *path,
                                        const float *row_weight, const uint16_t *q,
                                        const uint16_t *k_tree, const float *lse,
                                        const kvc_cache *cache, double *S, void *ws,
                                        size_t ws_bytes, void *stream);

/*
 * kvc_tree_commit -- append the accepted tokens and evict by accumulated
 * attention weight.
 *
 * Defined by: InertiaKV sec 3.1 eqs 2-4 and MomentKV Algorithm 1 as in
 * kvc_aggregate_evict, kvc_moment_update and kvc_compact, for a step that
 * appends a >= 0 tokens: the verification is one observation of weight S.
 * For unit u, n = len[u]:
 *   slots n .. n+a-1 receive the accepted tokens (k_tree, v_tree rows, vote
 *     1, positions pos + j, unscored);
 *   with S (from kvc_tree_weights): util of every slot i < n + a becomes S_i
 *     when unscored or under KVC_RULE_SINGLE, util + S_i (KVC_RULE_CUMULATIVE)
 *     or alpha util + (1 - alpha) S_i (KVC_RULE_EMA).  Without (S = NULL, a
 *     verification that does not refresh): utilities stay, the accepted
 *     tokens are unscored (protected);
 *   k = max(0, n + a - budget) victims: the lowest (util, pos) pairs among
 *     the scored slots, ties of both to the lower slot; evict_idx / evict_pos
 *     (optional, [U][kmax]) receive their slots and positions in ascending
 *     slot order, n_evict[u] = k;
 *   the victims are folded into the moments, weighted by their votes (mom
 *     NULL: they are dropped);
 *   with n' = n + a - k: the r-th victim slot below n' receives the r-th
 *     other slot at or above n' (kvc_compact's rule), len[u] = n'.  Slots at
 *     or behind n' are not written, except that the utilities of slots below
 *     the old n are updated.
 * Not combined with merging, KVC_RULE_MI (its score is not an attention
 * weight alone) or KVC_RULE_EMA_CHAINED (KVC_ERR_UNSUPPORTED).  kmax in
 * [1, 64] (KVC_ERR_UNSUPPORTED above: bring a cache that far over its budget
 * down with kvc_decode_step or kvc_aggregate_evict first).  max_len >=
 * len[u] on entry.  ws: the decode stream's workspace
 * (kvc_decode_workspace_size); the victim queue it keeps for lazy steps is
 * dropped.  Device-side errors, which leave the unit as it was with
 * n_evict = 0: KVC_ERR_SHAPE (len[u] outside [0, max_len], len[u] + a > cap,
 * budget[u] outside [1, L], k > kmax), KVC_ERR_INVALID_ARG (the path, as in
 * kvc_tree_weights; fewer than k scored slots, which is seen once the
 * utilities are updated).
 */
KVC_API kvc_status kvc_tree_commit(const kvc_params *p, int32_t max_len, const kvc_tree *tree,
                                   const kvc_path *path, const uint16_t *k_tree,
                                   const uint16_t *v_tree, const float *S,
                                   const kvc_cache *cache, const kvc_moments *mom, int32_t kmax,
                                   int32_t *evict_idx, int32_t *evict_pos, int32_t *n_evict,
                                   void *ws, size_t ws_bytes, void *stream);
/* The same with S in fp64 (8-byte aligned; NULL: no refresh). */
KVC_API kvc_status kvc_tree_commit_f64(const kvc_params *p, int32_t max_len,
                                       const kvc_tree *tree, const kvc_path *path,
                                       const uint16_t *k_tree, const uint16_t *v_tree,
                                       const double *S, const kvc_cache *cache,
                                       const kvc_moments *mom, int32_t kmax, int32_t *evict_idx,
                                       int32_t *evict_pos, int32_t *n_evict, void *ws,
                                       size_t ws_bytes, void *stream);

/* ------------------------------------------------------------------ */
/* in front of the cache: norms and rotation of a step's heads          */
/* ------------------------------------------------------------------ */

/*
 * The method's sources begin at q, k_new and v_new of a step; these calls, which
 * the sources do not describe, make them of a projection's rows.
 */
typedef struct {
    int32_t Hq, Hkv;        /* query and KV heads of a row; Hq = G Hkv, G in
                               {1, 2, 4, 8}, Hkv <= 4096                     */
    int32_t d;              /* head dimension (128)                          */
    int32_t rot;            /* leading dimensions of a head that are rotated:
                               0 (none) or a multiple of 16 up to d          */
    int32_t interleaved;    /* 0: pairs (i, i + rot/2); 1: (2i, 2i + 1)      */
    float eps;              /* of the norms, >= 0                            */
    float scale;            /* factor of cosine and sine (1; the length
                               extensions that scale attention have another) */
    const uint16_t *q_weight;   /* DEVICE [d] bf16: the norm's weights of the
                               query heads, or NULL: they are not normed     */
    const uint16_t *k_weight;   /* the same of the key heads                 */
    const double *inv_freq;     /* DEVICE [rot/2] radians per position, finite
                               (8-byte aligned; NULL with rot = 0)           */
    int32_t units;          /* units from one sequence to the next in the
                               outputs (NL Hkv; Hkv when the layers are
                               called one by one)                            */
    int32_t first_unit;     /* unit of KV head 0 within a sequence:
                               first_unit + Hkv <= units                     */
} kvc_rope;

/*
 * kvc_qk_norm_rope -- norms and rotation of the query and key heads of B
 * sequences of T tokens, in one pass, from the projection's rows to the unit
 * layouts of the other calls.
 *
 * Row (b, t) of qkv, at (b T + t) * row_stride elements, holds Hq query heads,
 * Hkv key heads and Hkv value heads of d elements each.  For a query or key
 * head x with weights w, position p = pos[b][t]:
 *   y = x w / sqrt(mean(x^2) + eps)                 (y = x without weights)
 *   pair i of the rotated dimensions, a_i = p inv_freq[i]:
 *     (y_1, y_2) -> scale (y_1 cos a_i - y_2 sin a_i, y_2 cos a_i + y_1 sin a_i)
 *   rounded once, to bf16; value heads are copied.
 * KV head g of sequence b is unit u = b units + first_unit + g, and query head
 * h belongs to KV head h / G: q [U][T][G][d], k and v [U][T][d] bf16, as
 * kvc_decode_step (T = 1), the drafted-token calls and the prefill calls take
 * them.  Any of q, k, v may be NULL (not written), one at least is not.
 * All in fp32 but the angles: these are fixed-point fractions of a turn, with
 * the product by the position exact modulo a turn (inv_freq / 2 pi rounded to
 * 53 bits), so far positions lose nothing.  A normed row whose squares sum
 * past fp32's range has y = 0 (NaN where it was infinite), a row of zeros with
 * eps = 0 is NaN; a dimension that is not turned reaches no other.
 * pos [B][T] int32 (any value).  n: DEVICE [B] live tokens of each sequence,
 * taken as within [0, T], or NULL = T: rows of the outputs at or behind it are
 * left as they were, rows of the inputs there are not used.
 * qkv, q, k, v and the weights are 16-byte aligned; row_stride >= (Hq + 2 Hkv)
 * d, a multiple of 8.  Outputs do not overlap inputs.
 */
KVC_API kvc_status kvc_qk_norm_rope(const kvc_rope *r, int32_t B, int32_t T, const uint16_t *qkv,
                                    int64_t row_stride, const int32_t *pos, const int32_t *n,
                                    uint16_t *q, uint16_t *k, uint16_t *v, void *stream);

/* ------------------------------------------------------------------ */
/* beside the budgeted cache: a cache in pages                          */
/* ------------------------------------------------------------------ */

/*
 * (Here a page is a piece of memory, not a source.)
 * A prompt before its selection, or a layer that keeps all of its tokens, lives
 * in pages of a pool that sequences share: no rows are reserved, and a row may
 * be held in 8 bits.  kvc_page_write puts rows in, kvc_page_attend appends one
 * token and attends over the pages, kvc_page_read gives rows back in bf16 (the
 * prompt for the prefill scorer, or what a selection keeps for the budgeted
 * cache).
 */
enum {
    KVC_PAGE_BF16 = 0,      /* rows of d bf16                                */
    KVC_PAGE_E4M3 = 1       /* rows of d e4m3 values with an fp32 scale each:
                               scale = max(max |x| / 448, 2^-126),
                               value = e4m3(x (1 / scale)), nearest even,
                               at most 448 in magnitude; a row that holds a
                               NaN or an infinity is NaN when read           */
};

typedef struct {
    int32_t U;              /* units                                         */
    int32_t d;              /* head dimension (128)                          */
    int32_t type;           /* KVC_PAGE_*                                    */
    int32_t heads;          /* units that share a table and a length: unit u
                               is head u % heads of sequence u / heads; 1: a
                               table per unit (a budget of its own).  Divides
                               U; S = U / heads                              */
    int32_t page;           /* slots per page: 16, 32, 64 or 128             */
    int32_t n_pages;        /* pages of the pool                             */
    int32_t stride;         /* entries per row of the table: a sequence has
                               room for stride * page slots (< 2^31 - 128)   */
    void *K, *V;            /* DEVICE [n_pages][heads][page][d]              */
    float *k_scale, *v_scale;   /* DEVICE [n_pages][heads][page]; NULL with
                               KVC_PAGE_BF16                                 */
    const int32_t *table;   /* DEVICE [S][stride]: slot i of a sequence is row
                               i % page of page table[i / page].  Entries
                               behind a call's last slot are not read (but
                               the first by kvc_page_attend)                 */
    const int32_t *len;     /* DEVICE [S] slots in use.  No call changes it:
                               one array may serve every layer of a step, and
                               the caller advances it once                   */
} kvc_pages;

/* Bytes of workspace the calls below need with G query heads per KV head
 * (kvc_page_write and kvc_page_read: the first 256).  Zero it once before the
 * first call; its first 256 bytes hold the status word kvc_get_device_status
 * reads.  Calls that overlap on the GPU need a workspace each.  0: invalid
 * parameters. */
KVC_API size_t kvc_page_workspace_size(const kvc_pages *pg, int32_t G);

/*
 * kvc_page_write -- rows into pages, quantised as they are written.
 *
 * k, v [U][T][d] bf16 (16-byte aligned): of every unit of sequence s, rows
 * t < count[s] go to slots first[s] + t.  first: DEVICE [S] or NULL (0);
 * count: DEVICE [S] or NULL (T).  len is not used (first may be it).  A slot
 * is written by one row of one sequence; pages shared by sequences (a common
 * prefix) are written through one of them.
 * Device-side errors: KVC_ERR_SHAPE (count outside [0, T], slots outside
 * [0, stride * page)), which leaves the sequence as it was;
 * KVC_ERR_INVALID_ARG (a page outside the pool), whose rows are not written.
 */
KVC_API kvc_status kvc_page_write(const kvc_pages *pg, int32_t T, const int32_t *first,
                                  const int32_t *count, const uint16_t *k, const uint16_t *v,
                                  void *ws, size_t ws_bytes, void *stream);

/*
 * kvc_page_read -- rows out of pages, in bf16 (value * scale, rounded once).
 *
 * For unit u and i < count[u], rows k_out[u][i], v_out[u][i] receive slot
 * slots[u][i] (any order, repeats allowed), or slot i where slots is NULL.
 * slots: DEVICE [U][M] or NULL; count: DEVICE [U] or NULL (M; without slots the
 * lesser of M and the length).  k_out, v_out [U][ld][d] bf16 (16-byte aligned),
 * ld >= M: with ld = cap the rows of a budgeted cache.  Rows at or behind the
 * count are left as they were.
 * Device-side errors: KVC_ERR_SHAPE (count outside [0, M], which leaves the
 * unit's rows as they were; a slot outside [0, len), whose row is left),
 * KVC_ERR_INVALID_ARG (a page outside the pool, whose rows are left).
 */
KVC_API kvc_status kvc_page_read(const kvc_pages *pg, int32_t M, int32_t ld, const int32_t *slots,
                                 const int32_t *count, uint16_t *k_out, uint16_t *v_out, void *ws,
                                 size_t ws_bytes, void *stream);

/*
 * kvc_page_attend -- append one token, then its attention over the pages.
 *
 * Defined by: MomentKV sec 2 as in kvc_decode_attend (append before the
 * attention), without votes.  For unit u of sequence s, n = len[s]:
 *   with k_new, v_new [U][d] bf16, slot n receives them (quantised) and n
 *   below is n + 1; with both NULL nothing is appended;
 *   x_i = q_h . k_i / sqrt(d), i in [0, n), over the values as they are held;
 *   lse = log sum_i exp(x_i), o = sum_i exp(x_i - lse) v_i.
 *   n = 0: lse = -inf, o = 0.
 * A sequence of length 0 whose first entry of the table is -1 is a free place of
 * the batch: a call that appends leaves its outputs as they were and records no
 * error.
 * A NaN or an infinity of a value row reaches o alone, not lse; one in a key row
 * makes the logits it enters NaN or infinite, and where one is NaN or +infinite
 * lse and o of the head are NaN (all of them -infinite: as n = 0).
 * q [U][G][d] bf16; o [U][G][d] bf16 (the type the output projection reads),
 * lse [U][G] fp32.  q, o, k_new, v_new are 16-byte aligned.  Logits, sums and
 * outputs are fp32 until that one rounding; weights enter the products as two
 * 16-bit terms (2^-17 of a weight is left out with bf16 values; with e4m3 ones
 * 2^-22, and 2^-31 of the largest contribution); one below 2^-126 of the
 * largest may count as none, and bf16 values whose sum, over weights of up to
 * 2^8 each, passes fp32's range are infinite.  Beside e4m3 keys an element of q
 * keeps its bits down to 2^-27 of its head's largest.  max_len bounds n with the
 * appended token, 1 <= max_len <= stride * page; a bound far above the lengths
 * costs short units a few microseconds, no more.  Outputs do not overlap inputs;
 * calls that append to the same units are ordered by the caller.
 * Device-side errors, which leave the outputs of the units concerned as they
 * were: KVC_ERR_SHAPE (len[s] < 0, or n with the appended token above
 * max_len), KVC_ERR_INVALID_ARG (a page outside the pool).
 */
KVC_API kvc_status kvc_page_attend(const kvc_pages *pg, int32_t G, int32_t max_len,
                                   const uint16_t *q, const uint16_t *k_new,
                                   const uint16_t *v_new, uint16_t *o, float *lse, void *ws,
                                   size_t ws_bytes, void *stream);

/* ------------------------------------------------------------------ */
/* prefill -> decode hand-off                                           */
/* ------------------------------------------------------------------ */

/* Bytes of workspace kvc_prefill_handoff needs for U units of N prompt
 * tokens. */
KVC_API size_t kvc_prefill_handoff_workspace_size(int32_t U, int32_t N);

/*
 * kvc_prefill_handoff -- start a decode stream from a prefill selection.
 *
 * Defined by: LaProx key design 3 (the kept set of a global or per-layer
 * selection gives every (layer, KV head) its own budget) and MomentKV's
 * setup (the prompt is compressed before decoding, sec A4; the moment
 * statistics start at zero at the start of each generation and every
 * evicted token is folded, Algorithm 1 / sec 4.1 "efficient statistics
 * update"); KeepKV eq 15 for the optional initial utilities.
 *
 * keep [U][N] uint8 is the kept mask of a prefill selection (the
 * [NL][Hkv][N] output of kvc_prefill_score / kvc_prefill_snapkv of one
 * sequence is [U][N] with U = NL * Hkv; B sequences stack their masks);
 * K_src, V_src [U][N][d] bf16 are the prompt's keys and values in the same
 * order; votes_src [U][N] int32 or NULL (all 1); util_init [U][N] fp64 or
 * NULL.  For every unit u, with c = the number of kept tokens:
 *   slots [0, c) of cache receive the kept tokens in ascending position
 *     (K, V rows; pos = the token's index i in the prompt; votes (when the
 *     cache has votes) = votes_src or 1; util = util_init[u][i], i.e.
 *     scored, or +inf (unscored) when util_init is NULL); len[u] = c;
 *   the moments are reset and every token not kept is folded into them,
 *     weighted by its vote (the vote-weighted mean / covariance of the
 *     prompt's evicted set);
 *   budget[u] (optional DEVICE output [U]) = max(c, 1): the budget to
 *     decode with (pass it as kvc_params.budget, with L >= every budget).
 *     A unit that kept nothing decodes with budget 1 (every decode step
 *     appends before it evicts); its first step leaves it at length 1, so
 *     that step must not take the fused steady-state path (pass max_len !=
 *     L + 1, e.g. L + 2 when cap allows).
 * p: the decode stream's parameters (U, G, d, cap; budget is not read
 * here).  A unit whose c exceeds cap - 1 records KVC_ERR_SHAPE and gets
 * len 0.  Device memory ws of kvc_prefill_handoff_workspace_size(U, N)
 * bytes (256-byte aligned) carries the evicted lists and a status word
 * (KVC_ERR_* of the call; read it with kvc_get_device_status(ws, ...)).
 */
KVC_API kvc_status kvc_prefill_handoff(const kvc_params *p, int32_t N, const uint8_t *keep,
                                       const uint16_t *K_src, const uint16_t *V_src,
                                       const int32_t *votes_src, const double *util_init,
                                       const kvc_cache *cache, const kvc_moments *mom,
                                       int32_t *budget, void *ws, size_t ws_bytes,
                                       void *stream);

/* ------------------------------------------------------------------ */
/* prefill scorer                                                       */
/* ------------------------------------------------------------------ */

/*
 * kvc_prefill_prepare -- per-group value-norm factors of the output
 * projection, once per weight set.
 *
 * Defined by: LaProx key design 1 (Output = sum_h A^h (V^h W_O^h)) and its
 * GQA group-mean paragraph.  Reading: the group's attention is the mean over
 * its query heads, so the group's product is A_bar V_g W_g with
 * W_g = sum of W_O^h over the group's heads (W_O^h = rows [h d, (h+1) d)).
 * Gram = W_g W_g^T is accumulated in fp64 and factored in fp64 by pivoted
 * Cholesky; R[l][g] (d x d, fp32) satisfies R^T R = Gram, so that
 * ||(V W_g)[i,:]||_2 = ||R v_i||_2 (a sum of squares, free of cancellation).
 * W_O [NL][Hq*d][D] bf16; R [NL][Hkv][d][d] fp32, 16-byte aligned.
 */
KVC_API kvc_status kvc_prefill_prepare(int32_t NL, int32_t Hq, int32_t Hkv, int32_t d,
                               int32_t D, const uint16_t *W_O, float *R,
                               void *stream);

/* Bytes of workspace kvc_prefill_score needs. */
KVC_API size_t kvc_prefill_workspace_size(int32_t NL, int32_t Hkv, int32_t N,
                                  int64_t B_total);

/*
 * kvc_prefill_score -- LaProx indicator, per-layer normalization and one
 * model-wide top-K.
 *
 * Defined by: LaProx key design 1 (p_i = ||A[:,i]||_2 ||(V W_O)[i,:]||_2),
 * key design 2 (s_{l,j} = p_{l,j} / sum_k p_{l,k}), key design 3 (global
 * top-K under B_total), the GQA group-mean attention paragraph; the
 * observation window of the last w prompt queries (SnapKV protocol, MomentKV
 * sec A4).
 *   window query j (0..w-1) sits at position N - w + j and sees keys
 *   0..N-w+j; A^h = row softmax of q K^T / sqrt(d); A_bar = mean over the
 *   group's G heads; c_i = ||A_bar[:, i]||_2; r_i = ||R v_i||_2;
 *   p = c r; s = p / (sum of p over the layer's heads and tokens) when
 *   normalize != 0, else s = p; keep the B_total largest s over all
 *   (l, g, i), equal scores kept in ascending flat index (l*Hkv + g)*N + i.
 * alloc selects the budget allocation of LaProx's ablation table:
 *   KVC_ALLOC_GLOBAL  the above (head- and layer-flatten: LaProx itself);
 *   KVC_ALLOC_LAYER   head-flatten only: each layer keeps its B_total / NL
 *                     largest s over its heads and tokens (Hkv <= 64);
 *   KVC_ALLOC_HEAD    uniform: each (layer, KV head) keeps its
 *                     B_total / (NL Hkv) largest s;
 *   B_total must be a multiple of the number of segments
 *   (KVC_ERR_INVALID_ARG); ties as above; idx stays ascending.
 * q_win [NL][Hq][w][d] bf16 (4-byte aligned), K, V [NL][Hkv][N][d] bf16
 * (16-byte aligned); R from kvc_prefill_prepare.  Outputs: scores
 * [NL][Hkv][N] fp32, keep [NL][Hkv][N] uint8 (0/1), counts [NL][Hkv] int32,
 * idx [B_total] int64 kept flat indices ascending.  Any output except keep
 * may be NULL.  Supported: d = 128, Hq = 4 Hkv, 1 <= w <= min(32, N),
 * NL * Hkv * N + 128 < 2^31 (else KVC_ERR_UNSUPPORTED).  ws: device memory of
 * kvc_prefill_workspace_size bytes, 256-byte aligned (KVC_ERR_WORKSPACE).
 * A kernel wait that ran out (a fault) leaves NaN scores.
 * Streams: the value norms run on a stream the library owns (one per
 * context and device, created on the first call in that context, never
 * destroyed), forked from and joined back into `stream` through events, so
 * every output is ordered on `stream` as usual and a stream capture of
 * `stream` takes both branches.  Calls on different caller streams share
 * that stream and queue there.
 */
KVC_API kvc_status kvc_prefill_score(int32_t NL, int32_t Hq, int32_t Hkv, int32_t d,
                             int32_t N, int32_t w, int64_t B_total,
                             int32_t normalize, int32_t alloc, const uint16_t *q_win,
                             const uint16_t *K, const uint16_t *V,
                             const float *R, float *scores, uint8_t *keep,
                             int32_t *counts, int64_t *idx, void *ws,
                             size_t ws_bytes, void *stream);

/*
 * kvc_prefill_window_attention -- weighted column sums of the group-mean
 * window attention.
 *
 * Defined by: KeepKV reading notes eq 15 at the end of the prefill
 * (S = sum over the last w queries of (1 - alpha) alpha^(age) s^k, the
 * windowed EMA initialization of the utilities: row_weight[j] =
 * (1 - alpha) alpha^(w-1-j)); MomentKV sec A4 setup, SnapKV's prefill
 * protocol (attention accumulated over the observation window:
 * row_weight[j] = 1).  With the window and the causal mask of
 * kvc_prefill_score (query j of w at position N - w + j sees keys
 * 0..N-w+j; A_bar the mean over the group's query heads of the row
 * softmax of q K^T / sqrt(d)):
 *   S[l][g][i] = sum_{j<w} row_weight[j] A_bar[j, i].
 * row_weight: HOST array of w floats.  q_win [NL][Hq][w][d], K
 * [NL][Hkv][N][d] bf16 as in kvc_prefill_score; S [NL][Hkv][N] fp32.
 * Supported: d = 128, Hq = 4 Hkv, 1 <= w <= min(32, N).  ws: device memory
 * of kvc_prefill_workspace_size(NL, Hkv, N, 0) bytes, 256-byte aligned.
 * Tensor cores (tcgen05) for the logits, fp32 probabilities.
 */
KVC_API kvc_status kvc_prefill_window_attention(int32_t NL, int32_t Hq, int32_t Hkv, int32_t d,
                                                int32_t N, int32_t w, const float *row_weight,
                                                const uint16_t *q_win, const uint16_t *K,
                                                float *S, void *ws, size_t ws_bytes,
                                                void *stream);

/*
 * kvc_prefill_snapkv -- the prompt selection of MomentKV's prefill protocol.
 *
 * Defined by: MomentKV sec A4 setup ("SnapKV's prefill protocol": attention
 * scores accumulated over a 32-token observation window at the end of the
 * prompt; the first token kept as the attention sink; adjacent tokens
 * merged into blocks of 4 before scoring; the cache budget allocated
 * adaptively over the heads of a layer from their attention).
 *   acc = kvc_prefill_window_attention with every row weight 1;
 *   scores[l][g][i] = mean of acc over the block of `pool` consecutive
 *     positions holding i ([b pool, (b + 1) pool), the last block ragged);
 *     with sink != 0, scores[l][g][0] = +infinity;
 *   each layer keeps its B_total / NL largest scores over all its KV heads
 *     and tokens (equal scores in ascending flat index).
 * Outputs as kvc_prefill_score (scores [NL][Hkv][N] fp32 optional, keep
 * [NL][Hkv][N] uint8 required, counts [NL][Hkv] and idx [B_total] optional,
 * idx ascending within each layer's slice [l B_total/NL, (l+1) B_total/NL)).
 * B_total must be a multiple of NL (KVC_ERR_INVALID_ARG); 1 <= pool <= 64;
 * Hkv <= 64; other limits and the workspace as kvc_prefill_window_attention.
 */
KVC_API kvc_status kvc_prefill_snapkv(int32_t NL, int32_t Hq, int32_t Hkv, int32_t d, int32_t N,
                                      int32_t w, int64_t B_total, int32_t pool, int32_t sink,
                                      const uint16_t *q_win, const uint16_t *K, float *scores,
                                      uint8_t *keep, int32_t *counts, int64_t *idx, void *ws,
                                      size_t ws_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* KVC_H */

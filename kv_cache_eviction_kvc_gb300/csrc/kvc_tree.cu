// kvc_tree.cu -- the extern "C" entry points for drafted tokens: host-side
// argument checks and dispatch (the kernels: kvc_tree_attend.cu,
// kvc_tree_weights.cu, kvc_tree_commit.cu).
#include "kvc_tree.h"

using namespace kvc;

#define TR_CHECK(cond, code, ...)      \
    do {                               \
        if (!(cond)) {                 \
            set_error(__VA_ARGS__);    \
            return (code);             \
        }                              \
    } while (0)

#define TR_TRY(expr)                      \
    do {                                  \
        kvc_status _s = (expr);           \
        if (_s != KVC_OK) return _s;      \
    } while (0)

static bool misaligned(const void *p, unsigned a) { return ((uintptr_t)p & (a - 1)) != 0; }

static kvc_status tr_cuda(cudaError_t e, const char *what)
{
    if (e == cudaSuccess) return KVC_OK;
    (void)cudaGetLastError();                    // it is reported here, not by the next call
    set_error("%s: %s", what, cudaGetErrorString(e));
    return KVC_ERR_CUDA;
}

static kvc_status check_tree(const char *fn, const kvc_params *p, int32_t max_len,
                             const kvc_tree *t, const kvc_cache *c)
{
    TR_TRY(check_params(p));
    TR_TRY(check_cache(c));
    TR_CHECK(max_len >= 1 && max_len <= p->cap, KVC_ERR_SHAPE,
             "%s: max_len = %d must satisfy 1 <= max_len <= cap = %d", fn, max_len, p->cap);
    TR_CHECK(t != nullptr && t->mask != nullptr, KVC_ERR_INVALID_ARG,
             "%s: the tree and its mask must be non-NULL", fn);
    TR_CHECK(t->T >= 1, KVC_ERR_INVALID_ARG, "%s: T = %d must be >= 1", fn, t->T);
    TR_CHECK(t->T <= kTreeMax, KVC_ERR_UNSUPPORTED, "%s: T = %d unsupported (at most %d)", fn, t->T,
             kTreeMax);
    TR_CHECK(t->units >= 1 && p->U % t->units == 0, KVC_ERR_INVALID_ARG,
             "%s: units = %d must divide U = %d", fn, t->units, p->U);
    TR_CHECK(!misaligned(t->mask, 8), KVC_ERR_INVALID_ARG, "%s: mask must be 8-byte aligned", fn);
    return KVC_OK;
}

static kvc_status check_path(const char *fn, const kvc_tree *t, const kvc_path *a)
{
    TR_CHECK(a != nullptr && a->token && a->n && a->pos, KVC_ERR_INVALID_ARG,
             "%s: the path and its arrays must be non-NULL", fn);
    TR_CHECK(a->A >= 1 && a->A <= t->T, KVC_ERR_INVALID_ARG,
             "%s: A = %d must satisfy 1 <= A <= T = %d", fn, a->A, t->T);
    return KVC_OK;
}

static kvc_status check_mom(const char *fn, const kvc_moments *m)
{
    TR_CHECK(m == nullptr || (m->n && m->mu_k && m->mu_v && m->C), KVC_ERR_INVALID_ARG,
             "%s: the moments' arrays must be non-NULL", fn);
    TR_CHECK(m == nullptr || !misaligned(m->C, 16), KVC_ERR_INVALID_ARG,
             "%s: moments C must be 16-byte aligned", fn);
    return KVC_OK;
}

static kvc_status check_tree_ws(const char *fn, const kvc_params *p, int32_t T, const void *ws,
                                size_t bytes)
{
    const size_t need = tree_ws_bytes(*p, T);
    TR_CHECK(ws != nullptr && !misaligned(ws, kAlign) && bytes >= need, KVC_ERR_WORKSPACE,
             "%s: a workspace of %zu bytes (256-byte aligned) is required", fn, need);
    return KVC_OK;
}

// S is fp64 when wide, else fp32
static kvc_status tree_weights(const char *fn, const kvc_params *p, int32_t max_len, const kvc_tree *tree,
                               const kvc_path *path, const float *row_weight, const uint16_t *q,
                               const uint16_t *k_tree, const float *lse, const kvc_cache *cache, void *S,
                               bool wide, void *ws, size_t ws_bytes, void *stream)
{
    TR_TRY(check_tree(fn, p, max_len, tree, cache));
    TR_TRY(check_path(fn, tree, path));
    TR_CHECK(q && k_tree && lse && S, KVC_ERR_INVALID_ARG,
             "%s: q, k_tree, lse and S must be non-NULL", fn);
    TR_CHECK(!misaligned(q, 16) && !misaligned(k_tree, 16), KVC_ERR_INVALID_ARG,
             "%s: q and k_tree must be 16-byte aligned", fn);
    TR_CHECK(!wide || !misaligned(S, 8), KVC_ERR_INVALID_ARG, "%s: S must be 8-byte aligned", fn);
    TR_TRY(check_tree_ws(fn, p, tree->T, ws, ws_bytes));
    const TreeArgs t{tree->mask, tree->n, tree->T, tree->units};
    const PathArgs a{path->token, path->n, path->pos, path->A};
    return tr_cuda(launch_tree_weights(*p, max_len, t, a, row_weight, q, k_tree, lse, *cache, S, wide,
                                       ws, static_cast<cudaStream_t>(stream)),
                   fn);
}

static kvc_status tree_commit(const char *fn, const kvc_params *p, int32_t max_len, const kvc_tree *tree,
                              const kvc_path *path, const uint16_t *k_tree, const uint16_t *v_tree,
                              const void *S, bool wide, const kvc_cache *cache, const kvc_moments *mom,
                              int32_t kmax, int32_t *evict_idx, int32_t *evict_pos, int32_t *n_evict,
                              void *ws, size_t ws_bytes, void *stream)
{
    TR_TRY(check_tree(fn, p, max_len, tree, cache));
    TR_TRY(check_path(fn, tree, path));
    TR_TRY(check_mom(fn, mom));
    TR_CHECK(p->merge == 0, KVC_ERR_UNSUPPORTED, "%s: not combined with merging", fn);
    TR_CHECK(p->rule == KVC_RULE_SINGLE || p->rule == KVC_RULE_CUMULATIVE || p->rule == KVC_RULE_EMA,
             KVC_ERR_UNSUPPORTED, "%s: rule %d does not aggregate attention weight per unit", fn,
             p->rule);
    TR_CHECK(k_tree && v_tree && n_evict, KVC_ERR_INVALID_ARG,
             "%s: k_tree, v_tree and n_evict must be non-NULL", fn);
    TR_CHECK(!misaligned(k_tree, 16) && !misaligned(v_tree, 16), KVC_ERR_INVALID_ARG,
             "%s: k_tree and v_tree must be 16-byte aligned", fn);
    TR_CHECK(!wide || !misaligned(S, 8), KVC_ERR_INVALID_ARG, "%s: S must be 8-byte aligned", fn);
    TR_CHECK(kmax >= 1, KVC_ERR_INVALID_ARG, "%s: kmax = %d must be >= 1", fn, kmax);
    TR_CHECK(kmax <= kTreeMax, KVC_ERR_UNSUPPORTED, "%s: kmax = %d unsupported (at most %d)", fn,
             kmax, kTreeMax);
    DecodeWs w = decode_ws_layout(*p, nullptr);
    TR_CHECK(ws != nullptr && !misaligned(ws, kAlign) && ws_bytes >= w.bytes, KVC_ERR_WORKSPACE,
             "%s: the decode workspace of %zu bytes (256-byte aligned) is required", fn, w.bytes);
    w = decode_ws_layout(*p, ws);
    const TreeArgs t{tree->mask, tree->n, tree->T, tree->units};
    const PathArgs a{path->token, path->n, path->pos, path->A};
    return tr_cuda(launch_tree_commit(*p, max_len, t, a, k_tree, v_tree, S, wide, *cache, mom,
                                      kmax, evict_idx, evict_pos, n_evict, w,
                                      static_cast<cudaStream_t>(stream)),
                   fn);
}

extern "C" {

size_t kvc_tree_workspace_size(const kvc_params *p, int32_t T)
{
    if (check_params(p) != KVC_OK || T < 1 || T > kTreeMax) return 0;
    return tree_ws_bytes(*p, T);
}

kvc_status kvc_tree_attend(const kvc_params *p, int32_t max_len, const kvc_tree *tree,
                           const uint16_t *q, const uint16_t *k_tree, const uint16_t *v_tree,
                           const kvc_cache *cache, const kvc_moments *mom, uint16_t *o, float *lse,
                           void *ws, size_t ws_bytes, void *stream)
{
    const char *fn = "kvc_tree_attend";
    TR_TRY(check_tree(fn, p, max_len, tree, cache));
    TR_TRY(check_mom(fn, mom));
    TR_CHECK(q && k_tree && v_tree && o && lse, KVC_ERR_INVALID_ARG,
             "%s: q, k_tree, v_tree, o and lse must be non-NULL", fn);
    TR_CHECK(!misaligned(q, 16) && !misaligned(k_tree, 16) && !misaligned(v_tree, 16) &&
                 !misaligned(o, 16),
             KVC_ERR_INVALID_ARG, "%s: q, k_tree, v_tree and o must be 16-byte aligned", fn);
    TR_TRY(check_tree_ws(fn, p, tree->T, ws, ws_bytes));
    const TreeArgs t{tree->mask, tree->n, tree->T, tree->units};
    return tr_cuda(launch_tree_attend(*p, max_len, t, q, k_tree, v_tree, *cache,
                                      p->correction == KVC_CORR_OFF ? nullptr : mom, o, lse, ws,
                                      static_cast<cudaStream_t>(stream)),
                   "kvc_tree_attend launch");
}

kvc_status kvc_tree_weights(const kvc_params *p, int32_t max_len, const kvc_tree *tree,
                            const kvc_path *path, const float *row_weight, const uint16_t *q,
                            const uint16_t *k_tree, const float *lse, const kvc_cache *cache,
                            float *S, void *ws, size_t ws_bytes, void *stream)
{
    return tree_weights("kvc_tree_weights", p, max_len, tree, path, row_weight, q, k_tree, lse, cache, S,
                        false, ws, ws_bytes, stream);
}

kvc_status kvc_tree_weights_f64(const kvc_params *p, int32_t max_len, const kvc_tree *tree,
                                const kvc_path *path, const float *row_weight, const uint16_t *q,
                                const uint16_t *k_tree, const float *lse, const kvc_cache *cache,
                                double *S, void *ws, size_t ws_bytes, void *stream)
{
    return tree_weights("kvc_tree_weights_f64", p, max_len, tree, path, row_weight, q, k_tree, lse, cache,
                        S, true, ws, ws_bytes, stream);
}

kvc_status kvc_tree_commit(const kvc_params *p, int32_t max_len, const kvc_tree *tree,
                           const kvc_path *path, const uint16_t *k_tree, const uint16_t *v_tree,
                           const float *S, const kvc_cache *cache, const kvc_moments *mom,
                           int32_t kmax, int32_t *evict_idx, int32_t *evict_pos, int32_t *n_evict,
                           void *ws, size_t ws_bytes, void *stream)
{
    return tree_commit("kvc_tree_commit", p, max_len, tree, path, k_tree, v_tree, S, false, cache, mom,
                       kmax, evict_idx, evict_pos, n_evict, ws, ws_bytes, stream);
}

kvc_status kvc_tree_commit_f64(const kvc_params *p, int32_t max_len, const kvc_tree *tree,
                               const kvc_path *path, const uint16_t *k_tree, const uint16_t *v_tree,
                               const double *S, const kvc_cache *cache, const kvc_moments *mom,
                               int32_t kmax, int32_t *evict_idx, int32_t *evict_pos,
                               int32_t *n_evict, void *ws, size_t ws_bytes, void *stream)
{
    return tree_commit("kvc_tree_commit_f64", p, max_len, tree, path, k_tree, v_tree, S, true, cache, mom,
                       kmax, evict_idx, evict_pos, n_evict, ws, ws_bytes, stream);
}

}  // extern "C"

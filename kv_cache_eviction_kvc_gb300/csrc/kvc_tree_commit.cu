// kvc_tree_commit.cu -- append the accepted tokens, update the utilities with
// the weight every slot gathered, evict the lowest (utility, position) pairs
// down to the budget into the moments, close the gaps.
//
// Its bytes: 20 per slot (utility read and written, weight read; 24 with weights in
// fp64), 128 KB per unit for C, and the rows that go and come.  One CTA per unit, of
// 256 threads and several per SM, so that one's loads run under another's
// selection, or of 512 when it has the SM to itself:
//   1. the utilities are updated in place; every thread keeps the lowest of
//      its slots;
//   2. at least k slots are at or below the k-th smallest minimum of any
//      partition of the slots, so it bounds the k-th lowest utility: the
//      threads are folded into 32 sets (128 for k > 16, where 32 would bound
//      loosely or not at all; with 128 throughout, 128 units of 2623 slots take
//      12.9 us for 6 victims and not 12.2) whose minima are ranked;
//   3. the slots at or below the bound, about 1.4 k of them, are looked up in the
//      threads' (long units: groups') slots whose minimum is, and ranked by
//      (utility, position, slot) against one another;
//   4. rows move, C is read and written in whole lines (prefetched to L2 at
//      the start).
// Long units are updated by a kernel of their own over the whole grid, which
// leaves the lowest utility of every 32 slots; step 1 is then a pass over those.
//
// Measured (a call among others): 128 units of 2623 slots on average, up to 6
// accepted, EMA, moments: 11.7 us (a chain of about ten dependent steps, most of
// them a trip to L2); 1024 units of 1024 slots, cumulative, votes, moments: 35 us for
// 162 MB (1.7 waves of four CTAs an SM, each such a chain: DRAM is a third busy); 8
// units of 131071 slots, 17 accepted: 18.7 us (update 7.9).  With kmax = 64 the rows of
// 64 victims leave room for two CTAs an SM: the 1024 units take 47 us without votes,
// 31 with kmax = 5.  Weights in fp64: 32.4 for 31.3 us.
//
// Many equal utilities (weights that underflow to 0) can make every slot a
// candidate: then the bound is taken again over whole (utility, position,
// slot) keys, which are distinct; and if the lowest keys sit in so few sets
// that even these are too many, the k lowest are found one after another.
#include "kvc_soft64.h"
#include "kvc_tree.h"

#include <stddef.h>

namespace kvc {
namespace {

constexpr int kThreads = 256;
constexpr int kCand = 1024;              // candidates held
constexpr int kLong = 32 * kThreads;     // slots of a unit that one CTA can update
constexpr int kSms = 152;
constexpr int kChunk = 2048;             // slots per CTA of the update kernel

struct Key {
    uint64_t u, t;                       // utility; position and slot
};

__device__ __forceinline__ bool key_less(const Key &a, const Key &b)
{
    return a.u < b.u || (a.u == b.u && a.t < b.t);
}

__device__ __forceinline__ Key key_min(const Key &a, const Key &b) { return key_less(b, a) ? b : a; }

// No key: above every scored slot's.
constexpr uint64_t kNone = ~0ull;

// Unscored slots (infinite utilities) are protected: they have no key.
__device__ __forceinline__ uint64_t util_key(double m)
{
    const uint64_t b = (uint64_t)__double_as_longlong(m);
    if ((b & 0x7fffffffffffffffull) == 0x7ff0000000000000ull) return kNone;
    return double_key(m);
}

__device__ __forceinline__ uint64_t tie_key(int32_t pos, int slot)
{
    return (uint64_t)((uint32_t)pos ^ 0x80000000u) << 32 | (uint32_t)slot;
}

struct ComArgs {
    TreeArgs t;
    PathArgs p;
    const uint16_t *kt, *vt;
    const void *S;                       // float, or (wide) double
    uint16_t *K, *V;
    int32_t *votes, *pos, *len;
    double *util;
    const int32_t *budget;
    float *mn, *mu_k, *mu_v, *C;
    int32_t *evict_idx, *evict_pos, *n_evict, *status, *pend;
    uint64_t *gmin;                      // [U][gstride] lowest keys of 32 slots each (long units)
    int gstride;
    double alpha, beta;                  // EMA: alpha util + beta weight
    int cap, L, rule, kmax, max_len;
    FastDiv by_units;
};

struct ComSmem {
    Key cand[kCand];
    Key set[128];
    Key bound;
    double fresh[kTreeMax];              // utilities of the accepted tokens
    float del[2][kD];                    // the batch means' distance from the moments'
    float w[kTreeMax];
    int32_t tok[kTreeMax];
    int vic[kTreeMax], src[kTreeMax], gone[kTreeMax];
    int scan[40];
    int n_cand, n_low, n_hole;
    alignas(16) float kv[4];             // [2][kmax][kD]: the victims' keys and values
};
static_assert(offsetof(ComSmem, kv) % 16 == 0 && offsetof(ComSmem, del) % 16 == 0, "read as float4");

// What a unit does: its lengths and counts, or why it is refused.  Warp-wide.
struct Plan {
    int n, acc, total, k, err;
};

__device__ __forceinline__ Plan plan_unit(const ComArgs &a, int u, int lane)
{
    const int b = a.by_units(u);
    Plan p;
    p.n = a.len[u];
    const int L = a.budget ? a.budget[u] : a.L;
    const int live = a.t.n ? a.t.n[b] : a.t.T;
    p.acc = a.p.n[b];
    // every entry of the row is read at once: which of them count is known with n
    int c0 = 0, c1 = 0;
    const int32_t *tok = a.p.token + (size_t)b * a.p.A;
    if (lane < a.p.A) c0 = tok[lane];
    if (lane + 32 < a.p.A) c1 = tok[lane + 32];
    const bool bad = (lane < p.acc && (c0 < 0 || c0 >= live)) ||
                     (lane + 32 < p.acc && (c1 < 0 || c1 >= live));
    p.total = p.n + p.acc;
    p.k = max(0, p.total - L);
    p.err = KVC_OK;
    if (p.n < 0 || p.n > a.max_len) p.err = KVC_ERR_SHAPE;
    else if (live < 0 || live > a.t.T || p.acc < 0 || p.acc > a.p.A || __any_sync(kFull, bad))
        p.err = KVC_ERR_INVALID_ARG;
    else if (p.total > a.cap || L < 1 || L > a.L || p.k > a.kmax) p.err = KVC_ERR_SHAPE;
    return p;
}

// Unusual operands (a call, so that the fp64 instructions are not in the way of
// the usual ones).
__device__ __noinline__ double odd_util(int rule, double alpha, double beta, double m, float weight)
{
    const double s = (double)weight;
    if (isinf(m) || rule == KVC_RULE_SINGLE) return s;
    return rule == KVC_RULE_CUMULATIVE ? m + s : fma(alpha, m, beta * s);
}

// fp32 to fp64 and the cumulative sum by integer operations where the operands
// are the usual ones (with fp64 instructions: 47 -> 42 us for 1024 units of 1024
// slots, 14.5 -> 10.3 for the update of 8 units of 131071).
__device__ __forceinline__ double new_util(const ComArgs &a, double m, float weight)
{
    const uint64_t b = (uint64_t)__double_as_longlong(m);
    const uint32_t w = __float_as_uint(weight);
    const bool fresh = a.rule == KVC_RULE_SINGLE || b == 0x7ff0000000000000ull;
    if ((w != 0 && (w >> 23) - 1u >= 254u) || !(fresh || soft_normal(b)))
        return odd_util(a.rule, a.alpha, a.beta, m, weight);
    const uint64_t s = w == 0 ? 0 : soft_widen(w);
    if (fresh) return __longlong_as_double((long long)s);
    if (a.rule == KVC_RULE_CUMULATIVE)
        return w == 0 ? m : __longlong_as_double((long long)soft_add(b, s));
    return fma(a.alpha, m, a.beta * __longlong_as_double((long long)s));
}

// The same with a weight in fp64, below fp32's range too.
__device__ __noinline__ double odd_util(int rule, double alpha, double beta, double m, double s)
{
    return rule == KVC_RULE_CUMULATIVE ? m + s : fma(alpha, m, beta * s);
}

__device__ __forceinline__ double new_util(const ComArgs &a, double m, double s)
{
    const uint64_t b = (uint64_t)__double_as_longlong(m), w = (uint64_t)__double_as_longlong(s);
    if (a.rule == KVC_RULE_SINGLE || (b & 0x7fffffffffffffffull) == 0x7ff0000000000000ull) return s;
    if (a.rule == KVC_RULE_EMA) return fma(a.alpha, m, a.beta * s);
    if (soft_normal(b) && soft_normal(w)) return __longlong_as_double((long long)soft_add(b, w));
    return odd_util(a.rule, a.alpha, a.beta, m, s);
}

// Long units: the utilities of kChunk slots, and the lowest keys of 32 slots
// each.  A group is what four neighbouring threads have (eight slots each, every
// kThreads-th), so that little goes between lanes.  grid (chunks, U)
constexpr int kGroups = kChunk / 32;     // groups of a chunk

__device__ __forceinline__ int group_slot(int g, int i)          // the i-th slot of a group
{
    return g / kGroups * kChunk + 4 * (g % kGroups) + (i & 3) + kThreads * (i >> 2);
}

template <typename W>
__global__ void __launch_bounds__(kThreads) tree_update_kernel(ComArgs a)
{
    const W *S = static_cast<const W *>(a.S);
    const int u = blockIdx.y, lane = threadIdx.x & 31;
    follow();
    const Plan p = plan_unit(a, u, lane);
    if (p.err != KVC_OK) return;
    const size_t cb = (size_t)u * a.cap;
    const int i0 = blockIdx.x * kChunk + threadIdx.x;
    uint64_t low = kNone;
    if (i0 - (int)threadIdx.x >= p.n) return;
    constexpr int kPer = kChunk / kThreads;
    double m[kPer];
    W s[kPer];
#pragma unroll
    for (int j = 0; j < kPer; j++) {
        const int i = i0 + j * kThreads;
        m[j] = i < p.n ? a.util[cb + i] : __longlong_as_double(0x7ff0000000000000ll);
        s[j] = S && i < p.n ? S[cb + i] : W(0);
    }
#pragma unroll
    for (int j = 0; j < kPer; j++) {
        const int i = i0 + j * kThreads;
        if (S && i < p.n) {
            m[j] = new_util(a, m[j], s[j]);
            a.util[cb + i] = m[j];
        }
        low = min((unsigned long long)low, (unsigned long long)util_key(m[j]));
    }
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) low = min((unsigned long long)low, __shfl_xor_sync(kFull, (unsigned long long)low, d));
    lead();                                                  // (not before: the next kernel's CTAs would crowd on the SMs that are free first, 49 us instead of 22)
    if ((lane & 3) == 0) a.gmin[(size_t)u * a.gstride + blockIdx.x * kGroups + (threadIdx.x >> 2)] = low;
}

// The k-th smallest of the sets' minima into s.bound.u (kNone when fewer than
// k sets have a key); `mine` is the thread's own minimum.
template <int kT>
__device__ __forceinline__ void rank_utils(ComSmem &s, uint64_t mine, int k)
{
    const int tid = threadIdx.x, fold = k <= 16 ? kT / 32 : kT / 128, sets = kT / fold, own = tid / fold;
    uint64_t *set = reinterpret_cast<uint64_t *>(s.set);
    for (int d = 1; d < fold; d <<= 1)
        mine = min((unsigned long long)mine, __shfl_xor_sync(kFull, (unsigned long long)mine, d));
    if (tid % fold == 0) set[own] = mine;
    if (tid == 0) s.n_cand = s.n_low = 0;
    __syncthreads();
    // a set's rank, counted by its threads together
    int r = 0;
#pragma unroll 8
    for (int j = tid % fold; j < sets; j += fold) {
        const uint64_t y = set[j];
        r += y < mine || (y == mine && j < own);
    }
    for (int d = 1; d < fold; d <<= 1) r += __shfl_xor_sync(kFull, r, d);
    if (r == k - 1 && tid % fold == 0) s.bound = Key{mine, kNone};
    __syncthreads();
}

// The same over whole keys, 128 sets.
template <int kT>
__device__ void rank_keys(ComSmem &s, Key mine, int k)
{
    const int tid = threadIdx.x;
    constexpr int fold = kT / 128;
    for (int d = 1; d < fold; d <<= 1)
        mine = key_min(mine, Key{__shfl_xor_sync(kFull, (unsigned long long)mine.u, d),
                                 __shfl_xor_sync(kFull, (unsigned long long)mine.t, d)});
    if (tid % fold == 0) s.set[tid / fold] = mine;
    if (tid == 0) s.n_cand = 0;
    __syncthreads();
    if (tid < 128) {
        const Key x = s.set[tid];
        int r = 0;
        for (int j = 0; j < 128; j++) {
            const Key y = s.set[j];
            r += key_less(y, x) || (j < tid && !key_less(x, y));
        }
        if (r == k - 1) s.bound = x;
    }
    __syncthreads();
}

__device__ __forceinline__ void add_candidate(ComSmem &s, const Key &k)
{
    const int c = atomicAdd(&s.n_cand, 1);
    if (c < kCand) s.cand[c] = k;
}

template <int kT, bool kSplit, typename W>
__global__ void __launch_bounds__(kT, kT > kThreads ? 1 : kSplit ? 2 : 4) tree_commit_kernel(ComArgs a)
{
    extern __shared__ __align__(16) unsigned char raw[];
    ComSmem &s = *reinterpret_cast<ComSmem *>(raw);
    const int u = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (!kSplit) follow();
    const size_t cb = (size_t)u * a.cap;
    double *util = a.util + cb;
    const W *S = a.S ? static_cast<const W *>(a.S) + cb : nullptr;
    // four slots a thread on their way while the four before are updated, the first
    // of them before it is known how many there are (what lies behind is not used)
    double m_next[4];
    W x_next[4];
    auto load = [&](int i0) {
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const int i = i0 + j * kT;
            m_next[j] = i < a.cap ? util[i] : 0.;
            x_next[j] = S && i < a.cap ? S[i] : W(0);
        }
    };
    if (!kSplit) load(tid);
    const Plan p = plan_unit(a, u, lane);
    if (p.err != KVC_OK) {
        if (tid == 0) {
            a.n_evict[u] = 0;
            record_status(a.status, p.err);
        }
        return;
    }
    const int n = p.n, acc = p.acc, total = p.total, k = p.k, b = a.by_units(u);
    const size_t tb = (size_t)u * a.t.T;
    int32_t *pos = a.pos + cb;
    const uint64_t *gmin = a.gmin + (size_t)u * a.gstride;
    const int pos0 = a.p.pos[b], groups = (n + kChunk - 1) / kChunk * kGroups;
    float *C = a.C + (size_t)u * kD * kD;
    if (a.C && k > 0) {
#pragma unroll
        for (int i = 0; i < 512 / kT; i++)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(C + (tid + i * kT) * 32) : "memory");
    }
    if (tid < acc) {
        s.tok[tid] = a.p.token[(size_t)b * a.p.A + tid];
        s.fresh[tid] = S ? (double)S[n + tid] : __longlong_as_double(0x7ff0000000000000ll);
    }
    // 1. the lowest key of the thread's slots (long units: of its groups of 32)
    uint64_t mine = kNone;
    constexpr int kAt = 8;                                   // loads of groups in flight
    uint64_t first[kAt];                                     // long units: the thread's first groups
    if (kSplit) {
        follow();
#pragma unroll
        for (int j = 0; j < kAt; j++) {
            const int g = tid + j * kT;
            first[j] = g < groups ? gmin[g] : kNone;
        }
#pragma unroll
        for (int j = 0; j < kAt; j++) mine = min((unsigned long long)mine, (unsigned long long)first[j]);
#pragma unroll 8
        for (int g = tid + kAt * kT; g < groups; g += kT)
            mine = min((unsigned long long)mine, (unsigned long long)gmin[g]);
    } else {
        for (int i0 = tid; i0 < n; i0 += 4 * kT) {
            double m[4];
            W x[4];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                m[j] = m_next[j];
                x[j] = x_next[j];
            }
            load(i0 + 4 * kT);
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const int i = i0 + j * kT;
                if (i >= n) m[j] = __longlong_as_double(0x7ff0000000000000ll);
                else if (S) util[i] = m[j] = new_util(a, m[j], x[j]);
                mine = min((unsigned long long)mine, (unsigned long long)util_key(m[j]));
            }
        }
    }
    // fewer scored slots than victims?  Minima of k threads answer it
    if (__syncthreads_count(mine != kNone) < k) {
        int c = tid < acc && util_key(s.fresh[tid]) != kNone, all;
        for (int i = tid; i < n; i += kT) c += util_key(util[i]) != kNone;
        block_exscan(c, s.scan, &all);
        if (all < k) {
            if (tid == 0) {
                a.n_evict[u] = 0;
                record_status(a.status, KVC_ERR_INVALID_ARG);
            }
            return;
        }
    }
    const int end = total - k;
    if (k > 0) {
        // 2., 3.
        rank_utils<kT>(s, mine, k);
        const uint64_t top = s.bound.u;
        if (tid < acc) {
            const uint64_t x = util_key(s.fresh[tid]);
            if (x != kNone) add_candidate(s, Key{x, tie_key(pos0 + tid, n + tid)});
        }
        // the groups of slots (long units: of 32; else: a thread's own) that have a low one
        int *low = reinterpret_cast<int *>(s.set);           // (the sets are done with)
        constexpr int kLow = sizeof(s.set) / sizeof(int);
        auto found = [&](int g) {
            const int c = atomicAdd(&s.n_low, 1);
            if (c < kLow) low[c] = g;
        };
        if (kSplit) {
#pragma unroll
            for (int j = 0; j < kAt; j++)
                if (first[j] != kNone && first[j] <= top) found(tid + j * kT);
            for (int g0 = tid + kAt * kT; g0 < groups; g0 += kAt * kT) {
                uint64_t x[kAt];
#pragma unroll
                for (int j = 0; j < kAt; j++) {
                    const int g = g0 + j * kT;
                    x[j] = g < groups ? gmin[g] : kNone;
                }
#pragma unroll
                for (int j = 0; j < kAt; j++)
                    if (x[j] != kNone && x[j] <= top) found(g0 + j * kT);
            }
        } else if (mine != kNone && mine <= top) {
            found(tid);
        }
        __syncthreads();
        // their slots, a lane each and four groups at once (more groups than places: every
        // slot is looked at below)
        const int n_low = s.n_low;
        if (n_low > kLow && tid == 0) s.n_cand = kCand + 1;
        for (int e0 = warp; n_low <= kLow && e0 < n_low; e0 += 4 * kT / 32) {
            double m[4];
            int32_t at[4];
            int slot[4];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const int e = e0 + j * kT / 32, g = low[min(e, n_low - 1)];
                slot[j] = kSplit ? group_slot(g, lane) : g + kT * lane;
                const bool in = e < n_low && slot[j] < n;
                m[j] = in ? util[slot[j]] : __longlong_as_double(0x7ff0000000000000ll);
                at[j] = in ? pos[slot[j]] : 0;
            }
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const uint64_t x = util_key(m[j]);
                if (x != kNone && x <= top) add_candidate(s, Key{x, tie_key(at[j], slot[j])});
            }
        }
        __syncthreads();
        auto key_at = [&](int i) {
            const uint64_t x = util_key(i < n ? util[i] : s.fresh[i - n]);
            return x == kNone ? Key{kNone, kNone}
                              : Key{x, tie_key(i < n ? pos[i] : pos0 + i - n, i)};
        };
        if (s.n_cand > kCand) {
            __syncthreads();
            Key low{kNone, kNone};
            for (int i = tid; i < total; i += kT) low = key_min(low, key_at(i));
            rank_keys<kT>(s, low, k);
            const Key top2 = s.bound;
            for (int i = tid; i < total; i += kT) {
                const Key x = key_at(i);
                if (x.u != kNone && !key_less(top2, x)) add_candidate(s, x);
            }
            __syncthreads();
        }
        if (s.n_cand > kCand) {
            Key last{0, 0};
            for (int r = 0; r < k; r++) {
                Key low{kNone, kNone};
                for (int i = tid; i < total; i += kT) {
                    const Key x = key_at(i);
                    if (r == 0 || key_less(last, x)) low = key_min(low, x);
                }
                __syncthreads();
                rank_keys<kT>(s, low, 1);
                last = s.bound;
                __syncthreads();
                if (tid == 0) s.vic[r] = (int)(uint32_t)last.t;
            }
        } else {
            // a slot's rank among the candidates; the k lowest are the victims
            const int c = s.n_cand;
            for (int i = tid; i < c; i += kT) {
                const Key x = s.cand[i];
                int r = 0;
#pragma unroll 4
                for (int j = 0; j < c; j++) r += key_less(s.cand[j], x);
                if (r < k) s.vic[r] = (int)(uint32_t)x.t;
            }
        }
        if (tid < k) s.gone[tid] = 0;
        if (tid == 0) s.n_hole = 0;
        __syncthreads();
        // into ascending slot order; which of the slots from `end` on go
        int v = 0, r = 0;
        if (tid < k) {
            v = s.vic[tid];
            for (int j = 0; j < k; j++) r += s.vic[j] < v;
            if (v >= end) s.gone[v - end] = 1;
        }
        __syncthreads();
        if (tid < k) {
            s.vic[r] = v;
            if (v < end) atomicAdd(&s.n_hole, 1);
            if (a.evict_idx) a.evict_idx[(size_t)u * a.kmax + r] = v;
            if (a.evict_pos) a.evict_pos[(size_t)u * a.kmax + r] = v < n ? pos[v] : pos0 + v - n;
            s.w[r] = v < n && a.votes ? (float)a.votes[cb + v] : 1.f;
            // the r-th hole below `end` takes the r-th slot at or above it that stays
            if (!s.gone[tid]) {
                int before = 0;
                for (int j = 0; j < tid; j++) before += !s.gone[j];
                s.src[before] = end + tid;
            }
        }
        __syncthreads();
        // the victims' rows, before any of them is overwritten
        if (a.C)
            for (int e0 = tid; e0 < k * 32; e0 += 4 * kT) {
                uint4 v[4];
#pragma unroll
                for (int x = 0; x < 4; x++) {
                    const int e = e0 + x * kT, j = e >> 5, ch = e & 15, which = e >> 4 & 1;
                    if (e >= k * 32) break;
                    const int i = s.vic[j];
                    const uint16_t *row = i < n ? (which ? a.V : a.K) + (cb + i) * kD
                                                : (which ? a.vt : a.kt) + (tb + s.tok[i - n]) * kD;
                    v[x] = reinterpret_cast<const uint4 *>(row)[ch];
                }
#pragma unroll
                for (int x = 0; x < 4; x++) {
                    const int e = e0 + x * kT, j = e >> 5, ch = e & 15, which = e >> 4 & 1;
                    if (e >= k * 32) break;
                    float f[8];
                    unpack8(v[x], f);
                    float4 *d = reinterpret_cast<float4 *>(s.kv + (which * a.kmax + j) * kD + ch * 8);
                    d[0] = make_float4(f[0], f[1], f[2], f[3]);
                    d[1] = make_float4(f[4], f[5], f[6], f[7]);
                }
            }
    } else if (tid == 0) {
        s.n_hole = 0;
    }
    __syncthreads();
    // rows: the moves (sources at or above `end`, destinations below), and the
    // accepted tokens below `end` that stay where they are appended
    const int nm = s.n_hole;
    for (int e = tid; e < (nm + acc) * 32; e += kT) {
        const int j = e >> 5, ch = e & 15, which = e >> 4 & 1;
        int from, to;
        if (j < nm) {
            from = s.src[j];
            to = s.vic[j];
        } else {
            from = to = n + j - nm;
            if (to >= end) continue;
            bool victim = false;
            for (int i = nm - 1; i >= 0 && s.vic[i] >= to; i--) victim |= s.vic[i] == to;
            if (victim) continue;
        }
        const uint16_t *row = from < n ? (which ? a.V : a.K) + (cb + from) * kD
                                       : (which ? a.vt : a.kt) + (tb + s.tok[from - n]) * kD;
        reinterpret_cast<uint4 *>((which ? a.V : a.K) + (cb + to) * kD)[ch] =
            reinterpret_cast<const uint4 *>(row)[ch];
        if ((e & 31) == 0) {
            util[to] = from < n ? util[from] : s.fresh[from - n];
            pos[to] = from < n ? pos[from] : pos0 + from - n;
            if (a.votes) a.votes[cb + to] = from < n ? a.votes[cb + from] : 1;
        }
    }
    if (tid == 0) {
        a.len[u] = end;
        a.n_evict[u] = k;
        a.pend[(size_t)u * kPendStride] = 0;      // a lazy step's victim queue is stale now
    }
    if (!a.C || k == 0) return;
    // the moments: the batch's weighted means and co-moment, merged (Chan,
    // Golub and LeVeque, 1979)
    float *kv = s.kv, *vv = s.kv + a.kmax * kD;
    const float n0 = a.mn[u];
    float nb = 0.f;
    for (int j = 0; j < k; j++) nb += s.w[j];
    const float n1 = n0 + nb;
    if (tid < 2 * kD) {
        const int which = tid >> 7, d = tid & 127;
        float *own = (which ? vv : kv) + d;
        float *mu = (which ? a.mu_v : a.mu_k) + (size_t)u * kD + d;
        const float mu0 = *mu;
        float x = 0.f;
        for (int j = 0; j < k; j++) x += s.w[j] * own[j * kD];
        x /= nb;
        s.del[which][d] = x - mu0;
        // the batch about its means, values weighted
        for (int j = 0; j < k; j++) own[j * kD] = which ? s.w[j] * (own[j * kD] - x) : own[j * kD] - x;
        *mu = mu0 + (x - mu0) * (nb / n1);
    }
    __syncthreads();
    // a warp has its share of the rows (value dimensions), a lane four columns
    constexpr int kShare = kD * 32 / kT;
    const float4 dk = reinterpret_cast<const float4 *>(s.del[0])[lane];
    const float cross = n0 * (nb / n1) / n1, keep = n0 / n1, inv = 1.f / n1;
    constexpr int kRowsAt = kT > kThreads ? 8 : 4;           // rows at once
#pragma unroll 1
    for (int r0 = 0; r0 < kShare; r0 += kRowsAt) {
        const int row = kShare * warp + r0;
        float4 *c = reinterpret_cast<float4 *>(C + row * kD) + lane;
        float4 old[kRowsAt], m[kRowsAt];
#pragma unroll
        for (int i = 0; i < kRowsAt; i++) {
            old[i] = c[i * (kD / 4)];
            m[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll 2
        for (int j = 0; j < k; j++) {
            const float4 y = reinterpret_cast<const float4 *>(kv + j * kD)[lane];
#pragma unroll
            for (int h = 0; h < kRowsAt / 4; h++) {
                const float4 x4 = *reinterpret_cast<const float4 *>(vv + j * kD + row + 4 * h);
                const float v[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    m[4 * h + i].x = fmaf(v[i], y.x, m[4 * h + i].x);
                    m[4 * h + i].y = fmaf(v[i], y.y, m[4 * h + i].y);
                    m[4 * h + i].z = fmaf(v[i], y.z, m[4 * h + i].z);
                    m[4 * h + i].w = fmaf(v[i], y.w, m[4 * h + i].w);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kRowsAt; i++) {
            const float dv = cross * s.del[1][row + i];
            c[i * (kD / 4)] = make_float4(fmaf(dv, dk.x, fmaf(keep, old[i].x, m[i].x * inv)),
                                          fmaf(dv, dk.y, fmaf(keep, old[i].y, m[i].y * inv)),
                                          fmaf(dv, dk.z, fmaf(keep, old[i].z, m[i].z * inv)),
                                          fmaf(dv, dk.w, fmaf(keep, old[i].w, m[i].w * inv)));
        }
    }
    if (tid == 0) a.mn[u] = n1;
    lead();
}

template <typename W>
cudaError_t launch(const kvc_params &p, int max_len, const TreeArgs &t, const PathArgs &pa,
                   const uint16_t *kt, const uint16_t *vt, const void *S, const kvc_cache &c,
                   const kvc_moments *m, int kmax, int32_t *evict_idx, int32_t *evict_pos,
                   int32_t *n_evict, const DecodeWs &ws, cudaStream_t st)
{
    ComArgs a{t, pa, kt, vt, S, c.K, c.V, c.votes, c.pos, c.len, c.util, p.budget,
              m ? m->n : nullptr, m ? m->mu_k : nullptr, m ? m->mu_v : nullptr, m ? m->C : nullptr,
              evict_idx, evict_pos, n_evict, ws.status, ws.pend,
              reinterpret_cast<uint64_t *>(ws.probs), (p.cap + kChunk - 1) / kChunk * kGroups, (double)p.alpha, 1.0 - (double)p.alpha, p.cap, p.L, p.rule, kmax,
              max_len, FastDiv(t.units)};
    // Half a device of units or fewer leaves SMs to the update kernel: 8 units of 8192
    // slots take 16.6 us in one kernel and 12.9 in two, 64 units 17.3 and 14.7, but 128
    // units 17.9 and 18.9; of 4096 slots 8 units take the same.
    const bool split = max_len > kLong || (max_len > kLong / 2 && p.U <= kSms / 2);
    const size_t smem = sizeof(ComSmem) + (m ? 2 * (size_t)kmax * kD * sizeof(float) : 0);
    // The attribute is the kernel's, shared by the host's threads: every call allows the
    // most that any call takes (a call that allowed its own size could take another
    // thread's away between that one's setting and its launch).
    constexpr size_t kMost = sizeof(ComSmem) + 2 * (size_t)kTreeMax * kD * sizeof(float);
    static_assert(kMost <= 227 * 1024, "one block's shared memory");
    // A unit that has an SM to itself gets twice the threads: 128 units of 2623 slots on
    // average 12.1 us with 256 and 11.7 with 512, 8 of 131071 19.8 and 18.8.
    const bool wide = p.U <= kSms;
    auto *kernel = wide ? split ? tree_commit_kernel<2 * kThreads, true, W> : tree_commit_kernel<2 * kThreads, false, W>
                   : split ? tree_commit_kernel<kThreads, true, W> : tree_commit_kernel<kThreads, false, W>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMost);
    if (e != cudaSuccess) return e;
    if (split) {
        if (p.U > 65535) return cudaErrorInvalidValue;
        e = launch_following(tree_update_kernel<W>, dim3((max_len + kChunk - 1) / kChunk, p.U), kThreads, 0, st, a);
        if (e != cudaSuccess) return e;
    }
    return launch_following(kernel, dim3(p.U), wide ? 2 * kThreads : kThreads, smem, st, a);
}

}  // namespace

cudaError_t launch_tree_commit(const kvc_params &p, int max_len, const TreeArgs &t,
                               const PathArgs &pa, const uint16_t *kt, const uint16_t *vt,
                               const void *S, bool wide, const kvc_cache &c, const kvc_moments *m,
                               int kmax, int32_t *evict_idx, int32_t *evict_pos, int32_t *n_evict,
                               const DecodeWs &ws, cudaStream_t st)
{
    return (wide ? launch<double> : launch<float>)(p, max_len, t, pa, kt, vt, S, c, m, kmax, evict_idx,
                                                   evict_pos, n_evict, ws, st);
}

}  // namespace kvc

// kvc_tree_commit.cu -- append the accepted tokens, update the utilities with
// the weight every slot gathered, evict the lowest (utility, position) pairs
// down to the budget into the moments, close the gaps.
//
// One CTA per unit, one pass over the utilities:
//   1. update in place; consecutive slots form groups (a power of two of
//      them, about 256 groups or more) whose lowest utility goes to shared
//      memory;
//   2. at least k slots are at or below the k-th smallest minimum of any
//      partition of the slots, so it bounds the k-th lowest utility: the
//      groups are folded into 128 sets whose minima are ranked;
//   3. the scored slots at or below the bound (in groups whose minimum is)
//      are the candidates, about 1.4 k of them, ranked by (utility, position,
//      slot) against one another.
// Many equal utilities (weights that underflow to 0) can make every slot a
// candidate: then the bound is taken again over whole (utility, position,
// slot) keys, which are distinct; and if the lowest keys sit in so few sets
// that even these are too many, the k lowest are found one after another.
#include "kvc_tree.h"

namespace kvc {
namespace {

constexpr int kThreads = 512;
constexpr int kSets = 128;               // minima ranked for the bound
constexpr int kCand = 1024;              // candidates held

struct Key {
    uint64_t u, t;                       // utility; position and slot
};

__device__ __forceinline__ bool key_less(const Key &a, const Key &b)
{
    return a.u < b.u || (a.u == b.u && a.t < b.t);
}

__device__ __forceinline__ Key key_min(const Key &a, const Key &b) { return key_less(b, a) ? b : a; }

__device__ __forceinline__ Key key_shfl(const Key &k, int m)
{
    return Key{__shfl_xor_sync(kFull, (unsigned long long)k.u, m),
               __shfl_xor_sync(kFull, (unsigned long long)k.t, m)};
}

// No key: above every scored slot's.
__device__ __forceinline__ Key key_none() { return Key{~0ull, ~0ull}; }

// Unscored slots (infinite utilities) are protected: they have no key.
__device__ __forceinline__ uint64_t util_key(double m)
{
    const uint64_t b = (uint64_t)__double_as_longlong(m);
    if ((b & 0x7fffffffffffffffull) == 0x7ff0000000000000ull) return ~0ull;
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
    const float *S;
    uint16_t *K, *V;
    int32_t *votes, *pos, *len;
    double *util;
    const int32_t *budget;
    float *mn, *mu_k, *mu_v, *C;
    int32_t *evict_idx, *evict_pos, *n_evict, *status, *pend;
    double alpha;
    int cap, L, rule, kmax, max_len, gshift;
};

struct ComSmem {
    float kv[2][kTreeMax][kD];           // the victims' keys and values
    Key cand[kCand];
    Key set[kSets];
    double fresh[kTreeMax];              // utilities of the accepted tokens
    float bar[2][kD], del[2][kD];        // batch means; their distance from the moments'
    float w[kTreeMax];
    int32_t tok[kTreeMax];
    int vic[kTreeMax], src[kTreeMax], dst[kTreeMax];
    int scan[40];
    Key bound;
    int n_cand, n_move;
};

__device__ __forceinline__ double new_util(const ComArgs &a, double m, double s)
{
    const uint64_t b = (uint64_t)__double_as_longlong(m);
    if ((b & 0x7fffffffffffffffull) == 0x7ff0000000000000ull || a.rule == KVC_RULE_SINGLE) return s;
    return a.rule == KVC_RULE_CUMULATIVE ? m + s : a.alpha * m + (1.0 - a.alpha) * s;
}

// The k-th smallest of the sets' minima into s.bound (none when fewer than k
// sets have a key).  `mine`: the thread's own minimum; four lanes are a set.
__device__ void rank_sets(ComSmem &s, Key mine, int k)
{
    mine = key_min(mine, key_shfl(mine, 1));
    mine = key_min(mine, key_shfl(mine, 2));
    if ((threadIdx.x & 3) == 0) s.set[threadIdx.x >> 2] = mine;
    if (threadIdx.x == 0) s.n_cand = 0;
    __syncthreads();
    if (threadIdx.x < kSets) {
        const Key x = s.set[threadIdx.x];
        int r = 0;
        for (int j = 0; j < kSets; j++) {
            const Key y = s.set[j];
            r += key_less(y, x) || (j < (int)threadIdx.x && !key_less(x, y));
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

__global__ void __launch_bounds__(kThreads) tree_commit_kernel(ComArgs a)
{
    extern __shared__ __align__(16) unsigned char raw[];
    ComSmem &s = *reinterpret_cast<ComSmem *>(raw);
    uint64_t *gmin = reinterpret_cast<uint64_t *>(raw + sizeof(ComSmem));
    const int u = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = u / a.t.units;
    const int n = a.len[u], acc = path_count(a.t, a.p, u, lane);
    const int L = a.budget ? a.budget[u] : a.L;
    const int total = n + acc, k = max(0, total - L);
    int err = KVC_OK;
    if (n < 0 || n > a.max_len) err = KVC_ERR_SHAPE;
    else if (acc < 0) err = KVC_ERR_INVALID_ARG;
    else if (total > a.cap || L < 1 || L > a.L || k > a.kmax) err = KVC_ERR_SHAPE;
    if (err != KVC_OK) {
        if (tid == 0) {
            a.n_evict[u] = 0;
            record_status(a.status, err);
        }
        return;
    }
    const size_t cb = (size_t)u * a.cap, tb = (size_t)u * a.t.T;
    double *util = a.util + cb;
    int32_t *pos = a.pos + cb;
    const float *S = a.S ? a.S + cb : nullptr;
    const int pos0 = a.p.pos[b];
    if (tid < acc) {
        s.tok[tid] = a.p.token[(size_t)b * a.p.A + tid];
        s.fresh[tid] = S ? (double)S[n + tid] : __longlong_as_double(0x7ff0000000000000ll);
    }
    // 1. utilities; the lowest of each group of 2^gshift consecutive slots
    const int groups = (n + (1 << a.gshift) - 1) >> a.gshift;
    int scored = 0;
    for (int i0 = 0; i0 < n; i0 += kThreads) {
        const int i = i0 + tid;
        uint64_t x = ~0ull;
        if (i < n) {
            double m = util[i];
            if (S) {
                m = new_util(a, m, S[i]);
                util[i] = m;
            }
            x = util_key(m);
            scored += x != ~0ull;
        }
        for (int d = 1; d < 1 << a.gshift; d <<= 1)
            x = min((unsigned long long)x, __shfl_xor_sync(kFull, (unsigned long long)x, d));
        if (i < n && (i & ((1 << a.gshift) - 1)) == 0) gmin[i >> a.gshift] = x;
    }
    if (tid < acc) scored += util_key(s.fresh[tid]) != ~0ull;
    int all;
    block_exscan(scored, s.scan, &all);
    if (all < k) {
        if (tid == 0) {
            a.n_evict[u] = 0;
            record_status(a.status, KVC_ERR_INVALID_ARG);
        }
        return;
    }
    if (k > 0) {
        // 2., 3.
        Key mine = key_none();
        for (int g = tid; g < groups; g += kThreads) mine = key_min(mine, Key{gmin[g], ~0ull});
        rank_sets(s, mine, k);
        const uint64_t top = s.bound.u;
        if (tid < acc && util_key(s.fresh[tid]) != ~0ull)
            add_candidate(s, Key{util_key(s.fresh[tid]), tie_key(pos0 + tid, n + tid)});
        for (int g = warp; g < groups; g += kThreads / 32) {
            if (gmin[g] > top || gmin[g] == ~0ull) continue;
            const int i = (g << a.gshift) + lane;
            if (lane < 1 << a.gshift && i < n) {
                const uint64_t x = util_key(util[i]);
                if (x <= top && x != ~0ull) add_candidate(s, Key{x, tie_key(pos[i], i)});
            }
        }
        __syncthreads();
        auto key_at = [&](int i) {
            const uint64_t x = util_key(i < n ? util[i] : s.fresh[i - n]);
            return x == ~0ull ? key_none()
                              : Key{x, tie_key(i < n ? pos[i] : pos0 + i - n, i)};
        };
        if (s.n_cand > kCand) {
            __syncthreads();
            mine = key_none();
            for (int i = tid; i < total; i += kThreads) mine = key_min(mine, key_at(i));
            rank_sets(s, mine, k);
            const Key top2 = s.bound;
            for (int i = tid; i < total; i += kThreads) {
                const Key x = key_at(i);
                if (x.u != ~0ull && !key_less(top2, x)) add_candidate(s, x);
            }
            __syncthreads();
        }
        if (s.n_cand > kCand) {
            Key last{0, 0};
            bool any = false;
            for (int r = 0; r < k; r++) {
                mine = key_none();
                for (int i = tid; i < total; i += kThreads) {
                    const Key x = key_at(i);
                    if (!any || key_less(last, x)) mine = key_min(mine, x);
                }
                __syncthreads();
                rank_sets(s, mine, 1);
                last = s.bound;
                any = true;
                __syncthreads();
                if (tid == 0) s.vic[r] = (int)(uint32_t)last.t;
            }
        } else {
            // a slot's rank among the candidates; the k lowest are the victims
            const int c = s.n_cand;
            for (int i = tid; i < c; i += kThreads) {
                const Key x = s.cand[i];
                int r = 0;
                for (int j = 0; j < c; j++) r += key_less(s.cand[j], x);
                if (r < k) s.vic[r] = (int)(uint32_t)x.t;
            }
        }
        __syncthreads();
        // into ascending slot order
        int v = 0, r = 0;
        if (tid < k) {
            v = s.vic[tid];
            for (int j = 0; j < k; j++) r += s.vic[j] < v;
        }
        __syncthreads();
        if (tid < k) s.vic[r] = v;
        __syncthreads();
        if (tid < k) {
            const int e = s.vic[tid];
            if (a.evict_idx) a.evict_idx[(size_t)u * a.kmax + tid] = e;
            if (a.evict_pos) a.evict_pos[(size_t)u * a.kmax + tid] = e < n ? pos[e] : pos0 + e - n;
            s.w[tid] = e < n && a.votes ? (float)a.votes[cb + e] : 1.f;
        }
    }
    const int end = total - k;
    // the holes below `end` take the slots at or above it that stay; both
    // lists ascend.  Accepted tokens below `end` that stay go where they are
    if (tid == 0) {
        int nm = 0, v = 0;
        while (v < k && s.vic[v] < end) v++;
        for (int i = end; i < total; i++) {
            if (v < k && s.vic[v] == i) { v++; continue; }
            s.src[nm] = i;
            s.dst[nm] = s.vic[nm];
            nm++;
        }
        s.n_move = nm;
    }
    // the victims' rows, before any of them is overwritten
    if (a.C)
        for (int e = tid; e < k * 32; e += kThreads) {
            const int j = e >> 5, ch = e & 15, which = e >> 4 & 1, i = s.vic[j];
            const uint16_t *r = i < n ? (which ? a.V : a.K) + (cb + i) * kD
                                      : (which ? a.vt : a.kt) + (tb + s.tok[i - n]) * kD;
            float f[8];
            unpack8(reinterpret_cast<const uint4 *>(r)[ch], f);
#pragma unroll
            for (int d = 0; d < 8; d++) s.kv[which][j][ch * 8 + d] = f[d];
        }
    __syncthreads();
    // rows: first the moves (sources at or above `end`, destinations below),
    // then the accepted tokens that stay where they were appended
    const int nm = s.n_move;
    auto is_victim = [&](int i) {
        for (int j = 0; j < k; j++)
            if (s.vic[j] == i) return true;
        return false;
    };
    for (int e = tid; e < (nm + acc) * 32; e += kThreads) {
        const int j = e >> 5, ch = e & 15, which = e >> 4 & 1;
        int from, to;
        if (j < nm) {
            from = s.src[j];
            to = s.dst[j];
        } else {
            from = to = n + j - nm;
            if (to >= end || is_victim(to)) continue;
        }
        const uint16_t *r = from < n ? (which ? a.V : a.K) + (cb + from) * kD
                                     : (which ? a.vt : a.kt) + (tb + s.tok[from - n]) * kD;
        uint4 *w = reinterpret_cast<uint4 *>((which ? a.V : a.K) + (cb + to) * kD);
        w[ch] = reinterpret_cast<const uint4 *>(r)[ch];
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
    float nb = 0.f;
    for (int j = 0; j < k; j++) nb += s.w[j];
    const float n0 = a.mn[u], n1 = n0 + nb;
    if (tid < 2 * kD) {
        const int which = tid >> 7, d = tid & 127;
        float x = 0.f;
        for (int j = 0; j < k; j++) x += s.w[j] * s.kv[which][j][d];
        float *mu = (which ? a.mu_v : a.mu_k) + (size_t)u * kD + d;
        x /= nb;
        s.bar[which][d] = x;
        s.del[which][d] = x - *mu;
        *mu += (x - *mu) * (nb / n1);
    }
    __syncthreads();
    const int r0 = 4 * (tid >> 4), c0 = 8 * (tid & 15);
    float m[4][8] = {};
    for (int j = 0; j < k; j++) {
#pragma unroll
        for (int x = 0; x < 4; x++) {
            const float v = s.w[j] * (s.kv[1][j][r0 + x] - s.bar[1][r0 + x]);
#pragma unroll
            for (int y = 0; y < 8; y++) m[x][y] += v * (s.kv[0][j][c0 + y] - s.bar[0][c0 + y]);
        }
    }
    float *C = a.C + (size_t)u * kD * kD;
    const float cross = n0 * (nb / n1) / n1;
#pragma unroll
    for (int x = 0; x < 4; x++)
#pragma unroll
        for (int y = 0; y < 8; y++) {
            float *c = C + (r0 + x) * kD + c0 + y;
            *c = (n0 * *c + m[x][y]) / n1 + cross * s.del[1][r0 + x] * s.del[0][c0 + y];
        }
    if (tid == 0) a.mn[u] = n1;
}

}  // namespace

cudaError_t launch_tree_commit(const kvc_params &p, int max_len, const TreeArgs &t,
                               const PathArgs &pa, const uint16_t *kt, const uint16_t *vt,
                               const float *S, const kvc_cache &c, const kvc_moments *m, int kmax,
                               int32_t *evict_idx, int32_t *evict_pos, int32_t *n_evict,
                               const DecodeWs &ws, cudaStream_t st)
{
    int gshift = 0;
    while (gshift < 5 && (max_len >> gshift) > 512) gshift++;
    const size_t smem = sizeof(ComSmem) + ((size_t)(max_len >> gshift) + 1) * sizeof(uint64_t);
    cudaError_t e = cudaFuncSetAttribute(tree_commit_kernel,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    ComArgs a{t, pa, kt, vt, S, c.K, c.V, c.votes, c.pos, c.len, c.util, p.budget,
              m ? m->n : nullptr, m ? m->mu_k : nullptr, m ? m->mu_v : nullptr, m ? m->C : nullptr,
              evict_idx, evict_pos, n_evict, ws.status, ws.pend, (double)p.alpha, p.cap, p.L, p.rule,
              kmax, max_len, gshift};
    tree_commit_kernel<<<p.U, kThreads, smem, st>>>(a);
    return cudaGetLastError();
}

}  // namespace kvc

// kvc_tree_weights.cu -- the attention weight that the accepted tokens gave
// to every slot of the cache and to the accepted tokens themselves.
//
// The sum runs over the query rows (accepted token, head), so the product is
// taken the other way round from the attention: D = K Q^T (tcgen05), 128
// slots on the tensor-memory lanes, the rows along the columns.  A thread has
// a slot and adds its columns up: no exchange between threads, no maximum (the
// lse is known), S written in whole lines.  exp(x - lse) w / G is one
// exponential, exp2(x' - c_row) with c_row = lse log2(e) - log2(w / G).
//
// Bound by the 256 bytes of key per slot up to about 128 rows (128 x 128
// exponentials take 512 clocks of the special-function units, a tile's 32 KB
// about 1200 of one SM's share of the bandwidth).  The 128-slot tiles of all
// units form one line, cut into equal parts for a persistent CTA per SM; every
// tile stands alone, so nothing is joined.  Measured (G = 4; a call among
// others): 128 units of 2623 slots on average, up to 6 accepted tokens: 18.8 us,
// 4.7 TB/s; 1024 units of 1024 slots, 5 accepted, votes: 47 us, 6.0 TB/s; 8 units
// of 131071 slots, 17 accepted: 45 us, 6.0 TB/s.  In between a tile takes 1320
// clocks, the bandwidth's; what is left is the start (about 6 us until the first
// product: lengths, paths, query rows).
//
// S in fp64 (kWide) takes the same times while the weights are in fp32's range
// (1024 units 47, 8 units 46 us).  Logits some hundred apart: 48 and 64 us, a tile's
// sums are then formed twice.
//
// 512 threads:
//   warps 0-7   two groups on alternate tiles, a thread per slot
//   warp 8      producer (TMA, a ring of 32 KB key tiles)
//   warp 9      tensor-memory owner and MMA issuer (up to four tiles ahead)
//   warp 10     walks the CTA's units ahead of the others
//   warp 11     gathers a unit's accepted rows of q (two buffers when they fit)
//   warps 12-15 the accepted tokens' own entries, a few dot products per unit
//               (mma.sync), 16 tokens of a unit at a time over the grid: a chain of
//               loads per eight rows (1024 units, G = 8, 24 accepted: one warp
//               284 us a call, four 144)
// Every wait is bounded (~2 s); a wait that ran out records KVC_ERR_TIMEOUT.
#include "kvc_soft64.h"
#include "kvc_tree.h"
#include "kvc_umma.cuh"

#include <stddef.h>

namespace kvc {
namespace {

constexpr int kTile = 128;
constexpr int kSlot = kTile * kD * 2;            // 32 KB: a tile of keys
constexpr int kHalf = kSlot / 2;
constexpr int kMaxRing = 6, kSegs = 3, kMaxRows = kTreeMax * 8;
constexpr int kThreads = 512;
constexpr int kProd = 8, kMma = 9, kWalk = 10, kGather = 11, kTail = 12;
constexpr int kTails = kThreads / 32 - kTail;
constexpr int kGrid = 152;
constexpr float kLog2e = 1.4426950408889634f;

struct WtArgs {
    TreeArgs t;
    PathArgs p;
    const float *w;
    const uint16_t *q, *kt;
    const float *lse;
    const int32_t *votes, *len;
    void *S;                               // float, or (wide) double
    int32_t *status;
    int U, G, gshift, cap, max_len;
    int rows, qbufs, ring, dbufs, dcols;   // rows of q per buffer (a multiple of 16); tiles in flight
    int blocks;                            // of 16 accepted tokens
    FastDiv by_units;
    float scale;                           // log2(e) / sqrt(d)
};

// The tiles of a unit that this CTA takes; tiles = 0: there is none left.
struct __align__(16) Seg {
    int u, n, t0, tiles, acc, b;
};

struct WtSmem {
    float c[2][kMaxRows];                  // c_row of a buffer's rows; read as float4
    Seg seg[kSegs];
    uint64_t full[kMaxRing], empty[kMaxRing];
    uint64_t segfull[kSegs], segempty[kSegs];
    uint64_t qfull[2], qempty[2], dfull[4], dempty[4];
    uint64_t drain;
    int scan[kThreads / 32];
    int start_unit, start_base;
    int bad;
    uint32_t tmem;
};
constexpr size_t kCtl = sizeof(WtSmem) + 1024;
constexpr int kMostSmem = 227 * 1024;            // of one block

// Accepted tokens of unit u, or -1 when the unit is refused.
__device__ __forceinline__ int unit_acc(const WtArgs &a, int u, int n, int32_t *err)
{
    const int b = a.by_units(u);
    const int live = a.t.n ? a.t.n[b] : a.t.T, acc = a.p.n[b];
    // (no token's load waits for another's: one by one they were 9 us of a call)
    const int32_t *tok = a.p.token + (size_t)b * a.p.A;
    bool bad = false;
    for (int j0 = 0; j0 < a.p.A; j0 += 8)
#pragma unroll
        for (int e = 0; e < 8; e++) {
            const int c = j0 + e < a.p.A ? tok[j0 + e] : 0;
            bad |= j0 + e < acc && (c < 0 || c >= live);
        }
    *err = KVC_ERR_INVALID_ARG;
    if (live < 0 || live > a.t.T || acc < 0 || acc > a.p.A || bad) return -1;
    *err = KVC_ERR_SHAPE;
    if (n < 0 || n > a.max_len || n + acc > a.cap) return -1;
    return acc;
}

__device__ __forceinline__ int unit_tiles(const WtArgs &a, int u)
{
    int32_t err;
    const int n = a.len[u];
    return unit_acc(a, u, n, &err) < 0 ? 0 : (n + kTile - 1) >> 7;
}

// 16 bytes to shared memory, zeros when the source is not to be read.
__device__ __forceinline__ void cp_async16(void *dst, const void *src, bool read)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
                 "r"(read ? 16 : 0)
                 : "memory");
}

// c_row: a row that weighs nothing (or saw nothing) has +inf.
__device__ __forceinline__ float row_c(const WtArgs &a, float lse, float w)
{
    return lse == -INFINITY ? INFINITY : lse * kLog2e - log2f(w / (float)a.G);
}

// exp2(x - c_row); nothing for a row of c = +inf, whatever its product is.
__device__ __forceinline__ float weight(uint32_t x, float scale, float c)
{
    const float e = ex2_approx(fmaf(__uint_as_float(x), scale, -c));
    return c == INFINITY ? 0.f : e;
}

// S in fp64 holds weights below fp32's range, which a method that orders the slots
// tells apart.  A sum of fp32 terms above kSmall is good as it is: a term that fp32
// loses is below 2^-126, 512 of them below 2^-27 of such a sum.  Below it the sum is
// formed again in units of 2^ref, the whole power of two below its largest term.
constexpr float kSmall = 0x1p-90f;
constexpr float kLeast = -1300.f;        // exponents from here down are 0 in fp64

// log2 of a term
__device__ __forceinline__ float weight_log(uint32_t x, float scale, float c)
{
    return c == INFINITY ? -INFINITY : fmaf(__uint_as_float(x), scale, -c);
}

// v as fp64 (by integer operations: fp64 ones are scarce).
__device__ __forceinline__ double widen(float v)
{
    const uint32_t b = __float_as_uint(v);
    return (b >> 23) - 1u < 254u ? __longlong_as_double((long long)soft_widen(b)) : (double)v;
}

// v 2^e for e < 0
__device__ __forceinline__ double widen(float v, int e)
{
    const uint64_t b = soft_widen(__float_as_uint(v));
    if (v >= 1.f && v < 0x1p100f && (int)(b >> 52) + e >= 1)
        return __longlong_as_double((long long)b + ((long long)e << 52));
    return ldexp((double)v, e);
}

template <bool kWide>
__global__ void __launch_bounds__(kThreads, 1)
tree_weights_kernel(const __grid_constant__ WtArgs a, const __grid_constant__ CUtensorMap tmK)
{
    extern __shared__ __align__(1024) unsigned char dyn[];
    const uint32_t qbytes = (uint32_t)a.rows * 256;      // a buffer: two halves of 64 columns
    unsigned char *ring = dyn, *qbuf = dyn + a.ring * kSlot;
    WtSmem &S = *reinterpret_cast<WtSmem *>(qbuf + a.qbufs * qbytes);
    if (smem_u32(dyn) & 1023) {                          // the swizzle counts on it
        if (threadIdx.x == 0) record_status(a.status, KVC_ERR_CUDA);
        return;
    }
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (warp == kProd && lane == 0)
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmK)) : "memory");
    if (tid == 0) {
        S.bad = 0;
        for (int i = 0; i < kMaxRing; i++) {
            mbar_init(&S.full[i], 1);
            mbar_init(&S.empty[i], 1);
        }
        for (int i = 0; i < kSegs; i++) {
            mbar_init(&S.segfull[i], 1);
            mbar_init(&S.segempty[i], 11);       // eight slot warps, producer, issuer, gatherer
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(&S.qfull[i], 1);
            mbar_init(&S.qempty[i], 9);          // eight slot warps, issuer
        }
        for (int i = 0; i < 4; i++) {
            mbar_init(&S.dfull[i], 1);
            mbar_init(&S.dempty[i], 4);
        }
        mbar_init(&S.drain, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMma) tmem_alloc(&S.tmem, 512);
    follow();

    // the line of tiles: every CTA counts it and finds where its part starts
    int lo, hi;
    {
        const int per = (a.U + kThreads - 1) / kThreads;
        const int u0 = min(a.U, tid * per), u1 = min(a.U, u0 + per);
        int sum = 0;
        for (int u = u0; u < u1; u++) {
            sum += unit_tiles(a, u);
            int32_t err;
            if (blockIdx.x == 0 && unit_acc(a, u, a.len[u], &err) < 0) record_status(a.status, err);
        }
        int incl = sum;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int t = __shfl_up_sync(kFull, incl, d);
            if (lane >= d) incl += t;
        }
        if (lane == 31) S.scan[warp] = incl;
        __syncthreads();
        const int of = lane < kThreads / 32 ? S.scan[lane] : 0;
        const int total = warp_isum(of);
        int b = incl - sum + warp_isum(lane < warp ? of : 0);
        const LineCuts c(gridDim.x, total);
        const int bid = min((int)blockIdx.x, c.parts);
        lo = c.start(bid);
        hi = c.start(min(bid + 1, c.parts));
        if (sum > 0 && lo < b + sum && lo >= b)
            for (int u = u0; u < u1; u++) {
                const int nt = unit_tiles(a, u);
                if (lo >= b && lo < b + nt) {
                    S.start_unit = u;
                    S.start_base = b;
                }
                b += nt;
            }
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = S.tmem;

    if (warp == kWalk) {
        // --------------------------------------------------------- walker
        if (elect_one()) {
            int u = lo < hi ? S.start_unit : a.U, base = S.start_base;
            bool ok = true;
            for (int i = 0; ok;) {
                Seg s;
                s.tiles = 0;
                if (u < a.U && base < hi) {
                    int32_t err;
                    s.u = u;
                    s.n = a.len[u];
                    s.b = a.by_units(u);
                    s.acc = unit_acc(a, u, s.n, &err);
                    const int nt = s.acc < 0 ? 0 : (s.n + kTile - 1) >> 7;
                    s.t0 = max(0, lo - base);
                    s.tiles = min(nt, hi - base) - s.t0;
                    base += nt;
                    u++;
                    if (s.tiles <= 0) continue;
                }
                if (i >= kSegs) ok = tree_wait(&S.segempty[i % kSegs], (i / kSegs - 1) & 1, &S.bad);
                if (!ok) break;
                S.seg[i % kSegs] = s;
                mbar_arrive(&S.segfull[i % kSegs]);
                i++;
                if (s.tiles == 0) break;
            }
        }
        __syncwarp();
    } else if (warp == kProd) {
        // ------------------------------------------------------- producer
        if (elect_one()) {
            int k = 0, slot = 0;
            uint32_t ph = 1;
            bool ok = true;
            const uint64_t pol = l2_policy_evict_first();
            for (int i = 0; ok; i++) {
                ok = tree_wait(&S.segfull[i % kSegs], (i / kSegs) & 1, &S.bad);
                if (!ok) break;
                const Seg s = S.seg[i % kSegs];
                mbar_arrive(&S.segempty[i % kSegs]);
                if (s.tiles == 0) break;
                for (int t = s.t0; t < s.t0 + s.tiles; t++) {
                    if (k >= a.ring) ok = tree_wait(&S.empty[slot], ph, &S.bad);
                    if (!ok) break;
                    unsigned char *d = ring + slot * kSlot;
                    const int boxes = s.n - t * kTile > 64 ? 2 : 1;
                    mbar_expect_tx(&S.full[slot], boxes * kHalf);
#pragma unroll
                    for (int h = 0; h < 2; h++)
                        for (int b = 0; b < boxes; b++)
                            tma_3d_hint(d + h * kHalf + b * (kHalf / 2), &tmK, 64 * h, t * kTile + 64 * b,
                                        s.u, &S.full[slot], pol);
                    k++;
                    if (++slot == a.ring) { slot = 0; ph ^= 1; }
                }
            }
            if (!ok) {
                S.bad = 1;
                // the copies in flight land before the block ends
                for (int i = max(0, k - a.ring); i < k; i++)
                    mbar_wait(&S.full[i % a.ring], (i / a.ring) & 1);
            }
        }
        __syncwarp();
    } else if (warp == kMma) {
        // ------------------------------------------------------ MMA issuer
        if (elect_one()) {
            bool ok = true;
            int slot = 0, db = 0, k = 0;
            uint32_t ph = 0, dph = 1;
            const uint64_t k0 = umma_sdesc(smem_u32(ring)), q0 = umma_sdesc(smem_u32(qbuf));
            for (int i = 0; ok; i++) {
                ok = tree_wait(&S.segfull[i % kSegs], (i / kSegs) & 1, &S.bad);
                if (!ok) break;
                const Seg s = S.seg[i % kSegs];
                mbar_arrive(&S.segempty[i % kSegs]);
                if (s.tiles == 0) break;
                const int qb = i % a.qbufs;
                ok = tree_wait(&S.qfull[qb], (i / a.qbufs) & 1, &S.bad);
                const int cols = max(16, (s.acc * a.G + 15) & ~15);
                const int n1 = min(cols, 256), n2 = cols - n1;
                const uint32_t id1 = umma_idesc_bf16(128, n1), id2 = umma_idesc_bf16(128, n2);
                const uint64_t qd = q0 + (uint64_t)(qb * qbytes >> 4);
                for (int t = 0; ok && t < s.tiles; t++) {
                    ok = tree_wait(&S.full[slot], ph, &S.bad);
                    if (k >= a.dbufs) ok = ok && tree_wait(&S.dempty[db], dph, &S.bad);
                    if (!ok) break;
                    tc_fence_after();
                    const uint64_t kd = k0 + (uint64_t)(slot * (kSlot >> 4));
                    const uint32_t d = tmem + db * a.dcols;
#pragma unroll
                    for (int ks = 0; ks < 8; ks++) {
                        const uint64_t b = qd + (uint64_t)((ks >> 2) * (a.rows * 8) + (ks & 3) * 2);
                        umma_bf16(d, umma_sdesc_step(kd, ks), b, id1, ks > 0);
                        if (n2) umma_bf16(d + 256, umma_sdesc_step(kd, ks), b + 256 * 8, id2, ks > 0);
                    }
                    umma_commit(&S.dfull[db]);
                    umma_commit(&S.empty[slot]);
                    if (t + 1 == s.tiles) umma_commit(&S.qempty[qb]);
                    if (++slot == a.ring) { slot = 0; ph ^= 1; }
                    if (++db == a.dbufs) { db = 0; dph ^= 1; }
                    k++;
                }
            }
            if (!ok) {
                // the MMAs in flight are done before tensor memory goes back
                S.bad = 1;
                umma_commit(&S.drain);
                mbar_wait(&S.drain, 0);
            }
        }
        __syncwarp();
    } else if (warp == kGather) {
        // ------------------------------------------------- accepted rows of q
        bool ok = true;
        for (int i = 0; ok; i++) {
            ok = __all_sync(kFull, tree_wait(&S.segfull[i % kSegs], (i / kSegs) & 1, &S.bad));
            if (!ok) break;
            const Seg s = S.seg[i % kSegs];
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.segempty[i % kSegs]);
            if (s.tiles == 0) break;
            const int qb = i % a.qbufs;
            if (i >= a.qbufs)
                ok = __all_sync(kFull, tree_wait(&S.qempty[qb], (i / a.qbufs - 1) & 1, &S.bad));
            if (!ok) break;
            const int rows = s.acc * a.G, cols = max(16, (rows + 15) & ~15);
            unsigned char *d = qbuf + qb * qbytes;
            const int32_t *tok = a.p.token + (size_t)s.b * a.p.A;
            const int t0 = lane < s.acc ? tok[lane] : 0, t1 = lane + 32 < s.acc ? tok[lane + 32] : 0;
            auto token = [&](int j) {                        // the j-th, for every lane its own j
                const int x = __shfl_sync(kFull, t0, j & 31), y = __shfl_sync(kFull, t1, j & 31);
                return j < 32 ? x : y;
            };
            // two rows of 16 chunks a step, all of them in flight together with what c_row
            // needs; rows past the last are zero
            for (int b0 = 0; b0 < cols; b0 += 128) {
                float lse[4], w[4];
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const int r = b0 + 32 * e + lane, j = min(r, rows - 1) >> a.gshift, t = token(max(j, 0));
                    lse[e] = -INFINITY;
                    w[e] = 1.f;
                    if (r < rows) {
                        lse[e] = a.lse[((size_t)s.u * a.t.T + t) * a.G + (r & (a.G - 1))];
                        if (a.w) w[e] = a.w[(size_t)s.b * a.p.A + j];
                    }
                }
                for (int r0 = b0; r0 < min(cols, b0 + 128); r0 += 2) {
                    const int r = r0 + (lane >> 4), c = lane & 15, t = token(min(r, max(rows - 1, 0)) >> a.gshift);
                    const uint16_t *from = a.q + (((size_t)s.u * a.t.T + t) * a.G + (r & (a.G - 1))) * kD + 8 * c;
                    cp_async16(d + (c >> 3) * (a.rows * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4), from, r < rows);
                }
#pragma unroll
                for (int e = 0; e < 4; e++)
                    if (b0 + 32 * e + lane < cols) S.c[qb][b0 + 32 * e + lane] = row_c(a, lse[e], w[e]);
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.qfull[qb]);
        }
    } else if (warp >= kTail) {
        // --------------------------------- the accepted tokens' own entries
        // a job: 16 of a unit's accepted tokens
        for (long long job = blockIdx.x + (long long)gridDim.x * (warp - kTail); job < (long long)a.U * a.blocks;
             job += (long long)gridDim.x * kTails) {
            const int u = (int)(job / a.blocks), m0 = 16 * (int)(job - (long long)u * a.blocks);
            int32_t err;
            const int n = a.len[u], acc = unit_acc(a, u, n, &err), b = a.by_units(u);
            if (acc <= m0) continue;
            const int32_t *tok = a.p.token + (size_t)b * a.p.A;
            const int g = lane >> 2, t = lane & 3, rows = acc * a.G;
            const int t0 = lane < acc ? tok[lane] : 0, t1 = lane + 32 < acc ? tok[lane + 32] : 0;
            auto token = [&](int j) {                        // the j-th, for every lane its own j
                const int x = __shfl_sync(kFull, t0, j & 31), y = __shfl_sync(kFull, t1, j & 31);
                return j < 32 ? x : y;
            };
            // eight rows of q: the thread's part of one, and what it needs of its two columns
            struct Rows {
                uint32_t q[16];
                float lse[2], w[2];
                uint64_t see[2];
            };
            auto fetch = [&](Rows &x, int r0) {
                const int r = min(r0 + g, rows - 1);
                const uint32_t *p = reinterpret_cast<const uint32_t *>(
                    a.q + (((size_t)u * a.t.T + token(r >> a.gshift)) * a.G + (r & (a.G - 1))) * kD) + t;
#pragma unroll
                for (int ks = 0; ks < 16; ks++) x.q[ks] = p[4 * ks];
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    const int rr = min(r0 + 2 * t + e, rows - 1), jj = rr >> a.gshift, ct = token(jj);
                    x.lse[e] = a.lse[((size_t)u * a.t.T + ct) * a.G + (rr & (a.G - 1))];
                    x.w[e] = a.w ? a.w[(size_t)b * a.p.A + jj] : 1.f;
                    x.see[e] = r0 + 2 * t + e < rows ? a.t.mask[(size_t)b * a.t.T + ct] : 0;
                }
            };
            // the 16 tokens' keys
            uint32_t ka[8][4];
            int c[2];
#pragma unroll
            for (int h = 0; h < 2; h++) {
                c[h] = token(min(m0 + g + 8 * h, acc - 1));
                const uint32_t *p = reinterpret_cast<const uint32_t *>(
                    a.kt + ((size_t)u * a.t.T + c[h]) * kD) + t;
#pragma unroll
                for (int ks = 0; ks < 8; ks++) {
                    ka[ks][h] = p[8 * ks];
                    ka[ks][2 + h] = p[8 * ks + 4];
                }
            }
            float sum[2] = {0.f, 0.f}, top[2] = {kLeast, kLeast}, ref[2], low[2] = {0.f, 0.f};
            // (a second time where a sum is small, in units of its largest term)
            for (int pass = 0; pass < (kWide ? 2 : 1); pass++) {
                Rows x, next;
                fetch(next, 0);
                for (int r0 = 0; r0 < rows; r0 += 8) {
                    x = next;
                    if (r0 + 8 < rows) fetch(next, r0 + 8);
                    float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int ks = 0; ks < 8; ks++)
                        mma16816(d, ka[ks][0], ka[ks][1], ka[ks][2], ka[ks][3], x.q[2 * ks], x.q[2 * ks + 1]);
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        const float cr = row_c(a, x.lse[e], x.w[e]);
#pragma unroll
                        for (int h = 0; h < 2; h++) {
                            if (!(x.see[e] >> c[h] & 1)) continue;
                            const uint32_t y = __float_as_uint(d[2 * h + e]);
                            if (!kWide || pass == 0) sum[h] += weight(y, a.scale, cr);
                            if (kWide && pass == 0) top[h] = fmaxf(top[h], weight_log(y, a.scale, cr));
                            if (kWide && pass == 1) low[h] += ex2_approx(weight_log(y, a.scale, cr) - ref[h]);
                        }
                    }
                }
                if (!kWide) break;
                bool again = false;
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    if (pass == 1) continue;
                    for (int x = 1; x < 4; x <<= 1) {
                        sum[h] += __shfl_xor_sync(kFull, sum[h], x);
                        top[h] = fmaxf(top[h], __shfl_xor_sync(kFull, top[h], x));
                    }
                    ref[h] = floorf(top[h]);
                    again |= m0 + g + 8 * h < acc && sum[h] < kSmall;
                }
                if (!__any_sync(kFull, again)) break;
            }
#pragma unroll
            for (int h = 0; h < 2; h++) {
                float &of = kWide ? low[h] : sum[h];
                of += __shfl_xor_sync(kFull, of, 1);
                of += __shfl_xor_sync(kFull, of, 2);
                if (t != 0 || m0 + g + 8 * h >= acc) continue;
                const size_t to = (size_t)u * a.cap + n + m0 + g + 8 * h;
                if (kWide)
                    static_cast<double *>(a.S)[to] =
                        sum[h] < kSmall ? widen(low[h], (int)ref[h]) : widen(sum[h]);
                else
                    static_cast<float *>(a.S)[to] = sum[h];
            }
        }
    } else {
        // ---------------------------------------------------------- slots
        const int w = warp >> 2, r = tid & 127;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        bool ok = true;
        int k = 0;                                           // the CTA's tiles so far
        for (int i = 0; ok; i++) {
            ok = __all_sync(kFull, tree_wait(&S.segfull[i % kSegs], (i / kSegs) & 1, &S.bad));
            if (!ok) break;
            const Seg s = S.seg[i % kSegs];
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.segempty[i % kSegs]);
            if (s.tiles == 0) break;
            const int qb = i % a.qbufs, cols = max(16, (s.acc * a.G + 15) & ~15);
            ok = __all_sync(kFull, tree_wait(&S.qfull[qb], (i / a.qbufs) & 1, &S.bad));
            // alternate tiles; with a single accumulator one group takes them all (a wait
            // for a phase must not begin before the phase ahead of it is over)
            const int step = a.dbufs > 1 ? 2 : 1;
            for (int t = step == 2 ? (k ^ w) & 1 : w ? s.tiles : 0; ok && t < s.tiles; t += step) {
                const int at = (s.t0 + t) * kTile + r, kk = k + t, db = kk % a.dbufs;
                const size_t slot = (size_t)s.u * a.cap + at;
                float vote = 1.f;
                if (a.votes && at < s.n) vote = (float)a.votes[slot];
                ok = __all_sync(kFull, tree_wait(&S.dfull[db], (kk / a.dbufs) & 1, &S.bad));
                if (!ok) break;
                tc_fence_after();
                float sum[4] = {0.f, 0.f, 0.f, 0.f}, top[2] = {kLeast, kLeast};
#pragma unroll 1
                for (int c0 = 0; c0 < cols; c0 += 16) {
                    uint32_t y[16];
                    tmem_ld16_async(tmem + lanes + db * a.dcols + c0, y);
                    float4 c[4];
#pragma unroll
                    for (int j = 0; j < 4; j++) c[j] = *reinterpret_cast<const float4 *>(&S.c[qb][c0 + 4 * j]);
                    tmem_wait_ld();
                    tmem_bind16(y);
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        sum[0] += weight(y[4 * j], a.scale, c[j].x);
                        sum[1] += weight(y[4 * j + 1], a.scale, c[j].y);
                        sum[2] += weight(y[4 * j + 2], a.scale, c[j].z);
                        sum[3] += weight(y[4 * j + 3], a.scale, c[j].w);
                        if (kWide) {
                            top[0] = fmaxf(fmaxf(top[0], weight_log(y[4 * j], a.scale, c[j].x)),
                                           weight_log(y[4 * j + 1], a.scale, c[j].y));
                            top[1] = fmaxf(fmaxf(top[1], weight_log(y[4 * j + 2], a.scale, c[j].z)),
                                           weight_log(y[4 * j + 3], a.scale, c[j].w));
                        }
                    }
                }
                const float all = (sum[0] + sum[1]) + (sum[2] + sum[3]);
                const float ref = floorf(fmaxf(top[0], top[1]));
                float low = 0.f;
                if (kWide && __any_sync(kFull, at < s.n && all < kSmall))
#pragma unroll 1
                    for (int c0 = 0; c0 < cols; c0 += 16) {
                        uint32_t y[16];
                        tmem_ld16_async(tmem + lanes + db * a.dcols + c0, y);
                        tmem_wait_ld();
                        tmem_bind16(y);
#pragma unroll
                        for (int j = 0; j < 16; j++)
                            low += ex2_approx(weight_log(y[j], a.scale, S.c[qb][c0 + j]) - ref);
                    }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&S.dempty[db]);
                if (at < s.n) {
                    if (kWide)
                        static_cast<double *>(a.S)[slot] =
                            all < kSmall ? widen(low * vote, (int)ref) : widen(all * vote);
                    else
                        static_cast<float *>(a.S)[slot] = all * vote;
                }
            }
            k += s.tiles;
            __syncwarp();
            if (ok && lane == 0) mbar_arrive(&S.qempty[qb]);
        }
    }
    __syncthreads();
    lead();
    if (warp == kMma) tmem_dealloc(tmem, 512);
    if (tid == 0 && S.bad) record_status(a.status, KVC_ERR_TIMEOUT);
}

}  // namespace

cudaError_t launch_tree_weights(const kvc_params &p, int max_len, const TreeArgs &t,
                                const PathArgs &pa, const float *row_weight, const uint16_t *q,
                                const uint16_t *kt, const float *lse, const kvc_cache &c, void *S,
                                bool wide, void *ws, cudaStream_t st)
{
    const long long tmax = (max_len + kTile - 1) / kTile, tiles = p.U * tmax;
    if (tiles > 0x7fffffffll) return cudaErrorInvalidValue;
    CUtensorMap mk;
    if (!make_unit_map(&mk, c.K, p.U, p.cap)) return cudaErrorInvalidValue;
    WtArgs a{t, pa, row_weight, q, kt, lse, c.votes, c.len, S, static_cast<int32_t *>(ws), p.U, p.G,
             p.G == 1 ? 0 : p.G == 2 ? 1 : p.G == 4 ? 2 : 3, p.cap, max_len};
    a.rows = (pa.A * p.G + 15) & ~15;
    a.blocks = (pa.A + 15) / 16;
    a.qbufs = a.rows <= 128 ? 2 : 1;
    a.dcols = a.rows <= 128 ? 128 : a.rows <= 256 ? 256 : 512;
    a.dbufs = 512 / a.dcols;
    a.ring = (int)((kMostSmem - kCtl - (size_t)a.qbufs * a.rows * 256) / kSlot);
    if (a.ring > kMaxRing) a.ring = kMaxRing;
    a.by_units = FastDiv(t.units);
    a.scale = kLog2e / sqrtf((float)kD);
    const size_t smem = (size_t)a.ring * kSlot + (size_t)a.qbufs * a.rows * 256 + sizeof(WtSmem);
    // (the attribute is the kernel's, shared by the host's threads: never one call's size)
    auto *kernel = wide ? tree_weights_kernel<true> : tree_weights_kernel<false>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostSmem);
    if (e != cudaSuccess) return e;
    long long grid = tiles > p.U ? tiles : p.U;
    if (grid > kGrid) grid = kGrid;
    return launch_following(kernel, dim3((unsigned)grid), kThreads, smem, st, a, mk);
}

}  // namespace kvc

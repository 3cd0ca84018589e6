// kvc_page_attend.cu -- one new token appended to a cache in pages and attended
// over it (kvc_page_attend).
//
//   x_i = q . k_i / sqrt(d),  lse = log sum exp(x_i),  o = sum exp(x_i - lse) v_i
//
// Bound by the bytes of the rows (512 per slot in bf16, 264 in e4m3): at eight
// heads 4 G d = 4096 operations per slot, 16 per byte, more than the CUDA cores
// keep up with beside the unpacking.  The products are mma.sync on fragments
// that are loaded from the pages straight into registers, slots on the M side
// (S' = K Q', O' = V' P', heads on the N side, eight of them): every lane's load
// is 16 bytes of one row, and no tile passes through shared memory.  What the
// operand layouts ask for is had by choosing the order of d: any order will do
// for K as long as Q has the same, and V's lanes hold four slots of the same
// dimensions, interleaved by byte permutes.  tcgen05 would need tiles of 128 rows
// in shared memory, in one type for both operands (e4m3 rows against bf16
// queries), for products that take a few percent of the time here.
//
// Precision.  Logits, maxima, sums and outputs are fp32; the tensor core cuts its sums
// off instead of rounding them, which adds up over a long run (3e-6 of o over 2300
// slots of a warp), so it has the 16 slots of a product alone and those are added with
// rounding (no cost but with eight heads over e4m3: 32 units x 16000 32.2 -> 33.3 us;
// the 32 slots of a tile at once spill, 146.5 -> 149.2 for 128 units x <= 32768).
// Weights enter O' as two 16-bit terms (bf16 beside bf16 values, 2^-17 of a weight left; f16 beside e4m3
// values, which f16 holds exactly).  Queries beside e4m3 keys are f16 after a
// power of two per head puts the largest at 2^13: bf16's 8 bits fit f16's 11 down
// to 2^-27 of it.  With e4m3 values there are two references: the weights' sum has the
// maximum of x, the contributions that of x + (the exponent of the value's scale), so
// that the largest contribution, not the largest weight, is near 2^7 in f16, whose steps
// (2^-24) are 2^-31 of it: a row of huge values that weighs nothing does not push the
// others below f16's range, and values of any magnitude leave the weights' sum alone.
// The second is held as its whole number of octaves above the first.
//
// A reference moves only when a weight or a contribution passes 2^8 of it: one vote per
// tile in place of six exchanges, and the sums are rarely scaled.  What a warp, or a part
// of a unit, gives to a join is its own o and the weights' maximum and sum.
//
// Work: tiles of 16 (bf16) or 32 slots of all units form one line, cut into equal
// parts for a fixed number of warps, whatever bound the caller gives for the
// lengths.  A warp walks its part alone, without a barrier, the next tile's rows
// on their way in registers across the ends of units.  A unit that is cut leaves
// its parts in the workspace, which a second kernel joins in the order of the line.
// Short units that all fit at once go whole to a cluster each, whose warps take its
// tiles in turn and join over distributed shared memory: no line, no second kernel.
//
// Measured, calls replayed as a graph: 8 units x 131071 slots bf16 85 us (6.3 TB/s),
// 128 units x <= 32768 e4m3 146.6 us (6.2; 145.4 with one reference for the weights' sum
// and the contributions), 1024 units x <= 1024 e4m3 43.2 us (4.9; 42.7), 128 x <= 3277
// bf16 with 8 heads 34.9 us (5.1), 8 x 64 3.7 us.  What is left is a chain of waits at
// either end: lengths, pages, first rows (about 3 us), the join (4 us, of which an empty
// kernel is 0.5 and reading the cuts 0.9).  Tried and slower: the next tiles in a ring of shared memory filled by
// cp.async (8 x 131071: 115); a tile of a CTA's four warps with a barrier per unit (1024
// units: 48); e4m3 tiles of 16 slots (47, and 44.5 with four CTAs per SM); joins by the
// last CTA or warp to come (registers spill); a CTA's parts joined in shared memory
// first (1024 units 43.9, 128 x <= 3277 37.1: the CTA waits for its slowest warp).
#include "kvc_page.h"

#include <cuda_fp16.h>
#include <float.h>
#include <limits.h>
#include <math.h>

namespace kvc {
namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32;
constexpr int kResident = 3, kGrid = 152 * kResident, kWorkers = kGrid * kWarps;
constexpr int kHeads = 8;                        // columns of the products
constexpr float kSlack = 8.f;                    // log2 that a logit may pass the reference by

struct AttendArgs {
    PageArgs pg;
    const uint16_t *q, *k_new, *v_new;
    uint16_t *o;
    float *lse;
    int32_t *status, *part_bad;                  // [2 kWorkers]
    int2 *cuts;                                  // [U] the first and the last worker that has a part
    float *part_o, *part_ml;                     // [2 kWorkers][G][d], [2 kWorkers][G][2]
    int S, G, max_len, cluster;
};

__device__ __forceinline__ uint4 ldg16(const void *p)
{
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p));
    return r;
}

// 16 bytes to shared memory in the background
__device__ __forceinline__ void copy16(void *dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ uint32_t word(const uint4 &r, int i)
{
    return i == 0 ? r.x : i == 1 ? r.y : i == 2 ? r.z : r.w;
}

// D += A (16x16, row) * B (16x8, col) of bf16, or of f16
template <bool kF16>
__device__ __forceinline__ void mma(float *d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                    uint32_t b0, uint32_t b1)
{
    if (kF16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        mma16816(d, a0, a1, a2, a3, b0, b1);
}

// the 8x8 matrix of 16-bit elements that the warp holds, transposed
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a)
{
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

// a and b as two 16-bit terms each, a in the low halves
template <bool kF16>
__device__ __forceinline__ void two_terms(float a, float b, uint32_t &hi, uint32_t &lo)
{
    if (kF16) {
        const __half2 h = __floats2half2_rn(a, b);
        const float2 f = __half22float2(h);
        const __half2 l = __floats2half2_rn(a - f.x, b - f.y);
        hi = *reinterpret_cast<const uint32_t *>(&h);
        lo = *reinterpret_cast<const uint32_t *>(&l);
    } else {
        hi = to_bf16x2(a, b);
        lo = to_bf16x2(a - bf_lo(hi), b - bf_hi(hi));
    }
}

// 2^x; results below fp32's normal range are zero
__device__ __forceinline__ float pow2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// 1 / x to an ulp; a NaN stays
__device__ __forceinline__ float reciprocal(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// The exponent field u of a value's scale 2^(u - 127) f, f in [1, 2).  A NaN or an infinity
// moves no reference (the product with it is NaN all the same): lse does not depend on values.
__device__ __forceinline__ float scale_exponent(float s)
{
    const uint32_t e = __float_as_uint(s) >> 23 & 0xff;
    return e == 0xff ? 0.f : (float)(int)e;
}

// What sums of contributions over 2^(e - 127) of the weights' reference become o by: two
// factors, neither past fp32's range, of the weights' sum l over its reference m (0 where
// there is no weight: o is 0 then).
template <bool kE4m3>
__device__ __forceinline__ float2 to_mean(float m, float l, float e)
{
    const float inv = m == -INFINITY && l == 0.f ? 0.f : reciprocal(l);
    if (!kE4m3) return make_float2(inv, 1.f);
    const float h = floorf((e - 127.f) * 0.5f);
    return make_float2(inv * pow2(h), pow2(e - 127.f - h));
}

// four e4m3 values as f16 (exact): the low two, the high two
__device__ __forceinline__ void e4m3_to_f16x4(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}\n"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}

template <bool kWhole>
struct Shared {
    __align__(16) uint16_t q[kWarps][kWhole ? 1 : 2][kHeads * kD];      // queries of the unit at hand and of the next
    __align__(16) uint16_t fresh[kWarps][2][kD];           // the new token's key and value
    __align__(16) uint8_t row[kWarps][2][kD * 2];          // as they are held
    int scratch[33];
    int seq[kWarps], at[kWarps];
    // kWhole: the warps' sums, whether a page was bad
    __align__(16) float o[kWhole ? kWarps : 1][kHeads][kD + 4];
    __align__(8) float2 ml[kWhole ? kWarps : 1][kHeads];
    int bad;
};

// what stands at the same place of CTA `rank` of the cluster
__device__ __forceinline__ uint32_t far_address(const void *p, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    return r;
}

__device__ __forceinline__ int far_int(const int *p, uint32_t rank)
{
    int r;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(r) : "r"(far_address(p, rank)) : "memory");
    return r;
}

__device__ __forceinline__ float2 far_float2(const float2 *p, uint32_t rank)
{
    float2 r;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                 : "=f"(r.x), "=f"(r.y)
                 : "r"(far_address(p, rank))
                 : "memory");
    return r;
}

__device__ __forceinline__ float4 far_float4(const float *p, uint32_t rank)
{
    float4 r;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(r.x), "=f"(r.y), "=f"(r.z), "=f"(r.w)
                 : "r"(far_address(p, rank))
                 : "memory");
    return r;
}

// What a lane holds of the slots a warp has of a tile: kBlocks blocks of 16.
template <bool kE4m3>
struct Frags {
    static constexpr int kBlocks = kE4m3 ? 2 : 1;
    static constexpr int kSlots = 16 * kBlocks;
    static constexpr int kRow = kE4m3 ? kD : kD * 2;       // bytes
    static constexpr int kK = kRow / 64, kV = kRow / 128;  // a lane's pieces of a key, of a value
    uint4 k[kBlocks * 2 * kK], v[kBlocks * 4 * kV];
    float ks[kBlocks * 2], vs[kBlocks * 2];
};

// A walk along the line, a tile at a time.
struct Walk {
    int s, h, n, tiles, tile;                    // sequence, head, its length, a unit's tiles, the tile
    int ahead;                                   // the next sequence's length
};

// o and lse of row i (unit and head), four dimensions a lane; L is the weights' sum over 2^M
__device__ __forceinline__ void store_row(const AttendArgs &a, size_t i, int lane, float M, float L, float4 o)
{
    *reinterpret_cast<uint2 *>(a.o + i * kD + lane * 4) = make_uint2(to_bf16x2(o.x, o.y), to_bf16x2(o.z, o.w));
    if (lane == 0) a.lse[i] = (M + log2f(L)) * 0.6931471805599453f;
}

enum { kNothing, kDone, kTooMany, kBad };

// 1 / L for sums of weights: 0 where there are none, and a NaN stays
__device__ __forceinline__ float share_of(float L) { return L == 0.f ? 0.f : reciprocal(L); }

// A share of the parts of row i (unit and head): its o, and the weights' sum L over 2^M, M
// the largest of the share.  kNothing where there are none; kTooMany, and nothing done, where there
// are more than `most`; kBad where one has a page outside the pool.
__device__ __forceinline__ int sum_parts(const AttendArgs &a, int i, int share, int shares, int lane, int most,
                                         float &M, float &L, float4 &o)
{
    const int G = a.G;
    const int u = i / G, hh = i - u * G;
    const int2 cut = a.cuts[u];
    const int n = a.pg.len[a.pg.by_heads(u)];
    // a unit that was refused has no parts, and what stands in cuts is another call's
    if (n < 0 || n > a.max_len - (a.k_new != nullptr) || cut.x >= cut.y) return kNothing;
    const int parts = cut.y - cut.x + 1;
    if (parts > most) return kTooMany;
    auto slot = [&](int p) { return 2 * (cut.x + p) + (p == 0); };
    const int mine = (uint32_t)(parts - 1) / (uint32_t)shares + 1, begin = share * mine, end = min(parts, begin + mine);
    // the first sums load beside their maxima: one wait for a share of up to eight parts
    float4 x[8];
    auto load = [&](int p) {
#pragma unroll
        for (int j = 0; j < 8; j++)
            if (p + j < end)
                x[j] = *reinterpret_cast<const float4 *>(a.part_o + ((size_t)slot(p + j) * G + hh) * kD + lane * 4);
    };
    load(begin);
    bool wrong = false;
    for (int p0 = begin; p0 < end; p0 += 32) {
        float2 ml = make_float2(-INFINITY, 0.f);
        if (p0 + lane < end) {
            ml = *reinterpret_cast<const float2 *>(a.part_ml + ((size_t)slot(p0 + lane) * G + hh) * 2);
            wrong |= a.part_bad[slot(p0 + lane)] != 0;
        }
        const float top = fmaxf(M, warp_max(ml.x));
        // weights of what there is and of the parts, as shares of their sum (0 keeps a NaN)
        float c = p0 == begin ? 0.f : (M == -INFINITY ? 0.f : pow2(M - top)) * L;
        float r = (ml.x == -INFINITY ? 0.f : pow2(ml.x - top)) * ml.y;
        M = top;
        L = c + warp_sum(r);
        const float inv = share_of(L);
        c *= inv, r *= inv;
        if (p0 > begin) o = make_float4(o.x * c, o.y * c, o.z * c, o.w * c);
        for (int j0 = 0; j0 < 32 && p0 + j0 < end; j0 += 8) {
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const float f = __shfl_sync(kFull, r, j0 + j);
                if (p0 + j0 + j < end)
                    o = make_float4(fmaf(f, x[j].x, o.x), fmaf(f, x[j].y, o.y), fmaf(f, x[j].z, o.z),
                                    fmaf(f, x[j].w, o.w));
            }
            load(p0 + j0 + 8);
        }
    }
    return __any_sync(kFull, wrong) ? kBad : kDone;
}

// The parts of units that were cut, joined in the order of the line: kShares warps
// per row (unit and head), each a share of the parts, whose sums meet in shared
// memory.  Four dimensions a lane; weights of 32 parts are formed in the lanes.  With
// one warp per row, rows of many parts (a long unit among short ones) are taken by the
// whole block; a unit's rows belong to different blocks.
template <int kShares>
__global__ void __launch_bounds__(kShares < 8 ? 256 : 32 * kShares, kShares < 8 ? 4 : 1) join_kernel(const __grid_constant__ AttendArgs a)
{
    constexpr int kJoinWarps = kShares < 8 ? 8 : kShares, kRows = kJoinWarps / kShares;
    constexpr int kMost = 24;                    // parts that a warp takes alone
    __shared__ float4 sums[kJoinWarps][32];
    __shared__ float part_m[kJoinWarps], part_l[kJoinWarps];
    __shared__ int got[kJoinWarps];
    follow();
    lead();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rows = a.S * a.pg.heads * a.G;
    for (int i0 = blockIdx.x; i0 < rows; i0 += gridDim.x * kRows) {
        // kShares = 1: first every warp its own row, then the block row after row of those left over
        constexpr int kTurns = kShares == 1 ? 1 + kRows : 1;
        uint32_t left = 0;                       // rows of the block that are left over
#pragma unroll 1
        for (int turn = 0; turn < kTurns; turn++) {
            const bool alone = kShares == 1 && turn == 0;
            if (turn > 0 && !(left >> (turn - 1) & 1)) continue;
            const int shares = alone ? 1 : kShares == 1 ? kJoinWarps : kShares, share = warp % shares;
            const int i = i0 + (turn > 0 ? turn - 1 : warp / shares) * gridDim.x;
            float M = -INFINITY, L = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            int done = i < rows ? sum_parts(a, i, share, shares, lane, alone ? kMost : INT_MAX, M, L, o) : kNothing;
            if (alone) {
                if (done == kDone) store_row(a, i, lane, M, L, o);
                if (done == kBad && lane == 0) record_status(a.status, KVC_ERR_INVALID_ARG);
                if (lane == 0) got[warp] = done;
                if (!__syncthreads_or(done == kTooMany)) break;
                for (int w = 0; w < kRows; w++) left |= (uint32_t)(got[w] == kTooMany) << w;
                __syncthreads();                 // got is written again
                continue;
            }
            sums[warp][lane] = o;
            if (lane == 0) part_m[warp] = M, part_l[warp] = L, got[warp] = done;
            __syncthreads();
            if (share == 0 && done != kNothing) {
                float top = M;
                for (int w = 1; w < shares; w++) {
                    top = fmaxf(top, part_m[warp + w]);
                    if (got[warp + w] == kBad) done = kBad;
                }
                // lane w has the weight of share w (0 keeps a NaN)
                float r = 0.f;
                if (lane < shares) r = (part_m[warp + lane] == -INFINITY ? 0.f : pow2(part_m[warp + lane] - top)) * part_l[warp + lane];
                L = warp_sum(r);
                r *= share_of(L);
                o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                for (int w = 0; w < shares; w++) {
                    const float c = __shfl_sync(kFull, r, w);
                    const float4 x = sums[warp + w][lane];
                    o = make_float4(fmaf(c, x.x, o.x), fmaf(c, x.y, o.y), fmaf(c, x.z, o.z), fmaf(c, x.w, o.w));
                }
                if (done == kDone) store_row(a, i, lane, top, L, o);
                else if (lane == 0) record_status(a.status, KVC_ERR_INVALID_ARG);
            }
            __syncthreads();
        }
    }
}

// kFew: at most four heads, whose weights' two terms are columns h and h + 4 of one
// product.
// kWhole: a unit goes whole to a cluster of a.cluster CTAs (1 to 8), whose warps take
// its tiles in turn and meet in shared memory: neither the line nor a second kernel is
// needed.
template <bool kE4m3, bool kFew, bool kWhole>
__global__ void __launch_bounds__(kThreads, kResident) attend_kernel(const __grid_constant__ AttendArgs a)
{
    using F = Frags<kE4m3>;
    constexpr int kBlocks = F::kBlocks, kTile = F::kSlots, kRow = F::kRow;
    __shared__ Shared<kWhole> sm;
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(kFull, tid >> 5, 0);   // uniform
    const int g = lane >> 2, c = lane & 3;
    const int app = a.k_new != nullptr, heads = a.pg.heads, G = a.G;
    follow();
    lead();

    // the line: tiles of every sequence's units in order, cut into equal parts for the warps
    auto length = [&](int s) { return s < a.S ? a.pg.len[s] : 0; };
    auto tiles_of = [&](int n) { return n < 0 || n > a.max_len - app ? 0 : max(1, (n + app + kTile - 1) / kTile); };
    Walk cur;                                    // the unit at hand
    int id = 0, t, t_end, unit_at = 0;           // the worker, its part of the line, the unit's first tile
    LineCuts cuts(1, 0);
    const int step = kWhole ? a.cluster * kWarps : 1;      // tiles from one of a warp to its next
    if (kWhole) {
        const int u = blockIdx.x / (unsigned)a.cluster;
        id = (blockIdx.x - u * a.cluster) * kWarps + warp;
        cur.s = a.pg.by_heads(u);
        cur.h = u - cur.s * heads;
        cur.n = a.pg.len[cur.s];
        cur.tiles = tiles_of(cur.n);
        cur.tile = cur.ahead = 0;
        t = 0, t_end = cur.tiles;
        if (t_end == 0) {
            if (tid == 0) record_status(a.status, KVC_ERR_SHAPE);
            return;                              // the whole cluster
        }
        cur.tile = id;
    } else {
        const int each = (a.S + kThreads - 1) / kThreads;
        const int s0 = min(a.S, tid * each), s1 = min(a.S, s0 + each);
        int mine = 0, refused = 0;
#pragma unroll 8
        for (int s = s0; s < s1; s++) {
            const int t = tiles_of(a.pg.len[s]);
            refused |= t == 0;
            mine += t * heads;
        }
        if (refused && blockIdx.x == 0) record_status(a.status, KVC_ERR_SHAPE);
        int total;
        const int before = block_exscan(mine, sm.scratch, &total);
        cuts = LineCuts(gridDim.x * kWarps, total);
#pragma unroll
        for (int w = 0; w < kWarps; w++) {
            const int id = w * gridDim.x + blockIdx.x, t = cuts.start(id);
            if (id < cuts.parts && t >= before && t < before + mine) {
                int at = before, s = s0, size;
                while (at + (size = tiles_of(a.pg.len[s]) * heads) <= t) at += size, s++;
                sm.seq[w] = s;
                sm.at[w] = at;
            }
        }
        __syncthreads();
        id = warp * gridDim.x + blockIdx.x;          // few tiles go to as many SMs as there are
        if (id >= cuts.parts) return;
        t = cuts.start(id);
        t_end = cuts.start(id + 1);
        cur.s = sm.seq[warp];
        cur.n = length(cur.s);
        cur.ahead = length(cur.s + 1);
        cur.tiles = tiles_of(cur.n);
        unit_at = sm.at[warp];
        cur.h = (t - unit_at) / cur.tiles;
        unit_at += cur.h * cur.tiles;
        cur.tile = t - unit_at;
    }
    auto next_unit = [&](Walk &w) {
        w.tile = 0;
        if (++w.h < heads) return;
        w.h = 0;
        do {
            w.s++;
            w.n = w.ahead;
            w.ahead = length(w.s + 1);
            w.tiles = tiles_of(w.n);
        } while (w.tiles == 0 && w.s < a.S);
    };

    // the tile after the one at hand is on its way, its successor's pages are known
    Walk far = cur;
    int far_left = kWhole ? (t_end - id + step - 1) / step : t_end - t;
    int far_h = 0, far_slot = 0, far_live = 0, ids[kBlocks];       // of what is loaded next
    bool far_bad = false;
    F f;
    auto look_up = [&]() {
        far_h = far.h;
        far_slot = far.tile * kTile;
        far_live = far_left > 0 ? far.n - far_slot : 0;           // slots from far_slot on that hold a row
#pragma unroll
        for (int b = 0; b < kBlocks; b++) ids[b] = far_live > 16 * b ? a.pg.entry(far.s, far_slot + 16 * b) : 0;
        --far_left;
        far.tile += step;
        if (!kWhole && far_left > 0 && far.tile == far.tiles) next_unit(far);
    };
    auto load = [&](bool keys) {
#pragma unroll
        for (int b = 0; b < kBlocks; b++) {
            int live = far_live - 16 * b;
            const bool ok = a.pg.in_pool(ids[b]);
            if (live > 0 && !ok) far_bad = true, live = 0;
            const size_t row = live > 0 ? a.pg.row(ids[b], far_h, far_slot + 16 * b) : 0;
            if (keys) {
                const uint8_t *p = a.pg.K + (row + g) * kRow + c * 16;
                const float *ps = a.pg.ks + row + g, *pv = a.pg.vs + row + g;
                if (live >= 16) {
#pragma unroll
                    for (int r = 0; r < 2; r++) {
#pragma unroll
                        for (int j = 0; j < F::kK; j++) f.k[(b * 2 + r) * F::kK + j] = ldg16(p + r * 8 * kRow + j * 64);
                        if (kE4m3) f.ks[b * 2 + r] = ps[8 * r], f.vs[b * 2 + r] = pv[8 * r];
                    }
                } else {
#pragma unroll
                    for (int r = 0; r < 2; r++) {
                        const bool on = g + 8 * r < live;
#pragma unroll
                        for (int j = 0; j < F::kK; j++)
                            f.k[(b * 2 + r) * F::kK + j] = on ? ldg16(p + r * 8 * kRow + j * 64) : make_uint4(0, 0, 0, 0);
                        if (kE4m3) f.ks[b * 2 + r] = on ? ps[8 * r] : 0.f, f.vs[b * 2 + r] = on ? pv[8 * r] : 0.f;
                    }
                }
            } else {
                const uint8_t *p = a.pg.V + (row + 2 * c) * kRow + g * 16;
                if (live >= 16) {
#pragma unroll
                    for (int i = 0; i < 4; i++)
#pragma unroll
                        for (int j = 0; j < F::kV; j++)
                            f.v[(b * 4 + i) * F::kV + j] = ldg16(p + ((i & 1) + 8 * (i >> 1)) * kRow + j * 128);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        const int r = (i & 1) + 8 * (i >> 1);
#pragma unroll
                        for (int j = 0; j < F::kV; j++)
                            f.v[(b * 4 + i) * F::kV + j] =
                                2 * c + r < live ? ldg16(p + r * kRow + j * 128) : make_uint4(0, 0, 0, 0);
                    }
                }
            }
        }
    };
    // the queries of a unit to shared memory
    auto fetch_q = [&](int buf, int u) {
        for (int i = lane; i < G * 16; i += 32) copy16(sm.q[warp][buf] + i * 8, a.q + (size_t)u * G * kD + i * 8);
    };
    int qbuf = 0;
    fetch_q(0, cur.s * heads + cur.h);
    look_up();
    load(true);
    load(false);
    look_up();

    const int head = kFew ? g & 3 : g;           // of the column that the lane's queries are
    const float log2e_d = 0.08838834764831845f * 1.4426950408889634f;   // log2(e) / sqrt(128)
    while (t < t_end) {
        const int u = cur.s * heads + cur.h, n = cur.n, tiles = cur.tiles;
        const int first = cur.tile, end = min(t_end - unit_at, tiles);
        // the new token's slot is in the last tile
        const bool has_new = app && end == tiles && (!kWhole || (tiles - 1) % step == id);
        copies_wait();
        __syncwarp();

        // queries: the lane's 32 dimensions of a head, in the order of the keys' loads
        uint32_t q[8][2];
        float ch0 = log2e_d, ch1 = log2e_d;      // what a product becomes a logit (base 2) by
        {
            uint4 w[4];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const int d = kE4m3 ? ((j >> 1) * 4 + c) * 16 + (j & 1) * 8 : (j * 4 + c) * 8;
                w[j] = head < G ? *reinterpret_cast<const uint4 *>(sm.q[warp][qbuf] + head * kD + d) : make_uint4(0, 0, 0, 0);
            }
            if (kE4m3) {
                uint32_t top = 0;                // magnitudes order as whole numbers
#pragma unroll
                for (int j = 0; j < 4; j++)
                    top = __vmaxu2(top, __vmaxu2(__vmaxu2(magnitudes(w[j].x), magnitudes(w[j].y)),
                                                 __vmaxu2(magnitudes(w[j].z), magnitudes(w[j].w))));
                top = __vmaxu2(top, __shfl_xor_sync(kFull, top, 1));
                top = __vmaxu2(top, __shfl_xor_sync(kFull, top, 2));
                top = max(top & 0xffffu, top >> 16) >> 7;      // the exponent
                // 2^e takes the largest to [2^13, 2^14)
                const int e = min(13 + 127 - (int)top, 120);
                const float f2 = __uint_as_float((uint32_t)(e + 127) << 23);
                const float back = __uint_as_float((uint32_t)(127 - e) << 23);
                ch0 *= __shfl_sync(kFull, back, 8 * c);
                ch1 *= __shfl_sync(kFull, back, 8 * c + 4);
#pragma unroll
                for (int j = 0; j < 4; j++)
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        const float2 y = scaled2(word(w[j], i), f2);
                        const __half2 x = __floats2half2_rn(y.x, y.y);
                        q[j * 2 + (i >> 1)][i & 1] = *reinterpret_cast<const uint32_t *>(&x);
                    }
            } else {
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    q[2 * j][0] = w[j].x, q[2 * j][1] = w[j].y;
                    q[2 * j + 1][0] = w[j].z, q[2 * j + 1][1] = w[j].w;
                }
            }
        }
        // what the unit's end and the next unit need comes in the background
        int fresh_page = 0;
        if (has_new) {
            copy16(sm.fresh[warp][lane >> 4] + (lane & 15) * 8,
                   (lane < 16 ? a.k_new : a.v_new) + (size_t)u * kD + (lane & 15) * 8);
            fresh_page = a.pg.entry(cur.s, n);
        }
        if (!kWhole && unit_at + tiles < t_end) {
            Walk then = cur;
            next_unit(then);
            fetch_q(qbuf ^ 1, then.s * heads + then.h);
        }

        float acc[8][4] = {}, m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
        float e0 = 1.f, e1 = 1.f;                // octaves of the contributions' reference over m, and 127
        bool bad = false;
        for (int tile = first; tile < end; tile += step) {
            int live = n - tile * kTile;
            bad |= far_bad;
            far_bad = false;
            if (has_new && tile + 1 == end) {
                // the new token's row: to its page, and into the registers as it is held
                const bool ok = a.pg.in_pool(fresh_page);
                bad |= !ok;
                const size_t row = ok ? a.pg.row(fresh_page, cur.h, n) : 0;
                copies_wait();
                __syncwarp();
                float sc[2] = {};
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    const uint2 w = reinterpret_cast<const uint2 *>(sm.fresh[warp][i])[lane];
                    uint8_t *pool = i ? a.pg.V : a.pg.K;
                    if (kE4m3) {
                        uint32_t top = __vmaxu2(magnitudes(w.x), magnitudes(w.y));
#pragma unroll
                        for (int j = 16; j; j >>= 1) top = __vmaxu2(top, __shfl_xor_sync(kFull, top, j));
                        sc[i] = row_scale(__uint_as_float(max(top << 16, top & 0xffff0000u)));
                        const uint32_t v = quantise4(w.x, w.y, __fdiv_rn(1.f, sc[i]));
                        reinterpret_cast<uint32_t *>(sm.row[warp][i])[lane] = v;
                        if (ok) {
                            *reinterpret_cast<uint32_t *>(pool + row * kRow + lane * 4) = v;
                            if (lane == 0) (i ? a.pg.vs : a.pg.ks)[row] = sc[i];
                        }
                    } else {
                        reinterpret_cast<uint2 *>(sm.row[warp][i])[lane] = w;
                        if (ok) *reinterpret_cast<uint2 *>(pool + row * kRow + lane * 8) = w;
                    }
                }
                __syncwarp();
#pragma unroll
                for (int b = 0; b < kBlocks; b++) {
                    const int at = live - 16 * b;                  // its place in the block
#pragma unroll
                    for (int r = 0; r < 2; r++)
                        if (at == g + 8 * r) {
#pragma unroll
                            for (int j = 0; j < F::kK; j++) f.k[(b * 2 + r) * F::kK + j] = lds_v4(sm.row[warp][0] + c * 16 + j * 64);
                            f.ks[b * 2 + r] = sc[0], f.vs[b * 2 + r] = sc[1];
                        }
#pragma unroll
                    for (int i = 0; i < 4; i++)
                        if (at == 2 * c + (i & 1) + 8 * (i >> 1))
#pragma unroll
                            for (int j = 0; j < F::kV; j++) f.v[(b * 4 + i) * F::kV + j] = lds_v4(sm.row[warp][1] + g * 16 + j * 128);
                }
                live++;
            }
            // S' = K Q'
            float x[kBlocks][4];
#pragma unroll
            for (int b = 0; b < kBlocks; b++) {
                float y[4] = {};
                x[b][0] = x[b][1] = x[b][2] = x[b][3] = 0.f;
#pragma unroll
                for (int j = 0; j < F::kK; j++) {
                    const uint4 &r0 = f.k[b * 2 * F::kK + j], &r1 = f.k[(b * 2 + 1) * F::kK + j];
                    if (kE4m3) {
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            uint32_t a0, a1, a2, a3;
                            e4m3_to_f16x4(word(r0, i), a0, a2);
                            e4m3_to_f16x4(word(r1, i), a1, a3);
                            mma<true>(i & 1 ? y : x[b], a0, a1, a2, a3, q[j * 4 + i][0], q[j * 4 + i][1]);
                        }
                    } else {
                        mma<false>(x[b], r0.x, r1.x, r0.y, r1.y, q[2 * j][0], q[2 * j][1]);
                        mma<false>(y, r0.z, r1.z, r0.w, r1.w, q[2 * j + 1][0], q[2 * j + 1][1]);
                    }
                }
#pragma unroll
                for (int j = 0; j < 4; j++) x[b][j] += y[j];
            }
            // logits in base 2 over the reference, what is not there at -inf; how far the tile passes
            // the references.  (The reference first: beside a large logit a scale's exponent is lost.
            // Products are rounded before it, so that equal ones stay equal.)
            const float ref0 = m0 == -INFINITY ? 0.f : m0, ref1 = m1 == -INFINITY ? 0.f : m1;
            float top0 = -INFINITY, top1 = -INFINITY, out0 = -INFINITY, out1 = -INFINITY;
            float vs[2 * kBlocks], high = 0.f;   // the values' scales, their largest exponent
#pragma unroll
            for (int b = 0; b < kBlocks; b++)
#pragma unroll
                for (int r = 0; r < 2; r++) {
                    const bool on = 16 * b + 8 * r + g < live;
                    float c0 = ch0, c1 = ch1, up = 0.f;
                    if (kE4m3) {
                        // finite, so that a product of zero stays a logit of zero
                        c0 = fminf(c0 * f.ks[b * 2 + r], FLT_MAX), c1 = fminf(c1 * f.ks[b * 2 + r], FLT_MAX);
                        vs[b * 2 + r] = f.vs[b * 2 + r];
                        up = scale_exponent(f.vs[b * 2 + r]);
                        high = fmaxf(high, up);
                    }
                    x[b][2 * r] = on ? __fmul_rn(x[b][2 * r], c0) - ref0 : -INFINITY;
                    x[b][2 * r + 1] = on ? __fmul_rn(x[b][2 * r + 1], c1) - ref1 : -INFINITY;
                    top0 = fmaxf(top0, x[b][2 * r]);
                    top1 = fmaxf(top1, x[b][2 * r + 1]);
                    if (kE4m3) {
                        out0 = fmaxf(out0, x[b][2 * r] + up);
                        out1 = fmaxf(out1, x[b][2 * r + 1] + up);
                    }
                }
            load(true);
            // contributions are at most 2^7 where their reference is met, 2^15 with the slack
            constexpr float kUp = 6.f;
            bool past = top0 > (m0 == -INFINITY ? -INFINITY : kSlack) || top1 > (m1 == -INFINITY ? -INFINITY : kSlack);
            if (kE4m3) past |= out0 > e0 + (kUp + kSlack) || out1 > e1 + (kUp + kSlack);
            if (__any_sync(kFull, past)) {
#pragma unroll
                for (int i = 4; i < 32; i <<= 1) {
                    top0 = fmaxf(top0, __shfl_xor_sync(kFull, top0, i));
                    top1 = fmaxf(top1, __shfl_xor_sync(kFull, top1, i));
                }
                // by how much m moves; from -inf the sums, which are zero, take no part
                const bool new0 = m0 == -INFINITY, new1 = m1 == -INFINITY;
                const float n0 = new0 ? top0 : m0 + fmaxf(top0, 0.f), n1 = new1 ? top1 : m1 + fmaxf(top1, 0.f);
                const float by0 = n0 == -INFINITY ? 0.f : n0 - ref0, by1 = n1 == -INFINITY ? 0.f : n1 - ref1;
                float d0 = new0 ? -INFINITY : -by0, d1 = new1 ? -INFINITY : -by1;
                l0 *= pow2(d0), l1 *= pow2(d1);
                m0 = n0, m1 = n1;
#pragma unroll
                for (int b = 0; b < kBlocks; b++) x[b][0] -= by0, x[b][1] -= by1, x[b][2] -= by0, x[b][3] -= by1;
                if (kE4m3) {
                    out0 = out1 = -INFINITY;
#pragma unroll
                    for (int b = 0; b < kBlocks; b++)
#pragma unroll
                        for (int r = 0; r < 2; r++) {
                            const float up = scale_exponent(vs[b * 2 + r]);
                            out0 = fmaxf(out0, x[b][2 * r] + up), out1 = fmaxf(out1, x[b][2 * r + 1] + up);
                        }
#pragma unroll
                    for (int i = 4; i < 32; i <<= 1) {
                        out0 = fmaxf(out0, __shfl_xor_sync(kFull, out0, i));
                        out1 = fmaxf(out1, __shfl_xor_sync(kFull, out1, i));
                    }
                    d0 += e0, d1 += e1;          // the old reference over the new m
                    e0 = fmaxf(ceilf(fmaxf(d0, out0 - kUp)), 1.f), e1 = fmaxf(ceilf(fmaxf(d1, out1 - kUp)), 1.f);
                    d0 -= e0, d1 -= e1;
                }
                const float r0 = pow2(d0), r1 = pow2(d1);
#pragma unroll
                for (int i = 0; i < 8; i++) acc[i][0] *= r0, acc[i][1] *= r1, acc[i][2] *= r0, acc[i][3] *= r1;
            }
            // weights, O' += V' P'
            const float s0 = pow2(127.f - e0), s1 = pow2(127.f - e1);
            // a value 2^100 above its reference, of a weight that fp32 may not hold: the
            // contribution is an exponential of its own
            const bool apart = kE4m3 && high - fminf(e0, e1) > 100.f;
#pragma unroll
            for (int b = 0; b < kBlocks; b++) {
                float p[4];
#pragma unroll
                for (int j = 0; j < 4; j++) p[j] = pow2(x[b][j]);
                l0 += p[0] + p[2];
                l1 += p[1] + p[3];
                if (kE4m3) {
#pragma unroll
                    for (int j = 0; j < 4; j++) p[j] *= vs[b * 2 + (j >> 1)] * (j & 1 ? s1 : s0);
                    if (apart)
#pragma unroll
                        for (int j = 0; j < 4; j++) {
                            const float v = vs[b * 2 + (j >> 1)], up = scale_exponent(v);
                            p[j] = pow2(x[b][j] + (up - (j & 1 ? e1 : e0))) *
                                   (up == 0.f ? v : __uint_as_float((__float_as_uint(v) & 0x807fffff) | 0x3f800000));
                        }
                }
                uint32_t hi0, lo0, hi1, lo1;
                two_terms<kE4m3>(p[0], p[1], hi0, lo0);
                two_terms<kE4m3>(p[2], p[3], hi1, lo1);
                if (kFew && c >= 2) hi0 = lo0, hi1 = lo1;
                hi0 = transpose8x8(hi0), hi1 = transpose8x8(hi1);
                if (!kFew) lo0 = transpose8x8(lo0), lo1 = transpose8x8(lo1);
                // a product's 16 rows are two dimensions of each lane's; it is added with rounding
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    uint32_t a0, a1, a2, a3;
                    if (kE4m3) {
                        // bytes of two slots side by side, dimensions 16 g + 2 i, + 1
                        const uint32_t sel = i & 1 ? 0x7362 : 0x5140;
                        e4m3_to_f16x4(__byte_perm(word(f.v[b * 4], i >> 1), word(f.v[b * 4 + 1], i >> 1), sel), a0, a1);
                        e4m3_to_f16x4(__byte_perm(word(f.v[b * 4 + 2], i >> 1), word(f.v[b * 4 + 3], i >> 1), sel), a2, a3);
                    } else {
                        // dimensions 8 g + 2 i, + 1 (and 64 on from the fourth)
                        const int j = i >> 2, w = i & 3;
                        a0 = __byte_perm(word(f.v[j], w), word(f.v[F::kV + j], w), 0x5410);
                        a1 = __byte_perm(word(f.v[j], w), word(f.v[F::kV + j], w), 0x7632);
                        a2 = __byte_perm(word(f.v[2 * F::kV + j], w), word(f.v[3 * F::kV + j], w), 0x5410);
                        a3 = __byte_perm(word(f.v[2 * F::kV + j], w), word(f.v[3 * F::kV + j], w), 0x7632);
                    }
                    float sum[4] = {};
                    mma<kE4m3>(sum, a0, a1, a2, a3, hi0, hi1);
                    if (!kFew) mma<kE4m3>(sum, a0, a1, a2, a3, lo0, lo1);
#pragma unroll
                    for (int j = 0; j < 4; j++) acc[i][j] += sum[j];
                }
            }
            load(false);
            look_up();
        }

        // the warp's sums: o and lse of a whole unit, else a part
        bad = __any_sync(kFull, bad);
        // a free place has no page for its token, which is no error
        auto record_bad = [&]() {
            if (!(app && n == 0 && a.pg.entry(cur.s, 0) == -1)) record_status(a.status, KVC_ERR_INVALID_ARG);
        };
#pragma unroll
        for (int i = 4; i < 32; i <<= 1) {
            l0 += __shfl_xor_sync(kFull, l0, i);
            l1 += __shfl_xor_sync(kFull, l1, i);
        }
        if (kFew)
#pragma unroll
            for (int i = 0; i < 8; i++)
#pragma unroll
                for (int j = 0; j < 4; j++) acc[i][j] += __shfl_xor_sync(kFull, acc[i][j], 2);
        const float2 f0 = to_mean<kE4m3>(m0, l0, e0), f1 = to_mean<kE4m3>(m1, l1, e1);
#pragma unroll
        for (int i = 0; i < 8; i++)
#pragma unroll
            for (int j = 0; j < 4; j++) acc[i][j] = acc[i][j] * (j & 1 ? f1.x : f0.x) * (j & 1 ? f1.y : f0.y);
        if (kWhole) {
            if (g == 0) {
                sm.ml[warp][2 * c] = make_float2(m0, l0);
                sm.ml[warp][2 * c + 1] = make_float2(m1, l1);
            }
#pragma unroll
            for (int j = 0; j < 2; j++)
                if (2 * c + j < G)
#pragma unroll
                    for (int i = 0; i < 8; i += 2) {
                        const int d = kE4m3 ? 16 * g + 2 * i : 8 * g + 2 * (i & 3) + 16 * (i & 4);
                        *reinterpret_cast<float4 *>(&sm.o[warp][2 * c + j][d]) =
                            make_float4(acc[i][j], acc[i][2 + j], acc[i + 1][j], acc[i + 1][2 + j]);
                    }
            const int any_bad = __syncthreads_or(bad);
            // a warp per head; lane w has the weight of the cluster's warp w
            auto join = [&](auto read_ml, auto read_o) {
                for (int hh = id; hh < G; hh += step) {
                    float2 ml = make_float2(-INFINITY, 0.f);
                    if (lane < step) ml = read_ml(hh);
                    const float M = warp_max(ml.x);
                    float r = (ml.x == -INFINITY ? 0.f : pow2(ml.x - M)) * ml.y;    // 0 keeps a NaN
                    const float L = warp_sum(r);
                    r *= share_of(L);
                    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
                    for (int w0 = 0; w0 < step; w0 += kWarps) {
                        float4 x[kWarps];
#pragma unroll
                        for (int w = 0; w < kWarps; w++) x[w] = read_o(w0, w, hh);
#pragma unroll
                        for (int w = 0; w < kWarps; w++) {
                            const float f = __shfl_sync(kFull, r, w0 + w);
                            o = make_float4(fmaf(f, x[w].x, o.x), fmaf(f, x[w].y, o.y), fmaf(f, x[w].z, o.z),
                                            fmaf(f, x[w].w, o.w));
                        }
                    }
                    store_row(a, (size_t)u * G + hh, lane, M, L, o);
                }
            };
            if (a.cluster == 1) {                // without the cluster's barriers (1 us of 4.6)
                if (!any_bad)
                    join([&](int hh) { return sm.ml[lane][hh]; },
                         [&](int, int w, int hh) { return *reinterpret_cast<const float4 *>(&sm.o[w][hh][lane * 4]); });
                else if (tid == 0)
                    record_bad();
                return;
            }
            if (tid == 0) sm.bad = any_bad;
            cluster_arrive();
            cluster_wait();
            const uint32_t there = lane / kWarps;
            if (!__any_sync(kFull, lane < step && far_int(&sm.bad, there) != 0))
                join([&](int hh) { return far_float2(&sm.ml[lane % kWarps][hh], there); },
                     [&](int w0, int w, int hh) { return far_float4(&sm.o[w][hh][lane * 4], w0 / kWarps); });
            else if (id == 0 && lane == 0)
                record_bad();
            // no CTA ends while another reads its sums
            cluster_arrive();
            cluster_wait();
            return;
        }
        const bool whole = first == 0 && end == tiles;
        const size_t part = 2 * id + (first == 0);
#pragma unroll
        for (int j = 0; j < 2; j++) {
            const int hh = 2 * c + j;
            if (hh >= G || (whole && bad)) continue;
            const float M = j ? m1 : m0, L = j ? l1 : l0;
            if (whole) {
                const size_t to = (size_t)u * G + hh;
#pragma unroll
                for (int i = 0; i < 8; i += 4) {
                    const int d = kE4m3 ? 16 * g + 2 * i : 8 * g + 16 * i;
                    *reinterpret_cast<uint4 *>(a.o + to * kD + d) =
                        make_uint4(to_bf16x2(acc[i][j], acc[i][2 + j]), to_bf16x2(acc[i + 1][j], acc[i + 1][2 + j]),
                                   to_bf16x2(acc[i + 2][j], acc[i + 2][2 + j]),
                                   to_bf16x2(acc[i + 3][j], acc[i + 3][2 + j]));
                }
                if (g == 0) a.lse[to] = (M + log2f(L)) * 0.6931471805599453f;
            } else {
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    const int d = kE4m3 ? 16 * g + 2 * i : 8 * g + 2 * (i & 3) + 16 * (i & 4);
                    *reinterpret_cast<float4 *>(a.part_o + (part * G + hh) * kD + d) =
                        make_float4(acc[i][j], acc[i][2 + j], acc[i + 1][j], acc[i + 1][2 + j]);
                }
                if (g == 0) *reinterpret_cast<float2 *>(a.part_ml + (part * G + hh) * 2) = make_float2(M, L);
            }
        }
        if (lane == 0) {
            if (whole && bad) record_bad();
            if (!whole) a.part_bad[part] = bad;
            if (first == 0) a.cuts[u] = make_int2(id, cuts.part(unit_at + tiles - 1));
        }

        // the next unit
        t = unit_at + end;
        unit_at += tiles;
        if (t < t_end) next_unit(cur);
        qbuf ^= 1;
    }
}

}  // namespace

size_t page_ws_bytes(const kvc_pages &pg, int G)
{
    return kAlign + align_up((size_t)pg.U * 8) + align_up(2 * kWorkers * 4) +
           align_up((size_t)2 * kWorkers * G * 2 * 4) + align_up((size_t)2 * kWorkers * G * kD * 4);
}

// as launch_following, in clusters
static cudaError_t launch_clusters(void (*kernel)(AttendArgs), int ctas, int cluster, cudaStream_t st,
                                   const AttendArgs &a)
{
    cudaLaunchConfig_t c{};
    c.gridDim = dim3(ctas);
    c.blockDim = dim3(kThreads);
    c.stream = st;
    cudaLaunchAttribute at[2] = {};
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    c.attrs = at;
    c.numAttrs = 2;
    return cudaLaunchKernelEx(&c, kernel, a);
}

cudaError_t launch_page_attend(const kvc_pages &pg, int G, int max_len, const uint16_t *q,
                               const uint16_t *k_new, const uint16_t *v_new, uint16_t *o, float *lse,
                               void *ws, cudaStream_t st)
{
    AttendArgs a{};
    a.pg = page_args(pg);
    a.q = q;
    a.k_new = k_new;
    a.v_new = v_new;
    a.o = o;
    a.lse = lse;
    uint8_t *at = static_cast<uint8_t *>(ws);
    a.status = &reinterpret_cast<WsHeader *>(at)->status;
    at += kAlign;
    a.cuts = reinterpret_cast<int2 *>(at);
    at += align_up((size_t)pg.U * 8);
    a.part_bad = reinterpret_cast<int32_t *>(at);
    at += align_up(2 * kWorkers * 4);
    a.part_ml = reinterpret_cast<float *>(at);
    at += align_up((size_t)2 * kWorkers * G * 2 * 4);
    a.part_o = reinterpret_cast<float *>(at);
    a.S = pg.U / pg.heads;
    a.G = G;
    a.max_len = max_len;
    const bool e4m3 = pg.type == KVC_PAGE_E4M3, few = G <= 4;
    const int tile = e4m3 ? Frags<true>::kSlots : Frags<false>::kSlots;
    // Short units go whole to a cluster each: as many CTAs as there are SMs for, four tiles at least
    // for each, at most ten for a warp.  In a graph, cluster / line (8 units in clusters of 8, 32 of
    // 4, 64 of 2, 128 and 456 alone): e4m3, 512 slots 7.0 / 8.4, 7.3 / 9.2, 8.2 / 10.7, 9.7 / 13.4,
    // 15.1 / 21.0 us; 1024 slots 7.7 / 8.6, 8.4 / 10.4, 11.0 / 13.7, 15.5 / 16.0, 23.7 / 29.5; 4096
    // slots 11.6 / 10.7, 16.7 / 15.2, 26.4 / 21.1, 46 / 31 (the first two go whole all the same, for
    // the lengths between); bf16, 1024 slots 6.7 / 7.7, 9.2 / 11.5, 4096 slots 12.9 / 12.3, 21.2 /
    // 18.0.  Larger clusters: 64 units of 512 slots in e4m3 8.9 in 4, 14.5 in 8.  Up to two CTAs'
    // worth of units: 768 of 256 slots 19.4 / 19.6 in e4m3, 21.1 / 24.1 in bf16; 1024 of them 25.5 /
    // 22.5 and 29.5 / 29.0.  With many units the line's warps lose about 1 us at the end of each,
    // which other CTAs hide: in bf16, of 128 slots on, 2048 units of 512 slots 88.3 / 91.5, 4096
    // 166 / 179, of 1024 slots 164 / 172 (4096 of 64 45.2 / 36.9; in e4m3 no gain: 2048 of 512 62.5 /
    // 57.2, 4096 of 256 78 / 64).
    const int tiles_each = (max_len - 1) / tile + 1;
    int cluster = 8;
    while (cluster > 1 && ((int64_t)pg.U * cluster > 152 || 4 * cluster > tiles_each)) cluster /= 2;
    a.cluster = cluster;
    if ((pg.U <= 2 * kGrid && tiles_each <= 10 * kWarps * cluster) ||
        (!e4m3 && pg.U >= 4 * kGrid && tiles_each >= 8 && tiles_each <= 20 * kWarps)) {
        void (*kernel)(AttendArgs) = e4m3 ? (few ? attend_kernel<true, true, true> : attend_kernel<true, false, true>)
                                          : (few ? attend_kernel<false, true, true> : attend_kernel<false, false, true>);
        return cluster == 1 ? launch_following(kernel, dim3(pg.U), kThreads, 0, st, a)
                            : launch_clusters(kernel, pg.U * cluster, cluster, st, a);
    }
    // no more CTAs than there can be tiles
    const int64_t tiles = (int64_t)pg.U * tiles_each;
    const dim3 grid((unsigned)(tiles < kGrid ? tiles : kGrid));
    void (*kernel)(AttendArgs) = e4m3 ? (few ? attend_kernel<true, true, false> : attend_kernel<true, false, false>)
                                      : (few ? attend_kernel<false, true, false> : attend_kernel<false, false, false>);
    const cudaError_t err = launch_following(kernel, grid, kThreads, 0, st, a);
    if (err != cudaSuccess) return err;
    const int64_t rows = (int64_t)pg.U * G, fill = 152 * 4;
    auto join = [&](void (*f)(AttendArgs), int per_block, int threads) {
        const int64_t blocks = (rows - 1) / per_block + 1;
        return launch_following(f, dim3((unsigned)(blocks < fill ? blocks : fill)), threads, 0, st, a);
    };
    // warps per row by the parts that a unit may have, each with a share of them (8 units of 131071
    // slots, 228 or 229 parts each: eight warps 85.4 us in a graph, 16 84.7, 32 85.4; 128 units, 16
    // parts of 8 heads: two warps 35.3, four 34.4, eight 39.1; 1024 units, two or three parts: one warp
    // 43.1, two 45.7)
    const int parts = kWorkers / pg.U + 2;
    if (parts <= 8) return join(join_kernel<1>, 8, 256);
    if (parts <= 32) return join(join_kernel<4>, 2, 256);
    return join(join_kernel<16>, 1, 512);
}

}  // namespace kvc

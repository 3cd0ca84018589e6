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
// Precision.  Logits, maxima, sums and outputs are fp32.  Weights enter O' as two
// 16-bit terms (bf16 beside bf16 values, 2^-17 of a weight left; f16 beside e4m3
// values, which f16 holds exactly).  Queries beside e4m3 keys are f16 after a
// power of two per head puts the largest at 2^13: bf16's 8 bits fit f16's 11 down
// to 2^-27 of it.  With e4m3 the reference of the exponentials is the maximum of
// x + (a power of two above the value's scale), so that the largest contribution,
// not the largest weight, is near 1 in f16: a row of huge values that weighs
// nothing does not push the others below f16's range.
//
// The reference moves only when a logit passes it by 2^8: one vote per tile in
// place of six exchanges, and the sums are rarely scaled.
//
// Work: tiles of all units form one line, cut into equal parts for a fixed number
// of persistent CTAs (three per SM), whatever bound the caller gives for the
// lengths.  A unit that is cut leaves its parts in the workspace; the CTA that
// comes last joins them in the order of the line, so results do not depend on it.
#include "kvc_page.h"

#include <cuda_fp16.h>
#include <math.h>

namespace kvc {
namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32;
constexpr int kGrid = 152 * 3;
constexpr int kHeads = 8;                        // columns of the products
constexpr int kPad = kD + 2;                     // row of a head in shared memory
constexpr float kSlack = 8.f;                    // log2 that a logit may pass the reference by

struct AttendArgs {
    PageArgs pg;
    const uint16_t *q, *k_new, *v_new;
    uint16_t *o;
    float *lse;
    int32_t *status, *arrived, *part_bad;        // [U], [2 kGrid]
    float *part_o, *part_ml;                     // [2 kGrid][G][d], [2 kGrid][G][2]
    int S, G, max_len;
};

__device__ __forceinline__ uint4 ldg16(const void *p)
{
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p));
    return r;
}

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

// log2 of a power of two above the scale, at least -100: weights over the reference
// are then at most 2^100, and their sum stays in range
__device__ __forceinline__ float scale_log2(float s)
{
    return fmaxf((float)((int)(__float_as_uint(s) >> 23) - 126), -100.f);
}

struct Shared {
    float o[kWarps][kHeads * kPad];
    float m[kWarps][kHeads], l[kWarps][kHeads];
    __align__(16) uint8_t row[2][kD * 2];        // the new token's key and value as held
    float row_scale[2];
    int scratch[33];
    int seq, at, last;
};

// What a lane holds of the slots a warp has of a tile: kBlocks blocks of 16.
template <bool kE4m3>
struct Frags {
    static constexpr int kBlocks = kE4m3 ? 2 : 1;
    static constexpr int kSlots = 16 * kBlocks;
    uint4 k[8], v[8];
    float ks[4], vs[4];
};

template <bool kE4m3>
__global__ void __launch_bounds__(kThreads, 3) attend_kernel(const __grid_constant__ AttendArgs a)
{
    using F = Frags<kE4m3>;
    constexpr int kTile = kWarps * F::kSlots;
    constexpr int kBytes = kE4m3 ? kD : kD * 2;
    __shared__ Shared sm;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, c = lane & 3;
    const int app = a.k_new != nullptr, heads = a.pg.heads, G = a.G;
    follow();
    lead();

    // the line: tiles of every sequence's units in order
    auto tiles_of = [&](int s) {
        const int n = a.pg.len[s];
        if (n < 0 || n > a.max_len - app) return 0;
        return max(1, (n + app + kTile - 1) / kTile);
    };
    const int each = (a.S + kThreads - 1) / kThreads;
    const int s0 = min(a.S, tid * each), s1 = min(a.S, s0 + each);
    int mine = 0;
    for (int s = s0; s < s1; s++) {
        const int t = tiles_of(s);
        if (t == 0 && blockIdx.x == 0) record_status(a.status, KVC_ERR_SHAPE);
        mine += t * heads;
    }
    int total;
    const int before = block_exscan(mine, sm.scratch, &total);
    const LineCuts cuts(gridDim.x, total);
    if ((int)blockIdx.x >= cuts.parts) return;
    int t = cuts.start(blockIdx.x);
    const int t_end = cuts.start(blockIdx.x + 1);
    if (t >= before && t < before + mine) {
        int at = before, s = s0, w;
        while (at + (w = tiles_of(s) * heads) <= t) at += w, s++;
        sm.seq = s;
        sm.at = at;
    }
    __syncthreads();
    int s = sm.seq, unit_at = sm.at, tiles = tiles_of(s);
    int h = (t - unit_at) / tiles;
    unit_at += h * tiles;

    const float log2e_d = 0.08838834764831845f * 1.4426950408889634f;   // log2(e) / sqrt(128)
    while (t < t_end) {
        const int u = s * heads + h, n = a.pg.len[s];
        const int first = t - unit_at, end = min(t_end - unit_at, tiles);
        const bool has_new = app && end == tiles;

        // queries: the lane's 32 dimensions of head g, in the order of the keys' loads
        uint32_t q[8][2];
        float ch0 = log2e_d, ch1 = log2e_d;      // what a product becomes a logit (base 2) by
        {
            uint4 w[4];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                const int d = kE4m3 ? ((j >> 1) * 4 + c) * 16 + (j & 1) * 8 : (j * 4 + c) * 8;
                w[j] = g < G ? *reinterpret_cast<const uint4 *>(a.q + ((size_t)u * G + g) * kD + d)
                             : make_uint4(0, 0, 0, 0);
            }
            if (kE4m3) {
                float amax = 0.f;
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    float f[8];
                    unpack8(w[j], f);
#pragma unroll
                    for (int i = 0; i < 8; i++) amax = fmaxf(amax, fabsf(f[i]));
                }
                amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 2));
                // 2^e takes the largest to [2^13, 2^14)
                const int e = min(13 + 127 - (int)(__float_as_uint(amax) >> 23), 120);
                const float f2 = __uint_as_float((uint32_t)(e + 127) << 23);
                const float back = __uint_as_float((uint32_t)(127 - e) << 23);
                ch0 *= __shfl_sync(kFull, back, 8 * c);
                ch1 *= __shfl_sync(kFull, back, 8 * c + 4);
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    float f[8];
                    unpack8(w[j], f);
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        const __half2 x = __floats2half2_rn(f[2 * i] * f2, f[2 * i + 1] * f2);
                        q[j * 2 + (i >> 1)][i & 1] = *reinterpret_cast<const uint32_t *>(&x);
                    }
                }
            } else {
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    q[2 * j][0] = w[j].x, q[2 * j][1] = w[j].y;
                    q[2 * j + 1][0] = w[j].z, q[2 * j + 1][1] = w[j].w;
                }
            }
        }

        float acc[8][4] = {}, m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
        F f;
        int ids[F::kBlocks];
        bool bad = false;
        const int mine_end = end + (has_new && warp == 0);   // one turn more, for the new token
        auto look_up = [&](int tile) {
#pragma unroll
            for (int b = 0; b < F::kBlocks; b++) {
                const int slot = tile * kTile + warp * F::kSlots + 16 * b;
                ids[b] = tile < end && slot < n ? a.pg.entry(s, slot) : 0;
            }
        };
        // slots of the tile that hold a row, from the lane's point of view: limit - 16 b
        auto load = [&](int tile, bool keys) {
#pragma unroll
            for (int b = 0; b < F::kBlocks; b++) {
                const int slot = tile * kTile + warp * F::kSlots + 16 * b;
                int live = tile < end ? n - slot : 0;         // rows of the block
                const bool ok = a.pg.in_pool(ids[b]);
                if (live > 0 && !ok) bad = true, live = 0;
                const size_t row = live > 0 ? a.pg.row(ids[b], h, slot) : 0;
                if (keys) {
                    const uint8_t *p = a.pg.K + (row + g) * kBytes + c * 16;
#pragma unroll
                    for (int r = 0; r < 2; r++) {
                        const bool on = g + 8 * r < live;
#pragma unroll
                        for (int j = 0; j < 4 / F::kBlocks; j++)
                            f.k[(b * 2 + r) * (4 / F::kBlocks) + j] =
                                on ? ldg16(p + r * 8 * kBytes + j * 64) : make_uint4(0, 0, 0, 0);
                        if (kE4m3) {
                            f.ks[b * 2 + r] = on ? a.pg.ks[row + g + 8 * r] : 0.f;
                            f.vs[b * 2 + r] = on ? a.pg.vs[row + g + 8 * r] : 0.f;
                        }
                    }
                } else {
                    const uint8_t *p = a.pg.V + (row + 2 * c) * kBytes + g * 16;
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        const int r = (i & 1) + 8 * (i >> 1);
                        const bool on = 2 * c + r < live;
#pragma unroll
                        for (int j = 0; j < 2 / F::kBlocks; j++)
                            f.v[(b * 4 + i) * (2 / F::kBlocks) + j] =
                                on ? ldg16(p + r * kBytes + j * 128) : make_uint4(0, 0, 0, 0);
                    }
                }
            }
        };

        look_up(first);
        load(first, true);
        load(first, false);
        look_up(first + 1);
        if (has_new && warp == 0) {
            // the new token's row: to its page, and to shared memory for the turn behind the last
            const int page = a.pg.entry(s, n);
            const bool ok = a.pg.in_pool(page);
            bad |= !ok;
            const size_t row = ok ? a.pg.row(page, h, n) : 0;
#pragma unroll
            for (int i = 0; i < 2; i++) {
                const uint2 w = *reinterpret_cast<const uint2 *>((i ? a.v_new : a.k_new) + (size_t)u * kD + lane * 4);
                uint8_t *pool = i ? a.pg.V : a.pg.K;
                if (kE4m3) {
                    uint32_t top = __vmaxu2(magnitudes(w.x), magnitudes(w.y));
#pragma unroll
                    for (int j = 16; j; j >>= 1) top = __vmaxu2(top, __shfl_xor_sync(kFull, top, j));
                    const float scale = row_scale(__uint_as_float(max(top << 16, top & 0xffff0000u)));
                    const uint32_t v = quantise4(w.x, w.y, __fdiv_rn(1.f, scale));
                    reinterpret_cast<uint32_t *>(sm.row[i])[lane] = v;
                    if (lane == 0) sm.row_scale[i] = scale;
                    if (ok) {
                        *reinterpret_cast<uint32_t *>(pool + row * kBytes + lane * 4) = v;
                        if (lane == 0) (i ? a.pg.vs : a.pg.ks)[row] = scale;
                    }
                } else {
                    reinterpret_cast<uint2 *>(sm.row[i])[lane] = w;
                    if (ok) *reinterpret_cast<uint2 *>(pool + row * kBytes + lane * 8) = w;
                }
            }
            __syncwarp();
        }

        for (int tile = first; tile < mine_end; tile++) {
            const bool extra = tile == end;
            int live = extra ? 1 : n - (tile * kTile + warp * F::kSlots);
            if (extra) {
                // the new token alone: row 0 of the block
                const uint4 none = make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int j = 0; j < 8; j++) f.k[j] = f.v[j] = none;
                if (g == 0)
#pragma unroll
                    for (int j = 0; j < 4 / F::kBlocks; j++) f.k[j] = lds_v4(sm.row[0] + c * 16 + j * 64);
                if (c == 0)
#pragma unroll
                    for (int j = 0; j < 2 / F::kBlocks; j++) f.v[j] = lds_v4(sm.row[1] + g * 16 + j * 128);
                f.ks[0] = sm.row_scale[0], f.vs[0] = sm.row_scale[1];
            }
            // S' = K Q'
            float x[F::kBlocks][4];
#pragma unroll
            for (int b = 0; b < F::kBlocks; b++) {
                float y[4] = {};
                x[b][0] = x[b][1] = x[b][2] = x[b][3] = 0.f;
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    float *to = i & 1 ? y : x[b];
                    if (kE4m3) {
                        const uint32_t r0 = word(f.k[b * 4 + (i >> 2)], i & 3);
                        const uint32_t r1 = word(f.k[b * 4 + 2 + (i >> 2)], i & 3);
                        mma<true>(to, e4m3_to_f16x2(r0), e4m3_to_f16x2(r1), e4m3_to_f16x2(r0 >> 16),
                                  e4m3_to_f16x2(r1 >> 16), q[i][0], q[i][1]);
                    } else {
                        const uint4 &r0 = f.k[i >> 1], &r1 = f.k[4 + (i >> 1)];
                        mma<false>(to, word(r0, 2 * (i & 1)), word(r1, 2 * (i & 1)), word(r0, 2 * (i & 1) + 1),
                                   word(r1, 2 * (i & 1) + 1), q[i][0], q[i][1]);
                    }
                }
#pragma unroll
                for (int j = 0; j < 4; j++) x[b][j] += y[j];
            }
            // logits in base 2, what is not there at -inf; the reference's candidates
            float top0 = -INFINITY, top1 = -INFINITY, vs[4];
#pragma unroll
            for (int b = 0; b < F::kBlocks; b++)
#pragma unroll
                for (int r = 0; r < 2; r++) {
                    const bool on = 16 * b + 8 * r + g < live;
                    float c0 = ch0, c1 = ch1, up = 0.f;
                    if (kE4m3) {
                        c0 *= f.ks[b * 2 + r], c1 *= f.ks[b * 2 + r];
                        vs[b * 2 + r] = on ? f.vs[b * 2 + r] : 0.f;
                        up = scale_log2(f.vs[b * 2 + r]);
                    }
                    x[b][2 * r] = on ? x[b][2 * r] * c0 : -INFINITY;
                    x[b][2 * r + 1] = on ? x[b][2 * r + 1] * c1 : -INFINITY;
                    top0 = fmaxf(top0, x[b][2 * r] + up);
                    top1 = fmaxf(top1, x[b][2 * r + 1] + up);
                }
            if (!extra) {
                if (tile + 1 < end) load(tile + 1, true);
            }
            if (__any_sync(kFull, top0 > m0 + kSlack || top1 > m1 + kSlack)) {
#pragma unroll
                for (int i = 4; i < 32; i <<= 1) {
                    top0 = fmaxf(top0, __shfl_xor_sync(kFull, top0, i));
                    top1 = fmaxf(top1, __shfl_xor_sync(kFull, top1, i));
                }
                const float n0 = fmaxf(m0, top0), n1 = fmaxf(m1, top1);
                const float r0 = m0 == n0 ? 1.f : exp2f(m0 - n0), r1 = m1 == n1 ? 1.f : exp2f(m1 - n1);
                m0 = n0, m1 = n1;
                l0 *= r0, l1 *= r1;
#pragma unroll
                for (int i = 0; i < 8; i++) acc[i][0] *= r0, acc[i][1] *= r1, acc[i][2] *= r0, acc[i][3] *= r1;
            }
            const float ref0 = m0 == -INFINITY ? 0.f : m0, ref1 = m1 == -INFINITY ? 0.f : m1;
            // weights, O' += V' P'
#pragma unroll
            for (int b = 0; b < F::kBlocks; b++) {
                float p[4];
#pragma unroll
                for (int j = 0; j < 4; j++) p[j] = exp2f(x[b][j] - (j & 1 ? ref1 : ref0));
                l0 += p[0] + p[2];
                l1 += p[1] + p[3];
                if (kE4m3) {
                    p[0] *= vs[b * 2], p[1] *= vs[b * 2];
                    p[2] *= vs[b * 2 + 1], p[3] *= vs[b * 2 + 1];
                }
                uint32_t hi0, lo0, hi1, lo1;
                two_terms<kE4m3>(p[0], p[1], hi0, lo0);
                two_terms<kE4m3>(p[2], p[3], hi1, lo1);
                hi0 = transpose8x8(hi0), hi1 = transpose8x8(hi1);
                lo0 = transpose8x8(lo0), lo1 = transpose8x8(lo1);
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    uint32_t a0, a1, a2, a3;
                    if (kE4m3) {
                        // bytes of two slots side by side, the lane's dimensions 16 g + 2 i, + 1
                        const uint32_t sel = i & 1 ? 0x7362 : 0x5140;
                        const uint32_t w0 = __byte_perm(word(f.v[b * 4], i >> 1), word(f.v[b * 4 + 1], i >> 1), sel);
                        const uint32_t w1 =
                            __byte_perm(word(f.v[b * 4 + 2], i >> 1), word(f.v[b * 4 + 3], i >> 1), sel);
                        a0 = e4m3_to_f16x2(w0), a1 = e4m3_to_f16x2(w0 >> 16);
                        a2 = e4m3_to_f16x2(w1), a3 = e4m3_to_f16x2(w1 >> 16);
                    } else {
                        // the lane's dimensions 8 g + 2 i, + 1 (and 64 on from the fourth)
                        const int j = i >> 2, w = i & 3;
                        a0 = __byte_perm(word(f.v[j], w), word(f.v[2 + j], w), 0x5410);
                        a1 = __byte_perm(word(f.v[j], w), word(f.v[2 + j], w), 0x7632);
                        a2 = __byte_perm(word(f.v[4 + j], w), word(f.v[6 + j], w), 0x5410);
                        a3 = __byte_perm(word(f.v[4 + j], w), word(f.v[6 + j], w), 0x7632);
                    }
                    mma<kE4m3>(acc[i], a0, a1, a2, a3, hi0, hi1);
                    mma<kE4m3>(acc[i], a0, a1, a2, a3, lo0, lo1);
                }
            }
            if (tile + 1 < end) {
                load(tile + 1, false);
                look_up(tile + 2);
            }
        }

        // the warps' sums meet in shared memory
#pragma unroll
        for (int i = 4; i < 32; i <<= 1) {
            l0 += __shfl_xor_sync(kFull, l0, i);
            l1 += __shfl_xor_sync(kFull, l1, i);
        }
        if (g == 0) {
            sm.m[warp][2 * c] = m0, sm.m[warp][2 * c + 1] = m1;
            sm.l[warp][2 * c] = l0, sm.l[warp][2 * c + 1] = l1;
        }
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const int d = kE4m3 ? 16 * g + 2 * i : 8 * g + 2 * (i & 3) + 64 * (i >> 2);
            *reinterpret_cast<float2 *>(&sm.o[warp][2 * c * kPad + d]) = make_float2(acc[i][0], acc[i][2]);
            *reinterpret_cast<float2 *>(&sm.o[warp][(2 * c + 1) * kPad + d]) = make_float2(acc[i][1], acc[i][3]);
        }
        const bool any_bad = __syncthreads_or(bad);

        // thread: head hh, eight dimensions
        const int hh = tid >> 4, d = (tid & 15) * 8;
        float M = -INFINITY, L = 0.f, O[8] = {};
#pragma unroll
        for (int w = 0; w < kWarps; w++) M = fmaxf(M, sm.m[w][hh]);
#pragma unroll
        for (int w = 0; w < kWarps; w++) {
            const float r = sm.m[w][hh] == -INFINITY ? 0.f : exp2f(sm.m[w][hh] - M);   // 0 keeps a NaN
            L = fmaf(r, sm.l[w][hh], L);
#pragma unroll
            for (int i = 0; i < 8; i++) O[i] = fmaf(r, sm.o[w][hh * kPad + d + i], O[i]);
        }
        auto write = [&]() {
            if (hh >= G) return;
            const float inv = M == -INFINITY && L == 0.f ? 0.f : 1.f / L;
            const size_t to = (size_t)u * G + hh;
            *reinterpret_cast<uint4 *>(a.o + to * kD + d) =
                make_uint4(to_bf16x2(O[0] * inv, O[1] * inv), to_bf16x2(O[2] * inv, O[3] * inv),
                           to_bf16x2(O[4] * inv, O[5] * inv), to_bf16x2(O[6] * inv, O[7] * inv));
            if (d == 0) a.lse[to] = (M + log2f(L)) * 0.6931471805599453f;
        };
        const int from = cuts.part(unit_at), upto = cuts.part(unit_at + tiles - 1);
        if (from == upto) {
            if (!any_bad) write();
            else if (tid == 0) record_status(a.status, KVC_ERR_INVALID_ARG);
        } else {
            // a part of the unit; the last to come joins them all
            const int slot = 2 * blockIdx.x + (first == 0);
            if (hh < G) {
                float *to = a.part_o + ((size_t)slot * G + hh) * kD + d;
                *reinterpret_cast<float4 *>(to) = make_float4(O[0], O[1], O[2], O[3]);
                *reinterpret_cast<float4 *>(to + 4) = make_float4(O[4], O[5], O[6], O[7]);
                if (d == 0) *reinterpret_cast<float2 *>(a.part_ml + ((size_t)slot * G + hh) * 2) = make_float2(M, L);
            }
            if (tid == 0) a.part_bad[slot] = any_bad;
            __threadfence();
            __syncthreads();
            if (tid == 0) sm.last = atomicAdd(a.arrived + u, 1) == upto - from;
            __syncthreads();
            if (sm.last) {
                __threadfence();
                bool wrong = false;
                M = -INFINITY, L = 0.f;
#pragma unroll
                for (int i = 0; i < 8; i++) O[i] = 0.f;
                for (int p = from; p <= upto; p++) wrong |= __ldcg(a.part_bad + 2 * p + (p == from)) != 0;
                if (hh < G) {
                    for (int p = from; p <= upto; p++)
                        M = fmaxf(M, __ldcg(a.part_ml + ((size_t)(2 * p + (p == from)) * G + hh) * 2));
#pragma unroll 4
                    for (int p = from; p <= upto; p++) {
                        const size_t at = (size_t)(2 * p + (p == from)) * G + hh;
                        const float2 ml = __ldcg(reinterpret_cast<const float2 *>(a.part_ml + at * 2));
                        const float r = ml.x == -INFINITY ? 0.f : exp2f(ml.x - M);
                        const float4 x = __ldcg(reinterpret_cast<const float4 *>(a.part_o + at * kD + d));
                        const float4 y = __ldcg(reinterpret_cast<const float4 *>(a.part_o + at * kD + d + 4));
                        L = fmaf(r, ml.y, L);
                        O[0] = fmaf(r, x.x, O[0]), O[1] = fmaf(r, x.y, O[1]);
                        O[2] = fmaf(r, x.z, O[2]), O[3] = fmaf(r, x.w, O[3]);
                        O[4] = fmaf(r, y.x, O[4]), O[5] = fmaf(r, y.y, O[5]);
                        O[6] = fmaf(r, y.z, O[6]), O[7] = fmaf(r, y.w, O[7]);
                    }
                }
                if (!wrong) write();
                if (tid == 0) {
                    if (wrong) record_status(a.status, KVC_ERR_INVALID_ARG);
                    a.arrived[u] = 0;            // for the next call
                }
            }
        }
        __syncthreads();

        // the next unit
        t = unit_at + end;
        if (t < t_end) {
            unit_at += tiles;
            if (++h == heads) {
                h = 0;
                do tiles = tiles_of(++s);
                while (tiles == 0);
            }
        }
    }
}

}  // namespace

size_t page_ws_bytes(const kvc_pages &pg, int G)
{
    return kAlign + align_up((size_t)pg.U * 4) + align_up(2 * kGrid * 4) +
           align_up((size_t)2 * kGrid * G * 2 * 4) + align_up((size_t)2 * kGrid * G * kD * 4);
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
    a.arrived = reinterpret_cast<int32_t *>(at);
    at += align_up((size_t)pg.U * 4);
    a.part_bad = reinterpret_cast<int32_t *>(at);
    at += align_up(2 * kGrid * 4);
    a.part_ml = reinterpret_cast<float *>(at);
    at += align_up((size_t)2 * kGrid * G * 2 * 4);
    a.part_o = reinterpret_cast<float *>(at);
    a.S = pg.U / pg.heads;
    a.G = G;
    a.max_len = max_len;
    // no more CTAs than there can be tiles
    const int tile = kWarps * (pg.type == KVC_PAGE_E4M3 ? 32 : 16);
    const int64_t tiles = (int64_t)pg.U * ((max_len + tile - 1) / tile);
    const dim3 grid((unsigned)(tiles < kGrid ? tiles : kGrid));
    return pg.type == KVC_PAGE_E4M3 ? launch_following(attend_kernel<true>, grid, kThreads, 0, st, a)
                                    : launch_following(attend_kernel<false>, grid, kThreads, 0, st, a);
}

}  // namespace kvc

// kvc_page_attend.cu -- one new token appended to a cache in pages and attended
// over it (kvc_page_attend): a CTA per unit, a warp per slot.
#include "kvc_page.h"

#include <math.h>

namespace kvc {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

struct AttendArgs {
    PageArgs pg;
    const uint16_t *q, *k_new, *v_new;
    uint16_t *o;
    float *lse;
    int32_t *status;
    int max_len;
};

// the lane's four values of a row
template <bool kE4m3>
__device__ __forceinline__ void load4(const uint8_t *pool, const float *scales, size_t row, int lane,
                                      float *f)
{
    if (kE4m3) {
        const uint32_t w = *reinterpret_cast<const uint32_t *>(pool + row * kD + lane * 4);
        const float s = scales[row];
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const uint32_t h = e4m3_to_f16x2(w >> (16 * i));
            const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&h));
            f[2 * i] = x.x * s;
            f[2 * i + 1] = x.y * s;
        }
    } else {
        const uint2 w = *reinterpret_cast<const uint2 *>(pool + (row * kD + lane * 4) * 2);
        f[0] = bf_lo(w.x), f[1] = bf_hi(w.x), f[2] = bf_lo(w.y), f[3] = bf_hi(w.y);
    }
}

template <bool kE4m3>
__device__ __forceinline__ void append4(uint8_t *pool, float *scales, size_t row, int lane,
                                        const uint16_t *x)
{
    const uint2 w = *reinterpret_cast<const uint2 *>(x + lane * 4);
    if (!kE4m3) {
        *reinterpret_cast<uint2 *>(pool + (row * kD + lane * 4) * 2) = w;
        return;
    }
    float f[4] = {bf_lo(w.x), bf_hi(w.x), bf_lo(w.y), bf_hi(w.y)}, amax = 0.f;
#pragma unroll
    for (int i = 0; i < 4; i++) amax = max_nan(amax, fabsf(f[i]));
#pragma unroll
    for (int m = 16; m; m >>= 1) amax = max_nan(amax, __shfl_xor_sync(kFull, amax, m));
    const float scale = row_scale(amax), inv = __fdiv_rn(1.f, scale);
    *reinterpret_cast<uint32_t *>(pool + row * kD + lane * 4) =
        to_e4m3(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv);
    if (lane == 0) scales[row] = scale;
}

template <bool kE4m3, int G>
__global__ void __launch_bounds__(kThreads) attend_kernel(const __grid_constant__ AttendArgs a)
{
    __shared__ float ms[kWarps][G], ls[kWarps][G], acc[kWarps][G][kD];
    __shared__ int bad;
    follow();
    lead();
    const int u = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int s = a.pg.by_heads(u), h = u - s * a.pg.heads;
    int n = a.pg.len[s];
    const int total = n + (a.k_new != nullptr);
    if (n < 0 || total > a.max_len) {
        if (threadIdx.x == 0) record_status(a.status, KVC_ERR_SHAPE);
        return;
    }
    if (threadIdx.x == 0) bad = 0;
    __syncthreads();
    if (total > n && warp < 2) {
        const int page = a.pg.entry(s, n);
        if (a.pg.in_pool(page)) {
            const size_t row = a.pg.row(page, h, n);
            if (warp == 0) append4<kE4m3>(a.pg.K, a.pg.ks, row, lane, a.k_new + (size_t)u * kD);
            if (warp == 1) append4<kE4m3>(a.pg.V, a.pg.vs, row, lane, a.v_new + (size_t)u * kD);
        }
    }
    __syncthreads();
    float q[G][4], m[G], l[G], f[G][4];
#pragma unroll
    for (int g = 0; g < G; g++) {
        const uint2 w = *reinterpret_cast<const uint2 *>(a.q + ((size_t)u * G + g) * kD + lane * 4);
        q[g][0] = bf_lo(w.x), q[g][1] = bf_hi(w.x), q[g][2] = bf_lo(w.y), q[g][3] = bf_hi(w.y);
        m[g] = -INFINITY, l[g] = 0.f;
        f[g][0] = f[g][1] = f[g][2] = f[g][3] = 0.f;
    }
    const float scale = 0.08838834764831845f;    // 1 / sqrt(128)
    for (int i = warp; i < total; i += kWarps) {
        const int page = a.pg.entry(s, i);
        if (!a.pg.in_pool(page)) {
            bad = 1;
            break;
        }
        const size_t row = a.pg.row(page, h, i);
        float k[4], v[4];
        load4<kE4m3>(a.pg.K, a.pg.ks, row, lane, k);
        load4<kE4m3>(a.pg.V, a.pg.vs, row, lane, v);
#pragma unroll
        for (int g = 0; g < G; g++) {
            const float x = warp_sum(q[g][0] * k[0] + q[g][1] * k[1] + q[g][2] * k[2] + q[g][3] * k[3]) * scale;
            const float top = fmaxf(m[g], x), was = m[g] == top ? 1.f : expf(m[g] - top), p = expf(x - top);
            m[g] = top;
            l[g] = l[g] * was + p;
#pragma unroll
            for (int e = 0; e < 4; e++) f[g][e] = f[g][e] * was + p * v[e];
        }
    }
#pragma unroll
    for (int g = 0; g < G; g++) {
        if (lane == 0) ms[warp][g] = m[g], ls[warp][g] = l[g];
#pragma unroll
        for (int e = 0; e < 4; e++) acc[warp][g][lane * 4 + e] = f[g][e];
    }
    __syncthreads();
    if (bad) {
        if (threadIdx.x == 0) record_status(a.status, KVC_ERR_INVALID_ARG);
        return;
    }
    for (int i = threadIdx.x; i < G * kD; i += kThreads) {
        const int g = i / kD, e = i % kD;
        float top = -INFINITY, sum = 0.f, x = 0.f;
        for (int w = 0; w < kWarps; w++) top = fmaxf(top, ms[w][g]);
        for (int w = 0; w < kWarps; w++) {
            if (ms[w][g] == -INFINITY && !(ls[w][g] != 0.f)) continue;    // a warp without slots
            const float c = expf(ms[w][g] - top);
            sum += c * ls[w][g];
            x += c * acc[w][g][e];
        }
        const size_t to = (size_t)u * G + g;
        a.o[to * kD + e] = __bfloat16_as_ushort(__float2bfloat16_rn(total ? x / sum : 0.f));
        if (e == 0) a.lse[to] = total ? top + logf(sum) : -INFINITY;
    }
}

template <bool kE4m3>
cudaError_t launch(const AttendArgs &a, int U, int G, cudaStream_t st)
{
    switch (G) {
        case 1: return launch_following(attend_kernel<kE4m3, 1>, dim3(U), kThreads, 0, st, a);
        case 2: return launch_following(attend_kernel<kE4m3, 2>, dim3(U), kThreads, 0, st, a);
        case 4: return launch_following(attend_kernel<kE4m3, 4>, dim3(U), kThreads, 0, st, a);
        default: return launch_following(attend_kernel<kE4m3, 8>, dim3(U), kThreads, 0, st, a);
    }
}

}  // namespace

size_t page_ws_bytes(const kvc_pages &pg, int G) { return kAlign; }

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
    a.status = &static_cast<WsHeader *>(ws)->status;
    a.max_len = max_len;
    return pg.type == KVC_PAGE_E4M3 ? launch<true>(a, pg.U, G, st) : launch<false>(a, pg.U, G, st);
}

}  // namespace kvc

// kvc_page.h -- shared by the calls over a cache in pages (kvc_page_write,
// kvc_page_read, kvc_page_attend) and the norms and rotation in front of it
// (kvc_qk_norm_rope): device views, addressing and launchers.
#pragma once

#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "kvc_common.cuh"
#include "kvc_internal.h"
#include "kvc_tree.h"

namespace kvc {

constexpr float kE4m3Max = 448.f;
constexpr float kLeastScale = 1.17549435e-38f;   // 2^-126: the reciprocal stays finite

// Device view of the pages.
struct PageArgs {
    uint8_t *K, *V;
    float *ks, *vs;
    const int32_t *table, *len;
    int heads, shift, n_pages, stride;           // shift: log2 of the slots per page
    FastDiv by_heads;

    __device__ __forceinline__ int entry(int s, int slot) const
    {
        return table[(size_t)s * stride + (slot >> shift)];
    }
    __device__ __forceinline__ bool in_pool(int page) const { return (uint32_t)page < (uint32_t)n_pages; }
    // row of the pool (K, V rows; scales) that holds the slot of head h, 64-bit: a long
    // cache passes 2^31 rows
    __device__ __forceinline__ size_t row(int page, int h, int slot) const
    {
        return (((size_t)page * heads + h) << shift) + (slot & ((1 << shift) - 1));
    }
};

PageArgs page_args(const kvc_pages &pg);

// Magnitudes of two bf16, which order as whole numbers; a NaN is above infinity.
__device__ __forceinline__ uint32_t magnitudes(uint32_t w) { return w & 0x7fff7fffu; }

// The scale of a row from its largest magnitude, and what its values are multiplied by.
__device__ __forceinline__ float row_scale(float amax)
{
    const float s = __fdiv_rn(amax, kE4m3Max);
    return s < kLeastScale ? kLeastScale : s;    // a NaN stays
}

// four e4m3 values, nearest even, at most 448
__device__ __forceinline__ uint32_t to_e4m3(float a, float b, float c, float d)
{
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
}

// two e4m3 values in the low half of w as two f16 (exact)
__device__ __forceinline__ uint32_t e4m3_to_f16x2(uint32_t w)
{
    uint32_t r;
    asm("{\n .reg .b16 h;\n cvt.u16.u32 h, %1;\n cvt.rn.f16x2.e4m3x2 %0, h;\n}\n" : "=r"(r) : "r"(w));
    return r;
}

// {lo, hi} rounded to bf16, lo in the low half
__device__ __forceinline__ uint32_t to_bf16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// packed fp32 pairs: one instruction for two
__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 z)
{
    float2 r;
    asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
        " fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}\n"
        : "=f"(r.x), "=f"(r.y)
        : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y), "f"(z.x), "f"(z.y));
    return r;
}

__device__ __forceinline__ float2 mul2(float2 x, float2 y)
{
    float2 r;
    asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mul.rn.f32x2 d, a, b;\n"
        " mov.b64 {%0, %1}, d;\n}\n"
        : "=f"(r.x), "=f"(r.y)
        : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
    return r;
}

// two bf16 times f
__device__ __forceinline__ float2 scaled2(uint32_t w, float f)
{
    return mul2(make_float2(bf_lo(w), bf_hi(w)), make_float2(f, f));
}

// four bf16 times inv as e4m3
__device__ __forceinline__ uint32_t quantise4(uint32_t w0, uint32_t w1, float inv)
{
    const float2 a = scaled2(w0, inv), b = scaled2(w1, inv);
    return to_e4m3(a.x, a.y, b.x, b.y);
}

size_t page_ws_bytes(const kvc_pages &pg, int G);

cudaError_t launch_qk_norm_rope(const kvc_rope &r, int B, int T, const uint16_t *qkv, int64_t row_stride,
                                const int32_t *pos, const int32_t *n, uint16_t *q, uint16_t *k,
                                uint16_t *v, cudaStream_t st);
cudaError_t launch_page_write(const kvc_pages &pg, int T, const int32_t *first, const int32_t *count,
                              const uint16_t *k, const uint16_t *v, void *ws, cudaStream_t st);
cudaError_t launch_page_read(const kvc_pages &pg, int M, int ld, const int32_t *slots,
                             const int32_t *count, uint16_t *k_out, uint16_t *v_out, void *ws,
                             cudaStream_t st);
cudaError_t launch_page_attend(const kvc_pages &pg, int G, int max_len, const uint16_t *q,
                               const uint16_t *k_new, const uint16_t *v_new, uint16_t *o, float *lse,
                               void *ws, cudaStream_t st);

}  // namespace kvc

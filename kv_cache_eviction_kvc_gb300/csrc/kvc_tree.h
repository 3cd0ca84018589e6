// kvc_tree.h -- shared by the drafted-token entry points (kvc_tree_attend,
// kvc_tree_weights, kvc_tree_commit): device-side checks, workspace carve-up
// and launchers.
#pragma once

#include <cuda_runtime.h>

#include "kvc_common.cuh"
#include "kvc_internal.h"
#include "kvc_tma.cuh"
#include "kvc_umma.cuh"

namespace kvc {

constexpr int kTreeMax = 64;          // drafted tokens per tree (one mask word)

// Device views of a tree and of an accepted path.
struct TreeArgs {
    const uint64_t *mask;             // [trees][T]
    const int32_t *n;                 // [trees] or NULL
    int T, units;
};

struct PathArgs {
    const int32_t *token, *n, *pos;   // [trees][A], [trees], [trees]
    int A;
};

// x / d for 0 <= x < 2^31 as a multiplication (Granlund and Montgomery, 1994)
struct FastDiv {
    uint32_t mul, shift;
    FastDiv(uint32_t d = 1)
    {
        shift = 0;
        while ((1u << shift) < d) shift++;               // d <= 2^31
        mul = (uint32_t)(((1ull << 32) * ((1ull << shift) - d)) / d + 1);
    }
    __device__ __forceinline__ int operator()(int x) const
    {
        return (int)((__umulhi((uint32_t)x, mul) + (uint32_t)x) >> shift);
    }
};

// The line of `total` tiles is cut into min(grid, total) parts, the first
// total % parts of them one tile longer.
struct LineCuts {
    int parts, q, rem;
    __device__ __forceinline__ LineCuts(int grid, int total)
        : parts(min(grid, total)), q(parts ? (uint32_t)total / (uint32_t)parts : 0), rem(total - q * parts)
    {
    }
    __device__ __forceinline__ int start(int c) const { return c * q + min(c, rem); }
    __device__ __forceinline__ int part(int tile) const        // that has the tile
    {
        const int longer = rem * (q + 1);
        return tile < longer ? (uint32_t)tile / (uint32_t)(q + 1)
                             : rem + (int)((uint32_t)(tile - longer) / (uint32_t)q);
    }
};

// True on one lane of a converged warp; the compiler keeps what the branch
// issues (descriptors and all) in uniform registers.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
    return p != 0;
}

// Bounded wait.  Once one has run out every wait ends at once and each role
// leaves its loop (all synchronisation among them is by such waits).
__device__ __forceinline__ bool tree_wait(uint64_t *b, uint32_t parity, volatile int *bad)
{
    if (mbar_try_wait(b, parity)) return true;
    const long long t0 = clock64();
    while (!mbar_try_wait(b, parity)) {
        if (*bad) return false;
        if (clock64() - t0 > kWaitCycles) {
            *bad = 1;
            return false;
        }
    }
    return true;
}

__device__ __forceinline__ void tmem_ld16_async(uint32_t addr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
        "%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(addr)
        : "memory");
}

__device__ __forceinline__ void tmem_bind16(uint32_t (&r)[16])
{
    asm volatile(""
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                   "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]),
                   "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
}

// 3D copies of a box of 64 columns x 64 rows of one unit.
__device__ __forceinline__ void tma_3d(void *dst, const CUtensorMap *map, int x, int y, int z,
                                       uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void tma_3d_hint(void *dst, const CUtensorMap *map, int x, int y, int z,
                                            uint64_t *bar, uint64_t policy)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}

// [units][rows][128] fp32, boxes of 32 columns x box_rows rows of a unit with
// the 128-byte swizzle.
inline bool make_f32_map(CUtensorMap *m, const void *base, uint64_t units, uint64_t rows, int box_rows)
{
    const cuuint64_t dims[3] = {(cuuint64_t)kD, (cuuint64_t)rows, (cuuint64_t)units};
    const cuuint64_t strides[2] = {(cuuint64_t)(kD * 4), (cuuint64_t)(rows * kD * 4)};
    const cuuint32_t box[3] = {32u, (cuuint32_t)box_rows, 1u};
    return encode_map(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, base, dims, strides, box);
}

// [units][rows][128] bf16, boxes of 64 columns x 64 rows of a unit with the
// 128-byte swizzle; rows past a unit's last read as zero.  A unit index and a
// row index fit 32 bits where their product does not.
inline bool make_unit_map(CUtensorMap *m, const void *base, uint64_t units, uint64_t rows)
{
    const cuuint64_t dims[3] = {(cuuint64_t)kD, (cuuint64_t)rows, (cuuint64_t)units};
    const cuuint64_t strides[2] = {(cuuint64_t)(kD * 2), (cuuint64_t)(rows * kD * 2)};
    const cuuint32_t box[3] = {64u, 64u, 1u};
    return encode_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, strides, box);
}

// Programmatic dependent launch: a kernel's launch and set-up overlap the end of
// the one before it in the stream (1 to 2.5 us of every call), and it calls
// follow() before it reads or writes anything of that one.  Every CTA calls it
// (or ends), so that a kernel that is done has all before it done too.  lead()
// comes after follow(): a kernel behind that one may read what both only read
// without waiting.  Where the next kernel's CTAs are small, lead() comes late:
// they would crowd on the SMs that are free first.
__device__ __forceinline__ void follow() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// In the kernel before: the next may be launched (it waits in follow()).
__device__ __forceinline__ void lead() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_following(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st,
                             const A &...args)
{
    cudaLaunchConfig_t c{};
    c.gridDim = grid;
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = smem;
    c.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    c.attrs = &at;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, kernel, P(args)...);
}

cudaError_t launch_tree_attend(const kvc_params &p, int max_len, const TreeArgs &t,
                               const uint16_t *q, const uint16_t *kt, const uint16_t *vt,
                               const kvc_cache &c, const kvc_moments *m, uint16_t *o, float *lse,
                               void *ws, cudaStream_t st);
cudaError_t launch_tree_weights(const kvc_params &p, int max_len, const TreeArgs &t,
                                const PathArgs &a, const float *row_weight, const uint16_t *q,
                                const uint16_t *kt, const float *lse, const kvc_cache &c, void *S,
                                bool wide, void *ws, cudaStream_t st);
cudaError_t launch_tree_commit(const kvc_params &p, int max_len, const TreeArgs &t,
                               const PathArgs &a, const uint16_t *kt, const uint16_t *vt,
                               const void *S, bool wide, const kvc_cache &c, const kvc_moments *m,
                               int kmax, int32_t *evict_idx, int32_t *evict_pos, int32_t *n_evict,
                               const DecodeWs &ws, cudaStream_t st);
// (S: fp64 when wide, else fp32)
size_t tree_ws_bytes(const kvc_params &p, int T);

}  // namespace kvc

// kvc_page_move.cu -- rows into a cache in pages (kvc_page_write: bf16, or e4m3
// with an fp32 scale per row) and out of it (kvc_page_read).
//
// Sixteen lanes hold a row: 16 bytes each of its bf16 form, 8 of its e4m3 form.
// The largest magnitude is four exchanges.  Both calls are bound by the bytes.
#include "kvc_page.h"

namespace kvc {
namespace {

constexpr int kThreads = 256;
constexpr int kTeams = kThreads / 16;

struct MoveArgs {
    PageArgs pg;
    const int32_t *first, *count, *slots;
    uint16_t *k, *v;                             // rows outside the pages
    int32_t *status;
    int rows, ld;                                // rows per unit, their stride
    FastDiv by_chunks;
    int chunks;
};

__device__ __forceinline__ unsigned team_mask() { return threadIdx.x & 16 ? 0xffff0000u : 0x0000ffffu; }

template <bool kE4m3>
__device__ __forceinline__ void store_row(uint8_t *pool, float *scales, size_t row, int lane, uint4 x)
{
    if (!kE4m3) {
        *reinterpret_cast<uint4 *>(pool + (row * kD + lane * 8) * 2) = x;
        return;
    }
    float f[8], amax = 0.f;
    unpack8(x, f);
#pragma unroll
    for (int i = 0; i < 8; i++) amax = max_nan(amax, fabsf(f[i]));
#pragma unroll
    for (int m = 8; m; m >>= 1) amax = max_nan(amax, __shfl_xor_sync(team_mask(), amax, m, 16));
    const float scale = row_scale(amax), inv = __fdiv_rn(1.f, scale);
#pragma unroll
    for (int i = 0; i < 8; i++) f[i] *= inv;
    *reinterpret_cast<uint2 *>(pool + row * kD + lane * 8) =
        make_uint2(to_e4m3(f[0], f[1], f[2], f[3]), to_e4m3(f[4], f[5], f[6], f[7]));
    if (lane == 0) scales[row] = scale;
}

template <bool kE4m3>
__device__ __forceinline__ uint4 load_row(const uint8_t *pool, const float *scales, size_t row, int lane)
{
    if (!kE4m3) return *reinterpret_cast<const uint4 *>(pool + (row * kD + lane * 8) * 2);
    const uint2 w = *reinterpret_cast<const uint2 *>(pool + row * kD + lane * 8);
    const float scale = scales[row];
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const uint32_t h = e4m3_to_f16x2((i < 2 ? w.x : w.y) >> (16 * (i & 1)));
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
        r[i] = to_bf16x2(f.x * scale, f.y * scale);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

template <bool kE4m3>
__global__ void __launch_bounds__(kThreads) write_kernel(const __grid_constant__ MoveArgs a)
{
    follow();
    lead();
    const int lane = threadIdx.x & 15, team = threadIdx.x >> 4;
    const int u = a.by_chunks(blockIdx.x), t = (blockIdx.x - u * a.chunks) * kTeams + team;
    const int s = a.pg.by_heads(u), h = u - s * a.pg.heads;
    const int count = a.count ? a.count[s] : a.rows, first = a.first ? a.first[s] : 0;
    if (count < 0 || count > a.rows || first < 0 ||
        (int64_t)first + count > ((int64_t)a.pg.stride << a.pg.shift)) {
        if (threadIdx.x == 0) record_status(a.status, KVC_ERR_SHAPE);
        return;
    }
    if (t >= count) return;
    const size_t from = ((size_t)u * a.ld + t) * kD + lane * 8;
    const uint4 k = *reinterpret_cast<const uint4 *>(a.k + from);
    const uint4 v = *reinterpret_cast<const uint4 *>(a.v + from);
    const int slot = first + t, page = a.pg.entry(s, slot);
    if (!a.pg.in_pool(page)) {
        if (lane == 0) record_status(a.status, KVC_ERR_INVALID_ARG);
        return;
    }
    const size_t row = a.pg.row(page, h, slot);
    store_row<kE4m3>(a.pg.K, a.pg.ks, row, lane, k);
    store_row<kE4m3>(a.pg.V, a.pg.vs, row, lane, v);
}

template <bool kE4m3>
__global__ void __launch_bounds__(kThreads) read_kernel(const __grid_constant__ MoveArgs a)
{
    follow();
    lead();
    const int lane = threadIdx.x & 15, team = threadIdx.x >> 4;
    const int u = a.by_chunks(blockIdx.x), i = (blockIdx.x - u * a.chunks) * kTeams + team;
    const int s = a.pg.by_heads(u), h = u - s * a.pg.heads;
    const int n = a.pg.len[s];
    const int count = a.count ? a.count[u] : a.slots ? a.rows : min(a.rows, max(n, 0));
    if (count < 0 || count > a.rows) {
        if (threadIdx.x == 0) record_status(a.status, KVC_ERR_SHAPE);
        return;
    }
    if (i >= count) return;
    const int slot = a.slots ? a.slots[(size_t)u * a.rows + i] : i;
    if (slot < 0 || slot >= n || (slot >> a.pg.shift) >= a.pg.stride) {
        if (lane == 0) record_status(a.status, KVC_ERR_SHAPE);
        return;
    }
    const int page = a.pg.entry(s, slot);
    if (!a.pg.in_pool(page)) {
        if (lane == 0) record_status(a.status, KVC_ERR_INVALID_ARG);
        return;
    }
    const size_t row = a.pg.row(page, h, slot), to = ((size_t)u * a.ld + i) * kD + lane * 8;
    *reinterpret_cast<uint4 *>(a.k + to) = load_row<kE4m3>(a.pg.K, a.pg.ks, row, lane);
    *reinterpret_cast<uint4 *>(a.v + to) = load_row<kE4m3>(a.pg.V, a.pg.vs, row, lane);
}

MoveArgs move_args(const kvc_pages &pg, int rows, int ld, const uint16_t *k, const uint16_t *v, void *ws)
{
    MoveArgs a{};
    a.pg = page_args(pg);
    a.k = const_cast<uint16_t *>(k);
    a.v = const_cast<uint16_t *>(v);
    a.status = &static_cast<WsHeader *>(ws)->status;
    a.rows = rows;
    a.ld = ld;
    a.chunks = (rows - 1) / kTeams + 1;
    a.by_chunks = FastDiv((uint32_t)a.chunks);
    return a;
}

}  // namespace

cudaError_t launch_page_write(const kvc_pages &pg, int T, const int32_t *first, const int32_t *count,
                              const uint16_t *k, const uint16_t *v, void *ws, cudaStream_t st)
{
    MoveArgs a = move_args(pg, T, T, k, v, ws);
    a.first = first;
    a.count = count;
    const dim3 grid(pg.U * a.chunks);
    return pg.type == KVC_PAGE_E4M3 ? launch_following(write_kernel<true>, grid, kThreads, 0, st, a)
                                    : launch_following(write_kernel<false>, grid, kThreads, 0, st, a);
}

cudaError_t launch_page_read(const kvc_pages &pg, int M, int ld, const int32_t *slots,
                             const int32_t *count, uint16_t *k_out, uint16_t *v_out, void *ws,
                             cudaStream_t st)
{
    MoveArgs a = move_args(pg, M, ld, k_out, v_out, ws);
    a.slots = slots;
    a.count = count;
    const dim3 grid(pg.U * a.chunks);
    return pg.type == KVC_PAGE_E4M3 ? launch_following(read_kernel<true>, grid, kThreads, 0, st, a)
                                    : launch_following(read_kernel<false>, grid, kThreads, 0, st, a);
}

}  // namespace kvc

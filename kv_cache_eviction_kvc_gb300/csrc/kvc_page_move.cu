// kvc_page_move.cu -- rows into a cache in pages (kvc_page_write: bf16, or e4m3
// with an fp32 scale per row) and out of it (kvc_page_read).
//
// Sixteen lanes hold a row: 16 bytes each of its bf16 form, 8 of its e4m3 form.
// Both calls are bound by the bytes (a slot read and written: 1024 in bf16, 776 to
// or from e4m3) once there are rows enough; before that by a chain of loads (count,
// slot, table, row, each waiting for the one before), of which a team has two rows
// in flight.
//
// Written in e4m3 the arithmetic is nearly as long as the bytes, so magnitudes are
// compared as 16-bit whole numbers, both rows' in one word (four exchanges for the
// two), and their quotients are formed once, side by side in the lanes.
//
// Measured: 8 units x 32768 rows to bf16 40.7 us (6.6 TB/s; 40.3 in a graph), to e4m3
// 33.2 (6.1); 8 x 131071 rows back 157 (6.8, what fits L2 among it) and 124 (6.5); 32
// units x <= 3277 listed rows of 32768 back 16.0 us (5.4) and from e4m3 14.1 (4.7 TB/s:
// the scale of a listed row brings 64 bytes from memory, 15 % more in all, and the
// chain of loads starts and ends it; loading the next rows' slots and pages ahead in
// longer-lived blocks took 14.5 to 16).  Rows in flight per team, the same
// three: one 35.2, 148, 18.6 us; two 33.6, 125, 14.1; three 33.3, 125, 14.2; four
// 35.7, 126, 14.6.
#include "kvc_page.h"

namespace kvc {
namespace {

constexpr int kThreads = 256;
constexpr int kTeams = kThreads / 16;
constexpr int kEach = 2, kRows = kTeams * kEach;   // rows of a team (in flight), of a block

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

__device__ __forceinline__ uint32_t largest(uint4 x)
{
    const uint32_t m = __vmaxu2(__vmaxu2(magnitudes(x.x), magnitudes(x.y)), __vmaxu2(magnitudes(x.z), magnitudes(x.w)));
    return __vmaxu2(m, m >> 16) & 0xffffu;
}

// A slot's key and value to row `row` of the pool.
template <bool kE4m3>
__device__ __forceinline__ void store_rows(const PageArgs &pg, size_t row, int lane, uint4 k, uint4 v)
{
    if (!kE4m3) {
        *reinterpret_cast<uint4 *>(pg.K + (row * kD + lane * 8) * 2) = k;
        *reinterpret_cast<uint4 *>(pg.V + (row * kD + lane * 8) * 2) = v;
        return;
    }
    // both rows' largest magnitudes in one word; even lanes have the key's quotients, odd
    // lanes the value's
    uint32_t top = largest(k) | largest(v) << 16;
#pragma unroll
    for (int m = 8; m; m >>= 1) top = __vmaxu2(top, __shfl_xor_sync(team_mask(), top, m, 16));
    const float scale = row_scale(__uint_as_float(lane & 1 ? top & 0xffff0000u : top << 16));
    const float inv = __fdiv_rn(1.f, scale);
    const float ki = __shfl_sync(team_mask(), inv, 0, 16), vi = __shfl_sync(team_mask(), inv, 1, 16);
    *reinterpret_cast<uint2 *>(pg.K + row * kD + lane * 8) =
        make_uint2(quantise4(k.x, k.y, ki), quantise4(k.z, k.w, ki));
    *reinterpret_cast<uint2 *>(pg.V + row * kD + lane * 8) =
        make_uint2(quantise4(v.x, v.y, vi), quantise4(v.z, v.w, vi));
    if (lane < 2) (lane ? pg.vs : pg.ks)[row] = scale;
}

// a row as it is held
template <bool kE4m3>
struct Held {
    uint4 w;                                     // e4m3: the first half
    float scale;

    __device__ __forceinline__ void load(const uint8_t *pool, const float *scales, size_t row, int lane)
    {
        if (kE4m3) {
            const uint2 x = *reinterpret_cast<const uint2 *>(pool + row * kD + lane * 8);
            w.x = x.x, w.y = x.y;
            scale = scales[row];
        } else {
            w = *reinterpret_cast<const uint4 *>(pool + (row * kD + lane * 8) * 2);
        }
    }
    __device__ __forceinline__ uint4 bf16() const
    {
        if (!kE4m3) return w;
        uint32_t r[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint32_t h = e4m3_to_f16x2((i < 2 ? w.x : w.y) >> (16 * (i & 1)));
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
            r[i] = to_bf16x2(f.x * scale, f.y * scale);
        }
        return make_uint4(r[0], r[1], r[2], r[3]);
    }
};

template <bool kE4m3>
__global__ void __launch_bounds__(kThreads) write_kernel(const __grid_constant__ MoveArgs a)
{
    follow();
    lead();
    const int lane = threadIdx.x & 15, team = threadIdx.x >> 4;
    const int u = a.by_chunks(blockIdx.x), t0 = (blockIdx.x - u * a.chunks) * kRows + team;
    const int s = a.pg.by_heads(u), h = u - s * a.pg.heads;
    const int count = a.count ? a.count[s] : a.rows, first = a.first ? a.first[s] : 0;
    uint4 k[kEach], v[kEach];
    int page[kEach];
    // a count that is refused below reads rows of the caller's arrays all the same
#pragma unroll
    for (int i = 0; i < kEach; i++) {
        const int t = t0 + i * kTeams;
        if (t >= min(count, a.rows)) break;
        const size_t from = ((size_t)u * a.ld + t) * kD + lane * 8;
        k[i] = *reinterpret_cast<const uint4 *>(a.k + from);
        v[i] = *reinterpret_cast<const uint4 *>(a.v + from);
    }
    if (count < 0 || count > a.rows || first < 0 ||
        (int64_t)first + count > ((int64_t)a.pg.stride << a.pg.shift)) {
        if (threadIdx.x == 0) record_status(a.status, KVC_ERR_SHAPE);
        return;
    }
#pragma unroll
    for (int i = 0; i < kEach; i++)
        if (t0 + i * kTeams < count) page[i] = a.pg.entry(s, first + t0 + i * kTeams);
#pragma unroll
    for (int i = 0; i < kEach; i++) {
        const int t = t0 + i * kTeams;
        if (t >= count) break;
        if (!a.pg.in_pool(page[i])) {
            if (lane == 0) record_status(a.status, KVC_ERR_INVALID_ARG);
            continue;
        }
        const size_t row = a.pg.row(page[i], h, first + t);
        store_rows<kE4m3>(a.pg, row, lane, k[i], v[i]);
    }
}

template <bool kE4m3>
__global__ void __launch_bounds__(kThreads) read_kernel(const __grid_constant__ MoveArgs a)
{
    follow();
    lead();
    const int lane = threadIdx.x & 15, team = threadIdx.x >> 4;
    const int u = a.by_chunks(blockIdx.x), i0 = (blockIdx.x - u * a.chunks) * kRows + team;
    const int s = a.pg.by_heads(u), h = u - s * a.pg.heads;
    int slot[kEach], page[kEach];
#pragma unroll
    for (int j = 0; j < kEach; j++) {
        const int i = i0 + j * kTeams;
        slot[j] = a.slots && i < a.rows ? a.slots[(size_t)u * a.rows + i] : i;
    }
    const int n = a.pg.len[s];
    const int count = a.count ? a.count[u] : a.slots ? a.rows : min(a.rows, max(n, 0));
    if (count < 0 || count > a.rows) {
        if (threadIdx.x == 0) record_status(a.status, KVC_ERR_SHAPE);
        return;
    }
#pragma unroll
    for (int j = 0; j < kEach; j++) {
        page[j] = -1;
        if (i0 + j * kTeams >= count) continue;
        if (slot[j] < 0 || slot[j] >= n || (slot[j] >> a.pg.shift) >= a.pg.stride) {
            if (lane == 0) record_status(a.status, KVC_ERR_SHAPE);
            continue;
        }
        page[j] = a.pg.entry(s, slot[j]);
        if (!a.pg.in_pool(page[j])) {
            if (lane == 0) record_status(a.status, KVC_ERR_INVALID_ARG);
            page[j] = -1;
        }
    }
    Held<kE4m3> k[kEach], v[kEach];
#pragma unroll
    for (int j = 0; j < kEach; j++) {
        if (page[j] < 0) continue;
        const size_t row = a.pg.row(page[j], h, slot[j]);
        k[j].load(a.pg.K, a.pg.ks, row, lane);
        v[j].load(a.pg.V, a.pg.vs, row, lane);
    }
#pragma unroll
    for (int j = 0; j < kEach; j++) {
        if (page[j] < 0) continue;
        const size_t to = ((size_t)u * a.ld + i0 + j * kTeams) * kD + lane * 8;
        *reinterpret_cast<uint4 *>(a.k + to) = k[j].bf16();
        *reinterpret_cast<uint4 *>(a.v + to) = v[j].bf16();
    }
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
    a.chunks = (rows - 1) / kRows + 1;
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

// kvc_tree_attend.cu -- attention of a tree of drafted tokens over the cache
// and the tree itself, with the normalization correction.
//
// The T G query rows of a unit share its keys and values, so a unit is one
// matrix product per tile of 128 slots each way: S = Q K^T (tcgen05, rows on
// the tensor-memory lanes), a softmax with a running maximum and sum (one
// thread per row), O += P V (P from tensor memory).  Up to 256 rows are bound
// by the 512 bytes per slot that stream from HBM (128 rows take 1024 tensor
// clocks per tile against about 2800 for its bytes at one SM's share of the
// bandwidth), so everything else is laid out to keep the loads going.
//
// Work split: the tiles of all (unit, block of 256 rows) items form one line
// that is cut into equal parts, one per CTA (a persistent CTA per SM).  An
// item inside one part is finished there; an item that a cut crosses leaves
// partial sums (maximum, sum, output) per part, which tree_join_kernel adds.
// With moments every item leaves its sums, and tree_moment_kernel mixes them
// with the evicted set's estimate.  The drafted tokens are the item's last
// tile.
//
// 576 threads:
//   warps 0-7, 8-15 two softmax groups, each with its own S, P and O in tensor
//                   memory.  Items of more than 128 rows give each group 128
//                   of them; otherwise the groups take alternate tiles of the
//                   same rows and add their sums at the end.  Two warps share
//                   32 rows: each has 64 of a tile's 128 slots, which halves
//                   the time from S to P that every tile waits for
//   warp 16         producer (TMA into a ring of 32 KB key and value tiles)
//   warp 17         tensor-memory owner and MMA issuer
// Tensor memory: O of group w at column 128 w, S at 256 + 128 w; P (bf16)
// overlays S, 32 columns at the start of each half.  The MMAs of one thread execute in the order
// of their issue, so the S that overwrites a P follows the product that reads
// it without a wait.
//
// What a row must not see: slots behind len and hidden drafted tokens are
// masked in S by selection (never by adding -inf to what may be NaN).  The
// value rows behind len are zeroed in shared memory up to the next multiple of
// 16 (the MMA reads 16 slots at a time).  Drafted tokens whose value is not
// finite are zeroed as well and added afterwards to the rows that see them.
// Every wait is bounded (~2 s); a wait that ran out records KVC_ERR_TIMEOUT.
#include "kvc_tree.h"
#include "kvc_umma.cuh"

#include <stddef.h>

namespace kvc {
namespace {

constexpr int kTile = 128;                       // slots per tile
constexpr int kRows = 256;                       // query rows per item
constexpr int kSlot = kTile * kD * 2;            // 32 KB: a tile of keys or values
constexpr int kHalf = kSlot / 2;                 // its 64-column half
constexpr int kRing = 5;
constexpr int kThreads = 576;
constexpr int kProd = 16, kMma = 17;
constexpr int kGrid = 152;                       // CTAs: one per SM
constexpr uint32_t kColS = 256;
constexpr float kLog2e = 1.4426950408889634f;
// the running maximum moves once a new one is above it by this much (in
// powers of two): weights stay below 2^8 and most tiles rescale nothing
constexpr float kSlack = 8.f;

constexpr uint32_t kIdescS = umma_idesc_bf16(128, 128);
constexpr uint32_t kIdescS64 = umma_idesc_bf16(128, 64);
constexpr uint32_t kIdescO = umma_idesc_bf16(128, 128) | (1u << 16);   // B (values) MN-major

struct AttArgs {
    TreeArgs t;
    const int32_t *votes, *len;
    const uint16_t *vt;
    uint16_t *o;
    float *lse;
    float *part;            // [items + CTAs][rows][128]
    float2 *ml;             // [items + CTAs][rows]
    int *first;             // [items + 1] tiles before each item
    int4 *cut;              // [CTAs] the item a part begins inside of: item, first and last part
    int32_t *status;
    int U, RB, TG, G, cap, max_len, rows, whole, join_all;
    float scale;            // log2(e) / sqrt(d)
};

struct AttSmem {
    union {                 // read as float4
        struct {
            float vote[kTile];               // votes of a tile's slots
            __nv_bfloat16 top[2][kTile];     // the halves' maxima
        };
        float2 ml[kTile];   // at an item's end: the rows' maxima and sums
    } g[2];
    int4 cut;
    uint64_t full[kRing], empty[kRing];
    uint64_t drain;
    uint64_t qfull[2], qempty[2], sfull[2], pready[2], pvdone[2];
    uint64_t odd[2];        // drafted tokens with a value that is not finite
    int scan[40];
    int start_item, start_base, total;
    int bad;
    uint32_t tmem;
};

// True on one lane of a converged warp; the compiler keeps what the branch
// issues (descriptors and all) in uniform registers.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
    return p != 0;
}

// Bounded wait.  Once one has run out every wait ends at once: each role then
// walks its loops to the end (so that the barriers among them stay matched)
// without issuing copies or MMAs.
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

// Everything is dynamic shared memory: the tiles fill all of it but 3 KB.
constexpr size_t kDyn = (size_t)(2 + kRing) * kSlot + sizeof(AttSmem);
static_assert(kDyn <= 227 * 1024, "one block's shared memory");
static_assert(offsetof(AttSmem, g) % 16 == 0 && offsetof(AttSmem, full) % 8 == 0, "alignment");

// Value operand: 128 slots of two 64-dimension boxes; leading byte offset
// between the boxes, stride byte offset between 8-slot groups, version 1,
// 128-byte swizzle.
__device__ __forceinline__ uint64_t v_desc(uint32_t saddr)
{
    uint64_t d = (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)((uint32_t)kHalf >> 4) << 16;
    d |= (uint64_t)(1024u >> 4) << 32;
    d |= (uint64_t)1u << 46;
    d |= (uint64_t)2u << 61;
    return d;
}

// D[tmem] (+)= A[tmem] * B[smem]
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc)
{
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
        : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
        "%14,%15,%16};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

__device__ __forceinline__ void tmem_st8(uint32_t addr, const uint32_t (&r)[8])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
        : "memory");
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

__device__ __forceinline__ void tmem_wait_st()
{
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

template <int kBar, int kCount>
__device__ __forceinline__ void bar_sync()
{
    asm volatile("bar.sync %0, %1;" ::"n"(kBar), "n"(kCount) : "memory");
}

// Barrier of one softmax group (2 + w) over its 256 threads.
__device__ __forceinline__ void group_sync(int w)
{
    if (w == 0) bar_sync<2, 256>();
    else bar_sync<3, 256>();
}

// Barrier of the two warps that share rows (ids 4 .. 11); the second form
// tells both whether either said yes.
__device__ __forceinline__ void pair_sync(int id)
{
    asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory");
}

__device__ __forceinline__ bool pair_any(int id, bool x)
{
    uint32_t r;
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.u32 p, %2, 0;\n bar.red.or.pred q, %1, 64, p;\n"
        " selp.u32 %0, 1, 0, q;\n}\n"
        : "=r"(r)
        : "r"(id), "r"((uint32_t)x)
        : "memory");
    return r != 0;
}

__device__ __forceinline__ void tmem_st1(uint32_t addr, float x)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(addr),
                 "r"(__float_as_uint(x))
                 : "memory");
}

__device__ __forceinline__ float tmem_ld1(uint32_t addr)
{
    uint32_t a;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\ntcgen05.wait::ld.sync.aligned;"
                 : "=r"(a)
                 : "r"(addr)
                 : "memory");
    return __uint_as_float(a);
}

// 32-byte stores: a whole sector per lane.
__device__ __forceinline__ void st_v8(void *p, const uint32_t *r)
{
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// Tiles of an item: the cache's and, last, the drafted tokens'; none when it
// has no live row or the unit is refused.
__device__ __forceinline__ int item_tiles(const AttArgs &a, int n, int live, int rb)
{
    if (n < 0 || n > a.max_len || live < 0 || live * a.G <= rb * kRows) return 0;
    return (n + kTile - 1) / kTile + 1;
}

// The line is cut into as many parts as there are CTAs, none of them empty.
__device__ __forceinline__ int parts_of(int grid, int total) { return min(grid, total); }

// The part of one item that this CTA takes.
struct Seg {
    int item, u, rb, n, live, nt;   // nt: tiles of the item
    int t0, t1;                     // this CTA's tiles of it
    int rows;                       // live rows of the item
};

struct Walk {
    const AttArgs &a;
    int item, base, lo, hi;
    int n_next, live_next;

    __device__ Walk(const AttArgs &a_, int item_, int base_, int lo_, int hi_)
        : a(a_), item(item_), base(base_), lo(lo_), hi(hi_)
    {
        peek(item);
    }
    __device__ void peek(int i)
    {
        if (i < a.U * a.RB) {
            const int u = i / a.RB;
            n_next = a.len[u];
            live_next = tree_live(a.t, u);
        }
    }
    __device__ bool next(Seg &s)
    {
        while (base < hi && item < a.U * a.RB) {
            s.item = item;
            s.u = item / a.RB;
            s.rb = item - s.u * a.RB;
            s.n = n_next;
            s.live = live_next;
            s.nt = item_tiles(a, s.n, s.live, s.rb);
            peek(item + 1);
            const int b = base;
            base += s.nt;
            item++;
            s.t0 = max(0, lo - b);
            s.t1 = min(s.nt, hi - b);
            if (s.t1 > s.t0) {
                s.rows = min(kRows, s.live * a.G - s.rb * kRows);
                return true;
            }
        }
        return false;
    }
};

// valid slots of tile t (the drafted tokens' tile: the live ones)
__device__ __forceinline__ int tile_valid(const Seg &s, int t)
{
    return t == s.nt - 1 ? s.live : min(kTile, s.n - t * kTile);
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(reinterpret_cast<uint64_t &>(d))
        : "l"(reinterpret_cast<const uint64_t &>(a)), "l"(reinterpret_cast<const uint64_t &>(b)),
          "l"(reinterpret_cast<const uint64_t &>(c)));
    return d;
}

__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    float2 d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(reinterpret_cast<uint64_t &>(d))
        : "l"(reinterpret_cast<const uint64_t &>(a)), "l"(reinterpret_cast<const uint64_t &>(b)));
    return d;
}

// Hidden slots of 16 raw products: -inf.
__device__ __forceinline__ void hide16(uint32_t (&y)[16], uint32_t keep)
{
#pragma unroll
    for (int j = 0; j < 16; j++) y[j] = keep >> j & 1 ? y[j] : 0xff800000u;
}

// Half a tile of the thread's row (64 of 128 slots; `half`): the row's maximum
// so far, the weights, which replace S as bf16 pairs, and their sum.  S is
// read twice, 16 columns at a time with the next 16 in flight: 64 held at once
// spill at 96 registers, and spills go through the memory that feeds the MMAs.
// A slot's vote multiplies its weight (exp(x + ln p) = p exp(x)).  The two
// halves agree on the maximum in shared memory, only when one of them has to
// move it, and as bf16: any reference near the maximum will do.  On the
// group's last tile of an item `last` l becomes the sum of both halves
// (through a column of S that is read by then).
template <bool kMask>
__device__ __forceinline__ void softmax_half(uint32_t tS, uint32_t tO, int half, int pair,
                                             float scale, const float *vote, uint64_t keep,
                                             __nv_bfloat16 (&xm)[2][kTile], int r, bool rescale,
                                             bool last, float &m, float &l)
{
    uint32_t y0[16], y1[16];
    float mx[2] = {-INFINITY, -INFINITY};
    const uint32_t at = tS + 64 * half;
    auto top_of = [&](uint32_t (&y)[16], uint32_t k) {
        if (kMask) hide16(y, k);
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
            mx[0] = fmaxf(fmaxf(mx[0], __uint_as_float(y[j])), __uint_as_float(y[j + 1]));
            mx[1] = fmaxf(fmaxf(mx[1], __uint_as_float(y[j + 2])), __uint_as_float(y[j + 3]));
        }
    };
    tmem_ld16_async(at, y0);
#pragma unroll
    for (int q = 0; q < 2; q++) {
        const uint32_t k = (uint32_t)(keep >> (32 * q));
        tmem_wait_ld();
        tmem_bind16(y0);
        tmem_ld16_async(at + 32 * q + 16, y1);
        top_of(y0, k);
        tmem_wait_ld();
        tmem_bind16(y1);
        tmem_ld16_async(q ? at : at + 32, y0);              // the last: the second pass's first
        top_of(y1, k >> 16);
    }
    float top = fmaxf(mx[0], mx[1]) * scale;
    if (pair_any(pair, top > m + kSlack || (m == -INFINITY && top > m))) {
        tmem_wait_ld();
        tmem_bind16(y0);
        xm[half][r] = __float2bfloat16_rn(top);
        pair_sync(pair);
        top = fmaxf(__bfloat162float(xm[0][r]), __bfloat162float(xm[1][r]));
        const bool move = top > m + kSlack || (m == -INFINITY && top > m);
        float f = 1.f;
        if (move) {
            f = m == -INFINITY ? 0.f : ex2_approx(m - top);
            m = top;
            l *= f;
        }
        if (rescale && __any_sync(kFull, move)) {
#pragma unroll 1
            for (int h = 0; h < 4; h++) {
                uint32_t y[16];
                const uint32_t o = tO + 64 * half + 16 * h;
                tmem_ld16_async(o, y);
                tmem_wait_ld();
                tmem_bind16(y);
#pragma unroll
                for (int j = 0; j < 16; j++) y[j] = __float_as_uint(__uint_as_float(y[j]) * f);
                tmem_st16(o, y);
            }
        }
    }
    const float nref = m == -INFINITY ? 0.f : -m;
    const float2 c2 = make_float2(scale, scale), r2 = make_float2(nref, nref);
    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    auto weights = [&](uint32_t (&y)[16], int h, uint32_t k) {
        if (kMask) hide16(y, k);
        uint32_t p[8];
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            float2 e[2];
#pragma unroll
            for (int i = 0; i < 2; i++) {
                const float2 x = make_float2(__uint_as_float(y[2 * (j + i)]),
                                             __uint_as_float(y[2 * (j + i) + 1]));
                const float2 t = fma2(x, c2, r2);
                e[i] = make_float2(ex2_approx(t.x), ex2_approx(t.y));
            }
            if (vote) {
                const float4 v = *reinterpret_cast<const float4 *>(vote + 64 * half + 16 * h + 2 * j);
                e[0].x *= v.x;
                e[0].y *= v.y;
                e[1].x *= v.z;
                e[1].y *= v.w;
            }
#pragma unroll
            for (int i = 0; i < 2; i++) {
                sum[i] = add2(sum[i], e[i]);
                p[j + i] = pack_bf16(e[i].x, e[i].y);
            }
        }
        tmem_st8(at + 8 * h, p);                             // over columns already read
    };
#pragma unroll
    for (int q = 0; q < 2; q++) {
        const uint32_t k = (uint32_t)(keep >> (32 * q));
        tmem_wait_ld();
        tmem_bind16(y0);
        tmem_ld16_async(at + 32 * q + 16, y1);
        weights(y0, 2 * q, k);
        tmem_wait_ld();
        tmem_bind16(y1);
        if (q == 0) tmem_ld16_async(at + 32, y0);
        weights(y1, 2 * q + 1, k >> 16);
    }
    l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
    if (last) tmem_st1(at + 32, l);
    tmem_wait_st();
    if (last) {
        tc_fence_before();
        pair_sync(pair);
        tc_fence_after();
        l += tmem_ld1(tS + 64 * (half ^ 1) + 32);
    }
}

__global__ void __launch_bounds__(kThreads, 1)
tree_attend_kernel(const __grid_constant__ AttArgs a, const __grid_constant__ CUtensorMap tmK,
                   const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmQ,
                   const __grid_constant__ CUtensorMap tmKt, const __grid_constant__ CUtensorMap tmVt)
{
    extern __shared__ __align__(1024) unsigned char dyn[];
    unsigned char *qbuf = dyn, *ring = qbuf + 2 * kSlot;
    AttSmem &S = *reinterpret_cast<AttSmem *>(ring + kRing * kSlot);
    if (smem_u32(dyn) & 1023) {                  // the swizzle counts on it
        if (threadIdx.x == 0) record_status(a.status, KVC_ERR_CUDA);
        return;
    }
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int items = a.U * a.RB;

    if (tid == 0) {
        S.bad = 0;
        for (int i = 0; i < kRing; i++) {
            mbar_init(&S.full[i], 1);
            mbar_init(&S.empty[i], 1);
        }
        mbar_init(&S.drain, 1);
        for (int i = 0; i < 2; i++) {
            mbar_init(&S.qfull[i], 1);
            mbar_init(&S.qempty[i], 1);
            mbar_init(&S.sfull[i], 1);
            mbar_init(&S.pready[i], 8);
            mbar_init(&S.pvdone[i], 1);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMma) tmem_alloc(&S.tmem, 512);

    // the line of tiles: every CTA counts it and finds where its part starts
    int lo, hi;
    {
        const int per = (items + kThreads - 1) / kThreads;
        const int i0 = min(items, tid * per), i1 = min(items, i0 + per);
        int sum = 0;
        for (int i = i0; i < i1; i++) {
            const int u = i / a.RB, n = a.len[u], live = tree_live(a.t, u);
            if (blockIdx.x == 0 && (n < 0 || n > a.max_len || live < 0) && i == u * a.RB)
                record_status(a.status, live < 0 ? KVC_ERR_INVALID_ARG : KVC_ERR_SHAPE);
            sum += item_tiles(a, n, live, i - u * a.RB);
        }
        int total;
        int base = block_exscan(sum, S.scan, &total);
        if (a.whole) {
            // parts of whole items: nothing to join
            const int c0 = (int)((long long)items * blockIdx.x / gridDim.x);
            const int c1 = (int)((long long)items * (blockIdx.x + 1) / gridDim.x);
            for (int i = i0, b = base; i < i1; i++) {
                const int u = i / a.RB;
                if (i == c0) { S.start_item = i; S.start_base = b; }
                b += item_tiles(a, a.len[u], tree_live(a.t, u), i - u * a.RB);
                if (i == c1 - 1) S.total = b;
            }
            __syncthreads();
            lo = c0 < c1 ? S.start_base : 0;
            hi = c0 < c1 ? S.total : 0;
        } else {
            const int g = parts_of(gridDim.x, total), c = min((int)blockIdx.x, g);
            lo = g ? (int)((long long)total * c / g) : 0;
            hi = g ? (int)((long long)total * min(c + 1, g) / g) : 0;
            if (tid == 0) S.cut = make_int4(-1, 0, 0, 0);
            __syncthreads();
            for (int i = i0, b = base; i < i1; i++) {
                const int u = i / a.RB;
                const int nt = item_tiles(a, a.len[u], tree_live(a.t, u), i - u * a.RB);
                if (blockIdx.x == 0) a.first[i] = b;
                if (lo >= b && lo < b + nt) {
                    S.start_item = i;
                    S.start_base = b;
                    // the part before has the item's start: this CTA names its parts
                    if (lo > b && b >= (long long)total * (c - 1) / g)
                        S.cut = make_int4(i, c - 1, (int)(((long long)(b + nt) * g - 1) / total), 0);
                }
                b += nt;
                if (blockIdx.x == 0 && i == items - 1) a.first[items] = b;
            }
            __syncthreads();
            if (tid == 0) a.cut[blockIdx.x] = S.cut;
        }
    }
    tc_fence_after();
    const uint32_t tmem = S.tmem;
    Walk walk(a, lo < hi ? S.start_item : items, S.start_base, lo, hi);
    Seg s;


    if (warp == kProd) {
        // ------------------------------------------------------- producer
        if (elect_one()) {
            int k = 0, slot = 0, nseg = 0, qn[2] = {0, 0};
            uint32_t ph = 1;                     // phase of the slot's last release
            bool ok = true;
            const uint64_t pol = l2_policy_evict_first();
            auto load = [&](const CUtensorMap *m, int u, int row, int rows, bool stream) {
                if (k >= kRing) ok = tree_wait(&S.empty[slot], ph, &S.bad);
                if (!ok) return;
                unsigned char *d = ring + slot * kSlot;
                const int boxes = rows > 64 ? 2 : 1;
                mbar_expect_tx(&S.full[slot], boxes * kHalf);
                for (int h = 0; h < 2; h++)
                    for (int b = 0; b < boxes; b++) {
                        if (stream)
                            tma_3d_hint(d + h * kHalf + b * (kHalf / 2), m, 64 * h, row + 64 * b, u,
                                        &S.full[slot], pol);
                        else
                            tma_3d(d + h * kHalf + b * (kHalf / 2), m, 64 * h, row + 64 * b, u,
                                   &S.full[slot]);
                    }
                k++;
                if (++slot == kRing) { slot = 0; ph ^= 1; }
            };
            auto load_q = [&](int half, int u, int row, int rows) {
                if (qn[half] > 0) ok = ok && tree_wait(&S.qempty[half], (qn[half] - 1) & 1, &S.bad);
                if (!ok) return;
                const int boxes = rows > 64 ? 2 : 1;
                unsigned char *d = qbuf + half * kSlot;
                mbar_expect_tx(&S.qfull[half], boxes * kHalf);
                for (int h = 0; h < 2; h++)
                    for (int b = 0; b < boxes; b++)
                        tma_3d(d + h * kHalf + b * (kHalf / 2), &tmQ, 64 * h, row + 64 * b, u,
                               &S.qfull[half]);
                qn[half]++;
            };
            while (ok && walk.next(s)) {
                const int qrow = s.rb * kRows;
                if (s.rows > 128) {
                    load_q(0, s.u, qrow, 128);
                    load_q(1, s.u, qrow + 128, s.rows - 128);
                } else {
                    // the halves alternate, so the next item's rows load early;
                    // an item of two halves takes both, whichever was last
                    load_q(nseg & 1, s.u, qrow, s.rows);
                }
                nseg++;
                for (int t = s.t0; ok && t < s.t1; t++) {
                    const int nv = tile_valid(s, t);
                    if (t == s.nt - 1) {
                        load(&tmKt, s.u, 0, 64, false);
                        if (ok) load(&tmVt, s.u, 0, 64, false);
                    } else {
                        load(&tmK, s.u, t * kTile, nv, a.RB == 1);
                        if (ok) load(&tmV, s.u, t * kTile, nv, a.RB == 1);
                    }
                }
            }
            if (!ok) {
                S.bad = 1;
                // the copies in flight land before the block ends
                for (int i = max(0, k - kRing); i < k; i++)
                    mbar_wait(&S.full[i % kRing], (i / kRing) & 1);
                for (int h = 0; h < 2; h++)
                    if (qn[h]) mbar_wait(&S.qfull[h], (qn[h] - 1) & 1);
            }
        }
        __syncwarp();
    } else if (warp == kMma) {
        // ------------------------------------------------------ MMA issuer
        if (elect_one()) {
            bool ok = true;
            // slot and phase of the ring's next key and value tile; phases of
            // the groups' barriers as bits
            int ks_slot = 0, vs_slot = 1;
            uint32_t ks_ph = 0, vs_ph = 0, q_ph = 0, p_ph = 0, nseg = 0;
            const uint64_t q0 = umma_sdesc(smem_u32(qbuf)), k0 = umma_sdesc(smem_u32(ring));
            const uint64_t v0 = v_desc(smem_u32(ring));
            constexpr uint32_t kStep = kSlot >> 4;           // a slot in descriptor units
            // S of group w from tile t; the key tile is waited for by its first
            // reader and given back by its last
            auto issue_s = [&](uint32_t w, uint32_t half, bool small, bool first, bool last_q) {
                if (first) ok = ok && tree_wait(&S.full[ks_slot], ks_ph, &S.bad);
                if (!ok) return;
                tc_fence_after();
                const uint32_t idesc = small ? kIdescS64 : kIdescS, d = tmem + kColS + 128 * w;
                const uint64_t qd = q0 + half * kStep, kd = k0 + (uint32_t)ks_slot * kStep;
#pragma unroll
                for (int ks = 0; ks < 8; ks++)
                    umma_bf16(d, umma_sdesc_step(qd, ks), umma_sdesc_step(kd, ks), idesc, ks > 0);
                umma_commit(&S.sfull[w]);
                if (last_q) umma_commit(&S.qempty[half]);
            };
            auto free_k = [&] {
                if (!ok) return;
                umma_commit(&S.empty[ks_slot]);
                ks_slot += 2;
                if (ks_slot >= kRing) { ks_slot -= kRing; ks_ph ^= 1; }
            };
            auto issue_o = [&](uint32_t w, int nv, bool first, bool keep) {
                if (first) ok = ok && tree_wait(&S.full[vs_slot], vs_ph, &S.bad);
                ok = ok && tree_wait(&S.pready[w], p_ph >> w & 1, &S.bad);
                p_ph ^= 1u << w;
                if (!ok) return;
                tc_fence_after();
                const uint64_t vd = v0 + (uint32_t)vs_slot * kStep;
                const uint32_t d = tmem + 128 * w, p = tmem + kColS + 128 * w;
                if (nv > kTile - 16) {
#pragma unroll
                    for (int ks = 0; ks < 8; ks++)
                        umma_ts(d, p + 8 * ks + 32 * (ks >> 2), vd + (uint64_t)(ks * (2048 >> 4)),
                                kIdescO, ks > 0 || keep);
                } else {
                    for (int ks = 0; 16 * ks < nv; ks++)
                        umma_ts(d, p + 8 * ks + 32 * (ks >> 2), vd + (uint64_t)(ks * (2048 >> 4)),
                                kIdescO, ks > 0 || keep);
                }
                umma_commit(&S.pvdone[w]);
            };
            auto free_v = [&] {
                if (!ok) return;
                umma_commit(&S.empty[vs_slot]);
                vs_slot += 2;
                if (vs_slot >= kRing) { vs_slot -= kRing; vs_ph ^= 1; }
            };
            auto wait_q = [&](uint32_t half) {
                ok = ok && tree_wait(&S.qfull[half], q_ph >> half & 1, &S.bad);
                q_ph ^= 1u << half;
            };
            while (ok && walk.next(s)) {
                const int nq = s.t1 - s.t0;
                const uint32_t qh = nseg++ & 1;
                if (s.rows > 128) {
                    wait_q(0);
                    wait_q(1);
                    bool small = tile_valid(s, s.t0) <= 64;
                    issue_s(0, 0, small, true, nq == 1);
                    issue_s(1, 1, small, false, nq == 1);
                    free_k();
                    for (int t = 0; ok && t < nq; t++) {
                        const int nv = tile_valid(s, s.t0 + t);
                        const bool more = t + 1 < nq, end = t + 2 == nq;
                        small = more && tile_valid(s, s.t0 + t + 1) <= 64;
                        issue_o(0, nv, true, t > 0);
                        if (more) issue_s(0, 0, small, true, end);
                        issue_o(1, nv, false, t > 0);
                        free_v();
                        if (more) {
                            issue_s(1, 1, small, false, end);
                            free_k();
                        }
                    }
                } else {
                    wait_q(qh);
                    issue_s(0, qh, tile_valid(s, s.t0) <= 64, true, nq == 1);
                    free_k();
                    if (nq > 1) {
                        issue_s(1, qh, tile_valid(s, s.t0 + 1) <= 64, true, nq == 2);
                        free_k();
                    }
                    for (int t = 0; ok && t < nq; t++) {
                        const uint32_t w = t & 1;
                        issue_o(w, tile_valid(s, s.t0 + t), true, t > 1);
                        free_v();
                        if (t + 2 < nq) {
                            issue_s(w, qh, tile_valid(s, s.t0 + t + 2) <= 64, true, t + 3 == nq);
                            free_k();
                        }
                    }
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
    } else if (warp < kProd) {
        // --------------------------------------------------------- softmax
        const int w = warp >> 3, half = warp >> 2 & 1, wl = warp & 3;
        const int r = wl * 32 + lane;                    // row of the group's 128
        const int pair = 4 + 4 * w + wl;
        const uint32_t lanes = (uint32_t)(wl * 32) << 16;
        const uint32_t tS = tmem + lanes + kColS + 128 * w, tO = tmem + lanes + 128 * w;
        bool ok = true;
        int k0 = 0, sn = 0, pn = 0, ntree = 0;
        while (walk.next(s)) {
            const bool dual = s.rows > 128;
            const int nq = s.t1 - s.t0;
            const int row = (dual ? 128 * w : 0) + r;        // row of the item
            const bool mine = row < s.rows;
            const bool busy = (dual ? 128 * w : 0) + wl * 32 < s.rows;   // the warp has rows
            const int grow = s.rb * kRows + row;             // row of the unit
            float m = -INFINITY, l = 0.f;
            int done = 0;                                    // this group's tiles so far
            uint64_t odd = 0;                                // drafted tokens added by hand
            uint64_t see = 0;
            if (mine)
                see = a.t.mask[(size_t)(s.u / a.t.units) * a.t.T + grow / a.G] &
                      (s.live >= 64 ? ~0ull : (1ull << s.live) - 1);
            int vote_next = 0;                               // loaded a tile ahead
            if (a.votes && half == 0) {
                const int i = (s.t0 + (dual ? 0 : w)) * kTile + r;
                if (i < s.n) vote_next = a.votes[(size_t)s.u * a.cap + i];
            }
            for (int t = dual ? 0 : w; t < nq; t += dual ? 1 : 2) {
                const int tile = s.t0 + t, nv = tile_valid(s, tile);
                const bool tree = tile == s.nt - 1;
                const int kv = k0 + 2 * t + 1, slot = kv % kRing;
                const bool votes = a.votes != nullptr && !tree;
                if (votes) {
                    group_sync(w);                           // the last tile's are read
                    if (half == 0) S.g[w].vote[r] = (float)vote_next;
                    const int i = (tile + (dual ? 1 : 2)) * kTile + r;
                    if (half == 0 && i < s.n) vote_next = a.votes[(size_t)s.u * a.cap + i];
                    group_sync(w);
                }
                // value rows the MMA reads that are no slot: zero
                if (!dual || w == 0) {
                    if (nv & 15 || tree) {
                        ok = tree_wait(&S.full[slot], (kv / kRing) & 1, &S.bad) && ok;
                        unsigned char *v = ring + slot * kSlot;
                        const int stop = (nv + 15) & ~15;
                        if (tree && half == 0 && r < 64) {
                            // thread r has row r: what is not finite is zeroed here and
                            // added to the rows that see it at the end
                            bool bad = false;
                            if (r < stop)
                                for (int c = 0; c < 16; c++) {
                                    unsigned char *p = v + (c >> 3) * kHalf + r * 128 + (((c & 7) ^ (r & 7)) << 4);
                                    const uint4 x = lds_v4(p);
                                    uint32_t q[4] = {x.x, x.y, x.z, x.w};
                                    bool hit = r >= nv;
#pragma unroll
                                    for (int e = 0; e < 4; e++) {
                                        const bool lo = (q[e] & 0x7f80u) == 0x7f80u;
                                        const bool hi = (q[e] & 0x7f800000u) == 0x7f800000u;
                                        hit |= lo || hi;
                                        if (lo || r >= nv) q[e] &= 0xffff0000u;
                                        if (hi || r >= nv) q[e] &= 0x0000ffffu;
                                    }
                                    if (hit)
                                        *reinterpret_cast<uint4 *>(p) = make_uint4(q[0], q[1], q[2], q[3]);
                                    bad |= hit;
                                }
                            const uint32_t bits = __ballot_sync(kFull, bad && r < nv);
                            if (lane == 0) reinterpret_cast<uint32_t *>(&S.odd[ntree & 1])[wl] = bits;
                        } else if (!tree && half == 0 && r >= nv && r < stop) {
                            for (int c = 0; c < 16; c++)
                                *reinterpret_cast<uint4 *>(v + (c >> 3) * kHalf + r * 128 +
                                                           ((c & 7) << 4)) = make_uint4(0, 0, 0, 0);
                        }
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        group_sync(w);
                    }
                }
                if (tree && dual) bar_sync<1, 512>();        // both groups see the odd tokens
                if (tree) odd = S.odd[ntree & 1];
                ok = tree_wait(&S.sfull[w], sn & 1, &S.bad) && ok;
                sn++;
                tc_fence_after();
                if (busy) {
                    const float *vote = votes ? S.g[w].vote : nullptr;
                    const bool last = t + (dual ? 1 : 2) >= nq;
                    if (tree || nv < kTile) {
                        uint64_t keep = 0;                   // slots the row may see
                        if (tree) {
                            keep = half ? 0 : see;
                        } else {
                            const int k = nv - 64 * half;
                            keep = k >= 64 ? ~0ull : k <= 0 ? 0ull : (1ull << k) - 1;
                        }
                        softmax_half<true>(tS, tO, half, pair, a.scale, vote, keep, S.g[w].top, r,
                                           done > 0, last, m, l);
                    } else {
                        softmax_half<false>(tS, tO, half, pair, a.scale, vote, ~0ull, S.g[w].top, r,
                                            done > 0, last, m, l);
                    }
                }
                done++;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&S.pready[w]);
                pn++;
            }
            k0 += 2 * nq;
            // ------------------------------------------------------ outputs
            if (done > 0) ok = tree_wait(&S.pvdone[w], (pn - 1) & 1, &S.bad) && ok;
            tc_fence_after();
            const bool all = s.t1 - s.t0 == s.nt;            // nothing to join
            const bool direct = all && !a.join_all;
            float c0 = 1.f, c1 = 0.f, M = m, Lsum = l;       // weights of the groups' sums
            if (!dual) {
                if (half == 0) S.g[w].ml[r] = make_float2(m, l);
                tc_fence_before();
                bar_sync<1, 512>();
                tc_fence_after();
                odd = S.odd[ntree & 1];          // written by the group that had the tokens' tile
                const float2 p0 = S.g[0].ml[r], p1 = S.g[1].ml[r];
                M = fmaxf(p0.x, p1.x);
                const float ref = M == -INFINITY ? 0.f : M;
                c0 = ex2_approx(p0.x - ref);
                c1 = ex2_approx(p1.x - ref);
                Lsum = p0.y * c0 + p1.y * c1;
            }
            const size_t sid = (size_t)s.item + blockIdx.x;
            const size_t orow = (size_t)s.u * a.TG + grow;
            const float inv = Lsum == 0.f ? 0.f : 1.f / Lsum;
            const float k_0 = direct ? c0 * inv : c0, k_1 = direct ? c1 * inv : c1;
            const bool has_tree = s.t1 == s.nt;
            const uint64_t by_hand = has_tree ? odd & see : 0;
            ntree += has_tree;
            // a warp writes 64 columns of its rows, or (alternate tiles) 32
            if (busy) {
                const int q0 = dual ? 2 * half : 2 * w + half, q1 = dual ? q0 + 2 : q0 + 1;
#pragma unroll 1
                for (int q = 2 * q0; q < 2 * q1; q++) {      // 16 columns at a time
                    uint32_t y[16], z[16];
                    tmem_ld16_async(tmem + lanes + (dual ? 128 * w : 0) + 16 * q, y);
                    if (!dual && nq > 1) tmem_ld16_async(tmem + lanes + 128 + 16 * q, z);
                    tmem_wait_ld();
                    tmem_bind16(y);
                    float f[16];
#pragma unroll
                    for (int j = 0; j < 16; j++) f[j] = __uint_as_float(y[j]) * k_0;
                    if (!dual && nq > 1) {
                        tmem_bind16(z);
#pragma unroll
                        for (int j = 0; j < 16; j++) f[j] = fmaf(__uint_as_float(z[j]), k_1, f[j]);
                    }
                    if (by_hand) {
                        // a visible value that is not finite: whatever its weight, the
                        // output is what weight x value gives, not finite
                        for (uint64_t rest = by_hand; rest; rest &= rest - 1) {
                            const int jt = __ffsll((long long)rest) - 1;
                            const uint16_t *vr = a.vt + ((size_t)s.u * a.t.T + jt) * kD + 16 * q;
#pragma unroll
                            for (int j = 0; j < 16; j++) {
                                const float v = bf2f(vr[j]);
                                f[j] += isfinite(v) ? 0.f : v;
                            }
                        }
                    }
                    if (mine && ok) {
                        if (direct) {
                            uint32_t h[8];
#pragma unroll
                            for (int j = 0; j < 8; j++) h[j] = pack_bf16(f[2 * j], f[2 * j + 1]);
                            uint4 *d = reinterpret_cast<uint4 *>(a.o + orow * kD + 16 * q);
                            d[0] = make_uint4(h[0], h[1], h[2], h[3]);
                            d[1] = make_uint4(h[4], h[5], h[6], h[7]);
                        } else {
                            float *d = a.part + (sid * a.rows + row) * kD + 16 * q;
                            st_v8(d, reinterpret_cast<const uint32_t *>(f));
                            st_v8(d + 8, reinterpret_cast<const uint32_t *>(f + 8));
                        }
                    }
                }
                if (mine && ok && half == 0 && (dual || w == 0)) {
                    if (direct)
                        a.lse[orow] = Lsum == 0.f ? -INFINITY
                                                  : (M + log2f(Lsum)) * 0.6931471805599453f;
                    else
                        a.ml[sid * a.rows + row] = make_float2(M, Lsum);
                }
            }
            // the other group reads this one's sums: both are done before either goes on
            tc_fence_before();
            if (!dual) bar_sync<1, 512>();
        }
    }
    __syncthreads();
    if (warp == kMma) tmem_dealloc(tmem, 512);
    if (tid == 0 && S.bad) record_status(a.status, KVC_ERR_TIMEOUT);
}

struct JoinArgs {
    AttArgs a;
    const uint16_t *q;
    const float *mn, *mu_k, *mu_v, *C;
    int first_order, grid;
};

// The sums of a cut item's parts added: one warp per row, a lane has four
// columns.  The result is the output, or (kKeep, when the moments follow) the
// first part's place takes it.  grid (CTAs of the attention, rows / 8): block
// x takes the item whose first cut is the start of part x.
template <bool kKeep>
__global__ void __launch_bounds__(256) tree_join_kernel(const __grid_constant__ JoinArgs j)
{
    const AttArgs &a = j.a;
    const int4 cut = a.cut[blockIdx.x];
    if (cut.x < 0) return;
    const int lane = threadIdx.x & 31, r = blockIdx.y * 8 + (threadIdx.x >> 5);
    const int u = cut.x / a.RB, rb = cut.x - u * a.RB;
    if (r >= min(kRows, tree_live(a.t, u) * a.G - rb * kRows)) return;
    const size_t at = ((size_t)cut.x + cut.y) * a.rows + r, step = (size_t)a.rows;
    const int np = cut.z - cut.y + 1;
    float M = -INFINITY;
    for (int k = lane; k < np; k += 32) M = fmaxf(M, a.ml[at + k * step].x);
    M = warp_max(M);
    const float ref = M == -INFINITY ? 0.f : M;
    float L = 0.f;
    float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = 0; k0 < np; k0 += 32) {
        float s = 0.f;
        if (k0 + lane < np) {
            const float2 ml = a.ml[at + (k0 + lane) * step];
            s = ex2_approx(ml.x - ref);
            L += ml.y * s;
        }
        const int m = min(32, np - k0);
#pragma unroll 8
        for (int k = 0; k < m; k++) {
            const float c = __shfl_sync(kFull, s, k);
            const float4 p =
                reinterpret_cast<const float4 *>(a.part + (at + (k0 + k) * step) * kD)[lane];
            f.x = fmaf(p.x, c, f.x);
            f.y = fmaf(p.y, c, f.y);
            f.z = fmaf(p.z, c, f.z);
            f.w = fmaf(p.w, c, f.w);
        }
    }
    L = warp_sum(L);
    if (kKeep) {
        __syncwarp();
        reinterpret_cast<float4 *>(a.part + at * kD)[lane] = f;
        if (lane == 0) a.ml[at] = make_float2(M, L);
        return;
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    const size_t row = (size_t)u * a.TG + (size_t)rb * kRows + r;
    reinterpret_cast<uint2 *>(a.o + row * kD)[lane] =
        make_uint2(pack_bf16(f.x * inv, f.y * inv), pack_bf16(f.z * inv, f.w * inv));
    if (lane == 0) a.lse[row] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
}

// The normalization correction: every row's sum normalised and mixed with the
// evicted set's estimate.  C q runs on tensor cores (mma.sync) with C as two
// bf16 terms (2^-16 of a product) in shared memory, 128-byte swizzled.  A CTA
// has 64 rows of an item, a warp 16 rows and half of the columns; grid
// (items, rows / 64).
constexpr int kMomRows = 64;
constexpr size_t kMomDyn = 2 * (size_t)kSlot;

__global__ void __launch_bounds__(256, 2) tree_moment_kernel(const __grid_constant__ JoinArgs j)
{
    const AttArgs &a = j.a;
    extern __shared__ __align__(1024) unsigned char cs[];   // C: high terms, low terms
    __shared__ float muk[kD], muv[kD];
    const int item = blockIdx.x, u = item / a.RB, rb = item - u * a.RB;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3, n0 = 64 * (warp & 1);
    const int n = a.len[u], live = tree_live(a.t, u);
    const float ne = j.mn[u];
    const bool mix = ne > 0.f;
    const int rows = min(kRows, live * a.G - rb * kRows), r0 = blockIdx.y * kMomRows + 16 * (warp >> 1);
    // the part that has the item's start (its place has the joined sums)
    int c0;
    if (a.whole) {
        c0 = (int)((((long long)item + 1) * j.grid - 1) / (a.U * a.RB));
    } else {
        const int W = a.first[a.U * a.RB];
        c0 = W ? (int)(((a.first[item] + 1ll) * parts_of(j.grid, W) - 1) / W) : 0;
    }
    if (n < 0 || n > a.max_len || live < 0 || (int)blockIdx.y * kMomRows >= rows) return;
    if (mix && j.first_order) {
        const float4 *C = reinterpret_cast<const float4 *>(j.C + (size_t)u * kD * kD);
        // 8 elements of a row of C a step, 16 bytes each of high and low terms
#pragma unroll 4
        for (int i = 0; i < kD * 16 / 256; i++) {
            const int e = i * 256 + tid, row = e >> 4, ch = e & 15;
            const float4 x = C[2 * e], y = C[2 * e + 1];
            const float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int k = 0; k < 4; k++) {
                hi[k] = pack_bf16(v[2 * k], v[2 * k + 1]);
                lo[k] = pack_bf16(v[2 * k] - bf_lo(hi[k]), v[2 * k + 1] - bf_hi(hi[k]));
            }
            unsigned char *d = cs + sw_off_t<128>(row, ch);
            *reinterpret_cast<uint4 *>(d) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4 *>(d + kSlot) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
    }
    if (mix && tid < kD) {
        muk[tid] = j.mu_k[(size_t)u * kD + tid];
        muv[tid] = j.mu_v[(size_t)u * kD + tid];
    }
    const size_t ubase = (size_t)u * a.TG + (size_t)rb * kRows;
    const size_t pbase = ((size_t)item + c0) * a.rows;
    const int ra[2] = {min(r0 + g, rows - 1), min(r0 + g + 8, rows - 1)};
    const float2 ml[2] = {a.ml[pbase + ra[0]], a.ml[pbase + ra[1]]};
    const float sd = rsqrtf((float)kD);
    uint32_t qa[8][4];
    if (mix) {
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const uint32_t *p = reinterpret_cast<const uint32_t *>(j.q + (ubase + ra[h]) * kD) + t;
#pragma unroll
            for (int ks = 0; ks < 8; ks++) {
                qa[ks][h] = p[8 * ks];
                qa[ks][2 + h] = p[8 * ks + 4];
            }
        }
    }
    __syncthreads();
    float z[2] = {0.f, 0.f};
    float d[8][4];
#pragma unroll
    for (int i = 0; i < 8; i++) d[i][0] = d[i][1] = d[i][2] = d[i][3] = 0.f;
    if (mix) {
#pragma unroll
        for (int ks = 0; ks < 8; ks++)
#pragma unroll
            for (int h = 0; h < 4; h++) {
                const int k = 16 * ks + 8 * (h >> 1) + 2 * t;
                z[h & 1] += bf_lo(qa[ks][h]) * muk[k] + bf_hi(qa[ks][h]) * muk[k + 1];
            }
        if (j.first_order) {
            // ldmatrix: a quarter-warp has the addresses of rows n0 + 8 i .. + 7 of C
            // in one 8-column chunk; four chunks are two k-steps
            const uint32_t base = smem_u32(cs);
#pragma unroll
            for (int i = 0; i < 8; i++) {
#pragma unroll
                for (int k4 = 0; k4 < 4; k4++) {
                    const uint32_t off = sw_off_t<128>(n0 + 8 * i + (lane & 7), 4 * k4 + (lane >> 3));
                    uint32_t b[4], c[4];
                    ldsm_x4(base + kSlot + off, b[0], b[1], b[2], b[3]);
                    ldsm_x4(base + off, c[0], c[1], c[2], c[3]);
                    const uint32_t(&q0)[4] = qa[2 * k4], (&q1)[4] = qa[2 * k4 + 1];
                    mma16816(d[i], q0[0], q0[1], q0[2], q0[3], b[0], b[1]);
                    mma16816(d[i], q1[0], q1[1], q1[2], q1[3], b[2], b[3]);
                    mma16816(d[i], q0[0], q0[1], q0[2], q0[3], c[0], c[1]);
                    mma16816(d[i], q1[0], q1[1], q1[2], q1[3], c[2], c[3]);
                }
            }
        }
    }
#pragma unroll
    for (int h = 0; h < 2; h++) {
        const float lse = ml[h].y == 0.f ? -INFINITY : (ml[h].x + log2f(ml[h].y)) * 0.6931471805599453f;
        float w = 1.f;
        if (mix) {
            float x = z[h];
            x += __shfl_xor_sync(kFull, x, 1);
            x += __shfl_xor_sync(kFull, x, 2);
            w = 1.f / (1.f + expf(logf(ne) + sd * x - lse));
        }
        const float wf = ml[h].y == 0.f ? 0.f : w / ml[h].y, we = 1.f - w;
        const float *p = a.part + (pbase + ra[h]) * kD + n0 + 2 * t;
        uint32_t *o = reinterpret_cast<uint32_t *>(a.o + (ubase + ra[h]) * kD + n0 + 2 * t);
        const bool mine = r0 + g + 8 * h < rows;
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const float2 x = *reinterpret_cast<const float2 *>(p + 8 * i);
            float f0 = wf * x.x, f1 = wf * x.y;
            if (mix) {
                f0 += we * (muv[n0 + 8 * i + 2 * t] + sd * d[i][2 * h]);
                f1 += we * (muv[n0 + 8 * i + 2 * t + 1] + sd * d[i][2 * h + 1]);
            }
            if (mine) o[4 * i] = pack_bf16(f0, f1);
        }
        if (mine && t == 0 && n0 == 0) a.lse[ubase + ra[h]] = lse;
    }
}

struct TreeWs {
    int32_t *status;
    int *first;
    int4 *cut;
    float2 *ml;
    float *part;
    size_t bytes;
};

TreeWs tree_ws(const kvc_params &p, int T, void *base)
{
    TreeWs w{};
    char *b = static_cast<char *>(base);
    size_t off = 0;
    auto take = [&](size_t n) {
        char *r = b ? b + off : nullptr;
        off += align_up(n);
        return r;
    };
    const size_t TG = (size_t)T * p.G, items = (size_t)p.U * ((TG + kRows - 1) / kRows);
    const size_t rows = TG < (size_t)kRows ? TG : (size_t)kRows;
    w.status = reinterpret_cast<int32_t *>(take(sizeof(WsHeader)));
    w.first = reinterpret_cast<int *>(take((items + 1) * sizeof(int)));
    w.cut = reinterpret_cast<int4 *>(take(kGrid * sizeof(int4)));
    w.ml = reinterpret_cast<float2 *>(take((items + kGrid) * rows * sizeof(float2)));
    w.part = reinterpret_cast<float *>(take((items + kGrid) * rows * kD * sizeof(float)));
    w.bytes = off;
    return w;
}

}  // namespace

size_t tree_ws_bytes(const kvc_params &p, int T) { return tree_ws(p, T, nullptr).bytes; }

cudaError_t launch_tree_attend(const kvc_params &p, int max_len, const TreeArgs &t,
                               const uint16_t *q, const uint16_t *kt, const uint16_t *vt,
                               const kvc_cache &c, const kvc_moments *m, uint16_t *o, float *lse,
                               void *ws, cudaStream_t st)
{
    const TreeWs w = tree_ws(p, t.T, ws);
    const int TG = t.T * p.G, RB = (TG + kRows - 1) / kRows;
    const long long items = (long long)p.U * RB, tmax = (max_len + kTile - 1) / kTile + 1;
    if (items * tmax > 0x7fffffffll) return cudaErrorInvalidValue;
    CUtensorMap mk, mv, mq, mkt, mvt;
    if (!make_unit_map(&mk, c.K, p.U, p.cap) || !make_unit_map(&mv, c.V, p.U, p.cap) ||
        !make_unit_map(&mq, q, p.U, TG) || !make_unit_map(&mkt, kt, p.U, t.T) ||
        !make_unit_map(&mvt, vt, p.U, t.T))
        return cudaErrorInvalidValue;
    const bool whole = tmax <= 4 || items >= 8 * kGrid;
    long long grid = whole ? items : (items * tmax + 3) / 4;
    if (grid < items) grid = items;
    if (grid > kGrid) grid = kGrid;
    AttArgs a{t, c.votes, c.len, vt, o, lse, w.part, w.ml, w.first, w.cut, w.status, p.U, RB, TG, p.G, p.cap,
              max_len, TG < kRows ? TG : kRows, whole, m != nullptr, kLog2e / sqrtf((float)kD)};
    cudaError_t e = cudaFuncSetAttribute(tree_attend_kernel,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kDyn);
    if (e != cudaSuccess) return e;
    tree_attend_kernel<<<(int)grid, kThreads, kDyn, st>>>(a, mk, mv, mq, mkt, mvt);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if (m == nullptr && whole) return cudaSuccess;
    JoinArgs j{a, q, m ? m->n : nullptr, m ? m->mu_k : nullptr, m ? m->mu_v : nullptr,
               m ? m->C : nullptr, p.correction == KVC_CORR_FIRST_ORDER, (int)grid};
    if (!whole) {
        const dim3 g((unsigned)grid, (a.rows + 7) / 8);
        if (m) tree_join_kernel<true><<<g, 256, 0, st>>>(j);
        else tree_join_kernel<false><<<g, 256, 0, st>>>(j);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    if (m) {
        e = cudaFuncSetAttribute(tree_moment_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)kMomDyn);
        if (e != cudaSuccess) return e;
        const dim3 g((unsigned)items, (a.rows + kMomRows - 1) / kMomRows);
        tree_moment_kernel<<<g, 256, kMomDyn, st>>>(j);
    }
    return cudaGetLastError();
}

}  // namespace kvc

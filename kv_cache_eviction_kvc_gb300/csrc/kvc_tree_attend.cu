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
// Work split: an item is a unit's block of 256 rows.  Items go to the CTAs (one
// per SM) whole, or each in parts of its own, or the tiles of all items form one
// line that is cut into equal parts (choose_cut has the rule).  An item inside
// one part is finished there; one that a cut crosses leaves partial sums
// (maximum, sum, output) per part, which tree_join_kernel adds.  With moments
// every item leaves its sums, and tree_moment_kernel mixes them with the evicted
// set's estimate.  The drafted tokens are the item's last tile.
//
// Measured (bf16, d = 128, G = 4; a call among others): 128 units of 2623 slots
// on average, 24 tokens: 36.5 us, 4.9 TB/s; 1024 units of 1024 slots, 16 tokens,
// votes and moments: 140 us, 4.6 TB/s; 8 units of 131071 slots, 63 tokens (252
// rows): 115 to 122 us, 4.5 TB/s and 1.13 PFLOP/s, 31 tokens: 91 us, 5.9 TB/s, 64
// tokens of 8 heads (512 rows, two blocks that read the slots once each): 210 us.  With
// two halves of rows a tile takes 3600 clocks for its 2048 of the tensor core:
// S overwrites P, so a group's product, softmax and next product follow one
// another.  (S in two halves of 64 slots, each made under the softmax of the
// other, took 141 us: half as wide a product is bound by its operands' reads.)
// 1024-slot units spend 6000 of 25000 clocks on their ends (sums of the two
// groups, outputs, the next unit's first S).
//
// 384 threads:
//   warps 0-3, 4-7  two softmax groups, each with its own S, P and O in tensor
//                   memory.  Items of more than 128 rows give each group 128
//                   of them; otherwise the groups take alternate tiles of the
//                   same rows and add their sums at the end
//   warp 8          producer (TMA into a ring of 32 KB key and value tiles)
//   warp 9          tensor-memory owner and MMA issuer
//   warp 10         walks the CTA's items ahead of the others and tells them
//                   through a ring in shared memory
//   warp 11         mends value tiles before their MMA (see below)
// (168 registers a thread: spills would go through the few KB of L1 that the
// tiles leave, to L2.)
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
// A warp of its own does it while the tile's S and softmax run: by the softmax
// threads it was 4000 of the 30000 clocks of a unit of 1024 slots.
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
constexpr int kThreads = 384;
constexpr int kProd = 8, kMma = 9, kWalk = 10, kMend = 11;
constexpr int kSegs = 4;                         // items told ahead
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
    int4 *cut;              // [CTAs] the item a part begins inside of: item, first and last part, rows
    int32_t *status;
    int U, RB, TG, gshift, cap, max_len, rows, whole, split, join_all;
    FastDiv by_rb, by_units;
    float scale;            // log2(e) / sqrt(d)

    __device__ __forceinline__ int live(int u) const
    {
        const int n = t.n ? t.n[by_units(u)] : t.T;
        return n < 0 || n > t.T ? -1 : n;
    }
};

// The part of one item that this CTA takes; rows = 0: there is none left.
struct __align__(16) Seg {
    int item, u, rb, n, live, nt;   // nt: tiles of the item
    int t0, t1;                     // this CTA's tiles of it
    int rows;                       // live rows of the item
    int mends;                      // value tiles to mend before the drafted tokens'
};

struct AttSmem {
    union {                 // read as float4
        float vote[2][kTile];   // votes of a tile's slots, and the next one's
        float2 ml[kTile];   // at an item's end: the rows' maxima and sums
    } g[2];
    Seg seg[kSegs];
    int4 cut;
    int4 mend[4];           // a value tile to mend: ring entry (-1: no more), phase, valid slots, drafted tokens'
    uint64_t full[kRing], empty[kRing];
    uint64_t segfull[kSegs], segempty[kSegs];
    uint64_t qfull[2], qempty[2];
    uint64_t sfull[2], pready[2][2];    // by group; by group and half of the tile
    uint64_t ohalf[2], odone[2];        // O of a tile's first half; of the group's last tile
    uint64_t gsync[2], xsync, drain;
    uint64_t armed[4], mended[4];
    uint64_t odd[4];        // drafted tokens with a value that is not finite
    int scan[kThreads / 32];
    int start_item, start_base;
    int bad;
    uint32_t tmem;
};

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

// 32 columns of 16 lanes: thread t has columns 8 b + 2 (t % 4) and the next of
// lane t / 4 in r[4 b], r[4 b + 1], and of lane t / 4 + 8 in the two after.
__device__ __forceinline__ void tmem_ld_16x256(uint32_t addr, uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
        "%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
          "=r"(r[14]), "=r"(r[15])
        : "r"(addr)
        : "memory");
}

// Pairs f[2 j], f[2 j + 1] of the four lanes of a quad as a 4 x 4 matrix,
// transposed: lane i's pair j becomes lane j's pair i.
__device__ __forceinline__ void quad_transpose(float (&f)[8], int lane)
{
#pragma unroll
    for (int s = 1; s < 4; s <<= 1) {
        const bool up = lane & s;
#pragma unroll
        for (int j = 0; j < 4; j++) {
            if (j & s) continue;
#pragma unroll
            for (int e = 0; e < 2; e++) {
                float &x = f[2 * j + e], &y = f[2 * (j + s) + e];
                const float got = __shfl_xor_sync(kFull, up ? x : y, s);
                if (up) x = got;
                else y = got;
            }
        }
    }
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
    if (n < 0 || n > a.max_len || live < 0 || (live << a.gshift) <= rb * kRows) return 0;
    return ((n + kTile - 1) >> 7) + 1;
}

__device__ __forceinline__ void check_unit(const AttArgs &a, int u)
{
    const int n = a.len[u], live = a.live(u);
    if (live < 0) record_status(a.status, KVC_ERR_INVALID_ARG);
    else if (n < 0 || n > a.max_len) record_status(a.status, KVC_ERR_SHAPE);
}

// Value rows that the MMA reads (16 at a time) and that are no slot, or drafted
// tokens: the tile is mended first.
__device__ __forceinline__ bool needs_mend(const Seg &s, int t)
{
    return t == s.nt - 1 || (t == s.nt - 2 && (s.n & 15));
}

// valid slots of tile t (the drafted tokens' tile: the live ones)
__device__ __forceinline__ int tile_valid(const Seg &s, int t)
{
    return t == s.nt - 1 ? s.live : min(kTile, s.n - t * kTile);
}

// The value of a load is used from here on (the compiler would convert it, and
// so wait for it, right behind the load).
__device__ __forceinline__ void late(int &x) { asm volatile("" : "+r"(x)); }
__device__ __forceinline__ void late(uint64_t &x) { asm volatile("" : "+l"(x)); }

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

// Hidden slots of 32 raw products: -inf.
template <bool kMask>
__device__ __forceinline__ void hide32(uint32_t (&y)[32], uint32_t keep)
{
    if (kMask)
#pragma unroll
        for (int j = 0; j < 32; j++) y[j] = keep >> j & 1 ? y[j] : 0xff800000u;
}

// A new maximum of the row: m, l and (rescale) the row of O follow it once it
// is above m by kSlack.
template <typename F>
__device__ __forceinline__ void move_max(float top, uint32_t tO, bool rescale, float &m, float &l, F before_o)
{
    const bool move = top > m + kSlack || (m == -INFINITY && top > m);
    if (__any_sync(kFull, move)) {
        float f = 1.f;
        if (move) {
            f = m == -INFINITY ? 0.f : ex2_approx(m - top);
            m = top;
            l *= f;
        }
        if (rescale) {
            before_o();
#pragma unroll 1
            for (int h = 0; h < 8; h++) {
                uint32_t z[16];
                tmem_ld16_async(tO + 16 * h, z);
                tmem_wait_ld();
                tmem_bind16(z);
#pragma unroll
                for (int j = 0; j < 16; j++) z[j] = __float_as_uint(__uint_as_float(z[j]) * f);
                tmem_st16(tO + 16 * h, z);
            }
        }
    }
}

// The weights of 32 raw products, added to sum and written to P as bf16 pairs.  The
// sum is of the weights before that rounding; each product of O is off by at most
// half a step of bf16, which is what o is rounded to itself (a second term for the
// rest would cost O's product a second time, 1024 of a tile's 3600 clocks with two
// halves of rows).
template <bool kVotes>
__device__ __forceinline__ void weights32(const uint32_t (&y)[32], uint32_t at, const float *v, float2 c2,
                                          float2 r2, float2 (&sum)[2])
{
            uint32_t p[16];
    #pragma unroll
            for (int j = 0; j < 16; j += 2) {
                float2 e[2];
    #pragma unroll
                for (int i = 0; i < 2; i++) {
                    const float2 x = make_float2(__uint_as_float(y[2 * (j + i)]),
                                                 __uint_as_float(y[2 * (j + i) + 1]));
                    const float2 t = fma2(x, c2, r2);
                    e[i] = make_float2(ex2_approx(t.x), ex2_approx(t.y));
                }
                if (kVotes) {
                    const float4 w = *reinterpret_cast<const float4 *>(v + 2 * j);
                    e[0].x *= w.x;
                    e[0].y *= w.y;
                    e[1].x *= w.z;
                    e[1].y *= w.w;
                }
    #pragma unroll
                for (int i = 0; i < 2; i++) {
                    sum[i] = add2(sum[i], e[i]);
                    p[j + i] = pack_bf16(e[i].x, e[i].y);
                }
            }
            tmem_st16(at, p);
}

// The largest of 32 raw products (hidden ones: -inf), kept in mx.
template <bool kMask>
__device__ __forceinline__ void top32(uint32_t (&y)[32], uint32_t keep, float (&mx)[2])
{
    hide32<kMask>(y, keep);
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
        mx[0] = fmaxf(fmaxf(mx[0], __uint_as_float(y[j])), __uint_as_float(y[j + 1]));
        mx[1] = fmaxf(fmaxf(mx[1], __uint_as_float(y[j + 2])), __uint_as_float(y[j + 3]));
    }
}

// 64 slots of the thread's row: the row's maximum so far, the weights, which
// replace S as bf16 pairs in the first 32 of the columns, and their sum.  A slot's
// vote multiplies its weight (exp(x + ln p) = p exp(x)).  All 64 products stay in
// registers meanwhile.  before_o() is called before O is rescaled.
template <bool kMask, bool kVotes, typename F>
__device__ __forceinline__ void softmax_half(uint32_t tS, uint32_t tO, float scale, const float *vote,
                                             uint64_t keep, bool rescale, float &m, float &l, F before_o)
{
    uint32_t a[32], b[32];
    float mx[2] = {-INFINITY, -INFINITY};
    tmem_ld32_async(tS, a);
    tmem_ld32_async(tS + 32, b);
    tmem_wait_ld();
    tmem_bind(a);
    tmem_bind(b);
    top32<kMask>(a, (uint32_t)keep, mx);
    top32<kMask>(b, (uint32_t)(keep >> 32), mx);
    move_max(fmaxf(mx[0], mx[1]) * scale, tO, rescale, m, l, before_o);
    const float nref = m == -INFINITY ? 0.f : -m;
    const float2 c2 = make_float2(scale, scale), r2 = make_float2(nref, nref);
    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    weights32<kVotes>(a, tS, vote, c2, r2, sum);
    weights32<kVotes>(b, tS + 16, vote + 32, c2, r2, sum);
    l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
}

template <bool kVotes>
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

    if (warp == kProd && lane < 5) {
        const CUtensorMap *m = lane == 0 ? &tmK : lane == 1 ? &tmV : lane == 2 ? &tmQ
                               : lane == 3 ? &tmKt : &tmVt;
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
    }
    if (tid == 0) {
        S.bad = 0;
        for (int i = 0; i < kRing; i++) {
            mbar_init(&S.full[i], 1);
            mbar_init(&S.empty[i], 1);
        }
        for (int i = 0; i < kSegs; i++) {
            mbar_init(&S.segfull[i], 1);
            mbar_init(&S.segempty[i], 10);       // eight softmax warps, producer, issuer
        }
        for (int i = 0; i < 2; i++) {
            mbar_init(&S.qfull[i], 1);
            mbar_init(&S.qempty[i], 1);
            mbar_init(&S.sfull[i], 1);
            mbar_init(&S.pready[i][0], 4);
            mbar_init(&S.pready[i][1], 4);
            mbar_init(&S.ohalf[i], 1);
            mbar_init(&S.odone[i], 1);
            mbar_init(&S.gsync[i], 4);
        }
        for (int i = 0; i < 4; i++) {
            mbar_init(&S.armed[i], 1);
            mbar_init(&S.mended[i], 1);
        }
        mbar_init(&S.xsync, 8);
        mbar_init(&S.drain, 1);
        S.cut = make_int4(-1, 0, 0, 0);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == kMma) tmem_alloc(&S.tmem, 512);
    follow();
    lead();

    // this CTA's items [item0, item1) and tiles [lo, hi) of the line
    int item0, item1, base0, lo, hi;
    if (a.split) {
        // each item in as many parts, a CTA each (fewer when it has fewer tiles)
        const int item = blockIdx.x / a.split, sub = blockIdx.x - item * a.split;
        const int u = a.by_rb(item), rb = item - u * a.RB, live = a.live(u);
        const int nt = item_tiles(a, a.len[u], live, rb), parts = min(a.split, nt);
        item0 = item;
        item1 = item + 1;
        base0 = 0;
        lo = sub < parts ? nt * sub / parts : 0;
        hi = sub < parts ? nt * (sub + 1) / parts : 0;
        if (tid == 0) {
            if (sub == 1 && parts > 1)
                S.cut = make_int4(item, blockIdx.x - 1, blockIdx.x + parts - 2,
                                  min(kRows, (live << a.gshift) - rb * kRows));
            a.cut[blockIdx.x] = S.cut;
            if (sub == 0 && rb == 0) check_unit(a, u);
        }
    } else if (a.whole) {
        // parts of whole items: nothing to count, nothing to join
        const LineCuts c(gridDim.x, items);
        item0 = c.start(blockIdx.x);
        item1 = c.start(blockIdx.x + 1);
        base0 = lo = 0;
        hi = 0x7fffffff;
        if (blockIdx.x == 0)
            for (int u = tid; u < a.U; u += kThreads) check_unit(a, u);
    } else {
        // every CTA counts the line and finds where its part starts
        const int per = (items + kThreads - 1) / kThreads;
        const int i0 = min(items, tid * per), i1 = min(items, i0 + per);
        int sum = 0;
        for (int i = i0; i < i1; i++) {
            const int u = a.by_rb(i);
            sum += item_tiles(a, a.len[u], a.live(u), i - u * a.RB);
            if (blockIdx.x == 0 && i == u * a.RB) check_unit(a, u);
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
        for (int i = i0; i < i1; i++) {
            const int u = a.by_rb(i);
            const int nt = item_tiles(a, a.len[u], a.live(u), i - u * a.RB);
            if (blockIdx.x == 0) a.first[i] = b;
            if (lo >= b && lo < b + nt) {
                S.start_item = i;
                S.start_base = b;
                // the part before has the item's start: this CTA names its parts
                if (lo > b && b >= c.start(bid - 1)) S.cut = make_int4(
                        i, bid - 1, c.part(b + nt - 1),
                        min(kRows, (a.live(u) << a.gshift) - (i - u * a.RB) * kRows));
            }
            b += nt;
            if (blockIdx.x == 0 && i == items - 1) a.first[items] = b;
        }
        __syncthreads();
        if (tid == 0) a.cut[blockIdx.x] = S.cut;
        item0 = lo < hi ? S.start_item : items;
        item1 = items;
        base0 = S.start_base;
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = S.tmem;

    if (warp == kWalk) {
        // --------------------------------------------------------- walker
        if (elect_one()) {
            int item = item0, base = base0, mends = 0, n = 0, live = 0;
            bool ok = true;
            if (item < item1) {
                n = a.len[a.by_rb(item)];
                live = a.live(a.by_rb(item));
            }
            for (int i = 0; ok; ) {
                Seg s;
                s.rows = 0;
                if (item < item1 && base < hi) {
                    s.item = item;
                    s.u = a.by_rb(item);
                    s.rb = item - s.u * a.RB;
                    s.n = n;
                    s.live = live;
                    s.nt = item_tiles(a, n, live, s.rb);
                    s.t0 = max(0, lo - base);
                    s.t1 = min(s.nt, hi - base);
                    base += a.whole ? 0 : s.nt;
                    if (++item < item1) {
                        n = a.len[a.by_rb(item)];
                        live = a.live(a.by_rb(item));
                    }
                    if (s.t1 <= s.t0) continue;
                    s.rows = min(kRows, (s.live << a.gshift) - s.rb * kRows);
                    mends += s.t0 <= s.nt - 2 && s.t1 >= s.nt - 1 && (s.n & 15);
                    s.mends = mends;
                    mends += s.t1 == s.nt;
                }
                if (i >= kSegs) ok = tree_wait(&S.segempty[i % kSegs], (i / kSegs - 1) & 1, &S.bad);
                if (!ok) break;
                S.seg[i % kSegs] = s;
                mbar_arrive(&S.segfull[i % kSegs]);
                i++;
                if (s.rows == 0) break;
            }
        }
        __syncwarp();
    } else if (warp == kProd) {
        // ------------------------------------------------------- producer
        if (elect_one()) {
            int k = 0, slot = 0, mends = 0, qn[2] = {0, 0};
            uint32_t ph = 1;                     // phase of the slot's last release
            bool ok = true;
            const uint64_t pol = l2_policy_evict_first();
            auto load = [&](const CUtensorMap *m, int u, int row, int rows, bool stream) {
                if (k >= kRing) ok = ok && tree_wait(&S.empty[slot], ph, &S.bad);
                if (!ok) return;
                unsigned char *d = ring + slot * kSlot;
                const int boxes = rows > 64 ? 2 : 1;
                mbar_expect_tx(&S.full[slot], boxes * kHalf);
#pragma unroll
                for (int h = 0; h < 2; h++)
                    for (int b = 0; b < boxes; b++) {
                        unsigned char *at = d + h * kHalf + b * (kHalf / 2);
                        if (stream) tma_3d_hint(at, m, 64 * h, row + 64 * b, u, &S.full[slot], pol);
                        else tma_3d(at, m, 64 * h, row + 64 * b, u, &S.full[slot]);
                    }
                k++;
                if (++slot == kRing) { slot = 0; ph ^= 1; }
            };
            // Told once the entry's phase has begun, so that the wait for it cannot end
            // with an earlier one.  At most three value tiles are in the ring: the fourth
            // place is free when it is needed.
            auto tell = [&](int entry, int nv, bool tree) {
                if (!ok) return;
                S.mend[mends & 3] = make_int4(entry, (k - 1) / kRing & 1, nv, tree);
                mbar_arrive(&S.armed[mends & 3]);
                mends++;
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
            for (int i = 0; ok; i++) {
                ok = tree_wait(&S.segfull[i % kSegs], (i / kSegs) & 1, &S.bad);
                if (!ok) break;
                const Seg s = S.seg[i % kSegs];
                mbar_arrive(&S.segempty[i % kSegs]);
                if (s.rows == 0) {
                    tell(-1, 0, false);
                    break;
                }
                const int qrow = s.rb * kRows;
                if (s.rows > 128) {
                    load_q(0, s.u, qrow, 128);
                    load_q(1, s.u, qrow + 128, s.rows - 128);
                } else {
                    // the halves alternate, so the next item's rows load early;
                    // an item of two halves takes both, whichever was last
                    load_q(i & 1, s.u, qrow, s.rows);
                }
                auto load_tile = [&](bool keys, int t) {
                    const bool tree = t == s.nt - 1;
                    const int nv = tree ? 64 : s.n - t * kTile, row = tree ? 0 : t * kTile;
                    const int entry = slot;
                    load(keys ? (tree ? &tmKt : &tmK) : (tree ? &tmVt : &tmV), s.u, row, nv,
                         !tree && a.RB == 1);
                    if (!keys && needs_mend(s, t)) tell(entry, tile_valid(s, t), tree);
                };
                // in the order of their use, so that no tile waits in the ring for
                // one behind it: alternate tiles have two S before the first O
                const int ahead = s.rows > 128 ? 1 : 2, nq = s.t1 - s.t0;
                for (int t = 0; ok && t < nq + ahead; t++) {
                    if (ahead == 2 && t >= ahead) load_tile(false, s.t0 + t - ahead);
                    if (t < nq) load_tile(true, s.t0 + t);
                    if (ahead == 1 && t < nq) load_tile(false, s.t0 + t);
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
            // next ring entry and its phase; the entries in use by S and by O (a byte of each
            // group)
            int slot = 0, mends = 0;
            uint32_t k_at = 0, v_at = 0;
            uint32_t ph = 0, q_ph = 0, p_ph = 0;             // phases; by half of q, by group and half as bits
            const uint64_t q0 = umma_sdesc(smem_u32(qbuf)), k0 = umma_sdesc(smem_u32(ring));
            const uint64_t v0 = v_desc(smem_u32(ring));
            constexpr uint32_t kStep = kSlot >> 4;           // a slot in descriptor units
            auto take = [&](uint32_t &at, uint32_t g) {      // the next entry, once it is there
                ok = ok && tree_wait(&S.full[slot], ph, &S.bad);
                at = (at & ~(0xffu << 8 * g)) | (uint32_t)slot << 8 * g;
                if (++slot == kRing) { slot = 0; ph ^= 1; }
            };
            // S of group w; the key tile is waited for by its first reader and given back by
            // its last; g: whose entry it is (two halves of rows share theirs)
            auto issue_s = [&](uint32_t w, uint32_t half, uint32_t g, int nv, bool first, bool last) {
                if (first) take(k_at, g);
                if (!ok) return;
                const uint32_t entry = k_at >> 8 * g & 0xff, idesc = nv <= 64 ? kIdescS64 : kIdescS;
                tc_fence_after();
                const uint32_t d = tmem + kColS + 128 * w;
                const uint64_t qd = q0 + half * kStep, kd = k0 + entry * kStep;
#pragma unroll
                for (int ks = 0; ks < 8; ks++)
                    umma_bf16(d, umma_sdesc_step(qd, ks), umma_sdesc_step(kd, ks), idesc, ks > 0);
                umma_commit(&S.sfull[w]);
                if (last) umma_commit(&S.empty[entry]);
            };
            // O of group w from a tile's nv slots, 16 a step, its second half once the softmax
            // has handed that over too; end: the group's last tile of the item
            auto issue_o = [&](uint32_t w, uint32_t g, int nv, bool mend, bool first, bool last, bool keep,
                               bool end) {
                if (first) take(v_at, g);
                if (first && mend) {
                    ok = ok && tree_wait(&S.mended[mends & 3], mends >> 2 & 1, &S.bad);
                    mends++;
                }
                auto half = [&](uint32_t h) {
                    ok = ok && tree_wait(&S.pready[w][h], p_ph >> (2 * h + w) & 1, &S.bad);
                    p_ph ^= 1u << (2 * h + w);
                    tc_fence_after();
                    return ok;
                };
                const uint32_t entry = v_at >> 8 * g & 0xff;
                const uint64_t vd = v0 + entry * kStep;
                const uint32_t d = tmem + 128 * w, p = tmem + kColS + 128 * w;
                auto step = [&](int ks) {
                    umma_ts(d, p + 8 * ks + 32 * (ks >> 2), vd + (uint64_t)(ks * (2048 >> 4)), kIdescO, keep || ks > 0);
                };
                if (!half(0)) return;
                if (nv > kTile - 16) {
#pragma unroll
                    for (int ks = 0; ks < 4; ks++) step(ks);
                    umma_commit(&S.ohalf[w]);
                    if (!half(1)) return;
#pragma unroll
                    for (int ks = 4; ks < 8; ks++) step(ks);
                } else {
                    for (int ks = 0; 16 * ks < nv; ks++) {
                        if (ks == 4) {
                            umma_commit(&S.ohalf[w]);
                            if (!half(1)) return;
                        }
                        step(ks);
                    }
                }
                if (last) umma_commit(&S.empty[entry]);
                if (end) umma_commit(&S.odone[w]);
            };
            auto wait_q = [&](uint32_t half) {
                ok = ok && tree_wait(&S.qfull[half], q_ph >> half & 1, &S.bad);
                q_ph ^= 1u << half;
            };
            for (int i = 0; ok; i++) {
                ok = tree_wait(&S.segfull[i % kSegs], (i / kSegs) & 1, &S.bad);
                if (!ok) break;
                const Seg s = S.seg[i % kSegs];
                mbar_arrive(&S.segempty[i % kSegs]);
                if (s.rows == 0) break;
                const int nq = s.t1 - s.t0;
                const uint32_t dual = s.rows > 128;
                // job j: tile j of the group j & 1, or with two halves of rows tile j / 2 of the
                // half j & 1.  S comes whole, O in halves: the first runs under the softmax of
                // the second.
                const int jobs = nq << dual;
                // whole tiles need no closer look (the issuer's instructions are what a tile
                // of two halves of rows waits for)
                const int whole = min(s.t1, s.n >> 7) - s.t0;
                if (dual) {
                    wait_q(0);
                    wait_q(1);
                } else {
                    wait_q(i & 1);
                }
                for (int j = 0; ok && j < jobs + 2; j++) {
                    const uint32_t w = j & 1, g = dual ? 0 : w, first = !dual || !w, last = !dual || w;
                    const int before = (j - 2) >> dual, now = j >> dual;
                    if (j >= 2) {
                        const bool easy = before < whole;
                        issue_o(w, g, easy ? kTile : tile_valid(s, s.t0 + before),
                                !easy && needs_mend(s, s.t0 + before), first, last, j - 2 >= 2, j >= jobs);
                    }
                    if (j < jobs)
                        issue_s(w, dual ? w : i & 1, g, now < whole ? kTile : tile_valid(s, s.t0 + now), first, last);
                    if (j == jobs - 1) {
                        if (dual || !(i & 1)) umma_commit(&S.qempty[0]);
                        if (dual || (i & 1)) umma_commit(&S.qempty[1]);
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
    } else if (warp == kMend) {
        // --------------------------------------------------------- mender
        bool ok = true;
        for (int x = 0; ok; x++) {
            ok = __all_sync(kFull, tree_wait(&S.armed[x & 3], x >> 2 & 1, &S.bad));
            if (!ok) break;
            const int4 f = S.mend[x & 3];
            if (f.x < 0) break;
            ok = __all_sync(kFull, tree_wait(&S.full[f.x], f.y, &S.bad));
            if (!ok) break;
            unsigned char *v = ring + f.x * kSlot;
            const int nv = f.z, stop = (nv + 15) & ~15;
            uint64_t odd = 0;
            // two rows of 16 chunks at a time: rows that are no slot become zero; of a
            // drafted token, what is not finite does, and is added to the rows that see
            // it at the end
#pragma unroll 4
            for (int r0 = f.w ? 0 : nv & ~1; r0 < stop; r0 += 2) {
                const int c = lane & 15, r = r0 + (lane >> 4);
                uint4 *p = reinterpret_cast<uint4 *>(v + (c >> 3) * kHalf + r * 128 + (((c & 7) ^ (r & 7)) << 4));
                const uint4 y = *p;
                uint32_t w[4] = {y.x, y.y, y.z, y.w};
                bool hit = false;
                if (f.w)
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        if ((w[e] & 0x7f80u) == 0x7f80u) { w[e] &= 0xffff0000u; hit = true; }
                        if ((w[e] & 0x7f800000u) == 0x7f800000u) { w[e] &= 0x0000ffffu; hit = true; }
                    }
                if (r >= nv) *p = make_uint4(0, 0, 0, 0);
                else if (hit) *p = make_uint4(w[0], w[1], w[2], w[3]);
                const unsigned bits = __ballot_sync(kFull, hit && r < nv);
                if (bits) odd |= (uint64_t)((bits & 0xffffu ? 1 : 0) | (bits >> 16 ? 2 : 0)) << r0;
            }
            if (lane == 0) S.odd[x & 3] = odd;
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.mended[x & 3]);
        }
        if (!ok && lane == 0) S.bad = 1;
    } else {
        // --------------------------------------------------------- softmax
        const int w = warp >> 2, r = tid & 127;              // group, row of its 128
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lanes + kColS + 128 * w, tO = tmem + lanes + 128 * w;
        uint32_t tiles = 0, gph = 0, xph = 0;                // tiles so far; barrier phases
        uint32_t half_ph = 0, done_ph = 0;                   // phases of ohalf and odone
        bool ok = true;
        auto wait = [&](uint64_t *b, uint32_t ph) {
            const bool x = tree_wait(b, ph, &S.bad);
            ok = __all_sync(kFull, x);
        };
        // barriers of the group's 128 threads and of all 256
        auto group_sync = [&] {
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.gsync[w]);
            wait(&S.gsync[w], gph);
            gph ^= 1;
        };
        auto all_sync = [&] {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.xsync);
            wait(&S.xsync, xph);
            xph ^= 1;
            tc_fence_after();
        };
        // what a thread needs of the next item from global memory: the drafted tokens its
        // row sees, the first votes
        uint64_t see_next = 0;
        int vote_first = 1;
        auto peek = [&](int i) {
            wait(&S.segfull[i % kSegs], (i / kSegs) & 1);
            if (!ok) return;
            const volatile Seg &s = S.seg[i % kSegs];
            const int rows = s.rows, u = s.u, row = (rows > 128 ? 128 * w : 0) + r;
            see_next = 0;
            if (row < rows)
                see_next = a.t.mask[(size_t)a.by_units(u) * a.t.T + ((s.rb * kRows + row) >> a.gshift)];
            if (kVotes) {
                const int at = (s.t0 + (rows > 128 ? 0 : w)) * kTile + r;
                vote_first = rows > 0 && at < s.n ? a.votes[(size_t)u * a.cap + at] : 1;
            }
        };
        peek(0);
        for (int i = 0; ok; i++) {
            const volatile Seg &s = S.seg[i % kSegs];
            const int rows = s.rows;
            if (rows == 0) break;
            const bool dual = rows > 128;
            const int step = dual ? 1 : 2;
            const int row = (dual ? 128 * w : 0) + r;        // row of the item
            const bool busy = row - lane < rows;             // the warp has rows
            late(see_next);
            late(vote_first);
            const int live = s.live;
            const uint64_t see = see_next & (live >= 64 ? ~0ull : (1ull << live) - 1);
            float m = -INFINITY, l = 0.f;
            bool begun = false;                              // O has a tile's product
            // the first tile's votes (a group without a tile here must not write: the
            // maxima and sums of the item's end share the space)
            if (kVotes && s.t0 + (dual ? 0 : w) < s.t1) {
                S.g[w].vote[tiles & 1][r] = (float)vote_first;
                group_sync();
                if (!ok) break;
            }
            for (int tile = s.t0 + (dual ? 0 : w); tile < s.t1; tile += step) {
                const bool tree = tile == s.nt - 1;
                const int nv = tree ? s.live : min(kTile, s.n - tile * kTile);
                // the next tile's votes, on their way while S is waited for
                int vote_next = 1;
                if (kVotes) {
                    const int at = (tile + step) * kTile + r;
                    if (at < s.n) vote_next = a.votes[(size_t)s.u * a.cap + at];
                }
                wait(&S.sfull[w], tiles & 1);
                if (!ok) break;
                tc_fence_after();
                // S was issued when all four warps had handed over the group's last weights:
                // they are done with the other buffer, and this one has been written
                if (kVotes) {
                    late(vote_next);
                    S.g[w].vote[(tiles + 1) & 1][r] = (float)vote_next;
                }
                // half by half: O of the first is made under the softmax of the second
#pragma unroll 1
                for (int h = 0; h < 2 && 64 * h < nv; h++) {
                    if (busy) {
                        const float *vote = S.g[w].vote[tiles & 1] + 64 * h;
                        // O must not be in the making when it is rescaled.  What came before
                        // this S is done (MMAs are in order); the first half's O need not be.
                        // The one before that is, so the parity is not an earlier phase's.
                        auto before_o = [&] {
                            if (h == 0) return;
                            wait(&S.ohalf[w], half_ph);
                            tc_fence_after();
                        };
                        if (tree || nv < 64 * h + 64) {
                            const uint64_t keep = tree ? see : (1ull << (nv - 64 * h)) - 1;
                            softmax_half<true, kVotes>(tS + 64 * h, tO, a.scale, vote, keep, begun, m, l, before_o);
                        } else {
                            softmax_half<false, kVotes>(tS + 64 * h, tO, a.scale, vote, 0, begun, m, l, before_o);
                        }
                        tmem_wait_st();
                    }
                    begun = true;
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&S.pready[w][h]);
                }
                if (!ok) break;
                tiles++;
                half_ph ^= nv > 64;
            }
            // ------------------------------------------------------ outputs
            if (ok) peek(i + 1);
            if (ok && begun) {
                wait(&S.odone[w], done_ph);
                done_ph ^= 1;
            }
            if (ok && s.t1 == s.nt) wait(&S.mended[s.mends & 3], s.mends >> 2 & 1);   // S.odd is written
            if (!ok) break;
            tc_fence_after();
            const int u = s.u, nq = s.t1 - s.t0;
            const bool direct = nq == s.nt && !a.join_all;   // nothing to join
            const bool has_tree = s.t1 == s.nt;
            float c0 = 1.f, c1 = 0.f, M = m, L = l;          // weights of the groups' sums
            if (!dual) S.g[w].ml[r] = make_float2(m, l);
            if (!dual) {
                all_sync();
                if (!ok) break;
                const float2 p0 = S.g[0].ml[r], p1 = S.g[1].ml[r];
                M = fmaxf(p0.x, p1.x);
                const float ref = M == -INFINITY ? 0.f : M;
                c0 = ex2_approx(p0.x - ref);
                c1 = ex2_approx(p1.x - ref);
                L = p0.y * c0 + p1.y * c1;
            }
            const size_t part = ((size_t)s.item + blockIdx.x) * a.rows + row;
            const size_t orow = (size_t)u * a.TG + (size_t)(s.rb * kRows + row);
            if (direct) {
                const float inv = L == 0.f ? 0.f : 1.f / L;
                c0 *= inv;
                c1 *= inv;
            }
            const uint64_t by_hand = has_tree ? S.odd[s.mends & 3] & see : 0;
            // a group writes its rows whole, or (alternate tiles) half of the columns
            const int q0 = dual ? 0 : 2 * w, q1 = dual ? 4 : q0 + 2;
            const bool two = !dual && nq > 1, mine = row < rows;
            if (busy) {
                // 32 columns of 16 rows at a time, in the layout that gives a thread two
                // columns of every eight; a transposition in each quad of lanes leaves it
                // eight in a row, so that a store covers whole lines
                uint32_t y[16], z[16];
                auto fetch = [&](int q) {
                    const uint32_t at = tmem + lanes + ((uint32_t)(16 * (q & 1)) << 16) + 32 * (q >> 1);
                    tmem_ld_16x256(at + (dual ? 128 * w : 0), y);
                    if (two) tmem_ld_16x256(at + 128, z);
                };
                fetch(2 * q0);
#pragma unroll 1
                for (int q = 2 * q0; q < 2 * q1; q++) {
                    const int h = q & 1, col = 32 * (q >> 1) + 8 * (lane & 3);
                    float f[2][8];
                    tmem_wait_ld();
                    tmem_bind16(y);
                    if (two) tmem_bind16(z);
#pragma unroll
                    for (int k = 0; k < 2; k++) {            // rows (lane / 4) and 8 more
                        const int of = 16 * h + 8 * k + (lane >> 2);
                        const float a0 = __shfl_sync(kFull, c0, of), a1 = __shfl_sync(kFull, c1, of);
#pragma unroll
                        for (int j = 0; j < 4; j++)
#pragma unroll
                            for (int e = 0; e < 2; e++) {
                                f[k][2 * j + e] = __uint_as_float(y[4 * j + 2 * k + e]) * a0;
                                if (two) f[k][2 * j + e] = fmaf(__uint_as_float(z[4 * j + 2 * k + e]), a1, f[k][2 * j + e]);
                            }
                    }
                    if (q + 1 < 2 * q1) fetch(q + 1);
#pragma unroll
                    for (int k = 0; k < 2; k++) quad_transpose(f[k], lane);
#pragma unroll
                    for (int k = 0; k < 2; k++) {
                        const int of = 16 * h + 8 * k + (lane >> 2), r2 = row - lane + of;
                        if (r2 >= rows) continue;
                        if (direct) {
                            *reinterpret_cast<uint4 *>(a.o + (orow - lane + of) * kD + col) =
                                make_uint4(pack_bf16(f[k][0], f[k][1]), pack_bf16(f[k][2], f[k][3]),
                                           pack_bf16(f[k][4], f[k][5]), pack_bf16(f[k][6], f[k][7]));
                        } else {
                            st_v8(a.part + (part - lane + of) * kD + col, reinterpret_cast<const uint32_t *>(f[k]));
                        }
                    }
                }
                // drafted tokens that the row sees and whose value is not finite: whatever
                // their weight, the output of such a column is not finite
                if (__any_sync(kFull, by_hand != 0)) {
                    __syncwarp();                            // what other lanes wrote of this row
                    if (mine)
                        for (uint64_t rest = by_hand; rest; rest &= rest - 1) {
                            const uint16_t *vr =
                                a.vt + ((size_t)u * a.t.T + __ffsll((long long)rest) - 1) * kD;
#pragma unroll 1
                            for (int c = 32 * q0; c < 32 * q1; c++) {
                                const float v = bf2f(vr[c]);
                                if (isfinite(v)) continue;
                                volatile uint16_t *o = a.o + orow * kD + c;
                                volatile float *p = a.part + part * kD + c;
                                if (direct) *o = (uint16_t)pack_bf16(bf2f(*o) + v, 0.f);
                                else *p = *p + v;
                            }
                        }
                }
                if (mine && (dual || w == 0)) {
                    if (direct)
                        a.lse[orow] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
                    else
                        a.ml[part] = make_float2(M, L);
                }
            }
            // the other group reads this one's sums: both are done before either goes on
            if (!dual) all_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.segempty[i % kSegs]);
        }
        if (!ok && lane == 0) S.bad = 1;
    }
    __syncthreads();
    if (warp == kMma) tmem_dealloc(tmem, 512);
    if (tid == 0 && S.bad) record_status(a.status, KVC_ERR_TIMEOUT);
}

// The kernels behind the attention.
struct JoinArgs {
    AttArgs a;
    const float *mn, *mu_k, *mu_v, *C;
    int first_order, grid;
};

// The sums of a cut item's parts added.  A warp has two rows, a lane four of
// their columns; the loads of eight parts are in flight together (four: 8 units
// of 4096 slots 14.7 us and not 13.4; of 240 rows 23.3 and not 23.9).  The result
// is the output, or (kKeep, when the moments follow) the first part's place
// takes it.  grid (CTAs of the attention, rows / 16): block x takes the item
// whose first cut is the start of part x.  Bound by latency: about 5 us behind
// the attention for 8 units of 131071 slots (152 parts of 252 rows, 20 MB).
constexpr int kJoinRows = 2, kJoinAt = 8;

template <bool kKeep>
__global__ void __launch_bounds__(256) tree_join_kernel(const __grid_constant__ JoinArgs j)
{
    const AttArgs &a = j.a;
    lead();
    follow();
    const int4 cut = a.cut[blockIdx.x];                     // item, first and last part, rows
    const int lane = threadIdx.x & 31, r0 = kJoinRows * (blockIdx.y * 8 + (threadIdx.x >> 5));
    if (cut.x < 0 || r0 >= cut.w) return;
    const int nr = min(kJoinRows, cut.w - r0), np = cut.z - cut.y + 1;
    const size_t at = ((size_t)cut.x + cut.y) * a.rows + r0, step = (size_t)a.rows;
    float M[kJoinRows], L[kJoinRows];
    float4 f[kJoinRows];
#pragma unroll
    for (int i = 0; i < kJoinRows; i++) {
        M[i] = -INFINITY;
        L[i] = 0.f;
        f[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int k0 = 0; k0 < np; k0 += kJoinAt) {
        // places past the last part or row are read again and weigh nothing
        float2 ml[kJoinAt][kJoinRows];
        float4 p[kJoinAt][kJoinRows];
#pragma unroll
        for (int k = 0; k < kJoinAt; k++)
#pragma unroll
            for (int i = 0; i < kJoinRows; i++) {
                const size_t x = at + min(k0 + k, np - 1) * step + min(i, nr - 1);
                ml[k][i] = a.ml[x];
                p[k][i] = reinterpret_cast<const float4 *>(a.part + x * kD)[lane];
            }
#pragma unroll
        for (int k = 0; k < kJoinAt; k++)
#pragma unroll
            for (int i = 0; i < kJoinRows; i++) {
                if (k0 + k >= np) continue;
                const float m = fmaxf(M[i], ml[k][i].x), ref = m == -INFINITY ? 0.f : m;
                const float c = ex2_approx(M[i] - ref), e = ex2_approx(ml[k][i].x - ref);
                M[i] = m;
                L[i] = fmaf(L[i], c, ml[k][i].y * e);
                f[i].x = fmaf(f[i].x, c, p[k][i].x * e);
                f[i].y = fmaf(f[i].y, c, p[k][i].y * e);
                f[i].z = fmaf(f[i].z, c, p[k][i].z * e);
                f[i].w = fmaf(f[i].w, c, p[k][i].w * e);
            }
    }
    const int u = a.by_rb(cut.x), rb = cut.x - u * a.RB;
    const size_t row = (size_t)u * a.TG + (size_t)rb * kRows + r0;
    if (kKeep) __syncwarp();                                // all lanes have read ml
#pragma unroll
    for (int i = 0; i < kJoinRows; i++) {
        if (i >= nr) break;
        if (kKeep) {
            reinterpret_cast<float4 *>(a.part + (at + i) * kD)[lane] = f[i];
            if (lane == 0) a.ml[at + i] = make_float2(M[i], L[i]);
        } else {
            const float inv = L[i] == 0.f ? 0.f : 1.f / L[i];
            reinterpret_cast<uint2 *>(a.o + (row + i) * kD)[lane] =
                make_uint2(pack_bf16(f[i].x * inv, f[i].y * inv), pack_bf16(f[i].z * inv, f[i].w * inv));
            if (lane == 0)
                a.lse[row + i] = L[i] == 0.f ? -INFINITY : (M[i] + log2f(L[i])) * 0.6931471805599453f;
        }
    }
}

// The normalization correction: every row's sum normalised and mixed with the
// evicted set's estimate.  Bound by bytes: 64 KB of C per unit, 1 KB per row.
// A persistent CTA per SM takes 64 rows of an item at a time.  C q runs on
// tcgen05 with C as two bf16 terms (2^-16 of a product), which warps of their
// own take apart in registers.  The roles are apart so that C of the jobs to
// come keeps loading; each knows 32 jobs ahead of their use (a lane each).
// 1024 units of 64 rows: 33 us behind the attention (134 MB, 4 TB/s; 24 us of
// it with the inputs that load before the attention ends).  One group of warps
// for everything took 36 us and began at the attention's end.
//   warps 0, 1, 4, 5    outputs: a thread per row (the tensor-memory lanes of
//                       64 rows), half of the columns each
//   warps 2, 3, 6, 7    q . mu_k of the rows, mu_v
//   warps 8-15          C to bf16 terms, loaded half a job ahead
//   warp 16             producer of q and the sums (TMA), warp 17 MMA issuer
constexpr int kMomRows = 64;
constexpr int kMomThreads = 576;
constexpr int kMomQ = kMomRows * kD * 2, kMomF = kMomRows * kD * 4;
struct MomSmem {
    float muv[2][kD], z[2][kMomRows];
    // (two of each: a wait for one job's phase is never two phases behind)
    uint64_t ffull[2], fempty[2], zready[2], pready[2], mdone[2], dfree[2];
    int bad;
    uint32_t tmem;
};
// the two terms of C, of two jobs | q of two jobs | sums of two jobs
constexpr size_t kMomDyn = 4 * (size_t)kSlot + 2 * (kMomQ + kMomF) + sizeof(MomSmem);
static_assert(kMomDyn <= 227 * 1024, "one block's shared memory");

// One job: 64 rows of an item.  rows <= 0: nothing to do.
struct MomJob {
    int u, row0, rows, sid;       // unit, first row of it, rows, place of the sums
    int r0;                       // first row of the item
    float ne;

    // The unit has evicted tokens to mix in.  All roles ask this, so that none is a job
    // ahead of another; a count that is NaN mixes (as in kvc_correct) and stays in its unit.
    __device__ __forceinline__ bool mixes() const { return !(ne <= 0.f); }
};

// sums: the place of the sums is wanted, which is known after the attention.
__device__ __forceinline__ MomJob mom_job(const JoinArgs &j, bool sums, int per, int job)
{
    const AttArgs &a = j.a;
    MomJob m;
    const int item = job / per;
    m.u = a.by_rb(item);
    const int rb = item - m.u * a.RB, n = a.len[m.u], live = a.live(m.u);
    m.r0 = (job - item * per) * kMomRows;
    m.row0 = rb * kRows + m.r0;
    m.rows = n < 0 || n > a.max_len || live < 0
                 ? 0 : min(kMomRows, min(kRows, (live << a.gshift) - rb * kRows) - m.r0);
    m.ne = j.mn[m.u];
    // the part that has the item's start (its place has the joined sums)
    m.sid = 0;
    if (sums && m.rows > 0) {
        const int items = a.U * a.RB;
        const LineCuts cuts(j.grid, a.whole ? items : a.split ? 0 : a.first[items]);
        m.sid = item + (a.split ? item * a.split : cuts.part(a.whole ? item : a.first[item]));
    }
    return m;
}

// A CTA's jobs with rows, one after another, for a whole warp.
struct MomJobs {
    const JoinArgs &j;
    bool sums;
    int per, jobs, k;             // k: the next one, in steps of the grid
    MomJob mine;                  // lane i: job k - k % 32 + i

    __device__ __forceinline__ MomJobs(const JoinArgs &j, bool sums, int per, int jobs)
        : j(j), sums(sums), per(per), jobs(jobs), k(0)
    {
    }
    __device__ __forceinline__ bool next(MomJob &m)
    {
        for (;; k++) {
            if ((long long)k * gridDim.x + blockIdx.x >= jobs) return false;
            if ((k & 31) == 0) {
                const long long job = (long long)(k + (threadIdx.x & 31)) * gridDim.x + blockIdx.x;
                mine.rows = 0;
                if (job < jobs) mine = mom_job(j, sums, per, (int)job);
            }
            m.rows = __shfl_sync(kFull, mine.rows, k & 31);
            if (m.rows > 0) break;
        }
        m.u = __shfl_sync(kFull, mine.u, k & 31);
        m.row0 = __shfl_sync(kFull, mine.row0, k & 31);
        m.sid = __shfl_sync(kFull, mine.sid, k & 31);
        m.r0 = __shfl_sync(kFull, mine.r0, k & 31);
        m.ne = __shfl_sync(kFull, mine.ne, k & 31);
        k++;
        return true;
    }
};

__global__ void __launch_bounds__(kMomThreads, 1)
tree_moment_kernel(const __grid_constant__ JoinArgs j, const __grid_constant__ CUtensorMap tmQ,
                   const __grid_constant__ CUtensorMap tmF)
{
    const AttArgs &a = j.a;
    extern __shared__ __align__(1024) unsigned char dyn[];
    unsigned char *planes = dyn, *qs = planes + 4 * kSlot, *fs = qs + 2 * kMomQ;
    MomSmem &S = *reinterpret_cast<MomSmem *>(fs + 2 * kMomF);
    if (smem_u32(dyn) & 1023) {
        if (threadIdx.x == 0) record_status(a.status, KVC_ERR_CUDA);
        return;
    }
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int items = a.U * a.RB, per = (a.rows + kMomRows - 1) / kMomRows;
    if (tid == 0) {
        S.bad = 0;
        for (int i = 0; i < 2; i++) {
            mbar_init(&S.ffull[i], 1);
            mbar_init(&S.fempty[i], 8);
            mbar_init(&S.zready[i], 4);
            mbar_init(&S.pready[i], 8);
            mbar_init(&S.mdone[i], 1);
            mbar_init(&S.dfree[i], 4);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 17) tmem_alloc(&S.tmem, 256);
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = S.tmem;
    // the sums, the place they are at and the outputs wait for the kernels before; the
    // rest of this one reads what they only read
    const bool sums = warp == 16 || (warp < 8 && !(warp & 2));
    if (sums) follow();
    MomJobs list(j, sums, per, items * per);
    MomJob m;
    const float sd = rsqrtf((float)kD);
    bool ok = true;
    int kf = 0, kc = 0;                                      // jobs and products before
    auto wait = [&](uint64_t *b, uint32_t ph) { ok = ok && __all_sync(kFull, tree_wait(b, ph, &S.bad)); };
    auto arrive = [&](uint64_t *b) {
        __syncwarp();
        if (lane == 0) mbar_arrive(b);
    };
    if (warp == 16) {
        // -------------------------------------------------------- producer
        for (; ok && list.next(m); kf++) {
            const bool mix = m.mixes();
            const int st = kf & 1;
            if (kf >= 2) wait(&S.fempty[st], (kf / 2 - 1) & 1);
            if (!ok) break;
            if (elect_one()) {
                mbar_expect_tx(&S.ffull[st], kMomF + (mix ? kMomQ : 0));
                for (int i = 0; i < 4; i++)
                    tma_3d(fs + st * kMomF + i * (kMomF / 4), &tmF, 32 * i, m.r0, m.sid, &S.ffull[st]);
                if (mix)
                    for (int i = 0; i < 2; i++)
                        tma_3d(qs + st * kMomQ + i * (kMomQ / 2), &tmQ, 64 * i, m.row0, m.u, &S.ffull[st]);
            }
            __syncwarp();
        }
        // (after a wait that ran out: the copies in flight land before the block ends)
        if (!ok)
            for (int i = max(0, kf - 2); i < kf; i++) mbar_wait(&S.ffull[i & 1], (i / 2) & 1);
    } else if (warp == 17) {
        // ------------------------------------------------------ MMA issuer
        const uint64_t c0 = umma_sdesc(smem_u32(planes));
        for (; ok && list.next(m); kf++) {
            const int st = kf & 1;
            if (!m.mixes() || !j.first_order) continue;
            wait(&S.ffull[st], (kf / 2) & 1);
            wait(&S.pready[kc & 1], (kc >> 1) & 1);
            if (kc >= 2) wait(&S.dfree[kc & 1], ((kc >> 1) - 1) & 1);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
                // rows 64 .. 127 of the operand are whatever lies behind: their lanes
                // are not read
                const uint64_t q0 = umma_sdesc(smem_u32(qs + st * kMomQ));
                const uint32_t d = tmem + 128 * (kc & 1);
#pragma unroll
                for (int x = 0; x < 16; x++) {
                    const int ks = x & 7;
                    umma_bf16(d, q0 + (uint64_t)((ks >> 2) * (kMomQ / 2 >> 4) + (ks & 3) * 2),
                              umma_sdesc_step(c0 + (uint64_t)((2 * (kc & 1) + (x >> 3)) * (kSlot >> 4)), ks),
                              kIdescS, x > 0);
                }
                umma_commit(&S.mdone[kc & 1]);
            }
            __syncwarp();
            kc++;
        }
        // (after a wait that ran out: the MMAs issued before are done when mdone says so)
        if (!ok && kc > 0) mbar_wait(&S.mdone[(kc - 1) & 1], ((kc - 1) >> 1) & 1);
    } else if (warp >= 8) {
        // ------------------------------------------------- C to bf16 terms
        // 16-byte chunks of eight elements; half of a unit's are taken apart while the
        // other half is on its way
        const int t = tid - 256;
        float4 x[8], y[8];
        auto fetch = [&](float4 (&r)[8], int u, int half) {
            const float4 *C = reinterpret_cast<const float4 *>(j.C + (size_t)u * kD * kD);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const int e = 2 * ((4 * half + i) * 256 + t);
                r[2 * i] = C[e];
                r[2 * i + 1] = C[e + 1];
            }
        };
        auto terms = [&](const float4 (&r)[8], int half) {
            unsigned char *to = planes + (kc & 1) * 2 * kSlot;
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const int e = (4 * half + i) * 256 + t;
                const float4 x = r[2 * i], y = r[2 * i + 1];
                const uint4 hi = make_uint4(pack_bf16(x.x, x.y), pack_bf16(x.z, x.w), pack_bf16(y.x, y.y),
                                            pack_bf16(y.z, y.w));
                const uint4 lo = make_uint4(pack_bf16(x.x - bf_lo(hi.x), x.y - bf_hi(hi.x)),
                                            pack_bf16(x.z - bf_lo(hi.y), x.w - bf_hi(hi.y)),
                                            pack_bf16(y.x - bf_lo(hi.z), y.y - bf_hi(hi.z)),
                                            pack_bf16(y.z - bf_lo(hi.w), y.w - bf_hi(hi.w)));
                unsigned char *d = to + sw_off_t<128>(e >> 4, e & 15);
                *reinterpret_cast<uint4 *>(d) = hi;
                *reinterpret_cast<uint4 *>(d + kSlot) = lo;
            }
        };
        auto next = [&] {                                    // the next job with a product
            while (list.next(m))
                if (m.mixes()) return true;
            return false;
        };
        bool more = j.first_order && next();
        if (more) {
            fetch(x, m.u, 0);
            fetch(y, m.u, 1);
        }
        for (; more && ok; kc++) {
            more = next();
            if (kc > 1) wait(&S.mdone[kc & 1], ((kc >> 1) - 1) & 1);   // the terms of two jobs ago are used up
            if (!ok) break;
            terms(x, 0);
            if (more) fetch(x, m.u, 0);
            terms(y, 1);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            tc_fence_before();
            arrive(&S.pready[kc & 1]);
            if (more) fetch(y, m.u, 1);
        }
    } else if (warp & 2) {
        // ------------------------------------------------- q . mu_k, mu_v
        // 16 rows a warp, eight lanes a row of 16 dimensions (two 16-byte chunks)
        const int q = 16 * (2 * (warp >> 2) + (warp & 1)), dim = 32 * (q >> 4) + lane;
        float k0[16], k1[16];                                // the lane's part of mu_k, and of the next job's
        float v0 = 0.f, v1 = 0.f;
        auto fetch = [&](float (&k)[16], float &v) {
            if (!m.mixes()) return;
            const float *mk = j.mu_k + (size_t)m.u * kD + 8 * (lane & 7);
#pragma unroll
            for (int i = 0; i < 16; i++) k[i] = mk[64 * (i >> 3) + (i & 7)];
            v = j.mu_v[(size_t)m.u * kD + dim];
        };
        bool more = list.next(m);
        if (more) fetch(k0, v0);
        for (; more && ok; kf++) {
            const int st = kf & 1;
            const float ne = m.ne;
            const bool mix = m.mixes();
            more = list.next(m);
            if (more) fetch(k1, v1);
            wait(&S.ffull[st], (kf / 2) & 1);
            if (!ok) break;
            if (mix) {
                const float ln = logf(ne);
                float z[4];
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const int r = q + 4 * i + (lane >> 3);
                    z[i] = 0.f;
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        float f[8];
                        unpack8(lds_v4(qs + st * kMomQ + sw_off_t<64>(r, (lane & 7) + 8 * h)), f);
#pragma unroll
                        for (int e = 0; e < 8; e++) z[i] = fmaf(f[e], k0[8 * h + e], z[i]);
                    }
                }
#pragma unroll
                for (int d = 1; d < 8; d <<= 1)
#pragma unroll
                    for (int i = 0; i < 4; i++) z[i] += __shfl_xor_sync(kFull, z[i], d);
                if ((lane & 7) == 0)
#pragma unroll
                    for (int i = 0; i < 4; i++) S.z[st][q + 4 * i + (lane >> 3)] = ln + sd * z[i];
                S.muv[st][dim] = v0;
            }
            arrive(&S.zready[st]);
            arrive(&S.fempty[st]);
#pragma unroll
            for (int i = 0; i < 16; i++) k0[i] = k1[i];
            v0 = v1;
        }
    } else {
        // --------------------------------------------------------- outputs
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const int col0 = 64 * (warp >> 2), row = 32 * (warp & 3) + lane;
        auto fetch = [&] { return a.ml[(size_t)m.sid * a.rows + m.r0 + min(row, m.rows - 1)]; };
        float2 ml0 = make_float2(0.f, 0.f), ml1 = ml0;
        bool more = list.next(m);
        if (more) ml0 = fetch();
        for (; more && ok; kf++) {
            const int st = kf & 1, c = kc;
            const MomJob g = m;
            const bool mix = g.mixes(), prod = mix && j.first_order;
            more = list.next(m);
            if (more) ml1 = fetch();
            wait(&S.ffull[st], (kf / 2) & 1);
            wait(&S.zready[st], (kf / 2) & 1);
            if (prod) {
                wait(&S.mdone[c & 1], (c >> 1) & 1);
                kc++;
            }
            if (!ok) break;
            tc_fence_after();
            if (row - lane < g.rows) {
                const float lse = ml0.y == 0.f ? -INFINITY : (ml0.x + log2f(ml0.y)) * 0.6931471805599453f;
                const float w = mix ? 1.f / (1.f + expf(S.z[st][row] - lse)) : 1.f;
                const float wf = ml0.y == 0.f ? 0.f : w / ml0.y, we = 1.f - w, ws = we * sd;
                const size_t orow = (size_t)g.u * a.TG + (size_t)(g.row0 + row);
#pragma unroll 2
                for (int h = 0; h < 4; h++) {
                    const int c0 = col0 + 16 * h;
                    uint32_t y[16];
                    if (prod) {
                        tmem_ld16_async(tmem + lanes + 128 * (c & 1) + c0, y);
                        tmem_wait_ld();
                        tmem_bind16(y);
                    }
                    float o[16];
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        const float4 x = *reinterpret_cast<const float4 *>(
                            fs + st * kMomF + (c0 >> 5) * (kMomF / 4) + row * 128 +
                            (((((c0 & 31) >> 2) + i) ^ (row & 7)) << 4));
                        o[4 * i] = wf * x.x;
                        o[4 * i + 1] = wf * x.y;
                        o[4 * i + 2] = wf * x.z;
                        o[4 * i + 3] = wf * x.w;
                        if (mix) {
                            const float4 v = *reinterpret_cast<const float4 *>(&S.muv[st][c0 + 4 * i]);
                            o[4 * i] = fmaf(we, v.x, o[4 * i]);
                            o[4 * i + 1] = fmaf(we, v.y, o[4 * i + 1]);
                            o[4 * i + 2] = fmaf(we, v.z, o[4 * i + 2]);
                            o[4 * i + 3] = fmaf(we, v.w, o[4 * i + 3]);
                        }
                    }
                    if (prod)
#pragma unroll
                        for (int i = 0; i < 16; i++) o[i] = fmaf(ws, __uint_as_float(y[i]), o[i]);
                    uint32_t b[8];
#pragma unroll
                    for (int i = 0; i < 8; i++) b[i] = pack_bf16(o[2 * i], o[2 * i + 1]);
                    if (row < g.rows) {
                        uint4 *d = reinterpret_cast<uint4 *>(a.o + orow * kD + c0);
                        d[0] = make_uint4(b[0], b[1], b[2], b[3]);
                        d[1] = make_uint4(b[4], b[5], b[6], b[7]);
                    }
                }
                if (row < g.rows && col0 == 0) a.lse[orow] = lse;
            }
            tc_fence_before();
            if (prod) arrive(&S.dfree[c & 1]);
            arrive(&S.fempty[st]);
            ml0 = ml1;
        }
    }
    if (!ok && lane == 0) S.bad = 1;
    __syncthreads();
    lead();
    if (warp == 17) tmem_dealloc(tmem, 256);
    if (tid == 0 && S.bad) record_status(a.status, KVC_ERR_TIMEOUT);
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

// How the items go to the CTAs: whole, each cut into `split` parts of its own,
// or (neither) the line of all tiles cut into kGrid parts.
struct Cut {
    bool whole;
    int split;
};

// In units of one tile's bytes at the whole device's bandwidth (9.65 ns): a CTA
// takes 80 of them for a tile (170 with two halves of rows) however little else
// runs, and 152 when all of them load.  A join is 320 and the sums' way to
// memory and back.  Measured (us), whole / parts of their own / line: 8 units
// of 512 slots 10.8 / 11.0 / -, of 1024 slots 14.1 / 11.1 / -, of 4096 slots
// - / 13.6 / 18.6; 40 of 2432 slots 23.8 / 17.6 / 21.3; 80 of 1408 slots 18.5 /
// - / 22.3, with 240 rows 30.9 / - / 41.4; 128 of up to 3277 slots 36.7 / - / 43.8;
// 160 of 1152 slots 30.5 / - / 26.5; 1024 of 1024 slots 140 / - / 147.
Cut choose_cut(long long items, long long tiles, int rows)
{
    const long long lat = rows > 128 ? 170 : 80, full = items / kGrid, rem = items % kGrid;
    auto larger = [](long long x, long long y) { return x > y ? x : y; };
    const long long whole = tiles * (full * larger(kGrid, lat) + (rem ? larger(lat, rem) : 0));
    // at least two tiles a part
    long long split = kGrid / items < (tiles + 1) / 2 ? kGrid / items : (tiles + 1) / 2;
    if (split < 2) split = 0;
    const long long parts = split ? items * split : items + kGrid;
    const long long each = split ? (tiles + split - 1) / split : (items * tiles + kGrid - 1) / kGrid;
    const long long cut = larger(items * tiles * 15 / 16, lat * each) + 320 + parts * rows / 64;
    return whole <= cut ? Cut{true, 0} : Cut{false, (int)split};
}

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
    const int rows = TG < kRows ? TG : kRows;
    const Cut cut = choose_cut(items, tmax, rows);
    const long long grid = cut.split ? items * cut.split : cut.whole && items < kGrid ? items : kGrid;
    AttArgs a{t, c.votes, c.len, vt, o, lse, w.part, w.ml, w.first, w.cut, w.status, p.U, RB, TG,
              p.G == 1 ? 0 : p.G == 2 ? 1 : p.G == 4 ? 2 : 3, p.cap, max_len, rows,
              cut.whole, cut.split, m != nullptr, FastDiv(RB), FastDiv(t.units), kLog2e / sqrtf((float)kD)};
    auto *kernel = c.votes ? tree_attend_kernel<true> : tree_attend_kernel<false>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kDyn);
    if (e != cudaSuccess) return e;
    e = launch_following(kernel, dim3((unsigned)grid), kThreads, kDyn, st, a, mk, mv, mq, mkt, mvt);
    if (e != cudaSuccess) return e;
    if (m == nullptr && cut.whole) return cudaSuccess;
    JoinArgs j{a, m ? m->n : nullptr, m ? m->mu_k : nullptr, m ? m->mu_v : nullptr, m ? m->C : nullptr,
               p.correction == KVC_CORR_FIRST_ORDER, (int)grid};
    if (!cut.whole) {
        const dim3 g((unsigned)grid, (a.rows + 8 * kJoinRows - 1) / (8 * kJoinRows));
        e = launch_following(m ? tree_join_kernel<true> : tree_join_kernel<false>, g, 256, 0, st, j);
        if (e != cudaSuccess) return e;
    }
    if (m) {
        CUtensorMap mf;
        if (!make_f32_map(&mf, w.part, items + kGrid, a.rows, kMomRows)) return cudaErrorInvalidValue;
        e = cudaFuncSetAttribute(tree_moment_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)kMomDyn);
        if (e != cudaSuccess) return e;
        const long long jobs = items * ((a.rows + kMomRows - 1) / kMomRows);
        e = launch_following(tree_moment_kernel, dim3((unsigned)(jobs < kGrid ? jobs : kGrid)), kMomThreads,
                             kMomDyn, st, j, mq, mf);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace kvc

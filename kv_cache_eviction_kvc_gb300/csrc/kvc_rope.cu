// kvc_rope.cu -- norms and rotation of a step's query and key heads
// (kvc_qk_norm_rope), from the projection's rows to the unit layouts.
//
//   y = x w / sqrt(mean(x^2) + eps), then pairs (y_1, y_2) turned by p f_i.
//
// Sixteen lanes hold a head, each four pairs (l < rot / 8) or eight dimensions
// that are not turned, so that both members of a pair are a lane's own in either
// pairing: a turn needs no exchange, the norm's sum four.
//
// Angles: f / 2 pi in turns, reduced modulo one turn, is a 64-bit fraction F; its
// product with the integer position, modulo 2^64, is the angle modulo a turn
// without rounding.  The only rounding is F's (53 bits of f / 2 pi), so position
// 2^20 at f = 1 is off by 2^-36 turns where an fp32 product would be off by 2^-7.
//
// Bound by the bytes, 512 per head read and written, with the instructions close
// behind (141 for two heads took 80 % of the issue slots of the time of the bytes):
// weights, cosine and sine are one 2x2 of a pair, formed once per token and kind of
// head, applied in packed fp32 pairs.  Value heads go along with the key heads, so
// that a tile waits for memory three times and not four (135.6 -> 133.2 us).
// Measured: one token of 48 heads 6.5 us (3.0 in a graph), 16 x 24 tokens 7.0 (4.2),
// 32768 tokens 129 (6.2 TB/s; a block per token without the 2x2 took 319), 262144 of
// 6 rows 176 (floor 120): a tile's turns are formed before its rows are asked for,
// though the rows do not depend on them.  Variants, measured at 131 to 133: four
// blocks of 64 registers and four rows in flight per team, against (with value heads
// by themselves): two rows 150, three 146, three blocks 152, two of 100 registers 181;
// loads and stores marked as streaming 141; the next position loaded ahead 146.
#include "kvc_page.h"

#include <algorithm>
#include <type_traits>

namespace kvc {
namespace {

constexpr int kThreads = 256;
constexpr int kTeams = kThreads / 16;            // of sixteen lanes: a head each
constexpr int kAhead = 4;                        // rows a team has in flight
constexpr int kResident = 4;                     // blocks per SM

struct RopeArgs {
    const uint16_t *qkv;
    int64_t row_stride;
    const int32_t *pos, *n;
    const uint16_t *qw, *kw;
    const double *inv_freq;
    uint16_t *q, *k, *v;
    int T, Hkv, gshift, rot, units, first_unit;
    float eps, scale;
    FastDiv by_T;
};

__device__ __forceinline__ uint64_t turn_fraction(double inv_freq)
{
    double t = fabs(inv_freq) * 0.15915494309189533577;   // 1 / (2 pi)
    t -= floor(t);
    const uint64_t f = (uint64_t)(t * 18446744073709551616.0);
    return inv_freq < 0 ? 0 - f : f;             // 1 - t would round a small t
}

__device__ __forceinline__ void unpack4(uint2 w, float *f)
{
    f[0] = bf_lo(w.x);
    f[1] = bf_hi(w.x);
    f[2] = bf_lo(w.y);
    f[3] = bf_hi(w.y);
}

// Where the sum of squares may have lost bits below fp32's range, and eps does not make up for
// them, the row is taken times 2^100 (exact): what it is multiplied by then.
constexpr float kLeastSquares = 0x1p-100f, kLeastEps = 0x1p-95f;

__device__ __forceinline__ float rescaled(uint2 &w0, uint2 &w1, float eps, unsigned mates)
{
    constexpr float kUp = 0x1p100f;
    float s = 0.f;
    auto take = [&](uint32_t &w) {
        const float2 y = scaled2(w, kUp);
        w = to_bf16x2(y.x, y.y);
        s = fmaf(y.x, y.x, fmaf(y.y, y.y, s));
    };
    take(w0.x), take(w0.y), take(w1.x), take(w1.y);
#pragma unroll
    for (int m = 8; m; m >>= 1) s += __shfl_xor_sync(mates, s, m, 16);
    return rsqrtf(s * (1.f / kD) + eps * kUp * kUp);
}

// Tiles of kTok tokens: their turns to shared memory (a thread per pair), then their
// rows [y rows, (y + 1) rows), 16 / kTok teams a token.  kAll: every dimension is turned,
// and no lane tells itself apart (32768 tokens of 48 rows 129 us, with the test 134).  kTiny:
// an eps below kLeastEps, so that rows of any magnitude keep their norm (the code for them
// costs every row 10 to 28 %, so it is not in the others).
template <int kTok, bool kInter, bool kAll, bool kTiny>
__global__ void __launch_bounds__(kThreads, kResident) rope_kernel(const __grid_constant__ RopeArgs a, int tokens,
                                                                   int rows)
{
    constexpr int kPer = kTeams / kTok;          // teams of a token
    __shared__ float4 turns[2][kTok][2][16];     // (c, s, c, s) of pairs 4l .. 4l + 3
    follow();
    lead();
    const int tid = threadIdx.x, lane = tid & 15, team = tid >> 4;
    const unsigned mates = team & 1 ? 0xffff0000u : 0x0000ffffu;
    const int half = a.rot >> 1;
    const bool turned = kAll || lane * 8 < a.rot;
    // the lane's two groups of four dimensions
    const int d0 = kInter || !turned ? lane * 8 : lane * 4;
    const int d1 = kInter || !turned ? d0 + 4 : half + d0;
    // a thread has one pair's turns: of token tid / 64 of the tile
    const int pair = tid & 63, pair_tok = tid >> 6;
    const bool turns_it = pair < half;
    const uint64_t fraction = turns_it ? turn_fraction(a.inv_freq[pair]) : 0;
    const int G = 1 << a.gshift, nq = a.Hkv << a.gshift, nk = nq + a.Hkv;
    const int r0 = blockIdx.y * rows, r1 = min(nk + a.Hkv, r0 + rows);
    // the rows of queries, and of keys with the values behind them, that are written
    const int q0 = a.q ? r0 : nq, q1 = min(r1, nq);
    const int kv0 = max(r0, a.k ? nq : nk), kv1 = min(r1, a.v ? nk + a.Hkv : nk);

    int buf = 0;
    for (int tok0 = blockIdx.x * kTok; tok0 < tokens; tok0 += gridDim.x * kTok, buf ^= 1) {
#pragma unroll
        for (int j = 0; j < kTok; j += kThreads / 64)
            if (turns_it && tok0 + pair_tok + j < tokens) {
                const uint64_t at = (uint64_t)(int64_t)a.pos[tok0 + pair_tok + j] * fraction;
                float s, c;
                sincospif(__ll2float_rn((long long)at) * 1.0842021724855044e-19f, &s, &c);   // 2^-63
                float2 *to = reinterpret_cast<float2 *>(&turns[buf][pair_tok + j][(pair >> 1) & 1][pair >> 2]);
                to[pair & 1] = make_float2(c * a.scale, s * a.scale);
            }
        __syncthreads();
        const int j = team / kPer, tok = tok0 + j;
        if (tok >= tokens) continue;
        const int b = a.by_T(tok), t = tok - b * a.T;
        if (a.n && t >= a.n[b]) continue;
        const uint16_t *src = a.qkv + (int64_t)tok * a.row_stride;
        const int64_t row = ((int64_t)b * a.units + a.first_unit) * a.T + t;   // of KV head 0 in k and v
        const int first = team % kPer;
#pragma unroll 1
        for (int keys = 0; keys < 2; keys++) {
            const int from = keys ? kv0 : q0, upto = keys ? kv1 : q1;
            if (from + first >= upto) continue;
            // a turn after the weights: (y_1, y_2) -> (A y_1 - B y_2, C y_2 + D y_1)
            const uint16_t *weight = keys ? a.kw : a.qw;
            float A[4], B[4], C[4], E[4];
            {
                float g[8];
#pragma unroll
                for (int i = 0; i < 8; i++) g[i] = 1.f;
                if (weight) {
                    unpack4(__ldg(reinterpret_cast<const uint2 *>(weight + d0)), g);
                    unpack4(__ldg(reinterpret_cast<const uint2 *>(weight + d1)), g + 4);
                }
                float cs[8];
                if (turned) {
                    *reinterpret_cast<float4 *>(cs) = turns[buf][j][0][lane];
                    *reinterpret_cast<float4 *>(cs + 4) = turns[buf][j][1][lane];
                } else {
#pragma unroll
                    for (int i = 0; i < 4; i++) cs[2 * i] = 1.f, cs[2 * i + 1] = 0.f;
                }
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const float g1 = g[kInter ? 2 * e : e], g2 = g[kInter ? 2 * e + 1 : e + 4];
                    A[e] = g1 * cs[2 * e], B[e] = -(g2 * cs[2 * e + 1]);
                    C[e] = g2 * cs[2 * e], E[e] = g1 * cs[2 * e + 1];
                }
            }
            for (int r = from + first; r < upto; r += kPer * kAhead) {
                uint2 w[kAhead][2];
#pragma unroll
                for (int i = 0; i < kAhead; i++) {
                    const uint16_t *x = src + min(r + i * kPer, upto - 1) * kD;
                    w[i][0] = __ldg(reinterpret_cast<const uint2 *>(x + d0));
                    w[i][1] = __ldg(reinterpret_cast<const uint2 *>(x + d1));
                }
                float inv[kAhead];
                if (weight) {
#pragma unroll
                    for (int i = 0; i < kAhead; i++) {
                        float2 s = make_float2(0.f, 0.f);
#pragma unroll
                        for (int e = 0; e < 4; e++) {
                            const uint32_t v = e == 0 ? w[i][0].x : e == 1 ? w[i][0].y : e == 2 ? w[i][1].x : w[i][1].y;
                            const float2 y = make_float2(bf_lo(v), bf_hi(v));
                            s = fma2(y, y, s);
                        }
                        inv[i] = s.x + s.y;
                    }
#pragma unroll
                    for (int m = 8; m; m >>= 1)
#pragma unroll
                        for (int i = 0; i < kAhead; i++) inv[i] += __shfl_xor_sync(mates, inv[i], m, 16);
#pragma unroll
                    for (int i = 0; i < kAhead; i++) {
                        if (kTiny && inv[i] < kLeastSquares && r + i * kPer < nk)
                            inv[i] = rescaled(w[i][0], w[i][1], a.eps, mates);
                        else
                            inv[i] = rsqrtf(inv[i] * (1.f / kD) + a.eps);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < kAhead; i++) inv[i] = 1.f;
                }
#pragma unroll
                for (int i = 0; i < kAhead; i++) {
                    const int at = r + i * kPer;
                    if (at >= upto) break;
                    if (at >= nk) {              // a value head goes as it is
                        uint16_t *dst = a.v + (row + (int64_t)(at - nk) * a.T) * kD;
                        *reinterpret_cast<uint2 *>(dst + d0) = w[i][0];
                        *reinterpret_cast<uint2 *>(dst + d1) = w[i][1];
                        continue;
                    }
                    const float2 n2 = make_float2(inv[i], inv[i]);
                    float2 y[4], z[4];
                    y[0] = mul2(make_float2(bf_lo(w[i][0].x), bf_hi(w[i][0].x)), n2);
                    y[1] = mul2(make_float2(bf_lo(w[i][0].y), bf_hi(w[i][0].y)), n2);
                    y[2] = mul2(make_float2(bf_lo(w[i][1].x), bf_hi(w[i][1].x)), n2);
                    y[3] = mul2(make_float2(bf_lo(w[i][1].y), bf_hi(w[i][1].y)), n2);
                    // a dimension that is not turned stays apart from its neighbour: 0 times an infinity is NaN
                    if (kInter) {
#pragma unroll
                        for (int e = 0; e < 4; e++) {
                            z[e] = mul2(make_float2(A[e], C[e]), y[e]);
                            if (turned) z[e] = fma2(make_float2(B[e], E[e]), make_float2(y[e].y, y[e].x), z[e]);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 2; e++) {
                            z[e] = mul2(make_float2(A[2 * e], A[2 * e + 1]), y[e]);
                            z[e + 2] = mul2(make_float2(C[2 * e], C[2 * e + 1]), y[e + 2]);
                            if (turned) {
                                z[e] = fma2(make_float2(B[2 * e], B[2 * e + 1]), y[e + 2], z[e]);
                                z[e + 2] = fma2(make_float2(E[2 * e], E[2 * e + 1]), y[e], z[e + 2]);
                            }
                        }
                    }
                    uint16_t *dst = keys ? a.k + (row + (int64_t)(at - nq) * a.T) * kD
                                         : a.q + (((row + (int64_t)(at >> a.gshift) * a.T) << a.gshift) + (at & (G - 1))) * kD;
                    *reinterpret_cast<uint2 *>(dst + d0) = make_uint2(to_bf16x2(z[0].x, z[0].y), to_bf16x2(z[1].x, z[1].y));
                    *reinterpret_cast<uint2 *>(dst + d1) = make_uint2(to_bf16x2(z[2].x, z[2].y), to_bf16x2(z[3].x, z[3].y));
                }
            }
        }
    }
}

}  // namespace

cudaError_t launch_qk_norm_rope(const kvc_rope &r, int B, int T, const uint16_t *qkv, int64_t row_stride,
                                const int32_t *pos, const int32_t *n, uint16_t *q, uint16_t *k,
                                uint16_t *v, cudaStream_t st)
{
    RopeArgs a{};
    a.qkv = qkv;
    a.row_stride = row_stride;
    a.pos = pos;
    a.n = n;
    a.qw = r.q_weight;
    a.kw = r.k_weight;
    a.inv_freq = r.inv_freq;
    a.q = q;
    a.k = k;
    a.v = v;
    a.T = T;
    a.Hkv = r.Hkv;
    while (r.Hkv << a.gshift < r.Hq) a.gshift++;
    a.rot = r.rot;
    a.units = r.units;
    a.first_unit = r.first_unit;
    a.eps = r.eps;
    a.scale = r.scale;
    a.by_T = FastDiv((uint32_t)T);
    const int tokens = B * T, rows = r.Hq + 2 * r.Hkv;
    // Tokens of a tile: enough rows for its 16 teams, not so many that few tiles have the work (4, 8
    // and 16 tokens, tiles of much work: 6 rows a token 445 / 297 / 184 us, 24 rows 161 / 131 / 133,
    // 48 rows 133 / 131 / 144, 80 rows 129 / 134 / 152; 1024 tokens of 24 rows 7.7 / 5.9 / 7.2; 64 of
    // 48 rows 3.6 / 4.7 / 7.0)
    const bool tiny = r.eps < kLeastEps && (r.q_weight || r.k_weight);
    int tok = tiny ? 4 : 16;
    while (tok > 4 && (tok * rows > 384 || tokens < 128 * tok)) tok /= 2;
    // Persistent blocks, four per SM (16 or 54 per SM in turn: within 3 %).  Few tokens: a token's
    // rows go to several blocks, as many as fill the device (384 tokens of 48 rows in tiles of 4: three
    // blocks 10.2, one 12.3 us; 1024: two 12.5, three 14.3, one 14.3; 4096: one 26.6, three 28.8)
    const int tiles = (tokens - 1) / tok + 1, fill = 152 * kResident;
    const int cuts = std::max(1, std::min((rows + kTeams - 1) / kTeams, fill / tiles));
    const int each = ((rows - 1) / cuts / kTeams + 1) * kTeams;
    const dim3 grid(std::min(tiles, fill), (rows - 1) / each + 1);
    auto pick = [&](auto inter, auto all) {
        constexpr bool kInter = decltype(inter)::value, kAll = decltype(all)::value;
        return tok == 4   ? rope_kernel<4, kInter, kAll, false>
               : tok == 8 ? rope_kernel<8, kInter, kAll, false>
                          : rope_kernel<16, kInter, kAll, false>;
    };
    const std::true_type yes;
    const std::false_type no;
    void (*kernel)(RopeArgs, int, int) = tiny          ? (r.interleaved ? rope_kernel<4, true, false, true> : rope_kernel<4, false, false, true>)
                                         : r.rot == kD ? (r.interleaved ? pick(yes, yes) : pick(no, yes))
                                                       : (r.interleaved ? pick(yes, no) : pick(no, no));
    return launch_following(kernel, grid, kThreads, 0, st, a, tokens, each);
}

}  // namespace kvc

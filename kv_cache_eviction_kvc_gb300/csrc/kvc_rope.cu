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
#include "kvc_page.h"

namespace kvc {
namespace {

constexpr int kThreads = 256;
constexpr int kTeams = kThreads / 16;            // of sixteen lanes: a head each

struct RopeArgs {
    const uint16_t *qkv;
    int64_t row_stride;
    const int32_t *pos, *n;
    const uint16_t *qw, *kw;
    const double *inv_freq;
    uint16_t *q, *k, *v;
    int T, Hkv, G, rot, units, first_unit;
    float eps, scale;
    FastDiv by_T;
};

__device__ __forceinline__ uint64_t turn_fraction(double inv_freq)
{
    double t = inv_freq * 0.15915494309189533577;   // 1 / (2 pi)
    t -= floor(t);
    return (uint64_t)(t * 18446744073709551616.0);
}

__device__ __forceinline__ void unpack4(uint2 w, float *f)
{
    f[0] = bf_lo(w.x);
    f[1] = bf_hi(w.x);
    f[2] = bf_lo(w.y);
    f[3] = bf_hi(w.y);
}

// One block: kTok tokens, `rows` of their heads.
template <int kTok, bool kInter>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs a, int tokens,
                                                        int rows_per_block)
{
    __shared__ float4 turns[kTok][2][16];        // (c, s, c, s) of pairs 4l .. 4l + 3
    follow();
    lead();
    const int tid = threadIdx.x, lane = tid & 15, team = tid >> 4;
    const int tok0 = blockIdx.x * kTok;
    const int half = a.rot >> 1;
    for (int i = tid; i < kTok * half; i += kThreads) {
        const int j = i / half, p = i - j * half, tok = tok0 + j;
        if (tok >= tokens) break;
        const uint64_t at = (uint64_t)(int64_t)a.pos[tok] * turn_fraction(a.inv_freq[p]);
        float s, c;
        sincospif(__ll2float_rn((long long)at) * 1.0842021724855044e-19f, &s, &c);   // 2^-63
        float2 *to = reinterpret_cast<float2 *>(&turns[j][(p >> 1) & 1][p >> 2]) + (p & 1);
        *to = make_float2(c * a.scale, s * a.scale);
    }
    __syncthreads();

    constexpr int kPer = kTeams / kTok;          // teams of a token
    const int j = team / kPer, tok = tok0 + j;
    if (tok >= tokens) return;
    const int b = a.by_T(tok), t = tok - b * a.T;
    if (a.n && t >= a.n[b]) return;
    const bool turned = lane * 8 < a.rot;
    // the lane's two groups of four dimensions
    const int d0 = kInter || !turned ? lane * 8 : lane * 4;
    const int d1 = kInter || !turned ? d0 + 4 : half + d0;
    float cs[8];
    if (turned) {
        *reinterpret_cast<float4 *>(cs) = turns[j][0][lane];
        *reinterpret_cast<float4 *>(cs + 4) = turns[j][1][lane];
    } else {
#pragma unroll
        for (int i = 0; i < 4; i++) cs[2 * i] = 1.f, cs[2 * i + 1] = 0.f;
    }
    const unsigned mates = team & 1 ? 0xffff0000u : 0x0000ffffu;
    const int G = a.G, nq = a.Hkv * G, all = nq + 2 * a.Hkv;
    const int end = min(all, (int)(blockIdx.y + 1) * rows_per_block);
    const uint16_t *src = a.qkv + (int64_t)tok * a.row_stride;
    const int64_t unit = (int64_t)b * a.units + a.first_unit;
    for (int r = blockIdx.y * rows_per_block + team % kPer; r < end; r += kPer) {
        const int kind = r < nq ? 0 : r < nq + a.Hkv ? 1 : 2;
        uint16_t *dst;
        if (kind == 0) {
            const int g = r / G;
            dst = a.q ? a.q + (((unit + g) * a.T + t) * G + (r - g * G)) * kD : nullptr;
        } else {
            dst = kind == 1 ? a.k : a.v;
            if (dst) dst += ((unit + (r - nq) % a.Hkv) * a.T + t) * kD;
        }
        if (!dst) continue;
        const uint16_t *x = src + r * kD;
        const uint2 w0 = __ldg(reinterpret_cast<const uint2 *>(x + d0));
        const uint2 w1 = __ldg(reinterpret_cast<const uint2 *>(x + d1));
        if (kind == 2) {
            *reinterpret_cast<uint2 *>(dst + d0) = w0;
            *reinterpret_cast<uint2 *>(dst + d1) = w1;
            continue;
        }
        float y[8];
        unpack4(w0, y);
        unpack4(w1, y + 4);
        const uint16_t *weight = kind == 0 ? a.qw : a.kw;
        if (weight) {
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < 8; i++) s = fmaf(y[i], y[i], s);
#pragma unroll
            for (int m = 8; m; m >>= 1) s += __shfl_xor_sync(mates, s, m, 16);
            const float inv = 1.f / sqrtf(s * (1.f / kD) + a.eps);
            float w[8];
            unpack4(__ldg(reinterpret_cast<const uint2 *>(weight + d0)), w);
            unpack4(__ldg(reinterpret_cast<const uint2 *>(weight + d1)), w + 4);
#pragma unroll
            for (int i = 0; i < 8; i++) y[i] *= inv * w[i];
        }
        float z[8];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int i1 = kInter ? 2 * i : i, i2 = kInter ? 2 * i + 1 : i + 4;
            z[i1] = y[i1] * cs[2 * i] - y[i2] * cs[2 * i + 1];
            z[i2] = y[i2] * cs[2 * i] + y[i1] * cs[2 * i + 1];
        }
        *reinterpret_cast<uint2 *>(dst + d0) = make_uint2(to_bf16x2(z[0], z[1]), to_bf16x2(z[2], z[3]));
        *reinterpret_cast<uint2 *>(dst + d1) = make_uint2(to_bf16x2(z[4], z[5]), to_bf16x2(z[6], z[7]));
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
    a.G = r.Hq / r.Hkv;
    a.rot = r.rot;
    a.units = r.units;
    a.first_unit = r.first_unit;
    a.eps = r.eps;
    a.scale = r.scale;
    a.by_T = FastDiv((uint32_t)T);
    const int tokens = B * T, rows = r.Hq + 2 * r.Hkv;
    const dim3 grid(tokens, (rows + kTeams - 1) / kTeams);
    return r.interleaved ? launch_following(rope_kernel<1, true>, grid, kThreads, 0, st, a, tokens, kTeams)
                         : launch_following(rope_kernel<1, false>, grid, kThreads, 0, st, a, tokens, kTeams);
}

}  // namespace kvc

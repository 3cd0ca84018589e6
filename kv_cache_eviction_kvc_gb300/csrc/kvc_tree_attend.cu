// kvc_tree_attend.cu -- attention of a tree of drafted tokens over the cache
// and the tree itself, with the normalization correction.
//
// One warp per query row (drafted token, head): a lane holds four dimensions
// of q and of the output, one pass over the slots with the running maximum
// and sum of the softmax.
#include "kvc_tree.h"

namespace kvc {
namespace {

struct AttArgs {
    TreeArgs t;
    const uint16_t *q, *kt, *vt, *K, *V;
    const int32_t *votes, *len;
    const float *mn, *mu_k, *mu_v, *C;
    uint16_t *o;
    float *lse;
    int32_t *status;
    int G, cap, max_len, first;
};

__device__ __forceinline__ uint32_t bf2(float a, float b)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

__global__ void __launch_bounds__(256) tree_attend_kernel(AttArgs a)
{
    const int u = blockIdx.x, lane = threadIdx.x & 31;
    const int row = blockIdx.y * 8 + (threadIdx.x >> 5);
    const int n = a.len[u], live = tree_live(a.t, u);
    if (n < 0 || n > a.max_len || live < 0) {
        if (threadIdx.x == 0) record_status(a.status, live < 0 ? KVC_ERR_INVALID_ARG : KVC_ERR_SHAPE);
        return;
    }
    if (row >= live * a.G) return;
    const size_t tb = (size_t)u * a.t.T, cb = (size_t)u * a.cap, qr = tb * a.G + row;
    const float scale = rsqrtf((float)kD);
    const uint2 qw = reinterpret_cast<const uint2 *>(a.q + qr * kD)[lane];
    const float q0 = bf_lo(qw.x), q1 = bf_hi(qw.x), q2 = bf_lo(qw.y), q3 = bf_hi(qw.y);
    float m = -INFINITY, l = 0.f, f0 = 0.f, f1 = 0.f, f2 = 0.f, f3 = 0.f;
    auto take = [&](const uint16_t *kp, const uint16_t *vp, float bias) {
        const uint2 kw = reinterpret_cast<const uint2 *>(kp)[lane];
        const uint2 vw = reinterpret_cast<const uint2 *>(vp)[lane];
        const float x = warp_sum(q0 * bf_lo(kw.x) + q1 * bf_hi(kw.x) + q2 * bf_lo(kw.y) +
                                 q3 * bf_hi(kw.y)) * scale + bias;
        const float mx = fmaxf(m, x);
        const float c = m == -INFINITY ? 0.f : expf(m - mx), e = x == -INFINITY ? 0.f : expf(x - mx);
        l = l * c + e;
        f0 = f0 * c + e * bf_lo(vw.x);
        f1 = f1 * c + e * bf_hi(vw.x);
        f2 = f2 * c + e * bf_lo(vw.y);
        f3 = f3 * c + e * bf_hi(vw.y);
        m = mx;
    };
    for (int i = 0; i < n; i++)
        take(a.K + (cb + i) * kD, a.V + (cb + i) * kD,
             a.votes ? logf((float)a.votes[cb + i]) : 0.f);
    uint64_t w = a.t.mask[(size_t)(u / a.t.units) * a.t.T + row / a.G];
    for (int j = 0; j < live; j++)
        if (w >> j & 1) take(a.kt + (tb + j) * kD, a.vt + (tb + j) * kD, 0.f);
    const bool none = l == 0.f;
    const float lse = none ? -INFINITY : m + logf(l);
    const float inv = none ? 0.f : 1.f / l;
    float f[4] = {f0 * inv, f1 * inv, f2 * inv, f3 * inv};
    const float ne = a.mn ? a.mn[u] : 0.f;
    if (ne > 0.f) {
        const float4 mk = reinterpret_cast<const float4 *>(a.mu_k + (size_t)u * kD)[lane];
        const float ze = logf(ne) + scale * warp_sum(q0 * mk.x + q1 * mk.y + q2 * mk.z + q3 * mk.w);
        const float wr = 1.f / (1.f + expf(ze - lse));
        for (int i = 0; i < kD; i++) {
            float g = a.mu_v[(size_t)u * kD + i];
            if (a.first) {
                const float4 c =
                    reinterpret_cast<const float4 *>(a.C + ((size_t)u * kD + i) * kD)[lane];
                g += scale * warp_sum(q0 * c.x + q1 * c.y + q2 * c.z + q3 * c.w);
            }
            if (lane == i >> 2) f[i & 3] = wr * f[i & 3] + (1.f - wr) * g;
        }
    }
    reinterpret_cast<uint2 *>(a.o + qr * kD)[lane] = make_uint2(bf2(f[0], f[1]), bf2(f[2], f[3]));
    if (lane == 0) a.lse[qr] = lse;
}

}  // namespace

size_t tree_ws_bytes(const kvc_params &, int) { return align_up(sizeof(WsHeader)); }

cudaError_t launch_tree_attend(const kvc_params &p, int max_len, const TreeArgs &t,
                               const uint16_t *q, const uint16_t *kt, const uint16_t *vt,
                               const kvc_cache &c, const kvc_moments *m, uint16_t *o, float *lse,
                               void *ws, cudaStream_t st)
{
    AttArgs a{t, q, kt, vt, c.K, c.V, c.votes, c.len, m ? m->n : nullptr, m ? m->mu_k : nullptr,
              m ? m->mu_v : nullptr, m ? m->C : nullptr, o, lse, static_cast<int32_t *>(ws), p.G,
              p.cap, max_len, p.correction == KVC_CORR_FIRST_ORDER};
    tree_attend_kernel<<<dim3(p.U, (t.T * p.G + 7) / 8), 256, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace kvc

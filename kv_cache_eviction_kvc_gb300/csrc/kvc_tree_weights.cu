// kvc_tree_weights.cu -- the attention weight that the accepted tokens gave
// to every slot of the cache and to the accepted tokens themselves.
//
// One thread per slot (the accepted tokens behind the cache's), over the
// accepted tokens and heads.
#include "kvc_tree.h"

namespace kvc {
namespace {

struct WtArgs {
    TreeArgs t;
    PathArgs p;
    const float *w;
    const uint16_t *q, *kt, *K;
    const float *lse;
    const int32_t *votes, *len;
    float *S;
    int32_t *status;
    int G, cap, max_len;
};

__global__ void __launch_bounds__(256) tree_weights_kernel(WtArgs a)
{
    const int u = blockIdx.y, i = blockIdx.x * 256 + threadIdx.x, b = u / a.t.units;
    const int n = a.len[u], acc = path_count(a.t, a.p, u, threadIdx.x & 31);
    if (n < 0 || n > a.max_len || acc < 0 || n + acc > a.cap) {
        if (i == 0) record_status(a.status, acc < 0 ? KVC_ERR_INVALID_ARG : KVC_ERR_SHAPE);
        return;
    }
    if (i >= n + acc) return;
    const int32_t *tok = a.p.token + (size_t)b * a.p.A;
    const size_t tb = (size_t)u * a.t.T, slot = (size_t)u * a.cap + i;
    const bool old = i < n;
    const int self = old ? 0 : tok[i - n];
    const uint16_t *k = old ? a.K + slot * kD : a.kt + (tb + self) * kD;
    const float scale = rsqrtf((float)kD);
    float s = 0.f;
    for (int j = 0; j < acc; j++) {
        const int c = tok[j];
        if (!old && !(a.t.mask[(size_t)b * a.t.T + c] >> self & 1)) continue;
        const float w = a.w ? a.w[(size_t)b * a.p.A + j] : 1.f;
        for (int h = 0; h < a.G; h++) {
            const size_t qr = (tb + c) * a.G + h;
            float x = 0.f;
            for (int d = 0; d < kD; d++) x += bf2f(a.q[qr * kD + d]) * bf2f(k[d]);
            const float lse = a.lse[qr];
            if (lse != -INFINITY) s += w / a.G * expf(x * scale - lse);
        }
    }
    a.S[slot] = old && a.votes ? s * (float)a.votes[slot] : s;
}

}  // namespace

cudaError_t launch_tree_weights(const kvc_params &p, int max_len, const TreeArgs &t,
                                const PathArgs &pa, const float *row_weight, const uint16_t *q,
                                const uint16_t *kt, const float *lse, const kvc_cache &c, float *S,
                                void *ws, cudaStream_t st)
{
    WtArgs a{t, pa, row_weight, q, kt, c.K, lse, c.votes, c.len, S, static_cast<int32_t *>(ws), p.G,
             p.cap, max_len};
    const int top = max_len + pa.A < p.cap ? max_len + pa.A : p.cap;
    tree_weights_kernel<<<dim3((top + 255) / 256, p.U), 256, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace kvc

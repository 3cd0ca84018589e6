// kvc_page.cu -- the extern "C" entry points of the cache in pages and of the
// norms and rotation in front of it: host-side argument checks and dispatch
// (the kernels: kvc_rope.cu, kvc_page_move.cu, kvc_page_attend.cu).
#include "kvc_page.h"

#include <math.h>

using namespace kvc;

#define PG_CHECK(cond, code, ...)      \
    do {                               \
        if (!(cond)) {                 \
            set_error(__VA_ARGS__);    \
            return (code);             \
        }                              \
    } while (0)

#define PG_TRY(expr)                      \
    do {                                  \
        kvc_status _s = (expr);           \
        if (_s != KVC_OK) return _s;      \
    } while (0)

static bool misaligned(const void *p, unsigned a) { return ((uintptr_t)p & (a - 1)) != 0; }

static kvc_status pg_cuda(cudaError_t e, const char *what)
{
    if (e == cudaSuccess) return KVC_OK;
    (void)cudaGetLastError();                    // it is reported here, not by the next call
    set_error("%s: %s", what, cudaGetErrorString(e));
    return KVC_ERR_CUDA;
}

static bool known_group(int G) { return G == 1 || G == 2 || G == 4 || G == 8; }

static kvc_status check_pages(const char *fn, const kvc_pages *pg)
{
    PG_CHECK(pg != nullptr, KVC_ERR_INVALID_ARG, "%s: pages is NULL", fn);
    PG_CHECK(pg->d == kD, KVC_ERR_UNSUPPORTED, "%s: d = %d unsupported (only 128)", fn, pg->d);
    PG_CHECK(pg->type == KVC_PAGE_BF16 || pg->type == KVC_PAGE_E4M3, KVC_ERR_INVALID_ARG,
             "%s: type = %d unknown", fn, pg->type);
    PG_CHECK(pg->page == 16 || pg->page == 32 || pg->page == 64 || pg->page == 128, KVC_ERR_UNSUPPORTED,
             "%s: pages of %d slots unsupported (16, 32, 64 or 128)", fn, pg->page);
    PG_CHECK(pg->U >= 1 && pg->heads >= 1 && pg->U % pg->heads == 0, KVC_ERR_INVALID_ARG,
             "%s: heads = %d must divide U = %d", fn, pg->heads, pg->U);
    PG_CHECK(pg->U <= 1 << 27, KVC_ERR_UNSUPPORTED, "%s: U = %d unsupported (at most 2^27)", fn, pg->U);
    PG_CHECK(pg->n_pages >= 1 && pg->stride >= 1, KVC_ERR_INVALID_ARG,
             "%s: n_pages = %d and stride = %d must be >= 1", fn, pg->n_pages, pg->stride);
    PG_CHECK((int64_t)pg->stride * pg->page < (1ll << 31) - 128, KVC_ERR_UNSUPPORTED,
             "%s: stride * page = %lld slots unsupported (below 2^31 - 128)", fn,
             (long long)pg->stride * pg->page);
    PG_CHECK(pg->K && pg->V && pg->table && pg->len, KVC_ERR_INVALID_ARG,
             "%s: K, V, table and len must be non-NULL", fn);
    PG_CHECK(!misaligned(pg->K, 16) && !misaligned(pg->V, 16), KVC_ERR_INVALID_ARG,
             "%s: K and V must be 16-byte aligned", fn);
    PG_CHECK(pg->type == KVC_PAGE_BF16 || (pg->k_scale && pg->v_scale), KVC_ERR_INVALID_ARG,
             "%s: pages in 8 bits need k_scale and v_scale", fn);
    return KVC_OK;
}

static kvc_status check_page_ws(const char *fn, size_t need, const void *ws, size_t bytes)
{
    PG_CHECK(ws != nullptr && !misaligned(ws, kAlign) && bytes >= need, KVC_ERR_WORKSPACE,
             "%s: a workspace of %zu bytes (256-byte aligned) is required", fn, need);
    return KVC_OK;
}

// Blocks of a launch with one per `rows` of every unit's rows.
static bool launchable(int64_t units, int64_t rows) { return units * rows < (1ll << 31); }

namespace kvc {

PageArgs page_args(const kvc_pages &pg)
{
    PageArgs a{};
    a.K = static_cast<uint8_t *>(pg.K);
    a.V = static_cast<uint8_t *>(pg.V);
    a.ks = pg.k_scale;
    a.vs = pg.v_scale;
    a.table = pg.table;
    a.len = pg.len;
    a.heads = pg.heads;
    a.shift = pg.page == 16 ? 4 : pg.page == 32 ? 5 : pg.page == 64 ? 6 : 7;
    a.n_pages = pg.n_pages;
    a.stride = pg.stride;
    a.by_heads = FastDiv((uint32_t)pg.heads);
    return a;
}

}  // namespace kvc

extern "C" {

kvc_status kvc_qk_norm_rope(const kvc_rope *r, int32_t B, int32_t T, const uint16_t *qkv,
                            int64_t row_stride, const int32_t *pos, const int32_t *n, uint16_t *q,
                            uint16_t *k, uint16_t *v, void *stream)
{
    const char *fn = "kvc_qk_norm_rope";
    PG_CHECK(r != nullptr, KVC_ERR_INVALID_ARG, "%s: the parameters are NULL", fn);
    PG_CHECK(r->d == kD, KVC_ERR_UNSUPPORTED, "%s: d = %d unsupported (only 128)", fn, r->d);
    PG_CHECK(r->Hkv >= 1 && r->Hq >= 1 && r->Hq % r->Hkv == 0, KVC_ERR_INVALID_ARG,
             "%s: Hkv = %d must divide Hq = %d", fn, r->Hkv, r->Hq);
    PG_CHECK(known_group(r->Hq / r->Hkv), KVC_ERR_UNSUPPORTED,
             "%s: %d query heads per KV head unsupported (1, 2, 4 or 8)", fn, r->Hq / r->Hkv);
    PG_CHECK(r->Hkv <= 4096, KVC_ERR_UNSUPPORTED, "%s: Hkv = %d unsupported (at most 4096)", fn, r->Hkv);
    PG_CHECK(r->rot >= 0 && r->rot <= kD && r->rot % 16 == 0, KVC_ERR_UNSUPPORTED,
             "%s: rot = %d must be a multiple of 16 up to d", fn, r->rot);
    PG_CHECK(r->interleaved == 0 || r->interleaved == 1, KVC_ERR_INVALID_ARG,
             "%s: interleaved = %d must be 0 or 1", fn, r->interleaved);
    PG_CHECK(r->eps >= 0.f && isfinite(r->eps) && isfinite(r->scale), KVC_ERR_INVALID_ARG,
             "%s: eps = %g must be finite and >= 0, scale = %g finite", fn, (double)r->eps,
             (double)r->scale);
    PG_CHECK(r->rot == 0 || (r->inv_freq && !misaligned(r->inv_freq, 8)), KVC_ERR_INVALID_ARG,
             "%s: inv_freq must be non-NULL and 8-byte aligned", fn);
    PG_CHECK(r->first_unit >= 0 && (int64_t)r->first_unit + r->Hkv <= r->units, KVC_ERR_INVALID_ARG,
             "%s: units %d .. %lld of a sequence's %d", fn, r->first_unit,
             (long long)r->first_unit + r->Hkv, r->units);
    PG_CHECK(B >= 1 && T >= 1, KVC_ERR_INVALID_ARG, "%s: B = %d and T = %d must be >= 1", fn, B, T);
    PG_CHECK((int64_t)B * r->units < (1ll << 31) && (int64_t)B * T <= (1ll << 30), KVC_ERR_UNSUPPORTED,
             "%s: B = %d sequences of T = %d tokens unsupported", fn, B, T);
    PG_CHECK(qkv && pos && (q || k || v), KVC_ERR_INVALID_ARG,
             "%s: qkv, pos and one of q, k, v must be non-NULL", fn);
    PG_CHECK(!misaligned(qkv, 16) && !misaligned(q, 16) && !misaligned(k, 16) && !misaligned(v, 16) &&
                 !misaligned(r->q_weight, 16) && !misaligned(r->k_weight, 16),
             KVC_ERR_INVALID_ARG, "%s: qkv, q, k, v and the weights must be 16-byte aligned", fn);
    PG_CHECK(row_stride >= (r->Hq + 2ll * r->Hkv) * kD && row_stride % 8 == 0, KVC_ERR_SHAPE,
             "%s: row_stride = %lld must be a multiple of 8 and at least %lld", fn, (long long)row_stride,
             (r->Hq + 2ll * r->Hkv) * kD);
    return pg_cuda(launch_qk_norm_rope(*r, B, T, qkv, row_stride, pos, n, q, k, v,
                                       static_cast<cudaStream_t>(stream)),
                   fn);
}

size_t kvc_page_workspace_size(const kvc_pages *pg, int32_t G)
{
    if (check_pages("kvc_page_workspace_size", pg) != KVC_OK || !known_group(G)) return 0;
    return page_ws_bytes(*pg, G);
}

kvc_status kvc_page_write(const kvc_pages *pg, int32_t T, const int32_t *first, const int32_t *count,
                          const uint16_t *k, const uint16_t *v, void *ws, size_t ws_bytes, void *stream)
{
    const char *fn = "kvc_page_write";
    PG_TRY(check_pages(fn, pg));
    PG_CHECK(T >= 1, KVC_ERR_INVALID_ARG, "%s: T = %d must be >= 1", fn, T);
    PG_CHECK(launchable(pg->U, (T + 15ll) / 16), KVC_ERR_UNSUPPORTED,
             "%s: T = %d rows of U = %d units unsupported", fn, T, pg->U);
    PG_CHECK(k && v, KVC_ERR_INVALID_ARG, "%s: k and v must be non-NULL", fn);
    PG_CHECK(!misaligned(k, 16) && !misaligned(v, 16), KVC_ERR_INVALID_ARG,
             "%s: k and v must be 16-byte aligned", fn);
    PG_TRY(check_page_ws(fn, kAlign, ws, ws_bytes));
    return pg_cuda(launch_page_write(*pg, T, first, count, k, v, ws, static_cast<cudaStream_t>(stream)),
                   fn);
}

kvc_status kvc_page_read(const kvc_pages *pg, int32_t M, int32_t ld, const int32_t *slots,
                         const int32_t *count, uint16_t *k_out, uint16_t *v_out, void *ws,
                         size_t ws_bytes, void *stream)
{
    const char *fn = "kvc_page_read";
    PG_TRY(check_pages(fn, pg));
    PG_CHECK(M >= 1, KVC_ERR_INVALID_ARG, "%s: M = %d must be >= 1", fn, M);
    PG_CHECK(ld >= M, KVC_ERR_SHAPE, "%s: ld = %d must be at least M = %d", fn, ld, M);
    PG_CHECK(launchable(pg->U, (M + 15ll) / 16), KVC_ERR_UNSUPPORTED,
             "%s: M = %d rows of U = %d units unsupported", fn, M, pg->U);
    PG_CHECK(k_out && v_out, KVC_ERR_INVALID_ARG, "%s: k_out and v_out must be non-NULL", fn);
    PG_CHECK(!misaligned(k_out, 16) && !misaligned(v_out, 16), KVC_ERR_INVALID_ARG,
             "%s: k_out and v_out must be 16-byte aligned", fn);
    PG_TRY(check_page_ws(fn, kAlign, ws, ws_bytes));
    return pg_cuda(launch_page_read(*pg, M, ld, slots, count, k_out, v_out, ws,
                                    static_cast<cudaStream_t>(stream)),
                   fn);
}

kvc_status kvc_page_attend(const kvc_pages *pg, int32_t G, int32_t max_len, const uint16_t *q,
                           const uint16_t *k_new, const uint16_t *v_new, uint16_t *o, float *lse,
                           void *ws, size_t ws_bytes, void *stream)
{
    const char *fn = "kvc_page_attend";
    PG_TRY(check_pages(fn, pg));
    PG_CHECK(known_group(G), KVC_ERR_UNSUPPORTED, "%s: G = %d unsupported (1, 2, 4 or 8)", fn, G);
    PG_CHECK(max_len >= 1 && max_len <= (int64_t)pg->stride * pg->page, KVC_ERR_SHAPE,
             "%s: max_len = %d must satisfy 1 <= max_len <= stride * page = %lld", fn, max_len,
             (long long)pg->stride * pg->page);
    PG_CHECK(launchable(pg->U, (max_len + 15ll) / 16), KVC_ERR_UNSUPPORTED,
             "%s: max_len = %d of U = %d units unsupported", fn, max_len, pg->U);
    PG_CHECK(q && o && lse, KVC_ERR_INVALID_ARG, "%s: q, o and lse must be non-NULL", fn);
    PG_CHECK((k_new == nullptr) == (v_new == nullptr), KVC_ERR_INVALID_ARG,
             "%s: k_new and v_new must both be given or both be NULL", fn);
    PG_CHECK(!misaligned(q, 16) && !misaligned(o, 16) && !misaligned(k_new, 16) && !misaligned(v_new, 16),
             KVC_ERR_INVALID_ARG, "%s: q, o, k_new and v_new must be 16-byte aligned", fn);
    PG_TRY(check_page_ws(fn, page_ws_bytes(*pg, G), ws, ws_bytes));
    return pg_cuda(launch_page_attend(*pg, G, max_len, q, k_new, v_new, o, lse, ws,
                                      static_cast<cudaStream_t>(stream)),
                   fn);
}

}  // extern "C"

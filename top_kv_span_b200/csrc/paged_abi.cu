// C ABI entry points of the paged cache and the packed prompts (declared in
// include/reatt.h): argument checks on the host, the workspace plan and the
// launches.  Nothing here allocates device memory.
#include <math.h>

#include "kernels.h"
#include "paged.cuh"
#include "reatt.h"

namespace reatt {
namespace {

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline int cuda_status(cudaError_t e) { return e == cudaSuccess ? REATT_OK : REATT_ECUDA; }

constexpr int64_t kMaxPositions = int64_t(1) << 24;   // exact fp32 positions in the RoPE angle

// Row stride of a packed operand of H heads: 0 means dense.
bool stride_of(int64_t given, int64_t H, const reatt_paged_dims *d, int64_t *out)
{
    const int64_t dense = H * d->d;
    *out = given ? given : dense;
    const int64_t vec = d->dtype == REATT_BF16 ? 8 : 4;
    return *out >= dense && *out % vec == 0 && *out < (int64_t(1) << 36);
}

int paged_geom(const reatt_paged_dims *d, PagedGeom *g)
{
    if (!d) return REATT_EINVAL;
    if (d->B < 1 || d->Hq < 1 || d->Hkv < 1 || d->Hq % d->Hkv != 0 || d->N < 0 || d->page < 1 ||
        (d->page & (d->page - 1)) != 0 || d->max_pages < 1 || d->n_pages < 1 || d->reserved != 0)
        return REATT_EINVAL;
    if (!(d->rope_base >= 0.0) || !isfinite(d->rope_base)) return REATT_EINVAL;
    if (d->dtype != REATT_F32 && d->dtype != REATT_BF16) return REATT_EUNSUPPORTED;
    if (d->d != 64 && d->d != 128) return REATT_EUNSUPPORTED;
    if (!stride_of(d->q_stride, d->Hq, d, &g->qs) || !stride_of(d->k_stride, d->Hkv, d, &g->ks) ||
        !stride_of(d->v_stride, d->Hkv, d, &g->vs) ||
        !stride_of(d->q_rot_stride, d->Hq, d, &g->qrs) ||
        !stride_of(d->k_rot_stride, d->Hkv, d, &g->krs))
        return REATT_EINVAL;
    if (d->B > 65536 || d->Hq > 4096 || d->Hq / d->Hkv > 128) return REATT_EUNSUPPORTED;
    if (int64_t(d->max_pages) * d->page > kMaxPositions) return REATT_EUNSUPPORTED;
    if (d->N >= (int64_t(1) << 28) || d->n_pages > 0x7fffffff) return REATT_EUNSUPPORTED;
    if (double(d->n_pages) * d->Hkv * d->page * d->d > 4e18) return REATT_EUNSUPPORTED;
    g->B = d->B;
    g->Hq = d->Hq;
    g->Hkv = d->Hkv;
    g->g = d->Hq / d->Hkv;
    g->d = d->d;
    g->dtype = d->dtype;
    g->page_shift = 0;
    while ((1 << g->page_shift) < d->page) ++g->page_shift;
    g->max_pages = d->max_pages;
    g->N = d->N;
    g->n_pages = d->n_pages;
    g->rotate = d->rope_base > 0.0;
    return REATT_OK;
}

// RoPE frequencies base^(-2i/d) in half-turns, hi + lo.  The powers of one
// extended-precision root (64 bits of significand: the 63rd is good to 2^-58)
// instead of 64 calls of pow, which took 3 us.
void rope_frequencies(const reatt_paged_dims *d, PagedGeom *g)
{
    const long double root = g->rotate ? powl((long double)d->rope_base, -2.0L / d->d) : 0.0L;
    long double f = 1.0L / 3.141592653589793238462643383279502884L;
    for (int i = 0; i < 64; ++i, f *= root) {
        const bool used = g->rotate && i < d->d / 2;
        g->rope_hi[i] = used ? float(f) : 0.f;
        g->rope_lo[i] = used ? float(f - (long double)g->rope_hi[i]) : 0.f;
    }
}

}  // namespace
}  // namespace reatt

using namespace reatt;

extern "C" {

int reatt_paged_workspace_bytes(const reatt_paged_dims *dims, size_t *bytes)
{
    PagedGeom g;
    const int rc = paged_geom(dims, &g);
    if (rc) return rc;
    if (!bytes) return REATT_EINVAL;
    const size_t decode = paged_decode_ws_bytes(g), prompt = prompt_ws_bytes(g);
    *bytes = (kWsHeader + (decode > prompt ? decode : prompt) + 255) / 256 * 256;
    return REATT_OK;
}

int reatt_paged_append(const reatt_paged_dims *dims, const void *q, const void *k, const void *v,
                       const int32_t *cu_seqlens, const int32_t *past_len, const int32_t *page_table,
                       void *q_rot, void *k_rot, void *k_pages, void *v_pages, int32_t *seq_len,
                       void *ws, reatt_stream stream)
{
    PagedGeom g;
    const int rc = paged_geom(dims, &g);
    if (rc) return rc;
    if (!cu_seqlens || !past_len || !page_table || !k_pages || !v_pages || !ws) return REATT_EINVAL;
    if (g.N > 0 && (!k || !v)) return REATT_EINVAL;
    if (g.N > 0 && (q == nullptr) != (q_rot == nullptr)) return REATT_EINVAL;
    // seq_len is written while other blocks still read past_len
    if (seq_len == past_len) return REATT_EINVAL;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(cu_seqlens) ||
        !aligned16(past_len) || !aligned16(page_table) || !aligned16(q_rot) || !aligned16(k_rot) ||
        !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(seq_len) || !aligned16(ws))
        return REATT_EINVAL;
    // in place only row by row: the same buffer has the same stride
    if ((q && q == q_rot && g.qs != g.qrs) || (k && k == k_rot && g.ks != g.krs)) return REATT_EINVAL;
    rope_frequencies(dims, &g);
    return cuda_status(launch_paged_append(g, q, k, v, cu_seqlens, past_len, page_table, q_rot, k_rot,
                                           k_pages, v_pages, seq_len, ws,
                                           reinterpret_cast<cudaStream_t>(stream)));
}

int reatt_paged_decode(const reatt_paged_dims *dims, const void *q, const void *k_pages,
                       const void *v_pages, const int32_t *page_table, const int32_t *seq_len,
                       void *out, void *ws, reatt_stream stream)
{
    PagedGeom g;
    const int rc = paged_geom(dims, &g);
    if (rc) return rc;
    if (g.N != g.B) return REATT_EINVAL;   // one query row per sequence
    if (!q || !k_pages || !v_pages || !page_table || !seq_len || !out || !ws) return REATT_EINVAL;
    if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(page_table) ||
        !aligned16(seq_len) || !aligned16(out) || !aligned16(ws))
        return REATT_EINVAL;
    return cuda_status(launch_paged_decode(g, q, k_pages, v_pages, page_table, seq_len, out,
                                           static_cast<uint8_t *>(ws) + kWsHeader, ws,
                                           reinterpret_cast<cudaStream_t>(stream)));
}

int reatt_prompt_attend(const reatt_paged_dims *dims, const void *q, const void *k, const void *v,
                        const int32_t *cu_seqlens, void *out, void *ws, reatt_stream stream)
{
    PagedGeom g;
    const int rc = paged_geom(dims, &g);
    if (rc) return rc;
    if (!cu_seqlens || !ws || (g.N > 0 && (!q || !k || !v || !out))) return REATT_EINVAL;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(cu_seqlens) || !aligned16(out) ||
        !aligned16(ws))
        return REATT_EINVAL;
    const cudaError_t e = launch_prompt(g, q, k, v, cu_seqlens, out, static_cast<uint8_t *>(ws) + kWsHeader,
                                        ws, reinterpret_cast<cudaStream_t>(stream));
    // more blocks than a grid holds (rows of one token each, thousands of heads)
    return e == cudaErrorInvalidConfiguration ? REATT_EUNSUPPORTED : cuda_status(e);
}

}  // extern "C"

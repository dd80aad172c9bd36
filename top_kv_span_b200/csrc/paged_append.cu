// Appending packed new tokens to a paged key-value cache, with the rotation at
// their positions on the way.
//
// Token i of sequence b sits at position p = past_len[b] + i.  With w_j =
// base^(-2j/d) the pairs (x_j, x_{j+d/2}) of a query or key head turn by p w_j:
//   y_j = x_j cos(p w_j) - x_{j+d/2} sin(p w_j)
//   y_{j+d/2} = x_{j+d/2} cos(p w_j) + x_j sin(p w_j)
// K goes rotated, V as it is, to slot p % page of the page that the table names
// for p / page; the rotated q (and k, if asked for) also go to packed rows.
// Every byte is read and written once, so memory bounds it: a block takes a few
// tokens, forms their d/2 angles once in shared memory (all heads of a token
// share them) and then moves 16-byte words.  16001 tokens of 32/8 heads of width 128
// take 79 us, 5.4 TB/s (84% of the copy bandwidth).  Against 80.5 us before it was
// launched beside the end of its predecessor: blocks of 128 or 512 threads 84 and 80,
// 8 tokens a block 84, streaming cache hints 82, the data loads ahead of the lookups 88.
// A call of one token takes 4 us of the GPU.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kernels.h"
#include "paged.cuh"

namespace reatt {
namespace {

constexpr int kAppThreads = 256;
constexpr int kAppMaxTokens = kAppThreads / 32;   // one warp looks up one token

template <typename T> struct Pack;
template <> struct Pack<float> {
    __device__ __forceinline__ static uint4 pack(const float (&v)[4])
    {
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                          __float_as_uint(v[3]));
    }
};
template <> struct Pack<uint16_t> {
    __device__ __forceinline__ static uint4 pack(const float (&v)[8])
    {
        uint4 w;
        uint32_t *u = reinterpret_cast<uint32_t *>(&w);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
            u[e] = *reinterpret_cast<const uint32_t *>(&t);
        }
        return w;
    }
};

struct AppendArgs {
    const void *q, *k, *v;
    const int32_t *cu, *past, *table;
    void *q_rot, *k_rot, *k_pages, *v_pages;
    int32_t *seq_len;
    void *ws;
    int tokens;   // tokens per block
};

template <typename T, int D>
__global__ void __launch_bounds__(kAppThreads)
paged_append_kernel(PagedGeom geo, AppendArgs a)
{
    constexpr int VEC = Elem<T>::kVec;       // elements of a 16-byte word
    constexpr int NCH = D / 2 / VEC;         // word pairs of a head row
    __shared__ float2 cs[kAppMaxTokens][D / 2];
    __shared__ int64_t dst[kAppMaxTokens];   // element offset of (page, head 0, slot), or < 0
    __shared__ int pos_s[kAppMaxTokens];     // position, or -1: not a row of any sequence
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t t0 = int64_t(blockIdx.x) * a.tokens;

    pdl_wait();
    if (a.seq_len)
        for (int64_t b = int64_t(blockIdx.x) * blockDim.x + tid; b < geo.B;
             b += int64_t(gridDim.x) * blockDim.x) {
            int s, e;
            packed_rows(a.cu, int(b), geo.N, s, e);
            a.seq_len[b] = a.past[b] + (e - s);
        }

    if (warp < a.tokens) {
        // the sequence of this token: the last one that starts at or before it
        const int64_t t = t0 + warp;
        const int n = count_up_to(a.cu, geo.B, t);
        int pos = -1;
        int64_t off = -1;
        if (n > 0 && t < geo.N) {
            int s, e;
            packed_rows(a.cu, n - 1, geo.N, s, e);
            if (t >= s && t < e) {
                const int64_t p = int64_t(a.past[n - 1]) + (t - s);
                const bool inside = p >= 0 && p < geo.capacity();
                pos = inside ? int(p) : 0;
                int id = -1;
                if (inside) id = a.table[int64_t(n - 1) * geo.max_pages + (p >> geo.page_shift)];
                if (id >= 0 && id < geo.n_pages)
                    off = ((int64_t(id) * geo.Hkv << geo.page_shift) +
                           (p & ((int64_t(1) << geo.page_shift) - 1))) * D;
                else if (lane == 0)
                    report_status(a.ws, REATT_EPAGE);
            }
        }
        if (lane == 0) {
            pos_s[warp] = pos;
            dst[warp] = off;
        }
        if (geo.rotate && pos >= 0)
            for (int i = lane; i < D / 2; i += 32) {
                float c, s;
                rope_cs(pos, geo.rope_hi[i], geo.rope_lo[i], c, s);
                cs[warp][i] = make_float2(c, s);
            }
    }
    __syncthreads();

    const int nq = a.q ? geo.Hq : 0;
    const int rows = nq + 2 * geo.Hkv, items = rows * NCH;
    const int64_t head = int64_t(D) << geo.page_shift;   // elements between a page's heads
    for (int x = tid; x < a.tokens * items; x += kAppThreads) {
        const int w = x / items, y = x - w * items, r = y / NCH, i0 = (y - r * NCH) * VEC;
        if (pos_s[w] < 0) continue;
        const int64_t t = t0 + w;
        const int h = r < nq ? r : (r - nq < geo.Hkv ? r - nq : r - nq - geo.Hkv);
        const bool is_q = r < nq, is_v = r >= nq + geo.Hkv;
        const T *src = is_q ? static_cast<const T *>(a.q) + t * geo.qs
                            : (is_v ? static_cast<const T *>(a.v) + t * geo.vs
                                    : static_cast<const T *>(a.k) + t * geo.ks);
        src += int64_t(h) * D + i0;
        uint4 lo = *reinterpret_cast<const uint4 *>(src);
        uint4 hi = *reinterpret_cast<const uint4 *>(src + D / 2);
        if (!is_v && geo.rotate) {
            float xl[VEC], xh[VEC], yl[VEC], yh[VEC];
            Elem<T>::unpack(lo, xl);
            Elem<T>::unpack(hi, xh);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float2 f = cs[w][i0 + e];
                yl[e] = xl[e] * f.x - xh[e] * f.y;
                yh[e] = xh[e] * f.x + xl[e] * f.y;
            }
            lo = Pack<T>::pack(yl);
            hi = Pack<T>::pack(yh);
        }
        auto put = [&](T *p) {
            *reinterpret_cast<uint4 *>(p) = lo;
            *reinterpret_cast<uint4 *>(p + D / 2) = hi;
        };
        if (is_q) {
            put(static_cast<T *>(a.q_rot) + t * geo.qrs + int64_t(h) * D + i0);
        } else {
            if (dst[w] >= 0)
                put(static_cast<T *>(is_v ? a.v_pages : a.k_pages) + dst[w] + h * head + i0);
            if (!is_v && a.k_rot)
                put(static_cast<T *>(a.k_rot) + t * geo.krs + int64_t(h) * D + i0);
        }
    }
}

}  // namespace

cudaError_t launch_paged_append(const PagedGeom &g, const void *q, const void *k, const void *v,
                                const int32_t *cu, const int32_t *past, const int32_t *table,
                                void *q_rot, void *k_rot, void *k_pages, void *v_pages,
                                int32_t *seq_len, void *ws, cudaStream_t st)
{
    AppendArgs a{q, k, v, cu, past, table, q_rot, k_rot, k_pages, v_pages, seq_len, ws, 1};
    // one token per block until there are enough for every SM, then several
    a.tokens = g.N <= int64_t(num_sms()) * 8 ? 1 : 4;
    int64_t blocks = (g.N + a.tokens - 1) / a.tokens;
    if (blocks < 1) {
        if (!seq_len) return cudaSuccess;
        blocks = 1;
    }
    auto kern = g.dtype == REATT_BF16
                    ? (g.d == 128 ? paged_append_kernel<uint16_t, 128> : paged_append_kernel<uint16_t, 64>)
                    : (g.d == 128 ? paged_append_kernel<float, 128> : paged_append_kernel<float, 64>);
    return launch_pdl(kern, dim3(unsigned(blocks)), dim3(kAppThreads), 0, st, g, a);
}

}  // namespace reatt

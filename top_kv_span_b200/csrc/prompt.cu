// Causal attention of packed prompts on the CUDA cores (fp32).
//
//   o_i = sum_{t <= i} softmax_t(q_i.k_t / sqrt(d)) v_t   within each sequence
//
// One CTA takes 64 consecutive tokens of one query head and walks its keys 64 at
// a time with the running maximum and sum of the softmax.  Scores and output
// stay in registers (4 x 4 and 4 x d/16 per thread); the arithmetic is fp32
// fused multiply-adds, which bound it.
#include <cuda_runtime.h>
#include <math.h>

#include "kernels.h"
#include "prompt.cuh"

namespace reatt {
namespace {

constexpr int kPrThreads = 256;
constexpr int kPrTile = 64;   // query tokens of a CTA, and keys of a tile

template <int D> struct PrSmem {
    static constexpr int QS = D + 4, PS = kPrTile + 4;   // padded rows: conflict-free columns
    static constexpr int oQ = 0, oK = oQ + kPrTile * QS, oV = oK + kPrTile * QS,
                         oP = oV + kPrTile * D;
    static constexpr size_t kBytes = size_t(oP + kPrTile * PS) * 4;
};

template <typename T, int D>
__global__ void __launch_bounds__(kPrThreads)
prompt_kernel(PagedGeom geo, const T *__restrict__ q, const T *__restrict__ k,
              const T *__restrict__ v, const int32_t *__restrict__ cu, T *__restrict__ out,
              float scale)
{
    using Sm = PrSmem<D>;
    constexpr int VEC = Elem<T>::kVec, CH = D / VEC, OC = D / 16;
    extern __shared__ __align__(16) float sm[];
    float *qs = sm + Sm::oQ, *ks = sm + Sm::oK, *vs = sm + Sm::oV, *ps = sm + Sm::oP;
    __shared__ PromptBlock blk_s;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    if (tid < 32) {
        const PromptBlock r = prompt_block(geo, cu, kPrTile, blockIdx.x / geo.Hq);
        if (tid == 0) blk_s = r;
    }
    __syncthreads();
    const PromptBlock blk = blk_s;
    if (!blk.live) return;
    const int j = blockIdx.x % geo.Hq, h = j / geo.g;
    const int nrow = min(kPrTile, blk.len - blk.q0);

    // rows [t0, t0 + 64) of a packed operand, rows from `n` on as zeros
    auto fill = [&](float *dst, int stride, const T *src, int64_t row_stride, int head, int t0, int n) {
        for (int x = tid; x < kPrTile * CH; x += kPrThreads) {
            const int r = x / CH, c = (x - r * CH) * VEC;
            float w[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) w[e] = 0.f;
            if (r < n)
                Elem<T>::unpack(*reinterpret_cast<const uint4 *>(
                                    src + int64_t(blk.begin + t0 + r) * row_stride + int64_t(head) * D + c),
                                w);
#pragma unroll
            for (int e = 0; e < VEC; e += 4)
                *reinterpret_cast<float4 *>(dst + r * stride + c + e) =
                    make_float4(w[e], w[e + 1], w[e + 2], w[e + 3]);
        }
    };
    fill(qs, Sm::QS, q, geo.qs, j, blk.q0, nrow);

    float o[4][OC], m[4], l[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.f;
#pragma unroll
        for (int c = 0; c < OC; ++c) o[r][c] = 0.f;
    }
    const int kend = blk.q0 + nrow;
    for (int k0 = 0; k0 < kend; k0 += kPrTile) {
        __syncthreads();
        fill(ks, Sm::QS, k, geo.ks, h, k0, kend - k0);
        fill(vs, D, v, geo.vs, h, k0, kend - k0);
        __syncthreads();
        const bool diag = k0 + kPrTile > blk.q0;
        float s[4][4];
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < 4; ++c) s[r][c] = 0.f;
#pragma unroll 4
        for (int e = 0; e < D; e += 4) {
            float4 a[4], b[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) a[r] = *reinterpret_cast<const float4 *>(qs + (ty * 4 + r) * Sm::QS + e);
#pragma unroll
            for (int c = 0; c < 4; ++c) b[c] = *reinterpret_cast<const float4 *>(ks + (tx + 16 * c) * Sm::QS + e);
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    s[r][c] = fmaf(a[r].x, b[c].x, s[r][c]);
                    s[r][c] = fmaf(a[r].y, b[c].y, s[r][c]);
                    s[r][c] = fmaf(a[r].z, b[c].z, s[r][c]);
                    s[r][c] = fmaf(a[r].w, b[c].w, s[r][c]);
                }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int tok = blk.q0 + ty * 4 + r;
            float mx = -INFINITY;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                s[r][c] = k0 + tx + 16 * c <= tok ? s[r][c] * scale : -INFINITY;
                mx = fmaxf(mx, s[r][c]);
            }
#pragma unroll
            for (int w = 1; w < 16; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
            const float mn = fmaxf(m[r], mx);
            const float fac = m[r] == -INFINITY ? 0.f : exp2f(m[r] - mn);
            m[r] = mn;
            l[r] *= fac;
#pragma unroll
            for (int c = 0; c < OC; ++c) o[r][c] *= fac;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float p = s[r][c] == -INFINITY ? 0.f : exp2f(s[r][c] - mn);
                l[r] += p;
                ps[(ty * 4 + r) * Sm::PS + tx + 16 * c] = p;
            }
        }
        __syncwarp();   // a row's probabilities come from the 16 threads that read them
#pragma unroll 4
        for (int kk = 0; kk < kPrTile; ++kk) {
            float vv[OC];
#pragma unroll
            for (int c = 0; c < OC; c += 4) {
                const float4 t = *reinterpret_cast<const float4 *>(vs + kk * D + (c / 4) * 64 + tx * 4);
                vv[c] = t.x; vv[c + 1] = t.y; vv[c + 2] = t.z; vv[c + 3] = t.w;
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                // a key after the row's token takes no part, whatever its value is
                const float p = ps[(ty * 4 + r) * Sm::PS + kk];
                if (!diag || k0 + kk <= blk.q0 + ty * 4 + r) {
#pragma unroll
                    for (int c = 0; c < OC; ++c) o[r][c] = fmaf(p, vv[c], o[r][c]);
                }
            }
        }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
#pragma unroll
        for (int w = 1; w < 16; w <<= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], w);
        if (ty * 4 + r < nrow) {
            const float il = 1.f / l[r];
            T *dst = out + (int64_t(blk.begin + blk.q0 + ty * 4 + r) * geo.Hq + j) * D;
#pragma unroll
            for (int c = 0; c < OC; c += 4) {
                *reinterpret_cast<float4 *>(dst + (c / 4) * 64 + tx * 4) =
                    make_float4(o[r][c] * il, o[r][c + 1] * il, o[r][c + 2] * il, o[r][c + 3] * il);
            }
        }
    }
}

template <typename T, int D>
cudaError_t run(const PagedGeom &g, const void *q, const void *k, const void *v, const int32_t *cu,
                void *out, cudaStream_t st)
{
    auto kern = prompt_kernel<T, D>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         int(PrSmem<D>::kBytes));
    if (e != cudaSuccess) return e;
    // every sequence has at most one block that is not full
    const int64_t blocks = (g.N / kPrTile + (g.B < g.N ? g.B : g.N)) * g.Hq;
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    kern<<<unsigned(blocks), kPrThreads, PrSmem<D>::kBytes, st>>>(
        g, static_cast<const T *>(q), static_cast<const T *>(k), static_cast<const T *>(v), cu,
        static_cast<T *>(out), float(1.4426950408889634 / sqrt(double(D))));
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prompt(const PagedGeom &g, const void *q, const void *k, const void *v,
                          const int32_t *cu, void *out, void *ws, cudaStream_t st)
{
    if (g.N == 0) return cudaSuccess;
    if (g.dtype == REATT_BF16) return launch_prompt_tc(g, q, k, v, cu, out, ws, st);
    return g.d == 128 ? run<float, 128>(g, q, k, v, cu, out, st) : run<float, 64>(g, q, k, v, cu, out, st);
}

}  // namespace reatt

// Causal attention of packed prompts on the CUDA cores (fp32).
//
//   o_i = sum_{t <= i} softmax_t(q_i.k_t / sqrt(d)) v_t   within each sequence
//
// One CTA takes 32 consecutive tokens of one query head and walks its keys 64 at
// a time with the running maximum and sum of the softmax.  Scores and output
// stay in registers (4 x 4 and 4 x d/16 per thread), and both products read four
// elements of either operand at a time from shared memory.  The next K tile loads
// during P.V and the next V tile during Q.K^T.  The arithmetic is fp32 fused
// multiply-adds, which bound it: MEASURED.
#include <cuda_runtime.h>
#include <math.h>

#include "kernels.h"
#include "prompt.cuh"

namespace reatt {
namespace {

constexpr int kPrRows = 32;   // query tokens of a CTA
constexpr int kPrKeys = 64;   // keys of a tile
constexpr int kPrThreads = kPrRows / 4 * 16;

// Padded rows: a column of them falls into different banks.
template <int D> struct PrSmem {
    static constexpr int RS = D + 4, PS = kPrKeys + 4;
    static constexpr int oQ = 0, oK = oQ + kPrRows * RS, oV = oK + kPrKeys * RS,
                         oP = oV + kPrKeys * RS;
    static constexpr size_t kBytes = size_t(oP + kPrRows * PS) * 4;
};

template <int D>
__global__ void __launch_bounds__(kPrThreads)
prompt_kernel(PagedGeom geo, const float *__restrict__ q, const float *__restrict__ k,
              const float *__restrict__ v, const int32_t *__restrict__ cu, float *__restrict__ out,
              float scale)
{
    using Sm = PrSmem<D>;
    constexpr int OC = D / 16;   // output columns of a thread, in fours 64 apart
    extern __shared__ __align__(16) float sm[];
    float *qs = sm + Sm::oQ, *ks = sm + Sm::oK, *vs = sm + Sm::oV, *ps = sm + Sm::oP;
    __shared__ PromptBlock blk_s;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    if (tid < 32) {
        const PromptBlock r = prompt_block(geo, cu, kPrRows, blockIdx.x / geo.Hq);
        if (tid == 0) blk_s = r;
    }
    __syncthreads();
    const PromptBlock blk = blk_s;
    if (!blk.live) return;
    const int j = blockIdx.x % geo.Hq, h = j / geo.g;
    const int nrow = min(kPrRows, blk.len - blk.q0), kend = blk.q0 + nrow;

    // `rows` rows of a packed operand from token t0 on, those past the block's last
    // token as zeros: a group of copies on its way
    auto fetch = [&](float *dst, int rows, const float *src, int64_t row_stride, int head, int t0) {
        for (int x = tid; x < rows * (D / 4); x += kPrThreads) {
            const int r = x / (D / 4), c = (x - r * (D / 4)) * 4;
            const bool in = t0 + r < kend;
            cp_async16(smem_addr(dst + r * Sm::RS + c),
                       src + (in ? int64_t(blk.begin + t0 + r) * row_stride + int64_t(head) * D + c : 0),
                       in);
        }
        cp_async_commit();
    };
    fetch(qs, kPrRows, q, geo.qs, j, blk.q0);
    fetch(ks, kPrKeys, k, geo.ks, h, 0);
    fetch(vs, kPrKeys, v, geo.vs, h, 0);

    float o[4][OC], m[4], l[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.f;
#pragma unroll
        for (int c = 0; c < OC; ++c) o[r][c] = 0.f;
    }
    for (int k0 = 0; k0 < kend; k0 += kPrKeys) {
        cp_async_wait<1>();   // Q and this K
        __syncthreads();
        float s[4][4];
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < 4; ++c) s[r][c] = 0.f;
#pragma unroll 4
        for (int e = 0; e < D; e += 4) {
            float4 a[4], b[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) a[r] = *reinterpret_cast<const float4 *>(qs + (ty * 4 + r) * Sm::RS + e);
#pragma unroll
            for (int c = 0; c < 4; ++c) b[c] = *reinterpret_cast<const float4 *>(ks + (tx + 16 * c) * Sm::RS + e);
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
        __syncthreads();
        if (k0 + kPrKeys < kend) fetch(ks, kPrKeys, k, geo.ks, h, k0 + kPrKeys);
        else cp_async_commit();
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
            const float fac = m[r] == -INFINITY ? 0.f : ex2_approx(m[r] - mn);
            m[r] = mn;
            l[r] *= fac;
#pragma unroll
            for (int c = 0; c < OC; ++c) o[r][c] *= fac;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float p = s[r][c] == -INFINITY ? 0.f : ex2_approx(s[r][c] - mn);
                l[r] += p;
                ps[(ty * 4 + r) * Sm::PS + tx + 16 * c] = p;
            }
        }
        cp_async_wait<1>();   // this V
        __syncthreads();
        // Four keys at a time.  In the last tiles a key after the row's token takes no
        // part, whatever its value is.
        auto products = [&](bool masked) {
#pragma unroll 2
            for (int kk = 0; kk < kPrKeys; kk += 4) {
                float4 p[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) p[r] = *reinterpret_cast<const float4 *>(ps + (ty * 4 + r) * Sm::PS + kk);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float vv[OC];
#pragma unroll
                    for (int c = 0; c < OC; c += 4) {
                        const float4 t = *reinterpret_cast<const float4 *>(vs + (kk + i) * Sm::RS + (c / 4) * 64 + tx * 4);
                        vv[c] = t.x; vv[c + 1] = t.y; vv[c + 2] = t.z; vv[c + 3] = t.w;
                    }
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        if (masked && k0 + kk + i > blk.q0 + ty * 4 + r) continue;
                        const float w = i == 0 ? p[r].x : i == 1 ? p[r].y : i == 2 ? p[r].z : p[r].w;
#pragma unroll
                        for (int c = 0; c < OC; ++c) o[r][c] = fmaf(w, vv[c], o[r][c]);
                    }
                }
            }
        };
        if (k0 + kPrKeys > blk.q0) products(true);
        else products(false);
        __syncthreads();
        if (k0 + kPrKeys < kend) fetch(vs, kPrKeys, v, geo.vs, h, k0 + kPrKeys);
        else cp_async_commit();
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
#pragma unroll
        for (int w = 1; w < 16; w <<= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], w);
        if (ty * 4 + r < nrow) {
            const float il = 1.f / l[r];
            float *dst = out + (int64_t(blk.begin + blk.q0 + ty * 4 + r) * geo.Hq + j) * D;
#pragma unroll
            for (int c = 0; c < OC; c += 4)
                *reinterpret_cast<float4 *>(dst + (c / 4) * 64 + tx * 4) =
                    make_float4(o[r][c] * il, o[r][c + 1] * il, o[r][c + 2] * il, o[r][c + 3] * il);
        }
    }
}

template <int D>
cudaError_t run(const PagedGeom &g, const void *q, const void *k, const void *v, const int32_t *cu,
                void *out, cudaStream_t st)
{
    auto kern = prompt_kernel<D>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         int(PrSmem<D>::kBytes));
    if (e != cudaSuccess) return e;
    // every sequence has at most one block that is not full
    const int64_t blocks = (g.N / kPrRows + (g.B < g.N ? g.B : g.N)) * g.Hq;
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    kern<<<unsigned(blocks), kPrThreads, PrSmem<D>::kBytes, st>>>(
        g, static_cast<const float *>(q), static_cast<const float *>(k), static_cast<const float *>(v), cu,
        static_cast<float *>(out), float(1.4426950408889634 / sqrt(double(D))));
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prompt(const PagedGeom &g, const void *q, const void *k, const void *v,
                          const int32_t *cu, void *out, void *ws, cudaStream_t st)
{
    if (g.N == 0) return cudaSuccess;
    if (g.dtype == REATT_BF16) return launch_prompt_tc(g, q, k, v, cu, out, ws, st);
    return g.d == 128 ? run<128>(g, q, k, v, cu, out, st) : run<64>(g, q, k, v, cu, out, st);
}

}  // namespace reatt

// Causal attention of packed prompts on the CUDA cores (fp32).
//
//   o_i = sum_{t <= i} softmax_t(q_i.k_t / sqrt(d)) v_t   within each sequence
//
// One CTA takes 32 consecutive tokens of one query head.  Its groups of four warps
// (four of them at width 64, one at 128) walk the keys 64 at a time in turn, each with a
// running maximum and sum of the softmax of its own, and join at the end, so that an SM
// works on few blocks at a time and the longest one does not outlast the others.  Scores
// and output stay in registers (4 x 4 and 4 x d/16 per thread), and both products read
// four elements of either operand at a time from shared memory.  A group's next K tile
// loads during P.V and its next V tile during Q.K^T.  The arithmetic is fp32
// multiply-adds; what bounds it are the registers' fills from shared memory, eight
// 16-byte loads for 64 multiply-adds of a
// thread.  K and V are read anew for every query head.  Two prompts of 4131 tokens
// together, 4/1 heads of width 64, take 154 us, 30 TFLOP/s (one group of four warps per
// CTA 210 us; mma.sync with operands split in two tf32 terms 160 us where this then took
// 162, at three times the error; tcgen05 was not tried).  Width 128 leaves room for two
// groups in one CTA or for two CTAs of one, which is faster: a prompt of 2000 tokens with
// 32/8 heads 988 us (962 now) against 1102.
#include <cuda_runtime.h>
#include <math.h>

#include "kernels.h"
#include "prompt.cuh"

namespace reatt {
namespace {

constexpr int kPrRows = 32;   // query tokens of a CTA
constexpr int kPrKeys = 64;   // keys of a tile
constexpr int kPrGroup = kPrRows / 4 * 16;   // threads of a group

// Padded rows: a column of them falls into different banks.  Q, then K, V and P of
// every group, as many groups as fit.
template <int D> struct PrSmem {
    static constexpr int kGroups = D == 64 ? 4 : 1;
    static constexpr int RS = D + 4, PS = kPrKeys + 4;
    static constexpr int oK = 0, oV = oK + kPrKeys * RS, oP = oV + kPrKeys * RS,
                         kOne = oP + kPrRows * PS, oGroups = kPrRows * RS;
    static constexpr int kThreads = kGroups * kPrGroup;
    static constexpr size_t kBytes = size_t(oGroups + kGroups * kOne) * 4;
};

template <int D>
__global__ void __launch_bounds__(PrSmem<D>::kThreads)
prompt_kernel(PagedGeom geo, const float *__restrict__ q, const float *__restrict__ k,
              const float *__restrict__ v, const int32_t *__restrict__ cu, float *__restrict__ out,
              float scale, const int32_t *plan)
{
    using Sm = PrSmem<D>;
    constexpr int OC = D / 16;   // output columns of a thread, in fours 64 apart
    extern __shared__ __align__(16) float sm[];
    __shared__ PromptBlock blk_s;
    __shared__ float2 row_ml[Sm::kGroups][kPrRows];
    const int group = threadIdx.x / kPrGroup, tid = threadIdx.x % kPrGroup, tx = tid & 15, ty = tid >> 4;
    float *qs = sm, *mine = sm + Sm::oGroups + group * Sm::kOne;
    float *ks = mine + Sm::oK, *vs = mine + Sm::oV, *ps = mine + Sm::oP;
    pdl_wait();
    if (threadIdx.x < 32) {
        const int i = blockIdx.x / geo.Hq;
        const PromptBlock r = plan ? planned_block(geo, cu, plan, kPrRows, i) : prompt_block(geo, cu, kPrRows, i);
        if (threadIdx.x == 0) blk_s = r;
    }
    __syncthreads();
    const PromptBlock blk = blk_s;
    if (!blk.live) return;
    const int j = blockIdx.x % geo.Hq, h = j / geo.g;
    const int nrow = min(kPrRows, blk.len - blk.q0), kend = blk.q0 + nrow;

    auto meet = [&] { named_sync(1 + group, kPrGroup); };
    // `rows` rows of a packed operand from token t0 on, those past the block's last
    // token as zeros: a group of copies on its way
    auto fetch = [&](float *dst, int rows, const float *src, int64_t row_stride, int head, int t0) {
        for (int x = tid; x < rows * (D / 4); x += kPrGroup) {
            const int r = x / (D / 4), c = (x - r * (D / 4)) * 4;
            const bool in = t0 + r < kend;
            cp_async16(smem_addr(dst + r * Sm::RS + c),
                       src + (in ? int64_t(blk.begin + t0 + r) * row_stride + int64_t(head) * D + c : 0),
                       in);
        }
        cp_async_commit();
    };
    constexpr int STEP = Sm::kGroups * kPrKeys;   // from one tile of a group to its next
    const int first = group * kPrKeys;
    if (group == 0) fetch(qs, kPrRows, q, geo.qs, j, blk.q0);
    cp_async_wait<0>();
    __syncthreads();
    if (first < kend) {
        fetch(ks, kPrKeys, k, geo.ks, h, first);
        fetch(vs, kPrKeys, v, geo.vs, h, first);
    }

    float m[4], l[4];
    uint64_t o[4][OC / 2];   // pairs of neighbouring columns
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.f;
#pragma unroll
        for (int c = 0; c < OC / 2; ++c) o[r][c] = 0;
    }
    for (int k0 = first; k0 < kend; k0 += STEP) {
        cp_async_wait<1>();   // this K
        meet();
        // sums over the even and the odd elements of d side by side
        uint64_t s2[4][4];
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < 4; ++c) s2[r][c] = 0;
#pragma unroll 4
        for (int e = 0; e < D; e += 4) {
            ulonglong2 a[4], b[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) a[r] = *reinterpret_cast<const ulonglong2 *>(qs + (ty * 4 + r) * Sm::RS + e);
#pragma unroll
            for (int c = 0; c < 4; ++c) b[c] = *reinterpret_cast<const ulonglong2 *>(ks + (tx + 16 * c) * Sm::RS + e);
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
                for (int c = 0; c < 4; ++c) s2[r][c] = fma2(a[r].y, b[c].y, fma2(a[r].x, b[c].x, s2[r][c]));
        }
        float s[4][4];
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                float even, odd;
                unpack2(s2[r][c], even, odd);
                s[r][c] = even + odd;
            }
        meet();
        if (k0 + STEP < kend) fetch(ks, kPrKeys, k, geo.ks, h, k0 + STEP);
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
            const uint64_t fac2 = pack2(fac, fac);
#pragma unroll
            for (int c = 0; c < OC / 2; ++c) o[r][c] = mul2(o[r][c], fac2);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const float p = s[r][c] == -INFINITY ? 0.f : ex2_approx(s[r][c] - mn);
                l[r] += p;
                ps[(ty * 4 + r) * Sm::PS + tx + 16 * c] = p;
            }
        }
        cp_async_wait<1>();   // this V
        meet();
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
                    uint64_t vv[OC / 2];
#pragma unroll
                    for (int c = 0; c < OC; c += 4) {
                        const ulonglong2 t = *reinterpret_cast<const ulonglong2 *>(vs + (kk + i) * Sm::RS + (c / 4) * 64 + tx * 4);
                        vv[c / 2] = t.x;
                        vv[c / 2 + 1] = t.y;
                    }
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        if (masked && k0 + kk + i > blk.q0 + ty * 4 + r) continue;
                        const float w = i == 0 ? p[r].x : i == 1 ? p[r].y : i == 2 ? p[r].z : p[r].w;
                        const uint64_t w2 = pack2(w, w);
#pragma unroll
                        for (int c = 0; c < OC / 2; ++c) o[r][c] = fma2(w2, vv[c], o[r][c]);
                    }
                }
            }
        };
        if (k0 + kPrKeys > blk.q0) products(true);
        else products(false);
        meet();
        if (k0 + STEP < kend) fetch(vs, kPrKeys, v, geo.vs, h, k0 + STEP);
        else cp_async_commit();
    }
    // join the groups: each leaves its rows' (m, l) and o (over its K tile), then every
    // thread adds up four elements
    meet();
#pragma unroll
    for (int r = 0; r < 4; ++r) {
#pragma unroll
        for (int w = 1; w < 16; w <<= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], w);
        if (tx == 0) row_ml[group][ty * 4 + r] = make_float2(m[r], l[r]);
#pragma unroll
        for (int c = 0; c < OC; c += 4)
            *reinterpret_cast<ulonglong2 *>(ks + (ty * 4 + r) * Sm::RS + (c / 4) * 64 + tx * 4) =
                make_ulonglong2(o[r][c / 2], o[r][c / 2 + 1]);
    }
    __syncthreads();
    for (int x = threadIdx.x; x < nrow * (D / 4); x += Sm::kThreads) {
        const int r = x / (D / 4), c = (x - r * (D / 4)) * 4;
        float M = row_ml[0][r].x;
#pragma unroll
        for (int i = 1; i < Sm::kGroups; ++i) M = fmaxf(M, row_ml[i][r].x);
        float L = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < Sm::kGroups; ++i) {
            const float2 ml = row_ml[i][r];
            const float f = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - M);
            const float4 t = *reinterpret_cast<const float4 *>(sm + Sm::oGroups + i * Sm::kOne + Sm::oK + r * Sm::RS + c);
            L = fmaf(f, ml.y, L);
            acc.x = fmaf(f, t.x, acc.x);
            acc.y = fmaf(f, t.y, acc.y);
            acc.z = fmaf(f, t.z, acc.z);
            acc.w = fmaf(f, t.w, acc.w);
        }
        const float il = 1.f / L;
        *reinterpret_cast<float4 *>(out + (int64_t(blk.begin + blk.q0 + r) * geo.Hq + j) * D + c) =
            make_float4(acc.x * il, acc.y * il, acc.z * il, acc.w * il);
    }
}

// The plan (prompt.cuh): one block of threads takes the sequences kPlanThreads at a time,
// once for every power of two that occurs, with a running sum over the block.
constexpr int kPlanThreads = 1024;
__global__ void __launch_bounds__(kPlanThreads)
prompt_plan_kernel(PagedGeom geo, const int32_t *__restrict__ cu, int TB, int32_t *plan)
{
    __shared__ uint32_t kinds;
    __shared__ int64_t warp_sum[kPlanThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int32_t *start = plan + 2, *order = start + geo.B + 1;
    if (tid == 0) kinds = 0;
    pdl_wait();
    __syncthreads();
    auto blocks_of = [&](int b) {
        int s, e;
        packed_rows(cu, b, geo.N, s, e);
        return (e - s + TB - 1) / TB;
    };
    uint32_t mine = 0;
    for (int b = tid; b < geo.B; b += kPlanThreads) {
        const int n = blocks_of(b);
        if (n > 0) mine |= 1u << (31 - __clz(n));
    }
    mine = __reduce_or_sync(0xffffffffu, mine);
    if (lane == 0) atomicOr(&kinds, mine);
    __syncthreads();
    int listed = 0;
    int64_t blocks = 0;   // (offsets that overlap can have more than 32 bits hold)
    for (uint32_t left = kinds; left;) {
        const int kind = 31 - __clz(left);
        left &= ~(1u << kind);
        for (int b0 = 0; b0 < geo.B; b0 += kPlanThreads) {
            const int b = b0 + tid, n = b < geo.B ? blocks_of(b) : 0;
            const bool in = n > 0 && 31 - __clz(n) == kind;
            // blocks of the listed ones up to this thread, and how many they are
            int64_t sum = in ? n : 0;
            int count = in;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t up = __shfl_up_sync(0xffffffffu, sum, o);
                const int up_count = __shfl_up_sync(0xffffffffu, count, o);
                if (lane >= o) {
                    sum += up;
                    count += up_count;
                }
            }
            // sums are below 2^41, counts of a block of threads below 2^11
            if (lane == 31) warp_sum[warp] = (sum << 12) | count;
            __syncthreads();
            int64_t before = 0, all = 0;
            for (int w = 0; w < kPlanThreads / 32; ++w) {
                if (w < warp) before += warp_sum[w];
                all += warp_sum[w];
            }
            if (in) {
                const int at = listed + int(before & 4095) + count - 1;
                const int64_t x = blocks + (before >> 12) + sum - n;
                start[at] = int32_t(x < 0x7fffffff ? x : 0x7fffffff);
                order[at] = b;
            }
            listed += int(all & 4095);
            blocks += all >> 12;
            __syncthreads();
        }
    }
    if (tid == 0) {
        plan[0] = listed;
        plan[1] = int32_t(blocks < 0x7fffffff ? blocks : 0x7fffffff);
    }
}

template <int D>
cudaError_t run(const PagedGeom &g, const void *q, const void *k, const void *v, const int32_t *cu,
                void *out, int32_t *plan, cudaStream_t st)
{
    const int64_t blocks = prompt_blocks(g, kPrRows) * g.Hq;
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    auto kern = prompt_kernel<D>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         int(PrSmem<D>::kBytes));
    if (e == cudaSuccess && plan) e = launch_prompt_plan(g, cu, kPrRows, plan, st);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(unsigned(blocks)), dim3(PrSmem<D>::kThreads), PrSmem<D>::kBytes, st, g,
                      static_cast<const float *>(q), static_cast<const float *>(k),
                      static_cast<const float *>(v), cu, static_cast<float *>(out),
                      float(1.4426950408889634 / sqrt(double(D))), static_cast<const int32_t *>(plan));
}

}  // namespace

size_t prompt_ws_bytes(const PagedGeom &g) { return prompt_plan_bytes(g); }

cudaError_t launch_prompt_plan(const PagedGeom &g, const int32_t *cu, int TB, int32_t *plan, cudaStream_t st)
{
    return launch_pdl(prompt_plan_kernel, dim3(1), dim3(kPlanThreads), 0, st, g, cu, TB, plan);
}

cudaError_t launch_prompt(const PagedGeom &g, const void *q, const void *k, const void *v,
                          const int32_t *cu, void *out, void *scratch, void *ws, cudaStream_t st)
{
    if (g.N == 0) return cudaSuccess;
    int32_t *plan = prompt_plan_bytes(g) ? static_cast<int32_t *>(scratch) : nullptr;
    if (g.dtype == REATT_BF16) return launch_prompt_tc(g, q, k, v, cu, out, plan, ws, st);
    return g.d == 128 ? run<128>(g, q, k, v, cu, out, plan, st) : run<64>(g, q, k, v, cu, out, plan, st);
}

}  // namespace reatt

// Causal attention of packed prompts on the tensor cores (bf16, tcgen05 + TMEM).
//
//   o_i = sum_{t <= i} softmax_t(q_i.k_t / sqrt(d)) v_t   within each sequence
//
// A row is one (token, query head) pair of a KV head, heads innermost, so the g
// query heads of a token lie in one tile and a K/V tile is read once for all of
// them.  A CTA takes two tiles of floor(128 / g) tokens each (TMEM lanes = rows)
// and walks the keys 128 at a time, S = Q.K^T and O += P.V as M128 x N128 (N = d)
// products, with the running maximum and sum of the softmax:
//   warps 0-3, 4-7  softmax of tile 0, 1: a thread owns a row; it reads its S
//            values from TMEM, masks, keeps a reference maximum that moves (and
//            rescales its row of O in TMEM) only when the row's maximum grows by
//            more than 2^8, and writes P = 2^(x - m) as bf16 over its own S tile
//   warp 8   TMA producer: K(0), V(0), K(1), V(1) ... through one ring
//   warps 9, 10  one thread per tile issues its products: P(j).V(j) and then
//            S(j+1), so that one tile's products run while the other's softmax
//            does.  S(j+1) may overwrite P(j) as the same thread issued P(j).V(j)
//            before it and products execute in the order of their issue
//   warp 11  TMEM allocation
// The logits are exact products summed in fp32; P rounds to bf16 (its operand
// type; the row sum takes the unrounded value), O is summed in fp32.
//
// Values behind the mask: a masked S is replaced before it is used, but a masked
// P = 0 still meets its V row in the product, so in the key tiles that hold any
// masked key the softmax warps first look V over: rows past the sequence become
// zeros, and so do infinities and NaN, which the last step then adds to the rows
// that do see them (a slow path that only such inputs take).
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <math.h>

#include "kernels.h"
#include "prompt.cuh"
#include "tc_ptx.cuh"

namespace reatt {
namespace {

using namespace tc;

constexpr int kPtThreads = 12 * 32;
constexpr int kPtRows = 128;    // rows of a tile (TMEM lanes)
constexpr int kPtKeys = 128;    // keys of a tile
constexpr float kPtMove = 8.f;  // log2 growth of a row's maximum that moves its reference
constexpr uint32_t kPtS = 0, kPtO = 256, kPtCols = 512;   // TMEM columns: S0 | S1 | O0 | O1

template <int D> struct PtSmem {
    static constexpr int NBOX = D / 64;                  // 64-element boxes of a row
    static constexpr int kQ = NBOX * kPtRows * 128;      // one Q tile
    static constexpr int kStage = NBOX * kPtKeys * 128;  // one K or V tile
    static constexpr int kStages = D == 128 ? 5 : 10;
    static constexpr int oQ = 0, oRing = 2 * kQ, oBar = oRing + kStages * kStage;
    static constexpr size_t kBytes = size_t(oBar) + 64 * 8 + 1024;
};

__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, int x, int y, int z,
                                            uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
        : "memory");
}
// 2^x on the special-function unit (relative error about 2^-22; 2^-inf = 0).
__device__ __forceinline__ float pt_ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ bool bf16x2_odd(uint32_t w)   // an infinity or NaN in either half
{
    return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

template <int D>
__global__ void __launch_bounds__(kPtThreads, 1)
prompt_tc_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                 const __grid_constant__ CUtensorMap vmap, PagedGeom geo,
                 const int32_t *__restrict__ cu, const uint16_t *__restrict__ v,
                 uint16_t *__restrict__ out, float scale, void *ws)
{
    using Sm = PtSmem<D>;
    constexpr int NS = Sm::kStages, NBOX = Sm::NBOX;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~uintptr_t(1023));
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Sm::oBar);
    uint64_t *qfull = bars, *full = bars + 1, *empty = full + NS, *sfull = empty + NS,
             *pfull = sfull + 2, *odone = pfull + 2, *done = odone + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + 2);
    __shared__ int abort_flag, odd_v;
    __shared__ PromptBlock blk_s;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int TPT = kPtRows / geo.g, TB = 2 * TPT;   // tokens of a tile, of the block
    const int h = blockIdx.x % geo.Hkv;
    if (warp == 8) {
        const PromptBlock r = prompt_block(geo, cu, TB, blockIdx.x / geo.Hkv);
        if (lane == 0) blk_s = r;
    } else if (warp == 11) {
        tmem_alloc(tmem_slot, kPtCols);
        tmem_relinquish();
    } else if (tid == 0) {
        abort_flag = odd_v = 0;
        mbar_init(qfull, 1);
        for (int s = 0; s < NS; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 2);   // both tiles' products have read the stage
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(&sfull[t], 1);
            mbar_init(&pfull[t], 4);   // P written (one arrival per softmax warp)
            mbar_init(&odone[t], 1);   // P.V complete
            mbar_init(&done[t], 1);    // all products of the tile complete
        }
        mbar_init_fence();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const PromptBlock blk = blk_s;
    if (!blk.live) {
        __syncthreads();
        if (warp == 11) tmem_dealloc(tmem_base, kPtCols);
        return;
    }
    // tokens and key tiles of each row tile (none past the sequence)
    auto tile_tokens = [&](int t) { return max(0, min(TPT, blk.len - blk.q0 - t * TPT)); };
    auto key_tiles = [&](int t) {
        const int n = tile_tokens(t);
        return n ? (blk.q0 + t * TPT + n + kPtKeys - 1) / kPtKeys : 0;
    };
    const int nt_all = max(key_tiles(0), key_tiles(1));
    const int j_odd = blk.q0 / kPtKeys;   // from this key tile on some key is masked

    auto fail = [&]() {
        report_status(ws, REATT_ETIMEOUT);
        *(volatile int *)&abort_flag = 1;
    };
    auto aborted = [&]() { return *(volatile int *)&abort_flag != 0; };
    auto wait = [&](uint64_t *bar, int use) {
        return mbar_wait_bounded(bar, uint32_t(use) & 1u, kWaitLimitNs);
    };

    if (warp == 8) {
        // ------------------------------------------------ TMA producer
        if (lane == 0) {
            const int nq = key_tiles(1) ? 2 : 1;
            mbar_arrive_expect_tx(qfull, uint32_t(nq * NBOX * TPT * geo.g * 128));
            for (int t = 0; t < nq; ++t)
                for (int bx = 0; bx < NBOX; ++bx)
                    tma_load_3d(smem + Sm::oQ + t * Sm::kQ + bx * kPtRows * 128, &qmap, 64 * bx,
                                h * geo.g, blk.begin + blk.q0 + t * TPT, qfull);
            int i = 0;
            for (; i < 2 * nt_all; ++i) {
                const int s = i % NS, u = i / NS;
                if (aborted() || (u > 0 && !wait(&empty[s], u - 1))) {
                    fail();
                    break;
                }
                mbar_arrive_expect_tx(&full[s], Sm::kStage);
                for (int bx = 0; bx < NBOX; ++bx)
                    tma_load_3d(smem + Sm::oRing + s * Sm::kStage + bx * kPtKeys * 128,
                                i & 1 ? &vmap : &kmap, 64 * bx, h, blk.begin + (i / 2) * kPtKeys,
                                &full[s]);
            }
            // the copies in flight land before the CTA may leave
            if (!wait(qfull, 0)) fail();
            for (int x = max(0, i - NS); x < i; ++x)
                if (!wait(&full[x % NS], x / NS)) fail();
        }
    } else if (warp == 9 || warp == 10) {
        // ------------------------------------------------ issuer of one tile's products
        if (lane == 0) {
            const int t = warp - 9, nt = key_tiles(t);
            constexpr uint32_t id_s = idesc_bf16(kPtRows, kPtKeys);
            constexpr uint32_t id_o = idesc_bf16(kPtRows, D) | (1u << 16);   // V read MN-major
            const uint32_t t_s = tmem_base + kPtS + uint32_t(t * kPtKeys);
            const uint32_t t_o = tmem_base + kPtO + uint32_t(t * 128);
            const uint8_t *qt = smem + Sm::oQ + t * Sm::kQ;
            bool ok = !aborted() && wait(qfull, 0);
            if (!ok) fail();
            for (int j = 0; ok && j < nt_all; ++j) {
                const int sk = (2 * j) % NS, sv = (2 * j + 1) % NS;
                if (aborted() || !wait(&full[sk], (2 * j) / NS)) {
                    fail();
                    break;
                }
                if (j < nt) {
                    tc_fence_after();
                    const uint8_t *kt = smem + Sm::oRing + sk * Sm::kStage;
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks)
                        tc_mma(t_s, sw128_desc(qt + (ks / 4) * kPtRows * 128) + uint64_t((ks % 4) * 2),
                               sw128_desc(kt + (ks / 4) * kPtKeys * 128) + uint64_t((ks % 4) * 2), id_s,
                               ks > 0 ? 1u : 0u);
                    tc_commit(&sfull[t]);
                    tc_commit(&empty[sk]);
                } else {
                    mbar_arrive(&empty[sk]);
                }
                if (aborted() || !wait(&full[sv], (2 * j + 1) / NS) || (j < nt && !wait(&pfull[t], j))) {
                    fail();
                    break;
                }
                if (j < nt) {
                    tc_fence_after();
                    const uint64_t vd = sw128_mn_desc(smem + Sm::oRing + sv * Sm::kStage, kPtKeys * 128);
#pragma unroll
                    for (int ks = 0; ks < kPtKeys / 16; ++ks)   // 16 keys are 2048 bytes of V rows
                        tc_mma_ts(t_o, t_s + uint32_t(ks * 8), vd + uint64_t(ks * 128), id_o,
                                  (j > 0 || ks > 0) ? 1u : 0u);
                    tc_commit(&odone[t]);
                    tc_commit(&empty[sv]);
                } else {
                    mbar_arrive(&empty[sv]);
                }
            }
            tc_commit(&done[t]);
            if (!wait(&done[t], 0)) fail();
        }
    } else if (warp < 8) {
        // ------------------------------------------------ softmax, one row per thread
        const int t = warp >> 2, nt = key_tiles(t);
        const int row = (warp & 3) * 32 + lane;
        const uint32_t lanes = tmem_base + (uint32_t((warp & 3) * 32) << 16);
        const uint32_t t_s = lanes + kPtS + uint32_t(t * kPtKeys), t_o = lanes + kPtO + uint32_t(t * 128);
        const int tok = blk.q0 + t * TPT + row / geo.g;   // token within the sequence
        const bool live = row < tile_tokens(t) * geo.g;
        const int lim = live ? tok : -1;                  // last key that the row sees
        float m = -INFINITY, l = 0.f;                     // reference maximum (of the raw products), sum
        bool ok = true;
        for (int j = 0; j < nt; ++j) {
            if (j >= j_odd) {
                // look V(j) over: 16-byte words of this thread; the swizzle only
                // permutes words within a key's 128-byte row
                const int sv = (2 * j + 1) % NS;
                ok = __all_sync(0xffffffffu, !aborted() && wait(&full[sv], (2 * j + 1) / NS));
                if (!ok) {
                    if (lane == 0) fail();
                    break;
                }
                uint8_t *vt = smem + Sm::oRing + sv * Sm::kStage;
                for (int x = row * 16; x < Sm::kStage; x += kPtRows * 16) {
                    uint4 *p = reinterpret_cast<uint4 *>(vt + x);
                    if (j * kPtKeys + ((x >> 7) & (kPtKeys - 1)) >= blk.len) {
                        *p = make_uint4(0, 0, 0, 0);
                        continue;
                    }
                    uint4 w = *p;
                    if (bf16x2_odd(w.x) || bf16x2_odd(w.y) || bf16x2_odd(w.z) || bf16x2_odd(w.w)) {
                        atomicOr(&odd_v, 1);
                        __threadfence_block();
                        uint32_t *u = reinterpret_cast<uint32_t *>(&w);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            if ((u[e] & 0x7f80u) == 0x7f80u) u[e] &= 0xffff0000u;
                            if ((u[e] & 0x7f800000u) == 0x7f800000u) u[e] &= 0xffffu;
                        }
                        *p = w;
                    }
                }
                fence_proxy_async_smem();   // before this warp's arrival for P(j)
            }
            ok = __all_sync(0xffffffffu, !aborted() && wait(&sfull[t], j));
            if (!ok) {
                if (lane == 0) fail();
                break;
            }
            tc_fence_after();
            float s[kPtKeys];
            {
                uint32_t a[32], b[32], c[32], d[32];
                tmem_ld32_nowait(t_s, a);
                tmem_ld32_nowait(t_s + 32, b);
                tmem_ld32_nowait(t_s + 64, c);
                tmem_ld32_nowait(t_s + 96, d);
                tmem_wait_ld();
                tmem_regs_after_wait(a);
                tmem_regs_after_wait(b);
                tmem_regs_after_wait(c);
                tmem_regs_after_wait(d);
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    s[i] = __uint_as_float(a[i]);
                    s[32 + i] = __uint_as_float(b[i]);
                    s[64 + i] = __uint_as_float(c[i]);
                    s[96 + i] = __uint_as_float(d[i]);
                }
            }
            const int k0 = j * kPtKeys;
            if (k0 + kPtKeys - 1 > lim) {
#pragma unroll
                for (int i = 0; i < kPtKeys; ++i)
                    if (k0 + i > lim) s[i] = -INFINITY;
            }
            float pm[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) pm[i] = s[i];
#pragma unroll
            for (int i = 8; i < kPtKeys; ++i) pm[i & 7] = fmaxf(pm[i & 7], s[i]);
            const float mx = fmaxf(fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3])),
                                   fmaxf(fmaxf(pm[4], pm[5]), fmaxf(pm[6], pm[7])));
            const bool first = m == -INFINITY;
            const bool move = mx != -INFINITY && (first || (mx - m) * scale > kPtMove);
            float fac = 1.f;
            if (move) {
                fac = first ? 0.f : pt_ex2((m - mx) * scale);
                m = mx;
                l *= fac;
            }
            if (j > 0 && __any_sync(0xffffffffu, move && !first)) {
                // O is at rest: P(j-1).V(j-1) is complete and P(j).V(j) waits for this P
                ok = __all_sync(0xffffffffu, !aborted() && wait(&odone[t], j - 1));
                if (!ok) {
                    if (lane == 0) fail();
                    break;
                }
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    float o[32];
                    tmem_ld32(t_o + uint32_t(c), o);
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] *= fac;
                    tmem_st32(t_o + uint32_t(c), o);
                }
            }
            // masked keys are -inf and give 0; without any key yet m is -inf: all give 0
            const float mc = m == -INFINITY ? 0.f : m * scale;
            float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float w[32];
#pragma unroll
                for (int i = 0; i < 64; i += 2) {
                    const float p0 = pt_ex2(fmaf(s[c * 64 + i], scale, -mc));
                    const float p1 = pt_ex2(fmaf(s[c * 64 + i + 1], scale, -mc));
                    sum[(i / 2) & 3] += p0 + p1;
                    const __nv_bfloat162 b2 = __floats2bfloat162_rn(p0, p1);
                    w[i / 2] = __uint_as_float(*reinterpret_cast<const uint32_t *>(&b2));
                }
                tmem_st32(t_s + uint32_t(c * 32), w);
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&pfull[t]);
        }
        if (ok && nt > 0) {
            ok = __all_sync(0xffffffffu, !aborted() && wait(&odone[t], nt - 1));
            if (!ok) {
                if (lane == 0) fail();
            } else {
                tc_fence_after();
                const bool odd = *(volatile int *)&odd_v != 0;
                const float il = 1.f / l;   // a live row sees itself; l = 0 only if all logits are -inf
                uint16_t *dst = out + (int64_t(blk.begin + tok) * geo.Hq + h * geo.g + row % geo.g) * D;
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    float o[32];
                    tmem_ld32(t_o + uint32_t(c), o);
                    if (odd && live)
                        for (int key = j_odd * kPtKeys; key <= tok; ++key) {
                            const uint16_t *vr = v + int64_t(blk.begin + key) * geo.vs + int64_t(h) * D + c;
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if ((vr[i] & 0x7f80u) == 0x7f80u)
                                    o[i] += __uint_as_float(uint32_t(vr[i]) << 16);
                        }
                    if (live) {
#pragma unroll
                        for (int i = 0; i < 32; i += 8) {
                            uint4 w;
                            uint32_t *u = reinterpret_cast<uint32_t *>(&w);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const __nv_bfloat162 b2 =
                                    __floats2bfloat162_rn(o[i + 2 * e] * il, o[i + 2 * e + 1] * il);
                                u[e] = *reinterpret_cast<const uint32_t *>(&b2);
                            }
                            *reinterpret_cast<uint4 *>(dst + c + i) = w;
                        }
                    }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 11) tmem_dealloc(tmem_base, kPtCols);
}

// Packed rows [N, H, d] at a row stride, boxes of 64 elements x heads x tokens.
bool packed_map(CUtensorMap *mp, const void *base, int64_t N, int H, int d, int64_t row_stride,
                uint32_t heads, uint32_t tokens)
{
    // the driver's encoder, looked up once (a magic static: thread-safe)
    static const PFN_cuTensorMapEncodeTiled_v12000 enc = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }();
    if (!enc) return false;
    cuuint64_t dims[3] = {cuuint64_t(d), cuuint64_t(H), cuuint64_t(N)};
    cuuint64_t strides[2] = {cuuint64_t(d) * 2, cuuint64_t(row_stride) * 2};
    cuuint32_t box[3] = {64, heads, tokens};
    cuuint32_t estr[3] = {1, 1, 1};
    return enc(mp, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box,
               estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t run(const PagedGeom &g, const void *q, const void *k, const void *v, const int32_t *cu,
                void *out, void *ws, cudaStream_t st)
{
    const int TPT = kPtRows / g.g, TB = 2 * TPT;
    CUtensorMap qm, km, vm;
    if (!packed_map(&qm, q, g.N, g.Hq, D, g.qs, uint32_t(g.g), uint32_t(TPT)) ||
        !packed_map(&km, k, g.N, g.Hkv, D, g.ks, 1, kPtKeys) ||
        !packed_map(&vm, v, g.N, g.Hkv, D, g.vs, 1, kPtKeys))
        return cudaErrorInvalidValue;
    // every sequence has at most one block that is not full
    const int64_t blocks = (g.N / TB + (g.B < g.N ? g.B : g.N)) * g.Hkv;
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    auto kern = prompt_tc_kernel<D>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         int(PtSmem<D>::kBytes));
    if (e != cudaSuccess) return e;
    kern<<<unsigned(blocks), kPtThreads, PtSmem<D>::kBytes, st>>>(
        qm, km, vm, g, cu, static_cast<const uint16_t *>(v), static_cast<uint16_t *>(out),
        float(1.4426950408889634 / sqrt(double(D))), ws);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prompt_tc(const PagedGeom &g, const void *q, const void *k, const void *v,
                             const int32_t *cu, void *out, void *ws, cudaStream_t st)
{
    return g.d == 128 ? run<128>(g, q, k, v, cu, out, ws, st) : run<64>(g, q, k, v, cu, out, ws, st);
}

}  // namespace reatt

// Causal attention of packed prompts on the tensor cores (bf16, tcgen05 + TMEM).
//
//   o_i = sum_{t <= i} softmax_t(q_i.k_t / sqrt(d)) v_t   within each sequence
//
// A row is one (token, query head) pair of a KV head, heads innermost, so the g
// query heads of a token lie in one tile and a K/V tile is read once for all of
// them.  A CTA takes two tiles of floor(128 / g) tokens each (TMEM lanes = rows)
// and walks the keys 64 at a time (a step), S = Q.K^T and O += P.V as products of
// M = 128 and N = 64 or d, with the running maximum and sum of the softmax:
//   warps 0-3, 4-7  softmax of tile 0, 1: a thread owns a row; it reads its S
//            values from TMEM, masks, keeps a reference maximum that moves (and
//            rescales its row of O in TMEM) only when the row's maximum grows by
//            more than 2^8, and writes P = 2^(x - m) as bf16 over its own S
//   warp 8   TMA producer: a ring of pairs, first {K(0), K(1)}, then {V(s), K(s+2)}
//   warps 9, 10  one thread per tile issues its products, P(s).V(s) and then
//            S(s+2).  Each tile has two S buffers, so S(s+1) waits there while the
//            softmax of step s runs and the softmax warps go from step to step
//            without a pause.  S(s+2) may overwrite P(s): the same thread issued
//            P(s).V(s) before it, and products execute in the order of their issue
//   warp 11  TMEM allocation
// What bounds it: the exponentials, 128 x 64 a tile and step at 16 per clock and SM,
// as long as the products take, and what the softmax warps do besides.  A prompt of
// 16384 tokens with 32/8 heads of width 128 takes 2.01 ms, 1.10 PFLOP/s.  Measured
// and dropped there: 128-key steps with one S buffer per tile, the other way to fill
// the 512 TMEM columns, which leave the chain S -> softmax -> P.V -> S open (2.22 ms);
// two threads per row (2.63 ms); a part of the exponentials as a polynomial on the FMA
// pipe, which costs more issue slots than it frees (2.05 ms for a quarter).
// The logits are exact products summed in fp32; P rounds to bf16 (its operand
// type; the row sum takes the unrounded value), O is summed in fp32.
//
// Values behind the mask: a masked S is replaced before it is used, but a masked
// P = 0 still meets its V row in the product, so in the steps that hold any
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

constexpr int kPtSoft = 8;      // softmax warps
constexpr int kPtThreads = (kPtSoft + 4) * 32;
constexpr int kPtRows = 128;    // rows of a tile (TMEM lanes)
constexpr int kPtKeys = 64;     // keys of a step
constexpr float kPtMove = 8.f;  // log2 growth of a row's maximum that moves its reference
// TMEM columns: tile 0's two S buffers, tile 1's, O of tile 0, of tile 1
constexpr uint32_t kPtS = 0, kPtO = 256, kPtCols = 512;

// Behind the operands in shared memory.
struct PtShared {
    uint64_t qfull, full[8], empty[8], sfull[2][2], pfull[2][2], odone[2], done[2], turn[2];
    uint32_t tmem;
    int abort_flag, odd_v;
    PromptBlock blk;
};

template <int D> struct PtSmem {
    static constexpr int NBOX = D / 64;                  // 64-element boxes of a row
    static constexpr int kQ = NBOX * kPtRows * 128;      // one Q tile
    static constexpr int kHalf = NBOX * kPtKeys * 128;   // K or V of a step
    static constexpr int kStage = 2 * kHalf;             // a pair
    static constexpr int kStages = D == 128 ? 5 : 8;
    static constexpr int oQ = 0, oRing = 2 * kQ, oBar = oRing + kStages * kStage;
    static constexpr size_t kBytes = size_t(oBar) + sizeof(PtShared);
    static_assert(kBytes <= 227 * 1024, "shared memory of a CTA");
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
// Two fp32 values in one 64-bit register and packed arithmetic on them.
__device__ __forceinline__ uint64_t pack2(float a, float b)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float &a, float &b)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// 16 registers into 16 consecutive columns of this thread's TMEM lane, without
// the wait.
__device__ __forceinline__ void tmem_st16_nowait(uint32_t taddr, const uint32_t (&v)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
        "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// One lane of the (converged) warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
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
    extern __shared__ __align__(1024) uint8_t smem[];   // no static shared memory before it
    PtShared &sh = *reinterpret_cast<PtShared *>(smem + Sm::oBar);
    if ((smem_addr(smem) & 1023u) != 0) return;   // never: the window starts aligned
    uint64_t *qfull = &sh.qfull, *full = sh.full, *empty = sh.empty, *odone = sh.odone,
             *done = sh.done;

    // the warp's index as a warp-uniform value
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int TPT = kPtRows / geo.g, TB = 2 * TPT;   // tokens of a tile, of the block
    const int h = blockIdx.x % geo.Hkv;
    if (warp == kPtSoft) {
        if (lane < 3) prefetch_tensormap(lane == 0 ? &qmap : lane == 1 ? &kmap : &vmap);
        const PromptBlock r = prompt_block(geo, cu, TB, blockIdx.x / geo.Hkv);
        if (lane == 0) sh.blk = r;
    } else if (warp == kPtSoft + 3) {
        tmem_alloc(&sh.tmem, kPtCols);
        tmem_relinquish();
    } else if (tid == 0) {
        sh.abort_flag = sh.odd_v = 0;
        mbar_init(qfull, 1);
        for (int s = 0; s < NS; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 2);   // both tiles' products have read the stage
        }
        for (int t = 0; t < 2; ++t) {
            for (int b = 0; b < 2; ++b) {
                mbar_init(&sh.sfull[t][b], 1);
                mbar_init(&sh.pfull[t][b], 4);   // P written (one arrival per softmax warp)
            }
            mbar_init(&sh.turn[t], 4);    // the tile's exponentials are done
            mbar_init(&odone[t], 1);   // P(n-2).V(n-2) complete
            mbar_init(&done[t], 1);    // all products of the tile complete
        }
        mbar_init_fence();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = sh.tmem;
    const PromptBlock blk = sh.blk;
    if (!blk.live) {
        __syncthreads();
        if (warp == kPtSoft + 3) tmem_dealloc(tmem_base, kPtCols);
        return;
    }
    // tokens and steps of each row tile (none past the sequence)
    auto tile_tokens = [&](int t) { return max(0, min(TPT, blk.len - blk.q0 - t * TPT)); };
    auto steps = [&](int t) {
        const int n = tile_tokens(t);
        return n ? (blk.q0 + t * TPT + n + kPtKeys - 1) / kPtKeys : 0;
    };
    const int ns = max(steps(0), steps(1));
    const int s_odd = blk.q0 / kPtKeys;   // from this step on some key is masked
    auto fail = [&]() {
        report_status(ws, REATT_ETIMEOUT);
        *(volatile int *)&sh.abort_flag = 1;
    };
    auto aborted = [&]() { return *(volatile int *)&sh.abort_flag != 0; };
    auto wait = [&](uint64_t *bar, int use) {
        return mbar_wait_bounded(bar, uint32_t(use) & 1u, kWaitLimitNs);
    };
    // the same by polling, for the waits of the chain S -> P -> O: a poll answers
    // sooner than a suspended wait, and reading the global timer would take longer
    // than most waits, so the limit counts polls (2^26 of at least 20 cycles)
    auto poll = [&](uint64_t *bar, int use) {
        for (int i = 1; !mbar_test(bar, uint32_t(use) & 1u); ++i)
            if ((i & 1023) == 0 && (aborted() || i >= (1 << 26))) return false;
        return true;
    };

    // registers move from the four service warps to the softmax warps:
    // 8 x 216 + 4 x 72 = 12 x 168 a lane
    if (warp >= kPtSoft) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == kPtSoft) {
        // ------------------------------------------------ TMA producer
        if (lane == 0) {
            const int nq = steps(1) ? 2 : 1;
            mbar_arrive_expect_tx(qfull, uint32_t(nq * NBOX * TPT * geo.g * 128));
            for (int t = 0; t < nq; ++t)
                for (int bx = 0; bx < NBOX; ++bx)
                    tma_load_3d(smem + Sm::oQ + t * Sm::kQ + bx * kPtRows * 128, &qmap, 64 * bx,
                                h * geo.g, blk.begin + blk.q0 + t * TPT, qfull);
            int i = 0;
            for (; i <= ns; ++i) {
                const int r = i % NS, u = i / NS, xk = i + 1;   // {V(i-1), K(i+1)}; i = 0: {K(0), K(1)}
                if (aborted() || (u > 0 && !wait(&empty[r], u - 1))) {
                    fail();
                    break;
                }
                uint8_t *st = smem + Sm::oRing + r * Sm::kStage;
                mbar_arrive_expect_tx(&full[r], xk < ns ? Sm::kStage : Sm::kHalf);
                for (int bx = 0; bx < NBOX; ++bx) {
                    tma_load_3d(st + bx * kPtKeys * 128, i ? &vmap : &kmap, 64 * bx, h,
                                blk.begin + (i ? i - 1 : 0) * kPtKeys, &full[r]);
                    if (xk < ns)
                        tma_load_3d(st + Sm::kHalf + bx * kPtKeys * 128, &kmap, 64 * bx, h,
                                    blk.begin + xk * kPtKeys, &full[r]);
                }
            }
            // the copies in flight land before the CTA may leave
            if (!wait(qfull, 0)) fail();
            for (int x = max(0, i - NS); x < i; ++x)
                if (!wait(&full[x % NS], x / NS)) fail();
        }
    } else if (warp <= kPtSoft + 2) {
        // ------------------------------------------------ issuer of one tile's products
        // The whole warp walks the steps, so that the operands' descriptors live in
        // uniform registers, and one elected lane issues (a loop of one lane alone
        // took 75 cycles per product for moving them there).
        const int t = warp - kPtSoft - 1, n = steps(t);
        constexpr uint32_t id_s = idesc_bf16(kPtRows, kPtKeys);
        constexpr uint32_t id_o = idesc_bf16(kPtRows, D) | (1u << 16);   // V read MN-major
        const uint32_t t_s = tmem_base + kPtS + uint32_t(t * 2 * kPtKeys);
        const uint32_t t_o = tmem_base + kPtO + uint32_t(t * 128);
        const uint64_t qd = sw128_desc(smem + Sm::oQ + t * Sm::kQ), ring = sw128_desc(smem + Sm::oRing),
                       ringv = sw128_mn_desc(smem + Sm::oRing, kPtKeys * 128);
        auto issue_s = [&](int x, uint64_t kd) {
            const uint32_t d = t_s + uint32_t((x & 1) * kPtKeys);
            if (elect_one()) {
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    tc_mma(d, qd + uint64_t((ks / 4) * (kPtRows * 128 / 16) + (ks % 4) * 2),
                           kd + uint64_t((ks / 4) * (kPtKeys * 128 / 16) + (ks % 4) * 2), id_s,
                           ks > 0 ? 1u : 0u);
                tc_commit(&sh.sfull[t][x & 1]);
            }
            __syncwarp();
        };
        auto release = [&](int r, bool used) {   // the stage, once the products issued so far are complete
            if (elect_one()) {
                if (used) tc_commit(&empty[r]);
                else mbar_arrive(&empty[r]);
            }
            __syncwarp();
        };
        bool ok = poll(qfull, 0) && poll(&full[0], 0);
        tc_fence_after();
        if (ok && n > 0) issue_s(0, ring);
        if (ok && n > 1) issue_s(1, ring + uint64_t(Sm::kHalf / 16));
        if (ok) release(0, n > 0);
        for (int x = 0; ok && x < ns; ++x) {
            const int r = (x + 1) % NS;
            ok = poll(&full[r], (x + 1) / NS) && (x >= n || poll(&sh.pfull[t][x & 1], x >> 1));
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            if (x < n) {
                tc_fence_after();
                const uint64_t vd = ringv + uint64_t(r * (Sm::kStage / 16));
                const uint32_t p = t_s + uint32_t((x & 1) * kPtKeys);
                if (elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < kPtKeys / 16; ++ks)   // 16 keys are 2048 bytes of V rows
                        tc_mma_ts(t_o, p + uint32_t(ks * 8), vd + uint64_t(ks * 128), id_o,
                                  (x > 0 || ks > 0) ? 1u : 0u);
                    if (x + 2 == n) tc_commit(&odone[t]);   // no S tells of P(n-2).V(n-2)
                }
                __syncwarp();
                if (x + 2 < n) issue_s(x + 2, ring + uint64_t((r * Sm::kStage + Sm::kHalf) / 16));
            }
            release(r, x < n);   // unused: the other tile has more steps
        }
        if (!ok && lane == 0) fail();
        if (elect_one()) tc_commit(&done[t]);
        __syncwarp();
        if (!wait(&done[t], 0) && lane == 0) fail();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        // ------------------------------------------------ softmax, one row per thread
        const int t = warp >> 2, n = steps(t), n_other = steps(t ^ 1);
        const int quad = warp & 3, row = quad * 32 + lane;
        const uint32_t lanes = tmem_base + (uint32_t(quad * 32) << 16);
        const uint32_t t_o = lanes + kPtO + uint32_t(t * 128);
        const int tok = blk.q0 + t * TPT + row / geo.g;   // token within the sequence
        const bool live = row < tile_tokens(t) * geo.g;
        const int lim = live ? tok : -1;                  // last key that the row sees
        const float lift = kPtMove / scale;               // growth that moves the reference
        float m = -INFINITY, l = 0.f;                     // reference maximum (of the raw products), sum
        bool ok = true;
        for (int j = 0; j < n; ++j) {
            const uint32_t t_s = lanes + kPtS + uint32_t((t * 2 + (j & 1)) * kPtKeys);
            if (j >= s_odd) {
                // look V(j) over: 16-byte words of this thread; the swizzle only
                // permutes words within a key's 128-byte row
                const int r = (j + 1) % NS;
                ok = ok && __all_sync(0xffffffffu, poll(&full[r], (j + 1) / NS));
                uint8_t *vt = smem + Sm::oRing + r * Sm::kStage;
                for (int x = row * 16; x < Sm::kHalf; x += kPtRows * 16) {
                    uint4 *p = reinterpret_cast<uint4 *>(vt + x);
                    if (j * kPtKeys + ((x >> 7) & (kPtKeys - 1)) >= blk.len) {
                        *p = make_uint4(0, 0, 0, 0);
                        continue;
                    }
                    uint4 w = *p;
                    if (bf16x2_odd(w.x) || bf16x2_odd(w.y) || bf16x2_odd(w.z) || bf16x2_odd(w.w)) {
                        atomicOr(&sh.odd_v, 1);
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
            ok = ok && __all_sync(0xffffffffu, poll(&sh.sfull[t][j & 1], j >> 1));
            if (!ok) {
                if (lane == 0) fail();
                break;
            }
            tc_fence_after();
            float s[kPtKeys];
            {
                uint32_t a[2][32];
#pragma unroll
                for (int c = 0; c < 2; ++c) tmem_ld32_nowait(t_s + uint32_t(c * 32), a[c]);
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    tmem_regs_after_wait(a[c]);
#pragma unroll
                    for (int i = 0; i < 32; ++i) s[c * 32 + i] = __uint_as_float(a[c][i]);
                }
            }
            const int k0 = j * kPtKeys;
            if (k0 + kPtKeys - 1 > lim) {
#pragma unroll
                for (int i = 0; i < kPtKeys; ++i)
                    if (k0 + i > lim) s[i] = -INFINITY;
            }
            // (a NaN logit is passed over here; its weight is NaN, and so is its row)
            float pm[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int i = 0; i < kPtKeys; i += 2) pm[i / 2 & 3] = fmaxf(pm[i / 2 & 3], fmaxf(s[i], s[i + 1]));
            const float mx = fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3]));
            // the reference stays while no row's maximum has grown by 2^8
            if (__any_sync(0xffffffffu, !(mx <= m + lift))) {
                const bool first = m == -INFINITY;
                const bool move = mx != -INFINITY && (first || !(mx <= m + lift));
                float fac = 1.f;
                if (move) {
                    fac = first ? 0.f : pt_ex2((m - mx) * scale);
                    m = mx;
                    l *= fac;
                }
                if (j > 0 && __any_sync(0xffffffffu, move && !first)) {
                    // O is at rest once P(j-1).V(j-1) is complete, as P(j).V(j) waits for
                    // this P; S(j+1) was issued after it and tells of it
                    ok = __all_sync(0xffffffffu, j + 1 < n ? poll(&sh.sfull[t][(j + 1) & 1], (j + 1) >> 1)
                                                           : poll(&odone[t], 0));
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
            }
            // masked keys are -inf and give 0; without any key yet m is -inf: all give 0
            const float mc = m == -INFINITY ? 0.f : m * scale;
            // The tiles' exponentials start in turn, half a step apart: one tile's
            // exponentials run beside the other's products and maxima.  (Left alone
            // the tiles fall into step and leave the special-function units, which
            // bound the kernel, idle in between: 2.14 instead of 2.01 ms.)
            const int jo = t ? j : j - 1;   // the other tile's step that goes first
            if (jo >= 0 && jo < n_other) {
                ok = __all_sync(0xffffffffu, poll(&sh.turn[t ^ 1], jo));
                if (!ok) {
                    if (lane == 0) fail();
                    break;
                }
            }
            const uint64_t sc2 = pack2(scale, scale), mc2 = pack2(-mc, -mc);
            uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t w[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const uint64_t x = fma2(pack2(s[c * 32 + 2 * i], s[c * 32 + 2 * i + 1]), sc2, mc2);
                    float p0, p1;
                    unpack2(x, p0, p1);
                    p0 = pt_ex2(p0);
                    p1 = pt_ex2(p1);
                    sum[i & 3] = add2(sum[i & 3], pack2(p0, p1));
                    const __nv_bfloat162 b2 = __floats2bfloat162_rn(p0, p1);
                    w[i] = *reinterpret_cast<const uint32_t *>(&b2);
                }
                tmem_st16_nowait(t_s + uint32_t(c * 16), w);
                if (c == 0) {   // half way, so that the hand-over costs no pause
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh.turn[t]);
                }
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.pfull[t][j & 1]);
            const uint64_t l2 = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
            float l0, l1;
            unpack2(l2, l0, l1);
            l += l0 + l1;
        }
        if (ok && n > 0) {
            ok = __all_sync(0xffffffffu, !aborted() && wait(&done[t], 0));
            if (!ok) {
                if (lane == 0) fail();
            } else {
                tc_fence_after();
                const bool odd = *(volatile int *)&sh.odd_v != 0;
                const float il = 1.f / l;   // a live row sees itself; l = 0 only if all logits are -inf
                uint16_t *dst = out + (int64_t(blk.begin + tok) * geo.Hq + h * geo.g + row % geo.g) * D;
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    float o[32];
                    tmem_ld32(t_o + uint32_t(c), o);
                    if (odd && live)
                        for (int key = s_odd * kPtKeys; key <= tok; ++key) {
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
    if (warp == kPtSoft + 3) tmem_dealloc(tmem_base, kPtCols);
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

// Causal attention of packed prompts on the tensor cores (bf16, tcgen05 + TMEM).
//
//   o_i = sum_{t <= i} softmax_t(q_i.k_t / sqrt(d)) v_t   within each sequence
//
// A row is one (token, query head) pair of a KV head, heads innermost, so the g
// query heads of a token lie in one tile and a K/V tile is read once for all of
// them.  A block is two tiles of floor(128 / g) tokens each (TMEM lanes = rows) of one
// KV head.  A CTA per SM takes one block after another (claiming the
// places of CTAs that have not started), the long ones first, and
// each block's keys 64 at a time (a step), S = Q.K^T and O += P.V as products of
// M = 128 and N = 64 or d, with the running maximum and sum of the softmax:
//   warps 0-3, 4-7  softmax of tile 0, 1: a thread owns a row; it reads its S
//            values from TMEM, masks, keeps a reference maximum that moves (and
//            rescales its row of O in TMEM) only when the row's maximum grows by
//            more than 2^8, and writes P = 2^(x - m) as bf16 over its own S; at the
//            block's end it divides its row of O by the sum and stores it
//   warp 8   claims and finds the blocks, and loads by TMA: Q as soon as the last block's S
//            products have read theirs, and a ring of pairs, first {K(0), K(1)}, then
//            {V(s), K(s+2)}, that runs on from block to block
//   warps 9, 10  issue one tile's products each, P(s).V(s) and then
//            S(s+2).  Each tile has two S buffers, so S(s+1) waits there while the
//            softmax of step s runs and the softmax warps go from step to step
//            without a pause.  S(s+2) may overwrite P(s): the same thread issued
//            P(s).V(s) before it, and products execute in the order of their issue
//   warp 11  TMEM allocation
// The roles meet only at barriers whose phases count on from block to block, so the
// next block's loads and first S run during the last steps and the stores of this one.
// What bounds it: the exponentials, 128 x 64 a tile and step at 16 per clock and SM,
// as long as the products take, and what the softmax warps do besides; in long runs the
// power limit.  A prompt of 16384 tokens, 32/8 heads of width 128, takes 1.74 ms by itself
// and 1.99 ms in a loop (1.26 and 1.10 PFLOP/s), seven prompts of 8191 tokens together
// 127 us: 86 steps an SM of 0.97 us, and 7 blocks, whose ends (the look over V, the wait for
// the last product, O on its way out, while the next block's softmax waits) take about
// 6 us each.  Measured and dropped, on the way there (16384 tokens, in a loop, against what
// stood then): 128-key steps with one S buffer per tile, the other way to fill the 512
// TMEM columns, which leave the chain S -> softmax -> P.V -> S open (2.22 ms, 2.01); two
// threads per row (2.63 ms, 2.31); a quarter of the exponentials as a polynomial on the
// FMA pipe (2.05 ms, 2.01); S loaded a step ahead, which spills (3.18 ms, 2.07); one
// block per CTA, whose loads and stores stand alone (152 us for the seven prompts, 133).
// The logits are exact products summed in fp32; P rounds to bf16 (its operand type), O is
// summed in fp32, and so is the row sum, of the rounded values: a weight's rounding then
// moves a row by its share of v - o, not of v (error against 64 bits of the seven prompts
// 0.0021 -> 0.0019, the fp32 form's 0.0016; values that all tokens share come back exact).
// Summing the unrounded values took 125 us and 1.96 ms, this then 128 us and 2.03 ms (with
// the halves widened by integer instructions 133 us and 2.13 ms).
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

#include <atomic>
#include <type_traits>

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

// Behind the operands in shared memory.  Index [2]: the tile, or the block's parity.
struct PtShared {
    uint64_t info_full[2], info_empty[2];   // blk[] written, read by every role
    uint64_t qfull, qempty;                 // Q landed, read by the block's last S products
    uint64_t full[8], empty[8];             // a ring stage landed, read by both tiles' products
    uint64_t sfull[2][2], pfull[2][2];      // S complete, P written: [tile][buffer]
    uint64_t odone[2];                      // P(n-2).V(n-2) complete
    uint64_t done[2], oempty[2];            // the block's O complete, read
    uint64_t last[2];                       // all products complete
    uint64_t turn[2];                       // a step's exponentials half done
    uint64_t claim;                         // the next block's index has come
    PromptBlock blk[2];
    int head[2];                            // its KV head
    alignas(16) uint8_t claimed[16];
    uint32_t tmem;
    int abort_flag;
    int odd[4];                             // block (mod 4) whose V had infinities or NaN, + 1
};

template <int D> struct PtSmem {
    static constexpr int NBOX = D / 64;                  // 64-element boxes of a row
    static constexpr int kQ = NBOX * kPtRows * 128;      // one Q tile
    static constexpr int kHalf = NBOX * kPtKeys * 128;   // K or V of a step
    static constexpr int kStage = 2 * kHalf;             // a pair
    static constexpr int kStages = D == 128 ? 4 : 8;
    static constexpr int kOut = kPtRows * 128;           // a tile's output on its way, 64 elements of a row
    static constexpr int oQ = 0, oRing = 2 * kQ, oOut = oRing + kStages * kStage, oBar = oOut + 2 * kOut;
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
// Cluster launch control: asks for a CTA of this grid that has not started; the 16-byte
// answer lands in shared memory and completes the mbarrier's transaction.
__device__ __forceinline__ void claim_cta(void *answer, uint64_t *bar)
{
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                     smem_addr(answer)),
                 "r"(smem_addr(bar))
                 : "memory");
}
// The claimed CTA's index, which will not start by itself, or -1: none was left.
__device__ __forceinline__ int claimed_cta(const void *answer)
{
    uint32_t got, x;
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b128 h;\n\t"
        "ld.shared.b128 h, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
        "selp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
        : "=r"(got), "=r"(x)
        : "r"(smem_addr(answer))
        : "memory");
    return got ? int(x) : -1;
}
// One lane of the (converged) warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}
// Adds the two bf16 values of a word to two fp32 sums, exactly widened.
__device__ __forceinline__ void add_bf16x2(float &a, float &b, uint32_t w)
{
    asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\t"
        "add.rn.f32.bf16 %0, x, %0;\n\tadd.rn.f32.bf16 %1, y, %1;\n\t}"
        : "+f"(a), "+f"(b)
        : "r"(w));
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
                 uint16_t *__restrict__ out, float scale, const int32_t *plan, void *ws)
{
    using Sm = PtSmem<D>;
    constexpr int NS = Sm::kStages, NBOX = Sm::NBOX;
    extern __shared__ __align__(1024) uint8_t smem[];   // no static shared memory before it
    PtShared &sh = *reinterpret_cast<PtShared *>(smem + Sm::oBar);
    if ((smem_addr(smem) & 1023u) != 0) return;   // never: the window starts aligned

    // the warp's index as a warp-uniform value
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int TPT = kPtRows / geo.g, TB = 2 * TPT;   // tokens of a tile, of a block
    if (warp == kPtSoft) {
        if (lane < 3) prefetch_tensormap(lane == 0 ? &qmap : lane == 1 ? &kmap : &vmap);
    } else if (warp == kPtSoft + 3) {
        tmem_alloc(&sh.tmem, kPtCols);
        tmem_relinquish();
    } else if (tid == 0) {
        sh.abort_flag = 0;
        for (int i = 0; i < 4; ++i) sh.odd[i] = 0;
        mbar_init(&sh.qfull, 1);
        mbar_init(&sh.claim, 1);
        mbar_init(&sh.qempty, 2);
        for (int r = 0; r < NS; ++r) {
            mbar_init(&sh.full[r], 1);
            mbar_init(&sh.empty[r], 2);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(&sh.turn[t], 4);
            mbar_init(&sh.info_full[t], 1);
            mbar_init(&sh.info_empty[t], kPtSoft + 2);
            for (int b = 0; b < 2; ++b) {
                mbar_init(&sh.sfull[t][b], 1);
                mbar_init(&sh.pfull[t][b], 4);   // one arrival per softmax warp
            }
            mbar_init(&sh.odone[t], 1);
            mbar_init(&sh.done[t], 1);
            mbar_init(&sh.oempty[t], 4);
            mbar_init(&sh.last[t], 1);
        }
        mbar_init_fence();
    }
    pdl_wait();   // the set-up above may run beside the end of the kernel before
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = sh.tmem;

    auto fail = [&]() {
        report_status(ws, REATT_ETIMEOUT);
        *(volatile int *)&sh.abort_flag = 1;
    };
    auto aborted = [&]() { return *(volatile int *)&sh.abort_flag != 0; };
    auto wait = [&](uint64_t *bar, int use) {
        return mbar_wait_bounded(bar, uint32_t(use) & 1u, kWaitLimitNs);
    };
    // the same by polling, for the waits of the chain S -> P -> O: a poll answers sooner
    // than a suspended wait, and reading the global timer would take longer than most
    // waits, so the limit counts polls (2^26 of at least 20 cycles); it also ends when
    // another wait has failed
    auto poll = [&](uint64_t *bar, int use) {
        for (int i = 1; !mbar_test(bar, uint32_t(use) & 1u); ++i)
            if ((i & 1023) == 0 && (aborted() || i >= (1 << 26))) return false;
        return true;
    };
    struct Block {
        int begin, len, q0, h;   // the sequence's first row and length, first token, KV head
        int rows0, rows1;        // tokens of each tile and its steps (none past the
        int n0, n1, ns;          // sequence), most steps
        bool live;
        __device__ int rows(int t) const { return t ? rows1 : rows0; }
        __device__ int n(int t) const { return t ? n1 : n0; }
    };
    auto block_of = [&](const PromptBlock &p, int h) {
        auto rows_of = [&](int t) { return max(0, min(TPT, p.len - p.q0 - t * TPT)); };
        auto steps = [&](int t, int rows) {
            return rows ? (p.q0 + t * TPT + rows + kPtKeys - 1) / kPtKeys : 0;
        };
        Block b;
        b.live = p.live;
        b.begin = p.begin;
        b.len = p.len;
        b.q0 = p.q0;
        b.h = h;
        b.rows0 = rows_of(0);
        b.rows1 = rows_of(1);
        b.n0 = steps(0, b.rows0);
        b.n1 = steps(1, b.rows1);
        b.ns = max(b.n0, b.n1);
        return b;
    };
    // block k as every role but the producer gets it (dead: no more, or a failed wait)
    auto next_block = [&](int k) {
        const bool got = __all_sync(0xffffffffu, poll(&sh.info_full[k & 1], k >> 1));
        PromptBlock p{0, 0, 0, false};
        int h = 0;
        if (got) {
            p = sh.blk[k & 1];
            h = sh.head[k & 1];
        }
        __syncwarp();
        if (got && lane == 0) mbar_arrive(&sh.info_empty[k & 1]);
        if (!got && lane == 0) fail();
        return block_of(p, h);
    };

    // registers move from the four service warps to the softmax warps:
    // 8 x 216 + 4 x 72 = 12 x 168 a lane
    if (warp >= kPtSoft) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == kPtSoft) {
            // ------------------------------------------------ blocks and loads
            int item = 0, loads = 0;   // ring items and Q tiles loaded so far
            bool ok = true;
            // this CTA's own place in the list of blocks, then those it claims from CTAs
            // that have not started: the list descends in work, so the SMs end together
            int i = blockIdx.x;
            for (int k = 0;; ++k) {
                PromptBlock p{0, 0, 0, false};
                if (i >= 0)
                    p = plan ? planned_block(geo, cu, plan, TB, i / geo.Hkv)
                             : prompt_block(geo, cu, TB, i / geo.Hkv);
                const Block b = block_of(p, i < 0 ? 0 : i % geo.Hkv);
                if (lane == 0) {
                    if (b.live) {
                        mbar_arrive_expect_tx(&sh.claim, 16);
                        claim_cta(sh.claimed, &sh.claim);
                    }
                    ok = k < 2 || wait(&sh.info_empty[k & 1], (k >> 1) - 1);
                    if (ok) {
                        sh.blk[k & 1] = p;
                        sh.head[k & 1] = b.h;
                        mbar_arrive(&sh.info_full[k & 1]);
                    }
                    if (ok && b.live) {
                        ok = k == 0 || wait(&sh.qempty, k - 1);
                        if (ok) {
                            const int nq = b.n1 ? 2 : 1;
                            ++loads;
                            mbar_arrive_expect_tx(&sh.qfull, uint32_t(nq * NBOX * TPT * geo.g * 128));
                            for (int t = 0; t < nq; ++t)
                                for (int bx = 0; bx < NBOX; ++bx)
                                    tma_load_3d(smem + Sm::oQ + t * Sm::kQ + bx * kPtRows * 128, &qmap,
                                                64 * bx, b.h * geo.g, b.begin + b.q0 + t * TPT, &sh.qfull);
                        }
                        for (int x = 0; ok && x <= b.ns; ++x, ++item) {
                            const int r = item % NS, u = item / NS, xk = x + 1;   // {V(x-1), K(x+1)}
                            ok = !aborted() && (u == 0 || wait(&sh.empty[r], u - 1));
                            if (!ok) break;
                            uint8_t *st = smem + Sm::oRing + r * Sm::kStage;
                            mbar_arrive_expect_tx(&sh.full[r], xk < b.ns ? Sm::kStage : Sm::kHalf);
                            for (int bx = 0; bx < NBOX; ++bx) {
                                tma_load_3d(st + bx * kPtKeys * 128, x ? &vmap : &kmap, 64 * bx, b.h,
                                            b.begin + (x ? x - 1 : 0) * kPtKeys, &sh.full[r]);
                                if (xk < b.ns)
                                    tma_load_3d(st + Sm::kHalf + bx * kPtKeys * 128, &kmap, 64 * bx, b.h,
                                                b.begin + xk * kPtKeys, &sh.full[r]);
                            }
                        }
                    }
                    if (b.live) {
                        ok = wait(&sh.claim, k) && ok;
                        i = claimed_cta(sh.claimed);
                        fence_proxy_async_smem();   // read before the next claim is answered there
                    }
                    if (!ok) fail();
                }
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok || !b.live) break;
                i = __shfl_sync(0xffffffffu, i, 0);
            }
            if (lane == 0) {
                // the copies in flight land before the CTA may leave
                if (loads > 0 && !wait(&sh.qfull, loads - 1)) fail();
                for (int x = max(0, item - NS); x < item; ++x)
                    if (!wait(&sh.full[x % NS], x / NS)) fail();
            }
        } else if (warp <= kPtSoft + 2) {
            // ------------------------------------------------ issuer of one tile's products
            // The whole warp walks the steps, so that the operands' descriptors live in
            // uniform registers, and one elected lane issues (a loop of one lane alone
            // took 75 cycles per product for moving them there).
            const int t = warp - kPtSoft - 1;
            constexpr uint32_t id_s = idesc_bf16(kPtRows, kPtKeys);
            constexpr uint32_t id_o = idesc_bf16(kPtRows, D) | (1u << 16);   // V read MN-major
            const uint32_t t_s = tmem_base + kPtS + uint32_t(t * 2 * kPtKeys);
            const uint32_t t_o = tmem_base + kPtO + uint32_t(t * 128);
            const uint64_t qd = sw128_desc(smem + Sm::oQ + t * Sm::kQ), ring = sw128_desc(smem + Sm::oRing),
                           ringv = sw128_mn_desc(smem + Sm::oRing, kPtKeys * 128);
            int item = 0, step = 0, used = 0;   // ring items, this tile's steps and blocks so far
            // S of the tile's step g, with the block's last one Q is free again
            auto issue_s = [&](int g, uint64_t kd, bool last) {
                const uint32_t d = t_s + uint32_t((g & 1) * kPtKeys);
                if (elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks)
                        tc_mma(d, qd + uint64_t((ks / 4) * (kPtRows * 128 / 16) + (ks % 4) * 2),
                               kd + uint64_t((ks / 4) * (kPtKeys * 128 / 16) + (ks % 4) * 2), id_s,
                               ks > 0 ? 1u : 0u);
                    tc_commit(&sh.sfull[t][g & 1]);
                    if (last) tc_commit(&sh.qempty);
                }
                __syncwarp();
            };
            auto release = [&](int r, bool read) {   // the stage, once the products issued so far are complete
                if (elect_one()) {
                    if (read) tc_commit(&sh.empty[r]);
                    else mbar_arrive(&sh.empty[r]);
                }
                __syncwarp();
            };
            bool ok = true;
            for (int k = 0; ok; ++k) {
                const Block b = next_block(k);
                if (!b.live) break;
                const int n = b.n(t);
                ok = poll(&sh.qfull, k) && poll(&sh.full[item % NS], item / NS);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                const uint64_t kd = ring + uint64_t((item % NS) * (Sm::kStage / 16));
                if (n > 0) issue_s(step, kd, n == 1);
                if (n > 1) issue_s(step + 1, kd + uint64_t(Sm::kHalf / 16), n == 2);
                if (n == 0) {
                    if (elect_one()) mbar_arrive(&sh.qempty);
                    __syncwarp();
                }
                release(item % NS, n > 0);
                ++item;
                for (int x = 0; x < b.ns; ++x, ++item) {
                    const int r = item % NS, g = step + x;
                    ok = poll(&sh.full[r], item / NS) && (x >= n || poll(&sh.pfull[t][g & 1], g >> 1)) &&
                         (x > 0 || n == 0 || used == 0 || poll(&sh.oempty[t], used - 1));
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    if (x < n) {
                        tc_fence_after();
                        const uint64_t vd = ringv + uint64_t(r * (Sm::kStage / 16));
                        const uint32_t p = t_s + uint32_t((g & 1) * kPtKeys);
                        if (elect_one()) {
#pragma unroll
                            for (int ks = 0; ks < kPtKeys / 16; ++ks)   // 16 keys are 2048 bytes of V rows
                                tc_mma_ts(t_o, p + uint32_t(ks * 8), vd + uint64_t(ks * 128), id_o,
                                          (x > 0 || ks > 0) ? 1u : 0u);
                            if (x + 2 == n) tc_commit(&sh.odone[t]);   // no S tells of P(n-2).V(n-2)
                            if (x + 1 == n) tc_commit(&sh.done[t]);
                        }
                        __syncwarp();
                        if (x + 2 < n)
                            issue_s(g + 2, ring + uint64_t((r * Sm::kStage + Sm::kHalf) / 16), x + 3 == n);
                    }
                    release(r, x < n);   // not read: the other tile has more steps
                }
                step += n;
                used += n > 0;
            }
            if (!ok && lane == 0) fail();
            if (elect_one()) tc_commit(&sh.last[t]);
            __syncwarp();
            if (!wait(&sh.last[t], 0) && lane == 0) fail();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        // ------------------------------------------------ softmax, one row per thread
        const int t = warp >> 2, quad = warp & 3, row = quad * 32 + lane;
        const uint32_t lanes = tmem_base + (uint32_t(quad * 32) << 16);
        const uint32_t t_o = lanes + kPtO + uint32_t(t * 128);
        const float lift = kPtMove / scale;    // growth that moves the reference
        const int inv_g = (65536 + geo.g - 1) / geo.g;
        int item = 0, step = 0, pace = 0;      // ring items, this tile's steps, the blocks' steps so far
        int used = 0, twos = 0;                // blocks of at least one step, of two
        bool ok = true;
        for (int k = 0; ok; ++k) {
            const Block b = next_block(k);
            if (!b.live) break;
            const int n = b.n(t);
            const int s_odd = b.q0 / kPtKeys;   // from this step on some key is masked
            const int tok = b.q0 + t * TPT + row / geo.g;   // token within the sequence
            const bool live = row < b.rows(t) * geo.g;
            const int lim = live ? tok : -1;                // last key that the row sees
            float m = -INFINITY, l = 0.f;                   // reference maximum (of the raw products), sum
            // The tiles' exponentials start in turn, half a step apart: one tile's
            // exponentials run beside the other's products and maxima.  (Left alone
            // the tiles fall into step and leave the special-function units, which
            // bound the kernel, idle in between: 2.14 instead of 2.01 ms.)  Both take
            // every turn of the block, a tile that has no such step too.
            auto my_turn = [&](int j) {
                const int first = pace + j - (t ? 0 : 1);   // the other tile's step that goes first
                return first < 0 || poll(&sh.turn[t ^ 1], first);
            };
            auto pass_on = [&] {
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.turn[t]);
            };
            // One step; only the edge steps (from s_odd on) hold keys that some row does
            // not see.  The others have a loop of their own without that code.
            auto one_step = [&](int j, auto edge) {
                const int g = step + j;
                const uint32_t t_s = lanes + kPtS + uint32_t((t * 2 + (g & 1)) * kPtKeys);
                if constexpr (decltype(edge)::value) {
                    // look V(j) over: 16-byte words of this thread; the swizzle only
                    // permutes words within a key's 128-byte row
                    const int it = item + 1 + j, r = it % NS;
                    if (!__all_sync(0xffffffffu, poll(&sh.full[r], it / NS))) return false;
                    uint8_t *vt = smem + Sm::oRing + r * Sm::kStage;
                    for (int x = row * 16; x < Sm::kHalf; x += kPtRows * 16) {
                        uint4 *p = reinterpret_cast<uint4 *>(vt + x);
                        if (j * kPtKeys + ((x >> 7) & (kPtKeys - 1)) >= b.len) {
                            *p = make_uint4(0, 0, 0, 0);
                            continue;
                        }
                        uint4 w = *p;
                        if (bf16x2_odd(w.x) || bf16x2_odd(w.y) || bf16x2_odd(w.z) || bf16x2_odd(w.w)) {
                            // the block is marked before the value goes, so whoever no
                            // longer sees the value sees the mark
                            *(volatile int *)&sh.odd[k & 3] = k + 1;
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
                // (one vote at the step's end asks whether the polls succeeded: until then
                // a failed one only means values that go nowhere)
                bool fine = poll(&sh.sfull[t][g & 1], g >> 1);
                __syncwarp();
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
                if constexpr (decltype(edge)::value) {
                    const int k0 = j * kPtKeys;
#pragma unroll
                    for (int i = 0; i < kPtKeys; ++i)
                        if (k0 + i > lim) s[i] = -INFINITY;
                }
                // (a NaN logit is passed over here; its weight is NaN, and so is its row)
                float pm[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int i = 0; i < kPtKeys; i += 2) pm[i / 2 & 3] = fmaxf(pm[i / 2 & 3], fmaxf(s[i], s[i + 1]));
                const float mx = fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3]));
                // the reference stays while no row's maximum has grown by 2^8 (rows that do
                // not exist hold anything and do not count)
                if (__any_sync(0xffffffffu, live && !(mx <= m + lift))) {
                    const bool first = m == -INFINITY;
                    const bool move = mx != -INFINITY && (first || !(mx <= m + lift));
                    float fac = 1.f;
                    if (move) {
                        fac = first ? 0.f : ex2_approx((m - mx) * scale);
                        m = mx;
                        l *= fac;
                    }
                    if (j > 0 && __any_sync(0xffffffffu, move && !first)) {
                        // O is at rest once P(j-1).V(j-1) is complete, as P(j).V(j) waits for
                        // this P; S(j+1) was issued after it and tells of it
                        if (!__all_sync(0xffffffffu, j + 1 < n ? poll(&sh.sfull[t][(g + 1) & 1], (g + 1) >> 1)
                                                               : poll(&sh.odone[t], twos)))
                            return false;
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
                fine = my_turn(j) && fine;
                __syncwarp();
                const uint64_t sc2 = pack2(scale, scale), mc2 = pack2(-mc, -mc);
                float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t w[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const uint64_t x = fma2(pack2(s[c * 32 + 2 * i], s[c * 32 + 2 * i + 1]), sc2, mc2);
                        float p0, p1;
                        unpack2(x, p0, p1);
                        p0 = ex2_approx(p0);
                        p1 = ex2_approx(p1);
                        const __nv_bfloat162 b2 = __floats2bfloat162_rn(p0, p1);
                        w[i] = *reinterpret_cast<const uint32_t *>(&b2);
                        add_bf16x2(sum[2 * (i & 3)], sum[2 * (i & 3) + 1], w[i]);
                    }
                    tmem_st16_nowait(t_s + uint32_t(c * 16), w);
                    if (c == 0) pass_on();   // half way, so that the hand-over costs no pause
                }
                tmem_wait_st();
                tc_fence_before();
                if (!__all_sync(0xffffffffu, fine)) return false;
                if (lane == 0) mbar_arrive(&sh.pfull[t][g & 1]);
                l += ((sum[0] + sum[1]) + (sum[2] + sum[3])) + ((sum[4] + sum[5]) + (sum[6] + sum[7]));
                return true;
            };
            int j = 0;
            for (const int inner = min(n, s_odd); ok && j < inner; ++j) ok = one_step(j, std::false_type());
            for (; ok && j < n; ++j) ok = one_step(j, std::true_type());
            for (; ok && j < b.ns; ++j) {   // steps that only the other tile has
                ok = __all_sync(0xffffffffu, my_turn(j));
                if (ok) pass_on();
            }
            if (ok && n > 0) {
                ok = __all_sync(0xffffffffu, poll(&sh.done[t], used));
                if (!ok) break;
                tc_fence_after();
                const bool odd = *(volatile int *)&sh.odd[k & 3] == k + 1;
                const float il = 1.f / l;   // a live row sees itself; l = 0 only if all logits are -inf
                // 64 elements of each row at a time go through shared memory, so that
                // eight lanes store 128 consecutive bytes of a row
                uint8_t *stage = smem + Sm::oOut + t * Sm::kOut + quad * 32 * 128;
                uint16_t *const tile_out = out + (int64_t(b.begin + b.q0 + t * TPT) * geo.Hq + b.h * geo.g) * D;
                const int stored = b.rows(t) * geo.g;   // rows of the tile that exist
#pragma unroll 1
                for (int c = 0; c < D; c += 64) {
                    float o[64];
                    {
                        uint32_t a0[32], a1[32];
                        tmem_ld32_nowait(t_o + uint32_t(c), a0);
                        tmem_ld32_nowait(t_o + uint32_t(c + 32), a1);
                        tmem_wait_ld();
                        tmem_regs_after_wait(a0);
                        tmem_regs_after_wait(a1);
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            o[i] = __uint_as_float(a0[i]);
                            o[32 + i] = __uint_as_float(a1[i]);
                        }
                    }
                    if (c + 64 == D) {   // O has been read
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sh.oempty[t]);
                    }
                    if (odd && live)
                        for (int key = s_odd * kPtKeys; key <= tok; ++key) {
                            const uint16_t *vr = v + int64_t(b.begin + key) * geo.vs + int64_t(b.h) * D + c;
#pragma unroll
                            for (int i = 0; i < 64; ++i)
                                if ((vr[i] & 0x7f80u) == 0x7f80u)
                                    o[i] += __uint_as_float(uint32_t(vr[i]) << 16);
                        }
#pragma unroll
                    for (int i = 0; i < 64; i += 8) {
                        uint4 w;
                        uint32_t *u = reinterpret_cast<uint32_t *>(&w);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const __nv_bfloat162 b2 =
                                __floats2bfloat162_rn(o[i + 2 * e] * il, o[i + 2 * e + 1] * il);
                            u[e] = *reinterpret_cast<const uint32_t *>(&b2);
                        }
                        *reinterpret_cast<uint4 *>(stage + lane * 128 + (((i / 8) ^ (lane & 7)) << 4)) = w;
                    }
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int rr = i * 4 + (lane >> 3), word = lane & 7, wr = quad * 32 + rr;
                        // wr / g for wr < 128, exactly: the quotient's error is below 1 / g
                        const int tk = (wr * inv_g) >> 16, hd = wr - tk * geo.g;
                        if (wr < stored)
                            *reinterpret_cast<uint4 *>(tile_out + (tk * geo.Hq + hd) * D + c + word * 8) =
                                *reinterpret_cast<const uint4 *>(stage + rr * 128 + ((word ^ (rr & 7)) << 4));
                    }
                    __syncwarp();
                }
            }
            item += b.ns + 1;
            step += n;
            pace += b.ns;
            used += n > 0;
            twos += n > 1;
        }
        if (!ok && lane == 0) fail();
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
    // the driver's encoder, looked up until it is found
    static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> found{nullptr};
    PFN_cuTensorMapEncodeTiled_v12000 enc = found.load(std::memory_order_relaxed);
    if (!enc) {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            enc = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
        found.store(enc, std::memory_order_relaxed);
    }
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
                void *out, int32_t *plan, void *ws, cudaStream_t st)
{
    const int TPT = kPtRows / g.g, TB = 2 * TPT;
    const int64_t blocks = prompt_blocks(g, TB) * g.Hkv;
    if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
    CUtensorMap qm, km, vm;
    if (!packed_map(&qm, q, g.N, g.Hq, D, g.qs, uint32_t(g.g), uint32_t(TPT)) ||
        !packed_map(&km, k, g.N, g.Hkv, D, g.ks, 1, kPtKeys) ||
        !packed_map(&vm, v, g.N, g.Hkv, D, g.vs, 1, kPtKeys))
        return cudaErrorInvalidValue;
    auto kern = prompt_tc_kernel<D>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         int(PtSmem<D>::kBytes));
    if (e == cudaSuccess && plan) e = launch_prompt_plan(g, cu, TB, plan, st);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(unsigned(blocks)), dim3(kPtThreads), PtSmem<D>::kBytes, st, qm, km, vm, g,
                      cu, static_cast<const uint16_t *>(v), static_cast<uint16_t *>(out),
                      float(1.4426950408889634 / sqrt(double(D))), static_cast<const int32_t *>(plan), ws);
}

}  // namespace

cudaError_t launch_prompt_tc(const PagedGeom &g, const void *q, const void *k, const void *v,
                             const int32_t *cu, void *out, int32_t *plan, void *ws, cudaStream_t st)
{
    return g.d == 128 ? run<128>(g, q, k, v, cu, out, plan, ws, st)
                      : run<64>(g, q, k, v, cu, out, plan, ws, st);
}

}  // namespace reatt

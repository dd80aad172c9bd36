// Dealing out the query blocks of packed causal prompts.
#pragma once

#include "paged.cuh"

namespace reatt {

// Blocks of TB tokens at most: every sequence has at most one that is not full.
inline int64_t prompt_blocks(const PagedGeom &g, int TB) { return g.N / TB + (g.B < g.N ? g.B : g.N); }

// A lane of a warp holds this many sequences, and so the warp all of them, up to which a
// block is found without a list of them.
constexpr int kPromptKept = 4, kPromptPlanned = 32 * kPromptKept;

struct PromptBlock {
    int begin, len;   // the sequence's first packed row and its length
    int q0;           // the block's first token within the sequence
    bool live;
};

// Blocks of TB tokens, the ones with the longest key range first: block index
// q of a sequence of n blocks attends about q key blocks, so all blocks q of
// every sequence come before all blocks q - 1.  f(q) = sum_b max(0, n_b - q)
// blocks have an index of at least q; the i-th block has the largest q with
// f(q) > i and belongs to the (i - f(q + 1))-th sequence with more than q
// blocks.  (Offsets that overlap, which no caller may pass, can only make blocks
// go missing.)  At most kPromptPlanned sequences.  One warp calls it; every lane gets the
// answer.
__device__ __forceinline__ PromptBlock prompt_block(const PagedGeom &geo,
                                                    const int32_t *__restrict__ cu, int TB, int i)
{
    const int lane = threadIdx.x & 31;
    auto blocks_of = [&](int b) {
        if (b >= geo.B) return 0;
        int s, e;
        packed_rows(cu, b, geo.N, s, e);
        return (e - s + TB - 1) / TB;
    };
    int kept[kPromptKept], most = 0;
#pragma unroll
    for (int c = 0; c < kPromptKept; ++c) {
        kept[c] = blocks_of(c * 32 + lane);
        most = max(most, kept[c]);
    }
    auto f = [&](int q) {
        int n = 0;
#pragma unroll
        for (int c = 0; c < kPromptKept; ++c) n += max(0, kept[c] - q);
        return __reduce_add_sync(0xffffffffu, n);   // at most N + B blocks, below 2^31
    };
    PromptBlock r{0, 0, 0, false};
    if (f(0) <= i) return r;
    int lo = 0, hi = __reduce_max_sync(0xffffffffu, most);   // f(lo) > i >= f(hi) = 0
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (f(mid) > i) lo = mid;
        else hi = mid;
    }
    int k = i - f(lo + 1);   // k-th sequence with more than lo blocks
    for (int b0 = 0; b0 < geo.B; b0 += 32) {
        const uint32_t mask = __ballot_sync(0xffffffffu, blocks_of(b0 + lane) > lo);
        const int c = __popc(mask);
        if (k >= 0 && k < c) {
            const int b = b0 + int(__fns(mask, 0, k + 1));
            int s, e;
            packed_rows(cu, b, geo.N, s, e);
            r.begin = s;
            r.len = e - s;
            r.q0 = lo * TB;
            r.live = true;
            return r;
        }
        k -= c;
    }
    return r;
}

// With more sequences every block would have to pass over all of them, again and again:
// 384 prompts of 200 tokens with 32/8 heads in bf16 took 947 us that way and 441 with
// the list below, 256 of 20 tokens 94 and 63; of one token 129 took 39 and 31, 65536
// with 8/2 heads 825 ms and 2.8 (fp32: 1.9 s and 23 ms).  So a kernel before lists those
// that have tokens, by falling powers of two of their blocks (the long ones still come
// first) and in order within each, with the number of blocks before them; a block is
// found in the list by bisection.  Layout: [0] sequences listed, [1] blocks in all, then
// start[B + 1] and order[B].
inline size_t prompt_plan_bytes(const PagedGeom &g)
{
    return g.B > kPromptPlanned ? (2 * size_t(g.B) + 3) * sizeof(int32_t) : 0;
}
cudaError_t launch_prompt_plan(const PagedGeom &g, const int32_t *cu, int TB, int32_t *plan, cudaStream_t st);

__device__ __forceinline__ PromptBlock planned_block(const PagedGeom &geo,
                                                     const int32_t *__restrict__ cu,
                                                     const int32_t *plan, int TB, int i)
{
    PromptBlock r{0, 0, 0, false};
    const int n = plan[0];
    const int32_t *start = plan + 2;
    if (n == 0 || i >= plan[1]) return r;
    const int at = max(count_up_to(start, n, i), 1) - 1;
    int s, e;
    packed_rows(cu, start[geo.B + 1 + at], geo.N, s, e);
    const int q = (e - s + TB - 1) / TB - 1 - (i - start[at]);   // its last block first
    r.begin = s;
    r.len = e - s;
    r.q0 = q * TB;
    r.live = q >= 0 && i >= start[at];
    return r;
}

}  // namespace reatt

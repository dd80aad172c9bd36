// Dealing out the query blocks of packed causal prompts.
#pragma once

#include "paged.cuh"

namespace reatt {

// Blocks of TB tokens at most: every sequence has at most one that is not full.
inline int64_t prompt_blocks(const PagedGeom &g, int TB) { return g.N / TB + (g.B < g.N ? g.B : g.N); }

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
// go missing.)  One warp calls it; every lane gets the answer.
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
    // this lane's first sequences stay in registers
    constexpr int KEEP = 4;
    int kept[KEEP], most = 0;
#pragma unroll
    for (int c = 0; c < KEEP; ++c) kept[c] = blocks_of(c * 32 + lane);
    auto f = [&](int q) {
        int n = 0;
#pragma unroll
        for (int c = 0; c < KEEP; ++c) n += max(0, kept[c] - q);
        for (int b = KEEP * 32 + lane; b < geo.B; b += 32) n += max(0, blocks_of(b) - q);
        return __reduce_add_sync(0xffffffffu, n);   // at most N + B blocks, below 2^31
    };
#pragma unroll
    for (int c = 0; c < KEEP; ++c) most = max(most, kept[c]);
    for (int b = KEEP * 32 + lane; b < geo.B; b += 32) most = max(most, blocks_of(b));
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

}  // namespace reatt

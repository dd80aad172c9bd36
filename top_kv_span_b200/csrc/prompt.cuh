// Dealing out the query blocks of packed causal prompts.
#pragma once

#include "paged.cuh"

namespace reatt {

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
// blocks.  One warp calls it; every lane gets the answer.
__device__ __forceinline__ PromptBlock prompt_block(const PagedGeom &geo,
                                                    const int32_t *__restrict__ cu, int TB, int64_t i)
{
    const int lane = threadIdx.x & 31;
    auto blocks_of = [&](int b) {
        int s, e;
        packed_rows(cu, b, geo.N, s, e);
        return (e - s + TB - 1) / TB;
    };
    auto f = [&](int q) {
        int64_t n = 0;
        for (int b = lane; b < geo.B; b += 32) n += max(0, blocks_of(b) - q);
#pragma unroll
        for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
        return n;
    };
    PromptBlock r{0, 0, 0, false};
    if (f(0) <= i) return r;
    int lo = 0, hi = int((geo.N + TB - 1) / TB);   // f(lo) > i >= f(hi)
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (f(mid) > i) lo = mid;
        else hi = mid;
    }
    int k = int(i - f(lo + 1));   // k-th sequence with more than lo blocks
    for (int b0 = 0; b0 < geo.B; b0 += 32) {
        const bool has = b0 + lane < geo.B && blocks_of(b0 + lane) > lo;
        const uint32_t mask = __ballot_sync(0xffffffffu, has);
        const int c = __popc(mask);
        if (k < c) {
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

// Geometry and helpers shared by the paged-cache operators: the append with
// rotation, the attention of one new token over pages and the causal attention
// of packed prompts.
#pragma once

#include "common.cuh"

namespace reatt {

// Derived sizes of one call (host-computed, passed by value to the kernels).
struct PagedGeom {
    int B, Hq, Hkv, g, d, dtype;
    int page_shift;      // log2 of the tokens per page
    int max_pages;       // page-table columns
    int64_t N;           // packed rows
    int64_t n_pages;     // pages in each pool
    int64_t qs, ks, vs;  // elements between the packed rows of q, k, v
    int64_t qrs, krs;    // the same of the rotated copies
    bool rotate;         // rope_base != 0
    float rope_hi[64];   // append: RoPE frequencies in half-turns, hi + lo (see rope_cs)
    float rope_lo[64];

    // tokens that a sequence's row of the page table can hold
    __host__ __device__ __forceinline__ int64_t capacity() const
    {
        return int64_t(max_pages) << page_shift;
    }
};

// Sequence b's packed rows [begin, end) from the row offsets, clamped to the
// packed rows so that malformed offsets never lead out of range.
__device__ __forceinline__ void packed_rows(const int32_t *__restrict__ cu, int b, int64_t N,
                                            int &begin, int &end)
{
    const int n = int(N);
    begin = min(max(cu[b], 0), n);
    end = max(min(cu[b + 1], n), begin);
}

}  // namespace reatt

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

// How many of n ascending numbers are t or less.  A warp halves the range five times at a
// time, until so few are left that loads all at once take no longer than another such
// step (the sequences of 65536 one-token appends: 926 us when every warp counted all of
// the offsets, 110 us now).  Numbers that do not ascend give any count from 0 to n.
__device__ __forceinline__ int count_up_to(const int32_t *x, int n, int64_t t)
{
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = n;   // numbers before lo are, numbers from hi on are not
    while (hi - lo > 256) {
        const int step = (hi - lo + 31) / 32, last = lo + (lane + 1) * step - 1;
        const int c = __popc(__ballot_sync(0xffffffffu, last < hi && x[last] <= t));
        hi = min(hi, lo + (c + 1) * step - 1);
        lo += c * step;
    }
    int c = 0;
    for (int i = lo + lane; i < hi; i += 32) c += x[i] <= t;
    return lo + __reduce_add_sync(0xffffffffu, c);
}

// 16 bytes global -> shared without passing registers; fill = false writes zeros.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool fill)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(fill ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// 2^x on the special-function unit (relative error about 2^-22; 2^-inf = 0).
__device__ __forceinline__ float ex2_approx(float x)
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
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

}  // namespace reatt

// What the decode kernels of the paged cache share: how the keys of a ragged
// batch are dealt out to the CTAs, and the layout of their partial results.
//
// A unit is one sequence's keys under one KV head and one chunk of its query
// heads; a tile is kTile keys of a unit.  All tiles of all units, in order, are
// cut into as many equal ranges as there are CTAs, so a batch of any mix of
// lengths loads every SM alike.  A unit that one range holds whole is finished
// there; a range's first and last unit may be cut, and then leave (m, l, acc):
// m the running maximum of the logits in the log2 domain, l the sum of
// 2^(x - m), acc the sum of 2^(x - m) v.  Slot 2i of the partials is range i's
// cut first unit (begun in an earlier range), slot 2i + 1 its cut last one
// (begun here, continued later).
#pragma once

#include "paged.cuh"

namespace reatt {

// Five warps a CTA with two tiles in flight each, two CTAs an SM, measured best of
// the shapes that fit (bf16, d = 128, 128K keys of 8 KV heads / 61 sequences of up to
// 8K / 256 of 1.5K keys of 2 KV heads): 89 / 96 / 76 us now, 94 / 96 / 76 when the others
// were measured: 4 warps x 3 tiles x 2 CTAs 114 / 119 / 92, 3 x 2 x 3 110 / 109 / 84,
// 6 x 2 x 1 92 / 108 / 86, 10 x 2 x 1 96 / 104 / 83, 8 x 2 x 1 112 / 131 / 100.
constexpr int kPdWarps = 5;             // warps of a CTA; each takes its own keys of a tile
constexpr int kPdThreads = kPdWarps * 32;
constexpr int kPdStages = 2;            // tiles in flight per warp
constexpr int kPdHalf = 4096;           // bytes of a warp's K (or V) rows of one tile
constexpr int kPdStage = 2 * kPdHalf;

// What range i left for the join (written by the main kernel, read by the join).
struct PdMeta {
    int32_t open_b, open_u;   // unit cut at the range's end that begins in it; open_b < 0: none
    int32_t first;            // slot 2i: 0 unused, 1 ends its unit, 2 the unit goes on
    int32_t pad;
};

struct PdArgs {
    const void *q, *k_pages, *v_pages;
    const int32_t *table, *lens;
    void *out;
    float *part_acc;   // [2 * ranges][HB][D]
    float2 *part_ml;   // [2 * ranges][HB]
    PdMeta *meta;      // [ranges]
    void *ws;
    int chunks;        // chunks of query heads per KV head
    float scale;       // log2(e) / sqrt(d)
};

__device__ __forceinline__ int pd_len(const PagedGeom &geo, const int32_t *lens, int b)
{
    const int64_t n = lens[b], cap = geo.capacity();
    return int(n < 0 ? 0 : (n > cap ? cap : n));
}

// For each thread its share of the sequences, `per` of them, and the first one there that
// has a key, or B (pd_range fills it).
__device__ __forceinline__ int (&pd_first_live())[kPdThreads]
{
    __shared__ int first[kPdThreads];
    return first;
}
__device__ __forceinline__ int pd_share(const PagedGeom &geo) { return (geo.B + kPdThreads - 1) / kPdThreads; }

// Position in the list of tiles.  A whole warp walks it together.
struct PdWalk {
    int b, u, tile, nt, len;
    // To sequence nb or the first one after it that has a key.  A run of empty ones (a batch
    // of fixed size that is mostly idle) is passed over 32 lengths at a time to the end of
    // its share, then by shares (one by one 65534 of them held a call up for 12 ms, now 0.03).
    template <int TILE>
    __device__ __forceinline__ void enter(const PagedGeom &geo, const int32_t *lens, int nb)
    {
        b = nb;
        len = b < geo.B ? pd_len(geo, lens, b) : 0;
        if (len == 0 && b < geo.B) {
            b = next_live(geo, lens, b);
            len = b < geo.B ? pd_len(geo, lens, b) : 0;
        }
        nt = (len + TILE - 1) / TILE;
    }
    // The first sequence behind `at` that has a key, or B.
    __device__ __forceinline__ static int next_live(const PagedGeom &geo, const int32_t *lens, int at)
    {
        const int lane = threadIdx.x & 31, per = pd_share(geo), share = at / per;
        const int end = min((share + 1) * per, geo.B);
        int found = geo.B;
        for (int s = at + 1; s < end && found == geo.B; s += 32) {
            const bool live = s + lane < end && pd_len(geo, lens, s + lane) > 0;
            const uint32_t some = __ballot_sync(0xffffffffu, live);
            if (some) found = s + __ffs(some) - 1;
        }
        for (int s = share + 1; s < kPdThreads && found == geo.B; s += 32) {
            const int first = s + lane < kPdThreads ? pd_first_live()[s + lane] : geo.B;
            found = __reduce_min_sync(0xffffffffu, first);   // the shares ascend
        }
        return found;
    }
    template <int TILE>
    __device__ __forceinline__ void next(const PagedGeom &geo, const int32_t *lens, int units)
    {
        if (++tile < nt) return;
        tile = 0;
        if (++u < units) return;
        u = 0;
        enter<TILE>(geo, lens, b + 1);
    }
};

// This CTA's range of tiles: where it starts and how many tiles it holds.
// Every thread of the CTA calls it.
template <int TILE>
__device__ __forceinline__ int64_t pd_range(const PagedGeom &geo, const int32_t *lens, int units,
                                            PdWalk &w)
{
    __shared__ int64_t warp_sum[kPdWarps];
    __shared__ int start[3];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = pd_share(geo);
    const int b0 = min(tid * per, geo.B), b1 = min(b0 + per, geo.B);
    int64_t sum = 0;
    int first = geo.B;
    for (int b = b0; b < b1; ++b) {
        const int len = pd_len(geo, lens, b);
        sum += int64_t((len + TILE - 1) / TILE) * units;
        if (len > 0) first = min(first, b);
    }
    pd_first_live()[tid] = first;
    int64_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
    }
    if (lane == 31) warp_sum[warp] = incl;
    if (tid == 0) start[0] = geo.B;
    __syncthreads();
    int64_t base = 0, total = 0;
#pragma unroll
    for (int x = 0; x < kPdWarps; ++x) {
        if (x < warp) base += warp_sum[x];
        total += warp_sum[x];
    }
    // with fewer tiles than CTAs the first `total` CTAs take one each
    const int64_t ranges = min(total, int64_t(gridDim.x)), i = blockIdx.x;
    const int64_t t0 = i < ranges ? total * i / ranges : total;
    const int64_t t1 = i < ranges ? total * (i + 1) / ranges : total;
    int64_t at = base + incl - sum;
    if (t0 < t1 && t0 >= at && t0 < at + sum)
        for (int b = b0; b < b1; ++b) {
            const int nt = (pd_len(geo, lens, b) + TILE - 1) / TILE;
            const int64_t n = int64_t(nt) * units;
            if (t0 < at + n) {
                start[0] = b;
                start[1] = int((t0 - at) / nt);
                start[2] = int((t0 - at) % nt);
                break;
            }
            at += n;
        }
    __syncthreads();
    w.b = start[0];
    w.u = w.tile = w.nt = w.len = 0;
    if (w.b < geo.B) {
        w.u = start[1];
        w.tile = start[2];
        w.len = pd_len(geo, lens, w.b);
        w.nt = (w.len + TILE - 1) / TILE;
    }
    return t1 - t0;
}

// Weight of a partial with maximum m under the joint maximum M.
__device__ __forceinline__ float pd_weight(float m, float M)
{
    return m == -INFINITY ? 0.f : ex2_approx(m - M);
}

}  // namespace reatt

// Attention of one new token per sequence over a paged key-value cache.
//
//   x_t = q.k_t / sqrt(d),  o = sum_t softmax_t(x) v_t,  t < seq_len[b]
//
// One pass over the keys with the running maximum and sum of the softmax; see
// paged_decode.cuh for how the keys are dealt out and joined again.  Every K
// and V byte is read once for all query heads of its KV head, so memory bounds
// it.  Each warp streams its own keys of a tile through its own ring with
// 16-byte asynchronous copies and never waits for the other warps until a unit
// ends; rows past the sequence, or on a page that the table does not name, are
// filled with zeros in shared memory, so nothing there can reach a sum.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>

#include "kernels.h"
#include "paged_decode.cuh"

namespace reatt {
namespace {

template <typename T> __device__ __forceinline__ void store_elem(T *p, float v);
template <> __device__ __forceinline__ void store_elem<float>(float *p, float v) { *p = v; }
template <> __device__ __forceinline__ void store_elem<uint16_t>(uint16_t *p, float v)
{
    *reinterpret_cast<__nv_bfloat16 *>(p) = __float2bfloat16_rn(v);
}

// E consecutive elements of a row, widened.
template <int E> __device__ __forceinline__ void load_slice(const float *p, float (&v)[E])
{
#pragma unroll
    for (int e = 0; e < E; e += 2) {
        const float2 t = *reinterpret_cast<const float2 *>(p + e);
        v[e] = t.x;
        v[e + 1] = t.y;
    }
}
template <> __device__ __forceinline__ void load_slice<4>(const float *p, float (&v)[4])
{
    const float4 t = *reinterpret_cast<const float4 *>(p);
    v[0] = t.x; v[1] = t.y; v[2] = t.z; v[3] = t.w;
}
template <int E> __device__ __forceinline__ void load_slice(const uint16_t *p, float (&v)[E])
{
#pragma unroll
    for (int e = 0; e < E; e += 2) {
        const uint32_t t = *reinterpret_cast<const uint32_t *>(p + e);
        v[e] = bf16lo(t);
        v[e + 1] = bf16hi(t);
    }
}

// Elements [offset, ...) of the page row of key `key`, or < 0.
__device__ __forceinline__ int64_t key_row(const PagedGeom &geo, int id, int h, int key, int D)
{
    if (id < 0 || id >= geo.n_pages) return -1;
    return ((((int64_t(id) * geo.Hkv + h) << geo.page_shift) +
             (key & ((1 << geo.page_shift) - 1)))) * D;
}

// HB query heads of one KV head per unit.  A lane owns D/32 elements of every
// row; the dot products of a tile's keys and heads are summed over the lanes by
// a transposed butterfly (31 shuffles for 32 sums), which leaves one (key, head)
// pair per lane for the exponentials.
template <typename T, int D, int HB>
__global__ void __launch_bounds__(kPdThreads)
paged_decode_kernel(PagedGeom geo, PdArgs a)
{
    constexpr int RB = D * int(sizeof(T));   // bytes of a row
    constexpr int KT = kPdHalf / RB;         // keys of a warp's part of a tile
    constexpr int TILE = KT * kPdWarps;
    constexpr int E = D / 32;                // elements of a row per lane
    constexpr int LPR = RB / 16;             // 16-byte words of a row
    constexpr int NB = KT * HB / 32;         // butterflies per tile part
    static_assert(NB * 32 == KT * HB && KT <= 32, "tile shape");
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float red_ml[kPdWarps][HB][2];
    float *red_o = reinterpret_cast<float *>(smem + kPdWarps * kPdStages * kPdStage);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int units = geo.Hkv * a.chunks;
    pdl_trigger();   // the join may be scheduled; it waits for this grid's end
    pdl_wait();

    // sequences without a key: zeros
    for (int b = blockIdx.x; b < geo.B; b += gridDim.x) {
        const int len = pd_len(geo, a.lens, b);
        if (len == 0)
            for (int i = tid; i < geo.Hq * D; i += kPdThreads)
                store_elem(static_cast<T *>(a.out) + int64_t(b) * geo.Hq * D + i, 0.f);
        if (tid == 0 && len != a.lens[b]) report_status(a.ws, REATT_EPAGE);
    }

    PdWalk cw;
    const int64_t n = pd_range<TILE>(geo, a.lens, units, cw);
    if (tid == 0) a.meta[blockIdx.x] = PdMeta{-1, 0, 0, 0};
    if (n == 0) return;
    PdWalk lw = cw;
    uint8_t *ring = smem + warp * kPdStages * kPdStage;
    const uint32_t ring_addr = smem_addr(ring);

    auto table_of = [&](const PdWalk &w) {
        const int key = w.tile * TILE + warp * KT + lane;
        return lane < KT && key < w.len
                   ? a.table[int64_t(w.b) * geo.max_pages + (key >> geo.page_shift)]
                   : 0;
    };
    int id = table_of(lw);   // this lane's page of the tile to load next
    int64_t loaded = 0;
    auto load = [&]() {
        if (loaded < n) {
            const int key0 = lw.tile * TILE + warp * KT, h = lw.u / a.chunks;
            int64_t off = -1;
            if (lane < KT && key0 + lane < lw.len) {
                off = key_row(geo, id, h, key0 + lane, D);
                if (off < 0) report_status(a.ws, REATT_EPAGE);
            }
            const uint32_t st = ring_addr + uint32_t(loaded % kPdStages) * kPdStage;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = i * (32 / LPR) + lane / LPR;
                const int64_t o = __shfl_sync(0xffffffffu, off, r);
                const uint32_t dst = st + uint32_t(i * 512 + lane * 16);
                const int64_t src = (o < 0 ? 0 : o) * int64_t(sizeof(T)) + (lane % LPR) * 16;
                cp_async16(dst, static_cast<const uint8_t *>(a.k_pages) + src, o >= 0);
                cp_async16(dst + kPdHalf, static_cast<const uint8_t *>(a.v_pages) + src, o >= 0);
            }
            if (++loaded < n) {
                lw.next<TILE>(geo, a.lens, units);
                id = table_of(lw);
            }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int s = 0; s < kPdStages - 1; ++s) load();

    float qv[HB][E], o[HB][E], m = -INFINITY, l = 0.f;   // m, l: of head lane % HB
    bool fresh = true;
    const int64_t seg0 = cw.tile;   // first tile of the current segment
    int64_t seg_begin = seg0;
    for (int64_t i = 0; i < n; ++i) {
        const int h = cw.u / a.chunks, j0 = (cw.u % a.chunks) * HB;   // first query head of the unit
        const int nh = min(HB, geo.g - j0);
        if (fresh) {
#pragma unroll
            for (int j = 0; j < HB; ++j) {
#pragma unroll
                for (int e = 0; e < E; ++e) qv[j][e] = o[j][e] = 0.f;
                if (j < nh)
                    load_slice<E>(static_cast<const T *>(a.q) + int64_t(cw.b) * geo.qs +
                                      int64_t(h * geo.g + j0 + j) * D + lane * E,
                                  qv[j]);
            }
            m = -INFINITY;
            l = 0.f;
            fresh = false;
        }
        load();
        cp_async_wait<kPdStages - 1>();
        __syncwarp();
        const T *kt = reinterpret_cast<const T *>(ring + (i % kPdStages) * kPdStage);
        const T *vt = reinterpret_cast<const T *>(ring + (i % kPdStages) * kPdStage + kPdHalf);
        const int key0 = cw.tile * TILE + warp * KT;
        float x[NB];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            constexpr int KPB = 32 / HB;   // keys of one butterfly
            float v[32];
#pragma unroll
            for (int kk = 0; kk < KPB; ++kk) {
                float kv[E];
                load_slice<E>(kt + (nb * KPB + kk) * D + lane * E, kv);
#pragma unroll
                for (int j = 0; j < HB; ++j) {
                    float s = qv[j][0] * kv[0];
#pragma unroll
                    for (int e = 1; e < E; ++e) s = fmaf(qv[j][e], kv[e], s);
                    v[kk * HB + j] = s;
                }
            }
#pragma unroll
            for (int w = 16; w >= 1; w >>= 1)
#pragma unroll
                for (int c = 0; c < w; ++c) {
                    const bool up = lane & w;
                    const float send = up ? v[c] : v[c + w], keep = up ? v[c + w] : v[c];
                    v[c] = keep + __shfl_xor_sync(0xffffffffu, send, w);
                }
            x[nb] = key0 + nb * KPB + lane / HB < cw.len ? v[0] * a.scale : -INFINITY;
        }
        float mx = x[0];
#pragma unroll
        for (int nb = 1; nb < NB; ++nb) mx = fmaxf(mx, x[nb]);
#pragma unroll
        for (int w = HB; w < 32; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
        const float mn = fmaxf(m, mx), fac = pd_weight(m, mn);
        m = mn;
        float p[NB], ps = 0.f;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
            // a masked key is -inf; a row of logits that are all -inf keeps l = 0
            p[nb] = x[nb] == -INFINITY ? 0.f : pd_ex2(x[nb] - m);
            ps += p[nb];
        }
        l = l * fac + ps;
#pragma unroll
        for (int j = 0; j < HB; ++j) {
            const float f = __shfl_sync(0xffffffffu, fac, j);
#pragma unroll
            for (int e = 0; e < E; ++e) o[j][e] *= f;
        }
#pragma unroll
        for (int kk = 0; kk < KT; ++kk) {
            float vv[E];
            load_slice<E>(vt + kk * D + lane * E, vv);
#pragma unroll
            for (int j = 0; j < HB; ++j) {
                const float pj = __shfl_sync(0xffffffffu, p[kk * HB / 32], (kk * HB) % 32 + j);
#pragma unroll
                for (int e = 0; e < E; ++e) o[j][e] = fmaf(pj, vv[e], o[j][e]);
            }
        }
        __syncwarp();   // the stage may be refilled
        const bool unit_end = cw.tile + 1 == cw.nt;
        if (unit_end || i + 1 == n) {
            // join the warps, then finish the unit or leave it for the join kernel
#pragma unroll
            for (int w = HB; w < 32; w <<= 1) l += __shfl_xor_sync(0xffffffffu, l, w);
            if (lane < HB) {
                red_ml[warp][lane][0] = m;
                red_ml[warp][lane][1] = l;
            }
#pragma unroll
            for (int j = 0; j < HB; ++j)
#pragma unroll
                for (int e = 0; e < E; ++e) red_o[(warp * HB + j) * D + lane * E + e] = o[j][e];
            __syncthreads();
            const bool begins = seg_begin == 0, whole = begins && unit_end;
            const int slot = 2 * blockIdx.x + (begins ? 1 : 0);
            for (int y = tid; y < HB * D; y += kPdThreads) {
                const int j = y / D, c = y - j * D;
                float M = red_ml[0][j][0];
#pragma unroll
                for (int w = 1; w < kPdWarps; ++w) M = fmaxf(M, red_ml[w][j][0]);
                float L = 0.f, acc = 0.f;
#pragma unroll
                for (int w = 0; w < kPdWarps; ++w) {
                    const float f = pd_weight(red_ml[w][j][0], M);
                    L += f * red_ml[w][j][1];
                    acc += f * red_o[(w * HB + j) * D + c];
                }
                if (whole) {
                    if (j < nh)
                        store_elem(static_cast<T *>(a.out) +
                                       (int64_t(cw.b) * geo.Hq + h * geo.g + j0 + j) * D + c,
                                   acc / L);
                } else {
                    a.part_acc[(int64_t(slot) * HB + j) * D + c] = acc;
                    if (c == 0) a.part_ml[slot * HB + j] = make_float2(M, L);
                }
            }
            if (tid == 0 && !whole) {
                if (begins) {
                    a.meta[blockIdx.x].open_b = cw.b;
                    a.meta[blockIdx.x].open_u = cw.u;
                } else {
                    a.meta[blockIdx.x].first = unit_end ? 1 : 2;
                }
            }
            __syncthreads();
            fresh = true;
            seg_begin = 0;
        }
        if (i + 1 < n) cw.next<TILE>(geo, a.lens, units);
    }
    cp_async_wait<0>();
}

// The join: block i finishes the unit that begins in range i and goes on in the
// following ranges, from its partials in order.
template <typename T, int D, int HB>
__global__ void __launch_bounds__(256)
paged_decode_join_kernel(PagedGeom geo, PdArgs a)
{
    __shared__ int last_s;
    pdl_wait();
    const PdMeta me = a.meta[blockIdx.x];
    if (me.open_b < 0) return;
    // the range that ends the unit: the first one after this whose slot says so
    const int tid = threadIdx.x, n = gridDim.x;
    if (tid == 0) last_s = n - 1;
    __syncthreads();
    for (int i = blockIdx.x + 1 + tid; i < n; i += 256)
        if (a.meta[i].first == 1) atomicMin(&last_s, i);
    __syncthreads();
    const int last = last_s;
    const int h = me.open_u / a.chunks, j0 = (me.open_u % a.chunks) * HB;
    const int nh = min(HB, geo.g - j0);
    for (int y = tid; y < nh * D; y += 256) {
        const int j = y / D, c = y - j * D;
        const int first = 2 * blockIdx.x + 1;
        float M = a.part_ml[first * HB + j].x;
        for (int i = blockIdx.x + 1; i <= last; ++i) M = fmaxf(M, a.part_ml[2 * i * HB + j].x);
        float2 ml = a.part_ml[first * HB + j];
        float f = pd_weight(ml.x, M);
        float L = f * ml.y, acc = f * a.part_acc[(int64_t(first) * HB + j) * D + c];
        for (int i = blockIdx.x + 1; i <= last; ++i) {
            ml = a.part_ml[2 * i * HB + j];
            f = pd_weight(ml.x, M);
            L += f * ml.y;
            acc += f * a.part_acc[(int64_t(2 * i) * HB + j) * D + c];
        }
        store_elem(static_cast<T *>(a.out) + (int64_t(me.open_b) * geo.Hq + h * geo.g + j0 + j) * D + c,
                   acc / L);
    }
}

constexpr int kMaxHeads = 16;   // query heads of a unit, at most

template <typename T, int D, int HB>
cudaError_t run(const PagedGeom &g, PdArgs a, int ranges, cudaStream_t st)
{
    a.chunks = (g.g + HB - 1) / HB;
    auto kern = paged_decode_kernel<T, D, HB>;
    const size_t smem = size_t(kPdWarps) * kPdStages * kPdStage + size_t(kPdWarps) * HB * D * 4;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e != cudaSuccess) return e;
    e = launch_pdl(kern, dim3(unsigned(ranges)), dim3(kPdThreads), smem, st, g, a);
    if (e != cudaSuccess) return e;
    return launch_pdl(paged_decode_join_kernel<T, D, HB>, dim3(unsigned(ranges)), dim3(256), 0, st, g, a);
}

int ranges_of() { return 2 * num_sms(); }   // two CTAs fit an SM

}  // namespace

size_t paged_decode_ws_bytes(const PagedGeom &g)
{
    const size_t n = size_t(ranges_of());
    return n * sizeof(PdMeta) + 2 * n * kMaxHeads * (sizeof(float2) + size_t(g.d) * sizeof(float));
}

cudaError_t launch_paged_decode(const PagedGeom &g, const void *q, const void *k_pages,
                                const void *v_pages, const int32_t *table, const int32_t *lens,
                                void *out, void *scratch, void *ws, cudaStream_t st)
{
    const int n = ranges_of();
    uint8_t *p = static_cast<uint8_t *>(scratch);
    PdArgs a{q, k_pages, v_pages, table, lens, out, nullptr, nullptr, nullptr, ws, 1,
             float(1.4426950408889634 / sqrt(double(g.d)))};
    a.part_acc = reinterpret_cast<float *>(p);
    a.part_ml = reinterpret_cast<float2 *>(p + size_t(2 * n) * kMaxHeads * g.d * sizeof(float));
    a.meta = reinterpret_cast<PdMeta *>(a.part_ml + size_t(2 * n) * kMaxHeads);
    if (g.dtype == REATT_BF16) {
        if (g.d == 128) return g.g <= 4 ? run<uint16_t, 128, 4>(g, a, n, st) : run<uint16_t, 128, 8>(g, a, n, st);
        return g.g <= 4 ? run<uint16_t, 64, 4>(g, a, n, st) : run<uint16_t, 64, 8>(g, a, n, st);
    }
    if (g.d == 128) return g.g <= 4 ? run<float, 128, 4>(g, a, n, st) : run<float, 128, 8>(g, a, n, st);
    return g.g <= 4 ? run<float, 64, 4>(g, a, n, st) : run<float, 64, 8>(g, a, n, st);
}

}  // namespace reatt

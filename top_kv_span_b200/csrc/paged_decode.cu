// Attention of one new token per sequence over a paged key-value cache.
//
//   x_t = q.k_t / sqrt(d),  o = sum_t softmax_t(x) v_t,  t < seq_len[b]
//
// One pass over the keys with the running maximum and sum of the softmax; see
// paged_decode.cuh for how the keys are dealt out and joined again.  Every K
// and V byte is read once for up to 16 query heads of its KV head (fp32: 8), so memory
// bounds it; a larger group is cut into chunks that each read all keys again.  Each
// warp streams its own keys of a tile through its own ring with
// 16-byte asynchronous copies and never waits for the other warps until a unit
// ends; rows past the sequence, or on a page that the table does not name, are
// filled with zeros in shared memory, so nothing there can reach a sum.
// One sequence of 131073 tokens, 32/8 heads of width 128 in bf16, takes 89 us, 6.0 TB/s
// (93% of the copy bandwidth, the join and both launches included); 61 sequences of up
// to 8K 96 us (92%); 256 of 1.5K tokens with 12/2 heads 76 us (84%).  By heads of a group,
// 269 MB of keys and values of width 128: 1 to 8 heads 50 to 53 us, 9 to 16 70 us (room for
// one CTA an SM), 32 121 us, 128 440 us; fp32 1 to 4 heads 54 us, 5 to 8 70 us, 16 123 us,
// 128 907 us.  Where units hold few keys their ends bound it: 256 sequences of 31 tokens,
// 32/8 heads, 22 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>

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

__device__ __forceinline__ void store4(float *p, const float4 &v) { *reinterpret_cast<float4 *>(p) = v; }
__device__ __forceinline__ void store4(uint16_t *p, const float4 &v)
{
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<const uint32_t *>(&a),
                                               *reinterpret_cast<const uint32_t *>(&b));
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
// Elements [offset, ...) of the page row of key `key`, or < 0.
__device__ __forceinline__ int64_t key_row(const PagedGeom &geo, int id, int h, int key, int D)
{
    if (id < 0 || id >= geo.n_pages) return -1;
    return ((((int64_t(id) * geo.Hkv + h) << geo.page_shift) +
             (key & ((1 << geo.page_shift) - 1)))) * D;
}

// One warp's stream of its K and V rows of the tiles, `n` tiles from `at` on, through
// its ring in shared memory.  The page of the next tile's rows is looked up one
// tile ahead, so that its latency is not waited for.
template <typename T, int D, bool SWIZZLE> struct PdStream {
    static constexpr int RB = D * int(sizeof(T));   // bytes of a row
    static constexpr int KT = kPdHalf / RB;         // keys of a warp's part of a tile
    static constexpr int TILE = KT * kPdWarps;
    static constexpr int LPR = RB / 16;             // 16-byte words of a row
    static_assert(KT <= 32, "a lane looks up one key");

    const PagedGeom &geo;
    const PdArgs &a;
    PdWalk at;
    int64_t left;              // tiles not issued yet
    int units, slot = 0, key_of_lane, id;
    uint32_t ring, dst[4];     // this lane's place in a stage, for four rows of words in turn
    bool one_page;             // the rows of a tile part lie in one page

    __device__ __forceinline__ PdStream(const PagedGeom &g, const PdArgs &args, const PdWalk &w,
                                        int64_t tiles, int u, uint32_t ring_addr)
        : geo(g), a(args), at(w), left(tiles), units(u), ring(ring_addr)
    {
        const int lane = threadIdx.x & 31;
        key_of_lane = int(threadIdx.x >> 5) * KT + lane;
        one_page = (1 << g.page_shift) >= KT;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = i * (32 / LPR) + lane / LPR, c = lane % LPR;
            dst[i] = uint32_t(r * RB + (SWIZZLE ? c ^ (r & 7) : c) * 16);
        }
        look_up();
    }
    __device__ __forceinline__ bool mine(int key) const
    {
        return int(threadIdx.x & 31) < KT && key < at.len;
    }
    __device__ __forceinline__ void look_up()
    {
        const int key = at.tile * TILE + key_of_lane;
        id = mine(key) ? a.table[int64_t(at.b) * geo.max_pages + (key >> geo.page_shift)] : 0;
    }
    // Issue the next tile's copies (none past the end); one group either way.
    __device__ __forceinline__ void load()
    {
        const int lane = threadIdx.x & 31, key = at.tile * TILE + key_of_lane;
        if (left > 0) {
            const uint32_t st = ring + uint32_t(slot) * kPdStage;
            const uint8_t *kp = static_cast<const uint8_t *>(a.k_pages);
            const uint8_t *vp = static_cast<const uint8_t *>(a.v_pages);
            if (key - lane >= at.len) {
                // no key of this warp's: the part is passed over
            } else if (one_page && key - lane + KT <= at.len && uint32_t(__shfl_sync(0xffffffffu, id, 0)) < geo.n_pages) {
                // all rows there and contiguous: every lane's words lie 512 bytes apart
                const int64_t first = key_row(geo, __shfl_sync(0xffffffffu, id, 0), at.u / a.chunks,
                                              key - lane, D) * int64_t(sizeof(T)) + lane * 16;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    // rows four instructions apart differ by a multiple of eight, or the
                    // words are not swizzled by rows that far apart
                    const uint32_t d = st + dst[i & 3] + uint32_t((i >> 2) * 2048);
                    cp_async16(d, kp + first + i * 512, true);
                    cp_async16(d + kPdHalf, vp + first + i * 512, true);
                }
            } else {
                int64_t off = -1;
                if (mine(key)) {
                    off = key_row(geo, id, at.u / a.chunks, key, D);
                    if (off < 0) report_status(a.ws, REATT_EPAGE);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int r = i * (32 / LPR) + lane / LPR;
                    const int64_t o = __shfl_sync(0xffffffffu, off, r);
                    const uint32_t d = st + dst[i & 3] + uint32_t((i >> 2) * 2048);
                    const int64_t src = (o < 0 ? 0 : o) * int64_t(sizeof(T)) + (lane % LPR) * 16;
                    cp_async16(d, kp + src, o >= 0);
                    cp_async16(d + kPdHalf, vp + src, o >= 0);
                }
            }
            slot = slot + 1 == kPdStages ? 0 : slot + 1;
            if (--left > 0) {
                at.next<TILE>(geo, a.lens, units);
                look_up();
            }
        }
        cp_async_commit();
    }
};

// What a range does besides its tiles: zeros for sequences without a key, and the
// status of lengths out of range.
template <typename T, int D>
__device__ __forceinline__ void pd_empty(const PagedGeom &geo, const PdArgs &a)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;   // a warp per sequence
    for (int b = blockIdx.x * kPdWarps + warp; b < geo.B; b += gridDim.x * kPdWarps) {
        const int len = pd_len(geo, a.lens, b);
        if (len == 0)
            for (int i = lane; i < geo.Hq * D; i += 32)
                store_elem(static_cast<T *>(a.out) + int64_t(b) * geo.Hq * D + i, 0.f);
        if (lane == 0 && len != a.lens[b]) report_status(a.ws, REATT_EPAGE);
    }
}

// Rows of the warps' o are padded by four floats: the lanes of a product's columns then
// write to different banks.
constexpr int kPdPad = 4;

// Joins the warps' (m, l, o) of a unit's part, which they have left in red_ml (l < 0:
// none, not even a key without weight, whose V may hold an infinity or NaN) and red_o,
// and finishes the unit or leaves the part for the join kernel.  Every thread of the CTA
// calls it after a barrier, and passes another one before it writes there again.
template <typename T, int D, int HB>
__device__ __forceinline__ void pd_finish(const PagedGeom &geo, const PdArgs &a, const PdWalk &w,
                                          bool begins, bool ends, const float2 (*red_ml)[HB],
                                          const float *red_o)
{
    const int h = w.u / a.chunks, j0 = (w.u % a.chunks) * HB, nh = min(HB, geo.g - j0);
    const bool whole = begins && ends;
    const int slot = 2 * blockIdx.x + (begins ? 1 : 0);
    for (int y = threadIdx.x; y < nh * (D / 4); y += kPdThreads) {
        const int j = y / (D / 4), c = (y - j * (D / 4)) * 4;
        float M = red_ml[0][j].x;
#pragma unroll
        for (int i = 1; i < kPdWarps; ++i) M = fmaxf(M, red_ml[i][j].x);
        float L = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kPdWarps; ++i) {
            const float2 ml = red_ml[i][j];
            if (ml.y < 0.f) continue;   // no key: its o was not left
            const float f = pd_weight(ml.x, M);
            const float4 t = *reinterpret_cast<const float4 *>(red_o + (i * HB + j) * (D + kPdPad) + c);
            L = fmaf(f, ml.y, L);
            acc.x = fmaf(f, t.x, acc.x);
            acc.y = fmaf(f, t.y, acc.y);
            acc.z = fmaf(f, t.z, acc.z);
            acc.w = fmaf(f, t.w, acc.w);
        }
        if (whole) {
            store4(static_cast<T *>(a.out) + (int64_t(w.b) * geo.Hq + h * geo.g + j0 + j) * D + c,
                   make_float4(acc.x / L, acc.y / L, acc.z / L, acc.w / L));
        } else {
            store4(a.part_acc + (int64_t(slot) * HB + j) * D + c, acc);
            if (c == 0) a.part_ml[slot * HB + j] = make_float2(M, L);
        }
    }
    if (threadIdx.x == 0 && !whole) {
        if (begins) {
            a.meta[blockIdx.x].open_b = w.b;
            a.meta[blockIdx.x].open_u = w.u;
        } else {
            a.meta[blockIdx.x].first = ends ? 1 : 2;
        }
    }
}

// fp32: HB query heads of one KV head per unit.  A lane owns D/32 elements of every
// row; the dot products of a tile's keys and heads are summed over the lanes by
// a transposed butterfly (31 shuffles for 32 sums), which leaves one (key, head)
// pair per lane for the exponentials.
template <int D, int HB>
__global__ void __launch_bounds__(kPdThreads)
paged_decode_f32_kernel(PagedGeom geo, PdArgs a)
{
    using Stream = PdStream<float, D, false>;
    constexpr int KT = Stream::KT, TILE = Stream::TILE;
    constexpr int E = D / 32;                // elements of a row per lane
    constexpr int NB = KT * HB / 32;         // butterflies per tile part
    static_assert(NB * 32 == KT * HB, "tile shape");
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float2 red_ml[kPdWarps][HB];
    float *red_o = reinterpret_cast<float *>(smem + kPdWarps * kPdStages * kPdStage);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int units = geo.Hkv * a.chunks;
    pdl_trigger();   // the join may be scheduled; it waits for this grid's end
    pdl_wait();
    PdWalk cw;
    const int64_t n = pd_range<TILE>(geo, a.lens, units, cw);
    if (tid == 0) a.meta[blockIdx.x] = PdMeta{-1, 0, 0, 0};
    if (n == 0) {
        pd_empty<float, D>(geo, a);
        return;
    }
    const uint8_t *ring = smem + warp * kPdStages * kPdStage;
    Stream stream(geo, a, cw, n, units, smem_addr(ring));
#pragma unroll
    for (int s = 0; s < kPdStages - 1; ++s) stream.load();
    pd_empty<float, D>(geo, a);   // behind the first loads

    float qv[HB][E], o[HB][E], m, l;   // m, l: of head lane % HB
    auto load_q = [&](const PdWalk &w) {
        const int h = w.u / a.chunks, j0 = (w.u % a.chunks) * HB, nh = min(HB, geo.g - j0);
#pragma unroll
        for (int j = 0; j < HB; ++j) {
#pragma unroll
            for (int e = 0; e < E; ++e) qv[j][e] = 0.f;
            if (j < nh)
                load_slice<E>(static_cast<const float *>(a.q) + int64_t(w.b) * geo.qs +
                                  int64_t(h * geo.g + j0 + j) * D + lane * E,
                              qv[j]);
        }
    };
    auto reset = [&] {
#pragma unroll
        for (int j = 0; j < HB; ++j)
#pragma unroll
            for (int e = 0; e < E; ++e) o[j][e] = 0.f;
        m = -INFINITY;
        l = 0.f;
    };
    load_q(cw);
    reset();
    bool begins = cw.tile == 0;   // this part of the unit starts at its first key
    bool any = false;             // some key of the part was this warp's
    int slot = 0;
    for (int64_t i = 0; i < n; ++i) {
        stream.load();
        cp_async_wait<kPdStages - 1>();
        __syncwarp();
        const float *kt = reinterpret_cast<const float *>(ring + slot * kPdStage);
        const float *vt = kt + kPdHalf / 4;
        const int key0 = cw.tile * TILE + warp * KT;
        const bool has = key0 < cw.len;   // some key of the tile is this warp's
        any |= has;
        float x[NB];
#pragma unroll
        for (int nb = 0; has && nb < NB; ++nb) {
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
        // the last product with this unit's q: the next one's is on its way meanwhile
        const bool unit_end = cw.tile + 1 == cw.nt, part_end = unit_end || i + 1 == n;
        PdWalk nw = cw;
        if (i + 1 < n) {
            nw.next<TILE>(geo, a.lens, units);
            if (part_end) load_q(nw);
        }
        if (has) {
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
                p[nb] = x[nb] == -INFINITY ? 0.f : ex2_approx(x[nb] - m);
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
        }
        __syncwarp();   // the stage may be refilled
        slot = slot + 1 == kPdStages ? 0 : slot + 1;
        if (part_end) {
            // join the warps, then finish the unit or leave it for the join kernel
#pragma unroll
            for (int w = HB; w < 32; w <<= 1) l += __shfl_xor_sync(0xffffffffu, l, w);
            __syncthreads();   // the last part's sums have been read
            if (lane < HB) red_ml[warp][lane] = make_float2(m, any ? l : -1.f);
#pragma unroll
            for (int j = 0; j < HB; ++j)
#pragma unroll
                for (int e = 0; e < E; e += 2)
                    *reinterpret_cast<float2 *>(red_o + (warp * HB + j) * (D + kPdPad) + lane * E + e) =
                        make_float2(o[j][e], o[j][e + 1]);
            __syncthreads();
            pd_finish<float, D, HB>(geo, a, cw, begins, unit_end, red_ml, red_o);
            begins = true;
            any = false;
            reset();
        }
        cw = nw;
    }
    cp_async_wait<0>();
}

// D (16 x 8, fp32) += A (16 x 16, bf16) . B (16 x 8, bf16)
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <bool TRANS> __device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr)
{
    if constexpr (TRANS)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// Transposes an 8 x 8 bf16 matrix that the warp holds two elements a lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t x)
{
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// bf16: the products run on the tensor cores with the keys as the rows, so that up
// to 8 query heads of the KV head are the 8 columns of one product (HT such
// groups): S^T = K.Q^T, 16 keys x 8 heads, and O^T += V^T.P^T, 16 elements of d x 8
// heads.  K and V come by ldmatrix from rows whose 16-byte words are swizzled by
// the row's low three bits (no bank conflicts), S^T turns into the operand P^T by
// 8 x 8 transposes between registers.  P stays a sum of two bf16 terms, the value cut
// off and what that left (up to 2^-7, rounded by 2^-8 of it: together good to 2^-14, so
// the row sum may take the fp32 value), at two products.  One bf16 term makes the result's
// error 1.1 to 1.5 times that of its own rounding; it took 89, 96 and 75 us where two take
// 89, 96 and 76, and for 16 heads of width 128 62 us where two take 70.  Both terms are above
// zero where the weight is (kPdMore sees to the second), so that an infinity in V stays
// one.  The reference maximum of a head moves only when some logit exceeds it by 2^8, so
// most tiles need no reduction over the keys.
// Memory bounds it, once enough warps hide the chain of one tile (paged_decode.cuh has
// the shapes measured); the same walk on the CUDA cores took 163, 168 and 194 us where
// this takes 89, 96 and 76.
constexpr float kPdMove = 8.f;
constexpr float kPdMore = 1.f / (1 << 16);   // of the weight, added to its second term
template <int D, int HT>
__global__ void __launch_bounds__(kPdThreads)
paged_decode_bf16_kernel(PagedGeom geo, PdArgs a)
{
    using Stream = PdStream<uint16_t, D, true>;
    constexpr int KT = Stream::KT, TILE = Stream::TILE, RB = Stream::RB, HB = 8 * HT;
    constexpr int KG = KT / 16;   // groups of 16 keys
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float2 red_ml[kPdWarps][HB];
    float *red_o = reinterpret_cast<float *>(smem + kPdWarps * kPdStages * kPdStage);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int gr = lane >> 2, tc = lane & 3;   // row and column pair of this lane in a product
    const int units = geo.Hkv * a.chunks;
    pdl_trigger();   // the join may be scheduled; it waits for this grid's end
    pdl_wait();
    PdWalk cw;
    const int64_t n = pd_range<TILE>(geo, a.lens, units, cw);
    if (tid == 0) a.meta[blockIdx.x] = PdMeta{-1, 0, 0, 0};
    if (n == 0) {
        pd_empty<uint16_t, D>(geo, a);
        return;
    }
    const uint32_t ring = smem_addr(smem + warp * kPdStages * kPdStage);
    Stream stream(geo, a, cw, n, units, ring);
#pragma unroll
    for (int s = 0; s < kPdStages - 1; ++s) stream.load();
    pd_empty<uint16_t, D>(geo, a);   // behind the first loads

    // this lane's rows for ldmatrix, and the swizzle of its words
    const uint32_t k_row = uint32_t((lane & 15) * RB), v_row = uint32_t(((lane & 7) + (lane >> 4) * 8) * RB);
    const uint32_t k_word = lane >> 4, v_word = (lane >> 3) & 1, swz = lane & 7;

    uint32_t q[HT][D / 16][2];
    float o[HT][D / 16][4], m[HT][2], l[HT][2];   // of heads 8 ht + 2 tc, + 1
    auto load_q = [&](const PdWalk &w) {
        const int h = w.u / a.chunks, j0 = (w.u % a.chunks) * HB, nh = min(HB, geo.g - j0);
#pragma unroll
        for (int t = 0; t < HT; ++t) {
            const bool in = 8 * t + gr < nh;
            const uint32_t *src = reinterpret_cast<const uint32_t *>(
                static_cast<const uint16_t *>(a.q) + int64_t(w.b) * geo.qs +
                int64_t(h * geo.g + j0 + (in ? 8 * t + gr : 0)) * D);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                q[t][ks][0] = in ? src[ks * 8 + tc] : 0u;
                q[t][ks][1] = in ? src[ks * 8 + 4 + tc] : 0u;
            }
        }
    };
    auto reset = [&] {
#pragma unroll
        for (int t = 0; t < HT; ++t) {
#pragma unroll
            for (int dt = 0; dt < D / 16; ++dt)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[t][dt][e] = 0.f;
            m[t][0] = m[t][1] = -INFINITY;
            l[t][0] = l[t][1] = 0.f;
        }
    };
    load_q(cw);
    reset();
    bool begins = cw.tile == 0;   // this part of the unit starts at its first key
    bool any = false;             // some key of the part was this warp's
    int slot = 0;
    for (int64_t i = 0; i < n; ++i) {
        stream.load();
        cp_async_wait<kPdStages - 1>();
        __syncwarp();
        const uint32_t kt = ring + uint32_t(slot) * kPdStage, vt = kt + kPdHalf;
        const int key0 = cw.tile * TILE + warp * KT;
        const bool has = key0 < cw.len;   // some key of the tile is this warp's
        any |= has;
        float x[KG][HT][4];
        if (has) {
#pragma unroll
            for (int kg = 0; kg < KG; ++kg) {
                // two chains of products each, added at the end
                float y[HT][4];
#pragma unroll
                for (int t = 0; t < HT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[kg][t][e] = y[t][e] = 0.f;
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    uint32_t f[4];
                    ldmatrix4<false>(f, kt + uint32_t(kg * 16 * RB) + k_row + (((2 * ks + k_word) ^ swz) << 4));
#pragma unroll
                    for (int t = 0; t < HT; ++t) mma16816(ks & 1 ? y[t] : x[kg][t], f, q[t][ks][0], q[t][ks][1]);
                }
#pragma unroll
                for (int t = 0; t < HT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[kg][t][e] = (x[kg][t][e] + y[t][e]) * a.scale;
            }
        }
        // the last product with this unit's q: the next one's is on its way meanwhile
        const bool unit_end = cw.tile + 1 == cw.nt, part_end = unit_end || i + 1 == n;
        PdWalk nw = cw;
        if (i + 1 < n) {
            nw.next<TILE>(geo, a.lens, units);
            if (part_end) load_q(nw);
        }
        if (has) {
            if (key0 + KT > cw.len) {
#pragma unroll
                for (int kg = 0; kg < KG; ++kg)
#pragma unroll
                    for (int t = 0; t < HT; ++t)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (key0 + kg * 16 + gr + (e >> 1) * 8 >= cw.len) x[kg][t][e] = -INFINITY;
            }
            bool lift = false;
#pragma unroll
            for (int kg = 0; kg < KG; ++kg)
#pragma unroll
                for (int t = 0; t < HT; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) lift |= x[kg][t][e] > m[t][e & 1] + kPdMove;
            if (__any_sync(0xffffffffu, lift)) {
#pragma unroll
                for (int t = 0; t < HT; ++t)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float mx = fmaxf(x[0][t][e], x[0][t][e + 2]);
#pragma unroll
                        for (int kg = 1; kg < KG; ++kg) mx = fmaxf(mx, fmaxf(x[kg][t][e], x[kg][t][e + 2]));
#pragma unroll
                        for (int w = 4; w < 32; w <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
                        const float mn = fmaxf(m[t][e], mx), f = pd_weight(m[t][e], mn);
                        m[t][e] = mn;
                        l[t][e] *= f;
#pragma unroll
                        for (int dt = 0; dt < D / 16; ++dt) {
                            o[t][dt][e] *= f;
                            o[t][dt][e + 2] *= f;
                        }
                    }
            }
            // before any maximum is known every logit is -inf, which has no weight
            float ref[HT][2];
#pragma unroll
            for (int t = 0; t < HT; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e) ref[t][e] = m[t][e] == -INFINITY ? 0.f : m[t][e];
#pragma unroll
            for (int kg = 0; kg < KG; ++kg) {
                uint32_t p[HT][2], rest[HT][2];   // P = p + rest, to 2^-14
#pragma unroll
                for (int t = 0; t < HT; ++t) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float w = ex2_approx(x[kg][t][e] - ref[t][e & 1]);
                        l[t][e & 1] += w;
                        x[kg][t][e] = w;
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float w0 = x[kg][t][2 * e], w1 = x[kg][t][2 * e + 1];
                        const uint32_t hi = __byte_perm(__float_as_uint(w0), __float_as_uint(w1), 0x7632);
                        const __nv_bfloat162 r2 = __floats2bfloat162_rn(
                            fmaf(w0, kPdMore, w0 - bf16lo(hi)), fmaf(w1, kPdMore, w1 - bf16hi(hi)));
                        p[t][e] = transpose8(hi);
                        rest[t][e] = transpose8(*reinterpret_cast<const uint32_t *>(&r2));
                    }
                }
#pragma unroll
                for (int dt = 0; dt < D / 16; ++dt) {
                    uint32_t f[4];
                    ldmatrix4<true>(f, vt + uint32_t(kg * 16 * RB) + v_row + (((2 * dt + v_word) ^ swz) << 4));
#pragma unroll
                    for (int t = 0; t < HT; ++t) {
                        mma16816(o[t][dt], f, p[t][0], p[t][1]);
                        mma16816(o[t][dt], f, rest[t][0], rest[t][1]);
                    }
                }
            }
        }
        __syncwarp();   // the stage may be refilled
        slot = slot + 1 == kPdStages ? 0 : slot + 1;
        if (part_end) {
            // join the warps, then finish the unit or leave it for the join kernel
            __syncthreads();   // the last part's sums have been read
#pragma unroll
            for (int t = 0; t < HT; ++t)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
#pragma unroll
                    for (int w = 4; w < 32; w <<= 1) l[t][e] += __shfl_xor_sync(0xffffffffu, l[t][e], w);
                    const int j = 8 * t + 2 * tc + e;
                    if (gr == 0) red_ml[warp][j] = make_float2(m[t][e], any ? l[t][e] : -1.f);
                    if (!any) continue;
#pragma unroll
                    for (int dt = 0; dt < D / 16; ++dt) {
                        red_o[(warp * HB + j) * (D + kPdPad) + dt * 16 + gr] = o[t][dt][e];
                        red_o[(warp * HB + j) * (D + kPdPad) + dt * 16 + gr + 8] = o[t][dt][e + 2];
                    }
                }
            __syncthreads();
            pd_finish<uint16_t, D, HB>(geo, a, cw, begins, unit_end, red_ml, red_o);
            begins = true;
            any = false;
            reset();
        }
        cw = nw;
    }
    cp_async_wait<0>();
}

// The join: block i finishes the unit that begins in range i and goes on in the
// following ranges.  Every partial's weight is formed once; then groups of threads
// take every so many-th partial, four elements a thread with several loads in
// flight, and the groups' sums are added in order.
constexpr int kJoinThreads = 512, kJoinParts = 64;
template <typename T, int D, int HB>
__global__ void __launch_bounds__(kJoinThreads)
paged_decode_join_kernel(PagedGeom geo, PdArgs a)
{
    static_assert(HB * D / 4 <= kJoinThreads, "a thread takes at most one word");
    __shared__ int last_s;
    __shared__ float top[HB], total[HB], weight[kJoinParts][HB];
    __shared__ float4 sums[kJoinThreads];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, n = gridDim.x, first = blockIdx.x;
    if (tid == 0) last_s = n - 1;
    __syncthreads();
    pdl_wait();
    // partial x is range first + x's: its last slot for x = 0, else its first one
    auto slot_of = [&](int x) { return x == 0 ? 2 * first + 1 : 2 * (first + x); };
    // What the next lines may need, all on its way at once: what this range left, which
    // later range ends the unit (the first one whose slot says so), and the first
    // partials' maxima and sums, a warp per head (of ranges that exist, used or not)
    const PdMeta me = a.meta[first];
    bool ends = false;
    if (first + 1 + tid < n) ends = a.meta[first + 1 + tid].first == 1;
    float2 pre[kJoinParts / 32];
#pragma unroll
    for (int u = 0; u < kJoinParts / 32; ++u) {
        const int x = u * 32 + lane;
        pre[u] = warp < HB && first + x < n ? a.part_ml[slot_of(x) * HB + warp] : make_float2(0.f, 0.f);
    }
    if (me.open_b < 0) return;
    if (ends) atomicMin(&last_s, first + 1 + tid);
    for (int i = first + 1 + kJoinThreads + tid; i < n; i += kJoinThreads)
        if (a.meta[i].first == 1) atomicMin(&last_s, i);
    __syncthreads();
    const int parts = last_s - first + 1;
    const int h = me.open_u / a.chunks, j0 = (me.open_u % a.chunks) * HB;
    const int nh = min(HB, geo.g - j0);
    // the joint maximum and sum of each head, and the first partials' weights
    if (warp < nh) {
        float M = -INFINITY, L = 0.f;
        auto take = [&](const float2 &ml) {
            const float mn = fmaxf(M, ml.x);
            L = L * pd_weight(M, mn) + pd_weight(ml.x, mn) * ml.y;
            M = mn;
        };
#pragma unroll
        for (int u = 0; u < kJoinParts / 32; ++u)
            if (u * 32 + lane < parts) take(pre[u]);
        for (int x = kJoinParts + lane; x < parts; x += 32) take(a.part_ml[slot_of(x) * HB + warp]);
        float all = M;
#pragma unroll
        for (int w = 16; w; w >>= 1) all = fmaxf(all, __shfl_xor_sync(0xffffffffu, all, w));
        L *= pd_weight(M, all);
#pragma unroll
        for (int w = 16; w; w >>= 1) L += __shfl_xor_sync(0xffffffffu, L, w);
        if (lane == 0) {
            top[warp] = all;
            total[warp] = L;
        }
#pragma unroll
        for (int u = 0; u < kJoinParts / 32; ++u)
            if (u * 32 + lane < parts) weight[u * 32 + lane][warp] = pd_weight(pre[u].x, all);
    }
    // groups of threads, one float4 word of the heads a thread
    const int words = nh * D / 4, groups = kJoinThreads / words, group = tid / words, word = tid % words;
    const int j = word * 4 / D;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int x0 = 0; x0 < parts; x0 += kJoinParts) {
        const int np = min(kJoinParts, parts - x0);
        __syncthreads();
        if (x0 > 0) {
            for (int y = tid; y < np * nh; y += kJoinThreads) {
                const int x = y / nh, i = y - x * nh;
                weight[x][i] = pd_weight(a.part_ml[slot_of(x0 + x) * HB + i].x, top[i]);
            }
            __syncthreads();
        }
        if (group < groups)
#pragma unroll 8
            for (int x = group; x < np; x += groups) {
                const float4 v =
                    reinterpret_cast<const float4 *>(a.part_acc + int64_t(slot_of(x0 + x)) * HB * D)[word];
                const float f = weight[x][j];
                acc.x = fmaf(f, v.x, acc.x);
                acc.y = fmaf(f, v.y, acc.y);
                acc.z = fmaf(f, v.z, acc.z);
                acc.w = fmaf(f, v.w, acc.w);
            }
    }
    sums[tid] = acc;
    __syncthreads();
    if (group > 0) return;
    for (int i = 1; i < groups; ++i) {
        const float4 v = sums[i * words + tid];
        acc.x += v.x;
        acc.y += v.y;
        acc.z += v.z;
        acc.w += v.w;
    }
    const int c = word * 4 - j * D;
    T *dst = static_cast<T *>(a.out) + (int64_t(me.open_b) * geo.Hq + h * geo.g + j0 + j) * D + c;
    const float il = 1.f / total[j];
    store_elem(dst, acc.x * il);
    store_elem(dst + 1, acc.y * il);
    store_elem(dst + 2, acc.z * il);
    store_elem(dst + 3, acc.w * il);
}

constexpr int kPdResident = 2;   // CTAs of an SM, at most
constexpr int kMaxHeads = 16;   // query heads of a unit, at most

template <typename T, int D, int HB>
cudaError_t run(void (*kern)(PagedGeom, PdArgs), const PagedGeom &g, PdArgs a, cudaStream_t st)
{
    a.chunks = (g.g + HB - 1) / HB;
    const size_t smem = size_t(kPdWarps) * kPdStages * kPdStage + size_t(kPdWarps) * HB * (D + kPdPad) * 4;
    // one range per CTA that the SMs hold at once (two, three or four, handed out as CTAs
    // end, even out SMs of different speed but cost more starts and partials: 97, 102 and
    // 109 us where one takes 88, one sequence of 131073 tokens)
    const int ranges = num_sms() * int(std::min<size_t>(kPdResident, 228 * 1024 / (smem + 2048)));
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e != cudaSuccess) return e;
    e = launch_pdl(kern, dim3(unsigned(ranges)), dim3(kPdThreads), smem, st, g, a);
    if (e != cudaSuccess) return e;
    return launch_pdl(paged_decode_join_kernel<T, D, HB>, dim3(unsigned(ranges)), dim3(kJoinThreads), 0, st, g, a);
}
// Query heads of a unit: as few as hold the group, at most 8 (fp32, whose products
// cost an instruction each) or 16.
template <int D> cudaError_t run_d(const PagedGeom &g, const PdArgs &a, cudaStream_t st)
{
    if (g.dtype == REATT_BF16)
        return g.g <= 8 ? run<uint16_t, D, 8>(paged_decode_bf16_kernel<D, 1>, g, a, st)
                        : run<uint16_t, D, 16>(paged_decode_bf16_kernel<D, 2>, g, a, st);
    return g.g <= 4 ? run<float, D, 4>(paged_decode_f32_kernel<D, 4>, g, a, st)
                    : run<float, D, 8>(paged_decode_f32_kernel<D, 8>, g, a, st);
}

int max_ranges() { return kPdResident * num_sms(); }

}  // namespace

size_t paged_decode_ws_bytes(const PagedGeom &g)
{
    const size_t n = size_t(max_ranges());
    return n * sizeof(PdMeta) + 2 * n * kMaxHeads * (sizeof(float2) + size_t(g.d) * sizeof(float));
}

cudaError_t launch_paged_decode(const PagedGeom &g, const void *q, const void *k_pages,
                                const void *v_pages, const int32_t *table, const int32_t *lens,
                                void *out, void *scratch, void *ws, cudaStream_t st)
{
    const int n = max_ranges();
    uint8_t *p = static_cast<uint8_t *>(scratch);
    PdArgs a{q, k_pages, v_pages, table, lens, out, nullptr, nullptr, nullptr, ws, 1,
             float(1.4426950408889634 / sqrt(double(g.d)))};
    a.part_acc = reinterpret_cast<float *>(p);
    a.part_ml = reinterpret_cast<float2 *>(p + size_t(2 * n) * kMaxHeads * g.d * sizeof(float));
    a.meta = reinterpret_cast<PdMeta *>(a.part_ml + size_t(2 * n) * kMaxHeads);
    return g.d == 128 ? run_d<128>(g, a, st) : run_d<64>(g, a, st);
}

}  // namespace reatt

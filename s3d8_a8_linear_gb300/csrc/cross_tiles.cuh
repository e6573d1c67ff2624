// What the cross attention kernels share (cross_attention.cu, cross_attention_backward.cu):
// tensor-memory accesses and MMAs whose A operand lies there, tensor maps of rows
// [tokens or states, heads, dim], and spans.
#pragma once

#include "launch.h"
#include "tcgen05.cuh"
#include "uniform.cuh"

namespace s3d8 {

namespace cross {

constexpr int kTile = 128;              // rows of a tile: query rows, or states
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// ---- tensor memory ----------------------------------------------------------

// 32 columns of the thread's lane.
__device__ __forceinline__ void tmem_ld32(uint32_t at, float *v)
{
    uint32_t r[32];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
                 "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
                   "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
                   "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
                   "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(at));
#pragma unroll
    for (int i = 0; i < 32; ++i)
        v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void tmem_st32(uint32_t at, const uint32_t *r)
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
                 "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(at),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
                 "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
                 "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
                 "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
                 : "memory");
}

__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// D (tensor memory) = A (tensor memory, bf16 pairs) B (shared memory) (+ D), one elected lane.
__device__ __forceinline__ void mma_tmem_a_elect(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n.reg .pred p, e;\nsetp.ne.b32 p, %4, 0;\nelect.sync _|e, 0xffffffff;\n"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

// A tile of rows x 64 columns of bf16 (128 bytes a row, 128-byte swizzle) as an operand whose
// sums run over the columns (tc::sw128_desc), or, here, over the rows: eight rows lie 1024
// bytes from the next eight, 64 columns `chunk` bytes from the next 64.
__device__ __forceinline__ uint64_t rows_desc(uint32_t a, uint32_t chunk)
{
    return (uint64_t)((a & 0x3FFFFu) >> 4) | ((uint64_t)(chunk >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) |
           (2ull << 61);
}

// Instruction descriptors: bf16 operands, fp32 sums, M = 128.
__device__ __forceinline__ uint32_t idesc_cols(int n) { return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | (8u << 24); }
__device__ __forceinline__ uint32_t idesc_rows(int n) { return idesc_cols(n) | (1u << 16); }
constexpr uint32_t kNegateA = 1u << 13;

__device__ __forceinline__ void tma_3d_elect(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar)
{
    asm volatile(
        "{\n.reg .pred e;\nelect.sync _|e, 0xffffffff;\n"
        "@e cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];\n}\n" ::"r"(dst),
        "l"((uint64_t)map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

// A wait of a warp that meets others at barriers: once one ran out it waits no more, and runs
// on to the end with what it finds, so that the others are not left waiting.
__device__ __forceinline__ void wait_on(bool &ok, uint32_t bar, uint32_t parity)
{
    if (ok)
        ok = tc::warp_wait(bar, parity);
    tc::tc_fence_after();
}

// ---- arithmetic -------------------------------------------------------------

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// What turns a product q . k into a base-2 exponent, but for its sign.  Not 0, so that a hidden
// score stays -inf: the least number that there is, which makes nothing of any other score.
__device__ __forceinline__ float exponents(float scale) { return fmaxf(fabsf(scale) * kLog2e, __uint_as_float(1u)); }

// Two bf16 in a word, lo first.
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two fp32 at once.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    uint64_t d, x = *reinterpret_cast<uint64_t *>(&a), y = *reinterpret_cast<uint64_t *>(&b), z = *reinterpret_cast<uint64_t *>(&c);
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(x), "l"(y), "l"(z));
    return *reinterpret_cast<float2 *>(&d);
}

__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    uint64_t d, x = *reinterpret_cast<uint64_t *>(&a), y = *reinterpret_cast<uint64_t *>(&b);
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(x), "l"(y));
    return *reinterpret_cast<float2 *>(&d);
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    uint64_t d, x = *reinterpret_cast<uint64_t *>(&a), y = *reinterpret_cast<uint64_t *>(&b);
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(x), "l"(y));
    return *reinterpret_cast<float2 *>(&d);
}

// ---- spans ------------------------------------------------------------------

// Token t's span, cut to the states; an empty one is (0, 0).  `record`: one that leaves the
// states is recorded.
__device__ __forceinline__ int2 span_of(const int32_t *spans, int S, int t, int *record)
{
    if (!spans)
        return make_int2(0, S);
    const int2 s = __ldg(reinterpret_cast<const int2 *>(spans) + t);
    if (s.x >= s.y)
        return make_int2(0, 0);
    if (record && (s.x < 0 || s.y > S))
        atomicExch(record, kStatusBounds);
    const int2 c = make_int2(max(s.x, 0), min(s.y, S));
    return c.x < c.y ? c : make_int2(0, 0);
}

// ---- work -------------------------------------------------------------------

// A piece of the work of every key/value head: a tile (of query rows, or of states) and the
// tiles j0 and on of the other kind; `begin`: such tiles of the pieces in front of it.  Lists
// end with an entry that has only that.
struct Item {
    int tile, j0, begin;
};

struct Piece {
    int item, tile, head, j0, n, slot;  // slot: -1 for a whole item, else where its sums go: 0 or 1
    int item_end;                       // tiles of all heads in front of the item's end
    bool begins;                        // the item, and not only a piece of it
};

// How many CTAs have a share: none of them an empty one.
__device__ __forceinline__ int64_t busy(int ctas, int64_t all) { return all < ctas ? all : ctas; }

// A CTA's share of the work of all heads: as many tiles as any other's, one behind the
// other, piece by piece.  (Launches keep the number of all tiles below 2^31.)
struct Share {
    const Item *items;
    int n_items, per_head, at, end;
    bool begun;

    __device__ __forceinline__ Share(const Item *list, int n, int heads, int ctas)
        : items(list), n_items(n), per_head(uniform(list[n].begin)), begun(false)
    {
        const int64_t all = (int64_t)heads * per_head, some = busy(ctas, all);
        at = blockIdx.x < some ? (int)(all * blockIdx.x / some) : 0;
        end = blockIdx.x < some ? (int)(all * (blockIdx.x + 1) / some) : 0;
    }

    __device__ __forceinline__ bool next(Piece &u)
    {
        if (at >= end)
            return false;
        u.head = at / per_head;
        const int r = at - u.head * per_head;
        int lo = 0, hi = n_items;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (uniform(items[mid].begin) <= r)
                lo = mid;
            else
                hi = mid;
        }
        const int off = r - uniform(items[lo].begin), left = uniform(items[lo + 1].begin) - r;
        u.item = lo;
        u.tile = uniform(items[lo].tile);
        u.j0 = uniform(items[lo].j0) + off;
        u.n = min(end - at, left);
        u.slot = off == 0 && u.n == left ? -1 : begun;
        u.begins = off == 0;
        u.item_end = at + left;
        at += u.n;
        begun = true;
        return true;
    }
};

// A run of tiles of states that some row of an item sees: its first, and how many come in
// front of it in the item's runs, which end with an entry that has only that.
struct Run {
    int first, begin;
};

// Which tile of states a piece's i-th one is, for growing i.
struct Walk {
    const Run *run;
    int off, end, shift;

    // `off`: tiles of the item's runs in front of the piece
    __device__ __forceinline__ Walk(const Run *runs, int off) : run(runs), off(off), end(0), shift(0) { load(); }
    __device__ __forceinline__ void load()
    {
        const int begin = uniform(run->begin);
        shift = uniform(run->first) - begin + off;
        end = uniform(run[1].begin) - off;
    }
    __device__ __forceinline__ int operator()(int i)
    {
        while (i >= end) {
            ++run;
            load();
        }
        return i + shift;
    }
};

// The runs of tokens t0 .. t0 + n - 1 (at most 32 E), at most `most` of them: the last one
// goes on over tiles that nobody sees.  One warp; how many tiles.
template <int E>
__device__ __forceinline__ int make_runs(const int32_t *spans, int S, int t0, int n, int most, Run *runs, int *record)
{
    const int lane = threadIdx.x & 31;
    int lo[E], hi[E], last = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int2 s = e * 32 + lane < n ? span_of(spans, S, t0 + e * 32 + lane, record) : make_int2(0, 0);
        lo[e] = s.x < s.y ? s.x / kTile : 0x7FFFFFFF;
        hi[e] = s.x < s.y ? (s.y + kTile - 1) / kTile : 0;
        last = max(last, hi[e]);
    }
    last = __reduce_max_sync(0xffffffffu, last);
    int end = 0, count = 0, made = 0;
    while (end < last) {
        int first = 0x7FFFFFFF;
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (hi[e] > end)
                first = min(first, max(lo[e], end));
        first = __reduce_min_sync(0xffffffffu, first);
        if (lane == 0)
            runs[made] = {first, count};
        ++made;
        end = first;
        if (made == most)
            end = last;
        for (bool more = end < last; more;) {
            int to = end;
#pragma unroll
            for (int e = 0; e < E; ++e)
                if (lo[e] <= end)
                    to = max(to, hi[e]);
            to = __reduce_max_sync(0xffffffffu, to);
            more = to > end;
            end = to;
        }
        count += end - first;
    }
    if (count == 0) {           // one, of which nothing is seen
        if (lane == 0)
            runs[0] = {0, 0};
        made = count = 1;
    }
    if (lane == 0)
        runs[made] = {0, count};
    return count;
}

// How a warp stores 32 columns of the rows that its lanes have: four lanes exchange 16-byte
// pieces, so that each store writes 64 bytes of eight rows and not 16 of 32 (which takes the
// load/store unit a step a row: a tile's 128 KB of results 4000 clocks).
struct RowStores {
    int64_t at[4];              // of the rows of this lane's four: where they begin, or -1

    __device__ __forceinline__ explicit RowStores(int64_t mine)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            at[i] = __shfl_sync(0xffffffffu, mine, (threadIdx.x & 28) + i);
    }
    // piece i of row j to row i of piece j, of four lanes
    static __device__ __forceinline__ void turn(uint4 (&x)[4])
    {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int b = 1; b < 4; b <<= 1)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (i & b)
                    continue;
                const uint4 to = lane & b ? x[i] : x[i | b];
                const uint4 from = make_uint4(__shfl_xor_sync(0xffffffffu, to.x, b), __shfl_xor_sync(0xffffffffu, to.y, b),
                                              __shfl_xor_sync(0xffffffffu, to.z, b), __shfl_xor_sync(0xffffffffu, to.w, b));
                if (lane & b)
                    x[i] = from;
                else
                    x[i | b] = from;
            }
    }
    // columns c .. c + 31 as bf16, those below dim
    __device__ __forceinline__ void bf16(__nv_bfloat16 *out, const float *o, int c, int dim, float by) const
    {
        uint4 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            x[i] = make_uint4(pack2(o[8 * i] * by, o[8 * i + 1] * by), pack2(o[8 * i + 2] * by, o[8 * i + 3] * by),
                              pack2(o[8 * i + 4] * by, o[8 * i + 5] * by), pack2(o[8 * i + 6] * by, o[8 * i + 7] * by));
        turn(x);
        c += 8 * (threadIdx.x & 3);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (at[i] >= 0 && c < dim)
                *reinterpret_cast<uint4 *>(out + at[i] + c) = x[i];
    }
    // as they are
    __device__ __forceinline__ void fp32(float *out, const float *o, int c) const
    {
#pragma unroll
        for (int h = 0; h < 32; h += 16) {
            uint4 x[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x[i] = make_uint4(__float_as_uint(o[h + 4 * i]), __float_as_uint(o[h + 4 * i + 1]), __float_as_uint(o[h + 4 * i + 2]),
                                  __float_as_uint(o[h + 4 * i + 3]));
            turn(x);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (at[i] >= 0)
                    *reinterpret_cast<uint4 *>(out + at[i] + c + h + 4 * (threadIdx.x & 3)) = x[i];
        }
    }
};

// A lane's columns of a row of DP fp32 sums: DP / 32 neighbouring ones.
template <int DP>
struct Columns;
template <>
struct Columns<64> {
    static __device__ __forceinline__ void get(const float *row, float (&x)[2])
    {
        const float2 v = reinterpret_cast<const float2 *>(row)[threadIdx.x & 31];
        x[0] = v.x, x[1] = v.y;
    }
    static __device__ __forceinline__ void put(__nv_bfloat16 *row, const float (&x)[2]) { reinterpret_cast<uint32_t *>(row)[threadIdx.x & 31] = pack2(x[0], x[1]); }
};
template <>
struct Columns<128> {
    static __device__ __forceinline__ void get(const float *row, float (&x)[4])
    {
        const float4 v = reinterpret_cast<const float4 *>(row)[threadIdx.x & 31];
        x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    }
    static __device__ __forceinline__ void put(__nv_bfloat16 *row, const float (&x)[4])
    {
        reinterpret_cast<uint2 *>(row)[threadIdx.x & 31] = make_uint2(pack2(x[0], x[1]), pack2(x[2], x[3]));
    }
};

// Most tiles of a launch that have sums of their own, where each may pass `others`.
inline int most_tiles(int64_t heads, int64_t others, int most)
{
    const int64_t fit = 0x7FFFFFFF / (heads * (others > 0 ? others : 1));
    return (int)(fit < most ? fit : most);
}

// What a CTA's share leaves to be joined: the item that begins in it and ends in a later one's.
// Its parts are in slot `slot` of this CTA and the first slots of those behind it, up to c1.
struct Cut {
    int tile, head, slot, c1;           // c1 < 0: nothing
};

// From the last piece of a share (`some`: there was one).
__device__ __forceinline__ Cut cut_of(const Share &share, const Piece &u, bool some, int heads, int ctas)
{
    Cut c = {0, 0, 0, -1};
    if (some && u.slot >= 0 && u.begins) {
        const int64_t all = (int64_t)heads * share.per_head;
        c = {u.tile, u.head, u.slot, (int)((u.item_end * busy(ctas, all) - 1) / all)};
    }
    return c;
}

// Whether two packed maxima of |bf16| bits are of finite values.
__device__ __forceinline__ bool finite2(uint32_t top) { return (top & 0xFFFFu) < 0x7F80u && (top >> 16) < 0x7F80u; }

// Where 16-byte chunk c of row r lies in a tile of 128-byte swizzled rows, 64 columns a block.
__device__ __forceinline__ uint32_t chunk_at(uint32_t tile, int r, int c)
{
    return tile + (c >> 3) * (kTile * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

// ---- host -------------------------------------------------------------------

// Rows [n, heads, dim] with strides (row, head) in elements, copied in pieces of `box_rows`
// rows x `box_heads` heads x 64 columns; what lies behind an end is zero.  The stride of an
// axis of one element means nothing (the binding passes 0).
inline cudaError_t row_map(CUtensorMap *map, const __nv_bfloat16 *p, int64_t n, int64_t heads, int64_t dim, const int64_t st[2],
                           int box_heads, int box_rows)
{
    auto encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(tensor_map_encoder_fn());
    if (!encode)
        return cudaErrorNotSupported;
    const cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)n};
    const cuuint64_t strides[2] = {(cuuint64_t)(heads > 1 ? st[1] : dim) * 2, (cuuint64_t)(n > 1 ? st[0] : dim) * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows}, es[3] = {1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<__nv_bfloat16 *>(p), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}

}  // namespace cross

}  // namespace s3d8

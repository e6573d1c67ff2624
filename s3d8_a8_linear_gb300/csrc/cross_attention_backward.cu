// The gradients of attention to an encoder's states (s3d8_cross_attention_backward):
//
//   delta = dout . out, p_j = exp(s_j - lse), ds_j = p_j (dout . v_j - delta)
//   dq = scale sum_j ds_j k_j, dk_j = scale sum ds_j q, dv_j = sum p_j dout
//
// Without atomics, so that equal inputs give equal bits: one kernel passes the states for
// each tile of 128 query rows (S = Q K^T, dP = dO V^T, dQ += dS K), one the query rows for
// each tile of 128 states (S^T = K Q^T, dP^T = V dO^T, dV += P^T dO, dK += dS^T Q): seven
// products where one pass with atomic sums would have five.  Tiles, sums in tensor memory,
// and shares of the work are as in the forward pass (cross_attention.cu); the two groups of
// four softmax warps take 64 columns each of every tile, and P and dS go back into tensor
// memory as bf16 A operands (2^-8 of each, which averages to about the rounding of the
// gradients).  Products are issued so that the tensor cores have two of them to do while a
// softmax step runs.
//
// Measured (2 x 2048 tokens of 32 / 8 heads of 128, 4 images of 3202 states): dq 210 us, its
// tensor pipe busy 65% of the time; dkv 340 us, 52%; with the first two kernels and the sums of
// what shares cut 580 us.  dkv's four products of a visit take 3200 clocks where 2060 would be the
// least: their operands and the copies use shared memory's bandwidth nearly whole (a product of
// two operands there takes 128 bytes a clock), and P and dS wait for one another.
//
// A first kernel makes delta and lse ready, a row a half warp, and the range of states that
// each query tile sees; one behind it delta of the rows that see few states.  Rows of the query
// tiles or the states that have no part in a tile are taken out of it where they hold infinities
// or NaN, which a weight of zero would not silence.
#include "bf16x8.cuh"
#include "cross_tiles.cuh"

namespace s3d8 {

namespace {

using namespace cross;

constexpr int kDqThreads = 512;         // warps: 0 copies, 1 and 2 products, 4 to 11 softmax, 12 to 15 look tiles over
constexpr int kThreads = 384;           // 0 copies, 1 products, 2 and 3 look tiles over, 4 to 11 softmax
constexpr int kMostTiles = 128;         // tiles of a launch that have sums of their own (their list fits beside five tiles of 32 KB)
constexpr int kJoinWarps = 8;

struct Plan {
    int tokens_a_tile, chunk_rows;      // query rows that a copy fills
    int q_tiles;                        // in all
    int first, tiles;                   // of this launch: query tiles or tiles of states
    int rows, ctas;                     // rows of a slot of partial sums
    float *info;                        // [q_tiles][heads][4][128]: -lse in base-2 exponents, -delta, the span's ends
    int2 *ranges;                       // [q_tiles]: states that some row sees
    float *parts;                       // [ctas][2][1 or 2][rows][DP]
    Cut *cuts;                          // [ctas]: what there is to add
    int negative;
};

// What there is to know about the rows of a tile of one key/value head.
__device__ __forceinline__ float *info_of(const Plan &p, int heads, int tile, int head) { return p.info + ((int64_t)tile * heads + head) * 4 * kTile; }

constexpr int kReadyRows = 32;          // of a block

// delta and lse of some of a tile's rows of one key/value head, and the tile's range.
__global__ __launch_bounds__(256) void cross_ready_kernel(const __grid_constant__ CrossArgs a, const __grid_constant__ Plan p)
{
    tc::pdl_launch_dependents();
    tc::pdl_wait();
    const int tile = blockIdx.x, head = blockIdx.y, group = a.Hq / a.heads, half = threadIdx.x >> 4, lane = threadIdx.x & 15;
    const int t0 = tile * p.tokens_a_tile;
    if (head == 0 && blockIdx.z == 0 && threadIdx.x < 32) {
        int lo = 0x7FFFFFFF, hi = 0;
        for (int i = threadIdx.x; i < p.tokens_a_tile && t0 + i < a.T; i += 32) {
            const int2 s = span_of(a.spans, a.S, t0 + i, a.status);
            if (s.x < s.y)
                lo = min(lo, s.x), hi = max(hi, s.y);
        }
        lo = __reduce_min_sync(0xffffffffu, lo);
        hi = __reduce_max_sync(0xffffffffu, hi);
        if (threadIdx.x == 0)
            p.ranges[tile] = make_int2(lo, hi);
    }
#pragma unroll
    for (int r = blockIdx.z * kReadyRows + half; r < (int)(blockIdx.z + 1) * kReadyRows; r += 16) {    // whole warps together
        const int t = t0 + r / group, h = head * group + r % group;
        const bool live = r < p.chunk_rows && t < a.T;
        float sum = 0.0f;
        if (live && 8 * lane < a.dim) {
            const uint4 x = ldg_stream_v4(a.dout + t * a.ds[0] + h * a.ds[1] + 8 * lane);
            const uint4 y = ldg_stream_v4(a.out + ((int64_t)t * a.Hq + h) * a.dim + 8 * lane);
            const uint32_t u[4] = {x.x, x.y, x.z, x.w}, w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                sum = fmaf(__uint_as_float(u[e] & 0xFFFF0000u), __uint_as_float(w[e] & 0xFFFF0000u),
                           fmaf(__uint_as_float(u[e] << 16), __uint_as_float(w[e] << 16), sum));
        }
#pragma unroll
        for (int o = 8; o > 0; o >>= 1)
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const int2 see = live ? span_of(a.spans, a.S, t, nullptr) : make_int2(0, 0);
        const bool some = see.x < see.y;
        if (lane == 0) {
            float *to = info_of(p, a.heads, tile, head) + r;
            to[0] = some ? -a.lse[(int64_t)t * a.Hq + h] * kLog2e : -INFINITY;
            to[kTile] = some ? -sum : 0.0f;
            to[2 * kTile] = __int_as_float(see.x);
            to[3 * kTile] = __int_as_float(see.y);
        }
    }
}

// delta is dout . out, but out is rounded to bf16: that is off by 2^-9 of a product whose size
// falls with the square root of the number n of states, as against the dout . v_j that it is
// taken from.  With few states it would be most of the error of dq and dk (n = 2: 2.4 times
// that of their own rounding, 19: 1.6 times, from 128 on 1.45 times, which is that of ds), so
// there it is summed from its parts, p_j (dout . v_j).
constexpr int kFew = 128;
constexpr int kFewWarps = 4;            // of a block
constexpr int kNever = 0x7FFFFFFF;

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A lane's part of a row: columns 8 (c + 4 i) .. + 7.
template <int N>
__device__ __forceinline__ void row_chunks(const __nv_bfloat16 *row, int c, int dim, bool some, uint4 (&x)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i)
        x[i] = some && 8 * (c + 4 * i) < dim ? __ldg(reinterpret_cast<const uint4 *>(row) + c + 4 * i) : make_uint4(0u, 0u, 0u, 0u);
}

// delta of a tile's rows that see few states.  A warp has 16 rows and passes the states that some
// of them see, 16 at a time.  Its products are mma.sync: a tcgen05 tile of 128 rows would pass the
// states of all their tokens, and here operands go from global memory straight into registers,
// whatever the spans are (a lane's chunks of 16 bytes are the columns of two products, in the same
// order for both operands).
// Measured (step of 8 x 1024 tokens of 32 / 8 heads of 128, 128 states each): 99 us of 320, 10 where
// no token sees few; half a warp a row with scalar sums took 2.06 ms of 2.24.
template <int DP>
__global__ __launch_bounds__(kFewWarps * 32, 3) void cross_few_kernel(const __grid_constant__ CrossArgs a, const __grid_constant__ Plan p)
{
    constexpr int N = DP / 32;
    tc::pdl_launch_dependents();
    tc::pdl_wait();
    const int tile = blockIdx.x, head = blockIdx.y, group = a.Hq / a.heads, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int r0 = (blockIdx.z * kFewWarps + warp_index()) * 16;
    int2 see[2];
#pragma unroll
    for (int y = 0; y < 2; ++y) {
        const int r = r0 + 8 * y + g, t = tile * p.tokens_a_tile + r / group;
        see[y] = r < p.chunk_rows && t < a.T ? span_of(a.spans, a.S, t, nullptr) : make_int2(0, 0);
        if (see[y].y - see[y].x > kFew)
            see[y] = make_int2(0, 0);
    }
    // the first state from `from` on that some row sees
    auto next = [&](int from) {
        int n = kNever;
#pragma unroll
        for (int y = 0; y < 2; ++y)
            if (see[y].y > from && see[y].x < see[y].y)
                n = min(n, max(see[y].x, from));
        return __reduce_min_sync(0xffffffffu, n);
    };
    int at = next(0);
    if (at == kNever)
        return;
    uint4 q[2][N], d[2][N];
    float lse[2], sum[2] = {0.0f, 0.0f};
#pragma unroll
    for (int y = 0; y < 2; ++y) {
        const int r = r0 + 8 * y + g, h = head * group + r % group;
        const int64_t t = tile * p.tokens_a_tile + r / group;
        const bool some = see[y].x < see[y].y;
        row_chunks(a.q + t * a.qs[0] + h * a.qs[1], c, a.dim, some, q[y]);
        row_chunks(a.dout + t * a.ds[0] + h * a.ds[1], c, a.dim, some, d[y]);
        lse[y] = some ? -a.lse[t * a.Hq + h] * kLog2e : 0.0f;
    }
    const float scale = a.scale * kLog2e;
    for (; at != kNever; at = next(at + 16)) {
        uint4 k[2][N], v[2][N];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int j = at + 8 * n + g;
            row_chunks(a.k + j * a.ks[0] + head * a.ks[1], c, a.dim, j < a.S, k[n]);
            row_chunks(a.v + j * a.vs[0] + head * a.vs[1], c, a.dim, j < a.S, v[n]);
        }
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            float s[4] = {0.0f, 0.0f, 0.0f, 0.0f}, dp[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const uint32_t q0[4] = {q[0][i].x, q[1][i].x, q[0][i].y, q[1][i].y}, q1[4] = {q[0][i].z, q[1][i].z, q[0][i].w, q[1][i].w};
                const uint32_t d0[4] = {d[0][i].x, d[1][i].x, d[0][i].y, d[1][i].y}, d1[4] = {d[0][i].z, d[1][i].z, d[0][i].w, d[1][i].w};
                mma_bf16(s, q0, k[n][i].x, k[n][i].y);
                mma_bf16(dp, d0, v[n][i].x, v[n][i].y);
                mma_bf16(s, q1, k[n][i].z, k[n][i].w);
                mma_bf16(dp, d1, v[n][i].z, v[n][i].w);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int y = e >> 1, j = at + 8 * n + 2 * c + (e & 1);
                const float part = ex2(fmaf(s[e], scale, lse[y])) * dp[e];
                sum[y] += j >= see[y].x && j < see[y].y ? part : 0.0f;
            }
        }
    }
#pragma unroll
    for (int y = 0; y < 2; ++y) {
        sum[y] += __shfl_xor_sync(0xffffffffu, sum[y], 1);
        sum[y] += __shfl_xor_sync(0xffffffffu, sum[y], 2);
        if (c == 0 && see[y].x < see[y].y)
            info_of(p, a.heads, tile, head)[kTile + r0 + 8 * y + g] = -sum[y];
    }
}

// The list of work of a launch: for each of its tiles, the tiles of the other kind that have
// a part in it, or one (of which nothing is seen).  One warp, from each tile's first and end.
template <typename Range>
__device__ __forceinline__ void make_list(int tiles, Item *items, Range range)
{
    const int lane = threadIdx.x & 31;
    int begin = 0;
    for (int base = 0; base < tiles; base += 32) {
        const int i = base + lane;
        int2 r = make_int2(0, 0);
        if (i < tiles) {
            r = range(i);
            if (r.x >= r.y)
                r = make_int2(0, 1);
        }
        const int size = r.y - r.x;
        int s = size;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int ps = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o)
                s += ps;
        }
        if (i < tiles)
            items[i] = {i, r.x, begin + s - size};
        begin += __shfl_sync(0xffffffffu, s, 31);
    }
    if (lane == 0)
        items[tiles] = {0, 0, begin};
}

// LONG places of the ring are for tiles in use from a visit's first product to its last (keys,
// or query rows), SHORT ones for the others (values, or dout).
template <int DP, int LONG_, int SHORT_>
struct Layout {
    static constexpr int CHUNKS = DP / 64;
    static constexpr int TILE = kTile * DP * 2;
    static constexpr int LONG = LONG_, SHORT = SHORT_, STAGES = LONG + SHORT;
    static constexpr int FIX = 0, RING = 2 * TILE, ITEMS = RING + STAGES * TILE;
    static constexpr int BARS = ITEMS + ((kMostTiles + 1) * (int)sizeof(Item) + 7) / 8 * 8, SLOT = BARS + 80 + 24 * STAGES;

    // where visit v's tile is, and how often its place was filled before
    static __device__ __forceinline__ int place(int v, int s) { return s ? LONG + v % SHORT : v % LONG; }
    static __device__ __forceinline__ int lap(int v, int s) { return s ? v / SHORT : v / LONG; }
};

// Five tiles of 32 KB are all that fits beside the two fixed ones: with four, dq waited for its
// keys (338 us of 2 x 2048 tokens' gradients, 216 with five and a product warp more).  dkv has
// four and its rows' statistics: a fifth with those in single places took 399 us for 351.
template <int DP>
struct DqLayout : Layout<DP, DP == 128 ? 3 : 6, DP == 128 ? 2 : 4> {
    static constexpr int DS_FREE = DqLayout::SLOT + 8, BYTES = DS_FREE + 16;
};

// Of a visit's query rows: [LONG][2] whether 64 of them see the whole tile, [LONG][128] the part of
// it that each sees, [LONG][2][128] -lse and -delta.
template <int DP>
struct DkvLayout : Layout<DP, DP == 128 ? 2 : 4, DP == 128 ? 2 : 4> {
    static constexpr int FULL = DkvLayout::SLOT + 8, SEEN = (FULL + DkvLayout::LONG * 8 + 15) / 16 * 16, INFO = SEEN + DkvLayout::LONG * kTile * 2;
    static constexpr int BYTES = INFO + DkvLayout::LONG * 2 * kTile * 4;
};

__device__ __forceinline__ void setup_common(uint32_t *tmem_slot, int warp)
{
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(tmem_slot)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
}

// Not before the last copies of `visits` visits have landed.
template <typename L>
__device__ __forceinline__ bool landed(uint32_t full, int visits)
{
    bool ok = true;
    for (int st = 0; st < L::STAGES; ++st) {
        const int s = st >= L::LONG, i = st - s * L::LONG, n = s ? L::SHORT : L::LONG, uses = (visits - i + n - 1) / n;
        if (visits > i)
            ok &= tc::warp_wait(full + 8 * st, (uses - 1) & 1);
    }
    return ok;
}

// A row of 128-byte swizzled chunks that holds an infinity or NaN.
template <int DP>
__device__ __forceinline__ bool bad_row(uint32_t tile, int r)
{
    uint32_t top = 0;
#pragma unroll 4
    for (int c = 0; c < DP / 8; ++c)
        top = absmax_bf16x8(lds_v4(chunk_at(tile, r, c)), top);
    return !finite2(top);
}

template <int DP>
__device__ __forceinline__ void clear_row(uint32_t tile, int r)
{
    for (int c = 0; c < DP / 8; ++c)
        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(chunk_at(tile, r, c)), "r"(0u) : "memory");
}

// ---- dq ---------------------------------------------------------------------

// Tensor memory: S 128 columns, dP twice 128 (dS over each), dQ.
template <int DP>
__global__ __launch_bounds__(kDqThreads, 1) void cross_dq_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_d,
                                                               const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                                                               const __grid_constant__ CrossArgs a, const __grid_constant__ Plan p)
{
    using L = DqLayout<DP>;
    extern __shared__ __align__(1024) unsigned char cross_mem_aligned[];
    unsigned char *mem = cross_mem_aligned;
    const uint32_t base = smem_addr(mem);
    if (base & 1023u) {         // (the first of the CTA's shared memory)
        record_timeout(a.status);
        return;
    }
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(mem + L::SLOT);
    Item *items = reinterpret_cast<Item *>(mem + L::ITEMS);
    const uint32_t bars = base + L::BARS;
    const uint32_t q_full = bars, q_empty = bars + 8, o_free = bars + 16, s_full = bars + 24, s_read = bars + 32, done = bars + 40;
    const uint32_t dp_full = bars + 48, ds_ready = bars + 64, ds_free = base + L::DS_FREE;     // two each: of either buffer
    const uint32_t kv_full = bars + 80, kv_empty = kv_full + 8 * L::STAGES, k_ok = kv_empty + 8 * L::STAGES;
    const int warp = warp_index(), lane = threadIdx.x & 31, group = a.Hq / a.heads;
    if (threadIdx.x == 0) {
        mbar_init(q_full, 1);
        mbar_init(q_empty, 1);
        mbar_init(o_free, 8);
        mbar_init(s_full, 1);
        mbar_init(s_read, 8);
        mbar_init(done, 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(dp_full + 8 * s, 1);
            mbar_init(ds_ready + 8 * s, 8);
            mbar_init(ds_free + 8 * s, 1);
        }
        for (int s = 0; s < L::STAGES; ++s) {
            mbar_init(kv_full + 8 * s, 1);
            mbar_init(kv_empty + 8 * s, 1);
            mbar_init(k_ok + 8 * s, 4);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    setup_common(tmem_slot, warp);
    if (p.chunk_rows < kTile)       // rows that no copy fills are zeros
        for (int i = threadIdx.x; i < 2 * L::TILE / 16; i += kDqThreads)
            reinterpret_cast<uint4 *>(mem + L::FIX)[i] = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
    __syncthreads();
    tc::pdl_launch_dependents();
    tc::pdl_wait();
    if (warp == 0) {
        make_list(p.tiles, items, [&](int i) {
            const int2 r = p.ranges[p.first + i];
            return make_int2(r.x / kTile, (r.y + kTile - 1) / kTile);
        });
    }
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    Share share(items, p.tiles, a.heads, p.ctas);
    Piece u;
    bool ok = true;

    // registers: 256 x 56 + 256 x 200 = 512 x 128
    if (warp < 4 || warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == 0) {                // copies
            int at = 0, last = 0;
            for (int units = 0; ok && share.next(u); ++units) {
                if (units > 0 && !(ok = tc::warp_wait(q_empty, (units - 1) & 1)))
                    break;
                tc::mbar_arrive_expect_tx_elect(q_full, 2 * L::CHUNKS * 128 * p.chunk_rows);
                for (int s = 0; s < 2; ++s)
                    for (int c = 0; c < L::CHUNKS; ++c)
                        tma_3d_elect(base + L::FIX + s * L::TILE + c * (kTile * 128), s ? &map_d : &map_q, 64 * c, u.head * group,
                                     (p.first + u.tile) * p.tokens_a_tile, q_full);
                for (int i = 0; ok && i < 2 * u.n; ++i) {
                    const int v = at + (i >> 1), s = i & 1, st = L::place(v, s), lap = L::lap(v, s);
                    if (lap > 0 && !(ok = tc::warp_wait(kv_empty + 8 * st, (lap - 1) & 1)))
                        break;
                    tc::mbar_arrive_expect_tx_elect(kv_full + 8 * st, L::TILE);
                    last = v + 1;
                    for (int c = 0; c < L::CHUNKS; ++c)
                        tma_3d_elect(base + L::RING + st * L::TILE + c * (kTile * 128), s ? &map_v : &map_k, 64 * c, u.head, (u.j0 + (i >> 1)) * kTile,
                                     kv_full + 8 * st);
                }
                at += u.n;
            }
            ok &= landed<L>(kv_full, last);
            if (lane == 0)
                p.cuts[blockIdx.x] = cut_of(share, u, at > 0, a.heads, p.ctas);
        } else if (warp == 1) {         // S and dP
            const int ksteps = (a.dim + 15) / 16;
            const uint32_t id_s = idesc_cols(kTile) | (p.negative ? kNegateA : 0u), id_p = idesc_cols(kTile);
            int job = 0;
            for (int units = 0; ok && share.next(u); ++units) {
                if (!(ok = tc::warp_wait(q_full, units & 1)))
                    break;
                for (int j = 0; ok && j < u.n; ++j, ++job) {
                    const int ks = L::place(job, 0), vs = L::place(job, 1);
                    if (!(ok = tc::warp_wait(k_ok + 8 * ks, L::lap(job, 0) & 1)))
                        break;
                    if (job > 0 && !(ok = tc::warp_wait(s_read, (job - 1) & 1)))
                        break;
                    tc::tc_fence_after();
                    for (int kk = 0; kk < ksteps; ++kk) {
                        const uint32_t off = (kk >> 2) * (kTile * 128) + (kk & 3) * 32;
                        tc::mma_bf16_elect(tmem, tc::sw128_desc(base + L::FIX + off), tc::sw128_desc(base + L::RING + ks * L::TILE + off), id_s, kk > 0);
                    }
                    tc::mma_commit_elect(s_full);
                    if (!(ok = tc::warp_wait(k_ok + 8 * vs, L::lap(job, 1) & 1)))
                        break;
                    if (job > 1 && !(ok = tc::warp_wait(ds_free + 8 * (job & 1), ((job >> 1) - 1) & 1)))
                        break;
                    tc::tc_fence_after();
                    for (int kk = 0; kk < ksteps; ++kk) {
                        const uint32_t off = (kk >> 2) * (kTile * 128) + (kk & 3) * 32;
                        tc::mma_bf16_elect(tmem + 128 + (job & 1) * 128, tc::sw128_desc(base + L::FIX + L::TILE + off),
                                           tc::sw128_desc(base + L::RING + vs * L::TILE + off), id_p, kk > 0);
                    }
                    tc::mma_commit_elect(dp_full + 8 * (job & 1));
                    tc::mma_commit_elect(kv_empty + 8 * vs);
                    if (j == u.n - 1)
                        tc::mma_commit_elect(q_empty);
                }
            }
        } else if (warp == 2) {         // dQ
            const uint32_t id_o = idesc_rows((a.dim + 15) / 16 * 16);
            int job = 0;
            for (int units = 0; ok && share.next(u); ++units) {
                if (units > 0 && !(ok = tc::warp_wait(o_free, (units - 1) & 1)))
                    break;
                for (int j = 0; ok && j < u.n; ++j, ++job) {
                    const int ks = L::place(job, 0);
                    if (!(ok = tc::warp_wait(ds_ready + 8 * (job & 1), (job >> 1) & 1)))
                        break;
                    tc::tc_fence_after();
                    for (int kk = 0; kk < kTile / 16; ++kk)
                        mma_tmem_a_elect(tmem + 384, tmem + 128 + (job & 1) * 128 + (kk >> 2) * 64 + (kk & 3) * 8,
                                         rows_desc(base + L::RING + ks * L::TILE + kk * 2048, kTile * 128), id_o, j > 0 || kk > 0);
                    tc::mma_commit_elect(kv_empty + 8 * ks);
                    tc::mma_commit_elect(ds_free + 8 * (job & 1));
                    if (j == u.n - 1)
                        tc::mma_commit_elect(done);
                }
            }
        } else if (warp >= 12) {        // looks the keys over
            int at = 0;
            while (ok && share.next(u)) {
                const int t0 = (p.first + u.tile) * p.tokens_a_tile;
                int lo = 0, hi = 0x7FFFFFFF;        // the states that every row with any sees
                for (int i = lane; i < p.tokens_a_tile && t0 + i < a.T; i += 32) {
                    const int2 see = span_of(a.spans, a.S, t0 + i, nullptr);
                    if (see.x < see.y)
                        lo = max(lo, see.x), hi = min(hi, see.y);
                }
                lo = __reduce_max_sync(0xffffffffu, lo);
                hi = __reduce_min_sync(0xffffffffu, hi);
                for (int i = 0; i < 2 * u.n; ++i) {
                    const int v = at + (i >> 1), st = L::place(v, i & 1), c0 = (u.j0 + (i >> 1)) * kTile;
                    if (!(ok = tc::warp_wait(kv_full + 8 * st, L::lap(v, i & 1) & 1)))
                        break;
                    if (!(i & 1) && (c0 < lo || c0 + kTile > hi)) {
                        const uint32_t tile = base + L::RING + st * L::TILE;
                        const int r = (warp - 12) * 32 + lane;
                        if (bad_row<DP>(tile, r)) {
                            bool seen = false;
                            for (int y = 0; y < p.tokens_a_tile && t0 + y < a.T; ++y) {
                                const int2 see = span_of(a.spans, a.S, t0 + y, nullptr);
                                seen |= see.x <= c0 + r && c0 + r < see.y;
                            }
                            if (!seen)
                                clear_row<DP>(tile, r);
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                    if (lane == 0)
                        tc::mbar_arrive(k_ok + 8 * st);
                }
                at += u.n;
            }
        }
    } else {                        // softmax: a row a thread, 64 columns a group of warps
        asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        const int half = (warp - 4) >> 2, row = threadIdx.x & 127;
        const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);
        const float scale = exponents(a.scale);
        int jobs = 0;
        for (int units = 0; ok && share.next(u); ++units) {
            const int t = (p.first + u.tile) * p.tokens_a_tile + row / group;
            const bool live = row < p.chunk_rows && t < a.T;
            const int64_t at = (int64_t)t * a.Hq + u.head * group + row % group;
            const int2 see = live ? span_of(a.spans, a.S, t, nullptr) : make_int2(0, 0);
            const float *known = info_of(p, a.heads, p.first + u.tile, u.head) + row;
            const float2 info = make_float2(known[0], known[kTile]);
            const float2 scale2 = make_float2(scale, scale), lse2 = make_float2(info.x, info.x), delta2 = make_float2(info.y, info.y);
            for (int i = 0; i < u.n; ++i, ++jobs) {
                const int c0 = (u.j0 + i) * kTile + 64 * half;
                if (!(ok = tc::warp_wait(s_full, jobs & 1)))
                    break;
                tc::tc_fence_after();
                float x[64], y[64];
                tmem_ld32(lanes + 64 * half, x);
                tmem_ld32(lanes + 64 * half + 32, x + 32);
                tmem_wait_ld();
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    tc::mbar_arrive(s_read);
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    const float2 e = fma2(make_float2(x[2 * c], x[2 * c + 1]), scale2, lse2);
                    x[2 * c] = ex2(e.x);
                    x[2 * c + 1] = ex2(e.y);
                }
                if (!(ok = tc::warp_wait(dp_full + 8 * (jobs & 1), (jobs >> 1) & 1)))
                    break;
                tc::tc_fence_after();
                const uint32_t dp = lanes + 128 + (jobs & 1) * 128 + 64 * half;
                tmem_ld32(dp, y);
                tmem_ld32(dp + 32, y + 32);
                tmem_wait_ld();
                uint32_t w[32];
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    const float2 g = mul2(make_float2(x[2 * c], x[2 * c + 1]), add2(make_float2(y[2 * c], y[2 * c + 1]), delta2));
                    x[2 * c] = g.x;
                    x[2 * c + 1] = g.y;
                }
                if (!__all_sync(0xffffffffu, see.x <= c0 && see.y >= c0 + 64)) {
                    const unsigned from = see.x - c0, n = see.y - see.x;
#pragma unroll
                    for (int c = 0; c < 64; ++c)
                        x[c] = c - from < n ? x[c] : 0.0f;
                }
#pragma unroll
                for (int c = 0; c < 32; ++c)
                    w[c] = pack2(x[2 * c], x[2 * c + 1]);
                tmem_st32(dp, w);
                tmem_wait_st();
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    tc::mbar_arrive(ds_ready + 8 * (jobs & 1));
            }
            if (!ok || !(ok = tc::warp_wait(done, units & 1)))
                break;
            tc::tc_fence_after();
            const bool whole = u.slot < 0;
            const RowStores rows(!live ? -1 : whole ? at * a.dim : (((int64_t)blockIdx.x * 2 + u.slot) * p.rows + row) * DP);
#pragma unroll
            for (int c = half * (DP / 2); c < (half + 1) * (DP / 2); c += 32) {
                if (c >= a.dim)
                    break;
                float o[32];
                tmem_ld32(lanes + 384 + c, o);
                tmem_wait_ld();
                if (whole)
                    rows.bf16(a.dq, o, c, a.dim, a.scale);
                else
                    rows.fp32(p.parts, o, c);
            }
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0)
                tc::mbar_arrive(o_free);
        }
    }
    if (!ok)
        record_timeout(a.status);
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// ---- dk, dv -----------------------------------------------------------------

// Tensor memory: S^T (P^T over it), dP^T (dS^T over it), dV, dK, 128 columns each.
template <int DP>
__global__ __launch_bounds__(kThreads, 1) void cross_dkv_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_d,
                                                                const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                                                                const __grid_constant__ CrossArgs a, const __grid_constant__ Plan p)
{
    using L = DkvLayout<DP>;
    extern __shared__ __align__(1024) unsigned char cross_mem_aligned[];
    unsigned char *mem = cross_mem_aligned;
    const uint32_t base = smem_addr(mem);
    if (base & 1023u) {         // (the first of the CTA's shared memory)
        record_timeout(a.status);
        return;
    }
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(mem + L::SLOT);
    Item *items = reinterpret_cast<Item *>(mem + L::ITEMS);
    int2 *ranges = reinterpret_cast<int2 *>(mem + L::RING);     // (while the list is made)
    const uint32_t bars = base + L::BARS;
    const uint32_t kv_full = bars, kv_empty = bars + 8, o_free = bars + 16, s_full = bars + 24, p_ready = bars + 32, dp_full = bars + 40, ds_ready = bars + 48,
                   done = bars + 56;
    const uint32_t q_full = bars + 64, q_empty = q_full + 8 * L::STAGES, q_ok = q_empty + 8 * L::STAGES;
    const int warp = warp_index(), lane = threadIdx.x & 31, group = a.Hq / a.heads;
    if (threadIdx.x == 0) {
        mbar_init(kv_full, 1);
        mbar_init(kv_empty, 1);
        mbar_init(o_free, 8);
        mbar_init(s_full, 1);
        mbar_init(p_ready, 8);
        mbar_init(dp_full, 1);
        mbar_init(ds_ready, 8);
        mbar_init(done, 1);
        for (int s = 0; s < L::STAGES; ++s) {
            mbar_init(q_full + 8 * s, 1);
            mbar_init(q_empty + 8 * s, 1);
            mbar_init(q_ok + 8 * s, 2);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    setup_common(tmem_slot, warp);
    __syncthreads();
    tc::pdl_launch_dependents();
    tc::pdl_wait();
    for (int i = threadIdx.x; i < p.tiles; i += kThreads) {       // the query tiles that see something of a tile of states
        const int c0 = (p.first + i) * kTile;
        int lo = 0x7FFFFFFF, hi = 0;
        for (int t = 0; t < p.q_tiles; ++t) {
            const int2 r = __ldg(p.ranges + t);
            if (r.x < c0 + kTile && r.y > c0)
                lo = min(lo, t), hi = t + 1;
        }
        ranges[i] = make_int2(lo, hi);
    }
    __syncthreads();
    if (warp == 0) {
        make_list(p.tiles, items, [&](int i) { return ranges[i]; });
    }
    __syncthreads();
    if (p.chunk_rows < kTile)       // rows that no copy fills are zeros
        for (int i = threadIdx.x; i < L::STAGES * L::TILE / 16; i += kThreads)
            reinterpret_cast<uint4 *>(mem + L::RING)[i] = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    Share share(items, p.tiles, a.heads, p.ctas);
    Piece u;
    bool ok = true;

    if (warp < 4) {
        if (warp == 0) {                // copies
            int at = 0, last = 0;
            for (int units = 0; ok && share.next(u); ++units) {
                if (units > 0 && !(ok = tc::warp_wait(kv_empty, (units - 1) & 1)))
                    break;
                tc::mbar_arrive_expect_tx_elect(kv_full, 2 * L::TILE);
                for (int s = 0; s < 2; ++s)
                    for (int c = 0; c < L::CHUNKS; ++c)
                        tma_3d_elect(base + L::FIX + s * L::TILE + c * (kTile * 128), s ? &map_v : &map_k, 64 * c, u.head, (p.first + u.tile) * kTile, kv_full);
                for (int i = 0; ok && i < 2 * u.n; ++i) {
                    const int v = at + (i >> 1), s = i & 1, st = L::place(v, s), lap = L::lap(v, s);
                    if (lap > 0 && !(ok = tc::warp_wait(q_empty + 8 * st, (lap - 1) & 1)))
                        break;
                    tc::mbar_arrive_expect_tx_elect(q_full + 8 * st, L::CHUNKS * 128 * p.chunk_rows);
                    last = v + 1;
                    for (int c = 0; c < L::CHUNKS; ++c)
                        tma_3d_elect(base + L::RING + st * L::TILE + c * (kTile * 128), s ? &map_d : &map_q, 64 * c, u.head * group,
                                     (u.j0 + (i >> 1)) * p.tokens_a_tile, q_full + 8 * st);
                }
                at += u.n;
            }
            ok &= landed<L>(q_full, last);
            if (lane == 0)
                p.cuts[blockIdx.x] = cut_of(share, u, at > 0, a.heads, p.ctas);
        } else if (warp == 1) {         // products
            const int ksteps = (a.dim + 15) / 16;
            const uint32_t id_s = idesc_cols(kTile) | (p.negative ? kNegateA : 0u), id_p = idesc_cols(kTile), id_o = idesc_rows(ksteps * 16);
            int jobs = 0;
            for (int units = 0; ok && share.next(u); ++units) {
                if (!(ok = tc::warp_wait(kv_full, units & 1)))
                    break;
                auto scores = [&](int v) {
                    const int qs = L::place(v, 0);
                    if (!(ok = tc::warp_wait(q_ok + 8 * qs, L::lap(v, 0) & 1)))
                        return;
                    tc::tc_fence_after();
                    for (int kk = 0; kk < ksteps; ++kk) {
                        const uint32_t off = (kk >> 2) * (kTile * 128) + (kk & 3) * 32;
                        tc::mma_bf16_elect(tmem, tc::sw128_desc(base + L::FIX + off), tc::sw128_desc(base + L::RING + qs * L::TILE + off), id_s, kk > 0);
                    }
                    tc::mma_commit_elect(s_full);
                };
                scores(jobs);
                for (int j = 0; ok && j < u.n; ++j, ++jobs) {
                    const int qs = L::place(jobs, 0), ds = L::place(jobs, 1);
                    if (!(ok = tc::warp_wait(q_ok + 8 * ds, L::lap(jobs, 1) & 1)))
                        break;
                    tc::tc_fence_after();
                    for (int kk = 0; kk < ksteps; ++kk) {
                        const uint32_t off = (kk >> 2) * (kTile * 128) + (kk & 3) * 32;
                        tc::mma_bf16_elect(tmem + 128, tc::sw128_desc(base + L::FIX + L::TILE + off), tc::sw128_desc(base + L::RING + ds * L::TILE + off), id_p,
                                           kk > 0);
                    }
                    tc::mma_commit_elect(dp_full);
                    if (j == u.n - 1)
                        tc::mma_commit_elect(kv_empty);
                    if (j == 0 && units > 0 && !(ok = tc::warp_wait(o_free, (units - 1) & 1)))
                        break;
                    if (!(ok = tc::warp_wait(p_ready, jobs & 1)))
                        break;
                    tc::tc_fence_after();
                    for (int kk = 0; kk < kTile / 16; ++kk)
                        mma_tmem_a_elect(tmem + 256, tmem + (kk >> 2) * 64 + (kk & 3) * 8, rows_desc(base + L::RING + ds * L::TILE + kk * 2048, kTile * 128), id_o,
                                         j > 0 || kk > 0);
                    tc::mma_commit_elect(q_empty + 8 * ds);
                    if (j + 1 < u.n)
                        scores(jobs + 1);
                    if (!ok || !(ok = tc::warp_wait(ds_ready, jobs & 1)))
                        break;
                    tc::tc_fence_after();
                    for (int kk = 0; kk < kTile / 16; ++kk)
                        mma_tmem_a_elect(tmem + 384, tmem + 128 + (kk >> 2) * 64 + (kk & 3) * 8, rows_desc(base + L::RING + qs * L::TILE + kk * 2048, kTile * 128),
                                         id_o, j > 0 || kk > 0);
                    tc::mma_commit_elect(q_empty + 8 * qs);
                    if (j == u.n - 1)
                        tc::mma_commit_elect(done);
                }
            }
        } else if (warp < 4) {          // looks the query rows over, and lays out what there is to know about them
            int at = 0;
            uint16_t *seen = reinterpret_cast<uint16_t *>(mem + L::SEEN);
            float *known = reinterpret_cast<float *>(mem + L::INFO);
            while (ok && share.next(u)) {
                const int c0 = (p.first + u.tile) * kTile, row = (warp - 2) * 64 + lane;
                float next[2][4];
                auto fetch = [&](int i) {
                    const float *info = info_of(p, a.heads, u.j0 + i, u.head) + row;
#pragma unroll
                    for (int y = 0; y < 2; ++y)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            next[y][e] = info[32 * y + e * kTile];
                };
                fetch(0);
                for (int i = 0; ok && i < u.n; ++i) {
                    const int v = at + i;
                    float info[2][2];
                    int lo[2], n[2];
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        info[y][0] = next[y][0], info[y][1] = next[y][1];
                        lo[y] = min(max(__float_as_int(next[y][2]) - c0, 0), kTile);
                        n[y] = max(min(__float_as_int(next[y][3]) - c0, kTile) - lo[y], 0);
                    }
                    if (i + 1 < u.n)
                        fetch(i + 1);
                    const bool all = __all_sync(0xffffffffu, n[0] == kTile && n[1] == kTile);
                    for (int s = 0; s < 2; ++s) {
                        const int st = L::place(v, s);
                        if (!(ok = tc::warp_wait(q_full + 8 * st, L::lap(v, s) & 1)))
                            break;
                        if (!all) {
#pragma unroll
                            for (int y = 0; y < 2; ++y)
                                if (n[y] == 0 && bad_row<DP>(base + L::RING + st * L::TILE, row + 32 * y))
                                    clear_row<DP>(base + L::RING + st * L::TILE, row + 32 * y);
                            fence_proxy_async_smem();
                        }
                        if (s == 0) {       // the tile before in this place is done with: its copy has begun anew
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                known[st * 2 * kTile + row + 32 * y] = info[y][0];
                                known[(st * 2 + 1) * kTile + row + 32 * y] = info[y][1];
                                seen[st * kTile + row + 32 * y] = (uint16_t)(lo[y] | n[y] << 8);
                            }
                            if (lane == 0)
                                reinterpret_cast<int *>(mem + L::FULL)[st * 2 + warp - 2] = all;
                        }
                        __syncwarp();
                        if (lane == 0)
                            tc::mbar_arrive(q_ok + 8 * st);
                    }
                }
                at += u.n;
            }
        }
    } else {                        // softmax: a state a thread, 64 query rows a group of warps
        const int half = (warp - 4) >> 2, row = threadIdx.x & 127;
        const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21), sc = lanes + 64 * half, dp = lanes + 128 + 64 * half;
        const float scale = exponents(a.scale);
        const float2 scale2 = make_float2(scale, scale);
        int jobs = 0;
        for (int units = 0; ok && share.next(u); ++units) {
            const int j = (p.first + u.tile) * kTile + row;
            for (int i = 0; i < u.n; ++i, ++jobs) {
                if (!(ok = tc::warp_wait(s_full, jobs & 1)))
                    break;
                tc::tc_fence_after();
                const int place = L::place(jobs, 0);
                const uint32_t info = base + L::INFO + (place * 2 * kTile + 64 * half) * 4, seen = base + L::SEEN + (place * kTile + 64 * half) * 2;
                const int *full = reinterpret_cast<const int *>(mem + L::FULL) + place * 2;
                const bool whole = uniform(full[half]) != 0;
                float x[64], y[64];
                uint32_t w[32];
                tmem_ld32(sc, x);
                tmem_ld32(sc + 32, x + 32);
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 64; c += 4) {
                    const uint4 l = lds_v4(info + 4 * c);
                    const float2 e = fma2(make_float2(x[c], x[c + 1]), scale2, make_float2(__uint_as_float(l.x), __uint_as_float(l.y)));
                    const float2 f = fma2(make_float2(x[c + 2], x[c + 3]), scale2, make_float2(__uint_as_float(l.z), __uint_as_float(l.w)));
                    x[c] = ex2(e.x), x[c + 1] = ex2(e.y), x[c + 2] = ex2(f.x), x[c + 3] = ex2(f.y);
                }
                if (!whole) {
#pragma unroll
                    for (int c = 0; c < 64; c += 8) {
                        const uint4 l = lds_v4(seen + 2 * c);
                        const uint32_t y[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const uint32_t part = y[e / 2] >> (16 * (e & 1));       // first, count
                            x[c + e] = row - (part & 0xFFu) < (part >> 8 & 0xFFu) ? x[c + e] : 0.0f;
                        }
                    }
                }
#pragma unroll
                for (int c = 0; c < 32; ++c)
                    w[c] = pack2(x[2 * c], x[2 * c + 1]);
                tmem_st32(sc, w);
                tmem_wait_st();
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    tc::mbar_arrive(p_ready);
                if (!(ok = tc::warp_wait(dp_full, jobs & 1)))
                    break;
                tc::tc_fence_after();
                tmem_ld32(dp, y);
                tmem_ld32(dp + 32, y + 32);
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 64; c += 4) {
                    const uint4 l = lds_v4(info + (kTile + c) * 4);
                    const float2 e = add2(make_float2(y[c], y[c + 1]), make_float2(__uint_as_float(l.x), __uint_as_float(l.y)));
                    const float2 f = add2(make_float2(y[c + 2], y[c + 3]), make_float2(__uint_as_float(l.z), __uint_as_float(l.w)));
                    y[c] = e.x, y[c + 1] = e.y, y[c + 2] = f.x, y[c + 3] = f.y;
                }
                if (!whole) {       // not 0 times what an unseen value gives
#pragma unroll
                    for (int c = 0; c < 64; ++c)
                        y[c] = x[c] == 0.0f ? 0.0f : y[c];
                }
#pragma unroll
                for (int c = 0; c < 32; ++c) {
                    const float2 g = mul2(make_float2(x[2 * c], x[2 * c + 1]), make_float2(y[2 * c], y[2 * c + 1]));
                    w[c] = pack2(g.x, g.y);
                }
                tmem_st32(dp, w);
                tmem_wait_st();
                tc::tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    tc::mbar_arrive(ds_ready);
            }
            if (!ok || !(ok = tc::warp_wait(done, units & 1)))
                break;
            tc::tc_fence_after();
            const bool whole = u.slot < 0;
            const RowStores rows(j >= a.S ? -1 : whole ? ((int64_t)j * a.heads + u.head) * a.dim : (((int64_t)blockIdx.x * 2 + u.slot) * 2 * kTile + row) * DP);
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int c = half * (DP / 2); c < (half + 1) * (DP / 2); c += 32) {
                    if (c >= a.dim)
                        break;
                    float o[32];
                    tmem_ld32(lanes + 256 + s * 128 + c, o);
                    tmem_wait_ld();
                    if (whole)
                        rows.bf16(s ? a.dk : a.dv, o, c, a.dim, s ? a.scale : 1.0f);
                    else
                        rows.fp32(p.parts + s * kTile * DP, o, c);
                }
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0)
                tc::mbar_arrive(o_free);
        }
    }
    if (!ok)
        record_timeout(a.status);
    tc::tc_fence_before();
    __syncthreads();
    if (warp == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// Adds the parts of what shares cut: a warp a row, in order.  Block (CTA, rows).  STATES: rows
// are states (dv and dk, one behind the other in a slot), else query rows.
template <int DP, bool STATES>
__global__ __launch_bounds__(kJoinWarps * 32) void cross_add_kernel(const __grid_constant__ CrossArgs a, const __grid_constant__ Plan p)
{
    constexpr int V = DP / 32;
    tc::pdl_launch_dependents();
    tc::pdl_wait();
    const Cut cut = p.cuts[blockIdx.x];
    if (cut.c1 < 0)
        return;
    const int tile = p.first + cut.tile, group = a.Hq / a.heads, warp = warp_index(), lane = threadIdx.x & 31, n = cut.c1 - (int)blockIdx.x + 1;
    const int slot_rows = STATES ? 2 * kTile : p.rows;
    const int r = blockIdx.y * kJoinWarps + warp;
    if (r >= slot_rows)
        return;
    const int row = STATES ? r % kTile : r;
    __nv_bfloat16 *out;
    float by = a.scale;
    if (STATES) {
        const int64_t j = (int64_t)tile * kTile + row;
        if (j >= a.S)
            return;
        out = (r < kTile ? a.dv : a.dk) + (j * a.heads + cut.head) * a.dim;
        by = r < kTile ? 1.0f : a.scale;
    } else {
        const int64_t t = (int64_t)tile * p.tokens_a_tile + row / group;
        if (row >= p.chunk_rows || t >= a.T)
            return;
        out = a.dq + (t * a.Hq + cut.head * group + row % group) * a.dim;
    }
    float acc[V] = {};
#pragma unroll 8
    for (int i = 0; i < n; ++i) {
        float part[V];
        Columns<DP>::get(p.parts + (((int64_t)(blockIdx.x + i) * 2 + (i == 0 ? cut.slot : 0)) * slot_rows + r) * DP, part);
#pragma unroll
        for (int v = 0; v < V; ++v)
            acc[v] += part[v];
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
        acc[v] *= by;
    if (lane * V < a.dim)
        Columns<DP>::put(out, acc);
}

// Where the workspace's parts are (the pointers as offsets), and how long it is.
Plan plan_of(int64_t T, int64_t Hq, int64_t heads, int DP, size_t *bytes)
{
    Plan p;
    const int group = (int)(Hq / heads);
    p.tokens_a_tile = kTile / group;
    p.chunk_rows = p.tokens_a_tile * group;
    p.q_tiles = (int)((T + p.tokens_a_tile - 1) / p.tokens_a_tile);
    p.rows = T * group < kTile ? (int)(T * group) : kTile;
    p.ctas = device_sm_count();
    p.first = p.tiles = p.negative = 0;
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t from = at;
        at += (n + 15) / 16 * 16;
        return from;
    };
    p.info = reinterpret_cast<float *>(take((size_t)p.q_tiles * heads * 4 * kTile * sizeof(float)));
    p.ranges = reinterpret_cast<int2 *>(take((size_t)p.q_tiles * sizeof(int2)));
    p.parts = reinterpret_cast<float *>(take((size_t)p.ctas * 2 * 2 * kTile * DP * sizeof(float)));
    p.cuts = reinterpret_cast<Cut *>(take(p.ctas * sizeof(Cut)));
    *bytes = at;
    return p;
}

template <int DP>
cudaError_t launch(const CrossArgs &a, cudaStream_t stream)
{
    using Lq = DqLayout<DP>;
    using L = DkvLayout<DP>;
    static_assert(Lq::BYTES <= 232448 && L::BYTES <= 232448 && L::BARS % 8 == 0 && L::INFO % 16 == 0, "shared memory");
    size_t bytes;
    Plan p = plan_of(a.T, a.Hq, a.heads, DP, &bytes);
    char *ws = static_cast<char *>(a.ws);
    p.info = reinterpret_cast<float *>(ws + reinterpret_cast<size_t>(p.info));
    p.ranges = reinterpret_cast<int2 *>(ws + reinterpret_cast<size_t>(p.ranges));
    p.parts = reinterpret_cast<float *>(ws + reinterpret_cast<size_t>(p.parts));
    p.cuts = reinterpret_cast<Cut *>(ws + reinterpret_cast<size_t>(p.cuts));
    p.negative = a.scale < 0.0f;
    CUtensorMap mq, md, mk, mv;
    cudaError_t e = row_map(&mq, a.q, a.T, a.Hq, a.dim, a.qs, a.Hq / a.heads, p.tokens_a_tile);
    if (e == cudaSuccess)
        e = row_map(&md, a.dout, a.T, a.Hq, a.dim, a.ds, a.Hq / a.heads, p.tokens_a_tile);
    if (e == cudaSuccess)
        e = row_map(&mk, a.k, a.S, a.heads, a.dim, a.ks, 1, kTile);
    if (e == cudaSuccess)
        e = row_map(&mv, a.v, a.S, a.heads, a.dim, a.vs, 1, kTile);
    static std::atomic<unsigned long long> allowed_q, allowed_kv;
    if (e == cudaSuccess)
        e = tc::allow_smem(cross_dq_kernel<DP>, Lq::BYTES, allowed_q);
    if (e == cudaSuccess)
        e = tc::allow_smem(cross_dkv_kernel<DP>, L::BYTES, allowed_kv);
    if (e == cudaSuccess)
        e = tc::launch_pdl(cross_ready_kernel, dim3(p.q_tiles, a.heads, kTile / kReadyRows), dim3(256), 0, stream, a, p);
    if (e == cudaSuccess && (a.spans || a.S <= kFew))
        e = tc::launch_pdl(cross_few_kernel<DP>, dim3(p.q_tiles, a.heads, kTile / (16 * kFewWarps)), dim3(kFewWarps * 32), 0, stream, a, p);
    const int tiles = (a.S + kTile - 1) / kTile, most_q = most_tiles(a.heads, tiles, kMostTiles), most_kv = most_tiles(a.heads, p.q_tiles, kMostTiles);
    for (p.first = 0; e == cudaSuccess && p.first < p.q_tiles; p.first += most_q) {
        p.tiles = p.q_tiles - p.first < most_q ? p.q_tiles - p.first : most_q;
        e = tc::launch_pdl(cross_dq_kernel<DP>, dim3(p.ctas), dim3(kDqThreads), Lq::BYTES, stream, mq, md, mk, mv, a, p);
        if (e == cudaSuccess)
            e = tc::launch_pdl(cross_add_kernel<DP, false>, dim3(p.ctas, (p.rows + kJoinWarps - 1) / kJoinWarps), dim3(kJoinWarps * 32), 0, stream, a, p);
    }
    for (p.first = 0; e == cudaSuccess && p.first < tiles; p.first += most_kv) {
        p.tiles = tiles - p.first < most_kv ? tiles - p.first : most_kv;
        e = tc::launch_pdl(cross_dkv_kernel<DP>, dim3(p.ctas), dim3(kThreads), L::BYTES, stream, mq, md, mk, mv, a, p);
        if (e == cudaSuccess)
            e = tc::launch_pdl(cross_add_kernel<DP, true>, dim3(p.ctas, 2 * kTile / kJoinWarps), dim3(kJoinWarps * 32), 0, stream, a, p);
    }
    return e;
}

}  // namespace

size_t cross_attention_backward_workspace(int64_t T, int64_t, int64_t Hq, int64_t heads, int64_t dim)
{
    size_t bytes;
    plan_of(T, Hq, heads, dim > 64 ? 128 : 64, &bytes);
    return bytes;
}

cudaError_t launch_cross_attention_backward(const CrossArgs &a, cudaStream_t stream)
{
    if (a.S == 0) {     // (and tokens: their gradients are zero)
        CrossArgs zeros = a;
        zeros.out = a.dq;
        zeros.lse = nullptr;
        return launch_cross_nothing(zeros, stream);
    }
    return a.dim > 64 ? launch<128>(a, stream) : launch<64>(a, stream);
}

}  // namespace s3d8

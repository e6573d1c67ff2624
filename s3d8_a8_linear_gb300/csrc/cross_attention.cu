// Attention of text tokens to an encoder's states, each token over a span of them
// (s3d8_cross_attention):
//
//   s_j = scale q . k_j (a <= j < b), out = sum softmax(s)_j v_j, lse = log sum exp s_j
//
// Tiles of 128 query rows: the query heads of a key/value head stand behind one another,
// token by token, so that they share its keys and values, and one token of 4 heads is four
// rows.  The states pass in tiles of 128.  S = Q K^T and O += P V run on the tensor cores
// (tcgen05, sums in tensor memory); the softmax's weights P go from registers into tensor
// memory as the second product's A operand, over the scores they come from.  A CTA an SM:
// one warp copies (bulk tensor copies into a ring), two issue the products, two groups of
// four warps have a row a thread each, and four warps look the values over (below).
//
// Two chains of score, softmax and product run in turn, so that the tensor cores work on
// one while the other is in its softmax: two query tiles over the same states where their
// spans are nearly the same (a prompt), or else one query tile whose states alternate (a
// decode step: every token its own image).  Every CTA looks over all spans, makes the same
// list of work from them, and takes an equal share of its state tiles, wherever that begins
// or ends; what a share cuts leaves fp32 sums, which a second kernel joins in order.
//
// Each chain has its own warp that issues products (one warp for both: 781 us where two take
// 720, 4 x 2047 tokens of 32 / 8 heads of 128 to 4 x 6404 states; two warps that share one
// chain's softmax rows: 1439 at that stage).  Its rate there is 1190 TFLOP/s, the tensor pipe
// busy half the time: a chain's scores, softmax and product follow one another, and two
// chains do not fill the gaps (three would need more tensor memory); timing copies without
// the exponentials, or with half of each copy, ran no faster.
//
// An item's states are those that some of its tokens see, in runs: a batch of single tokens
// jumps over the padding behind each image (48 tokens, 48 images of 0 .. 6404 of 6404 states:
// 119 us, 5.3 TB/s of what is seen; 197 when every tile between the first and the last was
// copied).
//
// The running maximum moves only where a tile exceeds it by 2^8 (rescaling O costs a round
// through tensor memory); sums are fp32 throughout.  The weights are rounded to bf16, the
// values' type, on their way into the product: 2^-8 of each, which averages to about the
// rounding of the output; 16 more bits would double the product.
//
// A weight of zero does not silence an infinity or NaN among the values: 0 * inf is NaN.
// Where some row of the query tiles does not see all of a state tile, the four other warps
// look at its values, replace what is not finite by zeros, and note which rows do see it;
// those rows get the infinity or NaN in that column at the end.
#include "cross_tiles.cuh"

namespace s3d8 {

namespace {

using namespace cross;

constexpr int kThreads = 512;
constexpr int kMostTiles = 512;         // query tiles of a launch
constexpr int kRuns = 1536;             // runs of states of all items, and their ends
constexpr int kJoinWarps = 8;

constexpr int kNoTile = 0xFFFF;         // of the two query tiles of a piece, low and high half of its `tile`

struct Plan {
    int tokens_a_tile, tiles, rows;     // rows: of a slot of partial sums
    int chunk_rows;                     // query rows that a copy fills
    int ctas;
    float *parts, *tops;                // [ctas][2][rows][DP], [ctas][2][rows][2]
    Cut *cuts;                          // [ctas]: what there is to join
    int negative;                       // scale < 0: the scores are those of -Q
};

template <int DP>
struct Layout {
    static constexpr int CHUNKS = DP / 64;
    static constexpr int TILE = kTile * DP * 2;             // bytes of a tile of Q, K or V
    static constexpr int STAGES = DP == 128 ? 4 : 8;
    static constexpr int Q = 0, KV = 2 * TILE, ITEMS = KV + STAGES * TILE;
    static constexpr int RUNS = ITEMS + ((kMostTiles + 1) * (int)sizeof(Item) + 15) / 16 * 16;   // at first the query tiles' ranges
    static constexpr int BAD = RUNS + kRuns * (int)sizeof(Run);     // [2][128][8]: columns of +inf, of -inf
    static constexpr int TOPS = BAD + 2 * 128 * 32;         // [2][128] maximum and sum of the second chain
    static constexpr int BARS = TOPS + 2 * 128 * 8;
    static constexpr int PLACES = BARS + 384;               // [STAGES]: the first state of the visits whose copies were issued last
    static constexpr int BYTES = 1024 + BARS + 512;
};

// A piece of a CTA's share: query tile a (and b, with the same states).
struct Unit : Piece {
    int ta, tb;
    bool pair;
};

__device__ __forceinline__ bool next_unit(Share &share, Unit &u)
{
    if (!share.next(u))
        return false;
    u.ta = u.tile & 0xFFFF;
    u.tb = u.tile >> 16 & 0xFFFF;
    u.pair = u.tb != kNoTile;
    return true;
}

// The list of items: for each pair of query tiles whether they go together.  One warp.
__device__ __forceinline__ int make_items(const int2 *ranges, int tiles, Item *items)
{
    const int lane = threadIdx.x & 31;
    int count = 0;
    auto span = [&](int t, int &j0, int &j1) {      // state tiles; one (of which nothing is seen) for an empty span
        const int2 r = ranges[t];
        j0 = r.x < r.y ? r.x / kTile : 0;
        j1 = r.x < r.y ? (r.y + kTile - 1) / kTile : 1;
    };
    for (int base = 0; base < (tiles + 1) / 2; base += 32) {
        const int a = 2 * (base + lane), b = a + 1;
        int n = 0, a0 = 0, a1 = 0, b0 = 0, b1 = 0;      // (the gaps of their spans counted in)
        bool pair = false;
        if (a < tiles) {
            n = 1;
            span(a, a0, a1);
            if (b < tiles) {
                span(b, b0, b1);
                // Together, both chains pass the states of either and each tile of states is copied
                // once; apart, each passes its own.  So they go together while that is at most a
                // quarter more visits than apart (prompts: a pair's visit takes 4060 clocks, one
                // of two alternating tiles half of that).
                const int u0 = min(a0, b0), u1 = max(a1, b1);
                pair = 8 * (u1 - u0) <= 5 * (a1 - a0 + b1 - b0) + 8;
                n = pair ? 1 : 2;
            }
        }
        int c = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int pc = __shfl_up_sync(0xffffffffu, c, o);
            if (lane >= o)
                c += pc;
        }
        if (n)
            items[count + c - n] = {a | (pair ? b : kNoTile) << 16, 0, 0};
        if (n == 2)
            items[count + c - 1] = {b | kNoTile << 16, 0, 0};
        count += __shfl_sync(0xffffffffu, c, 31);
    }
    return count;
}

// From the items' sizes (in `begin`) what lies in front of each.  One warp.
__device__ __forceinline__ void add_up(Item *items, int n)
{
    const int lane = threadIdx.x & 31;
    int sum = 0;
    for (int base = 0; base < n; base += 32) {
        const int size = base + lane < n ? items[base + lane].begin : 0;
        int s = size;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int ps = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o)
                s += ps;
        }
        if (base + lane < n)
            items[base + lane].begin = sum + s - size;
        sum += __shfl_sync(0xffffffffu, s, 31);
    }
    if (lane == 0)
        items[n] = {0, 0, sum};
}

// Scores of columns outside from .. from + n - 1: -inf.
__device__ __forceinline__ void hide(float (&x)[64], unsigned from, unsigned n)
{
#pragma unroll
    for (int c = 0; c < 64; ++c)
        x[c] = c - from < n ? x[c] : -INFINITY;
}

// A stage of the ring is free when both chains have used it, or the only one that does.
__device__ __forceinline__ void release(uint32_t empty, bool pair)
{
    tc::mma_commit_elect(empty);
    if (!pair)
        tc::mma_commit_elect(empty);
}

// Looks over a state tile's values (in shared memory at v): a row a thread at a time.
// What is not finite becomes zero, and is noted for the rows that see its state.
template <int DP>
__device__ __forceinline__ void look_over(uint32_t v, int c0, const CrossArgs &a, const Plan &p, const Unit &u, uint32_t *bad, int *any)
{
    {
        const int r = threadIdx.x & 127;
        uint32_t top = 0;
#pragma unroll 8
        for (int c = 0; c < DP / 8; ++c) {
            const uint4 x = lds_v4(chunk_at(v, r, c));
            top = absmax_bf16x8(x, top);
        }
        if (finite2(top))
            return;
        uint32_t plus[4] = {0, 0, 0, 0}, minus[4] = {0, 0, 0, 0};       // NaN: both
        for (int c = 0; c < DP / 8; ++c) {
            const uint32_t at = chunk_at(v, r, c);
            for (int e = 0; e < 8; ++e) {
                uint16_t x;
                asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(at + 2 * e));
                if ((x & 0x7FFF) < 0x7F80)
                    continue;
                asm volatile("st.shared.u16 [%0], %1;" ::"r"(at + 2 * e), "h"((uint16_t)0) : "memory");
                const int d = 8 * c + e;
                const uint32_t bit = 1u << (d & 31);
                if (x != 0xFF80)
                    plus[d >> 5] |= bit;
                if (x != 0x7F80)
                    minus[d >> 5] |= bit;
            }
        }
        const int j = c0 + r;
        if (j >= a.S)
            return;
        for (int s = 0; s < (u.pair ? 2 : 1); ++s)
            for (int i = 0; i < p.tokens_a_tile; ++i) {
                const int t = (s ? u.tb : u.ta) * p.tokens_a_tile + i;
                if (t >= a.T)
                    break;
                const int2 see = span_of(a.spans, a.S, t, nullptr);
                if (j < see.x || j >= see.y)
                    continue;
                const int group = a.Hq / a.heads;
                for (int g = 0; g < group; ++g)
                    for (int w = 0; w < 4; ++w) {
                        atomicOr(bad + (s * 128 + i * group + g) * 8 + w, plus[w]);
                        atomicOr(bad + (s * 128 + i * group + g) * 8 + 4 + w, minus[w]);
                    }
                atomicExch(any + s, 1);
            }
    }
}

template <int DP>
__global__ __launch_bounds__(kThreads, 1) void cross_forward_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                                                                    const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CrossArgs a,
                                                                    const __grid_constant__ Plan p)
{
    using L = Layout<DP>;
    extern __shared__ unsigned char cross_mem[];
    __shared__ uint32_t tmem_slot;
    __shared__ int item_count, bad_any[2];
    const uint32_t base = (smem_addr(cross_mem) + 1023u) & ~1023u;
    unsigned char *mem = cross_mem + (base - smem_addr(cross_mem));
    Item *items = reinterpret_cast<Item *>(mem + L::ITEMS);
    int2 *ranges = reinterpret_cast<int2 *>(mem + L::RUNS);
    Run *runs = reinterpret_cast<Run *>(mem + L::RUNS);
    uint32_t *bad = reinterpret_cast<uint32_t *>(mem + L::BAD);
    float2 *tops = reinterpret_cast<float2 *>(mem + L::TOPS);
    volatile int *places = reinterpret_cast<int *>(mem + L::PLACES);
    const uint32_t bars = base + L::BARS;
    const uint32_t q_full = bars, q_empty = bars + 8, o_free = bars + 16, s_full = bars + 24, p_ready = bars + 40, pv_done = bars + 56, p_half = bars + 72;
    const uint32_t kv_full = bars + 88, kv_empty = kv_full + 8 * L::STAGES, v_ok = kv_empty + 8 * L::STAGES;
    const int warp = warp_index(), lane = threadIdx.x & 31, group = a.Hq / a.heads;

    if (warp == 0 && lane == 0) {
        mbar_init(q_full, 1);
        mbar_init(q_empty, 2);
        mbar_init(o_free, 8);
        for (int s = 0; s < 2; ++s) {
            mbar_init(s_full + 8 * s, 1);
            mbar_init(p_half + 8 * s, 4);
            mbar_init(p_ready + 8 * s, 4);
            mbar_init(pv_done + 8 * s, 1);
        }
        for (int s = 0; s < L::STAGES; ++s) {
            mbar_init(kv_full + 8 * s, 1);
            mbar_init(kv_empty + 8 * s, 2);
            mbar_init(v_ok + 8 * s, 4);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&tmem_slot)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (threadIdx.x < 2)
        bad_any[threadIdx.x] = 0;
    for (int i = threadIdx.x; i < 2 * 128 * 8; i += kThreads)
        bad[i] = 0;
    if (p.chunk_rows < kTile)       // rows that no copy fills are zeros
        for (int i = threadIdx.x; i < 2 * L::TILE / 16; i += kThreads)
            reinterpret_cast<uint4 *>(mem + L::Q)[i] = make_uint4(0u, 0u, 0u, 0u);
    for (int i = threadIdx.x; i < p.tiles; i += kThreads)
        ranges[i] = make_int2(0x7FFFFFFF, 0);
    fence_proxy_async_smem();
    __syncthreads();
    tc::pdl_launch_dependents();
    tc::pdl_wait();
    int *record = blockIdx.x == 0 ? a.status : nullptr;
    int n_items = 1;
    if (p.tiles > 1) {
        for (int t = threadIdx.x; t < a.T; t += kThreads) {
            const int2 s = span_of(a.spans, a.S, t, record);
            if (s.x < s.y) {
                atomicMin(&ranges[t / p.tokens_a_tile].x, s.x);
                atomicMax(&ranges[t / p.tokens_a_tile].y, s.y);
            }
        }
        record = nullptr;
        __syncthreads();
        if (warp == 0) {
            const int n = make_items(ranges, p.tiles, items);
            if (lane == 0)
                item_count = n;
        }
        __syncthreads();
        n_items = uniform(item_count);
    } else if (threadIdx.x == 0) {
        items[0] = {kNoTile << 16, 0, 0};
    }
    __syncwarp();
    const int run_step = kRuns / n_items;
    for (int i = warp; i < n_items; i += kThreads / 32) {
        const int t0 = (items[i].tile & 0xFFFF) * p.tokens_a_tile;
        const int n = min(a.T - t0, (items[i].tile >> 16 & 0xFFFF) != kNoTile ? 2 * p.tokens_a_tile : p.tokens_a_tile);
        Run *to = runs + i * run_step;
        const int size = n <= 32 ? make_runs<1>(a.spans, a.S, t0, n, run_step - 1, to, record)
                                 : make_runs<8>(a.spans, a.S, t0, n, run_step - 1, to, record);
        if (lane == 0)
            items[i].begin = size;
    }
    if (p.tiles > 1)
        __syncthreads();
    __syncwarp();
    if (warp == 0)
        add_up(items, n_items);
    tc::tc_fence_before();
    __syncthreads();
    tc::tc_fence_after();
    const uint32_t tmem = tmem_slot;
    Share share(items, n_items, a.heads, p.ctas);
    Unit u;
    bool ok = true;

    // registers: 128 x (56 + 48) + 256 x 200 = 512 x 126
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == 0) {                // copies
            int at = 0;                 // tiles of K and V so far
            for (int units = 0; ok && next_unit(share, u); ++units) {
                if (units > 0 && !(ok = tc::warp_wait(q_empty, (units - 1) & 1)))
                    break;
                tc::mbar_arrive_expect_tx_elect(q_full, (u.pair ? 2 : 1) * L::CHUNKS * 128 * p.chunk_rows);
                for (int s = 0; s < (u.pair ? 2 : 1); ++s)
                    for (int c = 0; c < L::CHUNKS; ++c)
                        tma_3d_elect(base + L::Q + s * L::TILE + c * (kTile * 128), &map_q, 64 * c, u.head * group, (s ? u.tb : u.ta) * p.tokens_a_tile, q_full);
                Walk walk(runs + u.item * run_step, u.j0);
                int j = 0;
                for (int i = 0; ok && i < 2 * u.n; ++i, ++at) {
                    const int st = at % L::STAGES;
                    if (at >= L::STAGES && !(ok = tc::warp_wait(kv_empty + 8 * st, (at / L::STAGES - 1) & 1)))
                        break;
                    if (!(i & 1)) {     // (the values before these took the place of those half a ring back, which were used)
                        j = walk(i >> 1);
                        if (lane == 0)
                            places[(at >> 1) % L::STAGES] = j * kTile;
                        __syncwarp();
                    }
                    tc::mbar_arrive_expect_tx_elect(kv_full + 8 * st, L::TILE);
                    for (int c = 0; c < L::CHUNKS; ++c)
                        tma_3d_elect(base + L::KV + st * L::TILE + c * (kTile * 128), i & 1 ? &map_v : &map_k, 64 * c, u.head, j * kTile,
                                     kv_full + 8 * st);
                }
            }
            // not before the last copies have landed
            for (int i = at - L::STAGES < 0 ? 0 : at - L::STAGES; i < at; ++i)
                ok &= tc::warp_wait(kv_full + 8 * (i % L::STAGES), (i / L::STAGES) & 1);
            if (lane == 0)
                p.cuts[blockIdx.x] = cut_of(share, u, at > 0, a.heads, p.ctas);
        } else if (warp < 3) {          // products of a chain
            const int s = warp - 1, ksteps = (a.dim + 15) / 16;
            const uint32_t id_s = idesc_cols(kTile) | (p.negative ? kNegateA : 0u), id_o = idesc_rows(ksteps * 16);
            int at = 0, jobs = 0;       // tiles of K and V, and this chain's products, so far
            for (int units = 0; ok && next_unit(share, u); ++units) {
                const int mine = u.pair ? u.n : (u.n + 1 - s) / 2;
                const uint32_t q = base + L::Q + (u.pair ? s * L::TILE : 0);
                if (!(ok = tc::warp_wait(q_full, units & 1)))
                    break;
                for (int i = 0; ok && i < mine; ++i, ++jobs) {
                    const int k = at + 2 * (u.pair ? i : 2 * i + s), ks = k % L::STAGES, v = k + 1, vs = v % L::STAGES;
                    if (!(ok = tc::warp_wait(kv_full + 8 * ks, (k / L::STAGES) & 1)))
                        break;
                    tc::tc_fence_after();
                    const uint32_t kt = base + L::KV + ks * L::TILE, vt = base + L::KV + vs * L::TILE;
                    for (int kk = 0; kk < ksteps; ++kk) {
                        const uint32_t off = (kk >> 2) * (kTile * 128) + (kk & 3) * 32;
                        tc::mma_bf16_elect(tmem + s * 128, tc::sw128_desc(q + off), tc::sw128_desc(kt + off), id_s, kk > 0);
                    }
                    tc::mma_commit_elect(s_full + 8 * s);
                    release(kv_empty + 8 * ks, u.pair);
                    if (i == mine - 1)
                        tc::mma_commit_elect(q_empty);
                    if (!(ok = tc::warp_wait(v_ok + 8 * vs, (v / L::STAGES) & 1)))
                        break;
                    for (int half = 1; ok && half >= 0; --half) {     // the second half of the states is ready first
                        if (!(ok = tc::warp_wait((half ? p_half : p_ready) + 8 * s, jobs & 1)))
                            break;
                        tc::tc_fence_after();
                        for (int kk = 4 * half; kk < 4 * half + 4; ++kk)
                            mma_tmem_a_elect(tmem + 256 + s * 128, tmem + s * 128 + half * 64 + (kk & 3) * 8, rows_desc(vt + kk * 2048, kTile * 128), id_o,
                                             i > 0 || kk != 4);
                    }
                    tc::mma_commit_elect(pv_done + 8 * s);
                    release(kv_empty + 8 * vs, u.pair);
                }
                if (mine == 0 && lane == 0)     // (one state tile: the second chain has none)
                    tc::mbar_arrive(q_empty);
                at += 2 * u.n;
                // The last values, where they were the first chain's: a wait for a stage's next
                // phase means that one only once the phase before is known to be over.
                if (ok && s == 1 && !u.pair && u.n % 2 == 1)
                    ok = tc::warp_wait(v_ok + 8 * ((at - 1) % L::STAGES), ((at - 1) / L::STAGES) & 1);
            }
        }
    } else if (warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
        {                               // looks the values over
            int at = 0;
            for (int units = 0; ok && next_unit(share, u); ++units) {
                // the states that every row with any sees
                int lo = 0, hi = 0x7FFFFFFF;
                for (int s = 0; s < (u.pair ? 2 : 1); ++s)
                    for (int i = lane; i < p.tokens_a_tile; i += 32) {
                        const int t = (s ? u.tb : u.ta) * p.tokens_a_tile + i;
                        const int2 see = t < a.T ? span_of(a.spans, a.S, t, nullptr) : make_int2(0, 0);
                        if (see.x < see.y) {
                            lo = max(lo, see.x);
                            hi = min(hi, see.y);
                        }
                    }
                lo = __reduce_max_sync(0xffffffffu, lo);
                hi = __reduce_min_sync(0xffffffffu, hi);
                if (units > 0 && !(ok = tc::warp_wait(o_free, (units - 1) & 1)))   // the notes of the piece before are read
                    break;
                for (int i = 0; i < u.n; ++i) {
                    const int v = at + 2 * i + 1, st = v % L::STAGES;
                    if (!(ok = tc::warp_wait(kv_full + 8 * st, (v / L::STAGES) & 1)))
                        break;
                    const int c0 = uniform((int)places[(v >> 1) % L::STAGES]);
                    if (c0 < lo || c0 + kTile > hi) {
                        look_over<DP>(base + L::KV + st * L::TILE, c0, a, p, u, bad, bad_any);
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                    if (lane == 0)
                        tc::mbar_arrive(v_ok + 8 * st);
                }
                at += 2 * u.n;
            }
        }
    } else {                        // softmax, a row a thread
        asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        const int s = (warp - 4) >> 2, row = threadIdx.x & 127;
        const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21), sc = lanes + s * 128, oc = lanes + 256 + s * 128;
        const float scale = exponents(a.scale);
        int jobs = 0, visits = 0;       // of this chain, and of both before this piece
        int joins = 0;                  // of the two chains, so far
        while (next_unit(share, u)) {
            const int tile = u.pair && s ? u.tb : u.ta, t = tile * p.tokens_a_tile + row / group;
            const bool live = row < p.chunk_rows && t < a.T;
            const int2 see = live ? span_of(a.spans, a.S, t, nullptr) : make_int2(0, 0);
            const int mine = u.pair ? u.n : (u.n + 1 - s) / 2;
            float top = -INFINITY, sum = 0.0f;      // in units of base-2 exponents
            for (int i = 0; i < mine; ++i, ++jobs) {
                wait_on(ok, s_full + 8 * s, jobs & 1);
                const int c0 = places[(visits + (u.pair ? i : 2 * i + s)) % L::STAGES];
                float x[64], m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                const bool all = __all_sync(0xffffffffu, see.x <= c0 && see.y >= c0 + kTile);
                const unsigned from = see.x - c0, n = see.y - see.x;
                // the second half stays in registers; the first one is read twice
#pragma unroll
                for (int b = 0; b < kTile; b += 64) {
                    tmem_ld32(sc + b, x);
                    tmem_ld32(sc + b + 32, x + 32);
                    tmem_wait_ld();
                    if (!all)
                        hide(x, from - b, n);
#pragma unroll
                    for (int c = 0; c < 64; c += 4)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            m[e] = fmaxf(m[e], x[c + e]);
                }
                const float peak = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])) * scale;
                const bool rise = peak > top + 8.0f || top == -INFINITY;
                if (__any_sync(0xffffffffu, rise && peak > -INFINITY)) {
                    const float next = rise ? peak : top, turn = rise ? ex2(top - (next == -INFINITY ? 0.0f : next)) : 1.0f;
                    top = next;
                    sum *= turn;
                    if (i > 0) {
                        wait_on(ok, pv_done + 8 * s, (jobs - 1) & 1);
#pragma unroll
                        for (int c = 0; c < DP; c += 32) {
                            float o[32];
                            uint32_t b[32];
                            tmem_ld32(oc + c, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                b[e] = __float_as_uint(o[e] * turn);
                            tmem_st32(oc + c, b);
                        }
                    }
                }
                const float shift = top == -INFINITY ? 0.0f : -top;
                const float2 scale2 = make_float2(scale, scale), shift2 = make_float2(shift, shift);
                float2 part[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
#pragma unroll
                for (int b = 64; b >= 0; b -= 64) {     // each half of P over its half of the scores
                    if (b == 0) {
                        tmem_ld32(sc, x);
                        tmem_ld32(sc + 32, x + 32);
                        tmem_wait_ld();
                        if (!all)
                            hide(x, from, n);
                    }
                    uint32_t w[32];
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        const float2 e = fma2(make_float2(x[2 * c], x[2 * c + 1]), scale2, shift2), y = make_float2(ex2(e.x), ex2(e.y));
                        part[c & 1] = add2(part[c & 1], y);
                        w[c] = pack2(y.x, y.y);
                    }
                    tmem_st32(sc + b, w);
                    tmem_wait_st();
                    tc::tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        tc::mbar_arrive((b ? p_half : p_ready) + 8 * s);
                }
                part[0] = add2(part[0], part[1]);
                sum += part[0].x + part[0].y;
            }
            if (mine > 0)
                wait_on(ok, pv_done + 8 * s, (jobs - 1) & 1);
            // One query tile: the first group joins the two chains.  The second one may be through
            // with the next piece before that has read: in a piece of one visit it has nothing to
            // do, and so nothing to wait for.  It writes to the other half then, and to this one
            // again behind the next join's barrier, where the first group arrives after it has read.
            float turn[2] = {1.0f, 0.0f};
            if (!u.pair) {
                float2 *const at = tops + (joins++ & 1) * 128 + row;
                if (s == 1)
                    *at = make_float2(top, sum);
                tc::tc_fence_before();
                asm volatile("bar.sync 1, 256;" ::: "memory");
                tc::tc_fence_after();
                if (s == 0) {
                    const float2 other = *at;
                    const float next = fmaxf(top, other.x), from = next == -INFINITY ? 0.0f : next;
                    turn[0] = ex2(top - from);
                    turn[1] = ex2(other.x - from);
                    sum = sum * turn[0] + other.y * turn[1];
                    top = next;
                }
            }
            if (u.pair || s == 0) {
                const bool whole = u.slot < 0;
                const float by = whole ? (sum != 0.0f ? 1.0f / sum : 0.0f) : 1.0f;
                const bool both = !u.pair && u.n > 1, noted = uniform(bad_any[u.pair ? s : 0]);
                const uint32_t *note = bad + ((u.pair ? s : 0) * 128 + row) * 8;
                __nv_bfloat16 *out = a.out + ((int64_t)t * a.Hq + u.head * group + row % group) * a.dim;
                const int64_t slot = ((int64_t)blockIdx.x * 2 + u.slot) * p.rows + (u.pair ? s * 128 : 0) + row;
                const bool some = see.x < see.y;
#pragma unroll
                for (int c = 0; c < DP; c += 32) {
                    if (c >= a.dim)
                        break;
                    float o[32];
                    tmem_ld32(oc + c, o);
                    tmem_wait_ld();
                    if (!u.pair) {
                        float o2[32];
                        if (both) {
                            tmem_ld32(oc + 128 + c, o2);
                            tmem_wait_ld();
                        }
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            o[e] = o[e] * turn[0] + (both ? o2[e] * turn[1] : 0.0f);
                    }
                    if (noted) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            if (note[c / 32] >> e & 1)
                                o[e] += INFINITY;
                            if (note[4 + c / 32] >> e & 1)
                                o[e] -= INFINITY;
                        }
                    }
                    if (!live)
                        continue;
                    if (whole) {
#pragma unroll
                        for (int e = 0; e < 32; e += 8)
                            if (c + e < a.dim) {
                                uint32_t r[4];
#pragma unroll
                                for (int y = 0; y < 4; ++y)
                                    r[y] = some ? pack2(o[e + 2 * y] * by, o[e + 2 * y + 1] * by) : 0u;
                                *reinterpret_cast<uint4 *>(out + c + e) = make_uint4(r[0], r[1], r[2], r[3]);
                            }
                    } else if (some) {
                        float4 *part = reinterpret_cast<float4 *>(p.parts + slot * DP + c);
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            part[e / 4] = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
                    }
                }
                if (live) {
                    if (!whole)
                        reinterpret_cast<float2 *>(p.tops)[slot] = make_float2(some ? top : -INFINITY, some ? sum : 0.0f);
                    else if (a.lse)
                        a.lse[(int64_t)t * a.Hq + u.head * group + row % group] = some ? (top + __log2f(sum)) * kLn2 : -INFINITY;
                }
                if (noted) {        // used: gone, before the next piece
                    for (int w = 0; w < 8; ++w)
                        bad[((u.pair ? s : 0) * 128 + row) * 8 + w] = 0;
                    if (s == 0)
                        asm volatile("bar.sync 2, 128;" ::: "memory");
                    else
                        asm volatile("bar.sync 3, 128;" ::: "memory");
                    if (row == 0)
                        bad_any[u.pair ? s : 0] = 0;
                }
            }
            visits += u.n;
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

// Joins the parts of what shares cut: a warp a row, parts in order.  Block (CTA, rows).
template <int DP>
__global__ __launch_bounds__(kJoinWarps * 32) void cross_join_kernel(const __grid_constant__ CrossArgs a, const __grid_constant__ Plan p)
{
    constexpr int V = DP / 32;
    tc::pdl_launch_dependents();
    tc::pdl_wait();
    const Cut cut = p.cuts[blockIdx.x];
    if (cut.c1 < 0)
        return;
    const int warp = warp_index(), lane = threadIdx.x & 31, group = a.Hq / a.heads, n = cut.c1 - (int)blockIdx.x + 1;
    const int r = blockIdx.y * kJoinWarps + warp;
    if (r >= p.rows)
        return;
    const int tile = r < kTile ? cut.tile & 0xFFFF : cut.tile >> 16 & 0xFFFF, row = r % kTile;
    const int t = tile * p.tokens_a_tile + row / group;
    if (tile == kNoTile || row >= p.chunk_rows || t >= a.T)
        return;
    auto slot = [&](int i) { return ((int64_t)(blockIdx.x + i) * 2 + (i == 0 ? cut.slot : 0)) * p.rows + r; };
    float top = -INFINITY;
    float2 mine = make_float2(-INFINITY, 0.0f);     // maximum and sum of a lane's part
    if (lane < n)
        mine = reinterpret_cast<const float2 *>(p.tops)[slot(lane)];
    top = mine.x;
    for (int i = lane + 32; i < n; i += 32)
        top = fmaxf(top, p.tops[2 * slot(i)]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float zero = top == -INFINITY ? 0.0f : top;
    float sum = 0.0f, acc[V] = {};
    for (int base = 0; base < n; base += 32) {
        if (base > 0)
            mine = base + lane < n ? reinterpret_cast<const float2 *>(p.tops)[slot(base + lane)] : make_float2(-INFINITY, 0.0f);
        const float turn = mine.y == 0.0f ? 0.0f : ex2(mine.x - zero);      // saw nothing: its sums were not written
        float s = mine.y * turn;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            s += __shfl_xor_sync(0xffffffffu, s, o);
        sum += s;
        const int count = min(32, n - base);
#pragma unroll 8
        for (int i = 0; i < count; ++i) {
            const float by = __shfl_sync(0xffffffffu, turn, i), some = __shfl_sync(0xffffffffu, mine.y, i);
            float part[V];
            Columns<DP>::get(p.parts + slot(base + i) * DP, part);
#pragma unroll
            for (int v = 0; v < V; ++v)
                acc[v] = fmaf(some == 0.0f ? 0.0f : part[v], by, acc[v]);
        }
    }
    const int64_t at = (int64_t)t * a.Hq + cut.head * group + row % group;
    const int2 see = span_of(a.spans, a.S, t, nullptr);
    const bool some = see.x < see.y;
    const float by = some && sum != 0.0f ? 1.0f / sum : 0.0f;       // (no weight at all where every score is -inf)
#pragma unroll
    for (int v = 0; v < V; ++v)
        acc[v] = some ? acc[v] * by : 0.0f;
    if (lane * V < a.dim)
        Columns<DP>::put(a.out + at * a.dim, acc);
    if (a.lse && lane == 0)
        a.lse[at] = some ? (top + __log2f(sum)) * kLn2 : -INFINITY;
}

// No states at all: rows of zeros; a span that is not empty leaves the states.
__global__ void cross_nothing_kernel(const __grid_constant__ CrossArgs a)
{
    const int64_t rows = (int64_t)a.T * a.Hq, first = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, step = (int64_t)gridDim.x * blockDim.x;
    for (int64_t i = first; i < rows * a.dim / 8; i += step) {
        reinterpret_cast<uint4 *>(a.out)[i] = make_uint4(0u, 0u, 0u, 0u);
        if (a.lse && i < rows)
            a.lse[i] = -INFINITY;
    }
    for (int64_t t = first; t < a.T; t += step)
        span_of(a.spans, 0, (int)t, a.status);
}

// Of at most kMostTiles query tiles.
Plan plan_of(int64_t T, int64_t Hq, int64_t heads, int DP, size_t *bytes)
{
    Plan p;
    const int group = (int)(Hq / heads);
    p.tokens_a_tile = kTile / group;
    p.chunk_rows = p.tokens_a_tile * group;
    const int64_t tiles = (T + p.tokens_a_tile - 1) / p.tokens_a_tile;
    p.tiles = (int)(tiles < kMostTiles ? tiles : kMostTiles);
    p.rows = tiles > 1 ? 2 * kTile : (int)(T * group);
    p.ctas = device_sm_count();
    size_t at = (size_t)p.ctas * 2 * p.rows * DP * sizeof(float);
    p.parts = nullptr;
    p.tops = reinterpret_cast<float *>(at);
    at += ((size_t)p.ctas * 2 * p.rows * 2 * sizeof(float) + 15) / 16 * 16;
    p.cuts = reinterpret_cast<Cut *>(at);
    *bytes = at + p.ctas * sizeof(Cut);
    return p;
}

template <int DP>
cudaError_t launch(const CrossArgs &a, cudaStream_t stream)
{
    using L = Layout<DP>;
    static_assert(L::BYTES <= 232448 && L::BARS % 8 == 0 && L::ITEMS % 16 == 0 && 88 + 24 * L::STAGES <= 384, "shared memory");
    size_t bytes;
    Plan p = plan_of(a.T, a.Hq, a.heads, DP, &bytes);
    char *ws = static_cast<char *>(a.ws);
    p.parts = reinterpret_cast<float *>(ws);
    p.tops = reinterpret_cast<float *>(ws + reinterpret_cast<size_t>(p.tops));
    p.cuts = reinterpret_cast<Cut *>(ws + reinterpret_cast<size_t>(p.cuts));
    p.negative = a.scale < 0.0f;
    CUtensorMap mq, mk, mv;
    cudaError_t e = row_map(&mq, a.q, a.T, a.Hq, a.dim, a.qs, a.Hq / a.heads, p.tokens_a_tile);
    if (e == cudaSuccess)
        e = row_map(&mk, a.k, a.S, a.heads, a.dim, a.ks, 1, kTile);
    if (e == cudaSuccess)
        e = row_map(&mv, a.v, a.S, a.heads, a.dim, a.vs, 1, kTile);
    static std::atomic<unsigned long long> allowed;
    if (e == cudaSuccess)
        e = tc::allow_smem(cross_forward_kernel<DP>, L::BYTES, allowed);
    if (e == cudaSuccess)
        e = tc::launch_pdl(cross_forward_kernel<DP>, dim3(p.ctas), dim3(kThreads), L::BYTES, stream, mq, mk, mv, a, p);
    if (e == cudaSuccess)
        e = tc::launch_pdl(cross_join_kernel<DP>, dim3(p.ctas, (p.rows + kJoinWarps - 1) / kJoinWarps), dim3(kJoinWarps * 32), 0, stream, a, p);
    return e;
}

}  // namespace

size_t cross_attention_workspace(int64_t T, int64_t, int64_t Hq, int64_t heads, int64_t dim)
{
    size_t bytes;
    plan_of(T, Hq, heads, dim > 64 ? 128 : 64, &bytes);
    return bytes;
}

cudaError_t launch_cross_nothing(const CrossArgs &a, cudaStream_t stream)
{
    cross_nothing_kernel<<<device_sm_count(), 256, 0, stream>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_cross_attention(const CrossArgs &all, cudaStream_t stream)
{
    if (all.S == 0)
        return launch_cross_nothing(all, stream);
    const int64_t step = (int64_t)most_tiles(all.heads, (all.S + kTile - 1) / kTile, kMostTiles) * (kTile / (all.Hq / all.heads));
    for (int64_t t = 0; t < all.T; t += step) {
        CrossArgs a = all;
        a.T = (int)(all.T - t < step ? all.T - t : step);
        a.q += t * a.qs[0];
        a.out += t * a.Hq * a.dim;
        a.lse = a.lse ? a.lse + t * a.Hq : nullptr;
        a.spans = a.spans ? a.spans + 2 * t : nullptr;
        const cudaError_t e = a.dim > 64 ? launch<128>(a, stream) : launch<64>(a, stream);
        if (e != cudaSuccess)
            return e;
    }
    return cudaSuccess;
}

}  // namespace s3d8

// Attention of one new token per sequence over the paged cache
// (s3d8_paged_attention): the kernel.  Its instances are compiled in
// attention_{bf16,int8}_{8,16}.cu, the join of cut sequences and the dispatch in
// paged_attention.cu.
//
// Bound by HBM: every visible key and value is read once, for up to 16 query rows
// at a time.  The unit of work is a tile of 16 tokens of one (sequence, key/value
// head); the list of all tiles (a sequence's beginning counting as one more) is cut
// into contiguous runs, whatever the lengths are.  A warp streams its runs through
// a ring of its own in shared memory (cp.async, no barrier with other warps) and
// carries the softmax's running maximum m, sum l and the output sums O in fp32:
//   S = K Q^T (tensor cores, rows = tokens, columns = 8 or 16 query rows),
//   m' = max(m, S), O = 2^(m - m') O + V^T 2^(S - m'), l likewise.
// The matrix products are mma.sync (tcgen05's smallest tile is 64 rows, and the
// rate needed here is far below the tensor cores' limit).  The weights 2^(S - m')
// enter the second product as a 16-bit value and its 16-bit remainder: 16 bits of
// them in bf16.  With an int8 cache it is the weight times the value's scale, in fp16:
// 22 bits, or 2^-30 of the largest such product that its query row has met, whichever
// is coarser.
//
// Every warp begins with a run of three quarters of its even share; the last quarter
// of each share is in short runs that go to whichever warp is free (SMs differ by a
// quarter in the bandwidth they get: with even shares alone the slowest CTA of 64
// sequences of up to 8191 tokens ended at 174 us, the middle one at 146).  A run that
// ends inside a sequence leaves (m, l, O) in the workspace, and a second kernel joins
// the parts of each such sequence, in order of position.
//
// Measured with 32 / 8 heads of 128, join included: 8 sequences of up to 131072 tokens
// 531 to 547 us (6.6 to 6.8 TB/s), 64 of up to 8191 181 us (5.9 TB/s; 5 us until the first tiles
// arrive, 5 to 10 from the last ones through the join), 48 int8 sequences with a window
// 213 us (5.6 TB/s; 64% of the issue slots, a third of them turning codes into fp16).
#pragma once

#include <cfloat>

#include "async_copy.cuh"
#include "common.cuh"
#include "launch.h"
#include "tcgen05.cuh"

namespace s3d8 {

namespace attn {

constexpr int kTile = 16;          // tokens
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kSlack = 8.0f;     // weights reach 2^8
// int8 caches: what a value's code is multiplied with, its weight times its scale, is carried times a power of two of its
// query row (2^-kLeast to 2^kFar), which makes the row's largest product about 2^kUp when it is met and lets none pass
// 2^kFull: inside fp16.  By the products, not by the scales: a large scale on a token of no weight must not push the others down.
constexpr float kUp = 6.0f, kFull = 15.0f, kFar = 116.0f, kLeast = 120.0f;

template <int DP, bool INT8>
struct Shape {
    static constexpr int kRow = INT8 ? DP : 2 * DP;       // bytes of a key or value row in shared memory
    static constexpr int kChunks = kRow / 16;
    static constexpr int kKv = kTile * kRow;              // bytes of a tile's keys (and of its values)
    static constexpr int kScales = INT8 ? 2 * kTile * 4 : 0;
    static constexpr int kStage = 2 * kKv + kScales + 16; // + what the tile is
};

// ---- the plan: which tiles, and whose -----------------------------------------

struct Seq {
    int len, first, tiles;   // visible tokens first..len-1; tiles of 16 from the one that holds `first`

    // Places in the list: with a weight of 1 a sequence's beginning counts as one more (its query rows, its output), so that a
    // warp of many short sequences gets fewer tiles (64 of up to 1000 tokens 39 -> 35 us).
    __device__ __forceinline__ int places(int weight) const { return tiles ? tiles + weight : 0; }
};

__device__ __forceinline__ Seq sequence(const AttnArgs &a, int b)
{
    const int64_t room = a.width * a.kv.page_size;
    Seq s;
    s.len = (int)min((int64_t)max(a.lens[b], 0), room);
    s.first = a.window > 0 && s.len > a.window ? (int)(s.len - a.window) : 0;
    s.tiles = s.len > 0 ? (s.len + kTile - 1) / kTile - s.first / kTile : 0;
    return s;
}

// A place in the list: the beginning (k = 0) or tile k (from 1) of key/value head h,
// block of query rows blk, of sequence b.
struct Cursor {
    int b, h, blk, k;
    Seq s;

    __device__ __forceinline__ void next(const AttnArgs &a, int blocks)
    {
        if (++k <= s.tiles)
            return;
        k = 0;
        if (++blk < blocks)
            return;
        blk = 0;
        if (++h < a.kv.heads)
            return;
        h = 0;
        for (++b; b < a.B; ++b) {
            s = sequence(a, b);
            if (s.tiles > 0)
                return;
        }
    }
};

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void ldsm_x4_trans(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

template <bool F16>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if (F16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Transposes an 8 x 8 matrix of 16-bit values held two a lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t v)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// a b + c, 32 x 32 -> 64 bits.
__device__ __forceinline__ uint64_t wide(uint32_t a, uint32_t b, uint64_t c)
{
    return (uint64_t)a * b + c;
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float lg2(float x)
{
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// {lo, hi} as two 16-bit values in one register, and what their rounding left.
template <bool F16>
__device__ __forceinline__ void split2(float x, float y, uint32_t &top, uint32_t &rest)
{
    if (F16) {
        const __half2 h = __floats2half2_rn(x, y);
        const float2 f = __half22float2(h);
        const __half2 r = __floats2half2_rn(x - f.x, y - f.y);
        top = *reinterpret_cast<const uint32_t *>(&h);
        rest = *reinterpret_cast<const uint32_t *>(&r);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        const float2 f = __bfloat1622float2(h);
        const __nv_bfloat162 r = __floats2bfloat162_rn(x - f.x, y - f.y);
        top = *reinterpret_cast<const uint32_t *>(&h);
        rest = *reinterpret_cast<const uint32_t *>(&r);
    }
}

// 16-byte chunk c of row r of an int8 tile lies at chunk c ^ swz8(r): the reads
// below then meet no bank twice.
template <int CHUNKS>
__device__ __forceinline__ int swz8(int r)
{
    return CHUNKS >= 8 ? (r & 6) ^ ((r & 1) << 2) : (r >> 1) & (CHUNKS - 1);
}

// Four int8 codes (bytes of w) as two pairs of fp16, exactly: byte + 128 in the
// low bits of 1024 (0x6400), less 1152.
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t &p01, uint32_t &p23)
{
    const uint32_t u = w ^ 0x80808080u, magic = 0x64646464u;
    p01 = tc::f16x2_sub(prmt(u, magic, 0x4140), 0x64806480u);
    p23 = tc::f16x2_sub(prmt(u, magic, 0x4342), 0x64806480u);
}

// Byte i of either word as pair i of fp16, exactly.
__device__ __forceinline__ void pairs_to_f16(uint32_t w0, uint32_t w1, uint32_t (&f)[4])
{
    const uint32_t lo = prmt(w0, w1, 0x5140) ^ 0x80808080u, hi = prmt(w0, w1, 0x7362) ^ 0x80808080u, magic = 0x64646464u;
    f[0] = tc::f16x2_sub(prmt(lo, magic, 0x4140), 0x64806480u);
    f[1] = tc::f16x2_sub(prmt(lo, magic, 0x4342), 0x64806480u);
    f[2] = tc::f16x2_sub(prmt(hi, magic, 0x4140), 0x64806480u);
    f[3] = tc::f16x2_sub(prmt(hi, magic, 0x4342), 0x64806480u);
}

struct AttnPlan {
    int units, blocks, rows;     // per sequence: key/value heads x blocks of query rows; rows per block at most
    int group;                   // query heads per key/value head
    int log_page;                // of a page size that is a power of two, else -1
    uint32_t k16[3], v16[3], sc[3];   // strides of pages, tokens, heads: 16 bytes of keys and values, scales
    int alike;                   // keys and values have the same strides
    unsigned long long *queue;   // (kQueueTag, next short run): see grab
    int2 *joins;                 // [B units] first and last run of each sequence's parts, first < 0: nothing to join
    float *parts;                // [runs][2] partial states: of the sequence begun before the run, and of one that goes on behind it
};

// One partial state: rows x D output sums, then rows x (m, l); 16-byte aligned.
__host__ __device__ __forceinline__ size_t part_floats(int rows, int D)
{
    return (size_t)rows * D + ((2 * rows + 3) & ~3);
}

// ---- runs ------------------------------------------------------------------------------------
// The list in even shares, one a warp; of each share a long run, that its warp begins
// with, and short ones behind it, that are handed out.  Runs are numbered in the
// order of their places.
struct Runs {
    long long total;               // places of the call
    int share, head, rest, each;   // places of a share, of its long run, of a short one; runs of a share
    int count;                     // shares

    __device__ __forceinline__ Runs(long long places, int warps, bool short_runs) : total(places)
    {
        share = (int)((places + warps - 1) / warps);
        // Even shares alone where a short run's own cost (its query rows, a part to write and to join) passes what it evens
        // out (one sequence of 65536 tokens, 18 tiles a warp: 64 us, against 73 with short runs; 8 of up to 131072: 564 and
        // 550).
        const bool cut = share >= 32 && short_runs;
        head = cut ? share * 3 / 4 : share;
        rest = cut ? share / 8 : 1;
        each = 1 + (share - head + rest - 1) / rest;
        count = share ? (int)((places + share - 1) / share) : 0;
    }
    __device__ __forceinline__ long long begin(int r) const
    {
        const int s = r / each, j = r - s * each;
        return (long long)s * share + (j ? min(share, head + (j - 1) * rest) : 0);
    }
    // 0 or less where the list ends before it.
    __device__ __forceinline__ int length(int r) const
    {
        const int s = r / each, j = r - s * each;
        const int from = j ? min(share, head + (j - 1) * rest) : 0, to = min(share, head + j * rest);
        return (int)min((long long)(to - from), total - (long long)s * share - from);
    }
    __device__ __forceinline__ int of(long long place) const
    {
        const int s = (int)(place / share), at = (int)(place - (long long)s * share);
        return s * each + (at < head ? 0 : 1 + (at - head) / rest);
    }
};
constexpr int kRunsPerWarp = 4;    // a long one, and a quarter of a share and a tile in eighths of it

// The number of the next short run.  The join kernel leaves the counter at 0 under a
// tag; a workspace that holds anything else is set up by the first warp to ask.
constexpr unsigned long long kQueueTag = 0x53334438ull;
static __device__ int grab(unsigned long long *queue)
{
    for (;;) {
        unsigned long long old = atomicAdd(queue, 1ull);
        if (old >> 32 == kQueueTag)
            return (int)(uint32_t)old;
        ++old;
        for (;;) {
            const unsigned long long seen = atomicCAS(queue, old, kQueueTag << 32 | 1ull);
            if (seen == old)
                return 0;
            if (seen >> 32 == kQueueTag)
                break;
            old = seen;
        }
    }
}

// What a stage's tile is: visible tokens (16 bits) and flags; of a new state also its
// sequence, unit and run.
constexpr uint32_t kNew = 1u << 16;       // first tile of a state: of its run, or of its sequence
constexpr uint32_t kFirst = 1u << 17;     // first tile of its sequence
constexpr uint32_t kLast = 1u << 18;      // last tile of its sequence
constexpr uint32_t kStop = 1u << 19;      // last tile of its run

// ALIGNED: pages of a multiple of 16 tokens, so that a tile lies in one page and
// its rows follow one another at one stride.
// NB: blocks of 8 query rows.
template <int DP, bool INT8, int NB, bool ALIGNED, int WARPS, int STAGES>
__global__ __launch_bounds__(WARPS * 32, 1) void paged_attention_kernel(const __grid_constant__ AttnArgs a,
                                                                     const __grid_constant__ AttnPlan p)
{
    using Sh = Shape<DP, INT8>;
    constexpr int MT = DP / 16;                   // 16-column tiles of the output
    constexpr int kScanThreads = WARPS * 32;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    __shared__ long long scan[kScanThreads + 1];
    __shared__ long long warp_tiles[WARPS];
    __shared__ int warp_some[WARPS];
    __shared__ uint4 state[WARPS];                // what each warp's running state is of (as its first tile says)
    // int8: the powers of two that a lane's query rows carry (x = 0, 1 by y = 0, 1), and the value scale up to which no
    // product passes 2^kFull, whatever the weight.  In registers for 8 query rows (48 sequences with a window: 212 us, 219
    // from here); 16 leave none (64 sequences, 12 heads a key/value head of 128: 172 us from here, 183 in registers).
    constexpr bool kShared = INT8 && NB == 2;
    __shared__ __align__(16) float carried[kShared ? WARPS : 1][4][8];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int D = a.kv.dim, S = a.kv.page_size;
    tc::pdl_launch_dependents();
    tc::pdl_wait();

    // ---- places in front of each sequence ------------------------------------------
    // A beginning counts as a place where a warp gets several; with a tile a warp at most there is nothing to weigh.
    const int per = (a.B + kScanThreads - 1) / kScanThreads;   // sequences per scanning thread
    int weight;
    {
        long long tiles = 0;
        int some = 0;                             // sequences with tiles
        for (int i = 0; i < per; ++i) {
            const int b = threadIdx.x * per + i;
            if (b < a.B) {
                const int n = sequence(a, b).tiles;
                tiles += n;
                some += n > 0;
                if (blockIdx.x == 0 && a.lens[b] > a.width * S)
                    atomicExch(a.status, kStatusBounds);
            }
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long t = __shfl_up_sync(0xffffffffu, tiles, o);
            const int n = __shfl_up_sync(0xffffffffu, some, o);
            if (lane >= o) {
                tiles += t;
                some += n;
            }
        }
        if (lane == 31) {
            warp_tiles[warp] = tiles;
            warp_some[warp] = some;
        }
        __syncthreads();
        long long all = 0;
        for (int w = 0; w < WARPS; ++w) {
            all += warp_tiles[w];
            if (w < warp) {
                tiles += warp_tiles[w];
                some += warp_some[w];
            }
        }
        weight = all * p.units > (long long)gridDim.x * WARPS;
        scan[threadIdx.x + 1] = (tiles + (weight ? some : 0)) * p.units;
        if (threadIdx.x == 0)
            scan[0] = 0;
    }
    __syncthreads();
    const long long total = scan[kScanThreads];

    const Runs runs(total, gridDim.x * WARPS, !INT8);   // int8: bound by instructions, which every SM issues alike
    const int own = warp * gridDim.x + blockIdx.x;    // neighbouring runs on different SMs
    const size_t part_size = part_floats(p.rows, D);
    if (own < runs.count) {
        const uint32_t ring = smem_addr(smem_raw) + warp * (STAGES * Sh::kStage);
        Cursor in;                            // the tile to fetch next,
        int run = own * runs.each, left = 0;  // its run, and the places left of that, with it
        bool new_run = true, done = false;
        int asked = -1;                       // lane 0: the short run that comes next,
        bool pending = false;                 // once it has been asked for
        auto ask = [&]() {
            if (lane == 0 && runs.each > 1 && !pending) {
                const int i = grab(p.queue), s = i / (runs.each - 1);
                asked = s < runs.count ? s * runs.each + 1 + i - s * (runs.each - 1) : -1;
            }
            pending = true;
        };
        auto enter = [&]() {                  // to the first place of `run`
            const long long place = runs.begin(run);
            left = runs.length(run);
            new_run = true;
            // the scanning thread that holds it, then that one's sequences
            int lo = 0, hi = kScanThreads;
            while (hi - lo > 1) {
                const int mid = (lo + hi) / 2;
                if (scan[mid] <= place)
                    lo = mid;
                else
                    hi = mid;
            }
            long long ahead = place - scan[lo];
            in.b = lo * per;
            in.s = sequence(a, in.b);
            while (ahead >= (long long)in.s.places(weight) * p.units) {
                ahead -= (long long)in.s.places(weight) * p.units;
                in.s = sequence(a, ++in.b);
            }
            const uint32_t size = in.s.places(weight);
            uint32_t u, k;
            if (ahead >> 32) {
                u = (uint32_t)(ahead / size);
                k = (uint32_t)(ahead - (long long)u * size);
            } else {
                u = (uint32_t)ahead / size;
                k = (uint32_t)ahead - u * size;
            }
            in.k = (int)k + 1 - weight;
            in.h = p.blocks == 1 ? (int)u : (int)u / p.blocks;
            in.blk = (int)u - in.h * p.blocks;
        };
        auto settle = [&]() {                 // on to a tile: past a beginning, into the next run
            for (;;) {
                if (left > 0 && in.k == 0) {
                    left -= weight;
                    in.k = 1;
                }
                if (left > 0) {
                    if (left <= 2)
                        ask();                // the answer is there when this run ends
                    return;
                }
                ask();
                pending = false;
                run = __shfl_sync(0xffffffffu, asked, 0);
                if (run < 0) {
                    done = true;
                    return;
                }
                left = 0;
                if (runs.length(run) > 0)     // else behind the end of the list
                    enter();
            }
        };
        auto advance = [&]() {
            new_run = false;
            if (--left > 0)
                in.next(a, p.blocks);
            settle();
        };
        enter();
        settle();

        // ---- fetching: pages are looked up one tile ahead of the copies -----------------------
        const int side = lane >> 4;           // lanes 0-15 stand for the tile's keys, lanes 16-31 for its values
        constexpr int ES = INT8 ? 1 : 2, RPI = 32 / Sh::kChunks;   // element bytes; rows per round of 32 chunks
        const int fr = lane / Sh::kChunks, fc = lane % Sh::kChunks;
        const uint32_t lane_dst = fr * Sh::kRow + ((fc ^ (INT8 ? swz8<Sh::kChunks>(fr) : fr)) << 4);
        // round i of the copies: rows i RPI + fr; their swizzle differs from lane_dst's by a constant
        auto round_dst = [&](int i) {
            const uint32_t flip = (INT8 ? swz8<Sh::kChunks>((i * RPI) & 7) : (i * RPI) & 7) << 4;
            return i * RPI * Sh::kRow + (lane_dst ^ flip);
        };
        // this lane's chunk of the first rows of page 0, slot 0, head 0; its token's scale there
        const char *k_lane = static_cast<const char *>(a.kv.k) + (wide(fr, p.k16[1], fc) << 4);
        const char *v_lane = static_cast<const char *>(a.kv.v) + (wide(fr, p.v16[1], fc) << 4);
        const float *sc_lane = (side ? a.kv.v_scale : a.kv.k_scale) + (INT8 ? wide(lane & 15, p.sc[1], 0) : 0);
        int row_page = -1, row_slot = 0;      // of the next tile to fetch: its page and slot (ALIGNED: of its first token)
        bool row_seen = false;                // whether there is a visible token
        auto look_up = [&](bool live) {
            row_seen = false;
            if (!live)
                return;
            const int tok = (in.s.first / kTile + in.k - 1) * kTile + (ALIGNED ? 0 : lane & 15);
            if (!ALIGNED && (tok < in.s.first || tok >= in.s.len))
                return;
            row_seen = true;
            const int col = p.log_page >= 0 ? tok >> p.log_page : tok / S;
            row_slot = tok - col * S;
            row_page = a.table[in.b * a.width + col];
        };
        // Copies the tile that `in` stands at, looked up before.
        auto fetch = [&](uint32_t base) {
            const bool fresh = new_run || in.k == 1;
            if (fresh) {       // the query rows of a new state: into L1 by the time its first tile is there
                const int rows = min(p.group - in.blk * 16, p.rows);
                const char *src = reinterpret_cast<const char *>(a.q + ((int64_t)in.b * a.Hq + in.h * p.group + in.blk * 16) * D);
                for (int x = lane * 128; x < rows * D * 2; x += 32 * 128)
                    asm volatile("prefetch.global.L1 [%0];" ::"l"(src + x));
            }
            const bool ok = row_seen && row_page >= 0 && row_page < a.kv.pages;
            if (row_seen && !ok)
                atomicExch(a.status, kStatusBounds);   // its tokens stay masked
            const int row_bytes = D * ES;
            uint32_t mask;
            if (ALIGNED) {
                const int tok = (in.s.first / kTile + in.k - 1) * kTile;
                mask = 0xFFFFu;
                if (!ok || tok < in.s.first || tok + kTile > in.s.len) {
                    const int lo = max(in.s.first - tok, 0), hi = min(in.s.len - tok, kTile);
                    mask = ok ? ((1u << hi) - 1u) & ~((1u << lo) - 1u) : 0u;
                }
                const uint32_t page = ok ? row_page : 0;
                const uint64_t at_k = wide(page, p.k16[0], wide(row_slot, p.k16[1], wide(in.h, p.k16[2], 0))) << 4;
                const uint64_t at_v =
                    p.alike ? at_k : wide(page, p.v16[0], wide(row_slot, p.v16[1], wide(in.h, p.v16[2], 0))) << 4;
                if (INT8) {
                    const float *sc = sc_lane + wide(page, p.sc[0], wide(row_slot, p.sc[1], wide(in.h, p.sc[2], 0)));
                    cp_async4(base + 2 * Sh::kKv + lane * 4, sc, (mask >> (lane & 15)) & 1 ? 4 : 0);
                }
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    const char *src = kv ? v_lane + at_v : k_lane + at_k;
                    const uint64_t step = wide(kv ? p.v16[1] : p.k16[1], 16 * RPI, 0);
                    const uint32_t dst = base + kv * Sh::kKv;
                    if (mask == 0xFFFFu && D == DP) {
#pragma unroll
                        for (int i = 0; i < kTile / RPI; ++i, src += step)
                            cp_async16(dst + round_dst(i), src);
                    } else {
#pragma unroll
                        for (int i = 0; i < kTile / RPI; ++i, src += step) {
                            const bool live = ((mask >> (i * RPI + fr)) & 1) && fc * 16 < row_bytes;
                            cp_async16(dst + round_dst(i), live ? src : static_cast<const char *>(a.kv.k), live ? 16 : 0);
                        }
                    }
                }
            } else {
                const char *src = static_cast<const char *>(side ? a.kv.v : a.kv.k);
                if (ok) {
                    const uint32_t(&st)[3] = side ? p.v16 : p.k16;
                    src += wide(row_page, st[0], wide(row_slot, st[1], wide(in.h, st[2], 0))) << 4;
                }
                mask = __ballot_sync(0xffffffffu, ok);
                if (INT8) {
                    const float *sc = side ? a.kv.v_scale : a.kv.k_scale;
                    if (ok)
                        sc += wide(row_page, p.sc[0], wide(row_slot, p.sc[1], wide(in.h, p.sc[2], 0)));
                    cp_async4(base + 2 * Sh::kKv + lane * 4, sc, ok ? 4 : 0);
                }
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
#pragma unroll
                    for (int i = 0; i < kTile / RPI; ++i) {
                        const int r = i * RPI + fr;
                        const char *from = reinterpret_cast<const char *>(
                            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), kv * 16 + r));
                        const bool live = ((mask >> r) & 1) && fc * 16 < row_bytes;
                        cp_async16(base + kv * Sh::kKv + round_dst(i), live ? from + fc * 16 : from, live ? 16 : 0);
                    }
                }
            }
            if (lane == 0) {
                const uint32_t info = base + 2 * Sh::kKv + Sh::kScales;
                const int u = in.h * p.blocks + in.blk;
                const uint32_t what = (mask & 0xFFFFu) | (fresh ? kNew : 0u) | (in.k == 1 ? kFirst : 0u) |
                                      (in.k == in.s.tiles ? kLast : 0u) | (left == 1 ? kStop : 0u);
                asm volatile("st.shared.u32 [%0], %1;" ::"r"(info), "r"(what) : "memory");
                if (fresh) {
                    asm volatile("st.shared.u32 [%0], %1;" ::"r"(info + 4), "r"(in.b) : "memory");
                    asm volatile("st.shared.u32 [%0], %1;" ::"r"(info + 8), "r"(u) : "memory");
                    asm volatile("st.shared.u32 [%0], %1;" ::"r"(info + 12), "r"(run) : "memory");
                }
                if (in.k == 1) {
                    int2 join = make_int2(-1, -1);
                    if (in.s.tiles > left)    // goes on behind this run
                        join = make_int2(run, runs.of(runs.begin(run) + runs.length(run) - left + in.s.tiles - 1));
                    p.joins[(int64_t)in.b * p.units + u] = join;
                }
            }
        };

        look_up(!done);
        int fetched = 0;
#pragma unroll
        for (int s = 0; s < STAGES - 1; ++s) {
            if (!done) {
                fetch(ring + s * Sh::kStage);
                ++fetched;
                advance();
                look_up(!done);
            }
            cp_commit();
        }

        // ---- state of the current sequence: O^T, 16 columns x 8 query rows a tensor-core tile ----
        // lane (g, t) holds columns g and g + 8 of a tile for query rows 2t and 2t + 1
        float o[MT][NB][4], m[NB][2], l[NB][2];
        uint32_t q[DP / 16][NB][2];
        float qs[NB][2];                      // factor of a query row's scores, log2(e) in it
        float up[2][2], limit = 0.0f;
        float *const mine = carried[kShared ? warp : 0][t];
        auto read_powers = [&]() {
            if (!kShared)
                return;
            const uint4 v = lds_v4(smem_addr(mine));
            up[0][0] = __uint_as_float(v.x), up[0][1] = __uint_as_float(v.y);
            up[1][0] = __uint_as_float(v.z), up[1][1] = __uint_as_float(v.w);
        };
        auto write_powers = [&]() {
            if (kShared && g == 0) {
                *reinterpret_cast<float4 *>(mine) = make_float4(up[0][0], up[0][1], up[1][0], up[1][1]);
                mine[4] = limit;
            }
        };
        bool whole = false;                   // this run has the sequence from its first tile on

        uint32_t base = ring, filled = ring + (STAGES - 1) * Sh::kStage;   // stages of the tile, and of the next one to fetch
        auto turn = [&](uint32_t &stage) {
            stage += Sh::kStage;
            if (stage == ring + STAGES * Sh::kStage)
                stage = ring;
        };
        for (int i = 0; i < fetched; ++i, turn(base), turn(filled)) {
            __syncwarp();                     // every lane is done with tile i - 1, whose stage is filled again
            if (!done) {
                fetch(filled);
                ++fetched;
                advance();
                look_up(!done);
            }
            cp_commit();
            __syncwarp();
            const uint32_t mask = lds_u32(base + 2 * Sh::kKv + Sh::kScales);

            if (mask & kNew) {
                const uint4 info = lds_v4(base + 2 * Sh::kKv + Sh::kScales);
                if (lane == 0)
                    state[warp] = info;           // for the state's end
                const int unit = (int)info.z, h = p.blocks == 1 ? unit : unit / p.blocks, blk = unit - h * p.blocks;
                const int rows = min(p.group - blk * 16, p.rows);
                const int64_t head0 = (int64_t)info.y * a.Hq + h * p.group + blk * 16;   // query row of the state's row 0
                whole = mask & kFirst;
                up[0][0] = up[0][1] = up[1][0] = up[1][1] = 1.0f;
                limit = 0.0f;
                write_powers();
#pragma unroll
                for (int x = 0; x < NB; ++x) {
#pragma unroll
                    for (int j = 0; j < MT; ++j)
                        o[j][x][0] = o[j][x][1] = o[j][x][2] = o[j][x][3] = 0.0f;
                    m[x][0] = m[x][1] = INT8 ? -FLT_MAX : -INFINITY;
                    l[x][0] = l[x][1] = 0.0f;
                    qs[x][0] = qs[x][1] = a.scale * kLog2e;
                    const __nv_bfloat16 *src = a.q + (head0 + g + 8 * x) * D;
                    const bool in_row = g + 8 * x < rows;
                    if (!INT8) {
#pragma unroll
                        for (int ks = 0; ks < DP / 16; ++ks)
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                const int d = ks * 16 + y * 8 + 2 * t;
                                q[ks][x][y] = in_row && d < D ? __ldg(reinterpret_cast<const uint32_t *>(src + d)) : 0u;
                            }
                    } else {
                        // chunk order of the int8 keys: step 4 i + w, lane t <-> columns 16 (4 i + t) + 4 w ..+3.
                        // fp16 operands: the row times a power of two that puts its largest value near 2^14, exactly.
                        uint32_t top = 0u;
#pragma unroll
                        for (int ks = 0; ks < DP / 16; ++ks) {
                            const int d = 16 * (4 * (ks / 4) + t) + 4 * (ks % 4);
                            const uint2 v = in_row && d < D ? __ldg(reinterpret_cast<const uint2 *>(src + d)) : make_uint2(0u, 0u);
                            q[ks][x][0] = v.x;
                            q[ks][x][1] = v.y;
                            top = max_u16x2(top, v.x & 0x7FFF7FFFu);
                            top = max_u16x2(top, v.y & 0x7FFF7FFFu);
                        }
                        int e = (int)(max(top >> 16, top & 0xFFFFu) >> 7);        // largest biased exponent
                        e = max(e, __shfl_xor_sync(0xffffffffu, e, 1));
                        e = max(e, __shfl_xor_sync(0xffffffffu, e, 2));
                        e = min(max(e, 24), 254);
                        const float up = __uint_as_float((uint32_t)(127 + 13 + 127 - e) << 23);    // 2^(13 - (e - 127))
                        const float down = __uint_as_float((uint32_t)(e - 13) << 23);              // 2^((e - 127) - 13)
                        qs[x][0] *= __shfl_sync(0xffffffffu, down, 8 * t);       // rows 2t and 2t + 1
                        qs[x][1] *= __shfl_sync(0xffffffffu, down, 8 * t + 4);
#pragma unroll
                        for (int ks = 0; ks < DP / 16; ++ks)
#pragma unroll
                            for (int y = 0; y < 2; ++y) {
                                const __half2 f = __floats2half2_rn(__uint_as_float(q[ks][x][y] << 16) * up,
                                                                    __uint_as_float(q[ks][x][y] & 0xFFFF0000u) * up);
                                q[ks][x][y] = *reinterpret_cast<const uint32_t *>(&f);
                            }
                    }
                }
            }

            cp_wait<STAGES - 1>();
            __syncwarp();

            // ---- scores S^T = K Q^T: lane (g, t) holds tokens g and g + 8 of query rows 2t and 2t + 1 ----
            float sc[NB][4];
#pragma unroll
            for (int x = 0; x < NB; ++x)
                sc[x][0] = sc[x][1] = sc[x][2] = sc[x][3] = 0.0f;
            if (!INT8) {
                const int r = lane & 15;
                const uint32_t row = base + r * Sh::kRow;
#pragma unroll
                for (int ks = 0; ks < DP / 16; ++ks) {
                    uint32_t kf[4];
                    ldsm_x4(row + (((2 * ks + (lane >> 4)) ^ (r & 7)) << 4), kf);
#pragma unroll
                    for (int x = 0; x < NB; ++x)
                        mma<false>(sc[x], kf, q[ks][x][0], q[ks][x][1]);
                }
            } else {
#pragma unroll
                for (int y = 0; y < DP / 64; ++y) {
                    const int c = 4 * y + t;
                    const uint4 w0 = lds_v4(base + g * Sh::kRow + ((c ^ swz8<Sh::kChunks>(g)) << 4));
                    const uint4 w1 = lds_v4(base + (g + 8) * Sh::kRow + ((c ^ swz8<Sh::kChunks>(g + 8)) << 4));
                    const uint32_t u0[4] = {w0.x, w0.y, w0.z, w0.w}, u1[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                        uint32_t kf[4];
                        codes_to_f16(u0[z], kf[0], kf[2]);
                        codes_to_f16(u1[z], kf[1], kf[3]);
#pragma unroll
                        for (int x = 0; x < NB; ++x)
                            mma<true>(sc[x], kf, q[4 * y + z][x][0], q[4 * y + z][x][1]);
                    }
                }
            }
            float ks0 = 1.0f, ks1 = 1.0f, vs0 = 0.0f, vs1 = 0.0f;
            if (INT8) {
                const uint32_t at0 = base + 2 * Sh::kKv + g * 4;
                ks0 = __uint_as_float(lds_u32(at0));
                ks1 = __uint_as_float(lds_u32(at0 + 32));
                vs0 = __uint_as_float(lds_u32(at0 + kTile * 4));
                vs1 = __uint_as_float(lds_u32(at0 + kTile * 4 + 32));
            }
            const bool see0 = (mask >> g) & 1, see1 = (mask >> (g + 8)) & 1;
            // ---- running maximum, weights ---------------------------------------------------------------
            // The maximum moves only when a tile exceeds it by more than 2^kSlack: until then no lane has to hear of the others'
            // scores, and the weights stay below 2^kSlack.  int8 keeps the next whole number, and moves a row's power of two
            // only when a product passes 2^kFull, which takes a value scale above a limit: steps are by powers of two.
            if (kShared)
                limit = __uint_as_float(lds_u32(smem_addr(mine) + 16));
            bool above = false, heavy = INT8 && fmaxf(fabsf(vs0), fabsf(vs1)) > limit;
#pragma unroll
            for (int x = 0; x < NB; ++x)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    sc[x][y] = see0 ? sc[x][y] * (INT8 ? qs[x][y] * ks0 : qs[x][y]) : -INFINITY;
                    sc[x][2 + y] = see1 ? sc[x][2 + y] * (INT8 ? qs[x][y] * ks1 : qs[x][y]) : -INFINITY;
                    above |= fmaxf(sc[x][y], sc[x][2 + y]) > m[x][y] + kSlack;
                }
            bool move = __any_sync(0xffffffffu, above || heavy);
            if (INT8 && move) {
                read_powers();
#pragma unroll
                for (int x = 0; x < NB; ++x)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const float top = fmaxf(fabsf(ex2(sc[x][y] - m[x][y]) * vs0), fabsf(ex2(sc[x][2 + y] - m[x][y]) * vs1));
                        above |= top * up[x][y] > (float)(1 << (int)kFull);
                    }
                move = __any_sync(0xffffffffu, above);
            }
            if (move) {
                const float lv0 = INT8 ? lg2(fabsf(vs0)) : 0.0f, lv1 = INT8 ? lg2(fabsf(vs1)) : 0.0f;
                limit = FLT_MAX;
                float keep[NB][2];
#pragma unroll
                for (int x = 0; x < NB; ++x)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        float top = fmaxf(sc[x][y], sc[x][2 + y]);
                        float product = INT8 ? fmaxf(sc[x][y] + lv0, sc[x][2 + y] + lv1) : 0.0f;
#pragma unroll
                        for (int off = 4; off <= 16; off <<= 1) {
                            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
                            if (INT8)
                                product = fmaxf(product, __shfl_xor_sync(0xffffffffu, product, off));
                        }
                        const float was = m[x][y];
                        top = fmaxf(was, INT8 ? ceilf(top) : top);
                        keep[x][y] = top == was ? 1.0f : ex2(was - top);
                        m[x][y] = top;
                        l[x][y] *= keep[x][y];
                        if (INT8) {
                            // `same`: the exponent that leaves the output sums as they are
                            float &power = up[x][y];
                            const float same = (float)((int)(__float_as_uint(power) >> 23) - 127) + (top - was);
                            const float now = fmaxf(fminf(same, fminf(kUp - ceilf(product - top), kFar)), -kLeast);
                            keep[x][y] = now == same ? 1.0f : ex2(now - same);
                            power = __uint_as_float((uint32_t)((int)now + 127) << 23);
                            limit = fminf(limit, __uint_as_float((uint32_t)(127 + (int)(kFull - kSlack) - (int)now) << 23));
                        }
                    }
#pragma unroll
                for (int j = 0; j < MT; ++j)
#pragma unroll
                    for (int x = 0; x < NB; ++x) {
                        o[j][x][0] *= keep[x][0];
                        o[j][x][1] *= keep[x][1];
                        o[j][x][2] *= keep[x][0];
                        o[j][x][3] *= keep[x][1];
                    }
                write_powers();
                __syncwarp();
            }
            read_powers();
            uint32_t hi[NB][2], lo[NB][2];     // P^T as the second operand: tokens 2t, 2t + 1 (+ 8) of query row g
#pragma unroll
            for (int x = 0; x < NB; ++x) {
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    // nothing seen so far: every weight is 0
                    const float zero = !INT8 && m[x][y] == -INFINITY ? 0.0f : m[x][y];
                    const float w0 = ex2(sc[x][y] - zero), w1 = ex2(sc[x][2 + y] - zero);
                    l[x][y] += w0 + w1;
                    sc[x][y] = INT8 ? w0 * vs0 * up[x][y] : w0;
                    sc[x][2 + y] = INT8 ? w1 * vs1 * up[x][y] : w1;
                }
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    uint32_t top, rest;
                    split2<INT8>(sc[x][2 * y], sc[x][2 * y + 1], top, rest);
                    hi[x][y] = transpose8(top);
                    lo[x][y] = transpose8(rest);
                }
            }
            // ---- O^T += V^T P^T --------------------------------------------------------------------------
            const uint32_t vb = base + Sh::kKv;
            if (!INT8) {
                const int r = (lane & 7) + (lane >> 4) * 8;
                const uint32_t row = vb + r * Sh::kRow;
#pragma unroll
                for (int j = 0; j < MT; ++j) {
                    uint32_t vfr[4];
                    ldsm_x4_trans(row + (((2 * j + ((lane >> 3) & 1)) ^ (r & 7)) << 4), vfr);
#pragma unroll
                    for (int x = 0; x < NB; ++x) {
                        mma<false>(o[j][x], vfr, hi[x][0], hi[x][1]);
                        mma<false>(o[j][x], vfr, lo[x][0], lo[x][1]);
                    }
                }
            } else {
                // Lane (g, t) reads tokens 2t, 2t+1, 2t+8, 2t+9 at the columns of its g: columns 16 (8 x + g) ..+15 in 16-byte
                // chunks, two a tile (rows g and g + 8 of it); with 64 columns, 8 g ..+7.
                constexpr int X = DP >= 128 ? DP / 128 : 1, W = DP >= 128 ? 4 : 2;
#pragma unroll
                for (int x = 0; x < X; ++x) {
                    uint32_t w[4][W];
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const int r = 2 * t + (y & 1) + (y >> 1) * 8;
                        if (DP >= 128) {
                            const uint4 v = lds_v4(vb + r * Sh::kRow + (((8 * x + g) ^ swz8<Sh::kChunks>(r)) << 4));
                            w[y][0] = v.x;
                            w[y][1] = v.y;
                            w[y][W - 2] = v.z;
                            w[y][W - 1] = v.w;
                        } else {
                            asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                                         : "=r"(w[y][0]), "=r"(w[y][1])
                                         : "r"(vb + r * Sh::kRow + (((g >> 1) ^ swz8<Sh::kChunks>(r)) << 4) + (g & 1) * 8));
                        }
                    }
#pragma unroll
                    for (int z = 0; z < W; ++z) {
                        uint32_t f01[4], f89[4];
                        pairs_to_f16(w[0][z], w[1][z], f01);
                        pairs_to_f16(w[2][z], w[3][z], f89);
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const uint32_t vfr[4] = {f01[2 * y], f01[2 * y + 1], f89[2 * y], f89[2 * y + 1]};
                            const int j = x * 8 + 2 * z + y;
#pragma unroll
                            for (int b = 0; b < NB; ++b) {
                                mma<true>(o[j][b], vfr, hi[b][0], hi[b][1]);
                                mma<true>(o[j][b], vfr, lo[b][0], lo[b][1]);
                            }
                        }
                    }
                }
            }

            // ---- the end of the sequence, or of the run ----------------------------------------------------
            if (mask & (kLast | kStop)) {
                __syncwarp();
                read_powers();
                const uint4 info = state[warp];
                const int unit = (int)info.z, h = p.blocks == 1 ? unit : unit / p.blocks, blk = unit - h * p.blocks;
                const int rows = min(p.group - blk * 16, p.rows);
                const int64_t head0 = (int64_t)info.y * a.Hq + h * p.group + blk * 16;
#pragma unroll
                for (int off = 4; off <= 16; off <<= 1)
#pragma unroll
                    for (int x = 0; x < NB; ++x)
#pragma unroll
                        for (int y = 0; y < 2; ++y)
                            l[x][y] += __shfl_xor_sync(0xffffffffu, l[x][y], off);
                const bool final = (mask & kLast) && whole;
                float *part = p.parts + ((size_t)info.w * 2 + (whole ? 1 : 0)) * part_size;
#pragma unroll
                for (int x = 0; x < NB; ++x) {
                    float inv[2];
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const float f = INT8 ? __uint_as_float(0x7F000000u - __float_as_uint(up[x][y])) : 1.0f;   // 1 / up
                        inv[y] = final ? (l[x][y] == 0.0f ? 0.0f : f / l[x][y]) : f;
                    }
#pragma unroll
                    for (int j = 0; j < MT; ++j) {
                        // columns of the tile's rows g and g + 8
                        const int d0 = INT8 ? (DP >= 128 ? 16 * (8 * (j / 8) + g) + 2 * (j % 8) : 8 * g + 2 * j) : 16 * j + g;
                        const int d1 = INT8 ? d0 + 1 : d0 + 8;
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const int r = 8 * x + 2 * t + y;
                            if (r < rows) {
                                const float v0 = o[j][x][y] * inv[y], v1 = o[j][x][2 + y] * inv[y];
                                if (final) {
                                    __nv_bfloat16 *row = a.out + (head0 + r) * D;
                                    if (d0 < D)
                                        row[d0] = __float2bfloat16_rn(v0);
                                    if (d1 < D)
                                        row[d1] = __float2bfloat16_rn(v1);
                                } else {
                                    float *row = part + r * D;
                                    if (d0 < D)
                                        row[d0] = v0;
                                    if (d1 < D)
                                        row[d1] = v1;
                                }
                            }
                        }
                    }
                    if (g == 0) {
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const int r = 8 * x + 2 * t + y;
                            if (r < rows) {
                                if (!final) {
                                    *reinterpret_cast<float2 *>(part + p.rows * D + 2 * r) = make_float2(m[x][y], l[x][y]);
                                } else if (a.lse) {
                                    a.lse[head0 + r] = (m[x][y] + log2f(l[x][y])) * kLn2;
                                }
                            }
                        }
                    }
                }
            }
        }
        cp_wait<0>();
    }

    // ---- sequences of no tokens: zeros ------------------------------------------------
    for (int b = blockIdx.x * WARPS + warp; b < a.B; b += gridDim.x * WARPS) {
        if (a.lens[b] > 0 && a.width > 0)
            continue;
        for (int i = lane; i < p.units; i += 32)
            p.joins[(int64_t)b * p.units + i] = make_int2(-1, -1);
        for (int64_t i = lane; i < (int64_t)a.Hq * D; i += 32)
            a.out[(int64_t)b * a.Hq * D + i] = __float2bfloat16_rn(0.0f);
        if (a.lse)
            for (int i = lane; i < a.Hq; i += 32)
                a.lse[(int64_t)b * a.Hq + i] = -INFINITY;
    }
}

constexpr int kMaxWarps = 16;

template <int DP, bool INT8, int NB, bool ALIGNED, int WARPS, int STAGES>
cudaError_t launch(const AttnArgs &a, const AttnPlan &p, int ctas, cudaStream_t stream)
{
    constexpr int smem = WARPS * STAGES * Shape<DP, INT8>::kStage;
    static_assert(WARPS <= kMaxWarps && smem <= 226 * 1024, "the rings");
    auto kernel = paged_attention_kernel<DP, INT8, NB, ALIGNED, WARPS, STAGES>;
    static std::atomic<unsigned long long> allowed;
    const cudaError_t e = tc::allow_smem(kernel, smem, allowed);
    return e != cudaSuccess ? e : tc::launch_pdl(kernel, dim3(ctas), dim3(WARPS * 32), (size_t)smem, stream, a, p);
}

template <bool INT8, int NB, bool ALIGNED>
cudaError_t launch_dim(const AttnArgs &a, const AttnPlan &p, int ctas, cudaStream_t stream)
{
    if (a.kv.dim <= 64)
        return launch<64, INT8, NB, ALIGNED, NB == 1 ? 12 : 8, INT8 ? (NB == 1 ? 8 : 11) : (NB == 1 ? 4 : 6)>(a, p, ctas, stream);
    if (a.kv.dim <= 128)
        return launch<128, INT8, NB, ALIGNED, INT8 && NB == 1 ? 16 : 12, !INT8 ? 2 : NB == 1 ? 3 : 4>(a, p, ctas, stream);
    return launch<256, INT8, NB, ALIGNED, INT8 ? 8 : 4, 3>(a, p, ctas, stream);
}

template <bool INT8, int NB>
cudaError_t launch_pages(const AttnArgs &a, const AttnPlan &p, int ctas, cudaStream_t stream)
{
    return a.kv.page_size % kTile == 0 ? launch_dim<INT8, NB, true>(a, p, ctas, stream)
                                       : launch_dim<INT8, NB, false>(a, p, ctas, stream);
}

// The instances: queries of up to 8 or 16 heads per key/value head and block.
cudaError_t launch_bf16_8(const AttnArgs &a, const AttnPlan &p, int ctas, cudaStream_t stream);
cudaError_t launch_bf16_16(const AttnArgs &a, const AttnPlan &p, int ctas, cudaStream_t stream);
cudaError_t launch_int8_8(const AttnArgs &a, const AttnPlan &p, int ctas, cudaStream_t stream);
cudaError_t launch_int8_16(const AttnArgs &a, const AttnPlan &p, int ctas, cudaStream_t stream);

}  // namespace attn

}  // namespace s3d8

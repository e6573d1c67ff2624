// Rotary embedding of new queries and keys, and keys and values into the paged
// cache (s3d8_rope_append).
//
// HBM-bound: every (token, head) row of q, k and v is read once and written once.
// A row of D columns belongs to D/16 neighbouring lanes (rounded up to a power of
// two), two 16-byte chunks each, chosen so that a lane holds both columns of its
// rotary pairs; it reads its cosines and sines once and turns its columns of every
// head with them.  Few tokens, or heads that lie apart: one CTA per token.  Many:
// persistent CTAs fed by a ring of bulk copies, so that no load waits for another
// token's stores.  Measured: 61 tokens of 32 + 16 heads of 128 in 2.4 us, 16384 in
// 73 us (5.6 TB/s of what it has to move; 77 us without the ring), 4099 into int8 in
// 22 us (25 us).
#include "bf16x8.cuh"
#include "common.cuh"
#include "launch.h"
#include "rope_plan.h"
#include "tcgen05.cuh"

namespace s3d8 {

namespace {

// Codes of eight fp32 values of a row whose absmax gives s = RN(absmax / 127), r =
// RN(1 / s): as quant_chunk8 (the nearest integer of x r by the 1.5 2^23 sum, the
// rare near-ties again with the exact quotient), which takes bf16 values.
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float s, float r)
{
    if (s == 0.0f)
        return make_uint2(0u, 0u);
    uint32_t b[8];
    bool redo = s < kTinyScale;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float t = __fmul_rn(x[e], r);
        const float y = __fadd_rn(t, kRoundMagic);
        redo |= fabsf(__fsub_rn(t, __fsub_rn(y, kRoundMagic))) > kTieFloor;
        b[e] = __float_as_uint(y);
    }
    if (redo) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            b[e] = (uint32_t)quant_code(x[e], s, r);
    }
    return make_uint2(prmt(prmt(b[0], b[1], 0x0040), prmt(b[2], b[3], 0x0040), 0x5410),
                      prmt(prmt(b[4], b[5], 0x0040), prmt(b[6], b[7], 0x0040), 0x5410));
}

// Which two chunks a lane holds, and where the partners of its columns are.
enum RopeMode {
    kHalves,        // pairs (i, i + rotary/2), rotary a multiple of 16: both in one lane
    kNeighbours,    // pairs (2i, 2i + 1): two neighbouring chunks
    kHalvesOdd      // any other rotary: neighbouring chunks, partners read one by one
};

// A lane's part of every row: two chunks, and whether its pairs 8 lane .. 8 lane + 7 turn.
struct RopeLane {
    int lane, lanes, half, chunk[2];
    bool in_row, turns;

    __device__ __forceinline__ RopeLane(const RopeArgs &a, int mode, int log_lanes)
        : lane((int)threadIdx.x & ((1 << log_lanes) - 1)), lanes(1 << log_lanes), half(a.rotary / 2)
    {
        chunk[0] = 2 * lane;
        chunk[1] = 2 * lane + 1;
        if (mode == kHalves && lane < a.rotary / 16) {
            chunk[0] = lane;
            chunk[1] = lane + a.rotary / 16;
        }
        in_row = 16 * lane < a.kv.dim;
        turns = in_row && 8 * lane < half;
    }
};

template <int MODE>
__device__ __forceinline__ void turn(const RopeLane &l, float (&f)[2][8], const float (&cs)[8], const float (&sn)[8])
{
    if (MODE == kHalves) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float u = f[0][e], w = f[1][e];
            f[0][e] = u * cs[e] - w * sn[e];
            f[1][e] = w * cs[e] + u * sn[e];
        }
    } else if (MODE == kNeighbours) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {     // pair 8 lane + e: chunk e / 4, columns 2 (e % 4), + 1
            if (8 * l.lane + e >= l.half)
                continue;
            const float u = f[e / 4][2 * (e % 4)], w = f[e / 4][2 * (e % 4) + 1];
            f[e / 4][2 * (e % 4)] = u * cs[e] - w * sn[e];
            f[e / 4][2 * (e % 4) + 1] = w * cs[e] + u * sn[e];
        }
    }
}

// Writes a row: q as it is, keys and values into their page (page < 0: nowhere).
// Whole warps together (shuffles); `live`: this lane has a chunk of a row.
template <bool INT8>
__device__ __forceinline__ void put_row(const RopeArgs &a, const RopeLane &l, int64_t t, int head, bool live, int64_t page, int slot,
                                        const float (&f)[2][8])
{
    const int kind = head < a.Hq ? 0 : head < a.Hq + a.kv.heads ? 1 : 2;   // q, k, v
    const int h = kind == 0 ? head : kind == 1 ? head - a.Hq : head - a.Hq - a.kv.heads;
    if (live && kind == 0) {
        __nv_bfloat16 *o = a.q_out + (t * a.Hq + h) * a.kv.dim;
        *reinterpret_cast<uint4 *>(o + 8 * l.chunk[0]) = pack8(f[0]);
        *reinterpret_cast<uint4 *>(o + 8 * l.chunk[1]) = pack8(f[1]);
    }
    const int64_t *st = kind == 1 ? a.kv.ks : a.kv.vs;
    const int64_t at = page * st[0] + slot * st[1] + h * st[2];
    if (!INT8) {
        if (live && kind && page >= 0) {
            __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(kind == 1 ? a.kv.k : a.kv.v) + at;
            *reinterpret_cast<uint4 *>(o + 8 * l.chunk[0]) = pack8(f[0]);
            *reinterpret_cast<uint4 *>(o + 8 * l.chunk[1]) = pack8(f[1]);
        }
        return;
    }
    if (!__any_sync(0xffffffffu, live && kind))
        return;
    float top = 0.0f;     // of the row: codes of absmax / 127
#pragma unroll
    for (int e = 0; e < 8; ++e)
        top = fmaxf(top, fmaxf(fabsf(f[0][e]), fabsf(f[1][e])));
    for (int o = l.lanes >> 1; o > 0; o >>= 1)
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (!live || !kind || page < 0)
        return;
    const float s = __fdiv_rn(top, 127.0f);
    const float r = s > 0.0f ? __frcp_rn(s) : 0.0f;
    int8_t *o = static_cast<int8_t *>(kind == 1 ? a.kv.k : a.kv.v) + at;
#pragma unroll
    for (int y = 0; y < 2; ++y)
        *reinterpret_cast<uint2 *>(o + 8 * l.chunk[y]) = codes8(f[y], s, r);
    if (l.lane == 0)
        (kind == 1 ? a.kv.k_scale : a.kv.v_scale)[page * a.kv.ss[0] + slot * a.kv.ss[1] + h * a.kv.ss[2]] = s;
}

// Where token t goes: whether it is a token with an angle, and its page (-1: nowhere)
// and slot.  What is out of range is recorded once, by `one` thread.
__device__ __forceinline__ bool place(const RopeArgs &a, int pos, int64_t row, bool one, int &page, int &slot)
{
    page = -1;
    slot = 0;
    if (pos < 0)
        return false;
    bool bad = a.rotary && pos >= a.max_pos;
    const bool ok = !bad;
    if (ok) {
        const int col = pos / a.kv.page_size;
        slot = pos - col * a.kv.page_size;
        if (row >= 0 && row < a.table_rows && col < a.width)
            page = a.table[row * a.width + col];
        bad = page < 0 || page >= a.kv.pages;
        if (bad)
            page = -1;
    }
    if (bad && one)
        atomicExch(a.status, kStatusBounds);
    return ok;
}

// ROWS: rows of a lane whose loads leave together.
template <int MODE, bool INT8, int ROWS>
__global__ __launch_bounds__(kRopeThreads, 3) void rope_append_kernel(const __grid_constant__ RopeArgs a, int log_lanes, int vec)
{
    tc::pdl_launch_dependents();
    tc::pdl_wait();
    const int heads = a.Hq + 2 * a.kv.heads, slots = blockDim.x >> log_lanes;
    const int64_t t = blockIdx.x;
    const RopeLane l(a, MODE, log_lanes);

    // the rows do not depend on where the token stands: their loads leave first
    uint4 raw[ROWS][2];
    auto load_rows = [&](int base) {
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const int head = base + (threadIdx.x >> log_lanes) + i * slots;
            raw[i][0] = raw[i][1] = make_uint4(0u, 0u, 0u, 0u);
            if (head < heads && l.in_row) {
                const __nv_bfloat16 *x = head < a.Hq                ? a.q + t * a.qs[0] + head * a.qs[1]
                                         : head < a.Hq + a.kv.heads ? a.k + t * a.ks[0] + (head - a.Hq) * a.ks[1]
                                                                    : a.v + t * a.vs[0] + (head - a.Hq - a.kv.heads) * a.vs[1];
                raw[i][0] = ldg_stream_v4(x + 8 * l.chunk[0]);
                raw[i][1] = ldg_stream_v4(x + 8 * l.chunk[1]);
            }
        }
    };
    load_rows(0);
    const int pos = a.positions[t];
    int page, slot;
    const bool ok = place(a, pos, a.rows ? a.rows[t] : t, threadIdx.x == 0, page, slot);
    float cs[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f}, sn[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    if (ok && l.turns && MODE != kHalvesOdd) {
        const float *c = a.cos + (int64_t)pos * l.half + 8 * l.lane, *s = a.sin + (int64_t)pos * l.half + 8 * l.lane;
        if (vec) {
#pragma unroll
            for (int e = 0; e < 8; e += 4) {
                const float4 u = __ldg(reinterpret_cast<const float4 *>(c + e)), w = __ldg(reinterpret_cast<const float4 *>(s + e));
                cs[e] = u.x, cs[e + 1] = u.y, cs[e + 2] = u.z, cs[e + 3] = u.w;
                sn[e] = w.x, sn[e + 1] = w.y, sn[e + 2] = w.z, sn[e + 3] = w.w;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (8 * l.lane + e < l.half) {
                    cs[e] = __ldg(c + e);
                    sn[e] = __ldg(s + e);
                }
        }
    }

    for (int base = 0; base < heads; base += slots * ROWS) {   // whole warps together: there are shuffles below
        const int r0 = base + (threadIdx.x >> log_lanes);
        if (base > 0)
            load_rows(base);
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const int head = r0 + i * slots;
            const bool live = head < heads && l.in_row, keyed = head < a.Hq + a.kv.heads;   // q or k
            float f[2][8];
            const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
            unpack8(ok ? raw[i][0] : zero, f[0]);
            unpack8(ok ? raw[i][1] : zero, f[1]);
            if (keyed && l.turns)
                turn<MODE>(l, f, cs, sn);
            if (MODE == kHalvesOdd && keyed && live && ok) {
                const __nv_bfloat16 *x = head < a.Hq ? a.q + t * a.qs[0] + head * a.qs[1]
                                                     : a.k + t * a.ks[0] + (head - a.Hq) * a.ks[1];
                const float *c = a.cos + (int64_t)pos * l.half, *s = a.sin + (int64_t)pos * l.half;
                for (int e = 0; e < 16; ++e) {
                    const int d = 16 * l.lane + e;
                    float &v = f[e / 8][e % 8];
                    if (d < l.half)
                        v = v * c[d] - __bfloat162float(x[d + l.half]) * s[d];
                    else if (d < a.rotary)
                        v = v * c[d - l.half] + __bfloat162float(x[d - l.half]) * s[d - l.half];
                }
            }
            put_row<INT8>(a, l, t, head, live, page, slot, f);
        }
    }
}

// Many tokens whose heads follow one another: persistent CTAs, a token's q, k, v,
// cosines and sines by bulk copy into one stage of a ring.  The last warp copies
// (its lanes look up where 32 tokens go, a batch ahead of the copies), the others
// turn and store.  Many small CTAs, as the turning and the stores want warps:
// 16384 tokens of 48 heads of 128 take 78 us with two CTAs an SM of eight stages,
// 77 with three of five, 73 with five of three (int8: 102, 92, 70).
template <int MODE, bool INT8>
__global__ __launch_bounds__(kRopeThreads + 32, 3) void rope_append_ring_kernel(const __grid_constant__ RopeArgs a, int log_lanes,
                                                                              int stages, int stage_bytes)
{
    extern __shared__ __align__(128) unsigned char ring_mem[];
    __shared__ unsigned long long full_bar[kRingStages], empty_bar[kRingStages];
    __shared__ int4 meta[kRingStages];   // angle or not, page, slot
    const uint32_t ring = smem_addr(ring_mem), full = smem_addr(full_bar), empty = smem_addr(empty_bar);
    const int consumers = ((int)blockDim.x >> 5) - 1, warp = threadIdx.x >> 5;
    const int row_bytes = a.kv.dim * 2, heads = a.Hq + 2 * a.kv.heads, angles = heads * row_bytes;   // bytes of a stage's rows
    const int half_bytes = a.rotary * 2;
    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(full + 8 * s, 1);
            mbar_init(empty + 8 * s, consumers);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_proxy_async_smem();
    }
    __syncthreads();
    tc::pdl_launch_dependents();
    tc::pdl_wait();
    const int n = (int)((a.T - blockIdx.x + gridDim.x - 1) / gridDim.x);   // tokens blockIdx.x, + gridDim.x, ...
    bool timed_out = false;
    if (warp == consumers) {
        const int lane = threadIdx.x & 31;
        int pos = 0, page = -1, slot = 0, next_pos = 0, next_page = -1, next_slot = 0;
        bool ok = false, next_ok = false;
        auto look_up = [&](int i0) {
            if (i0 + lane < n) {
                const int64_t t = blockIdx.x + (int64_t)(i0 + lane) * gridDim.x;
                next_pos = a.positions[t];
                next_ok = place(a, next_pos, a.rows ? a.rows[t] : t, true, next_page, next_slot);
            }
        };
        look_up(0);
        int i = 0;
        for (; i < n; ++i) {
            if ((i & 31) == 0) {
                pos = next_pos;
                page = next_page;
                slot = next_slot;
                ok = next_ok;
                look_up(i + 32);
            }
            const int s = i % stages, from = i & 31;
            if (i >= stages && !tc::warp_wait(empty + 8 * s, ((i / stages) - 1) & 1)) {
                timed_out = true;
                break;
            }
            const int at = __shfl_sync(0xffffffffu, pos, from), pg = __shfl_sync(0xffffffffu, page, from);
            const int sl = __shfl_sync(0xffffffffu, slot, from), has = __shfl_sync(0xffffffffu, (int)ok, from);
            if (lane == 0) {
                const int64_t t = blockIdx.x + (int64_t)i * gridDim.x;
                const uint32_t to = ring + s * stage_bytes, bar = full + 8 * s;
                const bool angle = has && half_bytes;
                meta[s] = make_int4(has, pg, sl, 0);
                mbar_arrive_expect_tx(bar, (uint32_t)(angles + (angle ? 2 * half_bytes : 0)));
                bulk_load(to, a.q + t * a.qs[0], a.Hq * row_bytes, bar);
                bulk_load(to + a.Hq * row_bytes, a.k + t * a.ks[0], a.kv.heads * row_bytes, bar);
                bulk_load(to + (a.Hq + a.kv.heads) * row_bytes, a.v + t * a.vs[0], a.kv.heads * row_bytes, bar);
                if (angle) {
                    bulk_load(to + angles, a.cos + (int64_t)at * (a.rotary / 2), half_bytes, bar);
                    bulk_load(to + angles + half_bytes, a.sin + (int64_t)at * (a.rotary / 2), half_bytes, bar);
                }
            }
            __syncwarp();
        }
        // not before the last copies have landed
        for (int k = i - stages < 0 ? 0 : i - stages; k < i; ++k)
            if (!mbar_wait_bounded(full + 8 * (k % stages), (k / stages) & 1))
                timed_out = true;
    } else {
        const RopeLane l(a, MODE, log_lanes);
        const int slots = (consumers * 32) >> log_lanes;
        for (int i = 0; i < n; ++i) {
            const int s = i % stages;
            if (!tc::warp_wait(full + 8 * s, (i / stages) & 1)) {
                timed_out = true;
                break;
            }
            const int4 m = meta[s];
            const int64_t t = blockIdx.x + (int64_t)i * gridDim.x;
            const uint32_t from = ring + s * stage_bytes;
            float cs[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f}, sn[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
            if (m.x && l.turns) {
#pragma unroll
                for (int e = 0; e < 8; e += 4) {
                    const uint4 u = lds_v4(from + angles + (8 * l.lane + e) * 4), w = lds_v4(from + angles + half_bytes + (8 * l.lane + e) * 4);
                    cs[e] = __uint_as_float(u.x), cs[e + 1] = __uint_as_float(u.y), cs[e + 2] = __uint_as_float(u.z), cs[e + 3] = __uint_as_float(u.w);
                    sn[e] = __uint_as_float(w.x), sn[e + 1] = __uint_as_float(w.y), sn[e + 2] = __uint_as_float(w.z), sn[e + 3] = __uint_as_float(w.w);
                }
            }
            for (int base = 0; base < heads; base += slots) {   // whole warps together
                const int head = base + ((int)threadIdx.x >> log_lanes);
                const bool live = head < heads && l.in_row;
                const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
                float f[2][8];
                unpack8(live && m.x ? lds_v4(from + head * row_bytes + 16 * l.chunk[0]) : zero, f[0]);
                unpack8(live && m.x ? lds_v4(from + head * row_bytes + 16 * l.chunk[1]) : zero, f[1]);
                if (head < a.Hq + a.kv.heads && l.turns)
                    turn<MODE>(l, f, cs, sn);
                put_row<INT8>(a, l, t, head, live, m.y, m.z, f);
            }
            __syncwarp();
            if ((threadIdx.x & 31) == 0)
                tc::mbar_arrive(empty + 8 * s);
        }
    }
    if (timed_out)
        record_timeout(a.status);
}

template <int MODE, bool INT8>
cudaError_t launch_mode(const RopeArgs &a, cudaStream_t stream)
{
    int log_lanes = 0;
    while (16 << log_lanes < a.kv.dim)
        ++log_lanes;
    // One CTA per token: four rows a lane share one token's set-up (16384 tokens of 32 + 16 heads of 128: 79 us, against
    // 84 with three and 94 with two); two where the GPU has room for all tokens at once (61 tokens: 2.7 us against 3.4).
    const int heads = a.Hq + 2 * a.kv.heads, rows = a.T <= 2 * device_sm_count() ? 2 : 4;
    const int vec = a.rotary % 16 == 0 && ((uintptr_t)a.cos & 15) == 0 && ((uintptr_t)a.sin & 15) == 0;
    if constexpr (MODE != kHalvesOdd) {
        const RopeRing ring = rope_ring(heads, a.kv.dim, a.rotary, log_lanes);
        const bool whole = rope_whole(a.Hq, a.qs[1], a.kv.dim) && rope_whole(a.kv.heads, a.ks[1], a.kv.dim) &&
                           rope_whole(a.kv.heads, a.vs[1], a.kv.dim);
        // The ring from about as many tokens as there is room for at once (500 tokens of 48 heads of 128: 4.6 us against
        // 5.2).  Not for small rows in int8, which want more warps than it has (16384 tokens of 16 heads of 64: 31 us
        // against 27; of 12 heads of 256: 48 against 58).
        if (rows == 4 && vec && whole && ring.stages && (!INT8 || ring.stage >= 4096)) {
            const int64_t grid = (int64_t)device_sm_count() * ring.ctas;
            auto kernel = rope_append_ring_kernel<MODE, INT8>;
            static std::atomic<unsigned long long> allowed;
            const cudaError_t e = tc::allow_smem(kernel, kRingBytes, allowed);
            return e != cudaSuccess ? e
                                    : tc::launch_pdl(kernel, dim3((unsigned)(a.T < grid ? a.T : grid)), dim3(ring.threads + 32),
                                                     (size_t)ring.stages * ring.stage, stream, a, log_lanes, ring.stages, ring.stage);
        }
    }
    int threads = (((heads + rows - 1) / rows << log_lanes) + 31) / 32 * 32;
    threads = threads < kRopeThreads ? threads : kRopeThreads;
    return tc::launch_pdl(rows == 2 ? rope_append_kernel<MODE, INT8, 2> : rope_append_kernel<MODE, INT8, 4>,
                          dim3((unsigned)a.T), dim3(threads), 0, stream, a, log_lanes, vec);
}

template <int MODE>
cudaError_t launch_type(const RopeArgs &a, cudaStream_t stream)
{
    return a.kv.int8 ? launch_mode<MODE, true>(a, stream) : launch_mode<MODE, false>(a, stream);
}

}  // namespace

cudaError_t launch_rope_append(const RopeArgs &a, cudaStream_t stream)
{
    if (a.interleaved)
        return launch_type<kNeighbours>(a, stream);
    return a.rotary % 16 == 0 ? launch_type<kHalves>(a, stream) : launch_type<kHalvesOdd>(a, stream);
}

}  // namespace s3d8

// Rotary embedding of new queries and keys, and keys and values into the paged
// cache (s3d8_rope_append).
//
// HBM-bound: every (token, head) row of q, k and v is read once and written once.
// One CTA per token.  A row of D columns belongs to D/16 neighbouring lanes
// (rounded up to a power of two), two 16-byte chunks each, chosen so that a lane
// holds both columns of its rotary pairs; it reads its cosines and sines once and
// turns its columns of every head with them.  Measured: 16384 tokens of 32 + 16 heads
// of 128 in 77 us (5.4 TB/s of what it has to move; loads wait for one another only
// at a token's start), 61 tokens in 2.4 us.
#include "common.cuh"
#include "launch.h"
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

constexpr int kRopeThreads = 256;   // at most
// ROWS: rows of a lane whose loads leave together.
template <int MODE, bool INT8, int ROWS>
__global__ __launch_bounds__(kRopeThreads, 3) void rope_append_kernel(const __grid_constant__ RopeArgs a, int log_lanes, int vec)
{
    tc::pdl_launch_dependents();
    tc::pdl_wait();
    const int D = a.kv.dim, heads = a.Hq + 2 * a.kv.heads, half = a.rotary / 2;
    const int64_t t = blockIdx.x;
    const int lanes = 1 << log_lanes, lane = threadIdx.x & (lanes - 1), slots = blockDim.x >> log_lanes;
    int chunk[2] = {2 * lane, 2 * lane + 1};
    if (MODE == kHalves && lane < a.rotary / 16) {
        chunk[0] = lane;
        chunk[1] = lane + a.rotary / 16;
    }
    const bool in_row = 16 * lane < D;
    const bool turns = in_row && 8 * lane < half;    // this lane's pairs 8 lane .. 8 lane + 7

    // the rows do not depend on where the token stands: their loads leave first
    uint4 raw[ROWS][2];
    auto load_rows = [&](int base) {
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const int head = base + (threadIdx.x >> log_lanes) + i * slots;
            raw[i][0] = raw[i][1] = make_uint4(0u, 0u, 0u, 0u);
            if (head < heads && in_row) {
                const __nv_bfloat16 *x = head < a.Hq                ? a.q + t * a.qs[0] + head * a.qs[1]
                                         : head < a.Hq + a.kv.heads ? a.k + t * a.ks[0] + (head - a.Hq) * a.ks[1]
                                                                    : a.v + t * a.vs[0] + (head - a.Hq - a.kv.heads) * a.vs[1];
                raw[i][0] = ldg_stream_v4(x + 8 * chunk[0]);
                raw[i][1] = ldg_stream_v4(x + 8 * chunk[1]);
            }
        }
    };
    load_rows(0);
    const int pos = a.positions[t];
    bool ok = pos >= 0;
    if (ok && a.rotary && pos >= a.max_pos) {
        ok = false;
        if (threadIdx.x == 0)
            atomicExch(a.status, kStatusBounds);
    }
    int64_t page = -1;
    int slot = 0;
    if (ok) {
        const int64_t r = a.rows ? a.rows[t] : t;
        const int col = pos / a.kv.page_size;
        slot = pos - col * a.kv.page_size;
        if (r >= 0 && r < a.table_rows && col < a.width)
            page = a.table[r * a.width + col];
        if (page < 0 || page >= a.kv.pages) {
            page = -1;
            if (threadIdx.x == 0)
                atomicExch(a.status, kStatusBounds);
        }
    }
    float cs[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f}, sn[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    if (ok && turns && MODE != kHalvesOdd) {
        const float *c = a.cos + (int64_t)pos * half + 8 * lane, *s = a.sin + (int64_t)pos * half + 8 * lane;
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
                if (8 * lane + e < half) {
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
            const int kind = head < a.Hq ? 0 : head < a.Hq + a.kv.heads ? 1 : 2;   // q, k, v
            const int h = kind == 0 ? head : kind == 1 ? head - a.Hq : head - a.Hq - a.kv.heads;
            const bool live = head < heads && in_row;
            float f[2][8];
            const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
            unpack8(ok ? raw[i][0] : zero, f[0]);
            unpack8(ok ? raw[i][1] : zero, f[1]);
            if (kind < 2 && turns) {
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
                        if (8 * lane + e >= half)
                            continue;
                        const float u = f[e / 4][2 * (e % 4)], w = f[e / 4][2 * (e % 4) + 1];
                        f[e / 4][2 * (e % 4)] = u * cs[e] - w * sn[e];
                        f[e / 4][2 * (e % 4) + 1] = w * cs[e] + u * sn[e];
                    }
                }
            }
            if (MODE == kHalvesOdd && kind < 2 && live && ok) {
                const __nv_bfloat16 *x = kind == 0 ? a.q + t * a.qs[0] + h * a.qs[1] : a.k + t * a.ks[0] + h * a.ks[1];
                const float *c = a.cos + (int64_t)pos * half, *s = a.sin + (int64_t)pos * half;
                for (int e = 0; e < 16; ++e) {
                    const int d = 16 * lane + e;
                    float &v = f[e / 8][e % 8];
                    if (d < half)
                        v = v * c[d] - __bfloat162float(x[d + half]) * s[d];
                    else if (d < a.rotary)
                        v = v * c[d - half] + __bfloat162float(x[d - half]) * s[d - half];
                }
            }
            if (live && kind == 0) {
                __nv_bfloat16 *o = a.q_out + (t * a.Hq + h) * D;
                *reinterpret_cast<uint4 *>(o + 8 * chunk[0]) = pack8(f[0]);
                *reinterpret_cast<uint4 *>(o + 8 * chunk[1]) = pack8(f[1]);
            }
            const int64_t *st = kind == 1 ? a.kv.ks : a.kv.vs;
            const int64_t at = page * st[0] + slot * st[1] + h * st[2];
            if (!INT8) {
                if (live && kind && page >= 0) {
                    __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(kind == 1 ? a.kv.k : a.kv.v) + at;
                    *reinterpret_cast<uint4 *>(o + 8 * chunk[0]) = pack8(f[0]);
                    *reinterpret_cast<uint4 *>(o + 8 * chunk[1]) = pack8(f[1]);
                }
                continue;
            }
            if (!__any_sync(0xffffffffu, live && kind))
                continue;
            float top = 0.0f;     // of the row: codes of absmax / 127
#pragma unroll
            for (int e = 0; e < 8; ++e)
                top = fmaxf(top, fmaxf(fabsf(f[0][e]), fabsf(f[1][e])));
            for (int o = lanes >> 1; o > 0; o >>= 1)
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            if (!live || !kind || page < 0)
                continue;
            const float s = __fdiv_rn(top, 127.0f);
            const float r = s > 0.0f ? __frcp_rn(s) : 0.0f;
            int8_t *o = static_cast<int8_t *>(kind == 1 ? a.kv.k : a.kv.v) + at;
#pragma unroll
            for (int y = 0; y < 2; ++y)
                *reinterpret_cast<uint2 *>(o + 8 * chunk[y]) = codes8(f[y], s, r);
            if (lane == 0)
                (kind == 1 ? a.kv.k_scale : a.kv.v_scale)[page * a.kv.ss[0] + slot * a.kv.ss[1] + h * a.kv.ss[2]] = s;
        }
    }
}

template <int MODE, bool INT8>
cudaError_t launch_mode(const RopeArgs &a, cudaStream_t stream)
{
    int log_lanes = 0;
    while (16 << log_lanes < a.kv.dim)
        ++log_lanes;
    // Four rows a lane share one token's set-up (16384 tokens of 32 + 16 heads of 128: 79 us, against 84 with three
    // and 94 with two); two where the GPU has room for all tokens at once (61 tokens: 2.7 us against 3.4).
    const int heads = a.Hq + 2 * a.kv.heads, rows = a.T <= 2 * device_sm_count() ? 2 : 4;
    int threads = (((heads + rows - 1) / rows << log_lanes) + 31) / 32 * 32;
    threads = threads < kRopeThreads ? threads : kRopeThreads;
    const int vec = a.rotary % 16 == 0 && ((uintptr_t)a.cos & 15) == 0 && ((uintptr_t)a.sin & 15) == 0;
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

// Rotary embedding of new queries and keys, and keys and values into the paged
// cache (s3d8_rope_append).
//
// HBM-bound: every (token, head) row of q, k and v is read once and written once.
// A row of D columns belongs to D/8 neighbouring lanes (rounded up to a power of
// two), one 16-byte chunk each.
#include "common.cuh"
#include "launch.h"
#include "tcgen05.cuh"

namespace s3d8 {

namespace {

__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&f)[8])
{
    const uint4 v = ldg_stream_v4(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f[2 * j] = __uint_as_float(w[j] << 16);
        f[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint4 to_bf16x8(const float (&f)[8])
{
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t *>(&p);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

constexpr int kRopeThreads = 256;

__global__ __launch_bounds__(kRopeThreads) void rope_append_kernel(RopeArgs a, int lanes)
{
    tc::pdl_launch_dependents();
    tc::pdl_wait();
    const int D = a.kv.dim, heads = a.Hq + 2 * a.kv.heads;
    const int64_t unit = ((int64_t)blockIdx.x * kRopeThreads + threadIdx.x) / lanes;
    const int d0 = (int)(threadIdx.x % lanes) * 8;
    bool live = unit < a.T * heads && d0 < D;
    const int64_t t = live ? unit / heads : 0;
    const int head = live ? (int)(unit % heads) : 0;
    const int kind = head < a.Hq ? 0 : head < a.Hq + a.kv.heads ? 1 : 2;   // q, k, v
    float f[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    int64_t slot_page = -1;
    int slot = 0;
    const int h = kind == 0 ? head : kind == 1 ? head - a.Hq : head - a.Hq - a.kv.heads;
    if (live) {
        const int64_t pos = a.positions[t];
        bool ok = pos >= 0;
        if (ok && a.rotary && pos >= a.max_pos) {
            ok = false;
            atomicExch(a.status, kStatusBounds);
        }
        if (ok && kind) {
            const int64_t r = a.rows ? a.rows[t] : t;
            const int64_t col = pos / a.kv.page_size;
            slot = (int)(pos % a.kv.page_size);
            if (r >= 0 && r < a.table_rows && col < a.width) {
                const int p = a.table[r * a.width + col];
                if (p >= 0 && p < a.kv.pages)
                    slot_page = p;
            }
            if (slot_page < 0) {
                ok = false;
                atomicExch(a.status, kStatusBounds);
            }
        }
        if (ok) {
            const __nv_bfloat16 *x = kind == 0   ? a.q + t * a.qs[0] + h * a.qs[1]
                                     : kind == 1 ? a.k + t * a.ks[0] + h * a.ks[1]
                                                 : a.v + t * a.vs[0] + h * a.vs[1];
            load8(x + d0, f);
            if (kind < 2 && d0 < a.rotary) {
                const int half = a.rotary / 2;
                const float *c = a.cos + pos * half, *s = a.sin + pos * half;
                if (a.interleaved) {
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        if (d0 + e < a.rotary) {
                            const int i = (d0 + e) / 2;
                            const float u = f[e], w = f[e + 1];
                            f[e] = u * c[i] - w * s[i];
                            f[e + 1] = w * c[i] + u * s[i];
                        }
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int d = d0 + e;
                        if (d < half)
                            f[e] = f[e] * c[d] - __bfloat162float(x[d + half]) * s[d];
                        else if (d < a.rotary)
                            f[e] = f[e] * c[d - half] + __bfloat162float(x[d - half]) * s[d - half];
                    }
                }
            }
        }
        if (kind == 0)
            *reinterpret_cast<uint4 *>(a.q_out + (t * a.Hq + h) * D + d0) = to_bf16x8(f);
        live = ok && kind;
    }
    if (!a.kv.int8) {
        if (live) {
            const int64_t *st = kind == 1 ? a.kv.ks : a.kv.vs;
            __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(kind == 1 ? a.kv.k : a.kv.v) + slot_page * st[0] +
                               slot * st[1] + h * st[2] + d0;
            *reinterpret_cast<uint4 *>(o) = to_bf16x8(f);
        }
        return;
    }
    float top = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        top = fmaxf(top, fabsf(f[e]));
    for (int o = lanes >> 1; o > 0; o >>= 1)
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (!live)
        return;
    const float s = __fdiv_rn(top, 127.0f);
    const float r = s > 0.0f ? __frcp_rn(s) : 0.0f;
    uint32_t lo = 0, hi = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        lo |= (uint32_t)(quant_code(f[e], s, r) & 0xFF) << (8 * e);
        hi |= (uint32_t)(quant_code(f[e + 4], s, r) & 0xFF) << (8 * e);
    }
    const int64_t *st = kind == 1 ? a.kv.ks : a.kv.vs;
    int8_t *o = static_cast<int8_t *>(kind == 1 ? a.kv.k : a.kv.v) + slot_page * st[0] + slot * st[1] + h * st[2] + d0;
    *reinterpret_cast<uint2 *>(o) = make_uint2(lo, hi);
    if (d0 == 0)
        (kind == 1 ? a.kv.k_scale : a.kv.v_scale)[slot_page * a.kv.ss[0] + slot * a.kv.ss[1] + h * a.kv.ss[2]] = s;
}

}  // namespace

cudaError_t launch_rope_append(const RopeArgs &a, cudaStream_t stream)
{
    int lanes = 2;
    while (lanes * 8 < a.kv.dim)
        lanes *= 2;
    const int64_t units = a.T * (a.Hq + 2 * a.kv.heads), per = kRopeThreads / lanes;
    const int64_t grid = (units + per - 1) / per;
    if (grid > 0x7FFFFFFFLL)
        return cudaErrorInvalidValue;
    return tc::launch_pdl(rope_append_kernel, dim3((unsigned)grid), dim3(kRopeThreads), 0, stream, a, lanes);
}

}  // namespace s3d8

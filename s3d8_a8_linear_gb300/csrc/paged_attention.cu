// Attention of one new token per sequence over the paged cache
// (s3d8_paged_attention).
//
// One CTA per (sequence, query head); its warps walk the tokens with a running
// maximum and sum (lane l holds columns l, l + 32, ...) and join at the end.
#include "common.cuh"
#include "launch.h"
#include "tcgen05.cuh"

namespace s3d8 {

namespace {

constexpr int kWarps = 4;
constexpr int kCols = 8;   // 256 columns / 32 lanes

__device__ __forceinline__ float element(const void *base, int64_t at, int int8)
{
    return int8 ? (float)static_cast<const int8_t *>(base)[at]
                : __bfloat162float(static_cast<const __nv_bfloat16 *>(base)[at]);
}

__global__ __launch_bounds__(kWarps * 32) void paged_attention_kernel(AttnArgs a)
{
    __shared__ float om[kWarps], ol[kWarps], oo[kWarps][256];
    tc::pdl_launch_dependents();
    tc::pdl_wait();
    const int b = blockIdx.x / a.Hq, hq = blockIdx.x % a.Hq, h = hq / (a.Hq / a.kv.heads);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, D = a.kv.dim;
    int64_t len = a.lens[b];
    if (len > a.width * a.kv.page_size) {
        len = a.width * a.kv.page_size;
        if (threadIdx.x == 0)
            atomicExch(a.status, kStatusBounds);
    }
    const int64_t first = a.window > 0 && len > a.window ? len - a.window : 0;
    float q[kCols], o[kCols];
    for (int i = 0; i < kCols; ++i) {
        const int d = lane + 32 * i;
        q[i] = d < D ? __bfloat162float(a.q[((int64_t)b * a.Hq + hq) * D + d]) : 0.0f;
        o[i] = 0.0f;
    }
    float m = -INFINITY, l = 0.0f;
    for (int64_t j = first + warp; j < len; j += kWarps) {
        const int page = a.table[b * a.width + j / a.kv.page_size], t = (int)(j % a.kv.page_size);
        if (page < 0 || page >= a.kv.pages) {
            atomicExch(a.status, kStatusBounds);
            continue;
        }
        const int64_t ka = page * a.kv.ks[0] + t * a.kv.ks[1] + h * a.kv.ks[2];
        const int64_t va = page * a.kv.vs[0] + t * a.kv.vs[1] + h * a.kv.vs[2];
        const int64_t sa = page * a.kv.ss[0] + t * a.kv.ss[1] + h * a.kv.ss[2];
        float s = 0.0f;
        for (int i = 0; i < kCols; ++i)
            if (lane + 32 * i < D)
                s = fmaf(q[i], element(a.kv.k, ka + lane + 32 * i, a.kv.int8), s);
        for (int x = 16; x > 0; x >>= 1)
            s += __shfl_xor_sync(0xffffffffu, s, x);
        s *= a.scale * (a.kv.int8 ? a.kv.k_scale[sa] : 1.0f);
        const float top = fmaxf(m, s), base = top == -INFINITY ? 0.0f : top;
        const float old = expf(m - base), p = expf(s - base);
        m = top;
        l = l * old + p;
        const float pv = p * (a.kv.int8 ? a.kv.v_scale[sa] : 1.0f);
        for (int i = 0; i < kCols; ++i)
            if (lane + 32 * i < D)
                o[i] = fmaf(pv, element(a.kv.v, va + lane + 32 * i, a.kv.int8), o[i] * old);
    }
    if (lane == 0) {
        om[warp] = m;
        ol[warp] = l;
    }
    for (int i = 0; i < kCols; ++i)
        oo[warp][lane + 32 * i] = o[i];
    __syncthreads();
    float top = -INFINITY, sum = 0.0f;
    for (int w = 0; w < kWarps; ++w)
        top = fmaxf(top, om[w]);
    const float base = top == -INFINITY ? 0.0f : top;
    for (int w = 0; w < kWarps; ++w)
        sum += ol[w] * expf(om[w] - base);
    for (int d = threadIdx.x; d < D; d += kWarps * 32) {
        float v = 0.0f;
        for (int w = 0; w < kWarps; ++w)
            v += oo[w][d] * expf(om[w] - base);
        a.out[((int64_t)b * a.Hq + hq) * D + d] = __float2bfloat16_rn(sum == 0.0f ? 0.0f : v / sum);
    }
    if (threadIdx.x == 0 && a.lse)
        a.lse[(int64_t)b * a.Hq + hq] = top + logf(sum);
}

}  // namespace

size_t paged_attention_workspace(const KvCache &, int64_t, int64_t) { return 16; }

cudaError_t launch_paged_attention(const AttnArgs &a, cudaStream_t stream)
{
    return tc::launch_pdl(paged_attention_kernel, dim3((unsigned)(a.B * a.Hq)), dim3(kWarps * 32), 0, stream, a);
}

}  // namespace s3d8

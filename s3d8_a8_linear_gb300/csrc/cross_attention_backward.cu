// The gradients of attention to an encoder's states (s3d8_cross_attention_backward):
//
//   delta = dout . out, p_j = exp(s_j - lse), ds_j = p_j (dout . v_j - delta)
//   dq = scale sum_j ds_j k_j, dk_j = scale sum ds_j q, dv_j = sum p_j dout
#include "common.cuh"
#include "launch.h"
#include "tcgen05.cuh"

namespace s3d8 {

namespace {

constexpr int kWarps = 4;

__device__ __forceinline__ float warp_sum_f(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Token t's span, within the states; one that is not is cut to them and recorded.
__device__ __forceinline__ int2 span_of(const CrossArgs &a, int t)
{
    if (!a.spans)
        return make_int2(0, a.S);
    const int2 s = make_int2(a.spans[2 * (int64_t)t], a.spans[2 * (int64_t)t + 1]);
    if (s.x >= s.y)
        return make_int2(0, 0);
    if (s.x < 0 || s.y > a.S)
        atomicExch(a.status, kStatusBounds);
    return make_int2(max(s.x, 0), min(s.y, a.S));
}

struct Cols {
    float v[4];
};

__device__ __forceinline__ Cols columns(const __nv_bfloat16 *x, int dim)
{
    Cols c;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int d = (threadIdx.x & 31) + 32 * i;
        c.v[i] = d < dim ? __bfloat162float(x[d]) : 0.0f;
    }
    return c;
}

__device__ __forceinline__ float dot(const Cols &a, const Cols &b)
{
    return warp_sum_f(a.v[0] * b.v[0] + a.v[1] * b.v[1] + a.v[2] * b.v[2] + a.v[3] * b.v[3]);
}

__device__ __forceinline__ void store(__nv_bfloat16 *x, const Cols &c, float f, int dim)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int d = (threadIdx.x & 31) + 32 * i;
        if (d < dim)
            x[d] = __float2bfloat16_rn(c.v[i] * f);
    }
}

// A warp a (token, query head): dq, and delta for the other kernel.
__global__ __launch_bounds__(kWarps * 32) void cross_dq_kernel(const __grid_constant__ CrossArgs a)
{
    const int64_t row = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (row >= (int64_t)a.T * a.Hq)
        return;
    const int t = (int)(row / a.Hq), h = (int)(row % a.Hq), g = h / (a.Hq / a.heads);
    const int2 s = span_of(a, t);
    const Cols q = columns(a.q + t * a.qs[0] + h * a.qs[1], a.dim), d = columns(a.dout + t * a.ds[0] + h * a.ds[1], a.dim);
    const float delta = dot(d, columns(a.out + row * a.dim, a.dim)), lse = a.lse[row];
    Cols acc = {};
    for (int j = s.x; j < s.y; ++j) {
        const Cols k = columns(a.k + j * a.ks[0] + g * a.ks[1], a.dim);
        const float p = expf(a.scale * dot(q, k) - lse), ds = p * (dot(d, columns(a.v + j * a.vs[0] + g * a.vs[1], a.dim)) - delta);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            acc.v[i] += ds * k.v[i];
    }
    store(a.dq + row * a.dim, acc, a.scale, a.dim);
    if ((threadIdx.x & 31) == 0)
        static_cast<float *>(a.ws)[row] = delta;
}

// A warp a (state, key/value head).
__global__ __launch_bounds__(kWarps * 32) void cross_dkv_kernel(const __grid_constant__ CrossArgs a)
{
    const int64_t row = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (row >= (int64_t)a.S * a.heads)
        return;
    const int j = (int)(row / a.heads), g = (int)(row % a.heads), group = a.Hq / a.heads;
    const Cols k = columns(a.k + j * a.ks[0] + g * a.ks[1], a.dim), v = columns(a.v + j * a.vs[0] + g * a.vs[1], a.dim);
    Cols dk = {}, dv = {};
    for (int t = 0; t < a.T; ++t) {
        const int2 s = span_of(a, t);
        if (j < s.x || j >= s.y)
            continue;
        for (int h = g * group; h < (g + 1) * group; ++h) {
            const Cols q = columns(a.q + t * a.qs[0] + h * a.qs[1], a.dim), d = columns(a.dout + t * a.ds[0] + h * a.ds[1], a.dim);
            const int64_t at = (int64_t)t * a.Hq + h;
            const float p = expf(a.scale * dot(q, k) - a.lse[at]), ds = p * (dot(d, v) - static_cast<const float *>(a.ws)[at]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                dk.v[i] += ds * q.v[i];
                dv.v[i] += p * d.v[i];
            }
        }
    }
    store(a.dk + row * a.dim, dk, a.scale, a.dim);
    store(a.dv + row * a.dim, dv, 1.0f, a.dim);
}

unsigned blocks(int64_t rows) { return (unsigned)((rows + kWarps - 1) / kWarps); }

}  // namespace

size_t cross_attention_backward_workspace(int64_t T, int64_t, int64_t Hq, int64_t, int64_t) { return (size_t)(T * Hq) * sizeof(float) + 16; }

cudaError_t launch_cross_attention_backward(const CrossArgs &a, cudaStream_t stream)
{
    if (a.T > 0)
        cross_dq_kernel<<<blocks((int64_t)a.T * a.Hq), kWarps * 32, 0, stream>>>(a);
    if (a.S > 0)
        cross_dkv_kernel<<<blocks((int64_t)a.S * a.heads), kWarps * 32, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace s3d8

// The residual update behind a block fused with the norm in front of the next
// one, and its gradients (s3d8_residual_norm, s3d8_residual_norm_backward).
//
// Row by row, D columns, in fp32 from bf16:
//   h' = bf16(h + s * y * r' * w_post),  r' = rsqrt(mean(y^2) + eps), s = alpha g
//   x  = bf16(h' * r * w_pre),           r  = rsqrt(mean(h'^2) + eps)
// Both directions are bound by HBM: each row is read once into registers, its
// sums go through the CTA, and the outputs leave from the same registers.
#include "common.cuh"
#include "launch.h"
#include "tcgen05.cuh"

namespace s3d8 {

namespace {

__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f[2 * j] = __uint_as_float(w[j] << 16);
        f[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8])
{
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
        w[j] = *reinterpret_cast<const uint32_t *>(&p);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ float warp_sum_f(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sums of N values per thread over the CTA, the same in every thread.  `red`
// holds 32 N floats; two calls in a row need different `red`s (a third may take
// the first's again: every thread has passed the second's barrier by then, and so
// has read the first's).
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float *red)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = warp_sum_f(v[i]);
    if (nw == 1)
        return;
    if (lane == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            red[i * 32 + warp] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = warp_sum_f(lane < nw ? red[i * 32 + lane] : 0.0f);
}

__device__ __forceinline__ float gate_value(const NormArgs &a, int col)
{
    if (!a.gate)
        return 1.0f;
    const float g = __bfloat162float(a.gate[a.gate_n == 1 ? 0 : col]);
    return a.tanh_gate ? tanhf(g) : g;
}

// s * w_post of 8 columns, the factor of y r' in h'.
__device__ __forceinline__ void update_factor(const NormArgs &a, int chunk, float (&f)[8])
{
    if (a.w_post)
        unpack8(__ldg(reinterpret_cast<const uint4 *>(a.w_post) + chunk), f);
    const float one = a.gate_n == 1 || !a.gate ? a.alpha * gate_value(a, 0) : 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float s = a.gate && a.gate_n != 1 ? a.alpha * gate_value(a, 8 * chunk + e) : one;
        f[e] = a.w_post ? s * f[e] : s;
    }
}

template <int NS, int MAX_T>
__global__ __launch_bounds__(MAX_T) void residual_norm_kernel(NormArgs a)
{
    __shared__ float red[2][32];
    tc::pdl_launch_dependents();
    tc::pdl_wait();
    const int T = blockDim.x, chunks = a.D / 8;
    const float inv_d = 1.0f / (float)a.D;
    int flip = 0;
    for (int m = blockIdx.x; m < a.M; m += gridDim.x) {
        const size_t base = (size_t)m * chunks;
        uint4 hv[NS], yv[NS];
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            const int c = threadIdx.x + i * T;
            hv[i] = yv[i] = make_uint4(0u, 0u, 0u, 0u);
            if (c < chunks) {
                hv[i] = reinterpret_cast<const uint4 *>(a.h)[base + c];   // h_out may be h: an ordinary load
                if (a.y)
                    yv[i] = __ldg(reinterpret_cast<const uint4 *>(a.y) + base + c);
            }
        }
        if (a.y) {
            float r = 1.0f;
            if (a.w_post) {
                float s[1] = {0.0f};
#pragma unroll
                for (int i = 0; i < NS; ++i) {
                    float y[8];
                    unpack8(yv[i], y);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        s[0] = fmaf(y[e], y[e], s[0]);
                }
                block_sum(s, red[flip]);
                flip ^= 1;
                r = rsqrtf(s[0] * inv_d + a.eps);
            }
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                const int c = threadIdx.x + i * T;
                if (c < chunks) {
                    float h[8], y[8], f[8];
                    unpack8(hv[i], h);
                    unpack8(yv[i], y);
                    update_factor(a, c, f);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        h[e] = fmaf(y[e] * r, f[e], h[e]);
                    hv[i] = pack8(h);
                    reinterpret_cast<uint4 *>(a.h_out)[base + c] = hv[i];
                }
            }
        }
        if (!a.w_pre)
            continue;
        float s[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            float h[8];
            unpack8(hv[i], h);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                s[0] = fmaf(h[e], h[e], s[0]);
        }
        block_sum(s, red[flip]);
        flip ^= 1;
        const float r = rsqrtf(s[0] * inv_d + a.eps);
        uint32_t m2 = 0u;
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            const int c = threadIdx.x + i * T;
            if (c < chunks) {
                float h[8], w[8];
                unpack8(hv[i], h);
                unpack8(__ldg(reinterpret_cast<const uint4 *>(a.w_pre) + c), w);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    h[e] = h[e] * r * w[e];
                hv[i] = pack8(h);
                if (a.x)
                    reinterpret_cast<uint4 *>(a.x)[base + c] = hv[i];
                m2 = absmax_bf16x8(hv[i], m2);
            }
        }
        if (a.xq) {
            float top = absmax_bf16x2_value(m2);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const int nw = T >> 5, lane = threadIdx.x & 31;
            if (nw > 1) {
                if (lane == 0)
                    red[flip][threadIdx.x >> 5] = top;
                __syncthreads();
                top = lane < nw ? red[flip][lane] : 0.0f;
                flip ^= 1;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1)
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            }
            const float sc = __fdiv_rn(top, 127.0f);
            const float rs = sc > 0.0f ? __frcp_rn(sc) : 0.0f;
            if (threadIdx.x == 0)
                a.xscale[m] = sc;
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                const int c = threadIdx.x + i * T;
                if (c < chunks)
                    reinterpret_cast<uint2 *>(a.xq)[base + c] = quant_chunk8(hv[i], sc, rs);
            }
        }
    }
}

// One CTA walks rows blockIdx.x, + gridDim.x, ...; the column sums
//   P[d] = sum_m dx h' r   and   S[d] = sum_m G y r'
// stay in its threads' registers (in shared memory for rows over 8192 columns)
// and leave as one fp32 row of partials per CTA: dw_pre = P, dw_post = s S,
// dgate = alpha g' w_post S.
template <int NS, int MAX_T, bool WIDE>
__global__ __launch_bounds__(MAX_T) void residual_norm_backward_kernel(NormGradArgs g)
{
    extern __shared__ float wide_acc[];   // WIDE: [P, S][8][NS * T]
    __shared__ float red[2][3 * 32];
    const NormArgs &a = g.f;
    tc::pdl_launch_dependents();
    tc::pdl_wait();
    const int T = blockDim.x, chunks = a.D / 8;
    const float inv_d = 1.0f / (float)a.D;
    constexpr int NR = WIDE ? 1 : NS;
    float P[NR][8], S[NR][8];
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e)
            P[i][e] = S[i][e] = 0.0f;
    if (WIDE)
        for (int i = threadIdx.x; i < 2 * NS * T * 8; i += T)
            wide_acc[i] = 0.0f;
    __syncthreads();
    int flip = 0;
    for (int m = blockIdx.x; m < a.M; m += gridDim.x) {
        const size_t base = (size_t)m * chunks;
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        uint4 hv[NS], yv[NS], xv[NS], gv[NS];
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            const int c = threadIdx.x + i * T;
            const bool in = c < chunks;
            hv[i] = in ? __ldg(reinterpret_cast<const uint4 *>(a.h) + base + c) : zero;
            yv[i] = in && a.y ? __ldg(reinterpret_cast<const uint4 *>(a.y) + base + c) : zero;
            xv[i] = in && g.dx ? __ldg(reinterpret_cast<const uint4 *>(g.dx) + base + c) : zero;
            gv[i] = in && g.dh ? reinterpret_cast<const uint4 *>(g.dh)[base + c] : zero;
        }
        float s[3] = {0.0f, 0.0f, 0.0f};   // h'^2, a h', y^2
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            const int c = threadIdx.x + i * T;
            float h[8], x[8], y[8], w[8];
            unpack8(hv[i], h);
            unpack8(xv[i], x);
            unpack8(yv[i], y);
            unpack8(a.w_pre && c < chunks ? __ldg(reinterpret_cast<const uint4 *>(a.w_pre) + c) : zero, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                s[0] = fmaf(h[e], h[e], s[0]);
                s[1] = fmaf(x[e] * w[e], h[e], s[1]);
                s[2] = fmaf(y[e], y[e], s[2]);
            }
        }
        block_sum(s, red[flip]);
        flip ^= 1;
        const float r = rsqrtf(s[0] * inv_d + a.eps);
        const float ch = r * r * r * (s[1] * inv_d);
        const float rp = a.w_post ? rsqrtf(s[2] * inv_d + a.eps) : 1.0f;
        float t[1] = {0.0f};   // b y
        float G[NS][8];
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            const int c = threadIdx.x + i * T;
            float h[8], x[8], y[8], w[8], f[8];
            unpack8(hv[i], h);
            unpack8(xv[i], x);
            unpack8(yv[i], y);
            unpack8(gv[i], G[i]);
            if (c < chunks) {
                unpack8(a.w_pre ? __ldg(reinterpret_cast<const uint4 *>(a.w_pre) + c) : zero, w);
                if (a.y)
                    update_factor(a, c, f);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    G[i][e] = fmaf(r, x[e] * w[e], G[i][e]) - h[e] * ch;
                    const float dp = x[e] * h[e] * r, ds = G[i][e] * y[e] * rp;
                    if (WIDE) {
                        wide_acc[e * NS * T + c] += dp;
                        wide_acc[(8 + e) * NS * T + c] += ds;
                    } else {
                        P[i][e] += dp;
                        S[i][e] += ds;
                    }
                    if (a.y)
                        t[0] = fmaf(G[i][e] * f[e], y[e], t[0]);
                }
                reinterpret_cast<uint4 *>(g.dh_in)[base + c] = pack8(G[i]);
            }
        }
        float cy = 0.0f;
        if (a.w_post) {
            block_sum(t, red[flip]);
            flip ^= 1;
            cy = rp * rp * rp * (t[0] * inv_d);
        }
        if (a.y) {
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                const int c = threadIdx.x + i * T;
                if (c < chunks) {
                    float y[8], f[8];
                    unpack8(yv[i], y);
                    update_factor(a, c, f);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        f[e] = fmaf(rp * G[i][e], f[e], -y[e] * cy);
                    reinterpret_cast<uint4 *>(g.dy)[base + c] = pack8(f);
                }
            }
        }
    }
    // this CTA's row of partials: P, S, and sum_d w_post S for a single gate
    float *row = g.part + (size_t)blockIdx.x * (2 * a.D + 4);
    float dot[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        const int c = threadIdx.x + i * T;
        if (c < chunks) {
            float p[8], q[8], w[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                p[e] = WIDE ? wide_acc[e * NS * T + c] : P[WIDE ? 0 : i][e];
                q[e] = WIDE ? wide_acc[(8 + e) * NS * T + c] : S[WIDE ? 0 : i][e];
                w[e] = 1.0f;
            }
            if (a.w_post)
                unpack8(__ldg(reinterpret_cast<const uint4 *>(a.w_post) + c), w);
#pragma unroll
            for (int e = 0; e < 8; e += 4) {
                *reinterpret_cast<float4 *>(row + 8 * c + e) = make_float4(p[e], p[e + 1], p[e + 2], p[e + 3]);
                *reinterpret_cast<float4 *>(row + a.D + 8 * c + e) = make_float4(q[e], q[e + 1], q[e + 2], q[e + 3]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e)
                dot[0] = fmaf(w[e], q[e], dot[0]);
        }
    }
    block_sum(dot, red[flip]);
    if (threadIdx.x == 0)
        row[2 * a.D] = dot[0];
}

// Sums the CTAs' partial rows column by column, in the order of the CTAs.
__global__ void residual_norm_columns_kernel(NormGradArgs g, int ctas)
{
    const NormArgs &a = g.f;
    tc::pdl_wait();
    const int stride = 2 * a.D + 4;
    __shared__ float part[8][33];
    const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane;   // 0 .. 2 D: P, S, then the single gate's sum
    float s = 0.0f;
    if (col <= 2 * a.D)
        for (int i = grp; i < ctas; i += 8)
            s += g.part[(size_t)i * stride + col];
    part[grp][lane] = s;
    __syncthreads();
    if (grp != 0 || col > 2 * a.D)
        return;
#pragma unroll
    for (int i = 1; i < 8; ++i)
        s += part[i][lane];
    if (col < a.D) {
        if (g.dw_pre)
            g.dw_pre[col] = s;
        return;
    }
    const int d = col - a.D;
    if (col < 2 * a.D) {
        if (g.dw_post)
            g.dw_post[d] = a.alpha * gate_value(a, d) * s;
        if (!g.dgate || a.gate_n == 1)
            return;
        if (a.w_post)
            s *= __bfloat162float(a.w_post[d]);
    } else if (!g.dgate || a.gate_n != 1) {
        return;
    }
    const int k = col < 2 * a.D ? d : 0;
    float slope = 1.0f;
    if (a.tanh_gate) {   // 1 / cosh^2: 1 - tanh^2 would cancel for large gates
        const float c = 1.0f / coshf(__bfloat162float(a.gate[k]));
        slope = c * c;
    }
    g.dgate[k] = a.alpha * slope * s;
}

int norm_threads(int D, int ns)
{
    const int need = (D / 8 + ns - 1) / ns;
    return (need + 31) / 32 * 32;
}

// CTAs of the backward kernel: two per SM, each with one row of partials.
int backward_ctas(int M)
{
    const int most = 2 * device_sm_count();
    return M < most ? M : most;
}

}  // namespace

cudaError_t launch_residual_norm(const NormArgs &a, cudaStream_t stream)
{
    const int grid = a.M < 65536 ? a.M : 65536;
    if (a.D <= 256)
        return tc::launch_pdl(residual_norm_kernel<1, 32>, dim3(grid), dim3(norm_threads(a.D, 1)), 0, stream, a);
    if (a.D <= 8192)
        return tc::launch_pdl(residual_norm_kernel<2, 512>, dim3(grid), dim3(norm_threads(a.D, 2)), 0, stream, a);
    return tc::launch_pdl(residual_norm_kernel<2, 1024>, dim3(grid), dim3(norm_threads(a.D, 2)), 0, stream, a);
}

size_t residual_norm_backward_workspace(int64_t M, int64_t D)
{
    return (size_t)backward_ctas((int)M) * (2 * (size_t)D + 4) * sizeof(float);
}

cudaError_t launch_residual_norm_backward(const NormGradArgs &g, cudaStream_t stream)
{
    const int ctas = backward_ctas(g.f.M);
    cudaError_t e;
    if (g.f.D <= 256) {
        e = tc::launch_pdl(residual_norm_backward_kernel<1, 32, false>, dim3(ctas), dim3(norm_threads(g.f.D, 1)), 0, stream, g);
    } else if (g.f.D <= 8192) {
        e = tc::launch_pdl(residual_norm_backward_kernel<2, 512, false>, dim3(ctas), dim3(norm_threads(g.f.D, 2)), 0, stream, g);
    } else {
        const int T = norm_threads(g.f.D, 2);
        const size_t smem = (size_t)2 * 2 * T * 8 * sizeof(float);
        e = cudaFuncSetAttribute(residual_norm_backward_kernel<2, 1024, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)smem);
        if (e == cudaSuccess)
            e = tc::launch_pdl(residual_norm_backward_kernel<2, 1024, true>, dim3(ctas), dim3(T), smem, stream, g);
    }
    if (e != cudaSuccess)
        return e;
    if (!g.dw_pre && !g.dw_post && !g.dgate)
        return cudaSuccess;
    return tc::launch_pdl(residual_norm_columns_kernel, dim3((2 * g.f.D + 1 + 31) / 32), dim3(256), 0, stream, g, ctas);
}

}  // namespace s3d8

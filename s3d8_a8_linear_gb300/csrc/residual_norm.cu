// The residual update behind a block fused with the norm in front of the next
// one, and its gradients (s3d8_residual_norm, s3d8_residual_norm_backward).
//
// Row by row, D columns, in fp32 from bf16:
//   h' = bf16(h + s * y * r' * w_post),  r' = rsqrt(mean(y^2) + eps), s = alpha g
//   x  = bf16(h' * r * w_pre),           r  = rsqrt(mean(h'^2) + eps)
// Both directions are bound by HBM: each row is read once, its sums go through the
// CTA (or a group of lanes), and the outputs leave on the spot.  Forms, by the shape:
//   short rows (up to 1024 columns; 512 backward): a group of 8 to 32 lanes a row;
//   more rows than the GPU takes at once (and every backward call of up to 8192
//     columns): persistent CTAs, rows by bulk copy through a ring in shared memory,
//     the columns' factors in registers;
//   few rows (a token of 4096 columns is all latency, to which the ring's set-up
//     would only add), and backward calls of longer rows: a CTA a row, straight
//     from global memory.
// Measured, with a post-norm: forward of 16383 x 4096 88 us (6.1 TB/s of what it has
// to move), backward of 8192 x 4096 70 us (5.7 TB/s), forward of one token 2.7 us.
#include "bf16x8.cuh"
#include "common.cuh"
#include "launch.h"
#include "tcgen05.cuh"

namespace s3d8 {

namespace {

// Two fp32 lanes in a 64-bit register: one instruction for both, each rounded as the
// scalar one would.
typedef unsigned long long f2;
__device__ __forceinline__ f2 pair2(float lo, float hi)
{
    f2 d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ float2 split2(f2 v)
{
    float2 d;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(v));
    return d;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c)
{
    f2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b)
{
    f2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
// Eight bf16 values as four pairs, and back.
__device__ __forceinline__ void unpack4(uint4 v, f2 (&f)[4])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
        f[j] = pair2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u));
}
__device__ __forceinline__ uint4 pack4(const f2 (&f)[4])
{
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 v = split2(f[j]);
        const __nv_bfloat162 p = __floats2bfloat162_rn(v.x, v.y);
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

// Sums of eight values per thread over the CTA: total j is left in the lanes of
// every warp whose number is j modulo 8.  9 + 2 shuffles; `red`: 8 floats a warp,
// with the same rule for two calls in a row.
__device__ __forceinline__ float block_sum8(float (&v)[8], float *red)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
#pragma unroll
    for (int n = 8, o = 16; n > 1; n >>= 1, o >>= 1) {
        const bool upper = (lane & o) != 0;
#pragma unroll
        for (int i = 0; i < n / 2; ++i) {
            const float keep = upper ? v[i + n / 2] : v[i], send = upper ? v[i] : v[i + n / 2];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
    }
    float r = v[0];                       // value lane / 4, of this lane's share
    r += __shfl_xor_sync(0xffffffffu, r, 2);
    r += __shfl_xor_sync(0xffffffffu, r, 1);
    if ((lane & 3) == 0)
        red[warp * 8 + (lane >> 2)] = r;
    __syncthreads();
    r = 0.0f;
    for (int w = lane >> 3; w < nw; w += 4)
        r += red[w * 8 + (lane & 7)];
    r += __shfl_xor_sync(0xffffffffu, r, 8);
    return r + __shfl_xor_sync(0xffffffffu, r, 16);
}

// Sum, and maximum, over groups of GS neighbouring lanes.
template <int GS>
__device__ __forceinline__ float group_sum(float v)
{
#pragma unroll
    for (int o = GS / 2; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
template <int GS>
__device__ __forceinline__ float group_max(float v)
{
#pragma unroll
    for (int o = GS / 2; o > 0; o >>= 1)
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

__device__ __forceinline__ float block_max(float v, float *red)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    v = group_max<32>(v);
    if (nw == 1)
        return v;
    if (lane == 0)
        red[warp] = v;
    __syncthreads();
    return group_max<32>(lane < nw ? red[lane] : 0.0f);
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

__device__ __forceinline__ void update_factor(const NormArgs &a, int chunk, f2 (&f)[4])
{
    float v[8];
    update_factor(a, chunk, v);
#pragma unroll
    for (int e = 0; e < 4; ++e)
        f[e] = pair2(v[2 * e], v[2 * e + 1]);
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
            const float top = block_max(absmax_bf16x2_value(m2), red[flip]);
            flip ^= 1;
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

// What the three steps of a row do with one chunk of eight columns.
__device__ __forceinline__ float square_sum(uint4 v)
{
    float f[8], s = 0.0f;
    unpack8(v, f);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        s = fmaf(f[e], f[e], s);
    return s;
}
__device__ __forceinline__ uint4 updated(uint4 hv, uint4 yv, float r, const float (&f)[8])
{
    float h[8], y[8];
    unpack8(hv, h);
    unpack8(yv, y);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        h[e] = fmaf(y[e] * r, f[e], h[e]);
    return pack8(h);
}
__device__ __forceinline__ uint4 normed(uint4 hv, float r, uint4 wv)
{
    float h[8], w[8];
    unpack8(hv, h);
    unpack8(wv, w);
#pragma unroll
    for (int e = 0; e < 8; ++e)
        h[e] = h[e] * r * w[e];
    return pack8(h);
}

// Rows of up to GS * NS * 8 columns, one per group of GS lanes; the next row's
// loads leave before this one's work.
constexpr int kRowsThreads = 256;

template <int GS, int NS>
__global__ __launch_bounds__(kRowsThreads) void residual_norm_rows_kernel(NormArgs a)
{
    tc::pdl_launch_dependents();
    tc::pdl_wait();
    const int lane = threadIdx.x % GS, chunks = a.D / 8;
    const float inv_d = 1.0f / (float)a.D;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    float f[NS][8];
    uint4 w[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        const int c = lane + i * GS;
        w[i] = a.w_pre && c < chunks ? __ldg(reinterpret_cast<const uint4 *>(a.w_pre) + c) : zero;
        if (a.y && c < chunks)
            update_factor(a, c, f[i]);
    }
    const int step = gridDim.x * (kRowsThreads / GS);
    int m = blockIdx.x * (kRowsThreads / GS) + threadIdx.x / GS;
    uint4 hn[NS], yn[NS];
    auto load = [&](int row) {
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            const int c = lane + i * GS;
            hn[i] = yn[i] = zero;
            if (row < a.M && c < chunks) {
                hn[i] = reinterpret_cast<const uint4 *>(a.h)[(size_t)row * chunks + c];   // h_out may be h: an ordinary load
                if (a.y)
                    yn[i] = ldg_stream_v4(reinterpret_cast<const uint4 *>(a.y) + (size_t)row * chunks + c);
            }
        }
    };
    load(m);
    for (int m0 = blockIdx.x * (kRowsThreads / GS); m0 < a.M; m0 += step, m += step) {   // all groups of a CTA together
        uint4 hv[NS], yv[NS];
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            hv[i] = hn[i];
            yv[i] = yn[i];
        }
        load(m + step);
        const bool live = m < a.M;
        if (a.y) {
            float r = 1.0f;
            if (a.w_post) {
                float s = 0.0f;
#pragma unroll
                for (int i = 0; i < NS; ++i)
                    s += square_sum(yv[i]);
                r = rsqrtf(group_sum<GS>(s) * inv_d + a.eps);
            }
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                const int c = lane + i * GS;
                if (c < chunks) {
                    hv[i] = updated(hv[i], yv[i], r, f[i]);
                    if (live)
                        reinterpret_cast<uint4 *>(a.h_out)[(size_t)m * chunks + c] = hv[i];
                }
            }
        }
        if (!a.w_pre)
            continue;
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < NS; ++i)
            s += square_sum(hv[i]);
        const float r = rsqrtf(group_sum<GS>(s) * inv_d + a.eps);
        uint32_t m2 = 0u;
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            const int c = lane + i * GS;
            hv[i] = normed(hv[i], r, w[i]);
            if (c < chunks) {
                if (a.x && live)
                    reinterpret_cast<uint4 *>(a.x)[(size_t)m * chunks + c] = hv[i];
                m2 = absmax_bf16x8(hv[i], m2);
            }
        }
        if (a.xq) {
            const float sc = __fdiv_rn(group_max<GS>(absmax_bf16x2_value(m2)), 127.0f);
            const float rs = sc > 0.0f ? __frcp_rn(sc) : 0.0f;
            if (!live)
                continue;
            if (lane == 0)
                a.xscale[m] = sc;
#pragma unroll
            for (int i = 0; i < NS; ++i)
                if (lane + i * GS < chunks)
                    reinterpret_cast<uint2 *>(a.xq)[(size_t)m * chunks + lane + i * GS] = quant_chunk8(hv[i], sc, rs);
        }
    }
}

// ---- rows through a ring of bulk copies ---------------------------------------------------
// N tensors of the same shape, row m of each copied to one stage; rows blockIdx.x,
// + gridDim.x, ....  Thread 0 issues; a stage is filled again once every thread has
// passed a barrier behind its reads of it (release).
constexpr int kRingStages = 8;   // at most

struct RowRing {
    uint32_t data, bars;
    int stages, row_bytes, n;
    const char *src[4];
    int M, ahead;                 // rows issued so far, in steps of the grid

    __device__ __forceinline__ void issue()
    {
        const int64_t m = blockIdx.x + (int64_t)ahead * gridDim.x;
        if (m >= M)
            return;
        const int s = ahead % stages;
        mbar_arrive_expect_tx(bars + 8 * s, (uint32_t)(n * row_bytes));
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < n)
                bulk_load(data + (s * n + i) * row_bytes, src[i] + m * row_bytes, (uint32_t)row_bytes, bars + 8 * s);
        ++ahead;
    }
    __device__ __forceinline__ void start(unsigned char *smem, unsigned long long *bar_mem)
    {
        data = smem_addr(smem);
        bars = smem_addr(bar_mem);
        ahead = 0;
        if (threadIdx.x == 0) {
            for (int s = 0; s < stages; ++s)
                mbar_init(bars + 8 * s, 1);
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
            fence_proxy_async_smem();
        }
        __syncthreads();
    }
    __device__ __forceinline__ void fill()
    {
        if (threadIdx.x == 0)
            for (int s = 0; s < stages; ++s)
                issue();
    }
    __device__ __forceinline__ bool wait(int k) const { return mbar_wait_bounded(bars + 8 * (k % stages), (k / stages) & 1); }
    __device__ __forceinline__ uint4 chunk(int k, int tensor, int c) const
    {
        return lds_v4(data + ((k % stages) * n + tensor) * row_bytes + c * 16);
    }
    // After a wait that ran out: not before the copies in flight have landed, or as many waits have run out again.
    __device__ __forceinline__ void abandon(int k, int *status) const
    {
        if (threadIdx.x == 0) {
            record_timeout(status);
            for (int i = k; i < ahead; ++i)
                (void)wait(i);
        }
        __syncthreads();
    }
};

template <int NS, int T>
__global__ __launch_bounds__(T, T <= 256 ? 512 / T : 1) void residual_norm_ring_kernel(NormArgs a, int stages)
{
    extern __shared__ __align__(128) unsigned char ring_mem[];
    __shared__ float red[2][32];
    __shared__ unsigned long long bars[kRingStages];
    const int chunks = a.D / 8;
    const float inv_d = 1.0f / (float)a.D;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    RowRing ring;
    ring.stages = stages;
    ring.row_bytes = a.D * 2;
    ring.n = a.y ? 2 : 1;
    ring.M = a.M;
    ring.src[0] = reinterpret_cast<const char *>(a.h);
    ring.src[1] = reinterpret_cast<const char *>(a.y);
    ring.start(ring_mem, bars);
    tc::pdl_launch_dependents();
    tc::pdl_wait();
    ring.fill();
    float f[NS][8];
    uint4 w[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        const int c = threadIdx.x + i * T;
        w[i] = a.w_pre && c < chunks ? __ldg(reinterpret_cast<const uint4 *>(a.w_pre) + c) : zero;
        if (a.y && c < chunks)
            update_factor(a, c, f[i]);
    }
    int flip = 0, k = 0;
    for (int m = blockIdx.x; m < a.M; m += gridDim.x, ++k) {
        const size_t base = (size_t)m * chunks;
        if (!ring.wait(k)) {
            ring.abandon(k, a.status);
            return;
        }
        uint4 hv[NS], yv[NS];
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            const int c = threadIdx.x + i * T;
            hv[i] = c < chunks ? ring.chunk(k, 0, c) : zero;
            yv[i] = a.y && c < chunks ? ring.chunk(k, 1, c) : zero;
        }
        bool held = true;                 // until a barrier shows that every thread has read the stage
        if (a.y) {
            float r = 1.0f;
            if (a.w_post) {
                float s[1] = {0.0f};
#pragma unroll
                for (int i = 0; i < NS; ++i)
                    s[0] += square_sum(yv[i]);
                block_sum(s, red[flip]);
                flip ^= 1;
                r = rsqrtf(s[0] * inv_d + a.eps);
                held = false;
                if (threadIdx.x == 0)
                    ring.issue();
            }
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                const int c = threadIdx.x + i * T;
                if (c < chunks) {
                    hv[i] = updated(hv[i], yv[i], r, f[i]);
                    reinterpret_cast<uint4 *>(a.h_out)[base + c] = hv[i];
                }
            }
        }
        if (!a.w_pre) {
            if (held) {
                __syncthreads();
                if (threadIdx.x == 0)
                    ring.issue();
            }
            continue;
        }
        float s[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < NS; ++i)
            s[0] += square_sum(hv[i]);
        block_sum(s, red[flip]);
        flip ^= 1;
        if (held && threadIdx.x == 0)
            ring.issue();
        const float r = rsqrtf(s[0] * inv_d + a.eps);
        uint32_t m2 = 0u;
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            const int c = threadIdx.x + i * T;
            hv[i] = normed(hv[i], r, w[i]);
            if (c < chunks) {
                if (a.x)
                    reinterpret_cast<uint4 *>(a.x)[base + c] = hv[i];
                m2 = absmax_bf16x8(hv[i], m2);
            }
        }
        if (a.xq) {
            const float sc = __fdiv_rn(block_max(absmax_bf16x2_value(m2), red[flip]), 127.0f);
            flip ^= 1;
            const float rs = sc > 0.0f ? __frcp_rn(sc) : 0.0f;
            if (threadIdx.x == 0)
                a.xscale[m] = sc;
#pragma unroll
            for (int i = 0; i < NS; ++i)
                if (threadIdx.x + i * T < chunks)
                    reinterpret_cast<uint2 *>(a.xq)[base + threadIdx.x + i * T] = quant_chunk8(hv[i], sc, rs);
        }
    }
}

// ---- gradients ------------------------------------------------------------------------------
// Of a row, with a = dx w_pre and f = s w_post, the sums over columns of
//   h'^2, a h', y^2, f y dh, f y a, f y h'
// give everything: G = dh + r a - h' ch, ch = r^3 mean(a h'), and
//   sum(b y) = sum(f y G) = sum(f y dh) + r sum(f y a) - ch sum(f y h').
struct RowGrad {
    float r, ch, rp, cy;
};

__device__ __forceinline__ void grad_sums(uint4 hv, uint4 yv, uint4 xv, uint4 gv, uint4 wv, const f2 (&f)[4], f2 (&s)[6])
{
    f2 h[4], y[4], x[4], g[4], w[4];
    unpack4(hv, h);
    unpack4(yv, y);
    unpack4(xv, x);
    unpack4(gv, g);
    unpack4(wv, w);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const f2 ae = mul2(x[e], w[e]), fy = mul2(f[e], y[e]);
        s[0] = fma2(h[e], h[e], s[0]);
        s[1] = fma2(ae, h[e], s[1]);
        s[2] = fma2(y[e], y[e], s[2]);
        s[3] = fma2(fy, g[e], s[3]);
        s[4] = fma2(fy, ae, s[4]);
        s[5] = fma2(fy, h[e], s[5]);
    }
}
__device__ __forceinline__ void fold_sums(const f2 (&s)[6], float (&v)[8])
{
#pragma unroll
    for (int i = 0; i < 6; ++i) {
        const float2 t = split2(s[i]);
        v[i] = t.x + t.y;
    }
    v[6] = v[7] = 0.0f;
}

__device__ __forceinline__ RowGrad grad_factors(const NormArgs &a, float inv_d, float hh, float ah, float yy, float yg, float ya,
                                                float yh)
{
    // the cubes of the roots from the mean outwards: alone they would pass fp32's range for rows below 1e-13
    RowGrad q;
    q.r = rsqrtf(hh * inv_d + a.eps);
    q.ch = q.r * (q.r * (q.r * (ah * inv_d)));
    q.rp = a.w_post ? rsqrtf(yy * inv_d + a.eps) : 1.0f;
    q.cy = a.w_post ? q.rp * (q.rp * (q.rp * ((yg + q.r * ya - q.ch * yh) * inv_d))) : 0.0f;
    return q;
}

// One chunk's gradients, and its columns' sums P += dx h' r, S += G y r'.
__device__ __forceinline__ void grad_chunk(uint4 hv, uint4 yv, uint4 xv, uint4 gv, uint4 wv, const f2 (&f)[4], const RowGrad &q,
                                           f2 (&P)[4], f2 (&S)[4], uint4 &dh, uint4 &dy)
{
    f2 h[4], y[4], x[4], g[4], w[4];
    unpack4(hv, h);
    unpack4(yv, y);
    unpack4(xv, x);
    unpack4(gv, g);
    unpack4(wv, w);
    const f2 r = pair2(q.r, q.r), ch = pair2(-q.ch, -q.ch), rp = pair2(q.rp, q.rp), cy = pair2(-q.cy, -q.cy);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        g[e] = fma2(h[e], ch, fma2(r, mul2(x[e], w[e]), g[e]));
        P[e] = fma2(mul2(x[e], h[e]), r, P[e]);
        const f2 gr = mul2(rp, g[e]);
        S[e] = fma2(gr, y[e], S[e]);
        x[e] = fma2(gr, f[e], mul2(y[e], cy));
    }
    dh = pack4(g);
    dy = pack4(x);
}

// A CTA's row of partials: P, S, and sum_d w_post S for a single gate.
__device__ __forceinline__ float put_partials(const NormArgs &a, float *row, int c, const f2 (&P2)[4], const f2 (&S2)[4])
{
    float P[8], S[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 u = split2(P2[e]), v = split2(S2[e]);
        P[2 * e] = u.x, P[2 * e + 1] = u.y;
        S[2 * e] = v.x, S[2 * e + 1] = v.y;
    }
    float w[8] = {1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f}, dot = 0.0f;
    if (a.w_post)
        unpack8(__ldg(reinterpret_cast<const uint4 *>(a.w_post) + c), w);
#pragma unroll
    for (int e = 0; e < 8; e += 4) {
        *reinterpret_cast<float4 *>(row + 8 * c + e) = make_float4(P[e], P[e + 1], P[e + 2], P[e + 3]);
        *reinterpret_cast<float4 *>(row + a.D + 8 * c + e) = make_float4(S[e], S[e + 1], S[e + 2], S[e + 3]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        dot = fmaf(w[e], S[e], dot);
    return dot;
}

template <int GS, int NS>
__global__ __launch_bounds__(kRowsThreads) void residual_norm_backward_rows_kernel(NormGradArgs g)
{
    extern __shared__ __align__(16) float column_sums[];   // [2][D]
    __shared__ float red[32];
    const NormArgs &a = g.f;
    tc::pdl_launch_dependents();
    tc::pdl_wait();
    const int lane = threadIdx.x % GS, chunks = a.D / 8;
    const float inv_d = 1.0f / (float)a.D;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    f2 f[NS][4], P[NS][4], S[NS][4];
    uint4 w[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        const int c = lane + i * GS;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            P[i][e] = S[i][e] = f[i][e] = 0ull;
        w[i] = a.w_pre && c < chunks ? __ldg(reinterpret_cast<const uint4 *>(a.w_pre) + c) : zero;
        if (a.y && c < chunks)
            update_factor(a, c, f[i]);
    }
    const int groups = kRowsThreads / GS, group = threadIdx.x / GS;
    for (int m0 = blockIdx.x * groups; m0 < a.M; m0 += gridDim.x * groups) {
        const int m = m0 + group;
        const size_t base = (size_t)m * chunks;
        uint4 hv[NS], yv[NS], xv[NS], gv[NS];
        f2 s2[6] = {0ull, 0ull, 0ull, 0ull, 0ull, 0ull};
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            const int c = lane + i * GS;
            const bool in = m < a.M && c < chunks;
            hv[i] = in ? ldg_stream_v4(reinterpret_cast<const uint4 *>(a.h) + base + c) : zero;
            yv[i] = in && a.y ? ldg_stream_v4(reinterpret_cast<const uint4 *>(a.y) + base + c) : zero;
            xv[i] = in && g.dx ? ldg_stream_v4(reinterpret_cast<const uint4 *>(g.dx) + base + c) : zero;
            gv[i] = in && g.dh ? reinterpret_cast<const uint4 *>(g.dh)[base + c] : zero;   // dh_in may be dh
        }
#pragma unroll
        for (int i = 0; i < NS; ++i)
            grad_sums(hv[i], yv[i], xv[i], gv[i], w[i], f[i], s2);
        float s[8];
        fold_sums(s2, s);
#pragma unroll
        for (int i = 0; i < 6; ++i)
            s[i] = group_sum<GS>(s[i]);
        RowGrad q = grad_factors(a, inv_d, s[0], s[1], s[2], s[3], s[4], s[5]);
        if (m >= a.M)     // no row: nothing for the columns' sums, not even 0 times an infinite root (eps = 0)
            q.r = q.ch = q.rp = q.cy = 0.0f;
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            const int c = lane + i * GS;
            uint4 dh, dy;
            grad_chunk(hv[i], yv[i], xv[i], gv[i], w[i], f[i], q, P[i], S[i], dh, dy);
            if (m < a.M && c < chunks) {
                reinterpret_cast<uint4 *>(g.dh_in)[base + c] = dh;
                if (a.y)
                    reinterpret_cast<uint4 *>(g.dy)[base + c] = dy;
            }
        }
    }
    // the sums of a warp's groups, then one warp after another
#pragma unroll
    for (int o = GS; o < 32; o <<= 1)
#pragma unroll
        for (int i = 0; i < NS; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const f2 one = pair2(1.0f, 1.0f);
                P[i][e] = fma2(__shfl_xor_sync(0xffffffffu, P[i][e], o), one, P[i][e]);
                S[i][e] = fma2(__shfl_xor_sync(0xffffffffu, S[i][e], o), one, S[i][e]);
            }
    const int warp = threadIdx.x >> 5;
    for (int x = 0; x < kRowsThreads / 32; ++x) {
        if (warp == x && (threadIdx.x & 31) < GS) {
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                const int c = lane + i * GS;
                if (c < chunks) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        f2 *to = reinterpret_cast<f2 *>(column_sums + 8 * c) + e, *to_s = to + a.D / 2;
                        if (x) {
                            const f2 one = pair2(1.0f, 1.0f);
                            P[i][e] = fma2(*to, one, P[i][e]);
                            S[i][e] = fma2(*to_s, one, S[i][e]);
                        }
                        *to = P[i][e];
                        *to_s = S[i][e];
                    }
                }
            }
        }
        __syncthreads();
    }
    float *row = g.part + (size_t)blockIdx.x * (2 * a.D + 4);
    float dot[1] = {0.0f};
    if (warp == kRowsThreads / 32 - 1 && (threadIdx.x & 31) < GS) {
#pragma unroll
        for (int i = 0; i < NS; ++i)
            if (lane + i * GS < chunks)
                dot[0] += put_partials(a, row, lane + i * GS, P[i], S[i]);
    }
    block_sum(dot, red);
    if (threadIdx.x == 0)
        row[2 * a.D] = dot[0];
}

// One CTA walks rows blockIdx.x, + gridDim.x, ...; the columns' sums P and S stay in
// its threads' registers, and a row's chunks are read from the ring a second time
// instead of waiting there too (8192 x 4096: 72 us, against 82 with the chunks in the
// registers of twice the threads).
template <int NS, int T>
__global__ __launch_bounds__(T, T <= 256 ? 512 / T : 1) void residual_norm_backward_ring_kernel(NormGradArgs g, int stages)
{
    extern __shared__ __align__(128) unsigned char ring_mem[];
    __shared__ float red[2][8 * 32];
    __shared__ unsigned long long bars[kRingStages];
    const NormArgs &a = g.f;
    const int chunks = a.D / 8;
    const float inv_d = 1.0f / (float)a.D;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    RowRing ring;
    ring.stages = stages;
    ring.row_bytes = a.D * 2;
    ring.M = a.M;
    // h', then those of dh, dx and y that there are
    const char *dh = reinterpret_cast<const char *>(g.dh), *dx = reinterpret_cast<const char *>(g.dx);
    const char *y = reinterpret_cast<const char *>(a.y);
    const int at_g = dh ? 1 : -1, at_x = dx ? 1 + (dh != nullptr) : -1, at_y = y ? 1 + (dh != nullptr) + (dx != nullptr) : -1;
    ring.n = 1 + (dh != nullptr) + (dx != nullptr) + (y != nullptr);
    ring.src[0] = reinterpret_cast<const char *>(a.h);
    ring.src[1] = dh ? dh : dx ? dx : y;
    ring.src[2] = dh && dx ? dx : y;
    ring.src[3] = y;
    ring.start(ring_mem, bars);
    tc::pdl_launch_dependents();
    tc::pdl_wait();
    ring.fill();
    f2 f[NS][4], P[NS][4], S[NS][4];
    uint4 w[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        const int c = threadIdx.x + i * T;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            P[i][e] = S[i][e] = f[i][e] = 0ull;
        w[i] = a.w_pre && c < chunks ? __ldg(reinterpret_cast<const uint4 *>(a.w_pre) + c) : zero;
        if (a.y && c < chunks)
            update_factor(a, c, f[i]);
    }
    int flip = 0, k = 0;
    for (int m = blockIdx.x; m < a.M; m += gridDim.x, ++k) {
        const size_t base = (size_t)m * chunks;
        if (!ring.wait(k)) {
            ring.abandon(k, a.status);
            return;
        }
        uint4 hv[NS], yv[NS], xv[NS], gv[NS];
        auto read = [&](int i) {
            const int c = threadIdx.x + i * T;
            const bool in = c < chunks;
            hv[i] = in ? ring.chunk(k, 0, c) : zero;
            yv[i] = in && at_y > 0 ? ring.chunk(k, at_y, c) : zero;
            xv[i] = in && at_x > 0 ? ring.chunk(k, at_x, c) : zero;
            gv[i] = in && at_g > 0 ? ring.chunk(k, at_g, c) : zero;
        };
        f2 s2[6] = {0ull, 0ull, 0ull, 0ull, 0ull, 0ull};
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            read(i);
            grad_sums(hv[i], yv[i], xv[i], gv[i], w[i], f[i], s2);
        }
        float s[8];
        fold_sums(s2, s);
        const float total = block_sum8(s, red[flip]);
        flip ^= 1;
        float t[6];
#pragma unroll
        for (int i = 0; i < 6; ++i)
            t[i] = __shfl_sync(0xffffffffu, total, i);
        const RowGrad q = grad_factors(a, inv_d, t[0], t[1], t[2], t[3], t[4], t[5]);
#pragma unroll
        for (int i = 0; i < NS; ++i) {
            const int c = threadIdx.x + i * T;
            uint4 dh, dy;
            read(i);
            grad_chunk(hv[i], yv[i], xv[i], gv[i], w[i], f[i], q, P[i], S[i], dh, dy);
            if (c < chunks) {
                reinterpret_cast<uint4 *>(g.dh_in)[base + c] = dh;
                if (a.y)
                    reinterpret_cast<uint4 *>(g.dy)[base + c] = dy;
            }
        }
        __syncthreads();
        if (threadIdx.x == 0)
            ring.issue();
    }
    float *row = g.part + (size_t)blockIdx.x * (2 * a.D + 4);
    float dot[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NS; ++i)
        if (threadIdx.x + i * T < chunks)
            dot[0] += put_partials(a, row, threadIdx.x + i * T, P[i], S[i]);
    block_sum(dot, red[flip]);
    if (threadIdx.x == 0)
        row[2 * a.D] = dot[0];
}

// Rows of more than 8192 columns: straight from global memory, the columns' sums in
// shared memory.
constexpr int kWideThreads = 512, kWideChunks = 4;   // a thread's chunks of 8 columns

__global__ __launch_bounds__(kWideThreads) void residual_norm_backward_wide_kernel(NormGradArgs g)
{
    extern __shared__ __align__(16) f2 column_pairs[];   // [P, S][4][chunks] pairs
    __shared__ float red[2][8 * 32];
    const NormArgs &a = g.f;
    tc::pdl_launch_dependents();
    tc::pdl_wait();
    const int T = blockDim.x, chunks = a.D / 8;
    const float inv_d = 1.0f / (float)a.D;
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    for (int i = threadIdx.x; i < 8 * chunks; i += T)
        column_pairs[i] = 0ull;
    __syncthreads();
    int flip = 0;
    for (int m = blockIdx.x; m < a.M; m += gridDim.x) {
        const size_t base = (size_t)m * chunks;
        f2 s2[6] = {0ull, 0ull, 0ull, 0ull, 0ull, 0ull}, f[4] = {0ull, 0ull, 0ull, 0ull};
        uint4 hv[kWideChunks], yv[kWideChunks], xv[kWideChunks], gv[kWideChunks];
        auto weight = [&](int c) { return a.w_pre ? __ldg(reinterpret_cast<const uint4 *>(a.w_pre) + c) : zero; };
#pragma unroll
        for (int i = 0; i < kWideChunks; ++i) {
            const int c = threadIdx.x + i * T;
            const bool in = c < chunks;
            hv[i] = in ? ldg_stream_v4(reinterpret_cast<const uint4 *>(a.h) + base + c) : zero;
            yv[i] = in && a.y ? ldg_stream_v4(reinterpret_cast<const uint4 *>(a.y) + base + c) : zero;
            xv[i] = in && g.dx ? ldg_stream_v4(reinterpret_cast<const uint4 *>(g.dx) + base + c) : zero;
            gv[i] = in && g.dh ? reinterpret_cast<const uint4 *>(g.dh)[base + c] : zero;   // dh_in may be dh
        }
        // the next row comes as far as L2 meanwhile, a line for every eighth thread
        if ((threadIdx.x & 7) == 0 && m + (int)gridDim.x < a.M) {
            const __nv_bfloat16 *rows[4] = {a.h, a.y, g.dx, g.dh};
#pragma unroll
            for (int y = 0; y < 4; ++y)
                if (rows[y])
#pragma unroll
                    for (int i = 0; i < kWideChunks; ++i)
                        if (threadIdx.x + i * T < chunks)
                            asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<const uint4 *>(rows[y]) + base +
                                                                          (size_t)gridDim.x * chunks + threadIdx.x + i * T));
        }
#pragma unroll
        for (int i = 0; i < kWideChunks; ++i) {
            const int c = threadIdx.x + i * T;
            if (c < chunks) {
                if (a.y)
                    update_factor(a, c, f);
                grad_sums(hv[i], yv[i], xv[i], gv[i], weight(c), f, s2);
            }
        }
        float s[8];
        fold_sums(s2, s);
        const float total = block_sum8(s, red[flip]);
        flip ^= 1;
        float t[6];
#pragma unroll
        for (int i = 0; i < 6; ++i)
            t[i] = __shfl_sync(0xffffffffu, total, i);
        const RowGrad q = grad_factors(a, inv_d, t[0], t[1], t[2], t[3], t[4], t[5]);
#pragma unroll
        for (int i = 0; i < kWideChunks; ++i) {
            const int c = threadIdx.x + i * T;
            if (c < chunks) {
                if (a.y)
                    update_factor(a, c, f);
                f2 P[4], S[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    P[e] = column_pairs[e * chunks + c];
                    S[e] = column_pairs[(4 + e) * chunks + c];
                }
                uint4 dh, dy;
                grad_chunk(hv[i], yv[i], xv[i], gv[i], weight(c), f, q, P, S, dh, dy);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    column_pairs[e * chunks + c] = P[e];
                    column_pairs[(4 + e) * chunks + c] = S[e];
                }
                reinterpret_cast<uint4 *>(g.dh_in)[base + c] = dh;
                if (a.y)
                    reinterpret_cast<uint4 *>(g.dy)[base + c] = dy;
            }
        }
    }
    float *row = g.part + (size_t)blockIdx.x * (2 * a.D + 4);
    float dot[1] = {0.0f};
    for (int c = threadIdx.x; c < chunks; c += T) {
        f2 P[4], S[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            P[e] = column_pairs[e * chunks + c];
            S[e] = column_pairs[(4 + e) * chunks + c];
        }
        dot[0] += put_partials(a, row, c, P, S);
    }
    block_sum(dot, red[flip]);
    if (threadIdx.x == 0)
        row[2 * a.D] = dot[0];
}

// Sums the CTAs' partial rows column by column, in a fixed order.
constexpr int kColumnGroups = 16;

__global__ void residual_norm_columns_kernel(NormGradArgs g, int ctas)
{
    const NormArgs &a = g.f;
    tc::pdl_wait();
    const int stride = 2 * a.D + 4;
    __shared__ float part[kColumnGroups][33];
    const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane;   // 0 .. 2 D: P, S, then the single gate's sum
    float s = 0.0f;
    if (col <= 2 * a.D)
#pragma unroll 8
        for (int i = grp; i < ctas; i += kColumnGroups)
            s += g.part[(size_t)i * stride + col];
    part[grp][lane] = s;
    __syncthreads();
    if (grp != 0 || col > 2 * a.D)
        return;
#pragma unroll
    for (int i = 1; i < kColumnGroups; ++i)
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

// CTAs of the backward kernels that an SM holds, and how many have a row of partials.
int backward_ctas_per_sm(int D) { return D <= 512 ? 2 : D <= 1024 ? 6 : D <= 2048 ? 4 : D <= 4096 ? 2 : 1; }
int backward_ctas(int M, int D)
{
    const int most = backward_ctas_per_sm(D) * device_sm_count();
    return M < most ? M : most;
}

// Stages of a ring of n rows each, for `ctas` CTAs an SM.
int ring_stages(int D, int n, int ctas)
{
    const int fit = (220 * 1024 / ctas - 4096) / (n * D * 2);
    return fit < kRingStages ? fit : kRingStages;
}

// A kernel whose shared memory follows from the call's width: it is allowed all there is.
template <auto kernel, class... Args>
cudaError_t launch_big(int grid, int threads, size_t smem, cudaStream_t stream, Args... args)
{
    static std::atomic<unsigned long long> allowed;
    const cudaError_t e = tc::allow_smem(kernel, 224 * 1024, allowed);
    return e != cudaSuccess ? e : tc::launch_pdl(kernel, dim3(grid), dim3(threads), smem, stream, args...);
}

template <int GS, int NS>
cudaError_t launch_rows(const NormArgs &a, cudaStream_t stream)
{
    const int need = (a.M + kRowsThreads / GS - 1) / (kRowsThreads / GS), most = 4 * device_sm_count();
    return tc::launch_pdl(residual_norm_rows_kernel<GS, NS>, dim3(need < most ? need : most), dim3(kRowsThreads), 0, stream, a);
}

template <int GS, int NS>
cudaError_t launch_backward_rows(const NormGradArgs &g, int ctas, cudaStream_t stream)
{
    return tc::launch_pdl(residual_norm_backward_rows_kernel<GS, NS>, dim3(ctas), dim3(kRowsThreads), 2 * g.f.D * sizeof(float),
                          stream, g);
}

}  // namespace

cudaError_t launch_residual_norm(const NormArgs &a, cudaStream_t stream)
{
    const int sms = device_sm_count();
    if (a.D <= 1024) {
        return a.D <= 64    ? launch_rows<8, 1>(a, stream)
               : a.D <= 128 ? launch_rows<16, 1>(a, stream)
               : a.D <= 256 ? launch_rows<32, 1>(a, stream)
               : a.D <= 512 ? launch_rows<32, 2>(a, stream)
                            : launch_rows<32, 4>(a, stream);
    }
    if (a.M > 2 * sms) {
        const int n = a.y ? 2 : 1, per_sm = a.D <= 2048 ? 4 : a.D <= 4096 ? 2 : 1, stages = ring_stages(a.D, n, per_sm);
        const size_t smem = (size_t)stages * n * a.D * 2;
        return a.D <= 2048   ? launch_big<residual_norm_ring_kernel<2, 128>>(per_sm * sms, 128, smem, stream, a, stages)
               : a.D <= 4096 ? launch_big<residual_norm_ring_kernel<2, 256>>(per_sm * sms, 256, smem, stream, a, stages)
               : a.D <= 8192 ? launch_big<residual_norm_ring_kernel<2, 512>>(per_sm * sms, 512, smem, stream, a, stages)
                             : launch_big<residual_norm_ring_kernel<2, 1024>>(per_sm * sms, 1024, smem, stream, a, stages);
    }
    const int grid = a.M < 65536 ? a.M : 65536;
    if (a.D <= 8192)
        return tc::launch_pdl(residual_norm_kernel<2, 512>, dim3(grid), dim3(norm_threads(a.D, 2)), 0, stream, a);
    return tc::launch_pdl(residual_norm_kernel<2, 1024>, dim3(grid), dim3(norm_threads(a.D, 2)), 0, stream, a);
}

size_t residual_norm_backward_workspace(int64_t M, int64_t D)
{
    return (size_t)backward_ctas((int)M, (int)D) * (2 * (size_t)D + 4) * sizeof(float);
}

cudaError_t launch_residual_norm_backward(const NormGradArgs &g, cudaStream_t stream)
{
    const int D = g.f.D;
    int ctas = backward_ctas(g.f.M, D);
    cudaError_t e;
    if (D <= 512) {
        const int per = D <= 64 ? 32 : D <= 128 ? 16 : 8, need = (g.f.M + per - 1) / per;   // rows of a CTA at a time
        ctas = need < ctas ? need : ctas;
        e = D <= 64    ? launch_backward_rows<8, 1>(g, ctas, stream)
            : D <= 128 ? launch_backward_rows<16, 1>(g, ctas, stream)
            : D <= 256 ? launch_backward_rows<32, 1>(g, ctas, stream)
                       : launch_backward_rows<32, 2>(g, ctas, stream);
    } else if (D <= 8192) {
        const int n = 1 + (g.f.y != nullptr) + (g.dx != nullptr) + (g.dh != nullptr);
        const int stages = ring_stages(D, n, backward_ctas_per_sm(D));
        const size_t smem = (size_t)stages * n * D * 2;
        e = D <= 1024   ? launch_big<residual_norm_backward_ring_kernel<2, 64>>(ctas, 64, smem, stream, g, stages)
            : D <= 2048 ? launch_big<residual_norm_backward_ring_kernel<2, 128>>(ctas, 128, smem, stream, g, stages)
            : D <= 4096 ? launch_big<residual_norm_backward_ring_kernel<2, 256>>(ctas, 256, smem, stream, g, stages)
                        : launch_big<residual_norm_backward_ring_kernel<2, 512>>(ctas, 512, smem, stream, g, stages);
    } else {
        e = launch_big<residual_norm_backward_wide_kernel>(ctas, norm_threads(D, kWideChunks), (size_t)2 * D * sizeof(float),
                       stream, g);
    }
    if (e != cudaSuccess)
        return e;
    if (!g.dw_pre && !g.dw_post && !g.dgate)
        return cudaSuccess;
    return tc::launch_pdl(residual_norm_columns_kernel, dim3((2 * D + 1 + 31) / 32), dim3(32 * kColumnGroups), 0, stream, g, ctas);
}

}  // namespace s3d8

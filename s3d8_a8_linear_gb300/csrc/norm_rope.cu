// The norm of each query and key head with the rotation in the same pass, as tensors,
// and its gradients (s3d8_norm_rope, s3d8_norm_rope_backward).
//
//   r = rsqrt(mean x^2 + eps), y = x r w, z = R(position) y
//   dy = R^T dz, a = dy w, dx = r a - x r^3 mean(a x), dw = sum dy x r
//
// HBM-bound: 4 bytes an element forward, 6 backward.  A row of D columns belongs to
// D/16 neighbouring lanes, as in the append (rope_lane.cuh), so that the two sums of a
// row are a few shuffles and nothing else waits.  A warp takes a part of a token's rows
// and reads the token's cosines once; few tokens are cut into more parts.  The weights'
// gradients: a lane keeps its columns' sums in registers over all its rows, a CTA adds
// its lanes' in shared memory, a second kernel adds the CTAs' rows; every order is fixed,
// so equal inputs give equal bits.
#include "launch.h"
#include "rope_lane.cuh"
#include "tcgen05.cuh"

namespace s3d8 {

namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

struct Work {
    int parts;      // warps that share a token's rows
    int log_lanes, vec;
    int64_t items;  // tokens times parts
};

__device__ __forceinline__ const __nv_bfloat16 *row_of(const __nv_bfloat16 *const (&x)[2], const int64_t (&st)[2][2], int64_t t, int kind, int h)
{
    return x[kind] + t * st[kind][0] + h * st[kind][1];
}

// The position of token t; false for a padding token, or one without angles (recorded once).
__device__ __forceinline__ bool position(const NormRopeArgs &a, int64_t t, bool one, int64_t &pos)
{
    pos = a.positions ? a.positions[t] : t;
    if (pos < 0)
        return false;
    if (a.rotary && pos >= a.max_pos) {
        if (one)
            atomicExch(a.status, kStatusBounds);
        return false;
    }
    return true;
}

// ROWS: rows of a lane whose loads leave together.
template <int MODE, int ROWS>
__global__ __launch_bounds__(kThreads) void norm_rope_kernel(const __grid_constant__ NormRopeArgs a, const __grid_constant__ Work p)
{
    tc::pdl_launch_dependents();
    tc::pdl_wait();
    const RopeLane l(a.rotary, a.dim, MODE, p.log_lanes);
    const int slots = 32 >> p.log_lanes, slot = (threadIdx.x & 31) >> p.log_lanes, heads = a.heads[0] + a.heads[1];
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    for (int64_t item = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); item < p.items; item += (int64_t)gridDim.x * kWarps) {
        const int64_t t = item / p.parts;
        const int part = (int)(item - t * p.parts);
        float cs[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f}, sn[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
        int64_t pos = 0;
        bool ok = false;
        for (int base = part * slots * ROWS; base < heads; base += p.parts * slots * ROWS) {
            uint4 raw[ROWS][2];
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
                const int head = base + slot + i * slots, kind = head >= a.heads[0];
                raw[i][0] = raw[i][1] = zero;
                if (head < heads && l.in_row) {
                    const __nv_bfloat16 *x = row_of(a.x, a.xs, t, kind, kind ? head - a.heads[0] : head);
                    raw[i][0] = ldg_stream_v4(x + 8 * l.chunk[0]);
                    raw[i][1] = ldg_stream_v4(x + 8 * l.chunk[1]);
                }
            }
            if (base == part * slots * ROWS) {
                ok = position(a, t, part == 0 && (threadIdx.x & 31) == 0, pos);
                if (ok && l.turns && MODE != kHalvesOdd)
                    load_angles(l, a.cos + pos * l.half + 8 * l.lane, a.sin + pos * l.half + 8 * l.lane, p.vec, cs, sn);
            }
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
                const int head = base + slot + i * slots, kind = head >= a.heads[0], h = kind ? head - a.heads[0] : head;
                const bool live = head < heads && l.in_row;
                float f[2][8];
                unpack8(ok ? raw[i][0] : zero, f[0]);
                unpack8(ok ? raw[i][1] : zero, f[1]);
                float sum = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    sum = fmaf(f[0][e], f[0][e], fmaf(f[1][e], f[1][e], sum));
                const float r = rsqrtf(row_sum(sum, l.lanes) / (float)a.dim + a.eps);
                const __nv_bfloat16 *w = live && ok ? a.w[kind] : nullptr;
                if (w) {
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        float g[8];
                        unpack8(__ldg(reinterpret_cast<const uint4 *>(w) + l.chunk[y]), g);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            f[y][e] = f[y][e] * r * g[e];
                    }
                }
                if (l.turns)
                    turn<MODE>(l, f, cs, sn);
                if (MODE == kHalvesOdd && live && ok) {
                    const __nv_bfloat16 *x = row_of(a.x, a.xs, t, kind, h);
                    for (int e = 0; e < 16; ++e)
                        f[e / 8][e % 8] = turn_odd(16 * l.lane + e, l.half, f[e / 8][e % 8], a.cos + pos * l.half, a.sin + pos * l.half,
                                                   [&](int d) { return __bfloat162float(x[d]) * (w ? r * __bfloat162float(w[d]) : 1.0f); });
                }
                if (live) {
                    __nv_bfloat16 *o = a.out[kind] + (t * a.heads[kind] + h) * a.dim;
                    *reinterpret_cast<uint4 *>(o + 8 * l.chunk[0]) = pack8(f[0]);
                    *reinterpret_cast<uint4 *>(o + 8 * l.chunk[1]) = pack8(f[1]);
                }
            }
        }
    }
}

// A lane's share of one kind's rows (queries or keys) of a token.
template <int MODE, int ROWS>
__device__ __forceinline__ void back_rows(const NormRopeArgs &a, const Work &p, const RopeLane &l, int kind, int64_t t, int first, int step, bool ok,
                                          int64_t pos, const float (&cs)[8], const float (&sn)[8], const float (&w)[2][8], float (&dw)[2][8])
{
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    const int slots = 32 >> p.log_lanes, slot = (threadIdx.x & 31) >> p.log_lanes;
    for (int base = first; base < a.heads[kind]; base += step) {
        uint4 rx[ROWS][2], rz[ROWS][2];
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const int h = base + slot + i * slots;
            rx[i][0] = rx[i][1] = rz[i][0] = rz[i][1] = zero;
            if (ok && h < a.heads[kind] && l.in_row) {
                const __nv_bfloat16 *z = row_of(a.dz, a.dzs, t, kind, h), *x = row_of(a.x, a.xs, t, kind, h);
                rz[i][0] = ldg_stream_v4(z + 8 * l.chunk[0]);
                rz[i][1] = ldg_stream_v4(z + 8 * l.chunk[1]);
                if (a.w[kind]) {
                    rx[i][0] = ldg_stream_v4(x + 8 * l.chunk[0]);
                    rx[i][1] = ldg_stream_v4(x + 8 * l.chunk[1]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const int h = base + slot + i * slots;
            const bool live = h < a.heads[kind] && l.in_row;
            float f[2][8], x[2][8];
            unpack8(rz[i][0], f[0]);
            unpack8(rz[i][1], f[1]);
            unpack8(rx[i][0], x[0]);
            unpack8(rx[i][1], x[1]);
            if (l.turns)
                turn<MODE>(l, f, cs, sn);       // sn holds the sines with their signs turned
            if (MODE == kHalvesOdd && live && ok) {
                const __nv_bfloat16 *z = row_of(a.dz, a.dzs, t, kind, h);
                for (int e = 0; e < 16; ++e) {
                    const int d = 16 * l.lane + e;
                    const float *c = a.cos + pos * l.half, *s = a.sin + pos * l.half;
                    float &v = f[e / 8][e % 8];
                    if (d < l.half)
                        v = v * c[d] + __bfloat162float(z[d + l.half]) * s[d];
                    else if (d < a.rotary)
                        v = v * c[d - l.half] - __bfloat162float(z[d - l.half]) * s[d - l.half];
                }
            }
            if (a.w[kind]) {
                float sum = 0.0f, dot = 0.0f;
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        sum = fmaf(x[y][e], x[y][e], sum);
                        dot = fmaf(f[y][e] * w[y][e], x[y][e], dot);
                    }
                sum = row_sum(sum, l.lanes);
                dot = row_sum(dot, l.lanes);
                const float r = ok && h < a.heads[kind] ? rsqrtf(sum / (float)a.dim + a.eps) : 0.0f;   // no row: not 0 times infinity
                const float back = r * r * (dot / (float)a.dim);      // times r x: r^3 mean(a x) x
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        dw[y][e] = fmaf(f[y][e], x[y][e] * r, dw[y][e]);
                        f[y][e] = r * fmaf(-x[y][e], back, f[y][e] * w[y][e]);
                    }
            }
            if (live) {
                __nv_bfloat16 *o = a.out[kind] + (t * a.heads[kind] + h) * a.dim;
                *reinterpret_cast<uint4 *>(o + 8 * l.chunk[0]) = pack8(f[0]);
                *reinterpret_cast<uint4 *>(o + 8 * l.chunk[1]) = pack8(f[1]);
            }
        }
    }
}

// gridDim.x partial rows [2][dim] of the weights' gradients into a.part.
template <int MODE, int ROWS>
__global__ __launch_bounds__(kThreads) void norm_rope_backward_kernel(const __grid_constant__ NormRopeArgs a, const __grid_constant__ Work p)
{
    __shared__ float sums[2][kWarps][512];      // of a warp: its slots' columns side by side
    tc::pdl_launch_dependents();
    tc::pdl_wait();
    const RopeLane l(a.rotary, a.dim, MODE, p.log_lanes);
    const int slots = 32 >> p.log_lanes, slot = (threadIdx.x & 31) >> p.log_lanes, warp = threadIdx.x >> 5;
    float w[2][2][8], dw[2][2][8];
#pragma unroll
    for (int kind = 0; kind < 2; ++kind)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            unpack8(a.w[kind] && l.in_row ? __ldg(reinterpret_cast<const uint4 *>(a.w[kind]) + l.chunk[y]) : make_uint4(0u, 0u, 0u, 0u), w[kind][y]);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                dw[kind][y][e] = 0.0f;
        }
    for (int64_t item = (int64_t)blockIdx.x * kWarps + warp; item < p.items; item += (int64_t)gridDim.x * kWarps) {
        const int64_t t = item / p.parts;
        const int part = (int)(item - t * p.parts);
        float cs[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f}, sn[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
        int64_t pos;
        const bool ok = position(a, t, part == 0 && (threadIdx.x & 31) == 0, pos);
        if (ok && l.turns && MODE != kHalvesOdd) {
            load_angles(l, a.cos + pos * l.half + 8 * l.lane, a.sin + pos * l.half + 8 * l.lane, p.vec, cs, sn);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                sn[e] = -sn[e];
        }
        back_rows<MODE, ROWS>(a, p, l, 0, t, part * slots * ROWS, p.parts * slots * ROWS, ok, pos, cs, sn, w[0], dw[0]);
        back_rows<MODE, ROWS>(a, p, l, 1, t, part * slots * ROWS, p.parts * slots * ROWS, ok, pos, cs, sn, w[1], dw[1]);
    }
    // columns of a warp's slots, then of the warps, each in order
#pragma unroll
    for (int kind = 0; kind < 2; ++kind)
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (l.in_row)
                    sums[kind][warp][slot * (16 << p.log_lanes) + 8 * l.chunk[y] + e] = dw[kind][y][e];
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * a.dim; i += kThreads) {
        const int kind = i >= a.dim, d = kind ? i - a.dim : i;
        float s = 0.0f;
        for (int x = 0; x < kWarps; ++x)
            for (int y = 0; y < slots; ++y)
                s += sums[kind][x][y * (16 << p.log_lanes) + d];
        a.part[(int64_t)blockIdx.x * 2 * a.dim + i] = s;
    }
}

// Adds the CTAs' partial rows: a block 32 columns, its eight warps a share of the rows each.
__global__ __launch_bounds__(kThreads) void norm_rope_weights_kernel(const __grid_constant__ NormRopeArgs a, int rows)
{
    __shared__ float sums[kWarps][32];
    tc::pdl_launch_dependents();
    tc::pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, i = blockIdx.x * 32 + lane;
    float s = 0.0f;
    if (i < 2 * a.dim)
        for (int r = warp; r < rows; r += kWarps)
            s += a.part[(int64_t)r * 2 * a.dim + i];
    sums[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && i < 2 * a.dim) {
        for (int x = 1; x < kWarps; ++x)
            s += sums[x][lane];
        const int kind = i >= a.dim;
        if (a.dw[kind])
            a.dw[kind][kind ? i - a.dim : i] = s;
    }
}

Work plan(const NormRopeArgs &a, int rows)
{
    Work p;
    p.log_lanes = 0;
    while (16 << p.log_lanes < a.dim)
        ++p.log_lanes;
    p.vec = a.rotary % 16 == 0 && ((uintptr_t)a.cos & 15) == 0 && ((uintptr_t)a.sin & 15) == 0;
    // as many warps a token as its rows have loads for, as long as the GPU has room for them
    const int heads = a.heads[0] > a.heads[1] ? a.heads[0] : a.heads[1], each = (32 >> p.log_lanes) * rows;
    const int64_t most = (heads + each - 1) / each, room = (int64_t)device_sm_count() * 32 / (a.T > 0 ? a.T : 1);
    p.parts = (int)(room < 1 ? 1 : room < most ? room : most);
    p.items = a.T * p.parts;
    return p;
}

int grid_of(const Work &p, int ctas)
{
    const int64_t need = (p.items + kWarps - 1) / kWarps, most = (int64_t)device_sm_count() * ctas;
    return (int)(need < most ? need : most);
}

constexpr int kBackCtas = 2;     // an SM

template <int MODE>
cudaError_t forward(const NormRopeArgs &a, cudaStream_t stream)
{
    const Work p = plan(a, 4);
    return tc::launch_pdl(norm_rope_kernel<MODE, 4>, dim3(grid_of(p, 8)), dim3(kThreads), 0, stream, a, p);
}

template <int MODE>
cudaError_t backward(const NormRopeArgs &a, cudaStream_t stream)
{
    const Work p = plan(a, 2);
    const int grid = grid_of(p, kBackCtas);
    cudaError_t e = tc::launch_pdl(norm_rope_backward_kernel<MODE, 2>, dim3(grid), dim3(kThreads), 0, stream, a, p);
    if (e == cudaSuccess && (a.dw[0] || a.dw[1]))
        e = tc::launch_pdl(norm_rope_weights_kernel, dim3((2 * a.dim + 31) / 32), dim3(kThreads), 0, stream, a, grid);
    return e;
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs &a, cudaStream_t stream)
{
    if (a.interleaved)
        return forward<kNeighbours>(a, stream);
    return a.rotary % 16 == 0 ? forward<kHalves>(a, stream) : forward<kHalvesOdd>(a, stream);
}

size_t norm_rope_backward_workspace(int64_t, int, int dim) { return (size_t)device_sm_count() * kBackCtas * 2 * dim * sizeof(float); }

cudaError_t launch_norm_rope_backward(const NormRopeArgs &a, cudaStream_t stream)
{
    if (a.interleaved)
        return backward<kNeighbours>(a, stream);
    return a.rotary % 16 == 0 ? backward<kHalves>(a, stream) : backward<kHalvesOdd>(a, stream);
}

}  // namespace s3d8

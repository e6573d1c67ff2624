// The norm of each query and key head with the rotation in the same pass, as tensors,
// and its gradients (s3d8_norm_rope, s3d8_norm_rope_backward).
//
//   r = rsqrt(mean x^2 + eps), y = x r w, z = R(position) y
//   dy = R^T dz, a = dy w, dx = r a - x r^3 mean(a x), dw = sum dy x r
//
// HBM-bound: 4 bytes an element forward, 6 backward.  A row of D columns belongs to
// D/16 neighbouring lanes, as in the append (rope_lane.cuh), so that the two sums of a
// row are a few shuffles and nothing else waits; a warp has 32 lanes' worth of one token's
// rows at a time, a group.  Queries and keys are CTAs of their own, by their share of the
// rows (a warp keeps one weight's columns in registers, and one weight's sums), and each
// warp an equal run of its kind's groups.  It copies them through a ring of its own in
// shared memory, the token's angles with the first group of a token, five groups (backward
// three) in flight beside the one in use: what bounds it is HBM and, backward, the issue slots
// (70% busy). Measured: 25616 tokens of 8 heads of 128 in 22.5 to 23 us (4.6 TB/s of what it
// has to move; 33.5 with each warp waiting for the rows that it had asked for), 8191 tokens of
// 32 + 8 heads with rotation in 32 us (5.4 TB/s) and their gradients in 54 us (4.7 TB/s; 82.6).
// Shorter runs in two rounds of CTAs measured 25.6 and 56.6 us, four CTAs of 128 threads an SM
// 22.9 and 55.4.
//
// The weights' gradients: a lane keeps its columns' sums in registers over all its rows,
// a CTA adds its lanes' in shared memory, a second kernel adds the CTAs' rows; every order
// is fixed, so equal inputs give equal bits.  All arithmetic is fp32, rounded once.
#include "async_copy.cuh"
#include "cross_tiles.cuh"
#include "launch.h"
#include "rope_lane.cuh"
#include "tcgen05.cuh"
#include "uniform.cuh"

namespace s3d8 {

namespace {

using cross::add2;
using cross::fma2;
using cross::mul2;
using cross::pack2;

constexpr int kThreads = 512, kWarps = kThreads / 32;

struct Work {
    int log_lanes, vec;
    int ctas[2];    // of the queries, of the keys
};

template <bool BACK>
struct Ring {
    static constexpr int STAGES = BACK ? 4 : 6;
    static constexpr int DZ = 1024, ANGLES = BACK ? 2048 : 1024, STAGE = ANGLES + 1024;     // x first; cosines, sines
    static constexpr int BYTES = kWarps * STAGES * STAGE;
};

__device__ __forceinline__ float2 twice(float x) { return make_float2(x, x); }

// Sixteen values: two chunks of four pairs.
__device__ __forceinline__ void unpack(uint4 v, float2 (&f)[4])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
        f[j] = make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u));
}

__device__ __forceinline__ uint4 pack(const float2 (&f)[4])
{
    return make_uint4(pack2(f[0].x, f[0].y), pack2(f[1].x, f[1].y), pack2(f[2].x, f[2].y), pack2(f[3].x, f[3].y));
}

__device__ __forceinline__ float lds_f32(uint32_t at)
{
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at));
    return v;
}

// What a warp has to copy: a run of its kind's groups, in order of token and head.
template <int MODE, bool BACK>
struct Feed {
    using R = Ring<BACK>;
    const NormRopeArgs &a;
    const RopeLane &l;
    const int kind, slots, groups, vec;
    const uint32_t ring, angles;    // this lane's place in it, and the angles'
    int64_t left, t;
    int group, stage, next;
    bool fresh, ok;

    __device__ __forceinline__ Feed(const NormRopeArgs &a, const RopeLane &l, int kind, int slots, int slot, int vec, uint32_t ring, uint32_t angles, int64_t begin, int64_t n)
        : a(a), l(l), kind(kind), slots(slots), groups((a.heads[kind] + slots - 1) / slots), vec(vec), ring(ring), angles(angles), left(n), t(begin / groups),
          group((int)(begin - t * groups)), stage(0), next(0), fresh(true), ok(false)
    {
        if (a.positions && n > 0)
            next = __ldg(a.positions + t);
        head = group * slots + slot;
    }

    // Copies a group, if one is left; whether its token has a place.
    __device__ __forceinline__ bool operator()()
    {
        if (left > 0) {
            const uint32_t to = ring + stage * R::STAGE;
            const bool live = head < a.heads[kind] && l.in_row;
            const __nv_bfloat16 *x = a.x[kind] + t * a.xs[kind][0] + (live ? head * a.xs[kind][1] : 0);
            if (!BACK || a.w[kind]) {
                cp_async16(to, x + (live ? 8 * l.chunk[0] : 0), live ? 16 : 0);
                cp_async16(to + 512, x + (live ? 8 * l.chunk[1] : 0), live ? 16 : 0);
            }
            if (BACK) {
                const __nv_bfloat16 *z = a.dz[kind] + t * a.dzs[kind][0] + (live ? head * a.dzs[kind][1] : 0);
                cp_async16(to + R::DZ, z + (live ? 8 * l.chunk[0] : 0), live ? 16 : 0);
                cp_async16(to + R::DZ + 512, z + (live ? 8 * l.chunk[1] : 0), live ? 16 : 0);
            }
            if (fresh) {
                const int64_t pos = a.positions ? uniform(next) : t;
                if (a.positions && t + 1 < a.T)
                    next = __ldg(a.positions + t + 1);
                ok = pos >= 0;
                if (ok && a.rotary && pos >= a.max_pos) {
                    ok = false;
                    atomicExch(a.status, kStatusBounds);
                }
                if (ok && MODE != kHalvesOdd) {
                    const float *c = a.cos + pos * l.half, *s = a.sin + pos * l.half;
                    const int lane = threadIdx.x & 31, n = l.half;
                    if (vec) {
                        for (int i = lane; i < n / 2; i += 32)
                            cp_async16(angles + stage * R::STAGE + 16 * i, 4 * i < n ? c + 4 * i : s + 4 * i - n);
                    } else {
                        for (int i = lane; i < 2 * n; i += 32)
                            cp_async4(angles + stage * R::STAGE + 4 * i, i < n ? c + i : s + i - n, 4);
                    }
                }
                fresh = false;
            }
            head += slots;
            if (++group == groups) {
                head -= groups * slots;
                group = 0;
                ++t;
                fresh = true;
            }
            --left;
            stage = stage + 1 == R::STAGES ? 0 : stage + 1;
        }
        cp_commit();
        return ok;
    }

private:
    int head;
};

// BACK: gridDim.x partial rows [dim] of the weights' gradients into a.part, those of the queries' CTAs first.
template <int MODE, bool BACK>
__global__ __launch_bounds__(kThreads, 1) void norm_rope_kernel(const __grid_constant__ NormRopeArgs a, const __grid_constant__ Work p)
{
    using R = Ring<BACK>;
    extern __shared__ __align__(16) unsigned char norm_rope_mem[];
    const int warp = warp_index(), kind = (int)blockIdx.x >= p.ctas[0];
    const RopeLane l(a.rotary, a.dim, MODE, p.log_lanes);
    const int slots = 32 >> p.log_lanes, slot = (threadIdx.x & 31) >> p.log_lanes, heads = a.heads[kind], groups = (heads + slots - 1) / slots;
    const int64_t total = a.T * groups, part = (int64_t)(blockIdx.x - (kind ? p.ctas[0] : 0)) * kWarps + warp, parts = (int64_t)p.ctas[kind] * kWarps;
    const int64_t begin = total * part / parts, end = total * (part + 1) / parts;
    const uint32_t warps = smem_addr(norm_rope_mem) + warp * (R::STAGES * R::STAGE), ring = warps + (threadIdx.x & 31) * 16, angles = warps + R::ANGLES;
    const float inv = 1.0f / (float)a.dim;
    const bool normed = a.w[kind] != nullptr;
    tc::pdl_launch_dependents();
    tc::pdl_wait();
    float2 w[2][4], dw[2][4], cs[4], sn[4];
#pragma unroll
    for (int y = 0; y < 2; ++y) {
        unpack(normed && l.in_row ? __ldg(reinterpret_cast<const uint4 *>(a.w[kind]) + l.chunk[y]) : make_uint4(0u, 0u, 0u, 0u), w[y]);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            dw[y][e] = make_float2(0.0f, 0.0f);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        cs[e] = sn[e] = make_float2(0.0f, 0.0f);

    Feed<MODE, BACK> feed(a, l, kind, slots, slot, p.vec, ring, angles, begin, end - begin);
    int64_t t = begin / groups;
    int group = (int)(begin - t * groups), stage = 0;
    unsigned places = 0;        // of the groups in the ring: whether their token has one, the newest lowest
#pragma unroll
    for (int i = 0; i < R::STAGES - 1; ++i)
        places = places << 1 | feed();
    bool fresh = true;
    for (int64_t i = begin; i < end; ++i) {
        cp_wait<R::STAGES - 2>();
        __syncwarp();               // the angles are other lanes' copies, and the stage filled next is read
        places = places << 1 | feed();
        const bool ok = places >> (R::STAGES - 1) & 1;
        const int h = group * slots + slot;
        const bool live = h < heads && l.in_row;
        const uint32_t from = ring + stage * R::STAGE;
        float2 f[2][4], x[2][4];
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        if (!BACK || normed) {
            unpack(ok ? lds_v4(from) : zero, x[0]);
            unpack(ok ? lds_v4(from + 512) : zero, x[1]);
        }
        if (BACK) {
            unpack(ok ? lds_v4(from + R::DZ) : zero, f[0]);
            unpack(ok ? lds_v4(from + R::DZ + 512) : zero, f[1]);
        }
        if (fresh && ok && l.turns && MODE != kHalvesOdd) {
            // (beyond half, where it is no multiple of 8: not used)
            const uint32_t at = angles + stage * R::STAGE + 32 * l.lane;
            float c[8], sine[8];
            if (p.vec) {
#pragma unroll
                for (int e = 0; e < 8; e += 4) {
                    const uint4 u = lds_v4(at + 4 * e), v = lds_v4(at + 4 * (l.half + e));
                    c[e] = __uint_as_float(u.x), c[e + 1] = __uint_as_float(u.y), c[e + 2] = __uint_as_float(u.z), c[e + 3] = __uint_as_float(u.w);
                    sine[e] = __uint_as_float(v.x), sine[e + 1] = __uint_as_float(v.y), sine[e + 2] = __uint_as_float(v.z), sine[e + 3] = __uint_as_float(v.w);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    c[e] = lds_f32(at + 4 * e);
                    sine[e] = lds_f32(at + 4 * (l.half + e));
                }
            }
            const float by = BACK ? -1.0f : 1.0f;       // the gradient turns back
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                cs[e] = make_float2(c[2 * e], c[2 * e + 1]);
                sn[e] = make_float2(sine[2 * e] * by, sine[2 * e + 1] * by);
            }
        }
        float r = 0.0f;
        if (!BACK) {
            float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    sum = fma2(x[y][e], x[y][e], sum);
                    f[y][e] = x[y][e];
                }
            r = rsqrtf(fmaf(row_sum(sum.x + sum.y, l.lanes), inv, a.eps));
            if (normed && ok && live) {
#pragma unroll
                for (int y = 0; y < 2; ++y)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        f[y][e] = mul2(mul2(f[y][e], twice(r)), w[y][e]);
            }
        }
        if (l.turns && MODE == kHalves) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 u = f[0][e], v = f[1][e];
                f[0][e] = fma2(u, cs[e], mul2(v, make_float2(-sn[e].x, -sn[e].y)));
                f[1][e] = fma2(v, cs[e], mul2(u, sn[e]));
            }
        }
        if (l.turns && MODE == kNeighbours) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {     // pair 8 lane + e
                if (8 * l.lane + e >= l.half)
                    continue;
                const float2 u = f[e / 4][e % 4];
                const float c = e & 1 ? cs[e / 2].y : cs[e / 2].x, s = e & 1 ? sn[e / 2].y : sn[e / 2].x;
                f[e / 4][e % 4] = make_float2(fmaf(u.x, c, -(u.y * s)), fmaf(u.y, c, u.x * s));
            }
        }
        if (MODE == kHalvesOdd && live && ok && a.rotary) {
            const int64_t pos = a.positions ? __ldg(a.positions + t) : t;
            const float *c = a.cos + pos * l.half, *s = a.sin + pos * l.half;
            const __nv_bfloat16 *row = BACK ? a.dz[kind] + t * a.dzs[kind][0] + h * a.dzs[kind][1] : a.x[kind] + t * a.xs[kind][0] + h * a.xs[kind][1];
            auto partner = [&](int d) { return __bfloat162float(row[d]) * (BACK || !normed ? 1.0f : r * __bfloat162float(a.w[kind][d])); };
            auto turned = [&](int d, float v) {
                if (d < l.half)
                    return v * c[d] + partner(d + l.half) * (BACK ? s[d] : -s[d]);
                return d < a.rotary ? v * c[d - l.half] + partner(d - l.half) * (BACK ? -s[d - l.half] : s[d - l.half]) : v;
            };
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int d = 16 * l.lane + 2 * e;
                f[e / 4][e % 4] = make_float2(turned(d, f[e / 4][e % 4].x), turned(d + 1, f[e / 4][e % 4].y));
            }
        }
        if (BACK && normed) {
            float2 sum = make_float2(0.0f, 0.0f), dot = make_float2(0.0f, 0.0f), g[2][4];
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    g[y][e] = mul2(f[y][e], w[y][e]);
                    sum = fma2(x[y][e], x[y][e], sum);
                    dot = fma2(g[y][e], x[y][e], dot);
                }
            const float squares = row_sum(sum.x + sum.y, l.lanes), back = row_sum(dot.x + dot.y, l.lanes);
            r = ok && h < heads ? rsqrtf(fmaf(squares, inv, a.eps)) : 0.0f;   // no row: not 0 times infinity
            // from the mean outwards: r^2 alone passes fp32's range for rows below 5e-20
            const float2 r2 = twice(r), by = twice(-(r * (r * (back * inv))));
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    dw[y][e] = fma2(f[y][e], mul2(x[y][e], r2), dw[y][e]);
                    f[y][e] = mul2(r2, fma2(x[y][e], by, g[y][e]));
                }
        }
        if (live) {
            uint4 *o = reinterpret_cast<uint4 *>(a.out[kind] + (t * heads + h) * a.dim);
            o[l.chunk[0]] = pack(f[0]);
            o[l.chunk[1]] = pack(f[1]);
        }
        fresh = false;
        if (++group == groups) {
            group = 0;
            ++t;
            fresh = true;
        }
        stage = stage + 1 == R::STAGES ? 0 : stage + 1;
    }
    cp_wait<0>();
    if (!BACK)
        return;
    // columns of a warp's slots, then of the warps, each in order
    float *sums = reinterpret_cast<float *>(norm_rope_mem);     // [kWarps][512]: a warp's slots side by side
    __syncthreads();
#pragma unroll
    for (int y = 0; y < 2; ++y)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (l.in_row)
                *reinterpret_cast<float2 *>(sums + warp * 512 + slot * (16 << p.log_lanes) + 8 * l.chunk[y] + 2 * e) = dw[y][e];
    __syncthreads();
    for (int d = threadIdx.x; d < a.dim; d += kThreads) {
        float s = 0.0f;
        for (int x = 0; x < kWarps; ++x)
            for (int y = 0; y < slots; ++y)
                s += sums[x * 512 + y * (16 << p.log_lanes) + d];
        a.part[(int64_t)blockIdx.x * a.dim + d] = s;
    }
}

constexpr int kSumWarps = 8;

// Adds the CTAs' partial rows: a block 32 columns of a kind, its eight warps a share of the rows each.
__global__ __launch_bounds__(kSumWarps * 32) void norm_rope_weights_kernel(const __grid_constant__ NormRopeArgs a, const __grid_constant__ Work p)
{
    __shared__ float sums[kSumWarps][32];
    tc::pdl_launch_dependents();
    tc::pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, i = blockIdx.x * 32 + lane, kind = blockIdx.y;
    const int first = kind ? p.ctas[0] : 0;
    float s = 0.0f;
    if (i < a.dim)
        for (int r = warp; r < p.ctas[kind]; r += kSumWarps)
            s += a.part[(int64_t)(first + r) * a.dim + i];
    sums[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && i < a.dim) {
        for (int x = 1; x < kSumWarps; ++x)
            s += sums[x][lane];
        if (a.dw[kind])
            a.dw[kind][i] = s;
    }
}

Work plan(const NormRopeArgs &a)
{
    Work p;
    p.log_lanes = 0;
    while (16 << p.log_lanes < a.dim)
        ++p.log_lanes;
    p.vec = a.rotary % 16 == 0 && ((uintptr_t)a.cos & 15) == 0 && ((uintptr_t)a.sin & 15) == 0;
    const int slots = 32 >> p.log_lanes;
    int64_t groups[2];
    for (int kind = 0; kind < 2; ++kind)
        groups[kind] = a.T * ((a.heads[kind] + slots - 1) / slots);
    const int64_t all = groups[0] + groups[1], need = (all + kWarps - 1) / kWarps, most = device_sm_count();
    const int ctas = (int)(need < most ? need : most);
    p.ctas[1] = groups[1] == 0 ? 0 : (int)((groups[1] * ctas + all / 2) / all);
    if (groups[1] > 0 && p.ctas[1] == 0)
        p.ctas[1] = 1;
    p.ctas[0] = ctas > p.ctas[1] ? ctas - p.ctas[1] : 1;        // (together at most one more than the SMs)
    return p;
}

template <int MODE, bool BACK>
cudaError_t run(const NormRopeArgs &a, cudaStream_t stream)
{
    using R = Ring<BACK>;
    const Work p = plan(a);
    static std::atomic<unsigned long long> allowed;
    cudaError_t e = tc::allow_smem(norm_rope_kernel<MODE, BACK>, R::BYTES, allowed);
    if (e == cudaSuccess)
        e = tc::launch_pdl(norm_rope_kernel<MODE, BACK>, dim3(p.ctas[0] + p.ctas[1]), dim3(kThreads), R::BYTES, stream, a, p);
    if (BACK && e == cudaSuccess && (a.dw[0] || a.dw[1]))
        e = tc::launch_pdl(norm_rope_weights_kernel, dim3((a.dim + 31) / 32, 2), dim3(kSumWarps * 32), 0, stream, a, p);
    return e;
}

template <bool BACK>
cudaError_t run_mode(const NormRopeArgs &a, cudaStream_t stream)
{
    if (a.interleaved)
        return run<kNeighbours, BACK>(a, stream);
    return a.rotary % 16 == 0 ? run<kHalves, BACK>(a, stream) : run<kHalvesOdd, BACK>(a, stream);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs &a, cudaStream_t stream) { return run_mode<false>(a, stream); }

size_t norm_rope_backward_workspace(int64_t, int, int dim) { return (size_t)(device_sm_count() + 1) * dim * sizeof(float); }

cudaError_t launch_norm_rope_backward(const NormRopeArgs &a, cudaStream_t stream) { return run_mode<true>(a, stream); }

}  // namespace s3d8

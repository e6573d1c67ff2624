// Attention of one new token per sequence over the paged cache: the join of the
// sequences that were cut, and the dispatch (the kernel is in paged_attention.cuh).
#include "paged_attention.cuh"

namespace s3d8 {

namespace {

using namespace attn;

// Joins the parts of every sequence that was cut: block (unit of a sequence, query
// row or four of them), of 16 warps over one row's parts or four of a row each.  Run `first` left its part in its
// second slot, the runs behind it in their first.
// BATCH: parts whose loads leave together.
template <int DP, int kJoinWarps, int BATCH>
__global__ __launch_bounds__(kJoinWarps * 32) void paged_attention_join_kernel(const __grid_constant__ AttnArgs a,
                                                                             const __grid_constant__ AttnPlan p)
{
    constexpr int V = DP > 128 ? DP / 128 : 1;    // 16-byte pieces of a row in a lane
    __shared__ __align__(16) float sums[kJoinWarps][DP];
    __shared__ float tops[kJoinWarps], totals[kJoinWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, D = a.kv.dim;
    tc::pdl_launch_dependents();
    tc::pdl_wait();
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0)
        *p.queue = kQueueTag << 32;
    const int2 join = p.joins[blockIdx.x];
    if (join.x < 0)
        return;
    const int b = blockIdx.x / p.units, u = blockIdx.x % p.units, h = u / p.blocks, blk = u % p.blocks;
    const int rows = min(p.group - blk * 16, p.rows), count = join.y - join.x + 1;
    const size_t size = part_floats(p.rows, D);
    const float *parts = p.parts + (size_t)join.x * 2 * size;
    auto part = [&](int x) { return parts + (size_t)(2 * x + (x == 0)) * size; };
    auto rows_of_warps = [&]() {                  // a query row a warp, its parts in batches
        for (int r = blockIdx.y + warp * gridDim.y; r < rows; r += gridDim.y * kJoinWarps) {
            float top = -INFINITY, sum = 0.0f;
            float4 acc[V];
#pragma unroll
            for (int y = 0; y < V; ++y)
                acc[y] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            for (int x0 = 0; x0 < count; x0 += BATCH) {
                float2 ml = make_float2(-INFINITY, 0.0f);
                if (lane < BATCH && x0 + lane < count)
                    ml = *reinterpret_cast<const float2 *>(part(x0 + lane) + p.rows * D + 2 * r);
                float4 o[BATCH][V];
#pragma unroll
                for (int i = 0; i < BATCH; ++i)
#pragma unroll
                    for (int y = 0; y < V; ++y) {
                        o[i][y] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        if (x0 + i < count && 128 * y + 4 * lane < D)
                            o[i][y] = *reinterpret_cast<const float4 *>(part(x0 + i) + r * D + 128 * y + 4 * lane);
                    }
                float now = ml.x;
#pragma unroll
                for (int s = BATCH / 2; s > 0; s >>= 1)
                    now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, s));
                now = fmaxf(top, __shfl_sync(0xffffffffu, now, 0));
                const float zero = now == -INFINITY ? 0.0f : now;
                const float keep = ex2(top - zero), w = ex2(ml.x - zero), lw = ml.y * w;
                top = now;
                sum *= keep;
#pragma unroll
                for (int y = 0; y < V; ++y)
                    acc[y] = make_float4(acc[y].x * keep, acc[y].y * keep, acc[y].z * keep, acc[y].w * keep);
#pragma unroll
                for (int i = 0; i < BATCH; ++i) {
                    sum += __shfl_sync(0xffffffffu, lw, i);
                    const float wi = __shfl_sync(0xffffffffu, w, i);
#pragma unroll
                    for (int y = 0; y < V; ++y)
                        acc[y] = make_float4(fmaf(wi, o[i][y].x, acc[y].x), fmaf(wi, o[i][y].y, acc[y].y),
                                             fmaf(wi, o[i][y].z, acc[y].z), fmaf(wi, o[i][y].w, acc[y].w));
                }
            }
            const int64_t row = (int64_t)b * a.Hq + h * p.group + blk * 16 + r;
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
            for (int y = 0; y < V; ++y)
                if (128 * y + 4 * lane < D) {
                    const __nv_bfloat162 lo = __floats2bfloat162_rn(acc[y].x * inv, acc[y].y * inv);
                    const __nv_bfloat162 hi = __floats2bfloat162_rn(acc[y].z * inv, acc[y].w * inv);
                    *reinterpret_cast<uint2 *>(a.out + row * D + 128 * y + 4 * lane) =
                        make_uint2(*reinterpret_cast<const uint32_t *>(&lo), *reinterpret_cast<const uint32_t *>(&hi));
                }
            if (lane == 0 && a.lse)
                a.lse[row] = (top + log2f(sum)) * kLn2;
        }
    };
    if constexpr (kJoinWarps < 16) {
        rows_of_warps();
        return;
    } else {
        if (count <= BATCH) {
            rows_of_warps();
            return;
        }
        for (int r = blockIdx.y; r < rows; r += gridDim.y) {
            // this warp's parts, 32 at a time: lane i has the weight of part x0 + i kJoinWarps
            float top = -INFINITY, sum = 0.0f;
            float4 acc[V];
#pragma unroll
            for (int y = 0; y < V; ++y)
                acc[y] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            for (int x0 = warp; x0 < count; x0 += 32 * kJoinWarps) {
                const int x = x0 + lane * kJoinWarps, some = min(32, (count - x0 + kJoinWarps - 1) / kJoinWarps);
                float mx = -INFINITY, lx = 0.0f;
                if (x < count) {
                    const float2 ml = *reinterpret_cast<const float2 *>(part(x) + p.rows * D + 2 * r);
                    mx = ml.x;
                    lx = ml.y;
                }
                float4 o[BATCH][V];
                auto load = [&](int i0) {
#pragma unroll
                    for (int i = 0; i < BATCH; ++i)
#pragma unroll
                        for (int y = 0; y < V; ++y) {
                            o[i][y] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                            if (i0 + i < some && 128 * y + 4 * lane < D)
                                o[i][y] = *reinterpret_cast<const float4 *>(part(x0 + (i0 + i) * kJoinWarps) + r * D + 128 * y + 4 * lane);
                        }
                };
                load(0);
                float now = mx;
#pragma unroll
                for (int s = 16; s > 0; s >>= 1)
                    now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, s));
                now = fmaxf(top, now);
                const float zero = now == -INFINITY ? 0.0f : now;
                const float keep = ex2(top - zero), w = ex2(mx - zero);
                lx *= w;
#pragma unroll
                for (int s = 16; s > 0; s >>= 1)
                    lx += __shfl_xor_sync(0xffffffffu, lx, s);
                sum = sum * keep + lx;
                top = now;
#pragma unroll
                for (int y = 0; y < V; ++y)
                    acc[y] = make_float4(acc[y].x * keep, acc[y].y * keep, acc[y].z * keep, acc[y].w * keep);
                for (int i0 = 0; i0 < some; i0 += BATCH) {
                    if (i0)
                        load(i0);
#pragma unroll
                    for (int i = 0; i < BATCH; ++i) {
                        // a part beyond the last has a weight of 2^-inf, and zeros
                        const float wi = __shfl_sync(0xffffffffu, w, i0 + i);
#pragma unroll
                        for (int y = 0; y < V; ++y)
                            acc[y] = make_float4(fmaf(wi, o[i][y].x, acc[y].x), fmaf(wi, o[i][y].y, acc[y].y),
                                                 fmaf(wi, o[i][y].z, acc[y].z), fmaf(wi, o[i][y].w, acc[y].w));
                    }
                }
            }
            __syncthreads();                          // the row before has been read
            if (lane == 0) {
                tops[warp] = top;
                totals[warp] = sum;
            }
#pragma unroll
            for (int y = 0; y < V; ++y)
                if (128 * y + 4 * lane < DP)
                    *reinterpret_cast<float4 *>(&sums[warp][128 * y + 4 * lane]) = acc[y];
            __syncthreads();
            float all = -INFINITY, total = 0.0f;
#pragma unroll
            for (int x = 0; x < kJoinWarps; ++x)
                all = fmaxf(all, tops[x]);
            const float zero = all == -INFINITY ? 0.0f : all;
#pragma unroll
            for (int x = 0; x < kJoinWarps; ++x)
                total = fmaf(ex2(tops[x] - zero), totals[x], total);
            const int64_t row = (int64_t)b * a.Hq + h * p.group + blk * 16 + r;
            for (int d = threadIdx.x; d < D; d += kJoinWarps * 32) {
                float v = 0.0f;
#pragma unroll
                for (int x = 0; x < kJoinWarps; ++x)
                    v = fmaf(ex2(tops[x] - zero), sums[x][d], v);
                a.out[row * D + d] = __float2bfloat16_rn(total == 0.0f ? 0.0f : v / total);
            }
            if (threadIdx.x == 0 && a.lse)
                a.lse[row] = (all + log2f(total)) * kLn2;
        }
    }
}

template <int DP>
cudaError_t launch_join(const AttnArgs &a, const AttnPlan &p, cudaStream_t stream)
{
    // Few units of sequences that can be long: dozens of parts each, so 16 warps a query row, and all of their loads at once
    // where there is an SM for every row (one sequence of 60000 tokens 56 -> 53 us; 32 of up to 16000 186 -> 180).  Many
    // units, or short sequences: few parts, a warp a query row (32 of up to 100 tokens 12.6 -> 10.4 us).
    const unsigned units = (unsigned)a.B * p.units, sms = device_sm_count();
    int64_t longest = a.width * a.kv.page_size;
    longest = a.window > 0 && a.window < longest ? a.window : longest;
    if ((int64_t)units * p.rows > 4 * sms && (units > 2 * sms || longest <= 32 * kTile))
        return tc::launch_pdl(paged_attention_join_kernel<DP, 4, 8>, dim3(units, (p.rows + 3) / 4), dim3(4 * 32), 0, stream, a,
                              p);
    if (DP <= 128 && units * p.rows <= sms)
        return tc::launch_pdl(paged_attention_join_kernel<DP, 16, DP <= 128 ? 16 : 8>, dim3(units, p.rows), dim3(16 * 32), 0,
                              stream, a, p);
    return tc::launch_pdl(paged_attention_join_kernel<DP, 16, 8>, dim3(units, p.rows), dim3(16 * 32), 0, stream, a, p);
}

// The workspace's layout: the queue, what to join, partial states.
struct Layout {
    int ctas, rows;
    size_t joins, parts, bytes;
};

Layout layout(const KvCache &kv, int64_t B, int64_t Hq)
{
    Layout w;
    const int group = (int)(Hq / kv.heads);
    w.ctas = device_sm_count();
    w.rows = group < 16 ? group : 16;
    w.joins = 256;
    w.parts = w.joins + ((size_t)B * kv.heads * ((group + 15) / 16) * sizeof(int2) + 255) / 256 * 256;
    w.bytes = w.parts + (size_t)w.ctas * kMaxWarps * kRunsPerWarp * 2 * part_floats(w.rows, kv.dim) * sizeof(float);
    return w;
}

}  // namespace

size_t paged_attention_workspace(const KvCache &kv, int64_t B, int64_t Hq) { return layout(kv, B, Hq).bytes; }

cudaError_t launch_paged_attention(const AttnArgs &a, cudaStream_t stream)
{
    const Layout w = layout(a.kv, a.B, a.Hq);
    char *ws = static_cast<char *>(a.ws);
    AttnPlan p;
    p.group = a.Hq / a.kv.heads;
    p.rows = w.rows;
    p.blocks = (p.group + 15) / 16;
    p.units = a.kv.heads * p.blocks;
    p.queue = reinterpret_cast<unsigned long long *>(ws);
    p.joins = reinterpret_cast<int2 *>(ws + w.joins);
    p.parts = reinterpret_cast<float *>(ws + w.parts);
    for (int i = 0; i < 3; ++i) {
        p.k16[i] = (uint32_t)(a.kv.ks[i] / (a.kv.int8 ? 16 : 8));
        p.v16[i] = (uint32_t)(a.kv.vs[i] / (a.kv.int8 ? 16 : 8));
        p.sc[i] = (uint32_t)a.kv.ss[i];
    }
    p.alike = p.k16[0] == p.v16[0] && p.k16[1] == p.v16[1] && p.k16[2] == p.v16[2];
    p.log_page = -1;
    for (int i = 0; i < 31; ++i)
        if (a.kv.page_size == 1 << i)
            p.log_page = i;
    const auto launch = a.kv.int8 ? (p.group <= 8 ? attn::launch_int8_8 : attn::launch_int8_16)
                                  : (p.group <= 8 ? attn::launch_bf16_8 : attn::launch_bf16_16);
    const cudaError_t e = launch(a, p, w.ctas, stream);
    if (e != cudaSuccess)
        return e;
    return a.kv.dim <= 64    ? launch_join<64>(a, p, stream)
           : a.kv.dim <= 128 ? launch_join<128>(a, p, stream)
                             : launch_join<256>(a, p, stream);
}

}  // namespace s3d8

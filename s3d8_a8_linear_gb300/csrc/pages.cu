// Pages of a cache of several layers: copies, growth, forks, release and
// compaction (s3d8_copy_pages and the calls below it in the header).
//
// The bookkeeping (block table, lengths, reference counts) is a few hundred KB
// at most and runs in one CTA, which needs no ordering between CTAs; the page
// copies that follow read their list from the workspace and use the whole GPU.
// Measured: growth of 16 sequences 4 us, a fork of 16 in 40 layers 14 us (its copies
// move 40 MB), compaction of 250 pages in 40 layers 206 us (6.4 TB/s).
#include "common.cuh"
#include "launch.h"
#include "page_room.h"
#include "tcgen05.cuh"

namespace s3d8 {

namespace {

constexpr int kMetaThreads = 1024, kMetaWarps = kMetaThreads / 32;

// Exclusive prefix sum of one value per thread; `total` receives the sum.
template <class T>
__device__ T block_scan(T v, T *warp_sums, T &total)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    T inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o)
            inc += u;
    }
    __syncthreads();   // the previous call's sums have been read
    if (lane == 31)
        warp_sums[warp] = inc;
    __syncthreads();
    T w = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T u = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o)
            w += u;
    }
    total = __shfl_sync(0xffffffffu, w, 31);
    return inc - v + (warp ? __shfl_sync(0xffffffffu, w, warp - 1) : 0);
}

// Walks ids begin..end-1 in order over the whole CTA and calls f(id, rank) with
// the rank of each id for which pick(id) holds; returns how many there are.  f is
// called for the ranks below `most` only.
template <class Pick, class F>
__device__ int enumerate(int begin, int end, int most, int *warp_sums, Pick pick, F f)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // warp w takes a run of whole 32-id groups
    const int groups = (end - begin + 31) / 32, per = (groups + kMetaWarps - 1) / kMetaWarps;
    const int g0 = min(groups, warp * per), g1 = min(groups, g0 + per);
    int mine = 0;
#pragma unroll 4
    for (int g = g0; g < g1; ++g) {
        const int id = begin + g * 32 + lane;
        mine += __popc(__ballot_sync(0xffffffffu, id < end && pick(id)));
    }
    int total;
    int rank = block_scan(lane == 31 ? mine : 0, warp_sums, total);
    rank = __shfl_sync(0xffffffffu, rank, 0);
#pragma unroll 4
    for (int g = g0; g < g1; ++g) {
        if (rank >= most)
            break;
        const int id = begin + g * 32 + lane;
        const bool yes = id < end && pick(id);
        const uint32_t mask = __ballot_sync(0xffffffffu, yes);
        const int at = rank + __popc(mask & ((1u << lane) - 1u));
        if (yes && at < most)
            f(id, at);
        rank += __popc(mask);
    }
    return total;
}

// Workspace: ids [pages], more [pages], map [pages], then three lists of `rows`.
__device__ __forceinline__ int32_t *ws_list(const PagesArgs &a, int k)
{
    return a.ws + (k < 3 ? (size_t)k * a.pages : (size_t)3 * a.pages + (size_t)(k - 3) * a.rows);
}

__global__ __launch_bounds__(kMetaThreads) void extend_pages_kernel(PagesArgs a)
{
    __shared__ int sums[32];
    __shared__ long long wanted[32];
    tc::pdl_launch_dependents();
    tc::pdl_wait();
    int32_t *ids = ws_list(a, 0), *begins = ws_list(a, 3), *needs = ws_list(a, 4);
    long long asked = 0;   // a page for every column of every entry may pass 2^31
    for (int i0 = 0; i0 < a.n; i0 += kMetaThreads) {
        const int i = i0 + threadIdx.x;
        int need = -1;   // refused
        if (i < a.n) {
            const int s = a.who[i];
            const int64_t add = a.other[i];
            if (s < 0 || s >= a.rows) {
                atomicExch(a.status, kStatusBounds);
            } else {
                const int64_t len = max(a.lens[s], 0), S = a.page_size;
                const int64_t have = (len + S - 1) / S, want = (len + add + S - 1) / S;
                if (add >= 0 && want <= a.width && len + add <= 0x7FFFFFFF)
                    need = (int)(want - have);
            }
        }
        long long total;
        const long long begin = asked + block_scan((long long)max(need, 0), wanted, total);
        asked += total;
        if (i < a.n) {
            begins[i] = page_rank(begin);
            needs[i] = need;
        }
    }
    __syncthreads();
    const int32_t *refs = a.refs;
    const int free = enumerate(0, a.pages, min(page_rank(asked), a.pages), sums, [&](int id) { return refs[id] == 0; },
                               [&](int id, int at) { ids[at] = id; });
    __syncthreads();
    for (int i = threadIdx.x >> 5; i < a.n; i += kMetaWarps) {
        const int lane = threadIdx.x & 31, need = needs[i], begin = begins[i];
        const bool ok = page_room(begin, need, free);
        if (ok) {
            const int s = a.who[i];
            const int len = max(a.lens[s], 0);
            const int have = (int)(((int64_t)len + a.page_size - 1) / a.page_size);
            for (int k = lane; k < need; k += 32) {
                const int id = ids[begin + k];
                a.table[s * a.width + have + k] = id;
                a.refs[id] = 1;
            }
            __syncwarp();
            if (lane == 0)
                a.lens[s] = len + a.other[i];
        }
        if (lane == 0)
            a.got[i] = ok;
    }
}

__global__ __launch_bounds__(kMetaThreads) void fork_pages_kernel(PagesArgs a)
{
    __shared__ int sums[32];
    tc::pdl_launch_dependents();
    tc::pdl_wait();
    int32_t *ids = ws_list(a, 0), *src = ws_list(a, 3), *dst = ws_list(a, 4), *tokens = ws_list(a, 5);
    // what can be forked: a warp an entry, since every page of the parent is looked at before any is shared; four entries'
    // loads leave together (200 forks on one layer: 23 us, against 27 one after another)
    constexpr int kAhead = 4;
    for (int i0 = threadIdx.x >> 5; i0 < a.n; i0 += kAhead * kMetaWarps) {
        const int lane = threadIdx.x & 31;
        int64_t p[kAhead];
        int len[kAhead], id[kAhead];
        bool bad[kAhead];
#pragma unroll
        for (int x = 0; x < kAhead; ++x) {
            const int i = min(i0 + x * kMetaWarps, a.n - 1);
            const int64_t c = a.other[i];
            p[x] = a.who[i];
            bad[x] = p[x] < 0 || p[x] >= a.rows || c < 0 || c >= a.rows;
        }
#pragma unroll
        for (int x = 0; x < kAhead; ++x)
            len[x] = bad[x] ? 0 : a.lens[p[x]];
#pragma unroll
        for (int x = 0; x < kAhead; ++x) {
            bad[x] |= len[x] < 0 || len[x] > a.width * a.page_size;
            len[x] = bad[x] ? 0 : len[x];
            id[x] = (int64_t)lane * a.page_size < len[x] ? a.table[p[x] * a.width + lane] : 0;
        }
#pragma unroll
        for (int x = 0; x < kAhead; ++x) {
            const int i = i0 + x * kMetaWarps, full = len[x] / a.page_size, part = len[x] - full * a.page_size;
            bad[x] |= id[x] < 0 || id[x] >= a.pages;
            for (int k = lane + 32; k < full + (part > 0); k += 32) {
                const int more = a.table[p[x] * a.width + k];
                bad[x] |= more < 0 || more >= a.pages;
            }
            bad[x] = __any_sync(0xffffffffu, bad[x]);
            if (lane == 0 && i < a.n) {
                src[i] = bad[x] ? -2 : part ? full : -1;   // the partial page's column; -2: refused
                tokens[i] = bad[x] ? 0 : part;
                if (bad[x])
                    atomicExch(a.status, kStatusBounds);
            }
        }
    }
    __syncthreads();
    int asked = 0;
    for (int i0 = 0; i0 < a.n; i0 += kMetaThreads) {
        const int i = i0 + threadIdx.x;
        int total;
        const int begin = asked + block_scan((int)(i < a.n && tokens[i] > 0), sums, total);
        asked += total;
        if (i < a.n)
            dst[i] = begin;
    }
    __syncthreads();
    const int32_t *refs = a.refs;
    const int free = enumerate(0, a.pages, min(asked, a.pages), sums, [&](int id) { return refs[id] == 0; },
                               [&](int id, int at) { ids[at] = id; });
    __syncthreads();
    for (int i = threadIdx.x >> 5; i < a.n; i += kMetaWarps) {
        const int lane = threadIdx.x & 31, part = tokens[i], at = src[i], begin = dst[i];
        const int64_t p = a.who[i], c = a.other[i];
        const bool ok = at != -2 && (!part || begin < free);
        const int fresh = ok && part ? ids[begin] : -1;
        int from = -1;
        if (c >= 0 && c < a.rows) {
            const int full = ok ? a.lens[p] / a.page_size : 0;
            for (int64_t k = lane; k < a.width; k += 32) {
                int id = -1;
                if (k < full) {
                    id = a.table[p * a.width + k];
                    if (id >= 0 && id < a.pages)   // else the row is a child of this call as well
                        atomicAdd(a.refs + id, 1);
                    else
                        id = -1;
                } else if (k == full) {
                    id = fresh;
                }
                a.table[c * a.width + k] = id;
            }
            if (lane == 0) {
                a.lens[c] = ok ? a.lens[p] : 0;
                if (fresh >= 0) {
                    a.refs[fresh] = 1;
                    from = a.table[p * a.width + full];
                    if (from >= a.pages)
                        from = -1;
                }
            }
        }
        __syncwarp();     // every lane has read the entry's lists
        if (lane == 0) {
            src[i] = from;
            dst[i] = fresh;
            a.got[i] = ok;
        }
    }
}

__global__ __launch_bounds__(kMetaThreads) void free_pages_kernel(PagesArgs a)
{
    tc::pdl_launch_dependents();
    tc::pdl_wait();
    for (int i = threadIdx.x >> 5; i < a.n; i += kMetaWarps) {
        const int lane = threadIdx.x & 31;
        const int64_t s = a.who[i];
        if (s < 0 || s >= a.rows) {
            atomicExch(a.status, kStatusBounds);
            continue;
        }
        for (int64_t k = lane; k < a.width; k += 32) {
            const int id = a.table[s * a.width + k];
            const bool page = id >= 0 && id < a.pages;
            const bool counted = page && atomicSub(a.refs + id, 1) > 0;
            if (page && !counted)
                atomicAdd(a.refs + id, 1);   // held by more entries than counted: it stays free
            if (id >= 0 && !counted)
                atomicExch(a.status, kStatusBounds);
            a.table[s * a.width + k] = -1;
        }
        if (lane == 0)
            a.lens[s] = 0;
    }
}

// holes -> ids, movers -> more, map[mover] = its new id; refs and live follow.
__global__ __launch_bounds__(kMetaThreads) void compact_plan_kernel(PagesArgs a)
{
    __shared__ int sums[32];
    tc::pdl_launch_dependents();
    tc::pdl_wait();
    int32_t *holes = ws_list(a, 0), *movers = ws_list(a, 1), *map = ws_list(a, 2), *count = ws_list(a, 3);
    int32_t *refs = a.refs;
    const int live = enumerate(0, a.pages, 0, sums, [&](int id) { return refs[id] != 0; }, [](int, int) {});
    const int moves = enumerate(0, live, a.pages, sums, [&](int id) { return refs[id] == 0; },
                                [&](int id, int at) { holes[at] = id; });
    enumerate(live, a.pages, a.pages, sums, [&](int id) { return refs[id] != 0; },
              [&](int id, int at) { movers[at] = id; });
    for (int id = live + threadIdx.x; id < a.pages; id += kMetaThreads)
        map[id] = id;   // a dangling entry (of a page that nobody counts) stays
    __syncthreads();
    for (int i = threadIdx.x; i < moves; i += kMetaThreads) {
        const int from = movers[i], to = holes[i];
        map[from] = to;
        refs[to] = refs[from];
        refs[from] = 0;
    }
    if (threadIdx.x == 0) {
        *count = moves;
        a.got[0] = live;
    }
}

__global__ void compact_table_kernel(PagesArgs a)
{
    tc::pdl_launch_dependents();
    tc::pdl_wait();
    const int32_t *map = ws_list(a, 2);
    const int live = a.got[0];
    const int64_t n = a.rows * a.width;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
        const int id = a.table[i];
        if (id >= a.pages)
            atomicExch(a.status, kStatusBounds);
        else if (id >= live)
            a.table[i] = map[id];
    }
}

constexpr int kCopyThreads = 256;

// Copies the first nt tokens of a page, T at a time (per_row of them a row).  Rows
// that follow one another in memory go as one run; every thread has BATCH loads in
// flight (250 pages of 16 tokens x 8 heads x 128 in 40 layers, 1.3 GB: 202 us with
// eight, 208 with four, 269 with one and a row's address for each).
template <int BATCH, class T>
__device__ __forceinline__ void copy_rows(const T *from, T *to, int nt, int page_size, int heads, int per_row,
                                          const int64_t (&st)[3], int elements)
{
    const int64_t token = st[1] / elements, head = st[2] / elements;
    int runs, length;             // of T
    int64_t stride = 0;
    if (token == per_row && head == (int64_t)page_size * per_row && nt == page_size) {
        runs = 1, length = nt * heads * per_row;               // a whole page, heads outside
    } else if (head == per_row && token == (int64_t)heads * per_row) {
        runs = 1, length = nt * heads * per_row;               // tokens outside
    } else if (token == per_row) {
        runs = heads, length = nt * per_row, stride = head;    // a run a head
    } else {
        runs = nt * heads, length = per_row;                   // row by row
    }
    const int total = runs * length;
    const bool rows = runs == nt * heads && length == per_row && runs > 1;
    auto place = [&](int u) -> int64_t {
        if (runs == 1)
            return u;
        const int r = u / length, c = u - r * length;
        if (!rows)
            return r * stride + c;
        const int t = r / heads;
        return t * token + (r - t * heads) * head + c;
    };
    for (int u0 = threadIdx.x; u0 < total; u0 += kCopyThreads * BATCH) {
        T v[BATCH];
        int64_t at[BATCH];
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const int u = u0 + i * kCopyThreads;
            if (u < total) {
                at[i] = place(u);
                v[i] = __ldcs(from + at[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < BATCH; ++i)
            if (u0 + i * kCopyThreads < total)
                __stcs(to + at[i], v[i]);
    }
}

// One job = one page pair in one layer, keys or values (and, in int8, their scales).
template <int BATCH>
__global__ __launch_bounds__(kCopyThreads) void copy_pages_kernel(const __grid_constant__ PoolArgs p, const int32_t *src,
                                                                  const int32_t *dst, const int32_t *tokens, int n,
                                                                  const int32_t *count, int *status)
{
    tc::pdl_launch_dependents();
    tc::pdl_wait();
    if (count)
        n = *count;
    const int64_t jobs = (int64_t)n * p.layers * 2;
    const KvCache &g = p.geo;
    for (int64_t j = blockIdx.x; j < jobs; j += gridDim.x) {
        const int pair = (int)(j / (p.layers * 2)), rest = (int)(j - (int64_t)pair * (p.layers * 2)), layer = rest >> 1;
        const int from = src[pair], to = dst[pair], nt = tokens ? tokens[pair] : g.page_size;
        if (from < 0 || to < 0)
            continue;
        if (from >= g.pages || to >= g.pages) {
            if (threadIdx.x == 0)
                atomicExch(status, kStatusBounds);
            continue;
        }
        const bool value = rest & 1;
        const int64_t (&st)[3] = value ? g.vs : g.ks;
        const int es = g.int8 ? 1 : 2, epc = 16 / es;
        char *base = static_cast<char *>(value ? p.v[layer] : p.k[layer]);
        copy_rows<BATCH>(reinterpret_cast<const uint4 *>(base + from * st[0] * es), reinterpret_cast<uint4 *>(base + to * st[0] * es), nt,
                  g.page_size, g.heads, g.dim / epc, st, epc);
        if (g.int8) {
            float *sc = value ? p.v_scale[layer] : p.k_scale[layer];
            copy_rows<BATCH>(sc + from * g.ss[0], sc + to * g.ss[0], nt, g.page_size, g.heads, 1, g.ss, 1);
        }
    }
}

}  // namespace

size_t pages_workspace(int64_t pages, int64_t rows)
{
    return ((size_t)3 * pages + (size_t)3 * rows + 4) * sizeof(int32_t);
}

cudaError_t launch_copy_pages(const PoolArgs &p, const int32_t *src, const int32_t *dst, const int32_t *tokens, int n,
                              const int32_t *count, int *status, cudaStream_t stream)
{
    if (n == 0)
        return cudaSuccess;
    // Few pages: four loads a thread, so that more CTAs fit (16 pages of 40 layers: 13 us against 16); many:
    // eight.
    const int64_t jobs = (int64_t)n * p.layers * 2, sms = device_sm_count();
    const bool many = jobs > 32 * sms;
    return tc::launch_pdl(many ? copy_pages_kernel<8> : copy_pages_kernel<4>, dim3((unsigned)(jobs < 16 * sms ? jobs : 16 * sms)),
                          dim3(kCopyThreads), 0, stream, p, src, dst, tokens, n, count, status);
}

cudaError_t launch_extend_pages(const PagesArgs &a, cudaStream_t stream)
{
    return tc::launch_pdl(extend_pages_kernel, dim3(1), dim3(kMetaThreads), 0, stream, a);
}

cudaError_t launch_fork_pages(const PagesArgs &a, PagePairs *pairs, cudaStream_t stream)
{
    const int32_t *lists = a.ws + (size_t)3 * a.pages;
    *pairs = PagePairs{lists, lists + a.rows, lists + 2 * a.rows, nullptr};
    return tc::launch_pdl(fork_pages_kernel, dim3(1), dim3(kMetaThreads), 0, stream, a);
}

cudaError_t launch_free_pages(const PagesArgs &a, cudaStream_t stream)
{
    return tc::launch_pdl(free_pages_kernel, dim3(1), dim3(kMetaThreads), 0, stream, a);
}

cudaError_t launch_compact_pages(const PagesArgs &a, PagePairs *pairs, cudaStream_t stream)
{
    *pairs = PagePairs{a.ws + a.pages, a.ws, nullptr, a.ws + (size_t)3 * a.pages};
    cudaError_t e = tc::launch_pdl(compact_plan_kernel, dim3(1), dim3(kMetaThreads), 0, stream, a);
    if (e != cudaSuccess)
        return e;
    return tc::launch_pdl(compact_table_kernel, dim3(64), dim3(256), 0, stream, a);
}

}  // namespace s3d8

// The next token of each row from its logits (s3d8_sample): temperature, top-k, top-p and
// min-p, and one given uniform number a row.
//
// Tokens stand in the order of their logits, equal ones by index, with weights
// w = exp((l - max) / T); every limit keeps a beginning of that order, and u times the kept
// weight falls on one token of it.  A bf16 logit is one of 65536 values, so nothing is
// sorted: a row is counted into a histogram of its values, and weights are computed once
// per value instead of once per token.  That leaves time for exact ones: exp in pairs of
// fp32 (about 2^-43), summed as whole numbers of 2^-45 of the largest weight.  Such sums do
// not depend on their order, so equal inputs give equal bits, and a token next to a border
// is decided as in 64 bits.
//
// A cluster of CTAs takes a row, a part of the vocabulary each (16-bit counts in shared
// memory, so at most 65535 tokens a CTA).  The values are dealt in groups of 128, one power
// of two each; a CTA adds up the counts of its share of the groups from all CTAs of the
// cluster, skipping groups that none has.  The first CTA then finds the limits and the
// value by searching the groups' sums, and the CTA whose part holds the token reads its
// part again for it.
#include "launch.h"
#include "tcgen05.cuh"

namespace s3d8 {

namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kGroups = 512, kKeys = 128;       // groups of values, values of a group
constexpr int kHistWords = kGroups * kKeys / 2; // two 16-bit counts a word
constexpr int kMostTokens = 65528;              // of a CTA: counts stay below 2^16, parts begin on 8
constexpr int kScale = 45;                      // weights are whole numbers of 2^-45

struct Shared {
    uint32_t hist[kHistWords];
    uint32_t flags[kGroups / 32];               // groups that this CTA's part has
    uint32_t top;                               // its largest key
    // in the first CTA
    uint32_t count[kGroups], above[kGroups];    // of a group, all CTAs': tokens, those that min-p keeps
    unsigned long long mass[kGroups];
    // first: group sums, from the largest group downwards, in front of each
    uint32_t count_before[kGroups];
    unsigned long long mass_before[kGroups];
    uint32_t warp_count[kWarps], warp_above[kWarps];
    unsigned long long warp_mass[kWarps];
    uint32_t found_key, found_rank;             // the token: its value, and its rank among equals
    int found;
    uint32_t match[kWarps];
    unsigned long long best[kWarps];
    // what a search found
    uint32_t hit_count;
    unsigned long long hit_mass, hit_weight;
    uint32_t hit_key;
    int hit_group;
};

// Keys rise with the value; both zeros are one.  0: a token that is never drawn (-inf, NaN).
__device__ __forceinline__ uint32_t key_of(uint32_t bits)
{
    bits = bits == 0x8000u ? 0u : bits;
    const uint32_t key = bits & 0x8000u ? 0xFFFFu - bits : bits | 0x8000u;
    return (bits & 0x7FFFu) > 0x7F80u || bits == 0xFF80u ? 0u : key;
}

__device__ __forceinline__ float value_of(uint32_t key)
{
    return __uint_as_float((key & 0x8000u ? key & 0x7FFFu : 0xFFFFu - key) << 16);
}

// ---- pairs of fp32 (hi + lo, |lo| at most half a step of hi) ------------------

struct Pair {
    float hi, lo;
};

__device__ __forceinline__ Pair quick_sum(float a, float b)     // |a| >= |b|
{
    const float s = __fadd_rn(a, b);
    return {s, __fsub_rn(b, __fsub_rn(s, a))};
}

__device__ __forceinline__ Pair two_sum(float a, float b)
{
    const float s = __fadd_rn(a, b), bb = __fsub_rn(s, a);
    return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb))};
}

__device__ __forceinline__ Pair mul(Pair a, Pair b)
{
    const float p = __fmul_rn(a.hi, b.hi);
    return quick_sum(p, __fmaf_rn(a.hi, b.lo, __fmaf_rn(a.lo, b.hi, __fmaf_rn(a.hi, b.hi, -p))));
}

__device__ __forceinline__ Pair add(Pair a, Pair b)
{
    const Pair s = two_sum(a.hi, b.hi);
    return quick_sum(s.hi, __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo)));
}

// The two parts of a double (to 2^-48 of it).
__device__ __forceinline__ Pair pair_of(double x)
{
    const float hi = (float)x;
    return {hi, isfinite(hi) ? (float)(x - (double)hi) : 0.0f};
}

// 2^45 exp(x) to the nearest whole number, x <= 0: exp(x) = 2^n exp(r), r = x - n ln 2,
// with the series of exp(r), |r| <= ln(2) / 2: its terms from r^7 on in fp32 (below 2^-23 of
// the sum), the others in pairs.
__device__ __forceinline__ unsigned long long weight(Pair x)
{
    if (!(x.hi > -32.0f))       // below 2^-46
        return 0ull;
    const float n = rintf(x.hi * 1.44269504f);
    // ln 2 in three parts, of which the first has 12 bits, so that n times it is exact
    constexpr float l1 = 0.693115234375f, l2 = 3.19461833e-05f, l3 = 1.646595e-12f;
    Pair r = two_sum(__fmaf_rn(-n, l1, x.hi), __fmul_rn(-n, l2));
    r = add(r, {__fmaf_rn(-n, l2, -__fmul_rn(-n, l2)), __fmaf_rn(-n, l3, x.lo)});
    float t = 1.0f / 6227020800.0f;
    t = __fmaf_rn(t, r.hi, 1.0f / 479001600.0f);
    t = __fmaf_rn(t, r.hi, 1.0f / 39916800.0f);
    t = __fmaf_rn(t, r.hi, 1.0f / 3628800.0f);
    t = __fmaf_rn(t, r.hi, 1.0f / 362880.0f);
    t = __fmaf_rn(t, r.hi, 1.0f / 40320.0f);
    t = __fmaf_rn(t, r.hi, 1.0f / 5040.0f);
    constexpr double c6 = 1.0 / 720, c5 = 1.0 / 120, c4 = 1.0 / 24, c3 = 1.0 / 6;
    Pair y = mul({t, 0.0f}, r);
    y = mul(add(y, {(float)c6, (float)(c6 - (float)c6)}), r);
    y = mul(add(y, {(float)c5, (float)(c5 - (float)c5)}), r);
    y = mul(add(y, {(float)c4, (float)(c4 - (float)c4)}), r);
    y = mul(add(y, {(float)c3, (float)(c3 - (float)c3)}), r);
    y = mul(add(y, {0.5f, 0.0f}), r);
    y = mul(add(y, {1.0f, 0.0f}), r);
    y = add({1.0f, 0.0f}, y);
    const float scale = __uint_as_float((uint32_t)(127 + kScale + (int)n) << 23);
    return (unsigned long long)(__float2ll_rn(__fmul_rn(y.hi, scale)) + __float2ll_rn(__fmul_rn(y.lo, scale)));
}

struct Row {
    uint32_t top;       // the largest key
    float top_value;
    Pair inverse;       // 1 / T
};

__device__ __forceinline__ unsigned long long weight_of(uint32_t key, const Row &r)
{
    if (key == r.top)
        return 1ull << kScale;
    const Pair d = two_sum(value_of(key), -r.top_value);
    if (!isfinite(d.hi))        // an infinite largest logit takes all; -3.4e38 below 3.4e38 is nothing
        return 0ull;
    const float p = __fmul_rn(d.hi, r.inverse.hi);
    if (!(p > -40.0f))          // past what a weight can show (and NaN where 1 / T is infinite)
        return 0ull;
    return weight(mul(d, r.inverse));
}

__device__ __forceinline__ uint32_t remote_u32(uint32_t addr)
{
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}

__device__ __forceinline__ void remote_store_u32(uint32_t addr, uint32_t v)
{
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ void remote_store_u64(uint32_t addr, unsigned long long v)
{
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

// The counts of a lane's four neighbouring values of a group (values 4 lane .. 4 lane + 3), all CTAs'.
template <int C>
__device__ __forceinline__ void group_counts(Shared &s, int group, int lane, uint32_t (&n)[4])
{
    n[0] = n[1] = n[2] = n[3] = 0;
    const uint32_t at = smem_addr(s.hist) + (group * (kKeys / 2) + 2 * lane) * 4;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        uint32_t a, b;
        asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(a), "=r"(b) : "r"(tc::map_to_rank(at, c)));
        n[0] += a & 0xFFFFu, n[1] += a >> 16, n[2] += b & 0xFFFFu, n[3] += b >> 16;
    }
}

// The eight tokens from i on (i a multiple of 8; those at n and behind are no tokens).
__device__ __forceinline__ void eight(const uint16_t *x, int i, int n, bool vec, uint32_t (&key)[8])
{
    if (vec && i + 8 <= n) {
        const uint4 v = __ldg(reinterpret_cast<const uint4 *>(x + i));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 8; ++e)
            key[e] = key_of(e & 1 ? w[e / 2] >> 16 : w[e / 2] & 0xFFFFu);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            key[e] = i + e < n ? key_of(__ldg(x + i + e)) : 0u;
    }
}

// Searches the order of all tokens, by count or by mass: the value that holds the
// `target`-th unit (from 0).  All threads of the first CTA.  Leaves in s.hit_*: the value,
// its weight, and the tokens and mass in front of it.
template <int C>
__device__ __forceinline__ void search(Shared &s, const Row &row, bool by_mass, unsigned long long target)
{
    if (threadIdx.x < kGroups) {
        const int g = threadIdx.x;
        const unsigned long long before = by_mass ? s.mass_before[g] : s.count_before[g], n = by_mass ? s.mass[g] : s.count[g];
        if (target >= before && target < before + n)
            s.hit_group = g;
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        const int lane = 31 - threadIdx.x;      // the largest values first
        const int g = s.hit_group;
        uint32_t n[4];
        group_counts<C>(s, g, lane, n);
        unsigned long long w[4], mass = 0;
        uint32_t count = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            w[e] = n[e] ? weight_of(g * kKeys + 4 * lane + e, row) : 0;
            mass += n[e] * w[e];
            count += n[e];
        }
        uint32_t c = count;
        unsigned long long m = mass;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t pc = __shfl_up_sync(0xffffffffu, c, o);
            const unsigned long long pm = __shfl_up_sync(0xffffffffu, m, o);
            if (threadIdx.x >= o)
                c += pc, m += pm;
        }
        c += s.count_before[g] - count;
        m += s.mass_before[g] - mass;
#pragma unroll
        for (int e = 3; e >= 0; --e) {
            const unsigned long long before = by_mass ? m : c, size = by_mass ? n[e] * w[e] : n[e];
            if (target >= before && target < before + size) {
                s.hit_key = g * kKeys + 4 * lane + e;
                s.hit_weight = w[e];
                s.hit_count = c;
                s.hit_mass = m;
            }
            c += n[e];
            m += n[e] * w[e];
        }
    }
    __syncthreads();
}

template <int C>
__device__ __forceinline__ void row_sync()
{
    if (C > 1)
        tc::cluster_sync();
    else
        __syncthreads();
}

template <int C>
__global__ __launch_bounds__(kThreads) void sample_kernel(const __grid_constant__ SampleArgs a, int part, int vec)
{
    extern __shared__ __align__(16) unsigned char sample_mem[];
    Shared &s = *reinterpret_cast<Shared *>(sample_mem);
    const int rank = C > 1 ? (int)tc::cluster_rank() : 0, b = blockIdx.x / C;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int first = rank * part, n = max(0, min(part, a.V - first));
    for (int i = threadIdx.x; i < kHistWords / 4; i += kThreads)
        reinterpret_cast<uint4 *>(s.hist)[i] = make_uint4(0u, 0u, 0u, 0u);
    if (threadIdx.x < kGroups / 32)
        s.flags[threadIdx.x] = 0;
    if (threadIdx.x == 0) {
        s.top = 0;
        s.found = 0;
    }
    tc::pdl_launch_dependents();
    tc::pdl_wait();
    const uint16_t *x = reinterpret_cast<const uint16_t *>(a.logits) + (int64_t)b * a.stride + first;
    const float temp = a.temperature ? a.temperature[b] : 1.0f;
    __syncthreads();

    uint32_t top = 0;
    if (!(temp > 0.0f)) {       // the largest logit, the lowest index among equals
        unsigned long long best = 0;
        for (int i = threadIdx.x * 8; i < n; i += kThreads * 8) {
            uint32_t key[8];
            eight(x, i, n, vec, key);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                best = max(best, (unsigned long long)key[e] << 32 | (0xFFFFFFFFu - (uint32_t)(first + i + e)));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
        if (lane == 0)
            s.best[warp] = best;
        row_sync<C>();          // and the first CTA has begun
        if (warp == 0) {
            best = s.best[lane];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
            if (lane == 0)
                remote_store_u64(tc::map_to_rank(smem_addr(s.mass) + 8 * rank, 0), best);
        }
        row_sync<C>();
        if (rank == 0 && threadIdx.x == 0) {
            best = s.mass[0];
            for (int c = 1; c < C; ++c)
                best = max(best, s.mass[c]);
            const bool some = best >> 32;
            a.tokens[b] = some ? (int32_t)(0xFFFFFFFFu - (uint32_t)best) : -1;
            if (a.logprob)
                a.logprob[b] = some ? 0.0f : -INFINITY;
        }
        return;
    }

    for (int i = threadIdx.x * 8; i < n; i += kThreads * 8) {
        uint32_t key[8];
        eight(x, i, n, vec, key);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (key[e])
                atomicAdd(&s.hist[key[e] >> 1], key[e] & 1 ? 0x10000u : 1u);
            top = max(top, key[e]);
        }
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0)
        atomicMax(&s.top, top);
    __syncthreads();
    for (int g = warp; g < kGroups; g += kWarps) {
        const uint2 v = reinterpret_cast<const uint2 *>(s.hist)[g * (kKeys / 4) + lane];
        if (__any_sync(0xffffffffu, v.x | v.y) && lane == 0)
            atomicOr(&s.flags[g / 32], 1u << (g & 31));
    }
    row_sync<C>();

    Row row;
    row.top = 0;
#pragma unroll
    for (int c = 0; c < C; ++c)
        row.top = max(row.top, remote_u32(tc::map_to_rank(smem_addr(&s.top), c)));
    row.top_value = value_of(row.top);
    row.inverse = pair_of(1.0 / (double)temp);
    const double min_p = a.min_p ? (double)a.min_p[b] : 0.0;
    // the groups g, g + C, ... of this CTA, a warp each
    for (int g = rank + C * warp; g < kGroups; g += C * kWarps) {
        uint32_t some = 0;
#pragma unroll
        for (int c = 0; c < C; ++c)
            some |= remote_u32(tc::map_to_rank(smem_addr(s.flags) + 4 * (g / 32), c));
        uint32_t count = 0, above = 0;
        unsigned long long mass = 0;
        if (some >> (g & 31) & 1) {
            uint32_t cnt[4];
            group_counts<C>(s, g, lane, cnt);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (!cnt[e])
                    continue;
                const unsigned long long w = weight_of(g * kKeys + 4 * lane + e, row);
                count += cnt[e];
                mass += cnt[e] * w;
                above += (double)w >= min_p * (double)(1ull << kScale) ? cnt[e] : 0u;
            }
            count = __reduce_add_sync(0xffffffffu, count);
            above = __reduce_add_sync(0xffffffffu, above);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                mass += __shfl_xor_sync(0xffffffffu, mass, o);
        }
        if (lane == 0) {
            remote_store_u32(tc::map_to_rank(smem_addr(&s.count[g]), 0), count);
            remote_store_u32(tc::map_to_rank(smem_addr(&s.above[g]), 0), above);
            remote_store_u64(tc::map_to_rank(smem_addr(&s.mass[g]), 0), mass);
        }
    }
    row_sync<C>();

    if (rank == 0) {
        // sums in front of each group, from the largest values downwards
        uint32_t count = 0, above = 0;
        unsigned long long mass = 0;
        const int g = kGroups - 1 - (int)threadIdx.x;
        if (threadIdx.x < kGroups)
            count = s.count[g], above = s.above[g], mass = s.mass[g];
        uint32_t c = count, k = above;
        unsigned long long m = mass;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t pc = __shfl_up_sync(0xffffffffu, c, o), pk = __shfl_up_sync(0xffffffffu, k, o);
            const unsigned long long pm = __shfl_up_sync(0xffffffffu, m, o);
            if (lane >= o)
                c += pc, k += pk, m += pm;
        }
        if (lane == 31)
            s.warp_count[warp] = c, s.warp_above[warp] = k, s.warp_mass[warp] = m;
        __syncthreads();
        uint32_t all = 0, kept = 0;
        unsigned long long whole = 0;
        for (int w = 0; w < kGroups / 32; ++w) {
            if (w < warp)
                c += s.warp_count[w], m += s.warp_mass[w];
            all += s.warp_count[w], kept += s.warp_above[w], whole += s.warp_mass[w];
        }
        if (threadIdx.x < kGroups)
            s.count_before[g] = c - count, s.mass_before[g] = m - mass;
        __syncthreads();

        if (all == 0) {         // nothing to draw
            if (threadIdx.x == 0) {
                a.tokens[b] = -1;
                if (a.logprob)
                    a.logprob[b] = -INFINITY;
            }
        } else {
            uint32_t stay = all;        // a beginning of the order: its tokens and its mass
            unsigned long long held = whole;
            const int32_t top_k = a.top_k ? a.top_k[b] : 0;
            if (top_k > 0 && (uint32_t)top_k < stay) {
                search<C>(s, row, false, (unsigned long long)top_k - 1);
                stay = (uint32_t)top_k;
                held = s.hit_mass + (stay - s.hit_count) * s.hit_weight;
                __syncthreads();
            }
            const double top_p = a.top_p ? (double)a.top_p[b] : 1.0;
            if (top_p < 1.0) {          // the first tokens whose mass reaches top_p of what is held
                const double want = ceil(top_p * (double)held);
                const unsigned long long need = want > 1.0 ? min((unsigned long long)want, held) : 1ull;
                search<C>(s, row, true, need - 1);
                const uint32_t more = (uint32_t)((need - s.hit_mass + s.hit_weight - 1) / s.hit_weight);
                if (s.hit_count + more <= stay) {
                    stay = s.hit_count + more;
                    held = s.hit_mass + more * s.hit_weight;
                }
                __syncthreads();
            }
            if (kept < stay && a.min_p) {
                stay = max(kept, 1u);
                search<C>(s, row, false, (unsigned long long)stay - 1);
                held = s.hit_mass + (stay - s.hit_count) * s.hit_weight;
                __syncthreads();
            }
            const double want = (double)a.u[b] * (double)held;
            const unsigned long long t = want > 0.0 ? min((unsigned long long)want, held - 1) : 0ull;
            search<C>(s, row, true, t);
            if (threadIdx.x == 0) {
                const uint32_t key = s.hit_key, r = (uint32_t)((t - s.hit_mass) / s.hit_weight);
                for (int to = 0; to < C; ++to) {
                    remote_store_u32(tc::map_to_rank(smem_addr(&s.found_key), to), key);
                    remote_store_u32(tc::map_to_rank(smem_addr(&s.found_rank), to), r);
                    remote_store_u32(tc::map_to_rank(smem_addr(&s.found), to), 1u);
                }
                if (a.logprob) {
                    const double gap = key == row.top ? 0.0 : ((double)value_of(key) - (double)row.top_value) / (double)temp;
                    a.logprob[b] = (float)(gap - log((double)held / (double)(1ull << kScale)));
                }
            }
        }
    }
    row_sync<C>();

    // the found_rank-th token of the value found_key, over the CTAs' parts in order
    bool mine = s.found;
    if (mine) {
        const uint32_t key = s.found_key;
        uint32_t want = s.found_rank;
        for (int c = 0; c <= rank && mine; ++c) {
            const uint32_t w = remote_u32(tc::map_to_rank(smem_addr(&s.hist[key >> 1]), c)), has = key & 1 ? w >> 16 : w & 0xFFFFu;
            if (c == rank)
                mine = want < has;
            else if (want < has)
                mine = false;
            else
                want -= has;
        }
        if (mine) {     // each warp a run of the part
            const int run = ((n + kWarps - 1) / kWarps + 255) / 256 * 256, from = warp * run, to = min(n, from + run);
            uint32_t hits = 0;
            for (int i = from + lane * 8; i < to; i += 256) {
                uint32_t k[8];
                eight(x, i, n, vec, k);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    hits += k[e] == key;
            }
            hits = __reduce_add_sync(0xffffffffu, hits);
            if (lane == 0)
                s.match[warp] = hits;
            __syncthreads();
            uint32_t before_run = 0;
            for (int w = 0; w < warp; ++w)
                before_run += s.match[w];
            if (want >= before_run && want < before_run + hits) {
                want -= before_run;
                for (int i0 = from; i0 < to; i0 += 256) {
                    const int i = i0 + lane * 8;
                    uint32_t k[8], mask = 0;
                    if (i < to)
                        eight(x, i, n, vec, k);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        mask |= (i < to && k[e] == key ? 1u : 0u) << e;
                    uint32_t before = __popc(mask);
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const uint32_t p = __shfl_up_sync(0xffffffffu, before, o);
                        before += lane >= o ? p : 0;
                    }
                    const uint32_t sum = __shfl_sync(0xffffffffu, before, 31);
                    before -= __popc(mask);
                    if (want >= before && want < before + __popc(mask)) {
                        for (uint32_t skip = want - before; skip > 0; --skip)
                            mask &= mask - 1;
                        a.tokens[b] = first + i + __ffs(mask) - 1;
                    }
                    if (want < sum)
                        break;
                    want -= sum;
                }
            }
        }
    }
    if (C > 1)
        tc::cluster_sync();     // no CTA leaves while another may read its counts
}

template <int C>
cudaError_t launch(const SampleArgs &a, cudaStream_t stream)
{
    const int part = ((a.V + C - 1) / C + 7) / 8 * 8;
    const int vec = ((uintptr_t)a.logits & 15) == 0 && (a.stride & 7) == 0;
    auto kernel = sample_kernel<C>;
    static std::atomic<unsigned long long> allowed;
    cudaError_t e = tc::allow_smem(kernel, sizeof(Shared), allowed);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.B * C);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(Shared);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = C;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = C > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, a, part, vec);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs &a, cudaStream_t stream)
{
    // as few CTAs a row as fill the GPU (one fits an SM), and as many as 16-bit counts ask for
    const int64_t sms = device_sm_count(), most = kMostTokens;
    if (a.V <= 8192 || ((int64_t)a.B > sms / 2 && a.V <= most))
        return launch<1>(a, stream);
    if (a.B > sms / 4 && a.V <= 2 * most)
        return launch<2>(a, stream);
    if (a.B > sms / 8 && a.V <= 4 * most)
        return launch<4>(a, stream);
    return launch<8>(a, stream);
}

}  // namespace s3d8

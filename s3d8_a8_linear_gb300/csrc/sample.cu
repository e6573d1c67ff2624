// The next token of each row from its logits (s3d8_sample): temperature, top-k, top-p and
// min-p, and one given uniform number a row.
//
// Tokens stand in the order of their logits, equal ones by index, with weights
// w = exp((l - max) / T); every limit keeps a beginning of that order, and u times the kept
// weight falls on one token of it.  A bf16 logit is one of 65536 values, so nothing is
// sorted: tokens are counted into a histogram of their values, and weights are computed once
// per value instead of once per token.  That leaves time for exact ones: exp in pairs of
// fp32 (to 2^-43 of itself and 2^-46 of the largest weight), summed as whole numbers of 2^-45
// of the largest weight.  Such sums do not depend on their order, so equal inputs give equal
// bits, and are right to 2^-45 for each of their tokens.
//
// Counting costs an atomic addition in shared memory a token, so only the head of the order
// is counted, the values within 16 T of the largest logit; of the others only the sum of the
// weights is taken, in fp32: base-2 exponents of 23 to 64, which are rounded by up to 2^-19,
// ex2.approx (2^-22), and a dozen additions, together at most 2^-18 of that sum (which is at most
// 2^-6 of the largest weight with 128256 logits).  Where a limit or the drawn token turns out to
// lie behind the head, the row is counted again as a whole.
//
// A cluster of CTAs takes a row, a part of the vocabulary each (16-bit counts, so at most
// 65535 tokens a CTA), and reads it three times, from L2 but for the first.  Values form
// groups of 128, one power of two each.  The first CTA adds up the counts of the groups that
// have any from all CTAs, finds the limits and the value by searching the groups' sums, and
// tells the CTA whose part has the token.
//
// Bound by instructions and by the barriers between those steps (42% of the issue slots with
// 509 rows), not by HBM.  Measured with 128256 logits: one row 13 us, 64 rows with limits of
// their own 28 us, 509 rows 164 us (302 when every token was counted).
#include "launch.h"
#include "tcgen05.cuh"
#include "uniform.cuh"

namespace s3d8 {

namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kGroups = 512, kKeys = 128;       // groups of values, values of a group
constexpr int kHistWords = kGroups * kKeys / 2; // two 16-bit counts a word
constexpr int kMostTokens = 65528;              // of a CTA: counts stay below 2^16, parts begin on 8
constexpr int kScale = 45;                      // weights are whole numbers of 2^-45

constexpr int kUnits = 512;                      // runs of values that the first CTA adds up, at most
constexpr int kCached = 64;                     // runs of 32 whose values' counts and weights it keeps
constexpr float kHead = 16.0f;                  // counted: values within kHead T of the largest
constexpr float kHeadWeight = 1.2e-7f;          // exp(-kHead), and a little

// A value's tokens and weight, and what stands in front of it in its run.
struct Value {
    uint32_t count, count_before;
    unsigned long long weight, mass_before;
};

struct Shared {
    uint32_t hist[kHistWords];
    uint32_t flags[kGroups / 32];               // groups that this CTA's part has
    uint32_t top;                               // its largest key, times 2^16; the least of its lanes' largest (below)
    unsigned long long tail;                    // the weights that it has not counted
    uint32_t wave[kWarps];
    unsigned long long wide[kWarps];
    // told by the first CTA
    int verdict;                                // what a row comes to: below
    uint32_t key, rank;                         // the token: its value, and its rank among this CTA's
    // of the first CTA.  The groups that some CTA's part has, from the largest values downwards
    int groups;
    uint16_t order[kGroups];
    // Of run i, from the largest values downwards, all CTAs': tokens, those
    // that min-p keeps, weight; and what stands in front of it
    uint32_t count[kUnits], above[kUnits], count_before[kUnits];
    unsigned long long mass[kUnits], mass_before[kUnits];
    Value values[kCached][32];
};

enum Verdict { kNothing, kMine, kOther, kAgain };

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

// 1 / x (to 2^-46 of it; just rounded where that is 0 or infinite).
__device__ __forceinline__ Pair reciprocal(float x)
{
    const float r = __frcp_rn(x);
    return {r, isfinite(r) && r > 0.0f ? __fmul_rn(r, __fmaf_rn(-r, x, 1.0f)) : 0.0f};
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

// Two fp32 at once.
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    uint64_t d, x = *reinterpret_cast<uint64_t *>(&a), y = *reinterpret_cast<uint64_t *>(&b);
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(x), "l"(y));
    return *reinterpret_cast<float2 *>(&d);
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    uint64_t d, x = *reinterpret_cast<uint64_t *>(&a), y = *reinterpret_cast<uint64_t *>(&b), z = *reinterpret_cast<uint64_t *>(&c);
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(x), "l"(y), "l"(z));
    return *reinterpret_cast<float2 *>(&d);
}

struct Row {
    uint32_t top;       // the largest key
    float top_value;
    float unit;         // a power of two that brings T near enough to 1 for
    Pair inverse;       // 1 / (unit T)
};

// (Out of line, as search() is: a CTA passes its code once, and what is short is there sooner.)
__device__ __noinline__ unsigned long long weight_of(uint32_t key, Row r)
{
    if (key == r.top)
        return 1ull << kScale;
    const Pair d = two_sum(value_of(key) * r.unit, -r.top_value * r.unit);
    if (!isfinite(d.hi))        // an infinite largest logit takes all, and so does one far past a small unit
        return 0ull;
    const float p = __fmul_rn(d.hi, r.inverse.hi);
    if (!(p > -40.0f))          // past what a weight can show
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

// How the counted values are cut into runs, groups without any left out: runs of 32, a value a
// lane, or of 128 where those were too many.
struct Runs {
    int count;
    bool fine;
    __device__ __forceinline__ explicit Runs(int groups) : count(groups), fine(groups * 4 <= kUnits) { count *= fine ? 4 : 1; }
    // the largest of a lane's values of run i
    __device__ __forceinline__ int first(const Shared &s, int i) const
    {
        const int lane = threadIdx.x & 31;
        return fine ? s.order[i >> 2] * kKeys + (kKeys - 1) - 32 * (i & 3) - lane : s.order[i] * kKeys + (kKeys - 1) - 4 * lane;
    }
};

// Which groups some CTA's part has (most rows have few, but those around zero span many
// powers of two that they do not have).  One warp of the first CTA.
template <int C>
__device__ __forceinline__ void list_groups(Shared &s)
{
    const int lane = threadIdx.x & 31;
    uint32_t mine = 0;
    if (lane < kGroups / 32)
#pragma unroll
        for (int c = 0; c < C; ++c)
            mine |= remote_u32(tc::map_to_rank(smem_addr(s.flags) + 4 * lane, c));
    int count = 0;
    for (int w = kGroups / 32 - 1; w >= 0; --w) {
        const uint32_t some = __shfl_sync(0xffffffffu, mine, w);
        if (some >> lane & 1)
            s.order[count + __popc(some >> lane) - 1] = (uint16_t)(32 * w + lane);
        count += __popc(some);
    }
    if (lane == 0)
        s.groups = count;
}

// All CTAs' tokens of a lane's values of a run, the largest value first: value `first` - e, e
// < 4 (fine: e = 0 alone).
template <int C>
__device__ __forceinline__ void run_counts(Shared &s, const Runs &r, int first, uint32_t (&n)[4])
{
    n[0] = n[1] = n[2] = n[3] = 0;
    if (r.fine) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            uint16_t v;
            asm volatile("ld.shared::cluster.u16 %0, [%1];" : "=h"(v) : "r"(tc::map_to_rank(smem_addr(s.hist) + 2 * first, c)));
            n[0] += v;
        }
    } else {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            uint32_t a, b;
            asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];" : "=r"(a), "=r"(b) : "r"(tc::map_to_rank(smem_addr(s.hist) + 2 * (first - 3), c)));
            n[3] += a & 0xFFFFu, n[2] += a >> 16, n[1] += b & 0xFFFFu, n[0] += b >> 16;
        }
    }
}

// A run's tokens and weight in front of a lane's first value, and (at the last lane) with its
// values: inclusive sums over the lanes.
__device__ __forceinline__ void scan_run(const uint32_t (&n)[4], const unsigned long long (&w)[4], uint32_t &count, unsigned long long &mass)
{
    count = n[0] + n[1] + n[2] + n[3];
    mass = n[0] * w[0] + n[1] * w[1] + n[2] * w[2] + n[3] * w[3];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t pc = __shfl_up_sync(0xffffffffu, count, o);
        const unsigned long long pm = __shfl_up_sync(0xffffffffu, mass, o);
        const bool in = (int)(threadIdx.x & 31) >= o;
        count += in ? pc : 0u;
        mass += in ? pm : 0ull;
    }
}

// The eight tokens from i on (i a multiple of 8), two a word; those at n and behind are -inf.
__device__ __noinline__ uint4 eight_slowly(const uint16_t *x, int left)
{
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t lo = 2 * e < left ? __ldg(x + 2 * e) : 0xFF80u, hi = 2 * e + 1 < left ? __ldg(x + 2 * e + 1) : 0xFF80u;
        w[e] = lo | hi << 16;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint4 eight(const uint16_t *x, int i, int n, bool vec)
{
    return vec && i + 8 <= n ? __ldg(reinterpret_cast<const uint4 *>(x + i)) : eight_slowly(x + i, n - i);
}

// The larger of each two bf16 (of a NaN and a number, the number).
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

__device__ __forceinline__ uint32_t max_of(const uint4 &v) { return max_bf16x2(max_bf16x2(v.x, v.y), max_bf16x2(v.z, v.w)); }

__device__ __forceinline__ float lo_value(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_value(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Which of eight tokens have a value (bf16, twice in a word; both zeros are one).
__device__ __forceinline__ uint32_t equal(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("set.eq.u32.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

__device__ __forceinline__ uint32_t equal_mask(uint4 v, uint32_t value)
{
    // token 2 j is bit 2 j, token 2 j + 1 is bit 16 + 2 j + 1; then side by side
    const uint32_t m = (equal(v.x, value) & 0x00020001u) | (equal(v.y, value) & 0x00080004u) | (equal(v.z, value) & 0x00200010u) |
                       (equal(v.w, value) & 0x00800040u);
    return (m | m >> 16) & 0xFFu;
}

// Halves of a word that are at least those of another: 0xFFFF, else (and for NaN) 0.
__device__ __forceinline__ uint32_t at_least(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("set.ge.u32.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Counts those of eight tokens whose value is at least `cut` (bf16, twice in a word) and that
// are tokens.  A lane has few of them, so that a loop over a lane's takes fewer atomic
// instructions than eight.
__device__ __forceinline__ void count_eight(Shared &s, uint4 v, uint32_t cut)
{
    const unsigned long long lo = v.x | (unsigned long long)v.y << 32, hi = v.z | (unsigned long long)v.w << 32;
    uint32_t some = (at_least(v.x, cut) & 0x00010002u) | (at_least(v.y, cut) & 0x00040008u) | (at_least(v.z, cut) & 0x00100020u) |
                    (at_least(v.w, cut) & 0x00400080u);
    // the bits of odd tokens came from the low halves: token 2 j is bit 2 j + 1, token 2 j + 1 is bit 16 + 2 j
    while (__any_sync(0xffffffffu, some)) {
        if (some) {
            const int bit = __ffs(some) - 1, e = bit < 16 ? bit - 1 : bit - 15;
            some &= some - 1;
            const uint32_t key = key_of((uint32_t)((e < 4 ? lo : hi) >> (16 * (e & 3))) & 0xFFFFu);
            if (key)
                atomicAdd(&s.hist[key >> 1], key & 1 ? 0x10000u : 1u);
        }
        __syncwarp();
    }
}

// How the weights behind the head are taken: base-2 exponents y c + b, and the parts of c and
// b that fp32 does not hold, times ln 2.  Of rows that are not far: T between 2^-80 and 2^60 and
// the largest logit within 2^31, so that c, b and the rests of a logit of -2^68 are finite.
struct Behind {
    float cut;
    float2 c, b, c_rest, b_rest;

    __device__ __forceinline__ Behind(float cut, const Row &row)
        : cut(cut)
    {
        const Pair to2 = mul(row.inverse, {1.44269502f, 1.92596303e-08f}), top = mul(to2, {-row.top_value, 0.0f});
        c = make_float2(to2.hi, to2.hi);
        b = make_float2(top.hi, top.hi);
        c_rest = make_float2(to2.lo * 0.693147f, to2.lo * 0.693147f);
        b_rest = make_float2(top.lo * 0.693147f, top.lo * 0.693147f);
    }

    // Of two tokens, where they are not counted.
    __device__ __forceinline__ float2 operator()(uint32_t w) const
    {
        w = max_bf16x2(w, 0xE180E180u);         // -inf and NaN: -2^68, which is more than 100 T down and has no weight
        const float2 y = make_float2(lo_value(w), hi_value(w)), x = fma2(y, c, b), rest = fma2(y, c_rest, b_rest);
        float2 p;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(p.x) : "f"(x.x));
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(p.y) : "f"(x.y));
        p = fma2(p, rest, p);
        return make_float2(y.x < cut ? p.x : 0.0f, y.y < cut ? p.y : 0.0f);
    }
};

// A value of the order of all counted tokens, its weight, and the tokens and weight in front of it.
struct Hit {
    uint32_t key, count;
    unsigned long long mass, weight;
};

// The value that holds the `target`-th unit (from 0) of the tokens, or of their weight.  One
// warp of the first CTA.
template <int C>
__device__ __noinline__ Hit search(Shared &s, Row row, Runs runs, bool by_mass, unsigned long long target)
{
    const int lane = threadIdx.x & 31;
    int i = 0;
    for (int base = 0; base < runs.count; base += 32) {
        const int at = base + lane;
        const unsigned long long before = at >= runs.count ? 0 : by_mass ? s.mass_before[at] : s.count_before[at];
        const unsigned long long size = at >= runs.count ? 0 : by_mass ? s.mass[at] : s.count[at];
        const uint32_t in = __ballot_sync(0xffffffffu, target >= before && target < before + size);
        if (in) {
            i = base + __ffs(in) - 1;
            break;
        }
    }
    Hit hit = {0, 0, 0, 0};
    bool has = false;
    if (runs.fine && i < kCached) {
        const Value v = s.values[i][lane];
        hit = {(uint32_t)runs.first(s, i), s.count_before[i] + v.count_before, s.mass_before[i] + v.mass_before, v.weight};
        const unsigned long long before = by_mass ? hit.mass : hit.count, size = by_mass ? v.count * v.weight : v.count;
        has = target >= before && target < before + size;
    } else {
        const int first = runs.first(s, i);
        uint32_t n[4], c;
        run_counts<C>(s, runs, first, n);
        unsigned long long w[4], m;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            w[e] = n[e] ? weight_of(first - e, row) : 0;
        scan_run(n, w, c, m);
        c += s.count_before[i] - (n[0] + n[1] + n[2] + n[3]);
        m += s.mass_before[i] - (n[0] * w[0] + n[1] * w[1] + n[2] * w[2] + n[3] * w[3]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const unsigned long long before = by_mass ? m : c, size = by_mass ? n[e] * w[e] : n[e];
            if (target >= before && target < before + size) {
                hit = {(uint32_t)(first - e), c, m, w[e]};
                has = true;
            }
            c += n[e];
            m += n[e] * w[e];
        }
    }
    const int from = __ffs(__ballot_sync(0xffffffffu, has)) - 1;
    hit.key = __shfl_sync(0xffffffffu, hit.key, from);
    hit.count = __shfl_sync(0xffffffffu, hit.count, from);
    hit.mass = __shfl_sync(0xffffffffu, hit.mass, from);
    hit.weight = __shfl_sync(0xffffffffu, hit.weight, from);
    return hit;
}

template <int C>
__device__ __forceinline__ void row_sync()
{
    if (C > 1)
        tc::cluster_sync();
    else
        __syncthreads();
}

// Adds up the runs' counts of all CTAs and their weights, a warp a run.  All warps of the first CTA.
template <int C>
__device__ __forceinline__ void add_runs(Shared &s, const Row &row, unsigned long long least, const Runs &runs)
{
    const int warp = warp_index(), lane = threadIdx.x & 31;
    for (int i = warp; i < runs.count; i += kWarps) {
        const int first = runs.first(s, i);
        uint32_t n[4], count = 0, above = 0;
        unsigned long long w[4] = {0, 0, 0, 0}, mass = 0;
        run_counts<C>(s, runs, first, n);
        if (__any_sync(0xffffffffu, n[0] | n[1] | n[2] | n[3])) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                w[e] = n[e] ? weight_of(first - e, row) : 0;
                above += w[e] >= least ? n[e] : 0u;
            }
            above = __reduce_add_sync(0xffffffffu, above);
            scan_run(n, w, count, mass);
        }
        if (runs.fine && i < kCached)
            s.values[i][lane] = {n[0], count - n[0], w[0], mass - n[0] * w[0]};
        if (lane == 31) {
            s.count[i] = count;
            s.above[i] = above;
            s.mass[i] = mass;
        }
    }
}

// The token's value, its rank among its equals and its share, from the groups' sums; or that
// all tokens have to be counted.  One warp of the first CTA (the 64-bit arithmetic is slow).
template <int C>
__device__ __forceinline__ Verdict choose(Shared &s, const SampleArgs &a, int b, const Row &row, bool cold, bool whole, const Runs &runs, uint32_t &key,
                                          uint32_t &rank)
{
    const int lane = threadIdx.x & 31;
    uint32_t stay = 0, kept = 0;        // a beginning of the order: its tokens and its mass
    unsigned long long head = 0, held = 0;
    for (int base = 0; base < runs.count; base += 32) {     // sums in front of each run
        const int i = base + lane;
        const uint32_t count = i < runs.count ? s.count[i] : 0;
        const unsigned long long mass = i < runs.count ? s.mass[i] : 0;
        uint32_t c = count, k = i < runs.count ? s.above[i] : 0;
        unsigned long long m = mass;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t pc = __shfl_up_sync(0xffffffffu, c, o), pk = __shfl_up_sync(0xffffffffu, k, o);
            const unsigned long long pm = __shfl_up_sync(0xffffffffu, m, o);
            c += lane >= o ? pc : 0u;
            k += lane >= o ? pk : 0u;
            m += lane >= o ? pm : 0ull;
        }
        if (i < runs.count)
            s.count_before[i] = stay + c - count, s.mass_before[i] = head + m - mass;
        stay += __shfl_sync(0xffffffffu, c, 31);
        kept += __shfl_sync(0xffffffffu, k, 31);
        head += __shfl_sync(0xffffffffu, m, 31);
    }
    if (lane < C)
        asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(held) : "r"(tc::map_to_rank(smem_addr(&s.tail), lane)));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        held += __shfl_xor_sync(0xffffffffu, held, o);
    held += head;
    __syncwarp();

    const int32_t top_k = uniform(cold ? 1 : a.top_k ? a.top_k[b] : 0);
    if (top_k > 0 && (uint32_t)top_k > stay && !whole)
        return kAgain;
    if (top_k > 0 && (uint32_t)top_k <= stay) {
        const Hit hit = search<C>(s, row, runs, false, (unsigned long long)top_k - 1);
        stay = (uint32_t)top_k;
        held = hit.mass + (stay - hit.count) * hit.weight;
    } else if (!whole)
        stay = 0xFFFFFFFFu;             // with those that were not counted
    const float top_p = uniform(!cold && a.top_p ? a.top_p[b] : 1.0f);
    if (top_p < 1.0f) {                 // the first tokens whose mass reaches top_p of what is held
        const double want = ceil((double)top_p * (double)held);
        const unsigned long long need = want > 1.0 ? min((unsigned long long)want, held) : 1ull;
        if (need > head)
            return kAgain;
        const Hit hit = search<C>(s, row, runs, true, need - 1);
        const uint32_t more = (uint32_t)((need - hit.mass + hit.weight - 1) / hit.weight);
        if (hit.count + more <= stay) {
            stay = hit.count + more;
            held = hit.mass + more * hit.weight;
        }
    }
    const float min_p = uniform(!cold && a.min_p ? a.min_p[b] : 0.0f);
    if (!(min_p <= 0.0f) && kept < stay) {
        if (!whole && min_p <= kHeadWeight)
            return kAgain;
        stay = max(kept, 1u);
        const Hit hit = search<C>(s, row, runs, false, (unsigned long long)stay - 1);
        held = hit.mass + (stay - hit.count) * hit.weight;
    }
    const double want = (double)uniform(a.u[b]) * (double)held;
    const unsigned long long t = want > 0.0 ? min((unsigned long long)want, held - 1) : 0ull;
    if (t >= head)
        return kAgain;
    const Hit hit = search<C>(s, row, runs, true, t);
    key = hit.key;
    rank = (uint32_t)((t - hit.mass) / hit.weight);
    if (a.logprob && lane == 0) {
        const float d = value_of(key) * row.unit - row.top_value * row.unit, gap = key == row.top ? 0.0f : __fmaf_rn(d, row.inverse.hi, d * row.inverse.lo);
        a.logprob[b] = gap - log1pf((float)(held - (1ull << kScale)) * (1.0f / (float)(1ull << kScale)));
    }
    return kMine;
}

template <int C>
__global__ __launch_bounds__(kThreads) void sample_kernel(const __grid_constant__ SampleArgs a, int part, int vec, int ahead)
{
    extern __shared__ __align__(16) unsigned char sample_mem[];
    Shared &s = *reinterpret_cast<Shared *>(sample_mem);
    const int cta = C > 1 ? uniform((int)tc::cluster_rank()) : 0, b = blockIdx.x / C;
    const int warp = warp_index(), lane = threadIdx.x & 31;
    const int first = cta * part, n = max(0, min(part, a.V - first));
    tc::pdl_launch_dependents();
    tc::pdl_wait();
    const uint16_t *x = reinterpret_cast<const uint16_t *>(a.logits) + (int64_t)b * a.stride + first;
    // what a CTA of the next wave reads, into L2 meanwhile
    const int next = b + ahead;
    if (vec && threadIdx.x == 0 && ahead && next < a.B && n >= 8)
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(x + (int64_t)ahead * a.stride), "r"((uint32_t)(n / 8 * 16)) : "memory");
    uint32_t most = 0xFF80FF80u;        // of this thread's tokens; -inf
#pragma unroll 4
    for (int i = threadIdx.x * 8; i < n; i += kThreads * 8)
        most = max_bf16x2(most, max_of(eight(x, i, n, vec)));
    float temp = uniform(a.temperature ? a.temperature[b] : 1.0f);
    const bool cold = !(temp > 0.0f);   // the first token of the order alone
    temp = cold ? 1.0f : temp;
    if (threadIdx.x < kGroups / 32)
        s.flags[threadIdx.x] = 0;
    // The largest value, and one that 256 tokens reach, or as many as there are groups of 4 C
    // lanes with any: the least of the groups' largest.
    uint32_t top = max(key_of(most & 0xFFFFu), key_of(most >> 16));
#pragma unroll
    for (int o = 1; o < 4 * C; o <<= 1)
        top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const uint32_t low = __reduce_min_sync(0xffffffffu, top ? top : 0xFFFFu);
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0)
        s.wave[warp] = top << 16 | low;
    __syncthreads();
    if (warp == 0) {
        const uint32_t w = s.wave[lane];
        top = __reduce_max_sync(0xffffffffu, w >> 16);
        const uint32_t least = __reduce_min_sync(0xffffffffu, w & 0xFFFFu);
        if (lane == 0)
            s.top = top << 16 | least;
    }
    row_sync<C>();
    Row row;
    uint32_t reached;
    {
        const uint32_t t = lane < C ? remote_u32(tc::map_to_rank(smem_addr(&s.top), lane)) : 0xFFFFu;
        row.top = __reduce_max_sync(0xffffffffu, t >> 16);
        reached = __reduce_min_sync(0xffffffffu, t & 0xFFFFu);
    }
    if (row.top == 0) {                 // nothing to draw (all CTAs of the row alike)
        if (cta == 0 && threadIdx.x == 0) {
            a.tokens[b] = -1;
            if (a.logprob)
                a.logprob[b] = -INFINITY;
        }
        row_sync<C>();
        return;
    }
    row.top_value = value_of(row.top);
    // else 1 / T, or the part of it that fp32 does not hold, may pass fp32's range
    row.unit = temp >= 0x1p60f ? 0x1p-64f : temp <= 0x1p-80f ? 0x1p64f : 1.0f;
    row.inverse = reciprocal(temp * row.unit);
    const bool far = row.unit != 1.0f || !(fabsf(row.top_value) < 0x1p31f);
    const int last_group = row.top / kKeys;
    Verdict verdict;
    for (bool whole = false;; whole = true) {
        // counted: values from `cut` on; the second time all that have a weight (2^-46 is none)
        float cut = cold ? row.top_value : fminf(row.top_value - (whole ? 33.0f : kHead) * temp, whole ? INFINITY : value_of(reached));
        if (!(cut <= row.top_value))    // (infinite ones of both)
            cut = row.top_value;
        if (far)                        // all tokens, as Behind's terms may be infinite
            cut = -INFINITY;
        const uint32_t bits = __float_as_uint(cut) >> 16, cut2 = bits | bits << 16;     // bf16: towards zero
        const int first_group = bits == 0xFF80u ? 0 : key_of(bits) / kKeys;
        for (int i = first_group * (kKeys / 8) + threadIdx.x; i < (last_group + 1) * (kKeys / 8); i += kThreads)
            reinterpret_cast<uint4 *>(s.hist)[i] = make_uint4(0u, 0u, 0u, 0u);
        __syncthreads();
        const Behind behind(__uint_as_float(bits << 16), row);
        float2 tails = make_float2(0.0f, 0.0f);
        const uint4 none = make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u);      // -inf
        auto load = [&](int base) {
            const int i = base + (int)threadIdx.x * 8;
            return i < n ? eight(x, i, n, vec) : none;
        };
        uint4 ahead1 = load(0), ahead2 = load(kThreads * 8);    // loads do not pass the atomics
        for (int base = 0; base < n; base += kThreads * 8) {    // whole warps together
            const uint4 v = ahead1;
            ahead1 = ahead2;
            ahead2 = load(base + 2 * kThreads * 8);
            count_eight(s, v, cut2);
            if (!whole)
                tails = add2(tails, add2(add2(behind(v.x), behind(v.y)), add2(behind(v.z), behind(v.w))));
        }
        const float tail = tails.x + tails.y;
        unsigned long long sum = (unsigned long long)__float2ll_rn(tail * (float)(1ull << kScale));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0)
            s.wide[warp] = sum;
        __syncthreads();
        for (int g = first_group + warp; g <= last_group; g += kWarps) {
            const uint2 h = reinterpret_cast<const uint2 *>(s.hist)[g * (kKeys / 4) + lane];
            if (__any_sync(0xffffffffu, h.x | h.y) && lane == 0)
                atomicOr(&s.flags[g / 32], 1u << (g & 31));
        }
        if (warp == 0) {
            sum = lane < kWarps ? s.wide[lane] : 0ull;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (lane == 0)
                s.tail = sum;
        }
        row_sync<C>();

        if (cta == 0) {
            const float min_p = uniform(!cold && a.min_p ? a.min_p[b] : 0.0f);
            // the least weight that min-p keeps: min_p 2^45, and 0 (min_p NaN, or past 1: none)
            const unsigned long long least = min_p <= 0.0f ? 0ull : min_p <= 1.0f ? (unsigned long long)__float2ll_ru(min_p * (float)(1ull << kScale)) : ~0ull;
            if (warp == 0)
                list_groups<C>(s);
            __syncthreads();
            const Runs runs(uniform(s.groups));
            add_runs<C>(s, row, least, runs);
            __syncthreads();
            if (warp == 0) {            // whose part has the token, and its rank there
                uint32_t key = 0, rank = 0;
                const Verdict found = choose<C>(s, a, b, row, cold, whole, runs, key, rank);
                uint32_t has = 0;
                if (found == kMine && lane < C) {
                    const uint32_t w = remote_u32(tc::map_to_rank(smem_addr(&s.hist[key >> 1]), lane));
                    has = key & 1 ? w >> 16 : w & 0xFFFFu;
                }
                uint32_t before = has;
#pragma unroll
                for (int o = 1; o < C; o <<= 1) {
                    const uint32_t p = __shfl_up_sync(0xffffffffu, before, o);
                    before += lane >= o ? p : 0;
                }
                before -= has;
                if (lane < C) {
                    const bool mine = rank >= before && rank < before + has;
                    remote_store_u32(tc::map_to_rank(smem_addr(&s.key), lane), key);
                    remote_store_u32(tc::map_to_rank(smem_addr(&s.rank), lane), rank - before);
                    remote_store_u32(tc::map_to_rank(smem_addr(&s.verdict), lane), found == kMine && !mine ? kOther : found);
                }
            }
            __syncthreads();
        }
        row_sync<C>();
        verdict = (Verdict)uniform(s.verdict);
        if (verdict != kAgain)
            break;
    }
    if (verdict != kMine)
        return;

    // the token: a warp looks at a run of the part
    const uint32_t rank = s.rank, bits = __float_as_uint(value_of(s.key)) >> 16, value = bits | bits << 16;
    const int run = ((n + kWarps - 1) / kWarps + 255) / 256 * 256, from = warp * run, to = min(n, from + run);
    uint32_t hits = 0;
#pragma unroll 4
    for (int i = from + lane * 8; i < to; i += 256)
        hits += __popc(equal_mask(eight(x, i, to, vec), value));
    hits = __reduce_add_sync(0xffffffffu, hits);
    if (lane == 0)
        s.wave[warp] = hits;
    __syncthreads();
    const uint32_t in_front = __reduce_add_sync(0xffffffffu, lane < warp ? s.wave[lane] : 0u);
    if (rank < in_front || rank >= in_front + hits)
        return;
    uint32_t want = rank - in_front;
    for (int base = from; base < to; base += 256) {
        const int i = base + lane * 8;
        const uint32_t mask = i < to ? equal_mask(eight(x, i, to, vec), value) : 0u, mine = __popc(mask);
        uint32_t upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t p = __shfl_up_sync(0xffffffffu, upto, o);
            upto += lane >= o ? p : 0;
        }
        if (want >= upto - mine && want < upto) {
            uint32_t left = mask;
            for (uint32_t skip = want - (upto - mine); skip > 0; --skip)
                left &= left - 1;
            a.tokens[b] = first + i + __ffs(left) - 1;
        }
        const uint32_t all = __shfl_sync(0xffffffffu, upto, 31);
        if (want < all)
            return;
        want -= all;
    }
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
    return cudaLaunchKernelEx(&cfg, kernel, a, part, vec, device_sm_count() / C);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs &a, cudaStream_t stream)
{
    // One CTA fits an SM, and 16-bit counts ask for a CTA for every 65528 tokens.  More CTAs a
    // row shorten its counting while all rows still run at once (clusters of 8 and 4 do not fill
    // the last SMs of a group of them).  Measured with 1, 2, 4 and 8 CTAs (us): up to 8192 logits
    // 17, 18, 18, 18 with 8 rows; 32768 logits: 8 rows 26, 22, 20, 19, 16 rows 25, 22, 20, 24, 38
    // rows 26, 22, 31, 52, 152 rows 26, 44, 80, 171; 128256 logits: one row -, 31, 28, 15, 16 rows
    // -, 39, 28, 31, 38 rows -, 40, 38, 52, 64 rows -, 41, 53, 86.
    const int64_t sms = device_sm_count(), most = kMostTokens;
    if (a.V <= 8192 || ((int64_t)a.B > sms / 2 && a.V <= most))
        return launch<1>(a, stream);
    if (a.B > sms / 8 && a.V <= 2 * most)
        return launch<2>(a, stream);
    if (a.B > sms / 16 && a.V <= 4 * most)
        return launch<4>(a, stream);
    return launch<8>(a, stream);
}

}  // namespace s3d8

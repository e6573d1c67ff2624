// How the append's ring of bulk copies is laid out (rope_append.cu).
#pragma once

namespace s3d8 {

constexpr int kRopeThreads = 256;        // that turn and store, at most
constexpr int kRingStages = 8;           // at most
constexpr int kRingBytes = 110 * 1024;   // of a CTA, at most: what the kernel is allowed
constexpr int kRingThreads = 800;        // of an SM
constexpr int kRingSm = 227 * 1024;      // shared memory of an SM,
constexpr int kRingFixed = 1536;         // of which every CTA takes this much beside its stages

struct RopeRing {
    int threads, ctas, stages, stage;    // turning threads, CTAs an SM, stages of a CTA, their bytes
};

// Of tokens of `heads` rows in all (q, k and v); `stages` is 0 where three do not fit.
// Five CTAs of three stages at 48 heads of 128; more of them where a token has fewer rows.
inline RopeRing rope_ring(int heads, int dim, int rotary, int log_lanes)
{
    RopeRing r = {0, 0, 0, heads * dim * 2 + rotary * 4};
    if (3 * r.stage > kRingBytes)
        return r;
    r.threads = (((heads + 2) / 3 << log_lanes) + 31) / 32 * 32;
    r.threads = r.threads < kRopeThreads ? r.threads : kRopeThreads;
    r.ctas = kRingThreads / (r.threads + 32);
    r.stages = (kRingSm / r.ctas - kRingFixed) / r.stage;
    if (r.stages < 3) {
        r.stages = 3;
        r.ctas = kRingSm / (3 * r.stage + kRingFixed);
    }
    const int allowed = kRingBytes / r.stage;   // two CTAs an SM have room for a little more than that
    r.stages = r.stages < allowed ? r.stages : allowed;
    r.stages = r.stages < kRingStages ? r.stages : kRingStages;
    return r;
}

// Whether the rows of one token's `heads` heads, `stride` elements apart, lie in one
// piece.  The stride of a single head means nothing (the binding passes 0).
inline bool rope_whole(int heads, long long stride, int dim) { return heads == 1 || stride == dim; }

}  // namespace s3d8

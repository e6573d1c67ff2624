// What one lane has of a rotary row of D columns, and how it turns (rope_append.cu,
// norm_rope.cu): a row belongs to D/16 neighbouring lanes, rounded up to a power of
// two, of two 16-byte chunks each, chosen so that a lane holds both columns of its
// pairs.
#pragma once

#include "bf16x8.cuh"
#include "common.cuh"

namespace s3d8 {

// Which two chunks a lane holds, and where the partners of its columns are.
enum RopeMode {
    kHalves,        // pairs (i, i + rotary/2), rotary a multiple of 16: both in one lane
    kNeighbours,    // pairs (2i, 2i + 1): two neighbouring chunks
    kHalvesOdd      // any other rotary: neighbouring chunks, partners read one by one
};

// A lane's part of every row: two chunks, and whether its pairs 8 lane .. 8 lane + 7 turn.
struct RopeLane {
    int lane, lanes, half, chunk[2];
    bool in_row, turns;

    __device__ __forceinline__ RopeLane(int rotary, int dim, int mode, int log_lanes)
        : lane((int)threadIdx.x & ((1 << log_lanes) - 1)), lanes(1 << log_lanes), half(rotary / 2)
    {
        chunk[0] = 2 * lane;
        chunk[1] = 2 * lane + 1;
        if (mode == kHalves && lane < rotary / 16) {
            chunk[0] = lane;
            chunk[1] = lane + rotary / 16;
        }
        in_row = 16 * lane < dim;
        turns = in_row && 8 * lane < half;
    }
};

template <int MODE>
__device__ __forceinline__ void turn(const RopeLane &l, float (&f)[2][8], const float (&cs)[8], const float (&sn)[8])
{
    if (MODE == kHalves) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float u = f[0][e], w = f[1][e];
            f[0][e] = u * cs[e] - w * sn[e];
            f[1][e] = w * cs[e] + u * sn[e];
        }
    } else if (MODE == kNeighbours) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {     // pair 8 lane + e: chunk e / 4, columns 2 (e % 4), + 1
            if (8 * l.lane + e >= l.half)
                continue;
            const float u = f[e / 4][2 * (e % 4)], w = f[e / 4][2 * (e % 4) + 1];
            f[e / 4][2 * (e % 4)] = u * cs[e] - w * sn[e];
            f[e / 4][2 * (e % 4) + 1] = w * cs[e] + u * sn[e];
        }
    }
}

// The turned value of column d, whose own value is x and whose partner's value
// partner(column) gives; for the layouts in which a lane has no partners (kHalvesOdd).
template <typename Partner>
__device__ __forceinline__ float turn_odd(int d, int half, float x, const float *c, const float *s, Partner partner)
{
    if (d < half)
        return x * c[d] - partner(d + half) * s[d];
    return d < 2 * half ? x * c[d - half] + partner(d - half) * s[d - half] : x;
}

// Sum over the lanes of a row; every lane gets it.
__device__ __forceinline__ float row_sum(float v, int lanes)
{
    for (int o = lanes >> 1; o > 0; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The cosines and sines of the pairs 8 lane .. 8 lane + 7 of a position; `vec`:
// whole pieces of 16 bytes.
__device__ __forceinline__ void load_angles(const RopeLane &l, const float *c, const float *s, int vec, float (&cs)[8], float (&sn)[8])
{
    if (vec) {
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
            const float4 u = __ldg(reinterpret_cast<const float4 *>(c + e)), w = __ldg(reinterpret_cast<const float4 *>(s + e));
            cs[e] = u.x, cs[e + 1] = u.y, cs[e + 2] = u.z, cs[e + 3] = u.w;
            sn[e] = w.x, sn[e + 1] = w.y, sn[e + 2] = w.z, sn[e + 3] = w.w;
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (8 * l.lane + e < l.half) {
                cs[e] = __ldg(c + e);
                sn[e] = __ldg(s + e);
            }
    }
}

}  // namespace s3d8

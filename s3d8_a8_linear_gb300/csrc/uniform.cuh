// Values that all lanes of a warp have.
#pragma once

namespace s3d8 {

// Such a value as one that the compiler knows to be the same in all lanes: behind a branch on
// it, shuffles and votes need no check for lanes that are elsewhere (about 240 clocks each).
// Whole warps together.
template <typename T>
__device__ __forceinline__ T uniform(T x)
{
    return __shfl_sync(0xffffffffu, x, 0);
}

__device__ __forceinline__ int warp_index() { return uniform((int)threadIdx.x >> 5); }

}  // namespace s3d8

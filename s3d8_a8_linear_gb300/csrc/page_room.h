// Which entries of a call that takes pages find them (pages.cu).
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define S3D8_BOTH __host__ __device__ __forceinline__
#else
#define S3D8_BOTH inline
#endif

namespace s3d8 {

// The rank of an entry's first page among all that the call wants, from the sum of
// the needs in front of it.  Entries of wide tables can want more than 2^31 pages in
// all; their ranks stay at 2^31 - 1, which is beyond any pool.
S3D8_BOTH int32_t page_rank(int64_t wanted) { return wanted < 0x7FFFFFFF ? (int32_t)wanted : 0x7FFFFFFF; }

// Whether an entry's `need` pages (below 0: refused already) are among the `free` ones.
S3D8_BOTH bool page_room(int32_t rank, int32_t need, int32_t free)
{
    return need == 0 || (need > 0 && (int64_t)rank + need <= free);
}

}  // namespace s3d8

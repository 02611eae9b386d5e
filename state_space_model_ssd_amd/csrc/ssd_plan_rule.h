// How a packed batch's chunks are counted (internal; host code may include it too).
#pragma once

#ifdef __HIPCC__
#define SSD_PLAN_FN __host__ __device__ __forceinline__
#else
#define SSD_PLAN_FN inline
#endif

namespace ssd {

// a + b, but `most` at most (both are 0 to `most`): lengths that run back and forth over the
// tokens add up to more chunks than there is room for, 128 times 2^24 already among 256 sequences,
// which is past 32 bits.
SSD_PLAN_FN int add_chunks(int a, int b, int most) { return b < most - a ? a + b : most; }

}  // namespace ssd

#undef SSD_PLAN_FN

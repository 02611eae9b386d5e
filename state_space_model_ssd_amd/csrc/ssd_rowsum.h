// Sums over runs of lanes by register exchanges (internal).
#pragma once

#include "ssd_common.h"

namespace ssd {

// v plus the value of the lane that DPP control CTRL selects.
template <int CTRL>
__device__ __forceinline__ float dpp_xadd(float v) {
  const int o = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, false);
  return v + __builtin_bit_cast(float, o);
}

// run_sum's butterfly (ssd_gate.h) (lane i adds lane i ^ off, off = 1, 2, 4, ... below n),
// the same additions in the same order and so the same result bit for bit,
// with the exchanges in registers instead of LDS permutes.  Lanes ^1 and ^2
// come by quad permutes; ^4 and ^8 by mirroring within 8 and 16 lanes, which
// reaches a lane holding the same value once the smaller runs agree.  Then
// every row of 16 lanes holds one value r0..r3, so the ^16 step gives
// r0 + r1 in the lower half and r2 + r3 in the upper one (a lane's own row
// plus its partner's, in either order the same sum) and the ^32 step their
// sum.  n: a power of two <= 64, the same in every lane.
__device__ __forceinline__ float run_sum_dpp(float v, int n) {
  if (n > 1) v = dpp_xadd<0xb1>(v);    // quad_perm [1,0,3,2]
  if (n > 2) v = dpp_xadd<0x4e>(v);    // quad_perm [2,3,0,1]
  if (n > 4) v = dpp_xadd<0x141>(v);   // row_half_mirror
  if (n > 8) v = dpp_xadd<0x140>(v);   // row_mirror
  if (n > 16) {
    const int b = __builtin_bit_cast(int, v);
    const float r0 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 0));
    const float r1 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 16));
    const float r2 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 32));
    const float r3 = __builtin_bit_cast(float, __builtin_amdgcn_readlane(b, 48));
    const float lo = r0 + r1, hi = r2 + r3;
    v = n > 32 ? lo + hi : ((threadIdx.x & 32) ? hi : lo);
  }
  return v;
}

}  // namespace ssd

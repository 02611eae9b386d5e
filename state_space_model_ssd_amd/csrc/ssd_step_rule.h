// How the single-token state update divides a head's state (internal, host only).
#pragma once

#include <stdint.h>

namespace ssd {

// Lanes per row: N's accesses rounded up to a power of two, at most a wave.
inline int step_lpr(int N) {
  const int V = N >= 4 ? 4 : 1;
  int l = 1;
  while (l * V < N) l *= 2;
  return l;
}

// Rows per thread: more rows are more bytes in flight per wave and fewer
// workgroups to start, fewer rows more waves.  Measured (us, R = 1 / 2 / 4; P 64,
// N 128): one sequence of 24 heads 3.16 / 3.35 / 3.83, four 4.58 / 4.17 / 4.33, 32 18.0
// / 12.6 / 11.3; 64 sequences of 32 heads 38.9 / 24.6 / 23.4; 256, whose states pass
// the last-level cache, 156 / 103 / 106 (5.1 TB/s, a large copy's rate).  So four
// rows from one workgroup (of 256 threads) per CU on, two from half a one, and two
// again for states larger than the cache (256 MB).
inline int step_rows(int64_t batch, int64_t H, int64_t P, int N) {
  if (N < 4) return 1;
  const int64_t lanes = batch * H * P * step_lpr(N);
  if (lanes < 2 * 128 * 256) return 1;
  if (lanes < 4 * 256 * 256 || lanes >= 1 << 24) return 2;
  return 4;
}

}  // namespace ssd

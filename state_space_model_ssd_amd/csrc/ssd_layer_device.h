// Device-side building blocks of the operators around the SSD (internal):
// vector accesses at the element's own alignment, and the column sums that
// finish a weight gradient.
#pragma once

#include "ssd_common.h"

namespace ssd {

// V elements of T in registers as they lie in memory.  The type has the
// element's alignment, so a row may start at any element: gfx950 takes a
// global access of up to 16 bytes at any address.
template <int BYTES, int ALIGN> struct RawVec;
#define SSD_RAW(B, A, TYPE)                                                     \
  template <> struct RawVec<B, A> {                                             \
    typedef TYPE __attribute__((may_alias, aligned(A))) mem;                    \
    typedef TYPE reg;                                                           \
  };
SSD_RAW(16, 2, u32x4)
SSD_RAW(16, 4, u32x4)
typedef unsigned u32x2v __attribute__((ext_vector_type(2)));
SSD_RAW(8, 2, u32x2v)
SSD_RAW(8, 4, u32x2v)
SSD_RAW(4, 2, unsigned)
SSD_RAW(4, 4, unsigned)
SSD_RAW(2, 2, unsigned short)
#undef SSD_RAW

template <typename T, int V> struct Vec {
  static constexpr int B = (int)sizeof(T) * V;         // bytes
  static constexpr int NP = B > 16 ? B / 16 : 1;       // accesses
  static constexpr int PB = B / NP, PV = V / NP;
  using raw = RawVec<PB, (int)sizeof(T)>;
  typename raw::reg q[NP];

  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < NP; ++i) q[i] = *reinterpret_cast<const typename raw::mem*>(p + i * PV);
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < NP; ++i) *reinterpret_cast<typename raw::mem*>(p + i * PV) = q[i];
  }
  // The first n elements only (n < V: a row's end), zeros after them.
  __device__ __forceinline__ void load_some(const T* p, int n) {
    T e[V];
#pragma unroll
    for (int i = 0; i < V; ++i) e[i] = i < n ? p[i] : static_cast<T>(0.f);
    __builtin_memcpy(q, e, B);
  }
  __device__ __forceinline__ void store_some(T* p, int n) const {
    T e[V];
    __builtin_memcpy(e, q, B);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < n) p[i] = e[i];
  }
  __device__ __forceinline__ void clear() { __builtin_memset(q, 0, B); }
  __device__ __forceinline__ void clear_unless(bool keep) {
#pragma unroll
    for (int i = 0; i < NP; ++i) q[i] = keep ? q[i] : (typename raw::reg)(0);
  }
  __device__ __forceinline__ void get(float (&f)[V]) const {
    T e[V];
    __builtin_memcpy(e, q, B);
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = to_f32(e[i]);
  }
  __device__ __forceinline__ void set(const float (&f)[V]) {
    T e[V];
#pragma unroll
    for (int i = 0; i < V; ++i) e[i] = from_f32<T>(f[i]);
    __builtin_memcpy(q, e, B);
  }
};

// sigmoid(z) = 1 / (1 + e^-z).  fp32 tensors take the accurate exponential and
// division; bf16 ones the hardware's (a few units in the last place of fp32,
// far below one rounding to bf16).  e^-z may overflow to infinity: sigmoid 0.
template <typename T> __device__ __forceinline__ float sigmoid(float z) {
  if constexpr (sizeof(T) == 2) return __builtin_amdgcn_rcpf(1.f + __expf(-z));
  else return 1.f / (1.f + expf(-z));
}

// Whether a row of a single-token batch is padding: its slot lies outside
// the cache, or an earlier row has the same slot (the first row has it: no two
// workgroups ever write one state).  Every thread of the workgroup calls it.
// Costs one load per thread and 256 rows, in flight with the row's others.
__device__ __forceinline__ bool step_row_is_padding(const int32_t* slots, int row, int64_t nslots,
                                                    int64_t& slot) {
  if (!slots) {
    slot = row;
    return false;
  }
  const int32_t mine = slots[row];
  slot = mine;
  int seen = 0;
  for (int i = threadIdx.x; i < row; i += blockDim.x) seen |= slots[i] == mine;
  return __syncthreads_or(seen) || mine < 0 || mine >= nslots;
}

// Sums over the rows of part[nparts][cols]: OUT::put(column, sum).  One
// workgroup of 16 waves per 64 columns; wave w adds rows w, w + 16, ... in
// order, eight loads in flight, then the wave sums are added in wave order.
// No atomics: the order never changes.
constexpr int kColsumThreads = 1024;
template <typename OUT>
__global__ __launch_bounds__(kColsumThreads) void colsum_kernel(const float* __restrict__ part,
                                                                int nparts, int cols, OUT out) {
  __shared__ float sums[16][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int col = blockIdx.x * 64 + lane;
  const int c = col < cols ? col : cols - 1;
  float t = 0.f;
  int r = w;
  for (; r + 7 * 16 < nparts; r += 8 * 16) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = part[(int64_t)(r + 16 * i) * cols + c];
#pragma unroll
    for (int i = 0; i < 8; ++i) t += v[i];
  }
  for (; r < nparts; r += 16) t += part[(int64_t)r * cols + c];
  sums[w][lane] = t;
  __syncthreads();
  if (w > 0 || col >= cols) return;
#pragma unroll
  for (int q = 1; q < 16; ++q) t += sums[q][lane];
  out.put(col, t);
}

}  // namespace ssd

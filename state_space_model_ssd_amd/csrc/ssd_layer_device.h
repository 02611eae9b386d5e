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

// Accesses as a scalar base plus a 32-bit lane offset, which the memory unit adds.
// Left alone, the compiler adds the lane's offset to the tensor's base first, so
// that every row costs each lane a 64-bit addition and two registers, and forms
// the bases of all of an unrolled loop's rows up front, more than the scalar
// registers hold.  Two empty asm statements keep the form: one on the lane's
// offset, in the block of the access, and one on the base at each use, after
// which the next row's base can only be formed from it.
__device__ __forceinline__ uint32_t lane_offset(uint32_t off) {
  asm("" : "+v"(off));
  return off;
}

// The row a wave is at in a tensor: an address that is the same in every lane.
struct RowCursor {
  uint64_t at;
  template <typename T>
  __device__ __forceinline__ explicit RowCursor(const T* p) : at(reinterpret_cast<uint64_t>(p)) {}
  __device__ __forceinline__ __attribute__((address_space(1))) char* here() {
    asm("" : "+s"(at));
    return reinterpret_cast<__attribute__((address_space(1))) char*>(at);
  }
  __device__ __forceinline__ void move(int64_t bytes) { at += bytes; }
};

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
  // `off` (a lane_offset) bytes into the cursor's row.
  __device__ __forceinline__ void load_at(RowCursor& row, uint32_t off) {
    const __attribute__((address_space(1))) char* p = row.here() + off;
#pragma unroll
    for (int i = 0; i < NP; ++i)
      q[i] = *reinterpret_cast<const __attribute__((address_space(1))) typename raw::mem*>(p + i * PB);
  }
  __device__ __forceinline__ void store_at(RowCursor& row, uint32_t off) const {
    __attribute__((address_space(1))) char* p = row.here() + off;
#pragma unroll
    for (int i = 0; i < NP; ++i)
      *reinterpret_cast<__attribute__((address_space(1))) typename raw::mem*>(p + i * PB) = q[i];
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

// sigmoid(z) = 1 / (1 + e^-z) by the hardware's exponential and reciprocal, in
// fp32 for either type: the argument's rounding puts |z| 2^-23 and the functions
// some 2^-22 relative on e^-z, which weighs by its share of 1 + e^-z, so the
// result is off by a few units in the last place of fp32 for z >= -4 and by
// |z| of them below, where it is itself e^z.  e^-z may overflow to infinity:
// sigmoid 0.
__device__ __forceinline__ float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.f + __expf(-z));
}

// The slot of a row of a single-token batch.  A row is padding if its slot lies
// outside the cache, or if an earlier row has the same slot (the first row has
// it: no two rows ever write one state).  Every wave looks through the earlier
// rows by itself, 64 at a time, so no barrier is needed: begin() issues the
// loads of the nearest 256 without waiting for them, and the caller issues its
// own loads before repeated() uses them.
struct StepSlot {
  static constexpr int kAhead = 4;
  const int32_t* slots;
  int row, mine;
  int32_t near[kAhead];

  // False: outside the cache.  Uniform over the workgroup.
  __device__ __forceinline__ bool begin(const int32_t* s, int r, int64_t nslots) {
    slots = s;
    row = r;
    mine = s ? s[r] : r;
    if (mine < 0 || mine >= nslots) return false;
    if (s) {
      const int lane = threadIdx.x & 63;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) near[i] = s[max(row - 1 - lane - 64 * i, 0)];
    }
    return true;
  }
  __device__ __forceinline__ bool repeated() const {
    if (!slots) return false;
    const int lane = threadIdx.x & 63;
    bool seen = false;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) seen |= lane + 64 * i < row && near[i] == mine;
    for (int i = row - 1 - lane - 64 * kAhead; i >= 0; i -= 64) seen |= slots[i] == mine;
    return __any(seen);
  }
};

// Sums over the rows of part[nparts][cols]: OUT::put(column, sum).  One
// workgroup per 32 columns (whole lines of the partial rows): 32 groups of 32
// lanes, group g adding rows g, g + 32, ... in order with sixteen loads in
// flight, then the groups' sums are added in a fixed order.  No atomics: the
// order never changes.
constexpr int kColsumThreads = 1024, kColsumCols = 32;
template <typename OUT>
__global__ __launch_bounds__(kColsumThreads) void colsum_kernel(const float* __restrict__ part,
                                                                int nparts, int cols, OUT out) {
  constexpr int NG = kColsumThreads / kColsumCols, NL = 16;
  __shared__ float sums[NG][kColsumCols];
  const int lane = threadIdx.x % kColsumCols, g = threadIdx.x / kColsumCols;
  const int col = blockIdx.x * kColsumCols + lane;
  const int c = col < cols ? col : cols - 1;
  float t = 0.f;
  for (int r = g; r < nparts; r += NL * NG) {
    float v[NL];                                  // rows past the last: the last again, unused
#pragma unroll
    for (int i = 0; i < NL; ++i) v[i] = part[(int64_t)min(r + NG * i, nparts - 1) * cols + c];
#pragma unroll
    for (int i = 0; i < NL; ++i) t += r + NG * i < nparts ? v[i] : 0.f;
  }
  sums[g][lane] = t;
  __syncthreads();
  if (g >= 2) return;                             // the first wave: half the groups each
  t = 0.f;
#pragma unroll
  for (int q = 0; q < NG / 2; ++q) t += sums[g * (NG / 2) + q][lane];
  t += __shfl_xor(t, 32);
  if (g == 0 && col < cols) out.put(col, t);
}
template <typename OUT>
inline hipError_t colsum(const float* part, int nparts, int cols, const OUT& out, hipStream_t s) {
  hipLaunchKernelGGL(colsum_kernel<OUT>, dim3((cols + kColsumCols - 1) / kColsumCols),
                     dim3(kColsumThreads), 0, s, part, nparts, cols, out);
  return hipGetLastError();
}

}  // namespace ssd

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

// Partial sums of the weight gradients: one row per workgroup of the launch that
// makes them, `part_cols` columns per weight.  They lie in blocks of 32 columns (one
// line), [column / 32][row][32], so that the workgroup that adds a block reads one run
// of memory, 16 bytes per lane.  Measured with their kernel (us), rows of all columns /
// blocks of 32 / blocks of 16: convolution backward 1792 ch x 8192 24.2 / 23.3 / 23.8,
// 160 ch x 6349 10.4 / 10.1 / 10.2; norm backward 8192 x 768 37.0 / 36.5 / 37.1, 8192 x
// 2048 76.4 / 76.9 / 78.6 (blocks of 16 are written as half lines).
constexpr int kPartBlock = 32;
__host__ __device__ inline int64_t part_cols(int64_t C) {
  return (C + kPartBlock - 1) / kPartBlock * kPartBlock;
}
__device__ __forceinline__ float* part_at(float* part, int row, int nparts, int col) {
  return part + ((int64_t)(col / kPartBlock) * nparts + row) * kPartBlock + col % kPartBlock;
}

// Sums over the partial rows, one workgroup per block of columns: OUT::put(column,
// sum) for each.  LN lanes load a row's block, group g of them adds rows g, g + NG,
// ... in order, then the groups' sums are added in a fixed order.  No atomics: the
// order never changes.
template <typename OUT, int THREADS, int NL>
__global__ __launch_bounds__(THREADS) void colsum_kernel(const float* __restrict__ part, int nparts,
                                                         OUT out) {
  constexpr int LN = kPartBlock / 4, NG = THREADS / LN, NW = THREADS / 64;
  __shared__ float sums[NW][kPartBlock];
  const int g = threadIdx.x / LN, c = threadIdx.x % LN * 4;
  const float* p = part + (int64_t)blockIdx.x * nparts * kPartBlock + c;
  float t[4] = {0.f, 0.f, 0.f, 0.f};
  for (int r = g; r < nparts; r += NL * NG) {
    Vec<float, 4> q[NL];                          // rows past the last: the last again, unused
#pragma unroll
    for (int i = 0; i < NL; ++i) q[i].load(p + (int64_t)min(r + NG * i, nparts - 1) * kPartBlock);
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      float f[4];
      q[i].get(f);
#pragma unroll
      for (int e = 0; e < 4; ++e) t[e] += r + NG * i < nparts ? f[e] : 0.f;
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
#pragma unroll
    for (int d = LN; d < 64; d *= 2) t[e] += __shfl_xor(t[e], d);
  }
  if ((threadIdx.x & 63) < LN) {
#pragma unroll
    for (int e = 0; e < 4; ++e) sums[threadIdx.x / 64][c + e] = t[e];
  }
  __syncthreads();
  if (threadIdx.x >= kPartBlock) return;
  float v = 0.f;
#pragma unroll
  for (int w = 0; w < NW; ++w) v += sums[w][threadIdx.x];
  out.put((int)blockIdx.x * kPartBlock + (int)threadIdx.x, v);
}
// `cols` is whole blocks.  Few rows: small workgroups.
template <typename OUT>
inline hipError_t colsum(const float* part, int nparts, int64_t cols, const OUT& out, hipStream_t s) {
  const dim3 grid((unsigned)(cols / kPartBlock));
  if (nparts <= 256) hipLaunchKernelGGL((colsum_kernel<OUT, 256, 4>), grid, dim3(256), 0, s, part, nparts, out);
  else hipLaunchKernelGGL((colsum_kernel<OUT, 1024, 8>), grid, dim3(1024), 0, s, part, nparts, out);
  return hipGetLastError();
}

}  // namespace ssd

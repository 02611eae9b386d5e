// Device-side building blocks of the gated delta rule (internal): operands of 16x16
// matrix instructions over 32 values of the contracted axis, exact or as pairs.
//
// Every product here contracts 32 values per step.  Lane i holds eight consecutive ones,
// 8 (i / 16) .. + 7, of row (first operand) or column (second) i % 16; bf16 takes one
// 16x16x32 instruction, fp32 eight 16x16x4 ones, the e-th with value e of every lane.
// Either way the operands lie alike, so one kernel text serves both types.
//
// Results feed the next product without leaving their registers.  A result tile's lane i
// holds rows 4 (i / 16) .. + 3 of column i % 16.  With the rows of the two tiles of a
// 32-row block dealt out as tile_row() does, lane i's four values of the first and four of
// the second tile are rows 8 (i / 16) .. + 7 of the block: the second operand (or, turned,
// the first) of a product that contracts these rows.
//
// With bf16 inputs a value that is not an input goes into a product either rounded once
// (2^-8 of it at most, where the result is rounded to bf16 itself), or as the sum of two bf16
// (2^-17 of it, where it is part of a state, whose error would last): the products of two
// such pairs leave out the two low parts' product (2^-16 at most).
#pragma once

#include "ssd_common.h"
#include "ssd_delta.h"

namespace ssd {

struct Pair {             // hi + lo
  bf16x8 hi, lo;
};
struct F8 {
  float v[8];
};

template <typename T> struct Opnd;
template <> struct Opnd<bf16> {
  using X = bf16x8;                    // exact or rounded
  using S = Pair;                      // to 2^-17
  static constexpr int PX = 1, PS = 2; // 16-byte pieces per lane
  // Two values at a time, as the conversion takes them.
  __device__ __forceinline__ static X round(const float (&f)[8]) {
    u32x4 x;
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = pack(f[2 * e], f[2 * e + 1]);
    return __builtin_bit_cast(X, x);
  }
  __device__ __forceinline__ static S split(const float (&f)[8]) {
    u32x4 hi, lo;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      hi[e] = pack(f[2 * e], f[2 * e + 1]);
      lo[e] = pack(f[2 * e] - __builtin_bit_cast(float, hi[e] << 16),
                   f[2 * e + 1] - __builtin_bit_cast(float, hi[e] & 0xffff0000u));
    }
    return {__builtin_bit_cast(X, hi), __builtin_bit_cast(X, lo)};
  }
  __device__ __forceinline__ static uint32_t pack(float a, float b) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
  }
  __device__ __forceinline__ static X hi(const S& s) { return s.hi; }
  __device__ __forceinline__ static void get(const X& x, float (&f)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = static_cast<float>(x[e]);
  }
};
template <> struct Opnd<float> {
  using X = F8;
  using S = F8;
  static constexpr int PX = 2, PS = 2;
  __device__ __forceinline__ static X round(const float (&f)[8]) {
    X x;
#pragma unroll
    for (int e = 0; e < 8; ++e) x.v[e] = f[e];
    return x;
  }
  __device__ __forceinline__ static S split(const float (&f)[8]) { return round(f); }
  __device__ __forceinline__ static X hi(const S& s) { return s; }
  __device__ __forceinline__ static void get(const X& x, float (&f)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = x.v[e];
  }
};

// A product's instructions one by one: step i of `steps`.  Low parts come first.
__device__ __forceinline__ f32x4 mma16(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
// What is kept of a value for a later product: a pair, or rounded.
template <typename T, bool PAIR> struct Kept { using V = typename Opnd<T>::X; };
template <typename T> struct Kept<T, true> { using V = typename Opnd<T>::S; };

template <typename A, typename B> struct Steps;
template <> struct Steps<bf16x8, bf16x8> {
  static constexpr int n = 1;
  __device__ __forceinline__ static f32x4 step(int, bf16x8 a, bf16x8 b, f32x4 c) { return mma16(a, b, c); }
};
template <> struct Steps<bf16x8, Pair> {
  static constexpr int n = 2;
  __device__ __forceinline__ static f32x4 step(int i, bf16x8 a, const Pair& b, f32x4 c) {
    return mma16(a, i ? b.hi : b.lo, c);
  }
};
template <> struct Steps<Pair, bf16x8> {
  static constexpr int n = 2;
  __device__ __forceinline__ static f32x4 step(int i, const Pair& a, bf16x8 b, f32x4 c) {
    return mma16(i ? a.hi : a.lo, b, c);
  }
};
template <> struct Steps<Pair, Pair> {
  static constexpr int n = 3;
  __device__ __forceinline__ static f32x4 step(int i, const Pair& a, const Pair& b, f32x4 c) {
    return mma16(i == 0 ? a.lo : a.hi, i == 1 ? b.lo : b.hi, c);
  }
};
template <> struct Steps<F8, F8> {
  static constexpr int n = 8;
  __device__ __forceinline__ static f32x4 step(int i, const F8& a, const F8& b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[i], b.v[i], c, 0, 0, 0);
  }
};

template <typename A, typename B>
__device__ __forceinline__ f32x4 mma(const A& a, const B& b, f32x4 c) {
#pragma unroll
  for (int i = 0; i < Steps<A, B>::n; ++i) c = Steps<A, B>::step(i, a, b, c);
  return c;
}
// c[m] += a[m] b for M results: an instruction that adds to the result of the
// one before waits for it, so the results take turns.
template <int M, typename A, typename B>
__device__ __forceinline__ void mma_rows(const A (&a)[M], const B& b, f32x4* c) {
#pragma unroll
  for (int i = 0; i < Steps<A, B>::n; ++i)
#pragma unroll
    for (int m = 0; m < M; ++m) c[m] = Steps<A, B>::step(i, a[m], b, c[m]);
}

constexpr f32x4 kZero4 = {0.f, 0.f, 0.f, 0.f};

template <typename T, bool PAIR>
__device__ __forceinline__ typename Kept<T, PAIR>::V keep(const float (&f)[8]) {
  if constexpr (PAIR) return Opnd<T>::split(f);
  else return Opnd<T>::round(f);
}
template <typename T, bool PAIR>
__device__ __forceinline__ typename Kept<T, PAIR>::V keep(const typename Opnd<T>::S& s) {
  if constexpr (PAIR) return s;
  else return Opnd<T>::hi(s);
}
// Arrays of T that hold it: a pair's high and low parts.
template <typename T, bool PAIR> constexpr int kPlanes = PAIR && sizeof(T) == 2 ? 2 : 1;

// Row of result tile t (of 16) that lies in its row i of the instruction.
__device__ __forceinline__ int tile_row(int t, int i) {
  return 32 * (t >> 1) + 4 * (t & 1) + 8 * (i >> 2) + (i & 3);
}

// The eight values of a 32-row block's two tiles, in the order of their rows.
__device__ __forceinline__ void block8(f32x4 t0, f32x4 t1, float (&f)[8]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f[e] = t0[e];
    f[4 + e] = t1[e];
  }
}

// Operands from memory: 8 elements at p (16-byte aligned).
__device__ __forceinline__ bf16x8 load_opnd(const bf16* p) {
  return *reinterpret_cast<const bf16x8*>(p);
}
__device__ __forceinline__ F8 load_opnd(const float* p) {
  F8 f;
  const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
  block8(a, b, f.v);
  return f;
}
__device__ __forceinline__ bf16x8 load_opnd(__amdgpu_buffer_rsrc_t r, uint32_t off, bf16) {
  return __builtin_bit_cast(bf16x8, buf_load16(r, off));
}
__device__ __forceinline__ F8 load_opnd(__amdgpu_buffer_rsrc_t r, uint32_t off, float) {
  F8 f;
  block8(__builtin_bit_cast(f32x4, buf_load16(r, off)), __builtin_bit_cast(f32x4, buf_load16(r, off + 16)),
         f.v);
  return f;
}
__device__ __forceinline__ void store_opnd(bf16* p, bf16x8 v) { *reinterpret_cast<bf16x8*>(p) = v; }
__device__ __forceinline__ void store_opnd(float* p, const F8& v) {
  *reinterpret_cast<f32x4*>(p) = f32x4{v.v[0], v.v[1], v.v[2], v.v[3]};
  *reinterpret_cast<f32x4*>(p + 4) = f32x4{v.v[4], v.v[5], v.v[6], v.v[7]};
}

// Operands in memory and LDS: pieces of 64 lanes' 16 bytes, one lane after another, each a
// 16x32 tile of rounded bf16; a pair takes two (high parts, low parts), as does fp32 (values
// 0 to 3, 4 to 7).  A [N][64] matrix is in the order [32-block of columns][tile of rows].  Of a
// triangular [64][64] one the tiles that are not zero follow in the order (tile of rows,
// block of columns): lower (0,0) (1,0) (2,0) (3,0) (2,1) (3,1), upper (0,0) (1,0) (0,1) (1,1)
// (2,1) (3,1).
// Either way tile u of the second 32 columns follows two places behind.
__host__ __device__ constexpr int triangle_index(int u, int cb) { return u + 2 * cb; }
__device__ __forceinline__ int2 lower_tile(int i) { return i < 4 ? make_int2(i, 0) : make_int2(i - 2, 1); }
__device__ __forceinline__ int2 upper_tile(int i) { return i < 2 ? make_int2(i, 0) : make_int2(i - 2, 1); }

// The operand at `p`; `slot`: the lane's place in a piece.
__device__ __forceinline__ bf16x8 piece_x(const char* p, uint32_t slot, bf16) {
  return *reinterpret_cast<const bf16x8*>(p + slot);
}
__device__ __forceinline__ F8 piece_x(const char* p, uint32_t slot, float) {
  F8 f;
  block8(*reinterpret_cast<const f32x4*>(p + slot), *reinterpret_cast<const f32x4*>(p + kPiece + slot), f.v);
  return f;
}
// An operand from its 16-byte pieces.
__device__ __forceinline__ bf16x8 opnd_of(const uint4 (&q)[1], bf16) { return __builtin_bit_cast(bf16x8, q[0]); }
__device__ __forceinline__ F8 opnd_of(const uint4 (&q)[2], float) {
  F8 f;
  block8(__builtin_bit_cast(f32x4, q[0]), __builtin_bit_cast(f32x4, q[1]), f.v);
  return f;
}
__device__ __forceinline__ Pair piece_s(const char* p, uint32_t slot, bf16) {
  return {piece_x(p, slot, bf16{}), piece_x(p + kPiece, slot, bf16{})};
}
__device__ __forceinline__ F8 piece_s(const char* p, uint32_t slot, float) { return piece_x(p, slot, 0.f); }
__device__ __forceinline__ void put_piece(char* p, uint32_t slot, bf16x8 v) {
  *reinterpret_cast<bf16x8*>(p + slot) = v;
}
__device__ __forceinline__ void put_piece(char* p, uint32_t slot, const F8& v) {
  *reinterpret_cast<f32x4*>(p + slot) = f32x4{v.v[0], v.v[1], v.v[2], v.v[3]};
  *reinterpret_cast<f32x4*>(p + kPiece + slot) = f32x4{v.v[4], v.v[5], v.v[6], v.v[7]};
}
__device__ __forceinline__ void put_piece(char* p, uint32_t slot, const Pair& v) {
  put_piece(p, slot, v.hi);
  put_piece(p + kPiece, slot, v.lo);
}

// Sum over the four lanes that hold one column's rows.
__device__ __forceinline__ float column_sum(float v) {
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

}  // namespace ssd

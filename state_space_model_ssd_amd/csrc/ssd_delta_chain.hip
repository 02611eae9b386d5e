// The gated delta rule, the chain of states.  Per sequence, head and chunk, from the
// state S (P x N) entering the chunk and the chunk's T, A and decays (ssd_delta_prep.hip):
//   W = T (beta V - beta E K S^T)
//   O = scale E (Q S^T) + A W
//   S <- E_C S + (D W)^T K,     D_i = exp(G_C - G_i)
//
// Rows of S (values of the head) do not meet, so a wave owns 16 of them and carries them
// through the sequence in its registers, in fp32: S^T, W and the products between them
// chain result to operand without LDS.  Waves of a workgroup own neighbouring rows of one
// head and share what the chunk's products read besides: K, Q, K^T, T and A, copied to LDS
// as operands (64 lanes of 16 bytes each, one after another) by loads that write LDS
// directly, one chunk ahead where two chunks fit.
#include "ssd_delta_device.h"

#pragma clang fp contract(on)

namespace ssd {

namespace {

constexpr int C = kDeltaChunk;
constexpr int kPiece = 1024;              // 64 lanes of 16 bytes
constexpr int kLdsBytes = 160 * 1024;
typedef __attribute__((address_space(3))) void lds_void;

// 16 bytes per lane from `off` (zeros past the resource) to LDS, lane after lane.
__device__ __forceinline__ void copy_piece(__amdgpu_buffer_rsrc_t r, char* lds, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)lds, 16, off, 0, 0, 0);
}

// The operand at `p` in LDS: PX pieces, for pairs the high parts and then the low ones.
__device__ __forceinline__ bf16x8 lds_x(const char* p, int lane, bf16) {
  return *reinterpret_cast<const bf16x8*>(p + lane * 16);
}
__device__ __forceinline__ F8 lds_x(const char* p, int lane, float) {
  F8 f;
  block8(*reinterpret_cast<const f32x4*>(p + lane * 16),
         *reinterpret_cast<const f32x4*>(p + kPiece + lane * 16), f.v);
  return f;
}
__device__ __forceinline__ Pair lds_s(const char* p, int lane, bf16) {
  return {lds_x(p, lane, bf16{}), lds_x(p + kPiece, lane, bf16{})};
}
__device__ __forceinline__ F8 lds_s(const char* p, int lane, float) { return lds_x(p, lane, 0.f); }

// The six 16x32 tiles of a triangular [C][C] matrix that are not zero, in operand order:
// lower (0,0) (1,0) (2,0) (3,0) (2,1) (3,1) as (tile of rows, 32-block of columns).
__device__ __forceinline__ int2 lower_tile(int i) {
  return i < 4 ? make_int2(i, 0) : make_int2(i - 2, 1);
}
__device__ __forceinline__ constexpr int lower_at(int u, int cb) { return cb == 0 ? u : u + 2; }
// upper (0,0) (1,0) (0,1) (1,1) (2,1) (3,1)
__device__ __forceinline__ int2 upper_tile(int i) {
  return i < 2 ? make_int2(i, 0) : make_int2(i - 2, 1);
}
__device__ __forceinline__ constexpr int upper_at(int u, int cb) { return cb == 0 ? u : u + 2; }

// Copies the operands of a [rows][32 KB] matrix of T, pitch in bytes; `dealt`: tiles of
// rows as tile_row() deals them, else as they lie.
template <typename T, int TILES, int KB, bool DEALT, int NW>
__device__ __forceinline__ void copy_opnds(__amdgpu_buffer_rsrc_t r, char* lds, uint32_t pitch, int w,
                                           int lane) {
  constexpr int PX = Opnd<T>::PX;
  const int l16 = lane & 15;
  const uint32_t mine = (DEALT ? tile_row(0, l16) : l16) * pitch + (lane >> 4) * 8 * sizeof(T);
  for (int i = w; i < TILES * KB * PX; i += NW) {
    const int px = i % PX, kb = i / PX % KB, u = i / (PX * KB);
    const int base = DEALT ? 32 * (u >> 1) + 4 * (u & 1) : 16 * u;
    copy_piece(r, lds + i * kPiece, mine + base * pitch + kb * 32 * (uint32_t)sizeof(T) + px * 16);
  }
}
// The same of a triangular [C][C] matrix; PAIR: two bf16 planes where T is bf16.
template <typename T, bool LOWER, bool DEALT, bool PAIR, int NW>
__device__ __forceinline__ void copy_triangle(const void* m, char* lds, int w, int lane) {
  constexpr int PC = sizeof(T) == 4 || PAIR ? 2 : 1;
  constexpr uint32_t pitch = C * sizeof(T), step = sizeof(T) == 4 ? 16 : C * C * 2;
  const __amdgpu_buffer_rsrc_t r = buf_rsrc(m, C * C * (sizeof(T) == 4 ? 4 : 2 * PC));
  const int l16 = lane & 15;
  const uint32_t mine = (DEALT ? tile_row(0, l16) : l16) * pitch + (lane >> 4) * 8 * sizeof(T);
  for (int i = w; i < 6 * PC; i += NW) {
    const int2 t = LOWER ? lower_tile(i / PC) : upper_tile(i / PC);
    const int base = DEALT ? 32 * (t.x >> 1) + 4 * (t.x & 1) : 16 * t.x;
    copy_piece(r, lds + i * kPiece, mine + base * pitch + t.y * 32 * (uint32_t)sizeof(T) + i % PC * step);
  }
}

// A [C][16] tile of T, rows of the tile one after another: a wave's own columns.
template <typename T>
__device__ __forceinline__ void copy_columns(__amdgpu_buffer_rsrc_t r, char* lds, uint32_t pitch,
                                             int lane) {
  constexpr int LR = sizeof(T);                   // lanes per row of 16 values
  constexpr int RW = 64 / LR;                     // rows per piece
#pragma unroll
  for (int i = 0; i < C / RW; ++i)
    copy_piece(r, lds + i * kPiece, (i * RW + lane / LR) * pitch + lane % LR * 16);
}
// Rows 32 cb + 8 (lane / 16) .. + 7 of column lane % 16.
__device__ __forceinline__ bf16x8 column_opnd(const bf16* t, int cb, int lane) {
  return lds_operand_kmajor(t, 16, 32 * cb, 0, lane);
}
__device__ __forceinline__ F8 column_opnd(const float* t, int cb, int lane) {
  F8 f;
  const float* p = t + (32 * cb + 8 * (lane >> 4)) * 16 + (lane & 15);
#pragma unroll
  for (int e = 0; e < 8; ++e) f.v[e] = p[e * 16];
  return f;
}

// Values 32 cb + 8 (lane / 16) .. + 7 of a row of C floats.
__device__ __forceinline__ void row8(const float* p, int cb, int lane, float (&f)[8]) {
  p += 32 * cb + 8 * (lane >> 4);
  block8(*reinterpret_cast<const f32x4*>(p), *reinterpret_cast<const f32x4*>(p + 4), f);
}

// Bytes from the first of n rows to the end of the last one's `row` bytes.
__device__ __forceinline__ uint32_t rows_bytes(int n, uint32_t pitch, uint32_t row) {
  return n > 0 ? (uint32_t)(n - 1) * pitch + row : 0u;
}

// Workgroup -> (sequence, head) and its block of P: the blocks of one head, which read the
// same operands, run on the same XCD.
struct ChainTask {
  int seq, h, block;
  bool none;
};
__device__ __forceinline__ ChainTask chain_task(int b, int nstates, int H, int blocks) {
  const int x8 = b & 7, rest = b >> 3, unit = rest / blocks * 8 + x8;
  return {unit / H, unit % H, rest % blocks, unit >= nstates * H};
}
unsigned chain_grid(const DeltaArgs& a, int blocks) {
  return (unsigned)(((int64_t)a.nstates * a.H + 7) / 8 * 8 * blocks);
}

// S^T in its tiles from a state's rows, and back.
template <int N>
__device__ __forceinline__ void load_state(const float* p, int lane, f32x4 (&S)[N / 16]) {
#pragma unroll
  for (int kb = 0; kb < N / 32; ++kb) {
    const float* r = p + (int64_t)(lane & 15) * N + 32 * kb + 8 * (lane >> 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      S[2 * kb][e] = r[e];
      S[2 * kb + 1][e] = r[4 + e];
    }
  }
}
template <int N>
__device__ __forceinline__ void store_state(float* p, int lane, const f32x4 (&S)[N / 16]) {
#pragma unroll
  for (int kb = 0; kb < N / 32; ++kb) {
    float* r = p + (int64_t)(lane & 15) * N + 32 * kb + 8 * (lane >> 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      r[e] = S[2 * kb][e];
      r[4 + e] = S[2 * kb + 1][e];
    }
  }
}

// KEEP: for the backward, S and W are kept (as operands there: rounded) and O is not made.
template <typename T, int N, int NW, bool KEEP>
__global__ __launch_bounds__(64 * NW) void delta_chain_kernel(const DeltaArgs a, const ChunkMap cm,
                                                              int blocks) {
  using O = Opnd<T>;
  constexpr int NK = N / 32, NT = N / 16, PX = O::PX, PS = O::PS;
  constexpr int oK = 0, oT = oK + 4 * NK * PX, oKt = oT + 6 * PS, oQ = oKt + NT * 2 * PX;
  constexpr int oA = oQ + (KEEP ? 0 : 4 * NK * PX), oG = oA + (KEEP ? 0 : 6 * PX), oV = oG + 1;
  constexpr int VP = (int)sizeof(T);              // pieces of a wave's columns of V
  constexpr int SLOT = (oV + NW * VP) * kPiece;
  constexpr int NBUF = 2 * SLOT <= kLdsBytes ? 2 : 1;
  __shared__ __attribute__((aligned(16))) char lds[NBUF * SLOT];

  const ChainTask t = chain_task(blockIdx.x, a.nstates, a.H, blocks);
  if (t.none) return;
  const int w = wave_id(), lane = threadIdx.x & 63, l16 = lane & 15, la = lane >> 4;
  const int h = t.h, g = h / (a.H / a.G);
  const bool live = (t.block * NW + w) * 16 < a.P;
  const int p0 = live ? (t.block * NW + w) * 16 : 0;
  const int64_t srow = (((int64_t)t.seq * a.H + h) * a.P + p0) * N;
  const uint32_t qrow = (uint32_t)a.G * N * sizeof(T), vrow = (uint32_t)a.H * a.P * sizeof(T);

  f32x4 S[NT];
  if (a.init) {
    load_state<N>(a.init + srow, lane, S);
  } else {
#pragma unroll
    for (int i = 0; i < NT; ++i) S[i] = kZero4;
  }

  auto stage = [&](int j, char* b) {
    const ChunkDesc d = cm.desc(j);
    const int64_t jh = (int64_t)j * a.H + h, jg = (int64_t)j * a.G + g;
    const uint32_t qb = rows_bytes(d.len, qrow, N * sizeof(T));
    const int64_t qo = ((int64_t)d.start * a.G + g) * N;
    copy_opnds<T, 4, NK, true, NW>(buf_rsrc(static_cast<const T*>(a.k) + qo, qb), b + oK * kPiece, qrow, w, lane);
    copy_triangle<T, true, true, true, NW>(static_cast<const char*>(a.T) + jh * (C * C * 4), b + oT * kPiece, w, lane);
    copy_opnds<T, NT, 2, true, NW>(buf_rsrc(static_cast<const T*>(a.kt) + jg * N * C, N * C * sizeof(T)),
                                   b + oKt * kPiece, C * sizeof(T), w, lane);
    if constexpr (!KEEP) {
      copy_opnds<T, 4, NK, false, NW>(buf_rsrc(static_cast<const T*>(a.q) + qo, qb), b + oQ * kPiece, qrow, w, lane);
      copy_triangle<T, true, false, false, NW>(static_cast<const T*>(a.A) + jh * (C * C), b + oA * kPiece, w, lane);
    }
    if (w == 0) copy_piece(buf_rsrc(a.gates + jh * kGateFloats, kGateFloats * 4), b + oG * kPiece, lane * 16);
    const uint32_t vb = rows_bytes(d.len, vrow, 16 * sizeof(T));
    copy_columns<T>(buf_rsrc(static_cast<const T*>(a.v) + ((int64_t)d.start * a.H + h) * a.P + p0, vb),
                    b + (oV + w * VP) * kPiece, vrow, lane);
  };

  const int2 range = cm.seq_range(t.seq);
  if constexpr (NBUF == 2) {
    if (range.x < range.y) stage(range.x, lds);
  }
  for (int j = range.x; j < range.y; ++j) {
    char* b = lds + (NBUF == 2 ? ((j - range.x) & 1) * SLOT : 0);
    if constexpr (NBUF == 2) {
      __syncthreads();                            // chunk j is there, and chunk j - 1's slot free
      if (j + 1 < range.y) stage(j + 1, lds + ((j + 1 - range.x) & 1) * SLOT);
    } else {
      __syncthreads();
      stage(j, b);
      __syncthreads();
    }
    const ChunkDesc d = cm.desc(j);
    const int64_t jh = (int64_t)j * a.H + h;
    const float* gt = reinterpret_cast<const float*>(b + oG * kPiece);

    typename O::S sf[NK];
#pragma unroll
    for (int kb = 0; kb < NK; ++kb) {
      float f[8];
      block8(S[2 * kb], S[2 * kb + 1], f);
      sf[kb] = O::split(f);
    }
    f32x4 x[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      x[u] = kZero4;
#pragma unroll
      for (int kb = 0; kb < NK; ++kb) x[u] = mma(lds_x(b + (oK + (u * NK + kb) * PX) * kPiece, lane, T{}), sf[kb], x[u]);
    }
    typename O::S rf[2];
#pragma unroll
    for (int cb = 0; cb < 2; ++cb) {
      float f[8], v[8], be[8], E[8];
      block8(x[2 * cb], x[2 * cb + 1], f);
      O::get(column_opnd(reinterpret_cast<const T*>(b + (oV + w * VP) * kPiece), cb, lane), v);
      row8(gt, cb, lane, be);
      row8(gt + C, cb, lane, E);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = be[e] * (v[e] - E[e] * f[e]);
      rf[cb] = O::split(f);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      x[u] = kZero4;
#pragma unroll
      for (int cb = 0; cb <= u / 2; ++cb)
        x[u] = mma(lds_s(b + (oT + lower_at(u, cb) * PS) * kPiece, lane, T{}), rf[cb], x[u]);
    }
    typename O::X wf[2];
#pragma unroll
    for (int cb = 0; cb < 2; ++cb) {
      float f[8], D[8];
      block8(x[2 * cb], x[2 * cb + 1], f);
      wf[cb] = O::round(f);
      row8(gt + 2 * C, cb, lane, D);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] *= D[e];
      rf[cb] = O::split(f);
    }
    const float EC = gt[2 * C - 1];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      S[i] *= EC;
#pragma unroll
      for (int cb = 0; cb < 2; ++cb) S[i] = mma(lds_x(b + (oKt + (i * 2 + cb) * PX) * kPiece, lane, T{}), rf[cb], S[i]);
    }
    if constexpr (KEEP) {
      if (live) {
        T* s0 = static_cast<T*>(a.S0) + (jh * a.P + p0 + l16) * N + 8 * la;
#pragma unroll
        for (int kb = 0; kb < NK; ++kb) store_opnd(s0 + 32 * kb, O::hi(sf[kb]));
        T* wt = static_cast<T*>(a.Wt) + (jh * a.P + p0 + l16) * C + 8 * la;
#pragma unroll
        for (int cb = 0; cb < 2; ++cb) store_opnd(wt + 32 * cb, wf[cb]);
      }
    } else {
      // O with the state as first operand: rows are values, lane's column is a token
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        f32x4 o = kZero4;
#pragma unroll
        for (int kb = 0; kb < NK; ++kb) o = mma(O::hi(sf[kb]), lds_x(b + (oQ + (u * NK + kb) * PX) * kPiece, lane, T{}), o);
        o *= a.scale * gt[C + 16 * u + l16];
#pragma unroll
        for (int cb = 0; cb <= u / 2; ++cb)
          o = mma(wf[cb], lds_x(b + (oA + lower_at(u, cb) * PX) * kPiece, lane, T{}), o);
        const int c = 16 * u + l16;
        if (live && c < d.len) {
          T* out = static_cast<T*>(a.out) + ((int64_t)(d.start + c) * a.H + h) * a.P + p0 + 4 * la;
          T f[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) f[e] = from_f32<T>(o[e]);
          __builtin_memcpy(out, f, sizeof(f));
        }
      }
    }
  }
  if (!KEEP && a.final_states && live) store_state<N>(a.final_states + srow, lane, S);
}

// The chain backward: dS, the gradient of the state leaving the chunk, from the last chunk
// to the first.  With dO the output's gradient,
//   dW = A^T dO + D K dS^T,   dR = T^T dW       (dR: the gradient of beta V - beta E K S^T)
//   dS <- E_C dS + dO^T (scale E Q) - dR^T (beta E K)
// dS (before the update) and dR are kept for ssd_delta_local.hip.
template <typename T, int N, int NW>
__global__ __launch_bounds__(64 * NW) void delta_chain_bwd_kernel(const DeltaArgs a, const ChunkMap cm,
                                                                  int blocks) {
  using O = Opnd<T>;
  constexpr int NK = N / 32, NT = N / 16, PX = O::PX, PS = O::PS;
  constexpr int oK = 0, oA = oK + 4 * NK * PX, oT = oA + 6 * PS, oQt = oT + 6 * PS;
  constexpr int oKt = oQt + NT * 2 * PX, oG = oKt + NT * 2 * PX, oV = oG + 1;
  constexpr int VP = (int)sizeof(T);
  constexpr int SLOT = (oV + NW * VP) * kPiece;
  constexpr int NBUF = 2 * SLOT <= kLdsBytes ? 2 : 1;
  __shared__ __attribute__((aligned(16))) char lds[NBUF * SLOT];

  const ChainTask t = chain_task(blockIdx.x, a.nstates, a.H, blocks);
  if (t.none) return;
  const int w = wave_id(), lane = threadIdx.x & 63, l16 = lane & 15, la = lane >> 4;
  const int h = t.h, g = h / (a.H / a.G);
  const bool live = (t.block * NW + w) * 16 < a.P;
  const int p0 = live ? (t.block * NW + w) * 16 : 0;
  const int64_t srow = (((int64_t)t.seq * a.H + h) * a.P + p0) * N;
  const uint32_t qrow = (uint32_t)a.G * N * sizeof(T), vrow = (uint32_t)a.H * a.P * sizeof(T);

  f32x4 S[NT];
  if (a.dfinal) {
    load_state<N>(a.dfinal + srow, lane, S);
  } else {
#pragma unroll
    for (int i = 0; i < NT; ++i) S[i] = kZero4;
  }

  auto stage = [&](int j, char* b) {
    const ChunkDesc d = cm.desc(j);
    const int64_t jh = (int64_t)j * a.H + h, jg = (int64_t)j * a.G + g;
    const uint32_t qb = rows_bytes(d.len, qrow, N * sizeof(T));
    const int64_t qo = ((int64_t)d.start * a.G + g) * N;
    copy_opnds<T, 4, NK, true, NW>(buf_rsrc(static_cast<const T*>(a.k) + qo, qb), b + oK * kPiece, qrow, w, lane);
    copy_triangle<T, false, true, true, NW>(static_cast<const char*>(a.At) + jh * (C * C * 4), b + oA * kPiece, w, lane);
    copy_triangle<T, false, true, true, NW>(static_cast<const char*>(a.Tt) + jh * (C * C * 4), b + oT * kPiece, w, lane);
    copy_opnds<T, NT, 2, true, NW>(buf_rsrc(static_cast<const T*>(a.qt) + jg * N * C, N * C * sizeof(T)),
                                   b + oQt * kPiece, C * sizeof(T), w, lane);
    copy_opnds<T, NT, 2, true, NW>(buf_rsrc(static_cast<const T*>(a.kt) + jg * N * C, N * C * sizeof(T)),
                                   b + oKt * kPiece, C * sizeof(T), w, lane);
    if (w == 0) copy_piece(buf_rsrc(a.gates + jh * kGateFloats, kGateFloats * 4), b + oG * kPiece, lane * 16);
    const uint32_t vb = rows_bytes(d.len, vrow, 16 * sizeof(T));
    copy_columns<T>(buf_rsrc(static_cast<const T*>(a.dout) + ((int64_t)d.start * a.H + h) * a.P + p0, vb),
                    b + (oV + w * VP) * kPiece, vrow, lane);
  };

  const int2 range = cm.seq_range(t.seq);
  const int last = range.y - 1;
  if constexpr (NBUF == 2) {
    if (range.x < range.y) stage(last, lds);
  }
  for (int j = last; j >= range.x; --j) {
    char* b = lds + (NBUF == 2 ? ((last - j) & 1) * SLOT : 0);
    if constexpr (NBUF == 2) {
      __syncthreads();
      if (j > range.x) stage(j - 1, lds + ((last - j + 1) & 1) * SLOT);
    } else {
      __syncthreads();
      stage(j, b);
      __syncthreads();
    }
    const int64_t jh = (int64_t)j * a.H + h;
    const float* gt = reinterpret_cast<const float*>(b + oG * kPiece);

    typename O::S sf[NK];
#pragma unroll
    for (int kb = 0; kb < NK; ++kb) {
      float f[8];
      block8(S[2 * kb], S[2 * kb + 1], f);
      sf[kb] = O::split(f);
    }
    typename O::X of[2];
#pragma unroll
    for (int cb = 0; cb < 2; ++cb) of[cb] = column_opnd(reinterpret_cast<const T*>(b + (oV + w * VP) * kPiece), cb, lane);
    f32x4 x[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      x[u] = kZero4;
#pragma unroll
      for (int kb = 0; kb < NK; ++kb) x[u] = mma(lds_x(b + (oK + (u * NK + kb) * PX) * kPiece, lane, T{}), sf[kb], x[u]);
    }
    typename O::S rf[2];
#pragma unroll
    for (int cb = 0; cb < 2; ++cb) {
      float D[8];
      row8(gt + 2 * C, cb, lane, D);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int u = 2 * cb + i;
#pragma unroll
        for (int e = 0; e < 4; ++e) x[u][e] *= D[4 * i + e];
#pragma unroll
        for (int k = cb; k < 2; ++k) x[u] = mma(lds_s(b + (oA + upper_at(u, k) * PS) * kPiece, lane, T{}), of[k], x[u]);
      }
      float f[8];
      block8(x[2 * cb], x[2 * cb + 1], f);
      rf[cb] = O::split(f);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      x[u] = kZero4;
#pragma unroll
      for (int k = u / 2; k < 2; ++k) x[u] = mma(lds_s(b + (oT + upper_at(u, k) * PS) * kPiece, lane, T{}), rf[k], x[u]);
    }
    typename O::S qf[2];
#pragma unroll
    for (int cb = 0; cb < 2; ++cb) {
      float f[8], be[8], E[8], o[8];
      block8(x[2 * cb], x[2 * cb + 1], f);
      if (live) store_opnd(static_cast<T*>(a.dRt) + (jh * a.P + p0 + l16) * C + 32 * cb + 8 * la, O::round(f));
      row8(gt, cb, lane, be);
      row8(gt + C, cb, lane, E);
      O::get(of[cb], o);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        f[e] *= -be[e] * E[e];
        o[e] *= a.scale * E[e];
      }
      rf[cb] = O::split(f);
      qf[cb] = O::split(o);
    }
    if (live) {
      T* ds = static_cast<T*>(a.dS) + (jh * a.P + p0 + l16) * N + 8 * la;
#pragma unroll
      for (int kb = 0; kb < NK; ++kb) store_opnd(ds + 32 * kb, O::hi(sf[kb]));
    }
    const float EC = gt[2 * C - 1];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      S[i] *= EC;
#pragma unroll
      for (int cb = 0; cb < 2; ++cb) {
        S[i] = mma(lds_x(b + (oQt + (i * 2 + cb) * PX) * kPiece, lane, T{}), qf[cb], S[i]);
        S[i] = mma(lds_x(b + (oKt + (i * 2 + cb) * PX) * kPiece, lane, T{}), rf[cb], S[i]);
      }
    }
  }
  if (a.dinit && live) store_state<N>(a.dinit + srow, lane, S);
}

enum class Chain { fwd, keep, bwd };

template <Chain K, typename T, int N, int NW>
hipError_t chain_go(const DeltaArgs& a, hipStream_t s) {
  const int blocks = (a.P + 16 * NW - 1) / (16 * NW);
  const dim3 grid(chain_grid(a, blocks)), th(64 * NW);
  if constexpr (K == Chain::bwd)
    hipLaunchKernelGGL((delta_chain_bwd_kernel<T, N, NW>), grid, th, 0, s, a, a.cmap(), blocks);
  else
    hipLaunchKernelGGL((delta_chain_kernel<T, N, NW, K == Chain::keep>), grid, th, 0, s, a, a.cmap(), blocks);
  return hipGetLastError();
}

template <Chain K, typename T>
hipError_t chain_n(const DeltaArgs& a, hipStream_t s) {
  switch (a.N) {
    case 32: return chain_go<K, T, 32, 2>(a, s);
    case 64: return chain_go<K, T, 64, 2>(a, s);
    case 128: return chain_go<K, T, 128, K == Chain::bwd ? 2 : 4>(a, s);
  }
  return hipErrorInvalidValue;
}

template <Chain K>
hipError_t chain_type(const DeltaArgs& a, hipStream_t s) {
  if (a.nstates <= 0) return hipSuccess;
  return a.bf16 ? chain_n<K, bf16>(a, s) : chain_n<K, float>(a, s);
}

}  // namespace

hipError_t launch_delta_chain(const DeltaArgs& a, bool keep, hipStream_t s) {
  return keep ? chain_type<Chain::keep>(a, s) : chain_type<Chain::fwd>(a, s);
}
hipError_t launch_delta_chain_bwd(const DeltaArgs& a, hipStream_t s) { return chain_type<Chain::bwd>(a, s); }

}  // namespace ssd

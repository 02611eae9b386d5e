// The gated delta rule, what does not depend on the state: per chunk of 64 tokens and
// head, with G_i the running sum of the chunk's log decays, D_ij = exp(G_i - G_j) for
// j <= i, E_i = exp(G_i),
//   L_ij = beta_i D_ij k_i.k_j  (j < i),   T = (1 + L)^-1,   A_ij = scale D_ij q_i.k_j  (j <= i)
// so that the rows w (ssd_delta_chain.hip) are W = (T beta) (V - E K S^T).  For the backward, T^T
// and, with L = beta B,
//   T' = (1 + B beta)^-1 = 1 - B T beta,
// so that W = beta R, R = T' (V - E K S^T): what beta is multiplied with, also where it is 0.
//
// G is summed in fp64: its differences are what counts, and a chunk's sum may be large
// beside them.  T is inverted in fp32: the four 16x16 blocks of the diagonal by
// substitution, a column per lane, then
//   T_ij = -T_ii sum_{j <= k < i} L_ik T_kj
// by fp32 matrix instructions, whose results are the next product's second operand as they
// lie, and whose first operand L is as k k^T leaves it (which is symmetric).  (Powers of L,
// which would need no substitution, cancel: nearly equal keys give powers with entries of
// thousands for an inverse whose entries are at most one.)
//
// One wave per chunk and group, which walks over the group's heads: k k^T and q k^T are
// theirs in common.  A wave shares nothing with the others of its workgroup and waits for
// none; its LDS holds k's rows first, then each head's T.
//
// 4x8192 tokens, 32 heads in 16 groups of 128 x 128, bf16: 132 to 145 us for 617 MB read and written
// (4.5 TB/s), a bound of memory; for the backward 2x4096 50 us for 230 MB, of which T' takes 4.
// One chunk takes 10 us (7 of 32 tokens at most): loads, products, fp64 sums and the inverse, one
// after another in one wave.
#include "ssd_delta_device.h"

#pragma clang fp contract(on)

namespace ssd {

int device_cu_count();

namespace {

constexpr int C = kDeltaChunk;
constexpr int kPrepWaves = 4;
constexpr int LP = C + 4;                 // pitch of T in LDS

// A log decay below -512 is one of -512: exp is zero either way, and G stays finite, so
// that G_i - G_j of tokens after a reset (-inf) is a number.  A NaN stays one.
__device__ __forceinline__ double log_decay(float g) {
  return (double)__builtin_elementwise_maximum(g, -512.f);
}

// exp(x) to fp32: 2^n times 2 to a power of at most a half, of x log2(e) in fp64.
__device__ __forceinline__ float exp_of(double x) {
  const double t = x * 1.4426950408889634, n = rint(t);
  return ldexpf(__builtin_amdgcn_exp2f((float)(t - n)), (int)n);
}

__device__ __forceinline__ float load_gate(const void* p, bool b16, int64_t i) {
  return b16 ? to_f32(static_cast<const bf16*>(p)[i]) : static_cast<const float*>(p)[i];
}

// Columns 32 cb + 8 (lane / 16) .. + 7 of rows that are a [C][pitch] tile's columns, dealt tile
// u of them: the transposed tile's operand.
__device__ __forceinline__ F8 transposed_opnd(const float* t, int pitch, int u, int cb, int lane) {
  F8 f;
  const float* p = t + (32 * cb + 8 * (lane >> 4)) * pitch + tile_row(u, lane & 15);
#pragma unroll
  for (int e = 0; e < 8; ++e) f.v[e] = p[e * pitch];
  return f;
}

// Four of a lane's eight values of an operand (`half`: the first or the last four) at `slot`.
template <typename T>
__device__ __forceinline__ void put_half(char* p, uint32_t slot, int half, f32x4 f) {
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<f32x4*>(p + half * kPiece + slot) = f;
  } else {
    const uint2 v = {Opnd<bf16>::pack(f[0], f[1]), Opnd<bf16>::pack(f[2], f[3])};
    *reinterpret_cast<uint2*>(p + slot + 8 * half) = v;
  }
}
template <typename T>
__device__ __forceinline__ void put_half_pair(char* p, uint32_t slot, int half, f32x4 f) {
  put_half<T>(p, slot, half, f);
  if constexpr (sizeof(T) == 2) {
    f32x4 lo;
#pragma unroll
    for (int e = 0; e < 4; ++e) lo[e] = f[e] - static_cast<float>(static_cast<bf16>(f[e]));
    put_half<T>(p + kPiece, slot, half, lo);
  }
}

// The first ROWS [N] rows of a chunk to LDS, `pitch` elements apart; zeros past its end.  `then`: what
// is loaded behind them, before they are waited for.
template <typename T, int N, int ROWS, typename F>
__device__ __forceinline__ void stage_rows(T* lds, __amdgpu_buffer_rsrc_t r, uint32_t row, int pitch, int lane, F then) {
  constexpr int PR = N * (int)sizeof(T) / 16, PL = 64 / PR > 0 ? 64 / PR : 1;   // lanes a row, rows a load
  static_assert(PR <= 64, "a row is at most a wave's load");
  uint4 v[ROWS / PL];
#pragma unroll
  for (int i = 0; i < ROWS / PL; ++i) v[i] = buf_load16(r, (i * PL + lane / PR) * row + lane % PR * 16);
  then();
#pragma unroll
  for (int i = 0; i < ROWS / PL; ++i)
    *reinterpret_cast<uint4*>(lds + (i * PL + lane / PR) * pitch + lane % PR * (16 / (int)sizeof(T))) = v[i];
}

// The tile (block of rows i, block of columns j), j <= i, of a lower triangle of 16x16 blocks.
__device__ __forceinline__ constexpr int tri(int i, int j) { return i * (i + 1) / 2 + j; }

// BL: blocks of 16 tokens that a chunk has at most.
template <typename T, int N, bool BWD, int BL>
__global__ __launch_bounds__(64 * kPrepWaves, BWD ? 2 : 1) void delta_prep_kernel(const DeltaArgs a, const ChunkMap cm, int nh) {
  using O = Opnd<T>;
  using X = typename O::X;
  constexpr int V = 16 / (int)sizeof(T), XP = N + V, NK = N / 32, TP = N / 16 * 2;
  constexpr int kOwn = C * XP * (int)sizeof(T) > C * LP * 4 ? C * XP * (int)sizeof(T) : C * LP * 4;
  __shared__ __attribute__((aligned(16))) char own[kPrepWaves][kOwn];
  __shared__ double Gw[kPrepWaves][C];
  __shared__ float bw[kPrepWaves][C];
  const int wave = wave_id();
  // heads h0 .. of `nh` at a time: a group's, or part of one
  const int64_t item = (int64_t)blockIdx.x * kPrepWaves + wave;
  const int per = a.H / nh, j = (int)(item / per), h0 = (int)(item % per) * nh, rep = a.H / a.G, g = h0 / rep;
  if (j >= a.max_chunks) return;
  const ChunkDesc d = cm.desc(j);
  if (d.len <= 0) return;
  const int lane = threadIdx.x & 63, l16 = lane & 15, la = lane >> 4;
  const uint32_t slot = lane * 16;
  T* Ks = reinterpret_cast<T*>(own[wave]);
  float* Ts = reinterpret_cast<float*>(own[wave]);
  double* Gs = Gw[wave];
  float* bs = bw[wave];

  const uint32_t row = (uint32_t)a.G * N * sizeof(T), bytes = (uint32_t)(d.len - 1) * row + N * sizeof(T);
  const int64_t at0 = ((int64_t)d.start * a.G + g) * N, jg = (int64_t)j * a.G + g;
  const __amdgpu_buffer_rsrc_t kr = buf_rsrc(static_cast<const T*>(a.k) + at0, bytes);
  const __amdgpu_buffer_rsrc_t qr = buf_rsrc(static_cast<const T*>(a.q) + at0, bytes);
  auto q_opnd = [&](int i, int kb) {
    return load_opnd(qr, (16 * i + l16) * row + (32 * kb + 8 * la) * (uint32_t)sizeof(T), T{});
  };
  constexpr bool QF = sizeof(T) == 2;       // all of q on its way with k; fp32's would not fit the registers
  X qs[QF ? NK : 1][4];
  stage_rows<T, N, 16 * BL>(Ks, kr, row, XP, lane, [&]() {
    if constexpr (QF) {
#pragma unroll
      for (int kb = 0; kb < NK; ++kb)
#pragma unroll
        for (int i = 0; i < BL; ++i) qs[kb][i] = q_opnd(i, kb);
    }
  });
  // the first head's gates on their way
  const int64_t t0 = (int64_t)(d.start + lane) * a.H + h0;
  const bool in = lane < d.len;
  float gate = in ? load_gate(a.g, a.gate_bf16, t0) : 0.f, step = in ? load_gate(a.beta, a.gate_bf16, t0) : 0.f;
  wave_sync();

  // k_c.k_c' with the lane's row c = 16 i + l16 and columns c' = 16 j + 4 la + r; q_c.k_c' likewise,
  // or backward its transpose: the lane's key c = 16 j + l16 and queries 16 i + 4 la + r
  f32x4 kk[10], qk[10];
#pragma unroll
  for (int i = 0; i < 10; ++i) kk[i] = qk[i] = kZero4;
#pragma unroll
  for (int kb = 0; kb < NK; ++kb) {
    X kf[4];
#pragma unroll
    for (int i = 0; i < BL; ++i) kf[i] = load_opnd(&Ks[(16 * i + l16) * XP + 32 * kb + 8 * la]);
#pragma unroll
    for (int i = 0; i < BL; ++i) {
      const X qf = QF ? qs[QF ? kb : 0][i] : q_opnd(i, kb);
#pragma unroll
      for (int c = 0; c <= i; ++c) {
        kk[tri(i, c)] = mma(kf[c], kf[i], kk[tri(i, c)]);
        if constexpr (BWD) qk[tri(i, c)] = mma(qf, kf[c], qk[tri(i, c)]);
        else qk[tri(i, c)] = mma(kf[c], qf, qk[tri(i, c)]);
      }
    }
  }
  // fp32: k (and q) transposed, once per group; bf16's are read transposed out of LDS later
  if constexpr (sizeof(T) == 4) if (h0 % rep == 0) {
#pragma unroll 4
    for (int x = 0; x < TP; ++x)
      put_piece(static_cast<char*>(a.kt) + (jg * TP + x) * O::PX * kPiece, slot, transposed_opnd(Ks, XP, x % (N / 16), x / (N / 16), lane));
    if constexpr (BWD) {
      wave_sync();
      stage_rows<T, N, C>(Ks, qr, row, XP, lane, []() {});
      wave_sync();
#pragma unroll 4
      for (int x = 0; x < TP; ++x)
        put_piece(static_cast<char*>(a.qt) + (jg * TP + x) * O::PX * kPiece, slot, transposed_opnd(Ks, XP, x % (N / 16), x / (N / 16), lane));
    }
  }

  for (int h = h0; h < h0 + nh; ++h) {
    const int64_t jh = (int64_t)j * a.H + h;
    {
      double s = log_decay(gate);
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const double o = __shfl_up(s, off);
        if (lane >= off) s += o;
      }
      wave_sync();                                // the head before is done with G, beta and T
      Gs[lane] = s;
      bs[lane] = step;
      float* gt = a.gates + jh * kGateFloats;
      const float E = exp_of(s);
      gt[lane] = step;
      gt[C + lane] = E;
      gt[2 * C + lane] = exp_of(__shfl(s, 63) - s);
      gt[3 * C + lane] = step * E;
      reinterpret_cast<double*>(gt + 4 * C)[lane] = s;
      if (h + 1 < h0 + nh && in) {
        gate = load_gate(a.g, a.gate_bf16, t0 + h + 1 - h0);
        step = load_gate(a.beta, a.gate_bf16, t0 + h + 1 - h0);
      }
      wave_sync();
    }
    // L as first operands (backward: B), the diagonal's blocks to LDS; A (or its transpose)
    f32x4 L[10];
    float bi[4];
    if constexpr (BL < 4) {
#pragma unroll
      for (int x = 0; x < 6; ++x) {
        const int2 t = lower_tile(x);
        if (t.x >= BL) put_piece(static_cast<char*>(a.A) + (jh * 6 + x) * O::PX * kPiece, slot, X{});
      }
    }
#pragma unroll
    for (int i = 0; i < BL; ++i) {
      const int c = 16 * i + l16;
      const double Gc = Gs[c];
      const float bc = bi[i] = bs[c];
#pragma unroll
      for (int x = 0; x <= i; ++x) {
        f32x4 f;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int o = 16 * x + 4 * la + r;
          const float D = fexp<T>((float)(Gc - Gs[o]));
          L[tri(i, x)][r] = o < c ? (BWD ? 1.f : bc) * D * kk[tri(i, x)][r] : 0.f;
          if constexpr (!BWD) f[r] = o <= c ? a.scale * D * qk[tri(i, x)][r] : 0.f;
        }
        if (x == i) *reinterpret_cast<f32x4*>(&Ts[(16 * i + l16) * LP + 16 * i + 4 * la]) = BWD ? bc * L[tri(i, i)] : L[tri(i, i)];
        if constexpr (!BWD) {
          // four of the eight values of a lane
          const uint32_t at = 16u * (16 * (2 * (x & 1) + (la >> 1)) + l16);
          char* p = static_cast<char*>(a.A) + (jh * 6 + triangle_index(i, x / 2)) * O::PX * kPiece;
          put_half<T>(p, at, la & 1, f);
          // the block right of the diagonal's in the same 32 columns
          if (x == i && i % 2 == 0) put_half<T>(p, 16u * (16 * (2 + (la >> 1)) + l16), la & 1, kZero4);
        }
      }
    }
    if constexpr (BWD) {
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int c = 16 * x + l16;               // the key
        const double Gc = Gs[c];
        const int t = 2 * (c / 32) + (c / 4 & 1), i16 = c % 32 / 8 * 4 + c % 4;   // its place in the dealt tiles
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (i / 2 < x / 2) continue;            // a tile of zeros that is not kept
          f32x4 f = kZero4;
          if (i >= x) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int o = 16 * i + 4 * la + r;
              f[r] = c <= o ? a.scale * fexp<T>((float)(Gs[o] - Gc)) * qk[tri(i, x)][r] : 0.f;
            }
          }
          const uint32_t at = 16u * (16 * (2 * (i & 1) + (la >> 1)) + i16);
          char* p = static_cast<char*>(a.At) + (jh * 6 + triangle_index(t, i / 2)) * O::PS * kPiece;
          put_half_pair<T>(p, at, la & 1, f);
        }
      }
    }
    wave_sync();
    // the diagonal blocks: column l16 of block la
    {
      float t[16];
      float* B = Ts + 16 * la * LP + 16 * la;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float s0 = i == l16 ? 1.f : 0.f, s1 = 0.f;
#pragma unroll
        for (int m4 = 0; m4 < (i + 3) / 4; ++m4) {
          const f32x4 v = *reinterpret_cast<const f32x4*>(B + i * LP + 4 * m4);
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (4 * m4 + r < i) (r & 1 ? s1 : s0) -= v[r] * t[4 * m4 + r];
        }
        t[i] = s0 + s1;
      }
      wave_sync();
#pragma unroll
      for (int i = 0; i < 16; ++i) B[i * LP + l16] = t[i];
      wave_sync();
    }
    // below it, the blocks next to the diagonal first
    {
      f32x4 blk[10], dia[4];                      // T's blocks as second operands, the diagonal's as first
#pragma unroll
      for (int i = 0; i < BL; ++i) {
        dia[i] = *reinterpret_cast<const f32x4*>(&Ts[(16 * i + l16) * LP + 16 * i + 4 * la]);
#pragma unroll
        for (int r = 0; r < 4; ++r) blk[tri(i, i)][r] = Ts[(16 * i + 4 * la + r) * LP + 16 * i + l16];
      }
#pragma unroll
      for (int n = 1; n < BL; ++n) {
        f32x4 s[3], o[3];
#pragma unroll
        for (int c = 0; c < BL - n; ++c) s[c] = o[c] = kZero4;
#pragma unroll
        for (int k = 0; k < n; ++k)
#pragma unroll
          for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < BL - n; ++c)
              s[c] = __builtin_amdgcn_mfma_f32_16x16x4f32((BWD ? bi[c + n] : 1.f) * L[tri(c + n, c + k)][r], blk[tri(c + k, c)][r], s[c], 0, 0, 0);
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int c = 0; c < BL - n; ++c)
            o[c] = __builtin_amdgcn_mfma_f32_16x16x4f32(dia[c + n][r], s[c][r], o[c], 0, 0, 0);
#pragma unroll
        for (int c = 0; c < BL - n; ++c)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            blk[tri(c + n, c)][r] = -o[c][r];
            Ts[(16 * (c + n) + 4 * la + r) * LP + 16 * c + l16] = -o[c][r];
          }
      }
    }
    wave_sync();
    if constexpr (BWD) {
      // T's transpose; then T' where T was, a column of blocks at a time
#pragma unroll
      for (int x = 0; x < 6; ++x) {
        const int2 t = upper_tile(x);
        const int r = tile_row(t.x, l16), c0 = 32 * t.y + 8 * la;
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = Ts[(c0 + e) * LP + r];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = c0 + e >= r ? f[e] : 0.f;
        put_piece(static_cast<char*>(a.Tt) + (jh * 6 + x) * O::PS * kPiece, slot, O::split(f));
      }
      wave_sync();
#pragma unroll
      for (int c = 0; c < BL; ++c) {
        f32x4 t[4], o[4];                         // T's blocks as second operands
#pragma unroll
        for (int k = c; k < BL; ++k) {
          o[k] = kZero4;
#pragma unroll
          for (int r = 0; r < 4; ++r) t[k][r] = Ts[(16 * k + 4 * la + r) * LP + 16 * c + l16];
        }
#pragma unroll
        for (int k = c; k < BL; ++k)
#pragma unroll
          for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int i = k; i < BL; ++i)
              o[i] = __builtin_amdgcn_mfma_f32_16x16x4f32(L[tri(i, k)][r], t[k][r], o[i], 0, 0, 0);
#pragma unroll
        for (int i = c; i < BL; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            Ts[(16 * i + 4 * la + r) * LP + 16 * c + l16] = i == c && 4 * la + r == l16 ? 1.f : -bi[c] * o[i][r];
        __builtin_amdgcn_sched_barrier(0);
      }
      wave_sync();
    }
    // T, its columns times beta, or T'
#pragma unroll
    for (int x = 0; x < 6; ++x) {
      const int2 t = lower_tile(x);
      const int r = tile_row(t.x, l16), c0 = 32 * t.y + 8 * la;
      float f[8] = {};
      if (32 * (t.x / 2) < 16 * BL) {
        block8(*reinterpret_cast<const f32x4*>(&Ts[r * LP + c0]), *reinterpret_cast<const f32x4*>(&Ts[r * LP + c0 + 4]), f);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = c0 + e <= r ? (BWD ? f[e] : f[e] * bs[c0 + e]) : 0.f;
      }
      put_piece(static_cast<char*>(a.T) + (jh * 6 + x) * O::PS * kPiece, slot, O::split(f));
    }
  }
}

template <typename T, int N>
hipError_t prep_go(const DeltaArgs& a, bool bwd, hipStream_t s) {
  // a head per wave while that does not fill the device's SIMDs once (a forward of 32 heads: 17
  // tokens, 16 groups, 16.9 us, a group per wave 22.4; 4x2000 tokens, 8 groups, 103 and 97)
  const int cus = device_cu_count() > 0 ? device_cu_count() : 256;
  const int nh = (int64_t)a.max_chunks * a.G <= 4 * cus ? 1 : a.H / a.G;
  const int64_t items = (int64_t)a.max_chunks * (a.H / nh);
  const dim3 grid((unsigned)((items + kPrepWaves - 1) / kPrepWaves)), th(64 * kPrepWaves);
  if (bwd) {
    hipLaunchKernelGGL((delta_prep_kernel<T, N, true, 4>), grid, th, 0, s, a, a.cmap(), nh);
    return hipGetLastError();
  }
  // no more than 32 tokens: half of the blocks (a forward of 17 tokens, 32 heads: 13.5 us,
  // with all of them 16.9)
  if constexpr (sizeof(T) == 2) {
    if ((a.cu ? a.total : a.seqlen) <= 32) {
      hipLaunchKernelGGL((delta_prep_kernel<T, N, false, 2>), grid, th, 0, s, a, a.cmap(), nh);
      return hipGetLastError();
    }
  }
  hipLaunchKernelGGL((delta_prep_kernel<T, N, false, 4>), grid, th, 0, s, a, a.cmap(), nh);
  return hipGetLastError();
}

template <typename T>
hipError_t prep_type(const DeltaArgs& a, bool bwd, hipStream_t s) {
  switch (a.N) {
    case 32: return prep_go<T, 32>(a, bwd, s);
    case 64: return prep_go<T, 64>(a, bwd, s);
    case 128: return prep_go<T, 128>(a, bwd, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace

bool delta_dstate_ok(int64_t N) { return N == 32 || N == 64 || N == 128; }

hipError_t launch_delta_prep(const DeltaArgs& a, bool bwd, hipStream_t s) {
  if (a.max_chunks <= 0) return hipSuccess;
  return a.bf16 ? prep_type<bf16>(a, bwd, s) : prep_type<float>(a, bwd, s);
}

}  // namespace ssd

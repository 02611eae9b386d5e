// The gated delta rule, what does not depend on the state: per chunk of 64 tokens and
// head, with G_i the running sum of the chunk's log decays, D_ij = exp(G_i - G_j) for
// j <= i, E_i = exp(G_i),
//   L_ij = beta_i D_ij k_i.k_j  (j < i),   T = (1 + L)^-1,   A_ij = scale D_ij q_i.k_j  (j <= i)
// so that the rows w (ssd_delta_chain.hip) are W = T (beta V - beta E K S^T).
//
// G is summed in fp64: its differences are what counts, and a chunk's sum may be large
// beside them.  T is inverted in fp32: the four 16x16 blocks of the diagonal by
// substitution, one wave each, a column per lane; then, one wave per block column,
//   T_ij = -T_ii sum_{j <= k < i} L_ik T_kj
// by fp32 matrix instructions, whose results are the next product's second operand as they
// lie.  (Powers of L, which would need no substitution, cancel: nearly equal keys give
// powers with entries of thousands for an inverse whose entries are at most one.)
#include "ssd_delta_device.h"

#pragma clang fp contract(on)

namespace ssd {

namespace {

constexpr int C = kDeltaChunk;
constexpr int kPrepThreads = 256;
constexpr int LP = C + 4;                 // pitch of the fp32 matrices in LDS

// A log decay below -512 is one of -512: exp is zero either way, and G stays finite, so
// that G_i - G_j of tokens after a reset (-inf) is a number.  A NaN stays one.
__device__ __forceinline__ double log_decay(float g) {
  return (double)__builtin_elementwise_maximum(g, -512.f);
}

__device__ __forceinline__ float load_gate(const void* p, bool b16, int64_t i) {
  return b16 ? to_f32(static_cast<const bf16*>(p)[i]) : static_cast<const float*>(p)[i];
}

// Columns 32 cb + 8 (lane / 16) .. + 7 of rows that are a [C][pitch] tile's columns, dealt tile
// u of them: the transposed tile's operand.
__device__ __forceinline__ bf16x8 transposed_opnd(const bf16* t, int pitch, int u, int cb, int lane) {
  const int m = lane & 15;
  const bf16* p = t + (32 * cb + 8 * (lane >> 4) + (m >> 2)) * pitch + 32 * (u >> 1) + 8 * (m & 3) + 4 * (u & 1);
  const i16x4 lo = lds_tr16_b64(p), hi = lds_tr16_b64(p + 4 * pitch);
  typedef short i16x8v __attribute__((ext_vector_type(8)));
  const i16x8v v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  return __builtin_bit_cast(bf16x8, v);
}
__device__ __forceinline__ F8 transposed_opnd(const float* t, int pitch, int u, int cb, int lane) {
  F8 f;
  const float* p = t + (32 * cb + 8 * (lane >> 4)) * pitch + tile_row(u, lane & 15);
#pragma unroll
  for (int e = 0; e < 8; ++e) f.v[e] = p[e * pitch];
  return f;
}

template <typename T, int N, bool BWD>
__global__ __launch_bounds__(kPrepThreads) void delta_prep_kernel(const DeltaArgs a, const ChunkMap cm) {
  using O = Opnd<T>;
  constexpr int V = 16 / (int)sizeof(T), XP = N + V, NK = N / 32;
  __shared__ T Ks[C * XP];
  __shared__ T Qs[BWD ? C * XP : 1];
  __shared__ float Ls[C * LP];
  __shared__ float Ts[C * LP];
  __shared__ double Gs[C];
  __shared__ float bs[C];
  const int2 jh = xcd_chunk_head(blockIdx.x, a.H);
  const int j = jh.x, h = jh.y, rep = a.H / a.G, g = h / rep;
  if (j >= a.max_chunks) return;
  const ChunkDesc d = cm.desc(j);
  if (d.len <= 0) return;
  const int tid = threadIdx.x, w = wave_id(), lane = tid & 63, l16 = lane & 15, la = lane >> 4;
  const int64_t jhi = (int64_t)j * a.H + h, jgi = (int64_t)j * a.G + g;

  const int64_t row = (int64_t)a.G * N;
  const T* kp = static_cast<const T*>(a.k) + d.start * row + (int64_t)g * N;
  const T* qp = static_cast<const T*>(a.q) + d.start * row + (int64_t)g * N;
  for (int i = tid; i < C * (N / V); i += kPrepThreads) {
    const int r = i / (N / V), c = i % (N / V) * V;
    *reinterpret_cast<uint4*>(&Ks[r * XP + c]) = load16(kp + r * row + c, r < d.len);
    if constexpr (BWD) *reinterpret_cast<uint4*>(&Qs[r * XP + c]) = load16(qp + r * row + c, r < d.len);
  }
  if (w == 0) {
    double s = 0.0;
    float b = 0.f;
    if (lane < d.len) {
      const int64_t t = (int64_t)(d.start + lane) * a.H + h;
      s = log_decay(load_gate(a.g, a.gate_bf16, t));
      b = load_gate(a.beta, a.gate_bf16, t);
    }
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const double o = __shfl_up(s, off);
      if (lane >= off) s += o;
    }
    Gs[lane] = s;
    bs[lane] = b;
    float* gt = a.gates + jhi * kGateFloats;
    gt[lane] = b;
    const float E = (float)exp(s);
    gt[C + lane] = E;
    gt[3 * C + lane] = b * E;
    gt[2 * C + lane] = (float)exp(__shfl(s, 63) - s);
    reinterpret_cast<double*>(gt + 4 * C)[lane] = s;
  }
  __syncthreads();

  // wave w's 16 rows of L (columns up to its own), and its columns of A or A's transpose
  typename O::X own[NK], oth[NK];
#pragma unroll
  for (int kb = 0; kb < NK; ++kb) {
    const int at = (16 * w + l16) * XP + 32 * kb + 8 * la;
    own[kb] = load_opnd(&Ks[at]);
    if constexpr (BWD) {
      oth[kb] = own[kb];
    } else {
      const bool in = 16 * w + l16 < d.len;
      const T* p = qp + (in ? 16 * w + l16 : 0) * row + 32 * kb + 8 * la;
      oth[kb] = load_opnd(p);                     // rows past the end: never stored
    }
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    f32x4 kk = kZero4, qk = kZero4;
#pragma unroll
    for (int kb = 0; kb < NK; ++kb) {
      const int at = (16 * u + l16) * XP + 32 * kb + 8 * la;
      const typename O::X kf = load_opnd(&Ks[at]);
      if (u <= w) kk = mma(own[kb], kf, kk);
      if constexpr (BWD) qk = mma(load_opnd(&Qs[at]), oth[kb], qk);
      else qk = mma(kf, oth[kb], qk);
    }
    if (u <= w) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = 16 * w + 4 * la + r, c = 16 * u + l16;
        Ls[i * LP + c] = c < i ? bs[i] * fexp<T>((float)(Gs[i] - Gs[c])) * kk[r] : 0.f;
      }
    }
    // A forward: lane's row i = 16 w + l16, columns c = 16 u + 4 la + r; backward its transpose:
    // lane's row c = 16 w + l16, columns i.  Zero above the diagonal.
    const int mine = 16 * w + l16;
    float f[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int c = 16 * u + 4 * la + r, hi = BWD ? c : mine, lo = BWD ? mine : c;
      const bool in = lo <= hi && hi < d.len;
      f[r] = in ? a.scale * fexp<T>((float)(Gs[hi] - Gs[lo])) * qk[r] : 0.f;
    }
    // four of the eight values of a lane: forward rows as they lie, backward dealt
    const int cb = u / 2, t = BWD ? 2 * (mine / 32) + (mine / 4 & 1) : w;
    const int i = BWD ? mine % 32 / 8 * 4 + mine % 4 : l16;
    const uint32_t slot = 16u * (16 * (2 * (u & 1) + (la >> 1)) + i);
    const bool kept = BWD ? cb == 1 || t < 2 : cb == 0 || t >= 2;
    if (kept) {
      if constexpr (sizeof(T) == 4) {
        char* p = static_cast<char*>(BWD ? a.At : a.A) + (jhi * 12 + (BWD ? upper_index(t, cb) : lower_index(t, cb)) * 2) * kPiece;
        *reinterpret_cast<f32x4*>(p + (la & 1) * kPiece + slot) = f32x4{f[0], f[1], f[2], f[3]};
      } else {
        bf16x4 hi, lo;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          hi[r] = static_cast<bf16>(f[r]);
          lo[r] = static_cast<bf16>(f[r] - static_cast<float>(hi[r]));
        }
        if constexpr (BWD) {
          char* p = static_cast<char*>(a.At) + (jhi * 12 + upper_index(t, cb) * 2) * kPiece + slot + 8 * (la & 1);
          *reinterpret_cast<bf16x4*>(p) = hi;
          *reinterpret_cast<bf16x4*>(p + kPiece) = lo;
        } else {
          *reinterpret_cast<bf16x4*>(static_cast<char*>(a.A) + (jhi * 6 + lower_index(t, cb)) * kPiece + slot + 8 * (la & 1)) = hi;
        }
      }
    }
  }
  __syncthreads();

  // the diagonal blocks: lane's column of block w
  {
    float t[16];
    const float* L = &Ls[16 * w * LP + 16 * w];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float v = i == l16 ? 1.f : 0.f;
#pragma unroll
      for (int m = 0; m < i; ++m) v -= L[i * LP + m] * t[m];
      t[i] = v;
    }
    if (lane < 16) {
#pragma unroll
      for (int i = 0; i < 16; ++i) Ts[(16 * w + i) * LP + 16 * w + l16] = t[i];
    }
  }
  __syncthreads();
  // below it: wave w has block column w
  if (w < 3) {
    f32x4 blk[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) blk[k] = kZero4;
#pragma unroll
    for (int r = 0; r < 4; ++r) blk[0][r] = Ts[(16 * w + 4 * la + r) * LP + 16 * w + l16];
#pragma unroll
    for (int n = 1; n < 4; ++n) {                 // block row w + n
      if (w + n < 4) {
        const int i0 = 16 * (w + n) + l16;
        f32x4 s = kZero4, o = kZero4;
#pragma unroll
        for (int k = 0; k < n; ++k) {
          const f32x4 L = *reinterpret_cast<const f32x4*>(&Ls[i0 * LP + 16 * (w + k) + 4 * la]);
#pragma unroll
          for (int r = 0; r < 4; ++r) s = __builtin_amdgcn_mfma_f32_16x16x4f32(L[r], blk[k][r], s, 0, 0, 0);
        }
        const f32x4 t = *reinterpret_cast<const f32x4*>(&Ts[i0 * LP + 16 * (w + n) + 4 * la]);
#pragma unroll
        for (int r = 0; r < 4; ++r) o = __builtin_amdgcn_mfma_f32_16x16x4f32(t[r], s[r], o, 0, 0, 0);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          blk[n][r] = -o[r];
          Ts[(16 * (w + n) + 4 * la + r) * LP + 16 * w + l16] = -o[r];
        }
      }
    }
  }
  __syncthreads();

  // T, and for the backward its transpose
  const uint32_t slot = lane * 16;
  for (int x = w; x < 6; x += 4) {
    const int2 t = lower_tile(x);
    const int r = tile_row(t.x, l16), c0 = 32 * t.y + 8 * la;
    float f[8];
    block8(*reinterpret_cast<const f32x4*>(&Ts[r * LP + c0]), *reinterpret_cast<const f32x4*>(&Ts[r * LP + c0 + 4]), f);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = c0 + e <= r ? f[e] : 0.f;
    put_piece(static_cast<char*>(a.T) + (jhi * 12 + x * 2) * kPiece, slot, O::split(f));
  }
  if constexpr (BWD) {
    for (int x = w; x < 6; x += 4) {
      const int2 t = upper_tile(x);
      const int r = tile_row(t.x, l16), c0 = 32 * t.y + 8 * la;
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = c0 + e >= r ? Ts[(c0 + e) * LP + r] : 0.f;
      put_piece(static_cast<char*>(a.Tt) + (jhi * 12 + x * 2) * kPiece, slot, O::split(f));
    }
  }
  // k (and q) transposed, once per group
  if (h % rep == 0) {
    for (int x = w; x < N / 16 * 2; x += 4) {
      const int u = x % (N / 16), cb = x / (N / 16);
      const int64_t at = (jgi * (N / 16 * 2) + x) * O::PX * kPiece;
      put_piece(static_cast<char*>(a.kt) + at, slot, transposed_opnd(Ks, XP, u, cb, lane));
      if constexpr (BWD) put_piece(static_cast<char*>(a.qt) + at, slot, transposed_opnd(Qs, XP, u, cb, lane));
    }
  }
}

// Rows [0, cu[0]) and [cu[nstates], total) of a tensor, `row` bytes each (a multiple of 2).
__global__ __launch_bounds__(256) void delta_clear_kernel(const int32_t* __restrict__ cu, int nstates,
                                                          int total, void* p, int64_t row) {
  const int64_t n2 = row / 2, lo = min(max(cu[0], 0), total) * n2;
  const int64_t hi = min(max(cu[nstates], 0), total) * n2, end = total * n2;
  unsigned short* o = static_cast<unsigned short*>(p);
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x, step = (int64_t)gridDim.x * 256;
  for (int64_t i = at; i < lo; i += step) o[i] = 0;
  for (int64_t i = max(lo, hi) + at; i < end; i += step) o[i] = 0;
}

template <typename T, int N>
hipError_t prep_go(const DeltaArgs& a, bool bwd, hipStream_t s) {
  const dim3 grid((unsigned)xcd_grid(a.max_chunks, a.H));
  if (bwd) hipLaunchKernelGGL((delta_prep_kernel<T, N, true>), grid, dim3(kPrepThreads), 0, s, a, a.cmap());
  else hipLaunchKernelGGL((delta_prep_kernel<T, N, false>), grid, dim3(kPrepThreads), 0, s, a, a.cmap());
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

hipError_t launch_delta_clear(const DeltaArgs& a, void* p, int64_t row_bytes, hipStream_t s) {
  const int64_t blocks = ((int64_t)a.total * row_bytes / 2 + 256 * 16 - 1) / (256 * 16);
  hipLaunchKernelGGL(delta_clear_kernel, dim3((unsigned)(blocks < 1024 ? blocks : 1024)), dim3(256), 0, s,
                     a.cu, a.nstates, a.total, p, row_bytes);
  return hipGetLastError();
}

}  // namespace ssd

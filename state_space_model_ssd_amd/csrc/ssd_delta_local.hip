// The gated delta rule's backward inside each chunk, from what the two chains left
// (ssd_delta_chain.hip): the state S entering the chunk, the gradient dS of the state
// leaving it, the rows W and their gradient dR before T.  With L, A, D, E as there, and
//   P = tril(dO W^T) * D,   M = -tril(dR W^T, -1) * D   (the gradients of q k^T and, per beta, k k^T)
// the gradients are
//   dq = scale (E dO S + P K)
//   X  = M K - E dR S,    dbeta = dR.v + k.X,    dv = beta dR
//   dk = beta X + scale P^T Q + D_C W dS + (beta M)^T K
// and that of the log decay of token i sums what crosses it:
//   dg_i = sum over pairs c >= i > c' of (P scale q k^T + M beta k k^T)_cc'
//        + sum_{c >= i} (scale E q.(dO S) - beta E k.(dR S))_c  + sum_{c < i} (k.(D_C W dS))_c
//        + E_C <dS, S>
// (pairs by a running sum of column less row sums).  Spelled as k and q times their own
// gradients it would be shorter, but those cancel: a first token's is exactly zero.
//
// One workgroup per chunk and group; it walks over the group's heads, so dq and dk are
// summed over them in registers.  Wave w has tokens 16 w .. as the second operand's columns
// throughout: its results are columns of its own tokens, dot products with q and k are sums
// over a lane's rows, and P and M go into the next product as they lie.  P^T and M^T of its
// tokens are products of their own, not exchanged.  The axis of values is walked in slabs
// of 32, whose W, dR, S and dS lie in LDS with the values as rows (read transposed).
#include "ssd_delta_device.h"

#pragma clang fp contract(on)

namespace ssd {

namespace {

constexpr int C = kDeltaChunk;
constexpr int kLocalThreads = 256;
constexpr int kSlab = 32;

// [kSlab][COLS] tiles in LDS and the operands that contract their rows.
template <typename T, int COLS> struct Tile;
template <int COLS> struct Tile<bf16, COLS> {
  static constexpr int size = kSlab * COLS;
  __device__ __forceinline__ static bf16* piece(bf16* t, int r, int c) { return t + tile_at<COLS>(r, c); }
  __device__ __forceinline__ static bf16x8 at(const bf16* t, int r, int c) {
    const bf16* p = t + tile_at<COLS>(r, c);
    const i16x4 lo = lds_tr16_b64(p), hi = lds_tr16_b64(p + 4 * COLS);
    typedef short i16x8v __attribute__((ext_vector_type(8)));
    const i16x8v v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_bit_cast(bf16x8, v);
  }
  // columns of dealt tile u; of 16 neighbouring columns from c0
  __device__ __forceinline__ static bf16x8 dealt(const bf16* t, int u, int lane) {
    const int m = lane & 15;
    return at(t, 8 * (lane >> 4) + (m >> 2), 32 * (u >> 1) + 8 * (m & 3) + 4 * (u & 1));
  }
  __device__ __forceinline__ static bf16x8 plain(const bf16* t, int c0, int lane) {
    const int m = lane & 15;
    return at(t, 8 * (lane >> 4) + (m >> 2), c0 + 4 * (m & 3));
  }
};
template <int COLS> struct Tile<float, COLS> {
  static constexpr int pitch = COLS + 4, size = kSlab * pitch;
  __device__ __forceinline__ static float* piece(float* t, int r, int c) { return t + r * pitch + c; }
  __device__ __forceinline__ static F8 at(const float* t, int lane, int c) {
    F8 f;
#pragma unroll
    for (int e = 0; e < 8; ++e) f.v[e] = t[(8 * (lane >> 4) + e) * pitch + c];
    return f;
  }
  __device__ __forceinline__ static F8 dealt(const float* t, int u, int lane) {
    return at(t, lane, tile_row(u, lane & 15));
  }
  __device__ __forceinline__ static F8 plain(const float* t, int c0, int lane) {
    return at(t, lane, c0 + (lane & 15));
  }
};

// Copies `rows` rows (zeros up to kSlab) that lie one after another.
template <typename T, int COLS>
__device__ __forceinline__ void fill(T* t, const T* src, int rows) {
  constexpr int V = 16 / (int)sizeof(T), PR = COLS / V;
  for (int i = threadIdx.x; i < kSlab * PR; i += kLocalThreads) {
    const int r = i / PR, c = i % PR * V;
    *reinterpret_cast<uint4*>(Tile<T, COLS>::piece(t, r, c)) = load16(src + r * COLS + c, r < rows);
  }
}
__device__ __forceinline__ float dot16(uint4 x, uint4 y, bf16) {
  const bf16x8 a = __builtin_bit_cast(bf16x8, x), b = __builtin_bit_cast(bf16x8, y);
  float s = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) s += static_cast<float>(a[e]) * static_cast<float>(b[e]);
  return s;
}
__device__ __forceinline__ float dot16(uint4 x, uint4 y, float) {
  const f32x4 a = __builtin_bit_cast(f32x4, x), b = __builtin_bit_cast(f32x4, y);
  return a[0] * b[0] + a[1] * b[1] + a[2] * b[2] + a[3] * b[3];
}
// Two such copies, and the sum of their values' products.
template <typename T, int COLS>
__device__ __forceinline__ float fill_dot(T* t0, T* t1, const T* s0, const T* s1, int rows) {
  constexpr int V = 16 / (int)sizeof(T), PR = COLS / V;
  float s = 0.f;
  for (int i = threadIdx.x; i < kSlab * PR; i += kLocalThreads) {
    const int r = i / PR, c = i % PR * V;
    const uint4 x = load16(s0 + r * COLS + c, r < rows), y = load16(s1 + r * COLS + c, r < rows);
    s += dot16(x, y, T{});
    *reinterpret_cast<uint4*>(Tile<T, COLS>::piece(t0, r, c)) = x;
    *reinterpret_cast<uint4*>(Tile<T, COLS>::piece(t1, r, c)) = y;
  }
  return s;
}

__device__ __forceinline__ void store_gate(void* p, bool b16, int64_t i, float v) {
  if (b16) static_cast<bf16*>(p)[i] = static_cast<bf16>(v);
  else static_cast<float*>(p)[i] = v;
}

template <typename T, int N>
__global__ __launch_bounds__(kLocalThreads) void delta_local_bwd_kernel(const DeltaArgs a, const ChunkMap cm) {
  using O = Opnd<T>;
  using X = typename O::X;
  using TC = Tile<T, C>;
  using TN = Tile<T, N>;
  constexpr int NK = N / 32, NT = N / 16;
  __shared__ __attribute__((aligned(16))) T Ws[TC::size], Rs[TC::size], Ss[TN::size], Ds[TN::size];
  __shared__ double Gs[C];
  __shared__ float bs[C], left[C], mid[C], sdots[kLocalThreads / 64];
  const int2 jg = xcd_chunk_head(blockIdx.x, a.G);
  const int j = jg.x, g = jg.y, rep = a.H / a.G;
  if (j >= a.max_chunks) return;
  const ChunkDesc d = cm.desc(j);
  if (d.len <= 0) return;
  const int w = wave_id(), lane = threadIdx.x & 63, l16 = lane & 15, la = lane >> 4;
  const int c = 16 * w + l16;                     // the lane's token
  const uint32_t qrow = (uint32_t)a.G * N * sizeof(T), vrow = (uint32_t)a.H * a.P * sizeof(T);
  const int64_t qo = ((int64_t)d.start * a.G + g) * N;
  const uint32_t qbytes = (uint32_t)(d.len - 1) * qrow + N * sizeof(T);
  const __amdgpu_buffer_rsrc_t qr = buf_rsrc(static_cast<const T*>(a.q) + qo, qbytes);
  const __amdgpu_buffer_rsrc_t kr = buf_rsrc(static_cast<const T*>(a.k) + qo, qbytes);
  const int64_t tr = ((int64_t)j * a.G + g) * (NT * 2) * O::PX * kPiece;
  const char* kt = static_cast<const char*>(a.kt) + tr;
  const char* qt = static_cast<const char*>(a.qt) + tr;

  X ko[NK], qn[NK];                               // the token's k and q
#pragma unroll
  for (int kb = 0; kb < NK; ++kb) {
    const uint32_t off = c * qrow + (32 * kb + 8 * la) * (uint32_t)sizeof(T);
    ko[kb] = load_opnd(kr, off, T{});
    qn[kb] = load_opnd(qr, off, T{});
  }
  f32x4 dq[NT], dk[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) dq[i] = dk[i] = kZero4;

  for (int h = g * rep; h < (g + 1) * rep; ++h) {
    const int64_t jh = (int64_t)j * a.H + h;
    const float* gt = a.gates + jh * kGateFloats;
    if (threadIdx.x < C) {
      Gs[threadIdx.x] = reinterpret_cast<const double*>(gt + 3 * C)[threadIdx.x];
      bs[threadIdx.x] = gt[threadIdx.x];
    }
    const float be = gt[c], E = gt[C + c], Dc = gt[2 * C + c], EC = gt[2 * C - 1];
    const int64_t vo = ((int64_t)d.start * a.H + h) * a.P;
    const uint32_t vbytes = (uint32_t)(d.len - 1) * vrow + a.P * (uint32_t)sizeof(T);
    const __amdgpu_buffer_rsrc_t vr = buf_rsrc(static_cast<const T*>(a.v) + vo, vbytes);
    const __amdgpu_buffer_rsrc_t dor = buf_rsrc(static_cast<const T*>(a.dout) + vo, vbytes);

    f32x4 Pr[4], Lr[4], Pc[4], Lc[4];             // [c'][c]: c the query or k's reader (r), or the key (c)
#pragma unroll
    for (int u = 0; u < 4; ++u) Pr[u] = Lr[u] = Pc[u] = Lc[u] = kZero4;
    f32x4 yq[NT], yx[NT], yd[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) yq[i] = yx[i] = yd[i] = kZero4;
    float sdot = 0.f, rv = 0.f;
    for (int p0 = 0; p0 < a.P; p0 += kSlab) {
      const int rows = min(kSlab, a.P - p0);
      const int64_t at = jh * a.P + p0;
      __syncthreads();                            // the slab before is read
      fill<T, C>(Ws, static_cast<const T*>(a.Wt) + at * C, rows);
      fill<T, C>(Rs, static_cast<const T*>(a.dRt) + at * C, rows);
      sdot += fill_dot<T, N>(Ss, Ds, static_cast<const T*>(a.S0) + at * N, static_cast<const T*>(a.dS) + at * N, rows);
      const bool in = 8 * la < rows;              // values past P: none, whatever lies there
      const uint32_t vc = (uint32_t)(p0 + 8 * la) * sizeof(T);
      const X od = load_opnd(dor, in ? c * vrow + vc : 0xfffffff0u - 16u, T{});
      const X vv = load_opnd(vr, in ? c * vrow + vc : 0xfffffff0u - 16u, T{});
      X da[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        da[u] = load_opnd(dor, in ? tile_row(u, l16) * vrow + vc : 0xfffffff0u - 16u, T{});
      __syncthreads();
      const X wo = TC::plain(Ws, 16 * w, lane), ro = TC::plain(Rs, 16 * w, lane);
      {
        float r8[8], v8[8];
        O::get(ro, r8);
        O::get(vv, v8);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          rv += r8[e] * v8[e];
          r8[e] *= be;
        }
        if (in && c < d.len) store_opnd(static_cast<T*>(a.dv) + vo + (int64_t)c * a.H * a.P + p0 + 8 * la, O::round(r8));
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (u < 2 || w >= 2) {                    // c' in the token's 32-block or before
          const X f = TC::dealt(Ws, u, lane);
          Pr[u] = mma(f, od, Pr[u]);
          Lr[u] = mma(f, ro, Lr[u]);
        }
        if (u >= 2 || w < 2) {                    // or after
          Pc[u] = mma(da[u], wo, Pc[u]);
          Lc[u] = mma(TC::dealt(Rs, u, lane), wo, Lc[u]);
        }
      }
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const X s = TN::dealt(Ss, i, lane);
        yq[i] = mma(s, od, yq[i]);
        yx[i] = mma(s, ro, yx[i]);
        yd[i] = mma(TN::dealt(Ds, i, lane), wo, yd[i]);
      }
    }
    // the row sums that need the states' products alone
    float ql = 0.f, kx = 0.f, kd = 0.f;
#pragma unroll
    for (int kb = 0; kb < NK; ++kb) {
      float k8[8], q8[8];
      O::get(ko[kb], k8);
      O::get(qn[kb], q8);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int i = 2 * kb + e / 4, r = e % 4;
        ql += q8[e] * yq[i][r];
        kx += k8[e] * yx[i][r];
        kd += k8[e] * yd[i][r];
      }
    }
    // P and M, their transposes, and the pairs' sums
    X pr[2], mr[2], pc[2], mc[2];
    float pairs = 0.f;
#pragma unroll
    for (int cb = 0; cb < 2; ++cb) {
      float p8[8], m8[8], pt[8], mt[8];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int u = 2 * cb + t;
        f32x4 qkr = kZero4, qkc = kZero4, kk = kZero4;
#pragma unroll
        for (int kb = 0; kb < NK; ++kb) {
          const uint32_t off = tile_row(u, l16) * qrow + (32 * kb + 8 * la) * (uint32_t)sizeof(T);
          const X kf = load_opnd(kr, off, T{});
          kk = mma(kf, ko[kb], kk);
          if (u < 2 || w >= 2) qkr = mma(kf, qn[kb], qkr);
          if (u >= 2 || w < 2) qkc = mma(load_opnd(qr, off, T{}), ko[kb], qkc);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int e = 4 * t + r, o = 32 * cb + 8 * la + e;
          const float D = fexp<T>((float)(o > c ? Gs[o] - Gs[c] : Gs[c] - Gs[o]));
          const float bo = bs[o];
          p8[e] = o <= c ? Pr[u][r] * D : 0.f;
          m8[e] = o < c ? -Lr[u][r] * D : 0.f;
          pt[e] = o >= c ? Pc[u][r] * D * a.scale : 0.f;
          mt[e] = o > c ? -Lc[u][r] * D * bo : 0.f;
          // a pair's term is the same number as row and as column: what crosses no token cancels
          const float row = (Pr[u][r] * D * a.scale) * qkr[r] + (-Lr[u][r] * D * be) * kk[r];
          const float col = pt[e] * qkc[r] + mt[e] * kk[r];
          pairs += o > c ? col : o < c ? -row : 0.f;
        }
      }
      pr[cb] = O::round(p8);
      mr[cb] = O::round(m8);
      pc[cb] = O::round(pt);
      mc[cb] = O::round(mt);
    }
    float kX = 0.f;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      f32x4 q = yq[i] * E, x = yx[i] * -E, k = yd[i] * Dc;
#pragma unroll
      for (int cb = 0; cb < 2; ++cb) {
        const int at = (cb * NT + i) * O::PX * kPiece;
        const X kf = piece_x(kt + at, lane * 16, T{}), qf = piece_x(qt + at, lane * 16, T{});
        q = mma(kf, pr[cb], q);
        x = mma(kf, mr[cb], x);
        k = mma(qf, pc[cb], k);
        k = mma(kf, mc[cb], k);
      }
      float k8[8];
      O::get(ko[i / 2], k8);
#pragma unroll
      for (int r = 0; r < 4; ++r) kX += k8[4 * (i % 2) + r] * x[r];
      dq[i] += q * a.scale;
      dk[i] += k + x * be;
    }
    const float db = column_sum(rv + kX);
    const float lf = column_sum(a.scale * E * ql - be * E * kx), md = column_sum(Dc * kd + pairs);
    for (int off = 1; off < 64; off <<= 1) sdot += __shfl_xor(sdot, off);
    if (la == 0) {
      left[c] = lf;
      mid[c] = md;
      if (c < d.len) store_gate(a.dbeta, a.gate_bf16, (int64_t)(d.start + c) * a.H + h, db);
    }
    if (lane == 0) sdots[w] = sdot;
    __syncthreads();
    if (w == 0) {
      // sums over the tokens from this one on, and over those before it
      double s = left[63 - lane], b = mid[lane];
      const double own = b;
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const double x = __shfl_up(s, off), y = __shfl_up(b, off);
        if (lane >= off) {
          s += x;
          b += y;
        }
      }
      s = __shfl(s, 63 - lane);
      const double sd = (double)EC * ((double)sdots[0] + sdots[1] + sdots[2] + sdots[3]);
      if (lane < d.len)
        store_gate(a.dg, a.gate_bf16, (int64_t)(d.start + lane) * a.H + h, (float)(s + (b - own) + sd));
    }
  }
  if (c < d.len) {
#pragma unroll
    for (int kb = 0; kb < NK; ++kb) {
      float f[8];
      const int64_t at = qo + (int64_t)c * a.G * N + 32 * kb + 8 * la;
      block8(dq[2 * kb], dq[2 * kb + 1], f);
      store_opnd(static_cast<T*>(a.dq) + at, O::round(f));
      block8(dk[2 * kb], dk[2 * kb + 1], f);
      store_opnd(static_cast<T*>(a.dk) + at, O::round(f));
    }
  }
}

template <typename T>
hipError_t local_type(const DeltaArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)xcd_grid(a.max_chunks, a.G)), th(kLocalThreads);
  switch (a.N) {
    case 32: hipLaunchKernelGGL((delta_local_bwd_kernel<T, 32>), grid, th, 0, s, a, a.cmap()); break;
    case 64: hipLaunchKernelGGL((delta_local_bwd_kernel<T, 64>), grid, th, 0, s, a, a.cmap()); break;
    case 128: hipLaunchKernelGGL((delta_local_bwd_kernel<T, 128>), grid, th, 0, s, a, a.cmap()); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_local_bwd(const DeltaArgs& a, hipStream_t s) {
  if (a.max_chunks <= 0) return hipSuccess;
  return a.bf16 ? local_type<bf16>(a, s) : local_type<float>(a, s);
}

}  // namespace ssd

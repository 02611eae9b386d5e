// The norm of queries and keys in each head, and the rotation by the token's position, in
// one pass.  For every row (token, head) of D channels, with r = 1 / sqrt(mean(x^2) + eps)
// or 1 / sqrt(sum(x^2) + eps),
//   n = x r w,   (a, b) -> (a cos t - b sin t, b cos t + a sin t),  t = pos freq[i]
// for the R pairs of channels (i, i + R) or (2i, 2i + 1); channels from 2R on stay.
//
// What bounds it: each element read and written once (backward: two reads, one write).  A
// row lies over LPR lanes, 16 bytes each; a workgroup takes all heads of a few tokens, so
// a token's cosines and sines are made once and lie in LDS for all of them.  The other
// channel of a pair comes from the row in LDS, any R, D and pairing alike; a wave reads
// only rows that it wrote, so no barrier is needed there.
//
// Angles are taken by turns in fp64: pos freq / 2 pi less the nearest whole number, off by
// 2^-52 of the turns and then, in fp32, by 2^-26 of a turn at most.
#include "ssd_delta.h"
#include "ssd_layer_device.h"
#include "ssd_rowsum.h"

#pragma clang fp contract(on)

namespace ssd {

int device_cu_count();

namespace {

constexpr int kQnThreads = 256;
constexpr int kQnMaxTok = 4;            // most tokens a workgroup takes at a time
constexpr int kQnMaxParts = 1024;       // partial rows the workspace holds
constexpr int kQnSegment = 32;

__device__ __forceinline__ float2 turn(int pos, float freq) {
  const double t = (double)pos * (double)freq * 0.15915494309189533577;
  float2 cs;
  sincospif((float)(2.0 * (t - rint(t))), &cs.y, &cs.x);
  return cs;
}

// Where a row's elements lie over its lanes.
template <int V> struct RowLane {
  int ln, n, lpr, rows;                 // lane within the row, its first element; rows per pass
  bool mine[V];                         // not the lane before's, nor past the row's end
  __device__ __forceinline__ RowLane(int D, int lanes) : lpr(lanes) {
    ln = threadIdx.x & (lpr - 1);
    rows = kQnThreads / lpr;
    n = min(ln * V, D - V);
#pragma unroll
    for (int e = 0; e < V; ++e) mine[e] = n + e >= ln * V && ln * V < D;
  }
};

// One token's rows of q and k: row i of the workgroup's tokens.
struct RowAt {
  int which, head, tok;
  __device__ __forceinline__ RowAt(const QkNormArgs& a, int i) {
    const int all = a.heads[0] + a.heads[1];
    tok = i / all;
    head = i - tok * all;
    which = head >= a.heads[0];
    if (which) head -= a.heads[0];
  }
};

// f turned (or, BACK, turned back) by the token's angles; `row`: the row's D values in LDS.
template <int V, bool BACK>
__device__ __forceinline__ void rotate(const QkNormArgs& a, float* row, const float2* cs, int n, float (&f)[V]) {
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int e = 0; e < V; ++e) row[n + e] = f[e];
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const int c = n + e;
    const bool first = a.interleaved ? !(c & 1) : c < a.R;
    const int pair = a.interleaved ? c >> 1 : first ? c : c - a.R;
    if (c < 2 * a.R) {
      const float2 t = cs[pair];
      const float o = row[a.interleaved ? c ^ 1 : first ? c + a.R : c - a.R];
      const float s = first == BACK ? t.y : -t.y;
      f[e] = f[e] * t.x + o * s;
    }
  }
  __builtin_amdgcn_wave_barrier();
}

// The angles of `ntok` tokens from `tok`.
__device__ __forceinline__ void angles(const QkNormArgs& a, float2* cs, int64_t tok, int ntok) {
  for (int i = threadIdx.x; i < ntok * a.R; i += kQnThreads) {
    const int t = i / a.R;
    cs[i] = turn(a.pos[tok + t], a.freq[i - t * a.R]);
  }
}

template <typename T, int V, int RU>
__global__ __launch_bounds__(kQnThreads) void qk_norm_fwd_kernel(const QkNormArgs a, int lpr, int per) {
  extern __shared__ float lds[];        // angles of `per` tokens, then a pass's rows
  float2* cs = reinterpret_cast<float2*>(lds);
  const RowLane<V> L(a.D, lpr);
  const int64_t tok = (int64_t)blockIdx.x * per;
  const int ntok = (int)min((int64_t)per, a.tokens - tok);
  float* row = lds + 2 * per * a.R + threadIdx.x / lpr * a.D;
  if (a.R) {
    angles(a, cs, tok, ntok);
    __syncthreads();
  }
  float wt[2][V];
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int e = 0; e < V; ++e) wt[s][e] = a.w[s] ? a.w[s][L.n + e] : 1.f;
  const int all = ntok * (a.heads[0] + a.heads[1]);
  const float inv = a.l2 ? 1.f : 1.f / (float)a.D;
  for (int i0 = threadIdx.x / lpr; i0 < all; i0 += RU * L.rows) {
    Vec<T, V> x[RU];
#pragma unroll
    for (int u = 0; u < RU; ++u) {
      const RowAt at(a, min(i0 + u * L.rows, all - 1));
      x[u].load(static_cast<const T*>(a.x[at.which]) + (tok + at.tok) * a.stride[at.which] +
                (int64_t)at.head * a.D + L.n);
    }
#pragma unroll
    for (int u = 0; u < RU; ++u) {
      const int i = i0 + u * L.rows;
      const RowAt at(a, min(i, all - 1));
      float f[V], s = 0.f;
      x[u].get(f);
#pragma unroll
      for (int e = 0; e < V; ++e) s += L.mine[e] ? f[e] * f[e] : 0.f;
      const float r = rsqrtf(run_sum_dpp(s, lpr) * inv + a.eps);
#pragma unroll
      for (int e = 0; e < V; ++e) f[e] = f[e] * r * (at.which ? wt[1][e] : wt[0][e]);
      if (a.R) rotate<V, false>(a, row, cs + at.tok * a.R, L.n, f);
      x[u].set(f);
      if (i < all && L.ln * V < a.D)
        x[u].store(static_cast<T*>(a.out[at.which]) +
                   ((tok + at.tok) * a.heads[at.which] + at.head) * a.D + L.n);
    }
  }
}

// With d = dout turned back, n = x r and dn = d w:
//   dx = r (dn - n mean or sum(dn n)),   dw = sum over rows of d n
// The sums over rows: a lane's own rows (kQnSegment of the workgroup's token tiles in one
// register, then those sums in another, so that long inputs lose no more than short ones),
// then the workgroup's, then the partial rows' columns (q's, then k's).
template <typename T, int V>
__global__ __launch_bounds__(kQnThreads) void qk_norm_bwd_kernel(const QkNormArgs a, int lpr, int per) {
  extern __shared__ float lds[];
  float2* cs = reinterpret_cast<float2*>(lds);
  const RowLane<V> L(a.D, lpr);
  float* row = lds + 2 * per * a.R + threadIdx.x / lpr * a.D;
  float wt[2][V], dw[2][V], seg[2][V];
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int e = 0; e < V; ++e) {
      wt[s][e] = a.w[s] ? a.w[s][L.n + e] : 1.f;
      dw[s][e] = seg[s][e] = 0.f;
    }
  int until = kQnSegment;
  const float inv = a.l2 ? 1.f : 1.f / (float)a.D;
  const int heads = a.heads[0] + a.heads[1];
  for (int64_t tok = (int64_t)blockIdx.x * per; tok < a.tokens; tok += (int64_t)gridDim.x * per) {
    const int ntok = (int)min((int64_t)per, a.tokens - tok);
    if (a.R) {
      __syncthreads();
      angles(a, cs, tok, ntok);
      __syncthreads();
    }
    const int all = ntok * heads;
    for (int i = threadIdx.x / lpr; i < all; i += L.rows) {
      const RowAt at(a, i);
      Vec<T, V> xq, dq;
      xq.load(static_cast<const T*>(a.x[at.which]) + (tok + at.tok) * a.stride[at.which] +
              (int64_t)at.head * a.D + L.n);
      dq.load(static_cast<const T*>(a.dout[at.which]) +
              ((tok + at.tok) * a.heads[at.which] + at.head) * a.D + L.n);
      float x[V], d[V], s = 0.f;
      xq.get(x);
      dq.get(d);
      if (a.R) rotate<V, true>(a, row, cs + at.tok * a.R, L.n, d);
#pragma unroll
      for (int e = 0; e < V; ++e) s += L.mine[e] ? x[e] * x[e] : 0.f;
      const float r = rsqrtf(run_sum_dpp(s, lpr) * inv + a.eps);
      float m = 0.f;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        x[e] *= r;
        const float t = L.mine[e] ? d[e] * x[e] : 0.f;
        if (at.which) seg[1][e] += t;
        else seg[0][e] += t;
        d[e] *= at.which ? wt[1][e] : wt[0][e];
        m += L.mine[e] ? d[e] * x[e] : 0.f;
      }
      m = run_sum_dpp(m, lpr) * inv;
#pragma unroll
      for (int e = 0; e < V; ++e) d[e] = r * (d[e] - x[e] * m);
      dq.set(d);
      if (L.ln * V < a.D)
        dq.store(static_cast<T*>(a.dx[at.which]) + (tok + at.tok) * a.dstride[at.which] +
                 (int64_t)at.head * a.D + L.n);
    }
    if (--until == 0 || tok + (int64_t)gridDim.x * per >= a.tokens) {
      until = kQnSegment;
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int e = 0; e < V; ++e) {
          dw[s][e] += seg[s][e];
          seg[s][e] = 0.f;
        }
    }
  }
  if (!a.part) return;
  // the workgroup's sums of each channel, one row group after another
  const int cols = (int)part_cols(a.D);
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    __syncthreads();
    if (L.ln * V < a.D) {
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (L.mine[e]) lds[threadIdx.x / lpr * a.D + L.n + e] = dw[s][e];
    }
    __syncthreads();
    for (int c = threadIdx.x; c < cols; c += kQnThreads) {
      float v = 0.f;
      if (c < a.D)
        for (int g = 0; g < L.rows; ++g) v += lds[g * a.D + c];
      *part_at(a.part, blockIdx.x, gridDim.x, s * cols + c) = v;
    }
  }
}

struct QkNormOut {
  float* w[2];
  int D, cp;
  __device__ __forceinline__ void put(int col, float v) const {
    const int s = col >= cp, c = col - s * cp;
    if (c < D && w[s]) w[s][c] = v;
  }
};

int row_lanes(int D, int V) {
  int l = 1;
  while (l * V < D) l *= 2;
  return l;
}

template <typename T, int V>
hipError_t qn_go(const QkNormArgs& a, bool bwd, hipStream_t s) {
  const int lpr = row_lanes(a.D, V);
  // all tokens' workgroups at once where there are few, else four tokens share their angles'
  // barrier
  const int cus = device_cu_count() > 0 ? device_cu_count() : 256;
  const int per = a.tokens <= 4 * (int64_t)cus ? 1 : kQnMaxTok;
  const size_t rows = (size_t)kQnThreads / lpr * a.D * 4;
  const size_t lds = (size_t)per * a.R * 8 + (a.R || (bwd && a.part) ? rows : 0);
  const int64_t tiles = (a.tokens + per - 1) / per;
  if (!bwd) {
    if (tiles == 0) return hipSuccess;
    hipLaunchKernelGGL((qk_norm_fwd_kernel<T, V, 2>), dim3((unsigned)tiles), dim3(kQnThreads), lds, s, a, lpr, per);
    return hipGetLastError();
  }
  const int64_t most = a.part ? kQnMaxParts : (int64_t)1 << 24;
  const int grid = (int)(tiles < most ? tiles : most);
  if (grid > 0) hipLaunchKernelGGL((qk_norm_bwd_kernel<T, V>), dim3(grid), dim3(kQnThreads), lds, s, a, lpr, per);
  if (!a.part) return hipGetLastError();
  QkNormOut out;
  out.w[0] = a.dw[0];
  out.w[1] = a.dw[1];
  out.D = a.D;
  out.cp = (int)part_cols(a.D);
  return colsum(a.part, grid, 2 * part_cols(a.D), out, s);
}

hipError_t qn_type(const QkNormArgs& a, bool bwd, hipStream_t s) {
  if (a.bf16) return a.D >= 8 ? qn_go<bf16, 8>(a, bwd, s) : qn_go<bf16, 1>(a, bwd, s);
  return a.D >= 4 ? qn_go<float, 4>(a, bwd, s) : qn_go<float, 1>(a, bwd, s);
}

}  // namespace

int64_t qk_norm_bwd_floats(int64_t tokens, int64_t D) {
  return (tokens < kQnMaxParts ? tokens : kQnMaxParts) * 2 * part_cols(D);
}

hipError_t launch_qk_norm_fwd(const QkNormArgs& a, hipStream_t s) { return qn_type(a, false, s); }
hipError_t launch_qk_norm_bwd(const QkNormArgs& a, hipStream_t s) { return qn_type(a, true, s); }

}  // namespace ssd

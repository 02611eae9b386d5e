// The norm of queries and keys in each head, and the rotation by the token's position, in
// one pass.  For every row (token, head) of D channels, with r = 1 / sqrt(mean(x^2) + eps)
// or 1 / sqrt(sum(x^2) + eps),
//   n = x r w,   (a, b) -> (a cos t - b sin t, b cos t + a sin t),  t = pos freq[i]
// for the R pairs of channels (i, i + R) or (2i, 2i + 1); channels from 2R on stay.
//
// What bounds it: each element read and written once (backward: two reads, one write).  A
// row lies over LPR lanes, 16 bytes each.  A workgroup takes a few tokens, whose cosines and
// sines are made once, into LDS; a lane keeps its channels' in registers for all heads of its
// token.  The other channel of a pair is the lane's own (neighbours), or comes by a second load
// of the row from the cache (halves, where they are whole vectors); where rows or halves are no
// whole vectors it comes from the row in LDS.  32768 tokens of 16 + 16 heads of 128, bf16, forward
// without rotation: 99 us, 5.4 TB/s; 8192 of 32 + 8, backward with it: 47 us, 5.4 TB/s, and 4 for
// the weights' sums (through LDS for every pair, and a row's heads and tokens found by division: 79).
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
constexpr int kQnTok = 4;               // tokens a workgroup takes at a time where there are many
constexpr int kQnMaxParts = 1024;       // partial rows the workspace holds
constexpr int kQnSegment = 32;
constexpr int64_t kQnGridX = 1 << 18;

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

// V weights from element n on, ones without weights: a resource of no bytes and a select, for
// behind a branch they would be waited for at its end.
template <int V>
__device__ __forceinline__ void weights(const QkNormArgs& a, int k, int n, float (&w)[V]) {
  const __amdgpu_buffer_rsrc_t r = buf_rsrc(a.w[k], a.w[k] ? a.D * 4 : 0);
  if constexpr (V == 1) {
    w[0] = buf_load4(r, n * 4);
  } else {
#pragma unroll
    for (int e = 0; e < V; e += 4) {
      const f32x4 v = __builtin_bit_cast(f32x4, buf_load16(r, (n + e) * 4));
#pragma unroll
      for (int i = 0; i < 4; ++i) w[e + i] = v[i];
    }
  }
#pragma unroll
  for (int e = 0; e < V; ++e) w[e] = a.w[k] ? w[e] : 1.f;
}

// From a lane's first element to the other of its pair (halves of whole vectors); 0 from 2 R on.
__device__ __forceinline__ int other(const QkNormArgs& a, int n) { return n < a.R ? a.R : n < 2 * a.R ? -a.R : 0; }

// How the other channel of a pair is had: there is none; by a load (halves of whole vectors);
// in the lane (neighbours, rows of whole vectors); through LDS.
enum class Pairs { none, load, lane, lds };

// A lane's channels of one token: the cosine, and the sine with its sign, by which the other
// channel of the pair counts; (1, 0) from 2 R on.  BACK: turned back.
template <int V, Pairs M, bool BACK> struct Turns {
  float c[V], s[V];
  __device__ __forceinline__ void get(const QkNormArgs& a, const float2* cs, int n) {
    if constexpr (M == Pairs::none) return;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const int i = n + e;
      const bool first = a.interleaved ? !(i & 1) : i < a.R;
      const float2 t = cs[min(a.interleaved ? i >> 1 : first ? i : i - a.R, a.R - 1)];
      c[e] = i < 2 * a.R ? t.x : 1.f;
      s[e] = i < 2 * a.R ? first == BACK ? t.y : -t.y : 0.f;
    }
  }
  // f turned; `o`: the pairs' other values (load); `row`: the row's D values in LDS (lds)
  __device__ __forceinline__ void turn(const QkNormArgs& a, const float (&o)[V], float* row, int n, float (&f)[V]) const {
    if constexpr (M == Pairs::load) {
#pragma unroll
      for (int e = 0; e < V; ++e) f[e] = f[e] * c[e] + o[e] * s[e];
    } else if constexpr (M == Pairs::lane) {
#pragma unroll
      for (int e = 0; e + 1 < V; e += 2) {
        const float x = f[e], y = f[e + 1];
        f[e] = x * c[e] + y * s[e];
        f[e + 1] = y * c[e + 1] + x * s[e + 1];
      }
    } else if constexpr (M == Pairs::lds) {
      wave_sync();
#pragma unroll
      for (int e = 0; e < V; ++e) row[n + e] = f[e];
      wave_sync();
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const int i = n + e;
        if (i < 2 * a.R) f[e] = f[e] * c[e] + row[a.interleaved ? i ^ 1 : i < a.R ? i + a.R : i - a.R] * s[e];
      }
      wave_sync();
    }
  }
};

// The angles of `ntok` tokens from `tok`.
__device__ __forceinline__ void angles(const QkNormArgs& a, float2* cs, int64_t tok, int ntok) {
  for (int i = threadIdx.x; i < ntok * a.R; i += kQnThreads) {
    const int t = i / a.R;
    cs[i] = turn(a.pos[tok + t], a.freq[i - t * a.R]);
  }
}

// `per` tokens a workgroup; the row groups of a token share its heads.
template <typename T, int V, Pairs M, int RU>
__global__ __launch_bounds__(kQnThreads) void qk_norm_fwd_kernel(const QkNormArgs a, int lpr, int per) {
  extern __shared__ float lds[];        // angles of `per` tokens, then (lds) the groups' rows
  float2* cs = reinterpret_cast<float2*>(lds);
  const RowLane<V> L(a.D, lpr);
  const int64_t tok0 = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * per;
  if (tok0 >= a.tokens) return;
  const int ntok = (int)min((int64_t)per, a.tokens - tok0);
  const int group = threadIdx.x / lpr, gpt = L.rows / per, t = group / gpt, h0 = group % gpt;
  float* row = lds + 2 * per * a.R + group * a.D;
  // the first rows are on their way while the angles are made
  const T* src[2];
  Vec<T, V> x[2][RU], y[2][RU];
  float wt[2][V], wo[2][V];
  const int pair = other(a, L.n);
  auto load = [&](int k, int h) {
#pragma unroll
    for (int u = 0; u < RU; ++u) {
      const T* p = src[k] + (int64_t)min(h + u * gpt, a.heads[k] - 1) * a.D;
      x[k][u].load(p);
      if constexpr (M == Pairs::load) y[k][u].load(p + pair);
    }
  };
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    src[k] = static_cast<const T*>(a.x[k]) + (tok0 + min(t, ntok - 1)) * a.stride[k] + L.n;
    load(k, h0);
    weights(a, k, L.n, wt[k]);
    if constexpr (M == Pairs::load) weights(a, k, L.n + pair, wo[k]);
  }
  if constexpr (M != Pairs::none) {
    angles(a, cs, tok0, ntok);
    __syncthreads();
  }
  if (t >= ntok) return;
  Turns<V, M, false> tn;
  tn.get(a, cs + t * a.R, L.n);
  const float inv = a.l2 ? 1.f : 1.f / (float)a.D;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int heads = a.heads[k];
    T* dst = static_cast<T*>(a.out[k]) + (tok0 + t) * heads * a.D + L.n;
    for (int h = h0; h < heads; h += RU * gpt) {
      if (h > h0) load(k, h);
#pragma unroll
      for (int u = 0; u < RU; ++u) {
        float f[V], o[V], s = 0.f;
        x[k][u].get(f);
        if constexpr (M == Pairs::load) y[k][u].get(o);
#pragma unroll
        for (int e = 0; e < V; ++e) s += L.mine[e] ? f[e] * f[e] : 0.f;
        const float r = rsqrtf(run_sum_dpp(s, lpr) * inv + a.eps);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          f[e] = f[e] * r * wt[k][e];
          if constexpr (M == Pairs::load) o[e] = o[e] * r * wo[k][e];
        }
        tn.turn(a, o, row, L.n, f);
        x[k][u].set(f);
        if (h + u * gpt < heads && L.ln * V < a.D) x[k][u].store(dst + (int64_t)(h + u * gpt) * a.D);
      }
    }
  }
}

// With d = dout turned back, n = x r and dn = d w:
//   dx = r (dn - n mean or sum(dn n)),   dw = sum over rows of d n
// The sums over rows: a lane's own rows (kQnSegment of the workgroup's token tiles in one
// register, then those sums in another, so that long inputs lose no more than short ones),
// then the workgroup's, then the partial rows' columns (q's, then k's).
template <typename T, int V, Pairs M>
__global__ __launch_bounds__(kQnThreads, kQnMaxParts / 256) void qk_norm_bwd_kernel(const QkNormArgs a, int lpr, int per) {
  extern __shared__ float lds[];
  float2* cs = reinterpret_cast<float2*>(lds);
  const RowLane<V> L(a.D, lpr);
  const int group = threadIdx.x / lpr, gpt = L.rows / per, t = group / gpt, h0 = group % gpt;
  float* row = lds + 2 * per * a.R + group * a.D;
  float wt[2][V], dw[2][V], seg[2][V];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    weights(a, k, L.n, wt[k]);
#pragma unroll
    for (int e = 0; e < V; ++e) dw[k][e] = seg[k][e] = 0.f;
  }
  const int pair = other(a, L.n);
  int until = kQnSegment;
  const float inv = a.l2 ? 1.f : 1.f / (float)a.D;
  for (int64_t tok0 = (int64_t)blockIdx.x * per; tok0 < a.tokens; tok0 += (int64_t)gridDim.x * per) {
    const int ntok = (int)min((int64_t)per, a.tokens - tok0);
    if constexpr (M != Pairs::none) {
      __syncthreads();
      angles(a, cs, tok0, ntok);
      __syncthreads();
    }
    if (t < ntok) {
      Turns<V, M, true> tn;
      tn.get(a, cs + t * a.R, L.n);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int heads = a.heads[k];
        const T* src = static_cast<const T*>(a.x[k]) + (tok0 + t) * a.stride[k] + L.n;
        const T* dsrc = static_cast<const T*>(a.dout[k]) + (tok0 + t) * heads * a.D + L.n;
        T* dst = static_cast<T*>(a.dx[k]) + (tok0 + t) * a.dstride[k] + L.n;
#pragma unroll 2
        for (int h = h0; h < heads; h += gpt) {
          Vec<T, V> xq, dq, yq;
          xq.load(src + (int64_t)h * a.D);
          dq.load(dsrc + (int64_t)h * a.D);
          if constexpr (M == Pairs::load) yq.load(dsrc + (int64_t)h * a.D + pair);
          float x[V], d[V], o[V], s = 0.f;
          xq.get(x);
          dq.get(d);
          if constexpr (M == Pairs::load) yq.get(o);
          tn.turn(a, o, row, L.n, d);
#pragma unroll
          for (int e = 0; e < V; ++e) s += L.mine[e] ? x[e] * x[e] : 0.f;
          const float r = rsqrtf(run_sum_dpp(s, lpr) * inv + a.eps);
          float m = 0.f;
#pragma unroll
          for (int e = 0; e < V; ++e) {
            x[e] *= r;
            seg[k][e] += L.mine[e] ? d[e] * x[e] : 0.f;
            d[e] *= wt[k][e];
            m += L.mine[e] ? d[e] * x[e] : 0.f;
          }
          m = run_sum_dpp(m, lpr) * inv;
#pragma unroll
          for (int e = 0; e < V; ++e) d[e] = r * (d[e] - x[e] * m);
          dq.set(d);
          if (L.ln * V < a.D) dq.store(dst + (int64_t)h * a.D);
        }
      }
    }
    if (--until == 0 || tok0 + (int64_t)gridDim.x * per >= a.tokens) {
      until = kQnSegment;
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e) {
          dw[k][e] += seg[k][e];
          seg[k][e] = 0.f;
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

template <typename T, int V, Pairs M>
hipError_t qn_go(const QkNormArgs& a, bool bwd, hipStream_t s) {
  const int lpr = row_lanes(a.D, V), rows = kQnThreads / lpr;
  // a token's row groups: no more than its heads of q; a token a workgroup where there are few
  // tokens, else four at least, which share their angles' barrier (forward, 32 + 8 heads of 128:
  // 4 tokens 4.9 us, in fours 7.1; 16384 tokens 70 us, one by one 98)
  const int cus = device_cu_count() > 0 ? device_cu_count() : 256;
  int gpt = rows;
  while (gpt > 1 && gpt > a.heads[0]) gpt /= 2;
  if (a.tokens > 4 * (int64_t)cus && gpt > rows / kQnTok) gpt = rows / kQnTok;
  const int per = rows / gpt;
  const size_t row_lds = (size_t)rows * a.D * 4;
  const size_t lds = (size_t)per * a.R * 8 + (M == Pairs::lds || (bwd && a.part) ? row_lds : 0);
  const int64_t tiles = (a.tokens + per - 1) / per;
  if (!bwd) {
    if (tiles == 0) return hipSuccess;
    // rows of the grid, which may have 2^32 threads in each direction
    const int64_t x = tiles < kQnGridX ? tiles : kQnGridX;
    const dim3 grid((unsigned)x, (unsigned)((tiles + x - 1) / x));
    hipLaunchKernelGGL((qk_norm_fwd_kernel<T, V, M, 2>), grid, dim3(kQnThreads), lds, s, a, lpr, per);
    return hipGetLastError();
  }
  const int64_t most = a.part ? kQnMaxParts : (int64_t)1 << 22;
  const int grid = (int)(tiles < most ? tiles : most);
  if (grid > 0) hipLaunchKernelGGL((qk_norm_bwd_kernel<T, V, M>), dim3(grid), dim3(kQnThreads), lds, s, a, lpr, per);
  if (!a.part) return hipGetLastError();
  QkNormOut out;
  out.w[0] = a.dw[0];
  out.w[1] = a.dw[1];
  out.D = a.D;
  out.cp = (int)part_cols(a.D);
  return colsum(a.part, grid, 2 * part_cols(a.D), out, s);
}

template <typename T, int V>
hipError_t qn_pairs(const QkNormArgs& a, bool bwd, hipStream_t s) {
  if (a.R == 0) return qn_go<T, V, Pairs::none>(a, bwd, s);
  if constexpr (V > 1) {
    if (a.D % V == 0 && a.interleaved) return qn_go<T, V, Pairs::lane>(a, bwd, s);
    if (a.D % V == 0 && a.R % V == 0) return qn_go<T, V, Pairs::load>(a, bwd, s);
  }
  return qn_go<T, V, Pairs::lds>(a, bwd, s);
}

hipError_t qn_type(const QkNormArgs& a, bool bwd, hipStream_t s) {
  if (a.bf16) return a.D >= 8 ? qn_pairs<bf16, 8>(a, bwd, s) : qn_pairs<bf16, 1>(a, bwd, s);
  return a.D >= 4 ? qn_pairs<float, 4>(a, bwd, s) : qn_pairs<float, 1>(a, bwd, s);
}

}  // namespace

int64_t qk_norm_bwd_floats(int64_t tokens, int64_t D) {
  return (tokens < kQnMaxParts ? tokens : kQnMaxParts) * 2 * part_cols(D);
}

hipError_t launch_qk_norm_fwd(const QkNormArgs& a, hipStream_t s) { return qn_type(a, false, s); }
hipError_t launch_qk_norm_bwd(const QkNormArgs& a, hipStream_t s) { return qn_type(a, true, s); }

}  // namespace ssd

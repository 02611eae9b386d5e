// The norms around a block, forward and backward.  Per row of C channels:
//   p = x r1 post_w (or x),  u = p act(gate),  h = residual + alpha scale u,
//   out = h r2 pre_w,        r1 = rsqrt(mean x^2 + eps), r2 = rsqrt(mean h^2 + eps)
// and with n = h r2, m = x r1, f = alpha scale:
//   dn = dout pre_w,  dh = r2 (dn - n mean(dn n)) + dh_out
//   du = dh f,  dgate = du p act'(gate),  dp = du act,  dm = dp post_w
//   dx = r1 (dm - m mean(dm m))  (or dp),   dresidual = dh
//   dpre_w = sum dout n,  dscale = sum dh alpha u,  dpost_w = sum dp m
//
// What bounds it: memory; each input is read and each output written once.  A
// row stays in registers from its loads to its stores: it lies over W waves,
// KT vectors of V channels (16 bytes of x) per lane, and its sums (up to two
// forward, four backward, each needed before the next) are butterflies in
// registers, joined over the W waves in LDS.  W is the fewest waves that hold a
// row with KT = 2, so a row of up to 128 vectors needs no barrier at all.
//
// Weight gradients accumulate in registers over the rows a workgroup walks,
// leave as one partial row per workgroup and are added in workgroup order by a
// second launch.  No atomics.
#include "ssd_kernels.h"
#include "ssd_layer.h"
#include "ssd_layer_device.h"
#include "ssd_rowsum.h"

namespace ssd {

namespace {

template <typename T> constexpr int kBnV = 16 / (int)sizeof(T);

// Sum of v over the W waves of a row, the same in every lane.  `buf`: two
// buffers of W floats used in turn (`par`), so the barrier of one sum also
// frees the buffer of the sum before.
template <int W>
__device__ __forceinline__ float row_sum(float v, float (*buf)[W], int& par) {
  v = run_sum_dpp(v, 64);
  if constexpr (W > 1) {
    if ((threadIdx.x & 63) == 0) buf[par][threadIdx.x >> 6] = v;
    __syncthreads();
    v = buf[par][0];
#pragma unroll
    for (int w = 1; w < W; ++w) v += buf[par][w];
    par ^= 1;
  }
  return v;
}

// The channels [c, c + V) of a row of C channels, zeros past its end.
template <bool TAIL, typename E, int V>
__device__ __forceinline__ void bn_load(Vec<E, V>& q, const E* row, int c, int C) {
  if constexpr (TAIL) {
    if (c + V <= C) q.load(row + c);
    else q.load_some(row + c, C - c);
  } else {
    q.load(row + (c < C ? c : 0));
    q.clear_unless(c < C);
  }
}

template <bool TAIL, typename E, int V>
__device__ __forceinline__ void bn_store(const Vec<E, V>& q, E* row, int c, int C) {
  if (c + V <= C) q.store(row + c);
  else if (TAIL && c < C) q.store_some(row + c, C - c);
}

// Weights of the thread's channels: `one` where there is no weight, 0 past the
// row's end.
template <int KT, int V, int LANES>
__device__ __forceinline__ void bn_weights(const float* w, float mul, int t, int C,
                                           float (&out)[KT][V]) {
#pragma unroll
  for (int k = 0; k < KT; ++k)
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const int c = (t + k * LANES) * V + e;
      out[k][e] = c < C ? (w ? mul * w[c] : mul) : 0.f;
    }
}

// act(z) and its derivative.
__device__ __forceinline__ float bn_act(int kind, float z) {
  if (kind == 0) return z;
  const float s = sigmoid(z);
  return kind == 1 ? s : z * s;
}
__device__ __forceinline__ float bn_act_grad(int kind, float z, float& act) {
  if (kind == 0) {
    act = z;
    return 1.f;
  }
  const float s = sigmoid(z);
  act = kind == 1 ? s : z * s;
  return kind == 1 ? s * (1.f - s) : s * (1.f + z * (1.f - s));
}

// Threads of a workgroup: one row of W waves, or four rows of one wave.
template <int W> constexpr int kBnThreads = W > 1 ? W * 64 : 256;
template <int W> constexpr int kBnRows = kBnThreads<W> / (W * 64);

template <typename T, typename R, int W, int KT, bool TAIL>
__global__ __launch_bounds__(kBnThreads<W>) void block_norm_fwd_kernel(const BlockNormArgs a) {
  constexpr int V = kBnV<T>, LANES = W * 64, ROWS = kBnRows<W>;
  __shared__ float buf[2][W];
  int par = 0;
  const int t = threadIdx.x % LANES, C = a.C;
  const float inv = 1.f / (float)C;
  float pw[KT][V], fw[KT][V], nw[KT][V];
  bn_weights<KT, V, LANES>(a.post_w, 1.f, t, C, pw);
  bn_weights<KT, V, LANES>(a.scale, a.alpha, t, C, fw);
  bn_weights<KT, V, LANES>(a.pre_w, 1.f, t, C, nw);
  for (int64_t r = (int64_t)blockIdx.x * ROWS + threadIdx.x / LANES; r < a.rows;
       r += (int64_t)gridDim.x * ROWS) {
    const T* x = static_cast<const T*>(a.x) + r * C;
    const T* gate = static_cast<const T*>(a.gate) + r * C;
    const R* res = static_cast<const R*>(a.residual) + r * C;
    Vec<T, V> xq[KT], gq[KT];
    Vec<R, V> rq[KT];
#pragma unroll
    for (int k = 0; k < KT; ++k) {
      const int c = (t + k * LANES) * V;
      bn_load<TAIL>(xq[k], x, c, C);
      if (a.gate) bn_load<TAIL>(gq[k], gate, c, C);
      if (a.residual) bn_load<TAIL>(rq[k], res, c, C);
      else rq[k].clear();
    }
    float h[KT][V];
    float s = 0.f;
    if (a.post_w) {
#pragma unroll
      for (int k = 0; k < KT; ++k) {
        xq[k].get(h[k]);
#pragma unroll
        for (int e = 0; e < V; ++e) s += h[k][e] * h[k][e];
      }
      s = rsqrtf(row_sum<W>(s, buf, par) * inv + a.eps);
    }
    const float r1 = a.post_w ? s : 1.f;
    s = 0.f;
#pragma unroll
    for (int k = 0; k < KT; ++k) {
      float g[V], q[V];
      xq[k].get(h[k]);
      rq[k].get(q);
      if (a.gate) gq[k].get(g);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float u = h[k][e] * r1 * pw[k][e];
        if (a.gate) u *= bn_act(a.act, g[e]);
        h[k][e] = q[e] + fw[k][e] * u;
        s += h[k][e] * h[k][e];
      }
    }
    const float r2 = rsqrtf(row_sum<W>(s, buf, par) * inv + a.eps);
#pragma unroll
    for (int k = 0; k < KT; ++k) {
      const int c = (t + k * LANES) * V;
      float o[V];
#pragma unroll
      for (int e = 0; e < V; ++e) o[e] = h[k][e] * r2 * nw[k][e];
      Vec<T, V> oq;
      oq.set(o);
      bn_store<TAIL>(oq, static_cast<T*>(a.out) + r * C, c, C);
      if (a.res_out) {
        rq[k].set(h[k]);
        bn_store<TAIL>(rq[k], static_cast<R*>(a.res_out) + r * C, c, C);
      }
    }
  }
}

template <typename T, typename R, int W, int KT, bool TAIL>
__global__ __launch_bounds__(kBnThreads<W>) void block_norm_bwd_kernel(const BlockNormArgs a,
                                                                       int sec_scale, int sec_pre,
                                                                       int nsec) {
  constexpr int V = kBnV<T>, LANES = W * 64, ROWS = kBnRows<W>;
  __shared__ float buf[2][W];
  __shared__ float red[ROWS > 1 ? ROWS : 1][ROWS > 1 ? KT * LANES * V : 1];
  int par = 0;
  const int t = threadIdx.x % LANES, C = a.C;
  const float inv = 1.f / (float)C;
  float pw[KT][V], fw[KT][V], nw[KT][V];
  bn_weights<KT, V, LANES>(a.post_w, 1.f, t, C, pw);
  bn_weights<KT, V, LANES>(a.scale, a.alpha, t, C, fw);
  bn_weights<KT, V, LANES>(a.pre_w, 1.f, t, C, nw);
  float ap[KT][V], as[KT][V], an[KT][V];
#pragma unroll
  for (int k = 0; k < KT; ++k)
#pragma unroll
    for (int e = 0; e < V; ++e) ap[k][e] = as[k][e] = an[k][e] = 0.f;
  for (int64_t r = (int64_t)blockIdx.x * ROWS + threadIdx.x / LANES; r < a.rows;
       r += (int64_t)gridDim.x * ROWS) {
    const int64_t o = r * C;
    Vec<T, V> xq[KT], gq[KT], dq[KT];
    Vec<R, V> rq[KT], hq[KT];
#pragma unroll
    for (int k = 0; k < KT; ++k) {
      const int c = (t + k * LANES) * V;
      bn_load<TAIL>(xq[k], static_cast<const T*>(a.x) + o, c, C);
      bn_load<TAIL>(dq[k], static_cast<const T*>(a.dout) + o, c, C);
      if (a.gate) bn_load<TAIL>(gq[k], static_cast<const T*>(a.gate) + o, c, C);
      if (a.residual) bn_load<TAIL>(rq[k], static_cast<const R*>(a.residual) + o, c, C);
      else rq[k].clear();
      if (a.dres_out) bn_load<TAIL>(hq[k], static_cast<const R*>(a.dres_out) + o, c, C);
      else hq[k].clear();
    }
    float s = 0.f;
    if (a.post_w) {
#pragma unroll
      for (int k = 0; k < KT; ++k) {
        float x[V];
        xq[k].get(x);
#pragma unroll
        for (int e = 0; e < V; ++e) s += x[e] * x[e];
      }
      s = rsqrtf(row_sum<W>(s, buf, par) * inv + a.eps);
    }
    const float r1 = a.post_w ? s : 1.f;
    float h[KT][V];
    s = 0.f;
#pragma unroll
    for (int k = 0; k < KT; ++k) {
      float x[V], g[V], q[V];
      xq[k].get(x);
      rq[k].get(q);
      if (a.gate) gq[k].get(g);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float u = x[e] * r1 * pw[k][e];
        if (a.gate) u *= bn_act(a.act, g[e]);
        h[k][e] = q[e] + fw[k][e] * u;
        s += h[k][e] * h[k][e];
      }
    }
    const float r2 = rsqrtf(row_sum<W>(s, buf, par) * inv + a.eps);
    s = 0.f;
#pragma unroll
    for (int k = 0; k < KT; ++k) {
      float d[V];
      dq[k].get(d);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        h[k][e] *= r2;                            // n
        s += d[e] * nw[k][e] * h[k][e];
        an[k][e] += d[e] * h[k][e];
      }
    }
    const float mn = row_sum<W>(s, buf, par) * inv;
    s = 0.f;
#pragma unroll
    for (int k = 0; k < KT; ++k) {
      const int c = (t + k * LANES) * V;
      float x[V], g[V], d[V], dh[V], dg[V];
      xq[k].get(x);
      dq[k].get(d);
      hq[k].get(dh);
      if (a.gate) gq[k].get(g);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        dh[e] += r2 * (d[e] * nw[k][e] - h[k][e] * mn);
        const float m = x[e] * r1, p = m * pw[k][e], du = dh[e] * fw[k][e];
        float act = 1.f, da = 0.f;
        if (a.gate) da = bn_act_grad(a.act, g[e], act);
        as[k][e] += dh[e] * p * act;
        dg[e] = du * p * da;
        const float dp = du * act;
        ap[k][e] += dp * m;
        h[k][e] = dp * pw[k][e];                  // dm, or dp without a norm
        s += h[k][e] * m;
      }
      if (a.dres) {
        hq[k].set(dh);
        bn_store<TAIL>(hq[k], static_cast<R*>(a.dres) + o, c, C);
      }
      if (a.gate) {
        gq[k].set(dg);
        bn_store<TAIL>(gq[k], static_cast<T*>(a.dgate) + o, c, C);
      }
    }
    const float mm = a.post_w ? row_sum<W>(s, buf, par) * inv : 0.f;
#pragma unroll
    for (int k = 0; k < KT; ++k) {
      const int c = (t + k * LANES) * V;
      float x[V];
      xq[k].get(x);
#pragma unroll
      for (int e = 0; e < V; ++e) x[e] = r1 * (h[k][e] - x[e] * r1 * mm);
      xq[k].set(x);
      bn_store<TAIL>(xq[k], static_cast<T*>(a.dx) + o, c, C);
    }
  }
  // one partial row per workgroup and weight; four rows at a time are added
  // in LDS first
  float* part = a.part + (int64_t)blockIdx.x * nsec * C;
  auto put = [&](float(&v)[KT][V], int sec, float mul) {
    if constexpr (ROWS > 1) {
      const int row = threadIdx.x / LANES;
      __syncthreads();
#pragma unroll
      for (int k = 0; k < KT; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e) red[row][(t + k * LANES) * V + e] = v[k][e];
      __syncthreads();
      for (int c = threadIdx.x; c < C; c += kBnThreads<W>) {
        float u = red[0][c];
#pragma unroll
        for (int q = 1; q < ROWS; ++q) u += red[q][c];
        part[(int64_t)sec * C + c] = u * mul;
      }
    } else {
#pragma unroll
      for (int k = 0; k < KT; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const int c = (t + k * LANES) * V + e;
          if (c < C) part[(int64_t)sec * C + c] = v[k][e] * mul;
        }
    }
  };
  if (a.post_w) put(ap, 0, 1.f);
  if (a.scale) put(as, sec_scale, a.alpha);
  put(an, sec_pre, 1.f);
}

// Column sec C + c of the partial sums.
struct BlockNormOut {
  float* w[3];
  int C;
  __device__ __forceinline__ void put(int col, float v) const {
    const int sec = col / C;
    float* o = sec == 0 ? w[0] : sec == 1 ? w[1] : w[2];
    o[col - sec * C] = v;
  }
};

constexpr int kBnMaxParts = 1024;        // partial rows the workspace holds
int bn_grid(int64_t rows, int rows_per_group, int per_cu, int most) {
  const int cus = device_cu_count();
  int64_t want = (int64_t)(cus > 0 ? cus : 256) * per_cu;
  if (want > most) want = most;
  const int64_t groups = (rows + rows_per_group - 1) / rows_per_group;
  return (int)(groups < want ? groups : want);
}

template <bool BWD, typename T, typename R, int W, int KT, bool TAIL>
hipError_t bn_go(const BlockNormArgs& a, hipStream_t s) {
  if constexpr (!BWD) {
    const int grid = bn_grid(a.rows, kBnRows<W>, 8, 1 << 20);
    hipLaunchKernelGGL((block_norm_fwd_kernel<T, R, W, KT, TAIL>), dim3(grid),
                       dim3(kBnThreads<W>), 0, s, a);
  } else {
    const int nsec = 1 + (a.post_w ? 1 : 0) + (a.scale ? 1 : 0);
    const int sec_scale = a.post_w ? 1 : 0, sec_pre = nsec - 1;
    BlockNormOut out;
    out.C = a.C;
    out.w[0] = out.w[1] = out.w[2] = a.dpre_w;
    if (a.post_w) out.w[0] = a.dpost_w;
    if (a.scale) out.w[sec_scale] = a.dscale;
    const int grid = bn_grid(a.rows, kBnRows<W>, 4, kBnMaxParts);
    if (grid > 0)
      hipLaunchKernelGGL((block_norm_bwd_kernel<T, R, W, KT, TAIL>), dim3(grid),
                         dim3(kBnThreads<W>), 0, s, a, sec_scale, sec_pre, nsec);
    const int cols = nsec * a.C;
    hipLaunchKernelGGL(colsum_kernel<BlockNormOut>, dim3((cols + 63) / 64), dim3(kColsumThreads), 0,
                       s, (const float*)a.part, grid, cols, out);
  }
  return hipGetLastError();
}

template <bool BWD, typename T, typename R, bool TAIL>
hipError_t bn_rows(const BlockNormArgs& a, hipStream_t s) {
  const int nvec = (a.C + kBnV<T> - 1) / kBnV<T>;
  if (nvec <= 64) return bn_go<BWD, T, R, 1, 1, TAIL>(a, s);
  if (nvec <= 128) return bn_go<BWD, T, R, 1, 2, TAIL>(a, s);
  if (nvec <= 256) return bn_go<BWD, T, R, 2, 2, TAIL>(a, s);
  if (nvec <= 512) return bn_go<BWD, T, R, 4, 2, TAIL>(a, s);
  if (nvec <= 1024) return bn_go<BWD, T, R, 8, 2, TAIL>(a, s);
  if constexpr (sizeof(T) == 4) return bn_go<BWD, T, R, 16, 2, TAIL>(a, s);
  return hipErrorInvalidValue;
}

template <bool BWD, typename T, typename R>
hipError_t bn_tail(const BlockNormArgs& a, hipStream_t s) {
  return a.C % kBnV<T> ? bn_rows<BWD, T, R, true>(a, s) : bn_rows<BWD, T, R, false>(a, s);
}

template <bool BWD>
hipError_t bn_type(const BlockNormArgs& a, hipStream_t s) {
  if (!a.bf16) return bn_tail<BWD, float, float>(a, s);
  return a.res_bf16 ? bn_tail<BWD, bf16, bf16>(a, s) : bn_tail<BWD, bf16, float>(a, s);
}

}  // namespace

int64_t block_norm_bwd_floats(int64_t rows, int64_t C) {
  return (rows < kBnMaxParts ? rows : kBnMaxParts) * 3 * C;
}

hipError_t launch_block_norm_fwd(const BlockNormArgs& a, hipStream_t s) {
  if (a.rows <= 0) return hipSuccess;
  return bn_type<false>(a, s);
}

hipError_t launch_block_norm_bwd(const BlockNormArgs& a, hipStream_t s) {
  return bn_type<true>(a, s);
}

}  // namespace ssd

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
// row lies over W waves, one vector of four channels per lane (KT vectors in rows
// wider than 2048 channels), and stays in registers from its loads to its
// stores.  Its sums are butterflies in registers, joined over the W waves in LDS
// with one barrier: two exchanges forward (the norm after the block, then the
// one before the next), and two backward, whose later sums are arranged to need
// nothing that the second exchange computes.  Four channels per lane rather
// than eight: fewer registers, more rows in flight (forward at 8192 x 768 with an
// fp32 residual and a gate 23.5 -> 15.7 us, 5.6 TB/s; backward 82 -> 37 us, 3.8 TB/s with its
// second launch).
//
// A row that does not fill its waves pays for the last one: backward at 5003 rows of
// fp32 31.7 us for 1024 channels, 35.8 for 1028 (a fifth wave with one lane in use), 36.0
// for 1025; in bf16 at 8192 rows 21.9 for 768, 26.7 for 772.  Channels that are no whole
// vectors add the tail's loads one by one, each waited for: 35.9 for 771 (forward 9.7 / 13.1
// / 17.2).  Where rows start costs little: 1024 one element off 30.8.
//
// The forward keeps the next row's loads in flight; the backward, with twice
// the registers, gains nothing from that at 8192 x 768 (37.3 / 37.4 us with /
// without) and loses a wave in wider rows (8192 x 2048: 83 / 76 us).  Rows of one
// wave with three vectors per lane need no barrier, but 226 registers: 44 us.
//
// Weight gradients accumulate in registers over the rows a workgroup walks, in
// segments (bn_segment), leave as one partial row per workgroup and are added in
// workgroup order by a second launch.  No atomics.
#include "ssd_kernels.h"
#include "ssd_layer.h"
#include "ssd_layer_device.h"
#include "ssd_rowsum.h"

// Multiply-adds are fused only inside one expression, so every variant of a kernel
// rounds a value alike.
#pragma clang fp contract(on)

namespace ssd {

namespace {

// Sums of s[0..M) over the W waves of a row, the same in every lane.  `buf` holds
// two sets of W floats per sum and row, used in turn (`par`), so the barrier of
// one call also frees the set of the call before.  Every thread of the workgroup
// calls it.
template <int W, int RG, int M, int MAXM>
__device__ __forceinline__ void row_sums(float (&s)[M], float (*buf)[MAXM][RG][W], int rg, int& par) {
#pragma unroll
  for (int i = 0; i < M; ++i) s[i] = run_sum_dpp(s[i], 64);
  if constexpr (W > 1) {
    const int w = wave_id() - rg * W;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < M; ++i) buf[par][i][rg][w] = s[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < M; ++i) {
      s[i] = buf[par][i][rg][0];
#pragma unroll
      for (int j = 1; j < W; ++j) s[i] += buf[par][i][rg][j];
    }
    par ^= 1;
  }
}

// The channels [c, c + V) of a row of C channels, zeros past its end: with TAIL
// from the load itself, else after bn_trim, which the caller leaves until the
// values are needed (so that it does not wait for them any earlier).
template <bool TAIL, typename E, int V>
__device__ __forceinline__ void bn_load(Vec<E, V>& q, const E* row, int c, int C) {
  if constexpr (TAIL) {
    if (c + V <= C) q.load(row + c);
    else q.load_some(row + c, C - c);
  } else {
    q.load(row + (c < C ? c : 0));
  }
}
template <bool TAIL, typename E, int V>
__device__ __forceinline__ void bn_trim(Vec<E, V>& q, int c, int C) {
  if constexpr (!TAIL) q.clear_unless(c < C);
}

template <bool TAIL, typename E, int V>
__device__ __forceinline__ void bn_store(const Vec<E, V>& q, E* row, int c, int C) {
  if (c + V <= C) q.store(row + c);
  else if (TAIL && c < C) q.store_some(row + c, C - c);
}

// Weights of the thread's channels, times `mul`; `mul` where there is no weight,
// 0 past the row's end.
template <bool TAIL, int KT, int V, int LANES>
__device__ __forceinline__ void bn_weights(const float* w, float mul, int t, int C,
                                           float (&out)[KT][V]) {
#pragma unroll
  for (int k = 0; k < KT; ++k) {
    const int c = (t + k * LANES) * V;
    Vec<float, V> q;
    if (w) {
      bn_load<TAIL>(q, w, c, C);
      q.get(out[k]);
    }
#pragma unroll
    for (int e = 0; e < V; ++e) out[k][e] = c + e < C ? (w ? mul * out[k][e] : mul) : 0.f;
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

// The row of row group rg in the pass from row r0 on: past the last row, the last
// one again; past the last pass, the row of the pass before (whose lines are
// near; one row for all workgroups would be a hot spot).
__device__ __forceinline__ int64_t bn_row(int64_t r0, int rg, int64_t rows) {
  return min(r0 + rg, rows - 1);
}
__device__ __forceinline__ int64_t bn_next(int64_t r0, int64_t step, int rg, int64_t rows) {
  return bn_row(r0 + step < rows ? r0 + step : r0, rg, rows);
}

// A workgroup holds RG rows of W waves each and walks over rows with a stride of
// the grid; the next row's loads are in flight while a row is worked on.
template <typename T, typename R, int V, int W, int KT, int RG, bool TAIL>
__global__ __launch_bounds__(64 * W * RG) void block_norm_fwd_kernel(const BlockNormArgs a) {
  constexpr int LANES = W * 64;
  __shared__ float buf[2][1][RG][W];
  int par = 0;
  const int rg = RG > 1 ? wave_id() / W : 0, t = threadIdx.x - rg * LANES, C = a.C;
  const float inv = 1.f / (float)C;
  float pw[KT][V], fw[KT][V], nw[KT][V];
  Vec<T, V> xq[KT], gq[KT], nx[KT], ng[KT];
  Vec<R, V> rq[KT], nr[KT];
  auto load = [&](int64_t r, Vec<T, V>(&x)[KT], Vec<T, V>(&g)[KT], Vec<R, V>(&q)[KT]) {
#pragma unroll
    for (int k = 0; k < KT; ++k) {
      const int c = (t + k * LANES) * V;
      bn_load<TAIL>(x[k], static_cast<const T*>(a.x) + r * C, c, C);
      // where there is no gate or residual, x's row again: loaded, never used
      bn_load<TAIL>(g[k], static_cast<const T*>(a.gate ? a.gate : a.x) + r * C, c, C);
      if (a.residual) bn_load<TAIL>(q[k], static_cast<const R*>(a.residual) + r * C, c, C);
      else q[k].clear();
    }
  };
  load(bn_row((int64_t)blockIdx.x * RG, rg, a.rows), xq, gq, rq);
  bn_weights<TAIL, KT, V, LANES>(a.post_w, 1.f, t, C, pw);
  bn_weights<TAIL, KT, V, LANES>(a.scale, a.alpha, t, C, fw);
  bn_weights<TAIL, KT, V, LANES>(a.pre_w, 1.f, t, C, nw);
#pragma unroll 1
  for (int64_t r0 = (int64_t)blockIdx.x * RG; r0 < a.rows; r0 += (int64_t)gridDim.x * RG) {
    load(bn_next(r0, (int64_t)gridDim.x * RG, rg, a.rows), nx, ng, nr);
#pragma unroll
    for (int k = 0; k < KT; ++k) {
      bn_trim<TAIL>(xq[k], (t + k * LANES) * V, C);
      bn_trim<TAIL>(gq[k], (t + k * LANES) * V, C);
      bn_trim<TAIL>(rq[k], (t + k * LANES) * V, C);
    }
    float h[KT][V], s[1] = {0.f};
    float r1 = 1.f;
    if (a.post_w) {
#pragma unroll
      for (int k = 0; k < KT; ++k) {
        xq[k].get(h[k]);
#pragma unroll
        for (int e = 0; e < V; ++e) s[0] += h[k][e] * h[k][e];
      }
      row_sums<W, RG>(s, buf, rg, par);
      r1 = rsqrtf(s[0] * inv + a.eps);
      s[0] = 0.f;
    }
#pragma unroll
    for (int k = 0; k < KT; ++k) {
      float g[V], q[V];
      xq[k].get(h[k]);
      rq[k].get(q);
      gq[k].get(g);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float u = h[k][e] * r1 * pw[k][e];
        if (a.gate) u *= bn_act(a.act, g[e]);
        h[k][e] = q[e] + fw[k][e] * u;
        s[0] += h[k][e] * h[k][e];
      }
    }
    row_sums<W, RG>(s, buf, rg, par);
    const float r2 = rsqrtf(s[0] * inv + a.eps);
    const int64_t o = (r0 + rg) * C;
#pragma unroll
    for (int k = 0; k < KT; ++k) {
      const int c = (t + k * LANES) * V;
      if (r0 + rg < a.rows) {
        float out[V];
#pragma unroll
        for (int e = 0; e < V; ++e) out[e] = h[k][e] * r2 * nw[k][e];
        Vec<T, V> oq;
        oq.set(out);
        bn_store<TAIL>(oq, static_cast<T*>(a.out) + o, c, C);
        if (a.res_out) {
          rq[k].set(h[k]);
          bn_store<TAIL>(rq[k], static_cast<R*>(a.res_out) + o, c, C);
        }
      }
      xq[k] = nx[k];
      gq[k] = ng[k];
      rq[k] = nr[k];
    }
  }
}

// Backward.  With y = f act post_w m (what dh is multiplied by on its way to
// m), every sum after r1 is linear in quantities known before r2, so one
// exchange serves them all: mean(dn n) = r2 mean(dn h), and mean(dm m) =
// mean(y dh) = r2 mean(y dn) - r2^3 mean(dn h) mean(y h) + mean(y dh_out).
//
// The gate's factors are formed twice, and with several vectors per lane the
// weights wait in LDS, to keep the registers for rows in flight.
template <typename T, typename R, int V, int W, int KT, int RG, bool TAIL, bool SEG>
__global__ __launch_bounds__(64 * W * RG) void block_norm_bwd_kernel(const BlockNormArgs a,
                                                                     int sec_scale, int sec_pre,
                                                                     int64_t seg) {
  constexpr int LANES = W * 64, CC = LANES * KT * V;
  constexpr bool kLds = KT > 1;                   // weights in LDS
  static_assert(W == 1 || RG == 1, "rows of several waves do not share a workgroup's barriers");
  static_assert(!kLds || RG == 1, "one row per workgroup with the weights in LDS");
  __shared__ float buf[2][5][RG][W];
  __shared__ __align__(16) float wt[kLds ? 3 : 1][kLds || RG > 1 ? CC : 1];
  int par = 0;
  const int rg = RG > 1 ? wave_id() : 0, t = threadIdx.x - rg * LANES, C = a.C;
  const float inv = 1.f / (float)C;
  float wr[3][KT][V];
  if constexpr (kLds) {
    for (int c = threadIdx.x; c < CC; c += LANES) {
      wt[0][c] = c < C ? (a.post_w ? a.post_w[c] : 1.f) : 0.f;
      wt[1][c] = c < C ? a.alpha * (a.scale ? a.scale[c] : 1.f) : 0.f;
      wt[2][c] = c < C ? a.pre_w[c] : 0.f;
    }
    __syncthreads();
  } else {
    bn_weights<TAIL, KT, V, LANES>(a.post_w, 1.f, t, C, wr[0]);
    bn_weights<TAIL, KT, V, LANES>(a.scale, a.alpha, t, C, wr[1]);
    bn_weights<TAIL, KT, V, LANES>(a.pre_w, 1.f, t, C, wr[2]);
  }
  auto weights = [&](int k, int i, float(&w)[V]) {
    if constexpr (kLds) {
      Vec<float, V> q;
      q.load(&wt[i][(t + k * LANES) * V]);
      q.get(w);
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) w[e] = wr[i][k][e];
    }
  };
  // One partial row per workgroup and weight: a segment's sums, added to those of the
  // segments before by the same threads.  Rows of one wave are added in LDS first, in
  // the order of the waves.
  const int cp = (int)part_cols(C);
  auto put = [&](float(&v)[KT][V], int sec, float mul, bool add) {
    // read again in every segment, or its addresses would be held over the rows
    const int t = body_tid<SEG, 64 * W * RG>() - rg * LANES;
    if constexpr (RG > 1) {
      float* red = wt[0];
#pragma unroll 1
      for (int g = 0; g < RG; ++g) {
        __syncthreads();
        if (rg == g) {
#pragma unroll
          for (int k = 0; k < KT; ++k)
#pragma unroll
            for (int e = 0; e < V; ++e) {
              float* to = red + (t + k * LANES) * V + e;
              *to = g == 0 ? v[k][e] : *to + v[k][e];
            }
        }
      }
      __syncthreads();
      for (int c = threadIdx.x; c < C; c += LANES * RG) {
        float* to = part_at(a.part, (int)blockIdx.x, (int)gridDim.x, sec * cp + c);
        *to = add ? *to + red[c] * mul : red[c] * mul;
      }
    } else {
#pragma unroll
      for (int k = 0; k < KT; ++k) {
#pragma unroll
        for (int e = 0; e < V; ++e) v[k][e] *= mul;
        // a whole vector: its section's columns go to the end of a block
        const int c = (t + k * LANES) * V;
        if (c >= C) continue;
        float* to = part_at(a.part, (int)blockIdx.x, (int)gridDim.x, sec * cp + c);
        Vec<float, V> q;
        if (add) {
          float was[V];
          q.load(to);
          q.get(was);
#pragma unroll
          for (int e = 0; e < V; ++e) v[k][e] += was[e];
        }
        q.set(v[k]);
        q.store(to);
      }
    }
  };
  const int64_t first = (int64_t)blockIdx.x * RG, step = (int64_t)gridDim.x * RG;
#pragma unroll 1
  for (int64_t s0 = first; s0 < a.rows; s0 += seg * step) {
    const int64_t s1 = SEG ? min(s0 + seg * step, a.rows) : a.rows;
    float ap[KT][V], as[KT][V], an[KT][V];
#pragma unroll
    for (int k = 0; k < KT; ++k)
#pragma unroll
      for (int e = 0; e < V; ++e) ap[k][e] = as[k][e] = an[k][e] = 0.f;
#pragma unroll 1
    for (int64_t r = s0 + rg; r < s1; r += step) {
      // with segments the row's number goes through an empty asm statement, or each lane
      // would hold one address per tensor from row to row (up to 20 registers)
      int64_t row = r;
      if constexpr (SEG) asm("" : "+s"(row));
      const int64_t o = row * C;
      Vec<T, V> xq[KT], gq[KT], dq[KT];
      Vec<R, V> rq[KT], hq[KT];
#pragma unroll
      for (int k = 0; k < KT; ++k) {
        const int c = (t + k * LANES) * V;
        bn_load<TAIL>(xq[k], static_cast<const T*>(a.x) + o, c, C);
        // where there is no gate, x's row again: loaded, never used
        bn_load<TAIL>(gq[k], static_cast<const T*>(a.gate ? a.gate : a.x) + o, c, C);
        bn_load<TAIL>(dq[k], static_cast<const T*>(a.dout) + o, c, C);
        if (a.residual) bn_load<TAIL>(rq[k], static_cast<const R*>(a.residual) + o, c, C);
        else rq[k].clear();
        if (a.dres_out) bn_load<TAIL>(hq[k], static_cast<const R*>(a.dres_out) + o, c, C);
        else hq[k].clear();
      }
#pragma unroll
      for (int k = 0; k < KT; ++k) {
        bn_trim<TAIL>(xq[k], (t + k * LANES) * V, C);
        bn_trim<TAIL>(rq[k], (t + k * LANES) * V, C);
        bn_trim<TAIL>(gq[k], (t + k * LANES) * V, C);
        bn_trim<TAIL>(dq[k], (t + k * LANES) * V, C);
        bn_trim<TAIL>(hq[k], (t + k * LANES) * V, C);
      }
      float r1 = 1.f;
      if (a.post_w) {
        float s[1] = {0.f};
#pragma unroll
        for (int k = 0; k < KT; ++k) {
          float x[V];
          xq[k].get(x);
#pragma unroll
          for (int e = 0; e < V; ++e) s[0] += x[e] * x[e];
        }
        row_sums<W, RG>(s, buf, rg, par);
        r1 = rsqrtf(s[0] * inv + a.eps);
      }
      // sums of h^2, dn h, and with a norm of y dn, y h, y dh_out
      float h[KT][V], s[5] = {0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < KT; ++k) {
        float x[V], g[V], q[V], d[V], ho[V], pw[V], fw[V], nw[V];
        xq[k].get(x);
        rq[k].get(q);
        dq[k].get(d);
        gq[k].get(g);
        hq[k].get(ho);
        weights(k, 0, pw);
        weights(k, 1, fw);
        weights(k, 2, nw);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float act = a.gate ? bn_act(a.act, g[e]) : 1.f;
          const float y = x[e] * r1 * pw[e] * act * fw[e], dn = d[e] * nw[e];
          h[k][e] = q[e] + y;
          s[0] += h[k][e] * h[k][e];
          s[1] += dn * h[k][e];
          s[2] += y * dn;
          s[3] += y * h[k][e];
          s[4] += y * ho[e];
        }
      }
      row_sums<W, RG>(s, buf, rg, par);
      const float r2 = rsqrtf(s[0] * inv + a.eps);
      // dh = r2 (dn - c n) + dh_out.  Factors r2 only beside an h: r2^3 would leave fp32's
      // range for |h| beyond 1e12 (and under 1e-12 without eps).
      const float c2 = r2 * (s[1] * inv);
      const float mm = a.post_w ? (r2 * (s[2] - c2 * (r2 * s[3])) + s[4]) * inv : 0.f;
#pragma unroll
      for (int k = 0; k < KT; ++k) {
        const int c = (t + k * LANES) * V;
        float x[V], g[V], d[V], dh[V], dg[V], pw[V], fw[V], nw[V];
        xq[k].get(x);
        dq[k].get(d);
        gq[k].get(g);
        hq[k].get(dh);
        weights(k, 0, pw);
        weights(k, 1, fw);
        weights(k, 2, nw);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          float act = 1.f, da = 0.f;
          if (a.gate) da = bn_act_grad(a.act, g[e], act);
          const float n = h[k][e] * r2;
          an[k][e] += d[e] * n;
          dh[e] += r2 * (d[e] * nw[e] - c2 * n);
          const float m = x[e] * r1, p = m * pw[e], du = dh[e] * fw[e], dp = du * act;
          as[k][e] += dh[e] * (p * act);
          dg[e] = du * p * da;
          ap[k][e] += dp * m;
          x[e] = r1 * (dp * pw[e] - m * mm);
        }
        xq[k].set(x);
        bn_store<TAIL>(xq[k], static_cast<T*>(a.dx) + o, c, C);
        if (a.dres) {
          hq[k].set(dh);
          bn_store<TAIL>(hq[k], static_cast<R*>(a.dres) + o, c, C);
        }
        if (a.gate) {
          gq[k].set(dg);
          bn_store<TAIL>(gq[k], static_cast<T*>(a.dgate) + o, c, C);
        }
      }
    }
    const bool add = SEG && s0 > first;
    if (a.post_w) put(ap, 0, 1.f, add);
    if (a.scale) put(as, sec_scale, a.alpha, add);
    put(an, sec_pre, 1.f, add);
    if (!SEG) return;
  }
}

// Column c of section sec of the partial sums.
struct BlockNormOut {
  float* w[3];
  int C, cp;
  __device__ __forceinline__ void put(int col, float v) const {
    const int sec = col / cp, c = col - sec * cp;
    if (c >= C) return;
    float* o = sec == 0 ? w[0] : sec == 1 ? w[1] : w[2];
    o[c] = v;
  }
};

constexpr int kBnMaxParts = 2048;        // partial rows the workspace holds
int bn_grid(int64_t rows, int rows_per_group, int per_cu, int most) {
  const int cus = device_cu_count();
  int64_t want = (int64_t)(cus > 0 ? cus : 256) * per_cu;
  if (want > most) want = most;
  const int64_t groups = (rows + rows_per_group - 1) / rows_per_group;
  return (int)(groups < want ? groups : want);
}

// Rows whose terms of the weight gradients one register adds before they go to the
// partial row, of the `walk` rows that a wave walks: 64, and their square root where
// that is more, so that a term passes at most 64 + walk / 64 or 2 sqrt(walk) additions
// there, not one per row.  (2^23 rows of equal terms, 2048 a wave: off by 382 2^-24 in one
// register, by 15 in segments.  262144 x 768 900 and 912 us, 65536 x 8192 1447 and 1385.)
// Up to 64 rows a wave run the kernel without the segments' test.
int64_t bn_segment(int64_t walk) {
  int64_t seg = 64;
  while (seg * seg < walk) ++seg;
  return seg;
}

// Workgroups per CU: as many as are resident, so that each walks over rows to the
// end of the launch.  A forward wave needs about 50 registers (six waves per
// SIMD and more), a backward one about 100 (four per SIMD); with several vectors
// per lane the backward's LDS and registers leave one workgroup.  More than are
// resident costs a second, part-filled round: the backward at 8192 x 1536 took
// 91 us with three workgroups of six waves per CU, 73 with two.
template <bool BWD, typename T, typename R, int W, int KT, bool TAIL>
hipError_t bn_go(const BlockNormArgs& a, hipStream_t s) {
  constexpr int V = 4, RG = W == 1 ? 4 : 1;
  if constexpr (!BWD) {
    const int grid = bn_grid(a.rows, RG, 24 / (W * RG) > 1 ? 24 / (W * RG) : 1, 1 << 20);
    hipLaunchKernelGGL((block_norm_fwd_kernel<T, R, V, W, KT, RG, TAIL>), dim3(grid),
                       dim3(64 * W * RG), 0, s, a);
    return hipGetLastError();
  } else {
    const int nsec = 1 + (a.post_w ? 1 : 0) + (a.scale ? 1 : 0);
    const int sec_scale = a.post_w ? 1 : 0, sec_pre = nsec - 1;
    BlockNormOut out;
    out.C = a.C;
    out.cp = (int)part_cols(a.C);
    out.w[0] = out.w[1] = out.w[2] = a.dpre_w;
    if (a.post_w) out.w[0] = a.dpost_w;
    if (a.scale) out.w[sec_scale] = a.dscale;
    const int grid = bn_grid(a.rows, RG, KT == 1 ? 16 / (W * RG) : 1, kBnMaxParts);
    const int64_t walk = grid > 0 ? (a.rows + (int64_t)grid * RG - 1) / ((int64_t)grid * RG) : 0;
    const int64_t seg = bn_segment(walk);
    auto fn = seg < walk ? &block_norm_bwd_kernel<T, R, V, W, KT, RG, TAIL, true>
                         : &block_norm_bwd_kernel<T, R, V, W, KT, RG, TAIL, false>;
    if (grid > 0)
      hipLaunchKernelGGL(fn, dim3(grid), dim3(64 * W * RG), 0, s, a, sec_scale, sec_pre, seg);
    return colsum(a.part, grid, nsec * part_cols(a.C), out, s);
  }
}

template <bool BWD, typename T, typename R, bool TAIL>
hipError_t bn_rows(const BlockNormArgs& a, hipStream_t s) {
  const int nw = (a.C + 255) / 256;         // waves a row fills with one vector per lane
  switch (nw) {
#define SSD_BN(w) case w: return bn_go<BWD, T, R, w, 1, TAIL>(a, s);
    SSD_BN(1) SSD_BN(2) SSD_BN(3) SSD_BN(4) SSD_BN(5) SSD_BN(6) SSD_BN(7) SSD_BN(8)
#undef SSD_BN
  }
  // wider rows: sixteen waves forward; backward eight with more vectors per
  // lane, as 1024 threads leave too few registers (bf16 with an fp32 stream, all
  // parts: 4096 x 4096 208 us against 93, 2048 x 8192 306 against 135; today 92 and 118)
  constexpr int W = BWD ? 8 : 16;
  if (nw <= 16) return bn_go<BWD, T, R, W, 16 / W, TAIL>(a, s);
  return bn_go<BWD, T, R, W, 32 / W, TAIL>(a, s);
}

template <bool BWD, typename T, typename R>
hipError_t bn_tail(const BlockNormArgs& a, hipStream_t s) {
  return a.C % 4 ? bn_rows<BWD, T, R, true>(a, s) : bn_rows<BWD, T, R, false>(a, s);
}

template <bool BWD>
hipError_t bn_type(const BlockNormArgs& a, hipStream_t s) {
  if (!a.bf16) return bn_tail<BWD, float, float>(a, s);
  return a.res_bf16 ? bn_tail<BWD, bf16, bf16>(a, s) : bn_tail<BWD, bf16, float>(a, s);
}

}  // namespace

int64_t block_norm_bwd_floats(int64_t rows, int64_t C) {
  return (rows < kBnMaxParts ? rows : kBnMaxParts) * 3 * part_cols(C);
}

hipError_t launch_block_norm_fwd(const BlockNormArgs& a, hipStream_t s) {
  if (a.rows <= 0) return hipSuccess;
  return bn_type<false>(a, s);
}

hipError_t launch_block_norm_bwd(const BlockNormArgs& a, hipStream_t s) {
  return bn_type<true>(a, s);
}

}  // namespace ssd

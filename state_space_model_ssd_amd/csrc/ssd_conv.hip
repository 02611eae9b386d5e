// The short causal convolution over the channels x | B | C, its backward and
// its single-token form.  Per sequence, token t and channel c:
//   pre[t] = bias + sum_k w[k] in[t - (K-1) + k],   out = pre sigma(pre) or pre
//   dpre[t] = dout[t] act'(pre[t])
//   din[t] = sum_j w[K-1-j] dpre[t+j],  dw[k] = sum_t dpre[t] in[t - (K-1) + k]
//
// What bounds it: memory.  A forward reads and writes every element once for
// about 2 K + 10 operations, a backward reads two and writes one.  So a thread
// owns V neighbouring channels and a run of tokens, a wave 64 such vectors of one
// run, and a workgroup four runs in a row.  The forward loads all rows of a run,
// the K - 1 before it included, at once into registers; the backward a group of
// rows ahead.  The rows that two runs share come from the L1 and L2: the forward reads
// each element from memory once (6144 channels x 32768 tokens of bf16: 403.6 MB for
// 402.8, 150 us, 5.4 TB/s, a large copy's rate).  The backward, in column tiles of 256
// bytes, reads 78.2 MB for 58.7 at 1792 x 8192 out of rows of 3352 channels, which start
// anywhere in a 128-byte line: tiles share lines, and neighbouring tiles run on
// different XCDs.  It takes 23.3 us with its second launch (3.8 TB/s).
//
// Runs never straddle a sequence: a workgroup's tokens are the overlap of one
// WT-token tile of the token axis with one sequence.  Slot i of the grid is
// sequence s, tile i - s, for the largest s with tile(first token of s) + s <=
// i: those pairs are all different, cover every token, and there are at most
// tiles + sequences of them, so no table has to be built first.  Inside a run
// only the first K - 1 rows can lie before the sequence (initial state or
// zeros) and only the last K - 1 behind it, each decided per row by the whole
// wave at once.
#include "ssd_kernels.h"
#include "ssd_layer.h"
#include "ssd_layer_device.h"

// Multiply-adds are fused only inside one expression, so every variant of a kernel
// rounds a value alike.
#pragma clang fp contract(on)

namespace ssd {

namespace {

constexpr int kConvThreads = 256;
constexpr int kConvWaves = kConvThreads / kWave;

// The overlap of a tile with a sequence: tokens [lo, hi) of sequence s, which
// owns [start, end).
struct ConvTile {
  int s, start, end, lo, hi;
};

__device__ __forceinline__ int clamp_cu(const int32_t* cu, int s, int total) {
  return min(max(cu[s], 0), total);
}

// Tokens of sequence s.
__device__ __forceinline__ void conv_seq(const ConvArgs& a, int s, ConvTile& t) {
  t.s = s;
  t.start = a.cu ? clamp_cu(a.cu, s, a.total) : s * a.seqlen;
  t.end = a.cu ? max(t.start, clamp_cu(a.cu, s + 1, a.total)) : t.start + a.seqlen;
}

// Slots of a launch with WT-token tiles (an upper bound for a packed batch).
int conv_slots(const ConvArgs& a, int WT) {
  if (a.cu) return (a.total + WT - 1) / WT + a.nstates;
  return a.nstates * ((a.seqlen + WT - 1) / WT);
}

// Every lane of a wave calls it with the same slot and gets the same answer.
// The search probes 64 sequences at a time, one per lane.
template <int WT>
__device__ __forceinline__ ConvTile conv_tile(const ConvArgs& a, int slot) {
  ConvTile t;
  if (a.cu) {
    const int lane = threadIdx.x & 63;
    int lo = 0, n = a.nstates;
    while (n > 1) {
      const int step = (n + 63) / 64;
      const int i = lo + lane * step;
      const bool ok = lane * step < n && clamp_cu(a.cu, min(i, a.nstates), a.total) / WT + i <= slot;
      const int cnt = max(1, (int)__popcll(__ballot(ok)));
      const int end = lo + n;
      lo += (cnt - 1) * step;
      n = min(step, end - lo);
    }
    conv_seq(a, __builtin_amdgcn_readfirstlane(lo), t);
    const int tile = slot - t.s;
    t.lo = max(tile * WT, t.start);
    t.hi = min(tile * WT + WT, t.end);
  } else {
    const int per = (a.seqlen + WT - 1) / WT;
    conv_seq(a, slot / per, t);
    t.lo = t.start + (slot - t.s * per) * WT;
    t.hi = min(t.lo + WT, t.end);
  }
  // the same in every lane already; said so, row addresses stay scalar
  t.s = __builtin_amdgcn_readfirstlane(t.s);
  t.start = __builtin_amdgcn_readfirstlane(t.start);
  t.end = __builtin_amdgcn_readfirstlane(t.end);
  t.lo = __builtin_amdgcn_readfirstlane(t.lo);
  t.hi = __builtin_amdgcn_readfirstlane(t.hi);
  return t;
}

// The channels of a wave: tiles of 64 V channels that never straddle two of the
// three outputs, so every row base is the same in all lanes.  An output whose
// channels are not whole vectors (it has at least V) ends in a vector that
// overlaps the one before it: both compute and store the same values.
struct ConvCols {
  int i, ld;            // output and its channels
  int c;                // this lane's first channel, of all C (some channel if !ok)
  int co;               // the same within the output
  int tile;             // the tile's first channel within the output
  bool ok;              // the lane has channels
};

template <int V>
__host__ __device__ inline int conv_col_tiles(int n) { return (n + 64 * V - 1) / (64 * V); }
template <int V>
int conv_col_tiles(const ConvArgs& a) {
  return conv_col_tiles<V>(a.n[0]) + conv_col_tiles<V>(a.n[1]) + conv_col_tiles<V>(a.n[2]);
}

// First channel of vector v of an output of n channels.
template <int V>
__device__ __forceinline__ int conv_vec(int v, int n) { return min(v * V, n - V); }

template <int V>
__device__ __forceinline__ ConvCols conv_cols(const ConvArgs& a, int ct) {
  ConvCols k;
  const int t0 = conv_col_tiles<V>(a.n[0]), t1 = t0 + conv_col_tiles<V>(a.n[1]);
  k.i = ct < t0 ? 0 : ct < t1 ? 1 : 2;
  k.ld = ct < t0 ? a.n[0] : ct < t1 ? a.n[1] : a.n[2];
  const int first = ct < t0 ? 0 : ct < t1 ? a.n[0] : a.n[0] + a.n[1];
  ct -= ct < t0 ? 0 : ct < t1 ? t0 : t1;
  const int v = ct * 64 + (int)(threadIdx.x & 63);
  k.tile = ct * 64 * V;
  k.ok = v * V < k.ld;
  k.co = conv_vec<V>(v, k.ld);
  k.c = first + k.co;
  return k;
}

template <typename T>
__device__ __forceinline__ T* conv_pick(void* const* p, int i) {
  return static_cast<T*>(i == 0 ? p[0] : i == 1 ? p[1] : p[2]);
}

// Row p of sequence t.s's input, for tokens from K - 1 before the sequence on
// to its last: a token's row or a row of the initial state.  Without an initial
// state a row before the sequence is the tensor's first (some row that exists):
// conv_row_is_zero says so, and the caller clears it after all its loads are
// issued.  The tensor has a token.
template <typename T, int K>
__device__ __forceinline__ const T* conv_row(const ConvArgs& a, const ConvTile& t, int p) {
  const bool before = p < t.start, state = before && a.init;
  const T* base = static_cast<const T*>(state ? a.init : a.x);
  const int64_t row = state ? (int64_t)t.s * (K - 1) + (p - t.start + K - 1) : before ? 0 : p;
  return base + row * (state ? (int64_t)a.C : a.in_stride);
}
__device__ __forceinline__ bool conv_row_is_zero(const ConvArgs& a, const ConvTile& t, int p) {
  return p < t.start && !a.init;
}

// One more token: `win` holds the K rows up to it, oldest first.
template <typename T, int V, int K>
__device__ __forceinline__ void conv_slide(float (&win)[K][V], const Vec<T, V>& q) {
#pragma unroll
  for (int k = 0; k < K - 1; ++k)
#pragma unroll
    for (int e = 0; e < V; ++e) win[k][e] = win[k + 1][e];
  q.get(win[K - 1]);
}

// The K taps and the bias of V channels.
template <int V, int K>
__device__ __forceinline__ void conv_weights(const ConvArgs& a, int c, float (&w)[K][V],
                                             float (&b)[V]) {
#pragma unroll
  for (int e = 0; e < V; ++e) {
#pragma unroll
    for (int k = 0; k < K; ++k) w[k][e] = a.w[(int64_t)(c + e) * K + k];
    b[e] = a.bias ? a.bias[c + e] : 0.f;
  }
}

// The last K - 1 rows of a sequence behind its initial state (copies), by the
// workgroups after the convolution's own: V channels of one state row each.
template <typename T, int V, int K>
__device__ void conv_final_rows(const ConvArgs& a, int64_t i) {
  const int nvec = (a.C + V - 1) / V;
  if (i >= (int64_t)a.nstates * (K - 1) * nvec) return;
  const int c = conv_vec<V>((int)(i % nvec), a.C), r = (int)(i / nvec % (K - 1));
  const int s = (int)(i / nvec / (K - 1));
  ConvTile t;
  conv_seq(a, s, t);
  const int p = t.end - (K - 1) + r;
  Vec<T, V> q;
  if (conv_row_is_zero(a, t, p)) q.clear();
  else q.load(conv_row<T, K>(a, t, p) + c);
  q.store(static_cast<T*>(a.final_states) + ((int64_t)s * (K - 1) + r) * a.C + c);
}

// Zeros in the rows of tokens outside every sequence (before the first entry of
// cu_seqlens and from its last on): vectors i, i + step, ... of n channels of rows `stride`
// apart.
template <typename T, int V>
__device__ void conv_clear_rows(const ConvArgs& a, T* out, int n, int64_t stride, int64_t i,
                                int64_t step) {
  const int lo = clamp_cu(a.cu, 0, a.total), hi = max(lo, clamp_cu(a.cu, a.nstates, a.total));
  const int nvec = (n + V - 1) / V;
  const int64_t items = (int64_t)(lo + a.total - hi) * nvec;
  Vec<T, V> zero;
  zero.clear();
  for (; i < items; i += step) {
    const int64_t r = i / nvec;
    zero.store(out + (r < lo ? r : r - lo + hi) * stride + conv_vec<V>((int)(i - r * nvec), n));
  }
}

// One run of TT tokens from t0 on.  EDGE: its rows may lie before the sequence
// or the run may end early; the inner runs have neither test.
template <typename T, int V, int K, int TT, bool SILU, bool EDGE>
__device__ __forceinline__ void conv_fwd_run(const ConvArgs& a, const ConvTile& t, int t0,
                                             const ConvCols& col, const float (&w)[K][V],
                                             const float (&b)[V]) {
  Vec<T, V> q[TT + K - 1];
  const uint32_t cx = lane_offset((uint32_t)col.c * (uint32_t)sizeof(T));
  uint32_t co = lane_offset((uint32_t)col.co * (uint32_t)sizeof(T));
  const int64_t step = a.in_stride * (int64_t)sizeof(T);
  RowCursor row(static_cast<const T*>(a.x) + (int64_t)(EDGE ? t0 : t0 - (K - 1)) * a.in_stride);
  if constexpr (EDGE) {
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      RowCursor first(conv_row<T, K>(a, t, t0 - (K - 1) + j));
      q[j].load_at(first, cx);
    }
  }
#pragma unroll
  for (int j = EDGE ? K - 1 : 0; j < TT + K - 1; ++j) {
    q[j].load_at(row, cx);
    // past the run's end: its last row again
    row.move(!EDGE || t0 + j - (K - 1) < t.hi - 1 ? step : 0);
  }
  if constexpr (EDGE) {
#pragma unroll
    for (int j = 0; j < K - 1; ++j) q[j].clear_unless(!conv_row_is_zero(a, t, t0 - (K - 1) + j));
  }
  RowCursor out(conv_pick<T>(a.out, col.i) + (int64_t)t0 * col.ld);
  float win[K][V];
#pragma unroll
  for (int j = 0; j < K - 1; ++j) q[j].get(win[j + 1]);
#pragma unroll
  for (int i = 0; i < TT; ++i) {
    if (EDGE && t0 + i >= t.hi) continue;
    if (EDGE) co = lane_offset(co);
    conv_slide<T, V, K>(win, q[i + K - 1]);
    float o[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      float pre = b[e];
#pragma unroll
      for (int k = 0; k < K; ++k) pre += w[k][e] * win[k][e];
      o[e] = SILU ? pre * sigmoid(pre) : pre;
    }
    Vec<T, V> r;
    r.set(o);
    r.store_at(out, co);
    out.move((int64_t)col.ld * (int64_t)sizeof(T));
  }
}

// Workgroups after the nct * nparts of the convolution: nside for the final states,
// the rest for the rows to clear.
template <typename T, int V, int K, int TT, bool SILU>
__global__ __launch_bounds__(kConvThreads) void conv_fwd_kernel(const ConvArgs a, int nct,
                                                                int nslots, int nparts, int nside) {
  constexpr int WT = TT * kConvWaves;
  if ((int)blockIdx.x >= nct * nparts) {
    const int side = (int)blockIdx.x - nct * nparts;
    if (side < nside) {
      conv_final_rows<T, V, K>(a, (int64_t)side * kConvThreads + threadIdx.x);
    } else {
      const int64_t i = (int64_t)(side - nside) * kConvThreads + threadIdx.x;
      const int64_t step = (int64_t)((int)gridDim.x - nct * nparts - nside) * kConvThreads;
#pragma unroll 1
      for (int o = 0; o < 3; ++o) {
        const int n = o == 0 ? a.n[0] : o == 1 ? a.n[1] : a.n[2];
        if (n > 0) conv_clear_rows<T, V>(a, conv_pick<T>(a.out, o), n, n, i, step);
      }
    }
    return;
  }
  const int wv = wave_id();
  const ConvCols col = conv_cols<V>(a, blockIdx.x % nct);
  float w[K][V], b[V];
  conv_weights<V, K>(a, col.c, w, b);
  for (int slot = blockIdx.x / nct; slot < nslots; slot += nparts) {
    const ConvTile t = conv_tile<WT>(a, slot);
    const int t0 = t.lo + wv * TT;
    if (t0 >= t.hi || !col.ok) continue;
    if (t0 - (K - 1) >= t.start && t0 + TT <= t.hi) conv_fwd_run<T, V, K, TT, SILU, false>(a, t, t0, col, w, b);
    else conv_fwd_run<T, V, K, TT, SILU, true>(a, t, t0, col, w, b);
  }
}

// The gradient reaching the initial state, by the workgroups after the
// convolution's own: row r of it is tap k of the sequence's token r - k, and
// row len + i of a sequence shorter than K - 1 is row i of the final state.
template <typename T, int V, int K>
__device__ void conv_dinit_rows(const ConvArgs& a, int64_t i) {
  const int v0 = (a.n[0] + V - 1) / V, v1 = v0 + (a.n[1] + V - 1) / V;
  const int nvec = v1 + (a.n[2] + V - 1) / V;
  if (i >= (int64_t)a.nstates * nvec) return;
  const int s = (int)(i / nvec), v = (int)(i % nvec);
  const int o = v < v0 ? 0 : v < v1 ? 1 : 2;      // output that holds the channels
  const int ld = o == 0 ? a.n[0] : o == 1 ? a.n[1] : a.n[2];
  const int co = conv_vec<V>(v - (o == 0 ? 0 : o == 1 ? v0 : v1), ld);
  const int c = co + (o == 0 ? 0 : o == 1 ? a.n[0] : a.n[0] + a.n[1]);
  const T* dout = conv_pick<const T>(const_cast<void* const*>(a.dout), o) + co;
  ConvTile t;
  conv_seq(a, s, t);
  const int len = t.end - t.start;
  float w[K][V], b[V];
  conv_weights<V, K>(a, c, w, b);
  float acc[K - 1][V];
  Vec<T, V> q[2 * (K - 1)], dq[K - 1], fq[K - 1];
  const int past = max(t.end - 1, 0);             // rows of tokens there are not: any row
  if (a.total > 0) {
#pragma unroll
    for (int j = 0; j < 2 * (K - 1); ++j)
      q[j].load(conv_row<T, K>(a, t, j < K - 1 ? t.start - (K - 1) + j : min(t.start + j - (K - 1), past)) + c);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) dq[j].load(dout + (int64_t)min(t.start + j, past) * ld);
  }
#pragma unroll
  for (int r = 0; r < K - 1; ++r) {
    fq[r].clear();
    if (a.dfinal && r >= len)
      fq[r].load(static_cast<const T*>(a.dfinal) + ((int64_t)s * (K - 1) + r - len) * a.C + c);
  }
#pragma unroll
  for (int j = 0; j < K - 1; ++j) {
    fq[j].get(acc[j]);
    q[j].clear_unless(!conv_row_is_zero(a, t, t.start - (K - 1) + j));
  }
#pragma unroll
  for (int j = 0; j < K - 1; ++j) {
    if (j >= len) continue;
    float d[V], pre[V];
    dq[j].get(d);
#pragma unroll
    for (int e = 0; e < V; ++e) pre[e] = b[e];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float f[V];
      q[j + k].get(f);
#pragma unroll
      for (int e = 0; e < V; ++e) pre[e] += w[k][e] * f[e];
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
      if (a.silu) {
        const float sg = sigmoid(pre[e]);
        d[e] *= sg * (1.f + pre[e] * (1.f - sg));
      }
#pragma unroll
      for (int r = j; r < K - 1; ++r) acc[r][e] += w[r - j][e] * d[e];
    }
  }
#pragma unroll
  for (int r = 0; r < K - 1; ++r) {
    Vec<T, V> q;
    q.set(acc[r]);
    q.store(static_cast<T*>(a.dinit) + ((int64_t)s * (K - 1) + r) * a.C + c);
  }
}

// Backward, one run of TT = STEPS - (K - 1) tokens.  dpre is formed for them and
// the K - 1 tokens after, in order, from a sliding window of K input rows; din
// of a token is complete K - 1 tokens later.  The rows are loaded a group of GR
// tokens ahead of their use, so that the loads of one group are in flight while
// another is computed.  About 30 vector instructions and two transcendental ones (at a
// quarter of the rate) per element and step are 12 + 3 us at 1792 channels x 8192 tokens
// (bf16), where the bytes take 16.3; two channels per thread keep it at three waves per
// SIMD (four channels: 254 registers, 31 against 24 us).  EDGE as in the forward; the
// gradient of the final state reaches edge runs only.
template <typename T, int V, int K, int STEPS, int GR, bool SILU, bool EDGE>
__device__ __forceinline__ void conv_bwd_run(const ConvArgs& a, const ConvTile& t, int t0,
                                             const ConvCols& col, const float (&w)[K][V],
                                             const float (&b)[V], float (&acc)[K + 1][V]) {
  constexpr int TT = STEPS - (K - 1), NG = STEPS / GR;
  static_assert(STEPS % GR == 0, "whole groups");
  const int own = EDGE ? min(TT, t.hi - t0) : TT;     // tokens of this run
  uint32_t co = lane_offset((uint32_t)col.co * (uint32_t)sizeof(T));
  uint32_t cx = lane_offset((uint32_t)col.c * (uint32_t)sizeof(T));
  const T* x = static_cast<const T*>(a.x);
  const int64_t xstep = a.in_stride * (int64_t)sizeof(T), ostep = col.ld * (int64_t)sizeof(T);
  RowCursor xrow(x + (int64_t)(EDGE ? t0 : t0 - (K - 1)) * a.in_stride);
  RowCursor orow(conv_pick<const T>(const_cast<void* const*>(a.dout), col.i) + (int64_t)t0 * col.ld);
  Vec<T, V> h[K - 1], q[2][GR], dq[2][GR], fq[K - 1];
  // row j of the run; past the sequence's end its last row again
  auto load = [&](int j, Vec<T, V>& xv, Vec<T, V>& dv) {
    xv.load_at(xrow, cx);
    dv.load_at(orow, co);
    xrow.move(!EDGE || t0 + j < t.end - 1 ? xstep : 0);
    orow.move(!EDGE || t0 + j < t.end - 1 ? ostep : 0);
  };
#pragma unroll
  for (int j = 0; j < K - 1; ++j) {
    if constexpr (EDGE) {
      RowCursor first(conv_row<T, K>(a, t, t0 - (K - 1) + j));
      h[j].load_at(first, cx);
    } else {
      h[j].load_at(xrow, cx);
      xrow.move(xstep);
    }
  }
#pragma unroll
  for (int u = 0; u < GR; ++u) load(u, q[0][u], dq[0][u]);
  if constexpr (EDGE) {
#pragma unroll
    for (int k = 0; k < K - 1; ++k) {
      // any row that exists where there is no gradient of the final state
      RowCursor df(a.dfinal ? static_cast<const T*>(a.dfinal) + ((int64_t)t.s * (K - 1) + k) * a.C
                            : x + (int64_t)t.start * a.in_stride);
      fq[k].load_at(df, cx);
    }
  }
  RowCursor dx(static_cast<T*>(a.dx) + (int64_t)t0 * a.din_stride);
  float win[K][V], dp[K][V];
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    if (EDGE && g * GR >= own + K - 1) continue;
    if constexpr (EDGE) {                           // a block of its own: see lane_offset
      co = lane_offset(co);
      cx = lane_offset(cx);
    }
    if (g + 1 < NG) {
#pragma unroll
      for (int u = 0; u < GR; ++u) load((g + 1) * GR + u, q[(g + 1) & 1][u], dq[(g + 1) & 1][u]);
    }
    __builtin_amdgcn_sched_barrier(0);
    if (g == 0) {
#pragma unroll
      for (int j = 0; j < K - 1; ++j) {
        if (EDGE) h[j].clear_unless(!conv_row_is_zero(a, t, t0 - (K - 1) + j));
        h[j].get(win[j + 1]);
      }
    }
#pragma unroll
    for (int u = 0; u < GR; ++u) {
      const int j = g * GR + u;
      if (EDGE && j >= own + K - 1) continue;
      conv_slide<T, V, K>(win, q[g & 1][u]);
      conv_slide<T, V, K>(dp, dq[g & 1][u]);
      // past the sequence there is no token: whatever was loaded is dropped
      const bool in = !EDGE || t0 + j < t.end;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        if constexpr (SILU) {
          float pre = b[e];
#pragma unroll
          for (int k = 0; k < K; ++k) pre += w[k][e] * win[k][e];
          const float sg = sigmoid(pre);
          dp[K - 1][e] *= sg * (1.f + pre * (1.f - sg));
        }
        if (EDGE) dp[K - 1][e] = in ? dp[K - 1][e] : 0.f;
      }
      if (j < TT && (!EDGE || j < own)) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
#pragma unroll
          for (int k = 0; k < K; ++k) acc[k][e] += dp[K - 1][e] * win[k][e];
          acc[K][e] += dp[K - 1][e];
        }
      }
      if (j < K - 1) continue;
      float o[V];                                   // din of token t0 + j - (K - 1)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        o[e] = w[K - 1][e] * dp[0][e];
#pragma unroll
        for (int k = 1; k < K; ++k) o[e] += w[K - 1 - k][e] * dp[k][e];
      }
      if constexpr (EDGE) {
        const int f = t0 + j - t.end;               // the final state's row of this token
        if (a.dfinal && f >= 0) {
#pragma unroll
          for (int k = 0; k < K - 1; ++k) {
            float ff[V];
            fq[k].get(ff);
#pragma unroll
            for (int e = 0; e < V; ++e) o[e] += f == k ? ff[e] : 0.f;
          }
        }
      }
      Vec<T, V> r;
      r.set(o);
      if (EDGE) cx = lane_offset(cx);
      r.store_at(dx, cx);
      dx.move(a.din_stride * (int64_t)sizeof(T));
    }
    __builtin_amdgcn_sched_barrier(0);
  }
}

// dw and db accumulate in registers over `seg` of the workgroup's tiles, are added
// over its waves in LDS, and go to one partial row per workgroup, K + 1 sections of
// part_cols(C) columns, to which the next `seg` tiles are added (conv_segment).  SEG:
// there is more than one segment (in the kernel for one, the test alone costs 0.3 of
// the 8 us that a packed batch of 6349 tokens x 160 channels takes).
template <typename T, int V, int K, int STEPS, int GR, bool SILU, bool SEG>
__global__ __launch_bounds__(kConvThreads) void conv_bwd_kernel(const ConvArgs a, int nct,
                                                                int nslots, int nparts, int seg,
                                                                int nside) {
  constexpr int TT = STEPS - (K - 1), WT = TT * kConvWaves;
  __shared__ float red[kConvWaves][K + 1][64 * V];
  if ((int)blockIdx.x >= nct * nparts) {
    const int side = (int)blockIdx.x - nct * nparts;
    if (side < nside)
      conv_dinit_rows<T, V, K>(a, (int64_t)side * kConvThreads + threadIdx.x);
    else
      conv_clear_rows<T, V>(a, static_cast<T*>(a.dx), a.C, a.din_stride,
                            (int64_t)(side - nside) * kConvThreads + threadIdx.x,
                            (int64_t)((int)gridDim.x - nct * nparts - nside) * kConvThreads);
    return;
  }
  const int lane = threadIdx.x & 63, wv = wave_id();
  const int part = blockIdx.x / nct;
  const ConvCols col = conv_cols<V>(a, blockIdx.x % nct);
  float w[K][V], b[V];
  conv_weights<V, K>(a, col.c, w, b);
  for (int s0 = part;;) {                           // a segment; every workgroup has a tile
    float acc[K + 1][V];
#pragma unroll
    for (int k = 0; k <= K; ++k)
#pragma unroll
      for (int e = 0; e < V; ++e) acc[k][e] = 0.f;
    const int s1 = SEG ? min(s0 + seg * nparts, nslots) : nslots;
    for (int slot = s0; slot < s1; slot += nparts) {
      const ConvTile t = conv_tile<WT>(a, slot);
      const int t0 = t.lo + wv * TT;
      if (t0 >= t.hi || !col.ok) continue;
      if (t0 - (K - 1) >= t.start && t0 + TT <= t.hi && t0 + TT + K - 1 <= t.end)
        conv_bwd_run<T, V, K, STEPS, GR, SILU, false>(a, t, t0, col, w, b, acc);
      else
        conv_bwd_run<T, V, K, STEPS, GR, SILU, true>(a, t, t0, col, w, b, acc);
    }
    if (SEG && s0 != part) __syncthreads();         // the segment before has been read
#pragma unroll
    for (int k = 0; k <= K; ++k)
#pragma unroll
      for (int e = 0; e < V; ++e) red[wv][k][lane * V + e] = acc[k][e];
    __syncthreads();
    const int first = __builtin_amdgcn_readfirstlane(col.c - col.co);   // the output's first channel
    const int cp = (int)part_cols(a.C);
    for (int i = threadIdx.x; i < (K + 1) * 64 * V; i += kConvThreads) {
      const int k = i / (64 * V), cc = i % (64 * V), ch = col.tile + cc;
      if (ch >= col.ld) continue;
      // the value's place: its vector's lane, whose vector may start earlier
      const int at = cc / V * V + ch - conv_vec<V>(ch / V, col.ld);
      float s = red[0][k][at];
#pragma unroll
      for (int u = 1; u < kConvWaves; ++u) s += red[u][k][at];
      float* to = part_at(a.part, part, nparts, k * cp + first + ch);
      if (SEG && s0 != part) s += *to;              // the same thread in every segment
      *to = s;
    }
    s0 += seg * nparts;
    if (!SEG || s0 >= nslots) return;
  }
}

// Column c of section k of the partial sums: dweight[c][k], or dbias[c] for k = K.
struct ConvGradOut {
  float *dw, *db;
  int C, cp, K;
  __device__ __forceinline__ void put(int col, float v) const {
    const int k = col / cp, c = col - k * cp;
    if (c >= C) return;
    if (k < K) dw[(int64_t)c * K + k] = v;
    else if (db) db[c] = v;
  }
};

// One token per sequence: a thread owns V channels of one row and of its
// slot's state, so the shift in place needs no exchange.
template <typename T, int V, int K>
__global__ __launch_bounds__(kConvThreads) void conv_step_kernel(const ConvArgs a, int nblk) {
  const int row = blockIdx.x / nblk, v = (int)(blockIdx.x % nblk) * (int)blockDim.x + threadIdx.x;
  StepSlot slot;
  if (!slot.begin(a.slots, row, a.nslots)) return;
  const int c = min(v, a.C / V - 1) * V;
  T* st = static_cast<T*>(a.states) + (int64_t)slot.mine * (K - 1) * a.C + c;
  Vec<T, V> q[K];
#pragma unroll
  for (int k = 0; k < K - 1; ++k) q[k].load(st + (int64_t)k * a.C);
  q[K - 1].load(static_cast<const T*>(a.x) + row * a.in_stride + c);
  float w[K][V], o[V];
  conv_weights<V, K>(a, c, w, o);
  if (slot.repeated() || v >= a.C / V) return;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    float f[V];
    q[k].get(f);
#pragma unroll
    for (int e = 0; e < V; ++e) o[e] += w[k][e] * f[e];
  }
  if (a.silu) {
#pragma unroll
    for (int e = 0; e < V; ++e) o[e] *= sigmoid(o[e]);
  }
#pragma unroll
  for (int k = 0; k < K - 1; ++k) q[k + 1].store(st + (int64_t)k * a.C);
  const int i = c < a.n[0] ? 0 : c < a.n[0] + a.n[1] ? 1 : 2;
  const int ld = i == 0 ? a.n[0] : i == 1 ? a.n[1] : a.n[2];
  Vec<T, V> r;
  r.set(o);
  r.store(conv_pick<T>(a.out, i) + (int64_t)row * ld + c - (i == 0 ? 0 : i == 1 ? a.n[0] : a.n[0] + a.n[1]));
}

constexpr int kConvFwdLong = 16, kConvFwdShort = 4;     // tokens per run, forward
constexpr int kConvBwdLong = 64, kConvBwdShort = 16;    // steps per run, backward
constexpr int kConvBwdMaxParts = 256;
constexpr int kConvStepThreads = 128;
constexpr int64_t kConvMaxGroups = 1 << 21;   // workgroups of one launch

// Token groups of a launch: one per slot while the launch stays within
// `most` workgroups, each walking several slots beyond that.
int conv_parts(int nslots, int nct, int64_t most) {
  const int64_t p = most / nct;
  return (int)(nslots < p ? nslots : (p > 0 ? p : 1));
}

// Workgroups for the rows to clear, which only the device can count: one per 16 tokens
// up to one per CU, idle where there are none.
int conv_clear_groups(const ConvArgs& a) {
  if (!a.clear || !a.cu || a.total == 0) return 0;
  return a.total < 16 * 256 ? (a.total + 15) / 16 : 256;
}

// Tiles of a workgroup whose terms of dw and db one register adds before they go to
// the partial row: 256 tokens' worth, and the square root of the tokens a wave has
// where that is more, so that a term passes at most about 256 + tokens / 256 or
// 2 sqrt(tokens) additions there, not one per token.  (One register over all tiles: a sum
// of 2^23 equal terms per channel, 8192 a wave, was off by 1354 2^-24 of its value,
// with segments by 63; 2^20 tokens x 160 channels of fp32 512 and 520 us.)
int conv_segment(int nslots, int nparts, int TT) {
  const int runs = nparts > 0 ? (nslots + nparts - 1) / nparts : 0;
  int seg = (256 + TT - 1) / TT;
  while ((int64_t)seg * seg * TT < runs) ++seg;
  return seg;
}

template <typename T, int V, int K, int TT>
hipError_t conv_fwd_go(const ConvArgs& a, hipStream_t s) {
  const int nct = conv_col_tiles<V>(a);
  const int nslots = conv_slots(a, TT * kConvWaves);
  const int nparts = a.total > 0 ? conv_parts(nslots, nct, kConvMaxGroups) : 0;
  const int64_t fin = a.final_states ? (int64_t)a.nstates * (K - 1) * ((a.C + V - 1) / V) : 0;
  const int64_t nside = (fin + kConvThreads - 1) / kConvThreads;
  const int64_t grid = (int64_t)nct * nparts + nside + conv_clear_groups(a);
  if (grid == 0) return hipSuccess;
  auto fn = a.silu ? &conv_fwd_kernel<T, V, K, TT, true> : &conv_fwd_kernel<T, V, K, TT, false>;
  hipLaunchKernelGGL(fn, dim3((unsigned)grid), dim3(kConvThreads), 0, s, a, nct, nslots, nparts,
                     (int)nside);
  return hipGetLastError();
}

template <typename T, int V, int K, int STEPS>
hipError_t conv_bwd_go(const ConvArgs& a, hipStream_t s) {
  const int nct = conv_col_tiles<V>(a);
  const int nslots = conv_slots(a, (STEPS - (K - 1)) * kConvWaves);
  const int nparts = a.total > 0 ? conv_parts(nslots, 1, kConvBwdMaxParts) : 0;
  const int64_t ini = a.dinit ? (int64_t)a.nstates * ((a.C + 2) / V + 3) : 0;
  const int64_t nside = (ini + kConvThreads - 1) / kConvThreads;
  const int64_t grid = (int64_t)nct * nparts + nside + conv_clear_groups(a);
  const int seg = conv_segment(nslots, nparts, STEPS - (K - 1));
  const bool many = (int64_t)seg * nparts < nslots;
  auto fn = many ? (a.silu ? &conv_bwd_kernel<T, V, K, STEPS, 8, true, true>
                           : &conv_bwd_kernel<T, V, K, STEPS, 8, false, true>)
                 : (a.silu ? &conv_bwd_kernel<T, V, K, STEPS, 8, true, false>
                           : &conv_bwd_kernel<T, V, K, STEPS, 8, false, false>);
  if (grid > 0)
    hipLaunchKernelGGL(fn, dim3((unsigned)grid), dim3(kConvThreads), 0, s, a, nct, nslots, nparts, seg,
                       (int)nside);
  const int64_t cp = part_cols(a.C);
  return colsum(a.part, nparts, (K + 1) * cp, ConvGradOut{a.dw, a.dbias, a.C, (int)cp, K}, s);
}

template <typename T, int V, int K>
hipError_t conv_step_go(const ConvArgs& a, hipStream_t s) {
  const int nblk = (a.C / V + kConvStepThreads - 1) / kConvStepThreads;
  hipLaunchKernelGGL((conv_step_kernel<T, V, K>), dim3((unsigned)(a.batch * nblk)),
                     dim3(kConvStepThreads), 0, s, a, nblk);
  return hipGetLastError();
}

// Every output has a whole vector of V channels (or none).
bool conv_has(const ConvArgs& a, int V) {
  return a.n[0] >= V && (a.n[1] >= V || a.n[1] == 0) && (a.n[2] >= V || a.n[2] == 0);
}

// Long runs read fewer rows twice but leave few waves on a small problem, where
// one run's latency is the launch's.  Measured (us, long / short runs):
//   forward   1792 ch bf16: 256 tokens 5.0 / 3.0, 4096 8.8 / 8.1, 8192 13.2 / 12.9;
//             6144 ch bf16: 4096 tokens 24.4 / 25.3, 32768 149 / 166
//   backward  1792 ch bf16: 256 tokens 17.4 / 8.2, 4096 19.7 / 18.1, 8192 23.6 / 29.2;
//             6144 ch bf16: 2048 tokens 20.6 / 22.9; 256 ch: 32768 tokens 19.0 / 17.4
//             6144 ch fp32: 8192 tokens 127 / 119 (never long)
// so the forward takes them from 2^24 elements on, the backward from 10 2^20
// (bf16).  Two channels per thread in the short runs, again for more waves.
bool conv_long(const ConvArgs& a, int64_t from) { return (int64_t)a.total * a.C >= from; }

template <typename T, int K>
hipError_t conv_fwd_k(const ConvArgs& a, hipStream_t s) {
  if (conv_long(a, (int64_t)1 << 24) && conv_has(a, 4)) return conv_fwd_go<T, 4, K, kConvFwdLong>(a, s);
  if (conv_has(a, 2)) return conv_fwd_go<T, 2, K, kConvFwdShort>(a, s);
  return conv_fwd_go<T, 1, K, kConvFwdShort>(a, s);
}

template <typename T, int K>
hipError_t conv_bwd_k(const ConvArgs& a, hipStream_t s) {
  if constexpr (sizeof(T) == 2) {
    if (conv_long(a, (int64_t)10 << 20) && conv_has(a, 2)) return conv_bwd_go<T, 2, K, kConvBwdLong>(a, s);
  }
  if (conv_has(a, 2)) return conv_bwd_go<T, 2, K, kConvBwdShort>(a, s);
  return conv_bwd_go<T, 1, K, kConvBwdShort>(a, s);
}

// In place, so no two threads may share a channel: whole vectors only.
template <typename T, int K>
hipError_t conv_step_k(const ConvArgs& a, hipStream_t s) {
  const bool whole = a.n[0] % 2 == 0 && a.n[1] % 2 == 0 && a.n[2] % 2 == 0;
  return whole ? conv_step_go<T, 2, K>(a, s) : conv_step_go<T, 1, K>(a, s);
}

#define SSD_CONV_K(OP, T)                        \
  switch (a.K) {                                 \
    case 2: return conv_##OP##_k<T, 2>(a, s);    \
    case 3: return conv_##OP##_k<T, 3>(a, s);    \
    case 4: return conv_##OP##_k<T, 4>(a, s);    \
  }                                              \
  return hipErrorInvalidValue

}  // namespace

// As many partial rows as the launch with the shortest runs has.
int64_t conv_bwd_floats(int64_t tokens, int64_t nstates, int64_t C, int64_t K) {
  const int64_t wt = (kConvBwdShort - (K - 1)) * kConvWaves;
  const int64_t slots = (tokens + wt - 1) / wt + nstates;
  return (slots < kConvBwdMaxParts ? slots : kConvBwdMaxParts) * (K + 1) * part_cols(C);
}

hipError_t launch_conv_fwd(const ConvArgs& a, hipStream_t s) {
  if (a.bf16) { SSD_CONV_K(fwd, bf16); }
  SSD_CONV_K(fwd, float);
}
hipError_t launch_conv_bwd(const ConvArgs& a, hipStream_t s) {
  if (a.bf16) { SSD_CONV_K(bwd, bf16); }
  SSD_CONV_K(bwd, float);
}
hipError_t launch_conv_step(const ConvArgs& a, hipStream_t s) {
  if (a.batch <= 0) return hipSuccess;
  if (a.bf16) { SSD_CONV_K(step, bf16); }
  SSD_CONV_K(step, float);
}
#undef SSD_CONV_K

}  // namespace ssd

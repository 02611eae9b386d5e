// The short causal convolution over the channels x | B | C, its backward and
// its single-token form.  Per sequence, token t and channel c:
//   pre[t] = bias + sum_k w[k] in[t - (K-1) + k],   out = pre sigma(pre) or pre
//   dpre[t] = dout[t] act'(pre[t])
//   din[t] = sum_j w[K-1-j] dpre[t+j],  dw[k] = sum_t dpre[t] in[t - (K-1) + k]
//
// What bounds it: memory.  A forward reads and writes every element once for
// about 2 K + 10 operations, a backward reads two and writes one.  So a thread
// owns V neighbouring channels (16 bytes where the channel counts allow) and a
// run of TT tokens, a wave 64 such vectors of one run, and a workgroup four
// runs in a row.  All rows of a run, the K - 1 before it included, are loaded
// at once into registers and each element is read from memory once; the rows
// that two runs share come from the L1 and L2.
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
  return t;
}

// Pointer to channel c of token 0 in the output (or its gradient) that holds
// the channel, and that output's channels.
template <typename T>
__device__ __forceinline__ T* conv_split(const ConvArgs& a, void* const* out, int c, int& ld) {
  if (c < a.n[0]) {
    ld = a.n[0];
    return static_cast<T*>(out[0]) + c;
  }
  c -= a.n[0];
  if (c < a.n[1]) {
    ld = a.n[1];
    return static_cast<T*>(out[1]) + c;
  }
  ld = a.n[2];
  return static_cast<T*>(out[2]) + (c - a.n[1]);
}

// Row p of sequence t.s's input, for tokens from K - 1 before the sequence on
// to its last: a token's row, a row of the initial state, or zeros.  The
// sequence has a token.
template <typename T, int V, int K>
__device__ __forceinline__ Vec<T, V> conv_row(const ConvArgs& a, const ConvTile& t, int p, int c) {
  Vec<T, V> q;
  const bool before = p < t.start;
  const T* row = static_cast<const T*>(a.x) + (int64_t)p * a.in_stride;
  if (before) {
    // without an initial state: the sequence's first row, then cleared
    row = a.init ? static_cast<const T*>(a.init) + ((int64_t)t.s * (K - 1) + (p - t.start + K - 1)) * a.C
                 : static_cast<const T*>(a.x) + (int64_t)t.start * a.in_stride;
  }
  q.load(row + c);
  q.clear_unless(!before || a.init);
  return q;
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
  const int nvec = a.C / V;
  if (i >= (int64_t)a.nstates * (K - 1) * nvec) return;
  const int c = (int)(i % nvec) * V, r = (int)(i / nvec % (K - 1)), s = (int)(i / nvec / (K - 1));
  ConvTile t;
  conv_seq(a, s, t);
  const int p = t.end - (K - 1) + r;
  Vec<T, V> q;
  if (p < t.start && !a.init) q.clear();
  else q = conv_row<T, V, K>(a, t, p, c);
  q.store(static_cast<T*>(a.final_states) + ((int64_t)s * (K - 1) + r) * a.C + c);
}

template <typename T, int V, int K, int TT>
__global__ __launch_bounds__(kConvThreads) void conv_fwd_kernel(const ConvArgs a, int nct,
                                                                int nslots, int nparts) {
  constexpr int WT = TT * kConvWaves;
  if ((int)blockIdx.x >= nct * nparts) {
    conv_final_rows<T, V, K>(a, (int64_t)((int)blockIdx.x - nct * nparts) * kConvThreads + threadIdx.x);
    return;
  }
  const int lane = threadIdx.x & 63, wv = wave_id();
  const int nvec = a.C / V, v = (int)(blockIdx.x % nct) * 64 + lane;
  const int c = min(v, nvec - 1) * V;
  float w[K][V], b[V];
  conv_weights<V, K>(a, c, w, b);
  int ld;
  T* out = conv_split<T>(a, a.out, c, ld);
  for (int slot = blockIdx.x / nct; slot < nslots; slot += nparts) {
    const ConvTile t = conv_tile<WT>(a, slot);
    const int t0 = t.lo + wv * TT;
    if (t0 >= t.hi) continue;
    Vec<T, V> q[TT + K - 1];
#pragma unroll
    for (int j = 0; j < TT + K - 1; ++j)
      q[j] = conv_row<T, V, K>(a, t, min(t0 - (K - 1) + j, t.hi - 1), c);
    float win[K][V];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) q[j].get(win[j + 1]);
#pragma unroll
    for (int i = 0; i < TT; ++i) {
#pragma unroll
      for (int k = 0; k < K - 1; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e) win[k][e] = win[k + 1][e];
      q[i + K - 1].get(win[K - 1]);
      float o[V];
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float pre = b[e];
#pragma unroll
        for (int k = 0; k < K; ++k) pre += w[k][e] * win[k][e];
        o[e] = a.silu ? pre * sigmoid<T>(pre) : pre;
      }
      Vec<T, V> r;
      r.set(o);
      if (t0 + i < t.hi && v < nvec) r.store(out + (int64_t)(t0 + i) * ld);
    }
  }
}

// The gradient reaching the initial state, by the workgroups after the
// convolution's own: row r of it is tap k of the sequence's token r - k, and
// row len + i of a sequence shorter than K - 1 is row i of the final state.
template <typename T, int V, int K>
__device__ void conv_dinit_rows(const ConvArgs& a, int64_t i) {
  const int nvec = a.C / V;
  if (i >= (int64_t)a.nstates * nvec) return;
  const int c = (int)(i % nvec) * V, s = (int)(i / nvec);
  ConvTile t;
  conv_seq(a, s, t);
  const int len = t.end - t.start;
  float w[K][V], b[V];
  conv_weights<V, K>(a, c, w, b);
  int ld;
  const T* dout = conv_split<const T>(a, const_cast<void* const*>(a.dout), c, ld);
  float acc[K - 1][V];
#pragma unroll
  for (int r = 0; r < K - 1; ++r) {
#pragma unroll
    for (int e = 0; e < V; ++e) acc[r][e] = 0.f;
    if (a.dfinal && r >= len) {
      Vec<T, V> q;
      q.load(static_cast<const T*>(a.dfinal) + ((int64_t)s * (K - 1) + r - len) * a.C + c);
      q.get(acc[r]);
    }
  }
#pragma unroll
  for (int j = 0; j < K - 1; ++j) {
    if (j >= len) continue;
    float d[V], pre[V];
    Vec<T, V> q;
    q.load(dout + (int64_t)(t.start + j) * ld);
    q.get(d);
#pragma unroll
    for (int e = 0; e < V; ++e) pre[e] = b[e];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float f[V];
      conv_row<T, V, K>(a, t, t.start + j - (K - 1) + k, c).get(f);
#pragma unroll
      for (int e = 0; e < V; ++e) pre[e] += w[k][e] * f[e];
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
      if (a.silu) {
        const float sg = sigmoid<T>(pre[e]);
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

// Backward.  A run's dpre is formed for its TT tokens and the K - 1 after
// them, in order, from a sliding window of K input rows; din of a token is
// complete K - 1 tokens later.  dw and db accumulate in registers over the
// workgroup's tiles, are added over its waves in LDS at the end, and leave
// as one partial row per workgroup, [part][K + 1][C].
template <typename T, int V, int K, int TT>
__global__ __launch_bounds__(kConvThreads) void conv_bwd_kernel(const ConvArgs a, int nct,
                                                                int nslots, int nparts) {
  constexpr int WT = TT * kConvWaves;
  __shared__ float red[kConvWaves][K + 1][64 * V];
  if ((int)blockIdx.x >= nct * nparts) {
    conv_dinit_rows<T, V, K>(a, (int64_t)((int)blockIdx.x - nct * nparts) * kConvThreads + threadIdx.x);
    return;
  }
  const int lane = threadIdx.x & 63, wv = wave_id();
  const int ct = blockIdx.x % nct, part = blockIdx.x / nct;
  const int nvec = a.C / V, v = ct * 64 + lane;
  const int c = min(v, nvec - 1) * V;
  float w[K][V], b[V];
  conv_weights<V, K>(a, c, w, b);
  int ld;
  const T* dout = conv_split<const T>(a, const_cast<void* const*>(a.dout), c, ld);
  float acc[K + 1][V];
#pragma unroll
  for (int k = 0; k <= K; ++k)
#pragma unroll
    for (int e = 0; e < V; ++e) acc[k][e] = 0.f;
  for (int slot = part; slot < nslots; slot += nparts) {
    const ConvTile t = conv_tile<WT>(a, slot);
    const int t0 = t.lo + wv * TT;
    if (t0 >= t.hi) continue;
    const int own = min(TT, t.hi - t0);           // tokens of this run
    Vec<T, V> q[TT + 2 * (K - 1)], dq[TT + K - 1];
#pragma unroll
    for (int j = 0; j < TT + 2 * (K - 1); ++j)
      q[j] = conv_row<T, V, K>(a, t, min(t0 - (K - 1) + j, t.end - 1), c);
#pragma unroll
    for (int j = 0; j < TT + K - 1; ++j) dq[j].load(dout + (int64_t)min(t0 + j, t.end - 1) * ld);
    float win[K][V], dp[K][V];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) q[j].get(win[j + 1]);
#pragma unroll
    for (int j = 0; j < TT + K - 1; ++j) {
#pragma unroll
      for (int k = 0; k < K - 1; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e) {
          win[k][e] = win[k + 1][e];
          dp[k][e] = dp[k + 1][e];
        }
      q[j + K - 1].get(win[K - 1]);
      dq[j].get(dp[K - 1]);
      const bool in = t0 + j < t.end;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        if (a.silu) {
          float pre = b[e];
#pragma unroll
          for (int k = 0; k < K; ++k) pre += w[k][e] * win[k][e];
          const float sg = sigmoid<T>(pre);
          dp[K - 1][e] *= sg * (1.f + pre * (1.f - sg));
        }
        // past the sequence there is no token: whatever was loaded is dropped
        dp[K - 1][e] = in ? dp[K - 1][e] : 0.f;
      }
      if (j < own) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
#pragma unroll
          for (int k = 0; k < K; ++k) acc[k][e] += dp[K - 1][e] * win[k][e];
          acc[K][e] += dp[K - 1][e];
        }
      }
      const int i = j - (K - 1);                  // the token whose gradient is complete
      if (i >= 0 && i < own) {
        float o[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
          o[e] = 0.f;
#pragma unroll
          for (int k = 0; k < K; ++k) o[e] += w[K - 1 - k][e] * dp[k][e];
        }
        const int f = t0 + i - (t.end - (K - 1));
        if (a.dfinal && f >= 0) {
          Vec<T, V> df;
          float ff[V];
          df.load(static_cast<const T*>(a.dfinal) + ((int64_t)t.s * (K - 1) + f) * a.C + c);
          df.get(ff);
#pragma unroll
          for (int e = 0; e < V; ++e) o[e] += ff[e];
        }
        Vec<T, V> r;
        r.set(o);
        if (v < nvec) r.store(static_cast<T*>(a.dx) + (int64_t)(t0 + i) * a.din_stride + c);
      }
    }
  }
#pragma unroll
  for (int k = 0; k <= K; ++k)
#pragma unroll
    for (int e = 0; e < V; ++e) red[wv][k][lane * V + e] = acc[k][e];
  __syncthreads();
  for (int i = threadIdx.x; i < (K + 1) * 64 * V; i += kConvThreads) {
    const int k = i / (64 * V), cc = i % (64 * V), ch = ct * 64 * V + cc;
    if (ch >= a.C) continue;
    float t = red[0][k][cc];
#pragma unroll
    for (int u = 1; u < kConvWaves; ++u) t += red[u][k][cc];
    a.part[((int64_t)part * (K + 1) + k) * a.C + ch] = t;
  }
}

// Column k C + c of the partial sums: dweight[c][k], or dbias[c] for k = K.
struct ConvGradOut {
  float *dw, *db;
  int C, K;
  __device__ __forceinline__ void put(int col, float v) const {
    const int k = col / C, c = col - k * C;
    if (k < K) dw[(int64_t)c * K + k] = v;
    else if (db) db[c] = v;
  }
};

// One token per sequence: a thread owns V channels of one row and of its
// slot's state, so the shift in place needs no exchange.
template <typename T, int V, int K>
__global__ __launch_bounds__(kConvThreads) void conv_step_kernel(const ConvArgs a, int nblk) {
  const int row = blockIdx.x / nblk, v = (int)(blockIdx.x % nblk) * kConvThreads + threadIdx.x;
  int64_t slot;
  if (step_row_is_padding(a.slots, row, a.nslots, slot)) return;
  if (v >= a.C / V) return;
  const int c = v * V;
  T* st = static_cast<T*>(a.states) + slot * (K - 1) * a.C + c;
  Vec<T, V> q[K];
#pragma unroll
  for (int k = 0; k < K - 1; ++k) q[k].load(st + (int64_t)k * a.C);
  q[K - 1].load(static_cast<const T*>(a.x) + row * a.in_stride + c);
  float w[K][V], o[V];
  conv_weights<V, K>(a, c, w, o);
#pragma unroll
  for (int k = 0; k < K; ++k) {
    float f[V];
    q[k].get(f);
#pragma unroll
    for (int e = 0; e < V; ++e) o[e] += w[k][e] * f[e];
  }
  if (a.silu) {
#pragma unroll
    for (int e = 0; e < V; ++e) o[e] *= sigmoid<T>(o[e]);
  }
#pragma unroll
  for (int k = 0; k < K - 1; ++k) q[k + 1].store(st + (int64_t)k * a.C);
  int ld;
  T* out = conv_split<T>(a, a.out, c, ld);
  Vec<T, V> r;
  r.set(o);
  r.store(out + (int64_t)row * ld);
}

constexpr int kConvFwdTT = 16, kConvBwdTT = 8;
constexpr int kConvBwdMaxParts = 256;
constexpr int64_t kConvMaxGroups = 1 << 22;   // workgroups of one launch

// Token groups of a launch: one per slot while the launch stays within
// `most` workgroups, each walking several slots beyond that.
int conv_parts(int nslots, int nct, int64_t most) {
  const int64_t p = most / nct;
  return (int)(nslots < p ? nslots : (p > 0 ? p : 1));
}

template <typename T, int V, int K>
hipError_t conv_fwd_go(const ConvArgs& a, hipStream_t s) {
  const int nct = (a.C / V + 63) / 64;
  const int nslots = conv_slots(a, kConvFwdTT * kConvWaves);
  const int nparts = a.total > 0 ? conv_parts(nslots, nct, kConvMaxGroups) : 0;
  const int64_t fin = a.final_states ? (int64_t)a.nstates * (K - 1) * (a.C / V) : 0;
  const int64_t grid = (int64_t)nct * nparts + (fin + kConvThreads - 1) / kConvThreads;
  if (grid == 0) return hipSuccess;
  hipLaunchKernelGGL((conv_fwd_kernel<T, V, K, kConvFwdTT>), dim3((unsigned)grid),
                     dim3(kConvThreads), 0, s, a, nct, nslots, nparts);
  return hipGetLastError();
}

template <typename T, int V, int K>
hipError_t conv_bwd_go(const ConvArgs& a, hipStream_t s) {
  const int nct = (a.C / V + 63) / 64;
  const int nslots = conv_slots(a, kConvBwdTT * kConvWaves);
  const int nparts = a.total > 0 ? conv_parts(nslots, 1, kConvBwdMaxParts) : 0;
  const int64_t ini = a.dinit ? (int64_t)a.nstates * (a.C / V) : 0;
  const int64_t grid = (int64_t)nct * nparts + (ini + kConvThreads - 1) / kConvThreads;
  if (grid > 0)
    hipLaunchKernelGGL((conv_bwd_kernel<T, V, K, kConvBwdTT>), dim3((unsigned)grid),
                       dim3(kConvThreads), 0, s, a, nct, nslots, nparts);
  const int cols = (K + 1) * a.C;
  hipLaunchKernelGGL(colsum_kernel<ConvGradOut>, dim3((cols + 63) / 64), dim3(kColsumThreads), 0, s,
                     (const float*)a.part, nparts, cols, (ConvGradOut{a.dw, a.dbias, a.C, K}));
  return hipGetLastError();
}

template <typename T, int V, int K>
hipError_t conv_step_go(const ConvArgs& a, hipStream_t s) {
  const int nblk = (a.C / V + kConvThreads - 1) / kConvThreads;
  hipLaunchKernelGGL((conv_step_kernel<T, V, K>), dim3((unsigned)(a.batch * nblk)),
                     dim3(kConvThreads), 0, s, a, nblk);
  return hipGetLastError();
}

enum ConvOp { kFwd, kBwd, kStep };

template <int OP, typename T, int V, int K>
hipError_t conv_go(const ConvArgs& a, hipStream_t s) {
  if constexpr (OP == kFwd) return conv_fwd_go<T, V, K>(a, s);
  else if constexpr (OP == kBwd) return conv_bwd_go<T, V, K>(a, s);
  else return conv_step_go<T, V, K>(a, s);
}

template <int OP, typename T, int V>
hipError_t conv_width(const ConvArgs& a, hipStream_t s) {
  switch (a.K) {
    case 2: return conv_go<OP, T, V, 2>(a, s);
    case 3: return conv_go<OP, T, V, 3>(a, s);
    case 4: return conv_go<OP, T, V, 4>(a, s);
  }
  return hipErrorInvalidValue;
}

// 16-byte vectors where every output's channels are whole vectors, else one
// channel per thread.
template <int OP>
hipError_t conv_dispatch(const ConvArgs& a, hipStream_t s) {
  const int m = a.bf16 ? 8 : 4;
  const bool vec = a.n[0] % m == 0 && a.n[1] % m == 0 && a.n[2] % m == 0;
  if (a.bf16) return vec ? conv_width<OP, bf16, 8>(a, s) : conv_width<OP, bf16, 1>(a, s);
  return vec ? conv_width<OP, float, 4>(a, s) : conv_width<OP, float, 1>(a, s);
}

}  // namespace

int64_t conv_bwd_floats(int64_t tokens, int64_t nstates, int64_t C, int64_t K) {
  const int64_t slots = (tokens + kConvBwdTT * kConvWaves - 1) / (kConvBwdTT * kConvWaves) + nstates;
  return (slots < kConvBwdMaxParts ? slots : kConvBwdMaxParts) * (K + 1) * C;
}

hipError_t launch_conv_fwd(const ConvArgs& a, hipStream_t s) { return conv_dispatch<kFwd>(a, s); }
hipError_t launch_conv_bwd(const ConvArgs& a, hipStream_t s) { return conv_dispatch<kBwd>(a, s); }
hipError_t launch_conv_step(const ConvArgs& a, hipStream_t s) {
  if (a.batch <= 0) return hipSuccess;
  return conv_dispatch<kStep>(a, s);
}

}  // namespace ssd

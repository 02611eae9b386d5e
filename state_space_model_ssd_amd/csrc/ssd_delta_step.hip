// The gated delta rule for one new token per sequence: the recurrence's single update, in
// place on a cache of fp32 states.
//   w = beta (v - a S k),   S <- a S + w k^T,   o = scale S q = scale (a S_old q + w (k.q))
//
// What bounds it: the state, read and written once (8 P N H bytes a row); everything else
// is under two percent.  A row of a head's state lies over LPR lanes as in ssd_step.hip,
// four values a lane.  Both products with the old row, and k.q, are summed side by side in
// one butterfly, so the output waits for no second one.  256 rows of 300 slots, 32 heads of
// 128 x 128: 196 us, 5.4 TB/s; one row 4.1 us.
#include "ssd_delta.h"
#include "ssd_layer_device.h"
#include "ssd_rowsum.h"
#include "ssd_step_rule.h"

#pragma clang fp contract(on)

namespace ssd {

namespace {

constexpr int kStepThreads = 256;

// V: values per access (4, or 1 for N < 4); R: rows per thread.
template <typename T, typename GT, int V, int R>
__global__ __launch_bounds__(kStepThreads) void delta_step_kernel(const DeltaStepArgs a, int lpr, int nblk) {
  const int blk = blockIdx.x % nblk;              // block of rows of the head's state
  const int hb = blockIdx.x / nblk;
  const int h = hb % a.H, b = hb / a.H;
  const int g = h / (a.H / a.G);
  StepSlot slot;
  if (!slot.begin(a.slots, b, a.nslots)) return;
  const int ln = threadIdx.x & (lpr - 1);         // lane within the row
  const int rows = blockDim.x / lpr;              // rows per pass
  const int p0 = blk * rows * R + threadIdx.x / lpr;
  const bool in = ln * V < a.N;
  // the lane's first value: where N is no multiple of four, a row's last vector starts
  // early enough to end with the row, and its first values are the lane before's too
  const int n = min(ln * V, a.N - V);
  float* st = a.states + ((int64_t)slot.mine * a.H + h) * a.P * a.N + n;

  Vec<float, V> s[R];
#pragma unroll
  for (int r = 0; r < R; ++r) s[r].load(st + (int64_t)min(p0 + r * rows, a.P - 1) * a.N);
  Vec<T, V> qv, kv;
  qv.load(static_cast<const T*>(a.q) + b * a.q_stride + (int64_t)g * a.N + n);
  kv.load(static_cast<const T*>(a.k) + b * a.k_stride + (int64_t)g * a.N + n);
  const T* v = static_cast<const T*>(a.v) + b * a.v_stride + (int64_t)h * a.P;
  float vv[R];
#pragma unroll
  for (int r = 0; r < R; ++r) vv[r] = to_f32(v[min(p0 + r * rows, a.P - 1)]);
  const float decay = expf(to_f32(static_cast<const GT*>(a.g)[b * a.g_stride + h]));
  const float beta = to_f32(static_cast<const GT*>(a.beta)[b * a.beta_stride + h]);
  T* out = static_cast<T*>(a.out) + ((int64_t)b * a.H + h) * a.P;
  if (slot.repeated()) return;
  float q[V], k[V], kq = 0.f;
  qv.get(q);
  kv.get(k);
  bool mine[V];                                   // not the lane before's, nor past the row's end
#pragma unroll
  for (int e = 0; e < V; ++e) {
    mine[e] = n + e >= ln * V && in;
    kq += mine[e] ? k[e] * q[e] : 0.f;
  }
  kq = run_sum_dpp(kq, lpr);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int p = p0 + r * rows;
    float f[V], sk = 0.f, sq = 0.f;
    s[r].get(f);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      f[e] *= decay;
      sk += mine[e] ? f[e] * k[e] : 0.f;
      sq += mine[e] ? f[e] * q[e] : 0.f;
    }
    sk = run_sum_dpp(sk, lpr);
    sq = run_sum_dpp(sq, lpr);
    const float w = beta * (vv[r] - sk);
#pragma unroll
    for (int e = 0; e < V; ++e) f[e] += w * k[e];
    s[r].set(f);
    if (p < a.P && in) s[r].store(st + (int64_t)p * a.N);
    if (ln == 0 && p < a.P) out[p] = from_f32<T>(a.scale * (sq + w * kq));
  }
}

template <typename T, typename GT, int V, int R>
hipError_t step_go(const DeltaStepArgs& a, int lpr, hipStream_t s) {
  // one wave where a head's rows fill no more
  int threads = kStepThreads;
  while (threads > 64 && threads / 2 * R >= a.P * lpr) threads /= 2;
  const int rows = threads / lpr * R;
  const int nblk = (a.P + rows - 1) / rows;
  hipLaunchKernelGGL((delta_step_kernel<T, GT, V, R>), dim3((unsigned)(a.batch * (int64_t)a.H * nblk)),
                     dim3(threads), 0, s, a, lpr, nblk);
  return hipGetLastError();
}

template <typename T, typename GT>
hipError_t step_type(const DeltaStepArgs& a, hipStream_t s) {
  const int lpr = step_lpr(a.N);
  if (a.N < 4) return step_go<T, GT, 1, 1>(a, lpr, s);
  switch (step_rows(a.batch, a.H, a.P, a.N)) {
    case 4: return step_go<T, GT, 4, 4>(a, lpr, s);
    case 2: return step_go<T, GT, 4, 2>(a, lpr, s);
  }
  return step_go<T, GT, 4, 1>(a, lpr, s);
}

}  // namespace

hipError_t launch_delta_step(const DeltaStepArgs& a, hipStream_t s) {
  if (a.batch <= 0) return hipSuccess;
  if (!a.bf16) return step_type<float, float>(a, s);
  return a.gate_bf16 ? step_type<bf16, bf16>(a, s) : step_type<bf16, float>(a, s);
}

}  // namespace ssd

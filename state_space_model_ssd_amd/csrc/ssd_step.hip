// The SSD for one new token per sequence: the recurrence's single update, in
// place on a cache of fp32 states.
//   delta = clamp(softplus(dt + dt_bias)),  a = exp(delta A)
//   h[p,n] = a h[p,n] + (delta x[p]) B[n],   y[p] = sum_n h[p,n] C[n] + D x[p]
//
// What bounds it: the state, read and written once (8 P N H bytes a row);
// everything else is under a percent.  So a workgroup streams whole rows of
// one head's state: a row of N values lies over LPR lanes, four consecutive
// values (16 bytes) per lane, a wave covers 64 / LPR rows, and each thread has
// the R rows it owns in flight at once.  B and C are the same for all of a
// thread's rows and stay in its registers; a row's sum over n is a butterfly
// over its LPR lanes.  Where N is not a multiple of four, a row's last vector
// starts early enough to end with the row: it overlaps the vector before it, in
// the same wave, so both have loaded before either stores, store the same
// values, and the sum takes the shared ones once.
#include "ssd_layer.h"
#include "ssd_layer_device.h"
#include "ssd_rowsum.h"
#include "ssd_step_rule.h"

// Multiply-adds are fused only inside one expression, so every variant of a kernel
// rounds a value alike.
#pragma clang fp contract(on)

namespace ssd {

namespace {

constexpr int kStepThreads = 256;   // most threads of a workgroup

// softplus and the clamp as the scan forms them (step_from_raw in ssd_device.h), but a
// NaN stays one: fmaxf and fminf would take the clamp's bound for it.
__device__ __forceinline__ float step_size(float u, float dt_min, float dt_max) {
  const float sp = fmaxf(u, 0.f) + log1pf(expf(-fabsf(u)));
  return __builtin_elementwise_minimum(__builtin_elementwise_maximum(sp, dt_min), dt_max);
}

// V: values per access (4, or 1 for N < 4); R: rows per thread.
template <typename T, typename DT, int V, int R>
__global__ __launch_bounds__(kStepThreads) void step_kernel(const StepArgs a, int lpr, int nblk) {
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
  const int n = min(ln * V, a.N - V);             // the lane's first value
  float* st = a.states + ((int64_t)slot.mine * a.H + h) * a.P * a.N + n;

  Vec<float, V> s[R];
#pragma unroll
  for (int r = 0; r < R; ++r) s[r].load(st + (int64_t)min(p0 + r * rows, a.P - 1) * a.N);
  const T* x = static_cast<const T*>(a.x) + b * a.x_stride + (int64_t)h * a.P;
  Vec<T, V> Bq, Cq;
  Bq.load(static_cast<const T*>(a.B) + b * a.b_stride + (int64_t)g * a.N + n);
  Cq.load(static_cast<const T*>(a.C) + b * a.c_stride + (int64_t)g * a.N + n);
  float Bv[V], Cv[V], xv[R];
#pragma unroll
  for (int r = 0; r < R; ++r) xv[r] = to_f32(x[min(p0 + r * rows, a.P - 1)]);
  const float u = to_f32(static_cast<const DT*>(a.dt)[b * a.dt_stride + h]) +
                  (a.dt_bias ? a.dt_bias[h] : 0.f);
  const float delta = step_size(u, a.dt_min, a.dt_max);
  const float decay = expf(delta * a.A[h]);
  const float D = a.D ? a.D[h] : 0.f;
  T* out = static_cast<T*>(a.out) + ((int64_t)b * a.H + h) * a.P;
  if (slot.repeated()) return;
  Bq.get(Bv);
  Cq.get(Cv);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int p = p0 + r * rows;
    const float dx = delta * xv[r];
    float y = 0.f, f[V];
    s[r].get(f);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      f[e] = f[e] * decay + dx * Bv[e];
      // values before the lane's own place belong to the lane before it, and
      // lanes past the row's end have none
      y += n + e >= ln * V && in ? f[e] * Cv[e] : 0.f;
    }
    s[r].set(f);
    if (p < a.P && in) s[r].store(st + (int64_t)p * a.N);
    y = run_sum_dpp(y, lpr);
    if (ln == 0 && p < a.P) out[p] = from_f32<T>(a.D ? y + D * xv[r] : y);
  }
}

template <typename T, typename DT, int V, int R>
hipError_t step_go(const StepArgs& a, int lpr, hipStream_t s) {
  // one wave where a head's rows fill no more
  int threads = kStepThreads;
  while (threads > 64 && threads / 2 * R >= a.P * lpr) threads /= 2;
  const int rows = threads / lpr * R;
  const int nblk = (a.P + rows - 1) / rows;
  hipLaunchKernelGGL((step_kernel<T, DT, V, R>), dim3((unsigned)(a.batch * (int64_t)a.H * nblk)),
                     dim3(threads), 0, s, a, lpr, nblk);
  return hipGetLastError();
}

template <typename T, typename DT>
hipError_t step_type(const StepArgs& a, hipStream_t s) {
  const int lpr = step_lpr(a.N);
  if (a.N < 4) return step_go<T, DT, 1, 1>(a, lpr, s);
  switch (step_rows(a.batch, a.H, a.P, a.N)) {
    case 4: return step_go<T, DT, 4, 4>(a, lpr, s);
    case 2: return step_go<T, DT, 4, 2>(a, lpr, s);
  }
  return step_go<T, DT, 4, 1>(a, lpr, s);
}

}  // namespace

int64_t step_row_blocks(int64_t P, int64_t N) {
  const int rows = kStepThreads / step_lpr((int)N);
  return (P + rows - 1) / rows;
}

hipError_t launch_step(const StepArgs& a, hipStream_t s) {
  if (a.batch <= 0) return hipSuccess;
  if (!a.bf16) return step_type<float, float>(a, s);
  return a.dt_bf16 ? step_type<bf16, bf16>(a, s) : step_type<bf16, float>(a, s);
}

}  // namespace ssd

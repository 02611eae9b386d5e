// The SSD for one new token per sequence: the recurrence's single update, in
// place on a cache of fp32 states.
//   delta = clamp(softplus(dt + dt_bias)),  a = exp(delta A)
//   h[p,n] = a h[p,n] + (delta x[p]) B[n],   y[p] = sum_n h[p,n] C[n] + D x[p]
//
// What bounds it: the state, read and written once (8 P N H bytes a row);
// everything else is under a percent.  So a workgroup streams whole rows of
// one head's state: a row of N values lies over LPR lanes, V consecutive
// values (16 bytes) per lane, a wave covers 64 / LPR rows, and each thread has
// the R rows it owns in flight at once.  B and C are the same for all of a
// thread's rows and stay in its registers; a row's sum over n is a butterfly
// over its LPR lanes.
#include "ssd_device.h"
#include "ssd_layer.h"
#include "ssd_layer_device.h"
#include "ssd_rowsum.h"

namespace ssd {

namespace {

constexpr int kStepThreads = 256;

// V: values per access (4, or 1 where N is not a multiple of 4); NK: accesses
// of a lane per row; R: rows per thread.
template <typename T, typename DT, int V, int NK, int R>
__global__ __launch_bounds__(kStepThreads) void step_kernel(const StepArgs a, int lpr, int nblk) {
  const int blk = blockIdx.x % nblk;              // block of rows of the head's state
  const int hb = blockIdx.x / nblk;
  const int h = hb % a.H, b = hb / a.H;
  const int g = h / (a.H / a.G);
  int64_t slot;
  if (step_row_is_padding(a.slots, b, a.nslots, slot)) return;
  const int ln = threadIdx.x & (lpr - 1);         // lane within the row
  const int rows = kStepThreads / lpr;            // rows per pass
  const int p0 = blk * rows * R + threadIdx.x / lpr;
  float* st = a.states + (slot * a.H + h) * (int64_t)a.P * a.N;

  Vec<float, V> s[R][NK];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int p = min(p0 + r * rows, a.P - 1);
#pragma unroll
    for (int k = 0; k < NK; ++k) {
      const int n = (ln + k * lpr) * V;
      s[r][k].load(st + (int64_t)p * a.N + (n < a.N ? n : 0));
    }
  }
  const T* x = static_cast<const T*>(a.x) + b * a.x_stride + (int64_t)h * a.P;
  const T* Bp = static_cast<const T*>(a.B) + b * a.b_stride + (int64_t)g * a.N;
  const T* Cp = static_cast<const T*>(a.C) + b * a.c_stride + (int64_t)g * a.N;
  float Bv[NK][V], Cv[NK][V], xv[R];
#pragma unroll
  for (int k = 0; k < NK; ++k) {
    const int n = (ln + k * lpr) * V;
    Vec<T, V> q;
    q.load(Bp + (n < a.N ? n : 0));
    q.get(Bv[k]);
    q.load(Cp + (n < a.N ? n : 0));
    q.get(Cv[k]);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      Bv[k][e] = n < a.N ? Bv[k][e] : 0.f;
      Cv[k][e] = n < a.N ? Cv[k][e] : 0.f;
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) xv[r] = to_f32(x[min(p0 + r * rows, a.P - 1)]);
  const float u = to_f32(static_cast<const DT*>(a.dt)[b * a.dt_stride + h]) +
                  (a.dt_bias ? a.dt_bias[h] : 0.f);
  const float delta = step_from_raw(u, a.dt_min, a.dt_max);
  const float decay = expf(delta * a.A[h]);
  const float D = a.D ? a.D[h] : 0.f;
  T* out = static_cast<T*>(a.out) + ((int64_t)b * a.H + h) * a.P;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int p = p0 + r * rows;
    const float dx = delta * xv[r];
    float y = 0.f;
#pragma unroll
    for (int k = 0; k < NK; ++k) {
      const int n = (ln + k * lpr) * V;
      float f[V];
      s[r][k].get(f);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        f[e] = f[e] * decay + dx * Bv[k][e];
        // a lane past the row's end holds another value's copy: it adds nothing
        y += n < a.N ? f[e] * Cv[k][e] : 0.f;
      }
      s[r][k].set(f);
      if (p < a.P && n < a.N) s[r][k].store(st + (int64_t)p * a.N + n);
    }
    y = run_sum_dpp(y, lpr);
    if (ln == 0 && p < a.P) out[p] = from_f32<T>(a.D ? y + D * xv[r] : y);
  }
}

// Lanes per row: N's accesses rounded up to a power of two, at most a wave.
int step_lpr(int N, int V) {
  int l = 1;
  while (l < 64 && l * V < N) l *= 2;
  return l;
}

template <typename T, typename DT, int V, int NK, int R>
hipError_t step_go(const StepArgs& a, int lpr, hipStream_t s) {
  const int rows = kStepThreads / lpr * R;
  const int nblk = (a.P + rows - 1) / rows;
  hipLaunchKernelGGL((step_kernel<T, DT, V, NK, R>), dim3((unsigned)(a.batch * (int64_t)a.H * nblk)),
                     dim3(kStepThreads), 0, s, a, lpr, nblk);
  return hipGetLastError();
}

template <typename T, typename DT>
hipError_t step_type(const StepArgs& a, hipStream_t s) {
  if (a.N % 4 == 0) return step_go<T, DT, 4, 1, 1>(a, step_lpr(a.N, 4), s);
  const int lpr = step_lpr(a.N, 1);
  switch ((a.N + lpr - 1) / lpr) {
    case 1: return step_go<T, DT, 1, 1, 1>(a, lpr, s);
    case 2: return step_go<T, DT, 1, 2, 1>(a, lpr, s);
    case 3: return step_go<T, DT, 1, 3, 1>(a, lpr, s);
    case 4: return step_go<T, DT, 1, 4, 1>(a, lpr, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace

int64_t step_row_blocks(int64_t P, int64_t N) {
  const int rows = kStepThreads / step_lpr((int)N, N % 4 == 0 ? 4 : 1);
  return (P + rows - 1) / rows;
}

hipError_t launch_step(const StepArgs& a, hipStream_t s) {
  if (a.batch <= 0) return hipSuccess;
  if (!a.bf16) return step_type<float, float>(a, s);
  return a.dt_bf16 ? step_type<bf16, bf16>(a, s) : step_type<bf16, float>(a, s);
}

}  // namespace ssd

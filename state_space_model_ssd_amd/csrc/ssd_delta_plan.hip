// The gated delta rule's view of a packed batch: its chunk table, the rows outside every sequence
// cleared, and how long sequences are cut (DeltaSplit).
//
// Up to a wave's count of sequences in one launch, every workgroup of which adds up the sequences'
// chunks by itself; more take the scan's two launches and one that clears.  Each of these is 2 to
// 3 us and the gap before it (9 packed prompts of 14371 tokens, 24 heads of 64 x 128: 224 us a
// forward with four launches, 217 with one; 340 tokens in three sequences, 16 heads: 29.6 and 26.0, as
// measured when they were joined).
#include "ssd_delta.h"
#include "ssd_kernels.h"

namespace ssd {

int device_cu_count();

namespace {

constexpr int kPlanThreads = 256;
constexpr int kClearBlocks = 512;        // most workgroups that clear

// Rows [0, first) and [last, total) of a tensor, of n2 16-bit values each.
__device__ __forceinline__ void clear_rows(void* p, int64_t n2, int64_t first, int64_t last, int64_t total) {
  unsigned short* o = static_cast<unsigned short*>(p);
  const int64_t at = (int64_t)blockIdx.x * kPlanThreads + threadIdx.x, step = (int64_t)gridDim.x * kPlanThreads;
  for (int64_t i = at; i < first * n2; i += step) o[i] = 0;
  for (int64_t i = max(first, last) * n2 + at; i < total * n2; i += step) o[i] = 0;
}

__global__ __launch_bounds__(kPlanThreads) void delta_clear_kernel(const DeltaArgs a, const DeltaClear c) {
  const int first = min(max(a.cu[0], 0), a.total), last = min(max(a.cu[a.nstates], 0), a.total);
  for (int t = 0; t < c.n; ++t) clear_rows(c.p[t], c.row[t] / 2, first, last, a.total);
}

__global__ __launch_bounds__(kPlanThreads) void delta_plan_kernel(const DeltaArgs a, const DeltaClear c, int cus) {
  __shared__ int chunk[DeltaSplit::kSequences + 1], begin[DeltaSplit::kSequences], end[DeltaSplit::kSequences];
  const int tid = threadIdx.x, n = a.nstates;
  if (tid < DeltaSplit::kSequences) {              // one wave
    int from = 0, to = 0;
    if (tid < n) {
      from = min(max(a.cu[tid], 0), a.total);
      to = min(max(a.cu[tid + 1], from), a.total);
    }
    const int count = (to - from + kDeltaChunk - 1) / kDeltaChunk;
    int sum = count;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int o = __shfl_up(sum, off);
      if (tid >= off) sum += o;
    }
    // malformed lengths may add up to more chunks than there is room for
    begin[tid] = from;
    end[tid] = to;
    chunk[tid + 1] = min(sum, a.max_chunks);
    if (tid == 0) chunk[0] = 0;
    if (blockIdx.x == 0 && a.split.slots) {
      DeltaSplit::Sums v = {};
      v.add(a.split, min(sum, a.max_chunks) - min(sum - count, a.max_chunks), 1);
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        v.longest = max(v.longest, __shfl_xor(v.longest, off));
#pragma unroll
        for (int i = 0; i < DeltaSplit::kLengths; ++i) {
          v.first[i] += __shfl_xor(v.first[i], off);
          v.later[i] += __shfl_xor(v.later[i], off);
          v.chain[i] = max(v.chain[i], __shfl_xor(v.chain[i], off));
        }
      }
      const int all = min(__shfl(sum, 63), a.max_chunks);
      if (tid == 0) *a.split.chosen = DeltaSplit::best(a.split, v, all, a.H, a.P, a.N, a.split.block, cus);
    }
  }
  __syncthreads();
  if (blockIdx.x == 0 && tid <= n) a.seq_chunks[tid] = chunk[tid];
  const int j = blockIdx.x * kPlanThreads + tid;
  if (j < a.max_chunks) {
    int4 d = make_int4(0, 0, 0, 0);
    if (j < chunk[n]) {
      int lo = 0, hi = n - 1;                      // the last sequence whose first chunk is not behind j
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (chunk[mid] <= j) lo = mid;
        else hi = mid - 1;
      }
      const int k = j - chunk[lo], at = begin[lo] + k * kDeltaChunk, len = max(0, min(kDeltaChunk, end[lo] - at));
      d = make_int4(len > 0 ? at : 0, len, lo, k);
    }
    a.table[j] = d;
  }
  const int first = begin[0], last = min(max(a.cu[n], 0), a.total);
  for (int t = 0; t < c.n; ++t) clear_rows(c.p[t], c.row[t] / 2, first, last, a.total);
}

}  // namespace

hipError_t launch_delta_plan(const DeltaArgs& a, const DeltaClear& c, hipStream_t s) {
  if (!a.cu) return hipSuccess;
  int64_t most = 0;
  for (int i = 0; i < c.n; ++i) most = c.row[i] > most ? c.row[i] : most;
  int64_t clears = ((int64_t)a.total * most / 2 + kPlanThreads * 16 - 1) / (kPlanThreads * 16);
  if (clears > kClearBlocks) clears = kClearBlocks;
  if (a.nstates <= DeltaSplit::kSequences) {
    int64_t blocks = (a.max_chunks + kPlanThreads - 1) / kPlanThreads;
    if (blocks < clears) blocks = clears;
    if (blocks < 1) blocks = 1;
    hipLaunchKernelGGL(delta_plan_kernel, dim3((unsigned)blocks), dim3(kPlanThreads), 0, s, a, c,
                       device_cu_count() > 0 ? device_cu_count() : 256);
    return hipGetLastError();
  }
  FwdArgs f{};
  f.batch = 1;
  f.seqlen = a.total;
  f.L = kDeltaChunk;
  f.nstates = a.nstates;
  f.max_chunks = a.max_chunks;
  f.packed = true;
  f.cu_seqlens = a.cu;
  f.table = a.table;
  f.seq_chunks = a.seq_chunks;
  const hipError_t e = launch_plan(f, s);
  if (e != hipSuccess || clears == 0) return e;
  hipLaunchKernelGGL(delta_clear_kernel, dim3((unsigned)clears), dim3(kPlanThreads), 0, s, a, c);
  return hipGetLastError();
}

}  // namespace ssd

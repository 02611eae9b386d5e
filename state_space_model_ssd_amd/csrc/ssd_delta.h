// Host-side launch interface of the gated delta rule and of the norms of queries
// and keys (internal).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ssd_common.h"
#include "ssd_delta_cut.h"

namespace ssd {

constexpr int kDeltaChunk = 64;              // tokens per chunk
constexpr int kGateFloats = 6 * kDeltaChunk; // per (chunk, head): beta, E, D, beta E, and G in fp64
constexpr int kPiece = 1024;                 // bytes of 64 lanes' 16: operands lie in such pieces
// Pieces of a triangular 64x64 matrix (six 16x32 tiles of eight), rounded or as pairs, and of an
// fp32 [N][64] one.
__host__ __device__ constexpr int triangle_pieces(bool b16, bool pair) { return b16 && !pair ? 6 : 12; }
__host__ __device__ constexpr int transposed_pieces(int N) { return N / 16 * 2 * 2; }

// Cut sequences' slots: DeltaCut's rule, and where segments' states lie.  The sequences' first
// segments come first, then the others: a grid of slots has the workgroups without work behind
// all those of sequences that stay whole, which between them would take CUs from one another (12
// sequences of 1000 tokens, 16 heads of 64 x 128: 109 us for 78).
struct DeltaSplit : DeltaCut {
  static constexpr int kSequences = 64;  // most of a packed batch
  int slots;              // for segments of all sequences; 0: nothing is cut
  int per_row;            // segments of a row (equal rows)
  int fixed;              // the length: the host's (equal rows)
  int block;              // rows of a state that a workgroup has
  int* chosen;            // or in memory (packed batch); 0: nothing is cut
  float* ends;            // [slots][H][P + N][N] of zeros, and of a unit matrix
  float* starts;          // [slots][H][P][N] the states that segments start from

  __device__ __forceinline__ int length() const { return chosen ? *chosen : fixed; }
  // The first of the slots of a sequence's other segments than its first.
  __device__ __forceinline__ int others(const ChunkMap& cm, int n, int length, int seq) const {
    return chosen ? DeltaCut::others(n, length, cm.seq_range(seq).x) : n + seq * (per_row - 1);
  }
  __device__ __forceinline__ int2 segment(const ChunkMap& cm, int n, int length, int slot) const {
    if (!chosen && slot >= n) return make_int2((slot - n) / (per_row - 1), 1 + (slot - n) % (per_row - 1));
    int seq, part;
    DeltaCut::segment(n, length, slot, [&](int i) { return cm.seq_range(i).x; }, seq, part);
    return make_int2(seq, part);
  }
};

// The gated delta rule over whole prompts, forward and backward.
struct DeltaArgs {
  int total;              // tokens over all rows
  int seqlen;             // tokens per row
  int nstates;            // sequences
  int H, G, P, N;
  int max_chunks, nc_row;
  bool bf16, gate_bf16;
  bool back;              // the backward's launches
  bool pairs;             // backward: S, dS and R are kept as pairs (bf16), as dR always is
  float scale;
  const void* q;
  const void* k;
  const void* v;
  const void* g;
  const void* beta;
  const float* init;      // nullable
  const int32_t* cu;      // packed batch, else nullptr
  void* out;
  float* final_states;    // nullable
  // backward
  const void* dout;
  const float* dfinal;    // nullable
  void* dq;
  void* dk;
  void* dv;
  void* dg;
  void* dbeta;
  float* dinit;           // nullable
  // workspace; per (chunk, head) unless said otherwise.  Matrices that later launches
  // multiply by lie as operands: see ssd_delta_device.h.
  int4* table;            // packed batch: [max_chunks]
  int* seq_chunks;        // packed batch: [nstates + 1]
  float* gates;           // [kGateFloats]
  void* T;                // T beta, or for the backward T' (ssd_delta_prep.hip), lower, pairs
  void* A;                // scale (D * q k^T), lower (forward)
  void* kt;               // per (chunk, group), fp32: k transposed
  // backward
  void* Tt;               // T transposed, upper, pairs
  void* At;               // A transposed, upper, pairs
  void* qt;               // per (chunk, group), fp32: q transposed
  void* S0;               // [P][N] the state entering the chunk, dtype (two with pairs: high
                          // and low parts; so the next two)
  void* dS;               // [P][N] the gradient of the state leaving it
  void* Rt;               // [P][64] the rows r, transposed
  void* dRt;              // [P][64] the gradient of the rows w, transposed, fp32 or pairs
  DeltaSplit split;

  ChunkMap cmap() const {
    ChunkMap m;
    m.table = cu ? table : nullptr;
    m.seq_chunks = cu ? seq_chunks : nullptr;
    m.seqlen = seqlen;
    m.nc_row = nc_row;
    m.L = kDeltaChunk;
    return m;
  }
};

bool delta_dstate_ok(int64_t N);
// n tensors of `row` bytes a token, whose rows that no sequence of a packed batch has become zeros.
struct DeltaClear {
  int n;
  void* p[5];
  int64_t row[5];
};
// A packed batch's chunk table, its clearing, and how it is cut.
hipError_t launch_delta_plan(const DeltaArgs& a, const DeltaClear& c, hipStream_t s);
// The rows of a state that a workgroup of the chain has.
int delta_chain_rows(const DeltaArgs& a);
hipError_t launch_delta_prep(const DeltaArgs& a, bool bwd, hipStream_t s);
// The chain of states; `keep`: for the backward, which wants S0 and Rt and no output.
hipError_t launch_delta_chain(const DeltaArgs& a, bool keep, hipStream_t s);
hipError_t launch_delta_chain_bwd(const DeltaArgs& a, hipStream_t s);
hipError_t launch_delta_local_bwd(const DeltaArgs& a, hipStream_t s);

// One token per sequence.
struct DeltaStepArgs {
  int batch, H, G, P, N;
  int64_t nslots;
  int64_t q_stride, k_stride, v_stride, g_stride, beta_stride;
  bool bf16, gate_bf16;
  float scale;
  const void* q;
  const void* k;
  const void* v;
  const void* g;
  const void* beta;
  float* states;
  const int32_t* slots;   // nullable
  void* out;
};
hipError_t launch_delta_step(const DeltaStepArgs& a, hipStream_t s);

// The norm of queries and keys in each head, with the rotation.
struct QkNormArgs {
  int64_t tokens;
  int heads[2];           // of q and of k
  int D, R;               // channels of a head; pairs that are rotated
  bool bf16, l2, interleaved;
  float eps;
  int64_t stride[2], dstride[2];  // elements from token to token of the inputs and of dx
  const void* x[2];
  const float* w[2];      // nullable
  const int32_t* pos;     // with R > 0
  const float* freq;
  void* out[2];
  // backward
  const void* dout[2];
  void* dx[2];
  float* dw[2];           // with w
  float* part;
};
constexpr int kQkNormMaxD = 256;
hipError_t launch_qk_norm_fwd(const QkNormArgs& a, hipStream_t s);
hipError_t launch_qk_norm_bwd(const QkNormArgs& a, hipStream_t s);
// Floats of the backward's workspace: does not depend on the device.
int64_t qk_norm_bwd_floats(int64_t tokens, int64_t D);

}  // namespace ssd

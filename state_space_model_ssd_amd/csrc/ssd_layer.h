// Host-side launch interface of the operators around the SSD (internal): the
// short convolution, the single-token state update, the block norms.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ssd {

// The short convolution, whole prompts (forward and backward) and one token
// per sequence.
struct ConvArgs {
  int total;              // tokens over all rows
  int seqlen;             // tokens per row
  int nstates;            // sequences
  int K;                  // taps
  int n[3];               // channels of x, B and C
  int C;                  // their sum
  int64_t in_stride, din_stride;
  bool bf16, silu;
  bool clear;             // rows outside every sequence become zeros
  const void* x;
  const float* w;
  const float* bias;      // nullable
  const void* init;       // nullable
  const int32_t* cu;      // packed batch, else nullptr
  void* out[3];
  void* final_states;     // nullable
  // backward
  const void* dout[3];
  const void* dfinal;     // nullable
  void* dx;
  float* dw;
  float* dbias;           // nullable
  void* dinit;            // nullable
  float* part;            // partial sums of dw and dbias
  // one token per sequence
  void* states;
  const int32_t* slots;   // nullable
  int64_t nslots;
  int batch;
};
hipError_t launch_conv_fwd(const ConvArgs& a, hipStream_t s);
hipError_t launch_conv_bwd(const ConvArgs& a, hipStream_t s);
hipError_t launch_conv_step(const ConvArgs& a, hipStream_t s);
// Floats of the backward's workspace: does not depend on the device.
int64_t conv_bwd_floats(int64_t tokens, int64_t nstates, int64_t C, int64_t K);

// The single-token state update.
struct StepArgs {
  int batch, H, P, N, G;
  int64_t nslots;
  int64_t x_stride, dt_stride, b_stride, c_stride;
  bool bf16, dt_bf16;
  float dt_min, dt_max;
  const void* x;
  const void* dt;
  const float* dt_bias;   // nullable
  const float* A;
  const void* B;
  const void* C;
  const float* D;         // nullable
  float* states;
  const int32_t* slots;   // nullable
  void* out;
};
// Workgroups of a step's launch: batch * H * step_row_blocks at most.
int64_t step_row_blocks(int64_t P, int64_t N);
hipError_t launch_step(const StepArgs& a, hipStream_t s);

// The norms around a block.
struct BlockNormArgs {
  int64_t rows;
  int C;
  bool bf16, res_bf16;
  int act;                // 0: the gate itself, 1: sigmoid, 2: SiLU
  float alpha, eps;
  const void* x;
  const void* residual;   // nullable
  const void* gate;       // nullable
  const float* post_w;    // nullable
  const float* scale;     // nullable
  const float* pre_w;
  void* out;
  void* res_out;          // nullable
  // backward
  const void* dout;
  const void* dres_out;   // nullable
  void* dx;
  void* dres;             // nullable
  void* dgate;            // with gate
  float* dpost_w;         // with post_w
  float* dscale;          // with scale
  float* dpre_w;
  float* part;            // partial sums of the weight gradients
};
constexpr int kBlockNormMaxC = 8192;
hipError_t launch_block_norm_fwd(const BlockNormArgs& a, hipStream_t s);
hipError_t launch_block_norm_bwd(const BlockNormArgs& a, hipStream_t s);
// Floats of the backward's workspace: does not depend on the device.
int64_t block_norm_bwd_floats(int64_t rows, int64_t C);

}  // namespace ssd

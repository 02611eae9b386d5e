// C ABI of the operators around the SSD (declared in include/ssd.h): host-side
// argument checks and the launches on the caller's stream.
#include <math.h>

#include "ssd.h"
#include "ssd_layer.h"
#include "ssd_span.h"

namespace ssd {
namespace {

constexpr size_t kLayerAlign = 256;

bool dtype_ok(int32_t d) { return d == SSD_F32 || d == SSD_BF16; }

bool aligned_to(const void* p, int32_t dtype) {
  return reinterpret_cast<uintptr_t>(p) % (dtype == SSD_BF16 ? 2 : 4) == 0;
}

bool workspace_ok(const void* ws, size_t have, size_t need) {
  return need == 0 ||
         (ws && reinterpret_cast<uintptr_t>(ws) % kLayerAlign == 0 && have >= need);
}

// A row stride: 0 stands for contiguous rows.
bool stride_ok(int64_t stride, int64_t row) {
  return stride == 0 || (stride >= row && stride <= (int64_t)1 << 31);
}

ssd_status_t check_conv(const ssd_conv_problem_t* p) {
  if (!p) return SSD_ERR_INVALID_ARG;
  if (p->batch < 0 || p->seqlen < 0 || p->nseq < 0 || p->channels_x < 1 || p->channels_b < 0 ||
      p->channels_c < 0 || p->width < 1)
    return SSD_ERR_INVALID_ARG;
  if (!dtype_ok(p->dtype) || p->activation < 0 || p->activation > 1) return SSD_ERR_INVALID_ARG;
  if (p->clear_outside < 0 || p->clear_outside > 1) return SSD_ERR_INVALID_ARG;
  if (p->nseq > 0 && p->batch != 1) return SSD_ERR_INVALID_ARG;
  if (p->width < 2 || p->width > 4) return SSD_ERR_UNSUPPORTED;
  const int64_t most = (int64_t)1 << 20;
  if (p->channels_x > most || p->channels_b > most || p->channels_c > most) return SSD_ERR_UNSUPPORTED;
  const int64_t C = p->channels_x + p->channels_b + p->channels_c;
  if (C > most) return SSD_ERR_UNSUPPORTED;
  if (!stride_ok(p->in_stride, C) || !stride_ok(p->din_stride, C)) return SSD_ERR_INVALID_ARG;
  // int32 token indices on the device; grid limits
  const int64_t nstates = p->nseq > 0 ? p->nseq : p->batch;
  if (nstates > 65535 || p->seqlen > (int64_t)1 << 30) return SSD_ERR_UNSUPPORTED;
  const int64_t tokens = p->batch * p->seqlen;
  if (tokens > (int64_t)1 << 30 || tokens * C > (int64_t)1 << 40) return SSD_ERR_UNSUPPORTED;
  if (nstates * C > (int64_t)1 << 30) return SSD_ERR_UNSUPPORTED;
  return SSD_OK;
}

ConvArgs conv_args(const ssd_conv_problem_t* p) {
  ConvArgs a{};
  a.total = (int)(p->batch * p->seqlen);
  a.seqlen = (int)p->seqlen;
  a.nstates = (int)(p->nseq > 0 ? p->nseq : p->batch);
  a.K = (int)p->width;
  a.n[0] = (int)p->channels_x;
  a.n[1] = (int)p->channels_b;
  a.n[2] = (int)p->channels_c;
  a.C = a.n[0] + a.n[1] + a.n[2];
  a.in_stride = p->in_stride ? p->in_stride : a.C;
  a.din_stride = p->din_stride ? p->din_stride : a.C;
  a.bf16 = p->dtype == SSD_BF16;
  a.silu = p->activation == 1;
  a.clear = p->clear_outside == 1;
  a.batch = (int)p->batch;
  return a;
}

// The three outputs (or their gradients): present where they have channels.
bool conv_split_ok(const ssd_conv_problem_t* p, const void* x, const void* b, const void* c) {
  return x && (b || p->channels_b == 0) && (c || p->channels_c == 0) && aligned_to(x, p->dtype) &&
         aligned_to(b, p->dtype) && aligned_to(c, p->dtype);
}

// Packing as for ssd_fwd: exactly the packed batch has cu_seqlens, and with no
// tokens it may pass none (every sequence is then empty).
bool conv_packing_ok(const ssd_conv_problem_t* p, const int32_t* cu) {
  if (p->nseq == 0) return cu == nullptr;
  return cu != nullptr || p->seqlen == 0;
}

ssd_status_t check_step(const ssd_step_problem_t* p) {
  if (!p) return SSD_ERR_INVALID_ARG;
  if (p->batch < 0 || p->nheads < 1 || p->headdim < 1 || p->dstate < 1 || p->ngroups < 1 ||
      p->nslots < 0)
    return SSD_ERR_INVALID_ARG;
  if (p->nheads % p->ngroups != 0) return SSD_ERR_INVALID_ARG;
  if (!dtype_ok(p->dtype) || !dtype_ok(p->dt_dtype)) return SSD_ERR_INVALID_ARG;
  if (p->dtype == SSD_F32 && p->dt_dtype != SSD_F32) return SSD_ERR_INVALID_ARG;
  if (isnan(p->dt_min) || isnan(p->dt_max) || p->dt_min > p->dt_max) return SSD_ERR_INVALID_ARG;
  if (p->dstate > 256 || p->nheads > 65535 || p->batch > 65535 || p->headdim > 65535)
    return SSD_ERR_UNSUPPORTED;
  if (!stride_ok(p->x_stride, p->nheads * p->headdim) || !stride_ok(p->dt_stride, p->nheads) ||
      !stride_ok(p->b_stride, p->ngroups * p->dstate) ||
      !stride_ok(p->c_stride, p->ngroups * p->dstate))
    return SSD_ERR_INVALID_ARG;
  if (p->nslots > INT32_MAX) return SSD_ERR_UNSUPPORTED;
  if (p->batch * p->nheads * step_row_blocks(p->headdim, p->dstate) > (int64_t)1 << 23)
    return SSD_ERR_UNSUPPORTED;
  return SSD_OK;
}

ssd_status_t check_block_norm(const ssd_block_norm_problem_t* p) {
  if (!p) return SSD_ERR_INVALID_ARG;
  if (p->tokens < 0 || p->channels < 1) return SSD_ERR_INVALID_ARG;
  if (!dtype_ok(p->dtype) || !dtype_ok(p->residual_dtype)) return SSD_ERR_INVALID_ARG;
  if (p->dtype == SSD_F32 && p->residual_dtype != SSD_F32) return SSD_ERR_INVALID_ARG;
  if (p->gate_activation < 0 || p->gate_activation > 2) return SSD_ERR_INVALID_ARG;
  if (!(p->eps >= 0.f) || isinf(p->eps) || !isfinite(p->residual_scale)) return SSD_ERR_INVALID_ARG;
  if (p->channels > kBlockNormMaxC) return SSD_ERR_UNSUPPORTED;
  if (p->tokens > (int64_t)1 << 40 || p->tokens * p->channels > (int64_t)1 << 40)
    return SSD_ERR_UNSUPPORTED;
  return SSD_OK;
}

BlockNormArgs block_norm_args(const ssd_block_norm_problem_t* p) {
  BlockNormArgs a{};
  a.rows = p->tokens;
  a.C = (int)p->channels;
  a.bf16 = p->dtype == SSD_BF16;
  a.res_bf16 = p->residual_dtype == SSD_BF16;
  a.act = p->gate_activation;
  a.alpha = p->residual_scale;
  a.eps = p->eps;
  return a;
}

size_t elem_size(int32_t dtype) { return dtype == SSD_BF16 ? 2 : 4; }

// The buffers of a convolution call.
struct ConvSpans {
  uint64_t e, C, K, tokens;
  const ssd_conv_problem_t* p;
  explicit ConvSpans(const ssd_conv_problem_t* q, const ConvArgs& a)
      : e(elem_size(q->dtype)), C((uint64_t)a.C), K((uint64_t)a.K), tokens((uint64_t)a.total), p(q) {}
  Span xbc(const void* x, int64_t stride) const {
    return rows_of(x, (int64_t)tokens, (int64_t)C, stride, e);
  }
  Span part(const void* o, int64_t channels) const {
    return bytes_of(o, tokens * (uint64_t)channels * e);
  }
  Span weight(const void* w) const { return bytes_of(w, C * K * 4); }
  Span bias(const void* b) const { return bytes_of(b, C * 4); }
  Span states(const void* s, int64_t n) const { return bytes_of(s, (uint64_t)n * (K - 1) * C * e); }
  Span packing(const void* cu) const { return bytes_of(cu, (uint64_t)(p->nseq + 1) * 4); }
};

ssd_status_t status_of(hipError_t e) { return e == hipSuccess ? SSD_OK : SSD_ERR_HIP; }

}  // namespace
}  // namespace ssd

extern "C" {

ssd_status_t ssd_conv_fwd(const ssd_conv_problem_t* p, const void* xbc, const float* weight,
                          const float* bias, const void* initial_states,
                          const int32_t* cu_seqlens, void* out_x, void* out_b, void* out_c,
                          void* final_states, void* stream) {
  const ssd_status_t st = ssd::check_conv(p);
  if (st != SSD_OK) return st;
  if (!ssd::conv_packing_ok(p, cu_seqlens)) return SSD_ERR_INVALID_ARG;
  ssd::ConvArgs a = ssd::conv_args(p);
  if (a.total > 0 && (!xbc || !weight || !ssd::conv_split_ok(p, out_x, out_b, out_c)))
    return SSD_ERR_INVALID_ARG;
  if (!ssd::aligned_to(xbc, p->dtype) || !ssd::aligned_to(initial_states, p->dtype) ||
      !ssd::aligned_to(final_states, p->dtype))
    return SSD_ERR_INVALID_ARG;
  const ssd::ConvSpans m(p, a);
  if (ssd::aliased({m.part(out_x, p->channels_x), m.part(out_b, p->channels_b),
                    m.part(out_c, p->channels_c), m.states(final_states, a.nstates)},
                   {m.xbc(xbc, a.in_stride), m.weight(weight), m.bias(bias),
                    m.states(initial_states, a.nstates), m.packing(cu_seqlens)}))
    return SSD_ERR_INVALID_ARG;
  a.x = xbc; a.w = weight; a.bias = bias; a.init = initial_states; a.cu = cu_seqlens;
  a.out[0] = out_x; a.out[1] = out_b; a.out[2] = out_c;
  a.final_states = final_states;
  return ssd::status_of(ssd::launch_conv_fwd(a, static_cast<hipStream_t>(stream)));
}

size_t ssd_conv_bwd_workspace_size(const ssd_conv_problem_t* p) {
  if (ssd::check_conv(p) != SSD_OK) return 0;
  const ssd::ConvArgs a = ssd::conv_args(p);
  const size_t b = sizeof(float) * (size_t)ssd::conv_bwd_floats(a.total, a.nstates, a.C, a.K);
  return (b + ssd::kLayerAlign) / ssd::kLayerAlign * ssd::kLayerAlign;
}

ssd_status_t ssd_conv_bwd(const ssd_conv_problem_t* p, const void* xbc, const float* weight,
                          const float* bias, const void* initial_states,
                          const int32_t* cu_seqlens, const void* dout_x, const void* dout_b,
                          const void* dout_c, const void* dfinal_states, void* dxbc,
                          float* dweight, float* dbias, void* dinitial_states, void* workspace,
                          size_t workspace_bytes, void* stream) {
  const ssd_status_t st = ssd::check_conv(p);
  if (st != SSD_OK) return st;
  if (!ssd::conv_packing_ok(p, cu_seqlens)) return SSD_ERR_INVALID_ARG;
  ssd::ConvArgs a = ssd::conv_args(p);
  if (!dweight) return SSD_ERR_INVALID_ARG;
  if (a.total > 0 && (!xbc || !weight || !dxbc || !ssd::conv_split_ok(p, dout_x, dout_b, dout_c)))
    return SSD_ERR_INVALID_ARG;
  if (!ssd::aligned_to(xbc, p->dtype) || !ssd::aligned_to(initial_states, p->dtype) ||
      !ssd::aligned_to(dfinal_states, p->dtype) || !ssd::aligned_to(dxbc, p->dtype) ||
      !ssd::aligned_to(dinitial_states, p->dtype))
    return SSD_ERR_INVALID_ARG;
  // a gradient of the initial state of no token needs the taps as well
  if (dinitial_states && !weight) return SSD_ERR_INVALID_ARG;
  if (!ssd::workspace_ok(workspace, workspace_bytes, ssd_conv_bwd_workspace_size(p)))
    return SSD_ERR_WORKSPACE;
  const ssd::ConvSpans m(p, a);
  if (ssd::aliased({m.xbc(dxbc, a.din_stride), m.weight(dweight), m.bias(dbias),
                    m.states(dinitial_states, a.nstates),
                    ssd::bytes_of(workspace, ssd_conv_bwd_workspace_size(p))},
                   {m.xbc(xbc, a.in_stride), m.weight(weight), m.bias(bias),
                    m.states(initial_states, a.nstates), m.packing(cu_seqlens),
                    m.part(dout_x, p->channels_x), m.part(dout_b, p->channels_b),
                    m.part(dout_c, p->channels_c), m.states(dfinal_states, a.nstates)}))
    return SSD_ERR_INVALID_ARG;
  a.x = xbc; a.w = weight; a.bias = bias; a.init = initial_states; a.cu = cu_seqlens;
  a.dout[0] = dout_x; a.dout[1] = dout_b; a.dout[2] = dout_c;
  a.dfinal = dfinal_states;
  a.dx = dxbc; a.dw = dweight; a.dbias = dbias; a.dinit = dinitial_states;
  a.part = static_cast<float*>(workspace);
  return ssd::status_of(ssd::launch_conv_bwd(a, static_cast<hipStream_t>(stream)));
}

ssd_status_t ssd_conv_step(const ssd_conv_problem_t* p, const void* xbc, const float* weight,
                           const float* bias, void* conv_states, int64_t nslots,
                           const int32_t* slots, void* out_x, void* out_b, void* out_c,
                           void* stream) {
  const ssd_status_t st = ssd::check_conv(p);
  if (st != SSD_OK) return st;
  if (p->seqlen != 1 || p->nseq != 0 || nslots < 0) return SSD_ERR_INVALID_ARG;
  if (nslots > INT32_MAX) return SSD_ERR_UNSUPPORTED;
  if (!slots && nslots < p->batch) return SSD_ERR_INVALID_ARG;
  ssd::ConvArgs a = ssd::conv_args(p);
  if (a.batch > 0 && (!xbc || !weight || !ssd::conv_split_ok(p, out_x, out_b, out_c) ||
                      (nslots > 0 && !conv_states)))
    return SSD_ERR_INVALID_ARG;
  if (!ssd::aligned_to(xbc, p->dtype) || !ssd::aligned_to(conv_states, p->dtype))
    return SSD_ERR_INVALID_ARG;
  const ssd::ConvSpans m(p, a);
  if (ssd::aliased({m.states(conv_states, nslots), m.part(out_x, p->channels_x),
                    m.part(out_b, p->channels_b), m.part(out_c, p->channels_c)},
                   {m.xbc(xbc, a.in_stride), m.weight(weight), m.bias(bias),
                    ssd::bytes_of(slots, (uint64_t)p->batch * 4)}))
    return SSD_ERR_INVALID_ARG;
  a.x = xbc; a.w = weight; a.bias = bias;
  a.states = conv_states; a.nslots = nslots; a.slots = slots;
  a.out[0] = out_x; a.out[1] = out_b; a.out[2] = out_c;
  return ssd::status_of(ssd::launch_conv_step(a, static_cast<hipStream_t>(stream)));
}

ssd_status_t ssd_step(const ssd_step_problem_t* p, const void* x, const void* dt,
                      const float* dt_bias, const float* A, const void* B, const void* C,
                      const float* D, float* states, const int32_t* slots, void* out,
                      void* stream) {
  const ssd_status_t st = ssd::check_step(p);
  if (st != SSD_OK) return st;
  if (!slots && p->nslots < p->batch) return SSD_ERR_INVALID_ARG;
  if (p->batch > 0 && (!x || !dt || !A || !B || !C || !out || (p->nslots > 0 && !states)))
    return SSD_ERR_INVALID_ARG;
  if (!ssd::aligned_to(x, p->dtype) || !ssd::aligned_to(B, p->dtype) ||
      !ssd::aligned_to(C, p->dtype) || !ssd::aligned_to(out, p->dtype) ||
      !ssd::aligned_to(dt, p->dt_dtype) || !ssd::aligned_to(states, SSD_F32))
    return SSD_ERR_INVALID_ARG;
  ssd::StepArgs a{};
  a.batch = (int)p->batch; a.H = (int)p->nheads; a.P = (int)p->headdim; a.N = (int)p->dstate;
  a.G = (int)p->ngroups;
  a.nslots = p->nslots;
  a.x_stride = p->x_stride ? p->x_stride : p->nheads * p->headdim;
  a.dt_stride = p->dt_stride ? p->dt_stride : p->nheads;
  a.b_stride = p->b_stride ? p->b_stride : p->ngroups * p->dstate;
  a.c_stride = p->c_stride ? p->c_stride : p->ngroups * p->dstate;
  a.bf16 = p->dtype == SSD_BF16;
  a.dt_bf16 = p->dt_dtype == SSD_BF16;
  a.dt_min = p->dt_min; a.dt_max = p->dt_max;
  const int64_t HP = p->nheads * p->headdim, GN = p->ngroups * p->dstate;
  const uint64_t e = ssd::elem_size(p->dtype), H4 = (uint64_t)p->nheads * 4;
  if (ssd::aliased({ssd::bytes_of(states, ssd::capped(p->nslots, HP * p->dstate * 4)),
                    ssd::bytes_of(out, (uint64_t)p->batch * HP * e)},
                   {ssd::rows_of(x, p->batch, HP, a.x_stride, e),
                    ssd::rows_of(dt, p->batch, p->nheads, a.dt_stride, ssd::elem_size(p->dt_dtype)),
                    ssd::rows_of(B, p->batch, GN, a.b_stride, e),
                    ssd::rows_of(C, p->batch, GN, a.c_stride, e), ssd::bytes_of(dt_bias, H4),
                    ssd::bytes_of(A, H4), ssd::bytes_of(D, H4),
                    ssd::bytes_of(slots, (uint64_t)p->batch * 4)}))
    return SSD_ERR_INVALID_ARG;
  a.x = x; a.dt = dt; a.dt_bias = dt_bias; a.A = A; a.B = B; a.C = C; a.D = D;
  a.states = states; a.slots = slots; a.out = out;
  return ssd::status_of(ssd::launch_step(a, static_cast<hipStream_t>(stream)));
}

ssd_status_t ssd_block_norm_fwd(const ssd_block_norm_problem_t* p, const void* x,
                                const void* residual, const void* gate,
                                const float* post_weight, const float* scale,
                                const float* pre_weight, void* out, void* residual_out,
                                void* stream) {
  const ssd_status_t st = ssd::check_block_norm(p);
  if (st != SSD_OK) return st;
  if (p->tokens > 0 && (!x || !pre_weight || !out)) return SSD_ERR_INVALID_ARG;
  if (!ssd::aligned_to(x, p->dtype) || !ssd::aligned_to(gate, p->dtype) ||
      !ssd::aligned_to(out, p->dtype) || !ssd::aligned_to(residual, p->residual_dtype) ||
      !ssd::aligned_to(residual_out, p->residual_dtype))
    return SSD_ERR_INVALID_ARG;
  const uint64_t n = (uint64_t)(p->tokens * p->channels), c4 = (uint64_t)p->channels * 4;
  const uint64_t xb = n * ssd::elem_size(p->dtype), rb = n * ssd::elem_size(p->residual_dtype);
  // in place: the elements of out may be x's, those of residual_out residual's
  if (ssd::aliased({ssd::bytes_of(out, xb), ssd::bytes_of(residual_out, rb)},
                   {ssd::bytes_of(gate, xb), ssd::bytes_of(post_weight, c4),
                    ssd::bytes_of(scale, c4), ssd::bytes_of(pre_weight, c4)}) ||
      (out != x && ssd::overlap(ssd::bytes_of(out, xb), ssd::bytes_of(x, xb))) ||
      (residual_out != residual &&
       ssd::overlap(ssd::bytes_of(residual_out, rb), ssd::bytes_of(residual, rb))) ||
      ((residual != x || rb != xb) &&
       ssd::overlap(ssd::bytes_of(out, xb), ssd::bytes_of(residual, rb))) ||
      ((residual != x || rb != xb) &&
       ssd::overlap(ssd::bytes_of(residual_out, rb), ssd::bytes_of(x, xb))))
    return SSD_ERR_INVALID_ARG;
  ssd::BlockNormArgs a = ssd::block_norm_args(p);
  a.x = x; a.residual = residual; a.gate = gate;
  a.post_w = post_weight; a.scale = scale; a.pre_w = pre_weight;
  a.out = out; a.res_out = residual_out;
  return ssd::status_of(ssd::launch_block_norm_fwd(a, static_cast<hipStream_t>(stream)));
}

size_t ssd_block_norm_bwd_workspace_size(const ssd_block_norm_problem_t* p) {
  if (ssd::check_block_norm(p) != SSD_OK) return 0;
  const size_t b = sizeof(float) * (size_t)ssd::block_norm_bwd_floats(p->tokens, p->channels);
  return (b + ssd::kLayerAlign) / ssd::kLayerAlign * ssd::kLayerAlign;
}

ssd_status_t ssd_block_norm_bwd(const ssd_block_norm_problem_t* p, const void* x,
                                const void* residual, const void* gate,
                                const float* post_weight, const float* scale,
                                const float* pre_weight, const void* dout,
                                const void* dresidual_out, void* dx, void* dresidual,
                                void* dgate, float* dpost_weight, float* dscale,
                                float* dpre_weight, void* workspace, size_t workspace_bytes,
                                void* stream) {
  const ssd_status_t st = ssd::check_block_norm(p);
  if (st != SSD_OK) return st;
  if (!dpre_weight || !post_weight != !dpost_weight || !scale != !dscale) return SSD_ERR_INVALID_ARG;
  if (p->tokens > 0 && (!x || !pre_weight || !dout || !dx || !gate != !dgate))
    return SSD_ERR_INVALID_ARG;
  if (!ssd::aligned_to(x, p->dtype) || !ssd::aligned_to(gate, p->dtype) ||
      !ssd::aligned_to(dout, p->dtype) || !ssd::aligned_to(dx, p->dtype) ||
      !ssd::aligned_to(dgate, p->dtype) || !ssd::aligned_to(residual, p->residual_dtype) ||
      !ssd::aligned_to(dresidual_out, p->residual_dtype) ||
      !ssd::aligned_to(dresidual, p->residual_dtype))
    return SSD_ERR_INVALID_ARG;
  if (!ssd::workspace_ok(workspace, workspace_bytes, ssd_block_norm_bwd_workspace_size(p)))
    return SSD_ERR_WORKSPACE;
  const uint64_t n = (uint64_t)(p->tokens * p->channels), c4 = (uint64_t)p->channels * 4;
  const uint64_t xb = n * ssd::elem_size(p->dtype), rb = n * ssd::elem_size(p->residual_dtype);
  if (ssd::aliased({ssd::bytes_of(dx, xb), ssd::bytes_of(dresidual, rb), ssd::bytes_of(dgate, xb),
                    ssd::bytes_of(dpost_weight, c4), ssd::bytes_of(dscale, c4),
                    ssd::bytes_of(dpre_weight, c4),
                    ssd::bytes_of(workspace, ssd_block_norm_bwd_workspace_size(p))},
                   {ssd::bytes_of(x, xb), ssd::bytes_of(residual, rb), ssd::bytes_of(gate, xb),
                    ssd::bytes_of(post_weight, c4), ssd::bytes_of(scale, c4),
                    ssd::bytes_of(pre_weight, c4), ssd::bytes_of(dout, xb),
                    ssd::bytes_of(dresidual_out, rb)}))
    return SSD_ERR_INVALID_ARG;
  ssd::BlockNormArgs a = ssd::block_norm_args(p);
  a.x = x; a.residual = residual; a.gate = gate;
  a.post_w = post_weight; a.scale = scale; a.pre_w = pre_weight;
  a.dout = dout; a.dres_out = dresidual_out;
  a.dx = dx; a.dres = dresidual; a.dgate = dgate;
  a.dpost_w = dpost_weight; a.dscale = dscale; a.dpre_w = dpre_weight;
  a.part = static_cast<float*>(workspace);
  return ssd::status_of(ssd::launch_block_norm_bwd(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

// C ABI of the gated delta rule and of the norms of queries and keys (declared in
// include/ssd.h): host-side argument checks, workspace layout, and the launches on the
// caller's stream.
#include <math.h>

#include <type_traits>

#include "ssd.h"
#include "ssd_delta.h"
#include "ssd_kernels.h"
#include "ssd_layer.h"
#include "ssd_span.h"

namespace ssd {
namespace {

constexpr size_t kDeltaAlign = 256;

// Backward, bf16: S, dS and R are kept as pairs where the gates' gradients are wanted in fp32, and
// where there are few of them, else rounded to bf16.  A gate's gradient is a sum with cancellation
// of products of these, so single ones are off by more than many are together: dg of random keys
// without decay, rounded, is off by up to 5.5e-3 in the 2-norm over 64 gates, 3.8e-3 over 4096 and
// 3.2e-3 over 65536 (with pairs 2.4e-3 and 1.7e-3, the result's own rounding).  Pairs cost little
// while there are few, and a fifth where there are many: 1x1024 tokens, 32 heads of 128 x 128, 118
// -> 130 us; 1x2048 203 -> 230; 2x2048 295 -> 368; 2x4096 582 -> 711.
// dR is kept as pairs always: where keys are alike and beta is 1, dg is the small difference of
// <dS, S> and dv.v, and was off by 2.4e-2 with dR rounded (keys 0.02 apart) for 1.0e-2; 547 -> 582
// us at 2x4096 tokens.
constexpr int64_t kDeltaFewGates = 65536;

constexpr int kDeltaLeast = 16;          // chunks of the shortest segments of a sequence
// A quarter of an MI355X's 256 CUs; a number of its own, as the workspace must not depend on the device.
constexpr int kDeltaCutUnits = 64;

bool dtype_ok(int32_t d) { return d == SSD_F32 || d == SSD_BF16; }
size_t elem_size(int32_t dtype) { return dtype == SSD_BF16 ? 2 : 4; }
bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
bool elem_aligned(const void* p, int32_t dtype) { return aligned_to(p, elem_size(dtype)); }
bool stride_ok(int64_t stride, int64_t row) {
  return stride == 0 || (stride >= row && stride <= (int64_t)1 << 31);
}
bool workspace_ok(const void* ws, size_t have, size_t need) {
  return need == 0 || (ws && aligned_to(ws, kDeltaAlign) && have >= need);
}
size_t align_up(size_t v) { return (v + kDeltaAlign - 1) / kDeltaAlign * kDeltaAlign; }
ssd_status_t status_of(hipError_t e) { return e == hipSuccess ? SSD_OK : SSD_ERR_HIP; }

int64_t delta_chunks(const ssd_delta_problem_t* p) {
  const int64_t L = kDeltaChunk;
  if (p->nseq == 0) return p->batch * ((p->seqlen + L - 1) / L);
  // every sequence may end in a part-filled chunk; a chunk has a token at least
  const int64_t most = (p->seqlen + p->nseq * (L - 1)) / L;
  return most < p->seqlen ? most : p->seqlen;
}

ssd_status_t check_delta(const ssd_delta_problem_t* p) {
  if (!p) return SSD_ERR_INVALID_ARG;
  if (p->batch < 0 || p->seqlen < 0 || p->nseq < 0 || p->nheads < 1 || p->headdim < 1 ||
      p->dstate < 1 || p->ngroups < 1)
    return SSD_ERR_INVALID_ARG;
  if (p->nheads % p->ngroups != 0) return SSD_ERR_INVALID_ARG;
  if (!dtype_ok(p->dtype) || !dtype_ok(p->gate_dtype)) return SSD_ERR_INVALID_ARG;
  if (p->dtype == SSD_F32 && p->gate_dtype != SSD_F32) return SSD_ERR_INVALID_ARG;
  if (!isfinite(p->scale)) return SSD_ERR_INVALID_ARG;
  if (p->clear_outside < 0 || p->clear_outside > 1) return SSD_ERR_INVALID_ARG;
  if (p->nseq > 0 && p->batch != 1) return SSD_ERR_INVALID_ARG;
  if (!delta_dstate_ok(p->dstate) || p->headdim % 16 != 0 || p->headdim > 256) return SSD_ERR_UNSUPPORTED;
  // int32 token indices, 32-bit offsets inside a chunk
  if (p->nheads > 4096 || p->batch > 65535 || p->nseq > 65535 || p->seqlen > (int64_t)1 << 30)
    return SSD_ERR_UNSUPPORTED;
  const int64_t nstates = p->nseq > 0 ? p->nseq : p->batch;
  if (p->batch * p->seqlen > (int64_t)1 << 30) return SSD_ERR_UNSUPPORTED;
  // launches of at most 2^31 threads: 512 for each chunk and group, or each sequence, head and
  // 32 rows of its state
  if (delta_chunks(p) * p->nheads > (int64_t)1 << 22 ||
      nstates * p->nheads * ((p->headdim + 31) / 32) > (int64_t)1 << 22)
    return SSD_ERR_UNSUPPORTED;
  return SSD_OK;
}
DeltaArgs delta_args(const ssd_delta_problem_t* p) {
  DeltaArgs a{};
  a.total = (int)(p->batch * p->seqlen);
  a.seqlen = (int)p->seqlen;
  a.nstates = (int)(p->nseq > 0 ? p->nseq : p->batch);
  a.H = (int)p->nheads;
  a.G = (int)p->ngroups;
  a.P = (int)p->headdim;
  a.N = (int)p->dstate;
  a.max_chunks = (int)delta_chunks(p);
  a.nc_row = (int)((p->seqlen + kDeltaChunk - 1) / kDeltaChunk);
  a.bf16 = p->dtype == SSD_BF16;
  a.gate_bf16 = p->gate_dtype == SSD_BF16;
  a.scale = p->scale;
  // sequences may be cut where one's heads fill at most a quarter of the device (16384 tokens of 64
  // workgroups: 467 -> 376 us; 8192 of 128: 273 -> 321); a packed batch's lengths are not known here
  const int block = a.bf16 || a.N < 128 ? 64 : 32, blocks = (a.P + block - 1) / block, longest = p->nseq > 0 ? a.max_chunks : a.nc_row;
  const int least = longest / 64 > kDeltaLeast ? (longest + 63) / 64 : kDeltaLeast;
  const bool few = p->nseq > 0 ? a.nstates <= DeltaSplit::kSequences && a.H * blocks <= kDeltaCutUnits
                               : (int64_t)a.nstates * a.H * blocks <= kDeltaCutUnits;
  // to find that nothing is to be cut takes a packed batch 4 to 5 us, backward 15 to 24 (17 sequences
  // of 400 tokens, 32 heads of 64 x 128: 95 -> 100 and 421 -> 445 us; 12 of 1000, 16 heads: 74 -> 78 and
  // 333 -> 350); 9 of which one has half the tokens, 24 heads, gain 67 and 157 (285 -> 218, 982 -> 825)
  if (few && longest >= (p->nseq > 0 ? 4 : 2) * least) {
    a.split.least = least;
    // a row's segments are no more than these; how many, the launch says
    a.split.per_row = a.nc_row / least + 1;
    a.split.slots = p->nseq > 0 ? a.nstates + a.max_chunks / least : a.nstates * a.split.per_row;
  }
  a.pairs = a.bf16 && (!a.gate_bf16 || (int64_t)a.total * a.H < kDeltaFewGates);
  return a;
}

// The workspace's parts from `base` on (counted only, where it is null); returns its size.
size_t delta_layout(DeltaArgs& a, bool packed, bool bwd, void* base) {
  size_t off = 0;
  auto part = [&](auto& ptr, size_t bytes) {
    ptr = reinterpret_cast<std::remove_reference_t<decltype(ptr)>>(static_cast<char*>(base) + off);
    off = align_up(off + bytes);
  };
  const size_t mc = (size_t)a.max_chunks, e = a.bf16 ? 2 : 4, C = kDeltaChunk;
  const size_t mh = mc * a.H, mg = mc * a.G;
  if (packed) {
    part(a.table, mc * sizeof(int4));
    part(a.seq_chunks, ((size_t)a.nstates + 1) * 4);
  }
  if (a.split.slots) {
    const size_t n = (size_t)a.split.slots * a.H;
    if (packed) part(a.split.chosen, 4);
    part(a.split.ends, n * (a.P + a.N) * a.N * 4);
    part(a.split.starts, n * a.P * a.N * 4);
  }
  part(a.gates, mh * kGateFloats * 4);
  const size_t pair = (size_t)triangle_pieces(a.bf16, true) * kPiece;
  const size_t tr = a.bf16 ? 0 : (size_t)transposed_pieces(a.N) * kPiece;
  part(a.T, mh * pair);
  if (tr) part(a.kt, mg * tr);
  if (!bwd) {
    part(a.A, mh * triangle_pieces(a.bf16, false) * kPiece);
    return off;
  }
  part(a.Tt, mh * pair);
  part(a.At, mh * pair);
  if (tr) part(a.qt, mg * tr);
  const size_t ke = a.pairs ? 4 : e;
  part(a.S0, mh * a.P * a.N * ke);
  part(a.dS, mh * a.P * a.N * ke);
  part(a.Rt, mh * a.P * C * ke);
  part(a.dRt, mh * a.P * C * 4);
  return off;
}

size_t delta_workspace(const ssd_delta_problem_t* p, bool bwd) {
  if (check_delta(p) != SSD_OK) return 0;
  DeltaArgs a = delta_args(p);
  const size_t b = delta_layout(a, p->nseq > 0, bwd, nullptr);
  return b > kDeltaAlign ? b : kDeltaAlign;
}

// Packing as for ssd_fwd: exactly the packed batch has cu_seqlens, and with no tokens it
// may pass none (every sequence is then empty).
bool packing_ok(const ssd_delta_problem_t* p, const int32_t* cu) {
  if (p->nseq == 0) return cu == nullptr;
  return cu != nullptr || p->seqlen == 0;
}

// The buffers of a call.
struct DeltaSpans {
  uint64_t M, H, G, P, N, e, ge, n;
  const ssd_delta_problem_t* p;
  DeltaSpans(const ssd_delta_problem_t* q, const DeltaArgs& a)
      : M((uint64_t)a.total), H((uint64_t)a.H), G((uint64_t)a.G), P((uint64_t)a.P), N((uint64_t)a.N),
        e(elem_size(q->dtype)), ge(elem_size(q->gate_dtype)), n((uint64_t)a.nstates), p(q) {}
  Span qk(const void* x) const { return bytes_of(x, M * G * N * e); }
  Span v(const void* x) const { return bytes_of(x, M * H * P * e); }
  Span gate(const void* x) const { return bytes_of(x, M * H * ge); }
  Span states(const void* x) const { return bytes_of(x, n * H * P * N * 4); }
  Span packing(const void* cu) const { return bytes_of(cu, (uint64_t)(p->nseq + 1) * 4); }
};

ssd_status_t check_delta_step(const ssd_delta_step_problem_t* p) {
  if (!p) return SSD_ERR_INVALID_ARG;
  if (p->batch < 0 || p->nheads < 1 || p->headdim < 1 || p->dstate < 1 || p->ngroups < 1 || p->nslots < 0)
    return SSD_ERR_INVALID_ARG;
  if (p->nheads % p->ngroups != 0) return SSD_ERR_INVALID_ARG;
  if (!dtype_ok(p->dtype) || !dtype_ok(p->gate_dtype)) return SSD_ERR_INVALID_ARG;
  if (p->dtype == SSD_F32 && p->gate_dtype != SSD_F32) return SSD_ERR_INVALID_ARG;
  if (!isfinite(p->scale)) return SSD_ERR_INVALID_ARG;
  if (p->dstate > 256 || p->nheads > 65535 || p->batch > 65535 || p->headdim > 65535)
    return SSD_ERR_UNSUPPORTED;
  if (!stride_ok(p->q_stride, p->ngroups * p->dstate) || !stride_ok(p->k_stride, p->ngroups * p->dstate) ||
      !stride_ok(p->v_stride, p->nheads * p->headdim) || !stride_ok(p->g_stride, p->nheads) ||
      !stride_ok(p->beta_stride, p->nheads))
    return SSD_ERR_INVALID_ARG;
  if (p->nslots > INT32_MAX) return SSD_ERR_UNSUPPORTED;
  if (p->batch * p->nheads * step_row_blocks(p->headdim, p->dstate) > (int64_t)1 << 23)
    return SSD_ERR_UNSUPPORTED;
  return SSD_OK;
}

ssd_status_t check_qk_norm(const ssd_qk_norm_problem_t* p) {
  if (!p) return SSD_ERR_INVALID_ARG;
  if (p->tokens < 0 || p->q_heads < 1 || p->k_heads < 1 || p->headdim < 1 || p->rotary_pairs < 0)
    return SSD_ERR_INVALID_ARG;
  if (2 * p->rotary_pairs > p->headdim) return SSD_ERR_INVALID_ARG;
  if (!dtype_ok(p->dtype) || p->norm < 0 || p->norm > 1 || p->interleaved < 0 || p->interleaved > 1)
    return SSD_ERR_INVALID_ARG;
  if (!(p->eps >= 0.f) || isinf(p->eps)) return SSD_ERR_INVALID_ARG;
  if (p->headdim > kQkNormMaxD || p->q_heads > 4096 || p->k_heads > 4096 || p->tokens > (int64_t)1 << 30)
    return SSD_ERR_UNSUPPORTED;
  const int64_t q = p->q_heads * p->headdim, k = p->k_heads * p->headdim;
  if (!stride_ok(p->q_stride, q) || !stride_ok(p->k_stride, k) || !stride_ok(p->dq_stride, q) ||
      !stride_ok(p->dk_stride, k))
    return SSD_ERR_INVALID_ARG;
  return SSD_OK;
}

QkNormArgs qk_norm_args(const ssd_qk_norm_problem_t* p) {
  QkNormArgs a{};
  a.tokens = p->tokens;
  a.heads[0] = (int)p->q_heads;
  a.heads[1] = (int)p->k_heads;
  a.D = (int)p->headdim;
  a.R = (int)p->rotary_pairs;
  a.bf16 = p->dtype == SSD_BF16;
  a.l2 = p->norm == 1;
  a.interleaved = p->interleaved == 1;
  a.eps = p->eps;
  const int64_t in[2] = {p->q_stride, p->k_stride}, out[2] = {p->dq_stride, p->dk_stride};
  for (int i = 0; i < 2; ++i) {
    const int64_t row = (int64_t)a.heads[i] * a.D;
    a.stride[i] = in[i] ? in[i] : row;
    a.dstride[i] = out[i] ? out[i] : row;
  }
  return a;
}

}  // namespace
}  // namespace ssd

extern "C" {

size_t ssd_delta_fwd_workspace_size(const ssd_delta_problem_t* p) { return ssd::delta_workspace(p, false); }
size_t ssd_delta_bwd_workspace_size(const ssd_delta_problem_t* p) { return ssd::delta_workspace(p, true); }

ssd_status_t ssd_delta_fwd(const ssd_delta_problem_t* p, const void* q, const void* k, const void* v,
                           const void* g, const void* beta, const float* initial_states,
                           const int32_t* cu_seqlens, void* out, float* final_states, void* workspace,
                           size_t workspace_bytes, void* stream) {
  const ssd_status_t st = ssd::check_delta(p);
  if (st != SSD_OK) return st;
  if (!ssd::packing_ok(p, cu_seqlens)) return SSD_ERR_INVALID_ARG;
  ssd::DeltaArgs a = ssd::delta_args(p);
  if (a.total > 0 && (!q || !k || !v || !g || !beta || !out)) return SSD_ERR_INVALID_ARG;
  if (!ssd::aligned_to(q, 16) || !ssd::aligned_to(k, 16) || !ssd::aligned_to(v, 16) ||
      !ssd::aligned_to(out, 16) || !ssd::elem_aligned(g, p->gate_dtype) ||
      !ssd::elem_aligned(beta, p->gate_dtype) || !ssd::aligned_to(initial_states, 4) ||
      !ssd::aligned_to(final_states, 4))
    return SSD_ERR_INVALID_ARG;
  if (!ssd::workspace_ok(workspace, workspace_bytes, ssd_delta_fwd_workspace_size(p)))
    return SSD_ERR_WORKSPACE;
  const ssd::DeltaSpans m(p, a);
  if (ssd::aliased({m.v(out), m.states(final_states),
                    ssd::bytes_of(workspace, ssd_delta_fwd_workspace_size(p))},
                   {m.qk(q), m.qk(k), m.v(v), m.gate(g), m.gate(beta), m.states(initial_states),
                    m.packing(cu_seqlens)}))
    return SSD_ERR_INVALID_ARG;
  a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta;
  a.init = initial_states; a.cu = a.total > 0 ? cu_seqlens : nullptr;
  a.out = out; a.final_states = final_states;
  if (a.total == 0) a.nc_row = a.max_chunks = a.split.slots = 0;
  ssd::delta_layout(a, p->nseq > 0, false, workspace);
  a.split.block = ssd::delta_chain_rows(a);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e = ssd::launch_delta_plan(a, {p->clear_outside, {out}, {(int64_t)(m.H * m.P * m.e)}}, s);
  if (e == hipSuccess) e = ssd::launch_delta_prep(a, false, s);
  if (e == hipSuccess) e = ssd::launch_delta_chain(a, false, s);
  return ssd::status_of(e);
}

ssd_status_t ssd_delta_bwd(const ssd_delta_problem_t* p, const void* q, const void* k, const void* v,
                           const void* g, const void* beta, const float* initial_states,
                           const int32_t* cu_seqlens, const void* dout, const float* dfinal_states,
                           void* dq, void* dk, void* dv, void* dg, void* dbeta,
                           float* dinitial_states, void* workspace, size_t workspace_bytes,
                           void* stream) {
  const ssd_status_t st = ssd::check_delta(p);
  if (st != SSD_OK) return st;
  if (!ssd::packing_ok(p, cu_seqlens)) return SSD_ERR_INVALID_ARG;
  ssd::DeltaArgs a = ssd::delta_args(p);
  if (a.total > 0 && (!q || !k || !v || !g || !beta || !dout || !dq || !dk || !dv || !dg || !dbeta))
    return SSD_ERR_INVALID_ARG;
  if (!ssd::aligned_to(q, 16) || !ssd::aligned_to(k, 16) || !ssd::aligned_to(v, 16) ||
      !ssd::aligned_to(dout, 16) || !ssd::aligned_to(dq, 16) || !ssd::aligned_to(dk, 16) ||
      !ssd::aligned_to(dv, 16) || !ssd::elem_aligned(g, p->gate_dtype) ||
      !ssd::elem_aligned(beta, p->gate_dtype) || !ssd::elem_aligned(dg, p->gate_dtype) ||
      !ssd::elem_aligned(dbeta, p->gate_dtype) || !ssd::aligned_to(initial_states, 4) ||
      !ssd::aligned_to(dfinal_states, 4) || !ssd::aligned_to(dinitial_states, 4))
    return SSD_ERR_INVALID_ARG;
  if (!ssd::workspace_ok(workspace, workspace_bytes, ssd_delta_bwd_workspace_size(p)))
    return SSD_ERR_WORKSPACE;
  const ssd::DeltaSpans m(p, a);
  if (ssd::aliased({m.qk(dq), m.qk(dk), m.v(dv), m.gate(dg), m.gate(dbeta), m.states(dinitial_states),
                    ssd::bytes_of(workspace, ssd_delta_bwd_workspace_size(p))},
                   {m.qk(q), m.qk(k), m.v(v), m.gate(g), m.gate(beta), m.states(initial_states),
                    m.packing(cu_seqlens), m.v(dout), m.states(dfinal_states)}))
    return SSD_ERR_INVALID_ARG;
  a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta;
  a.init = initial_states; a.cu = a.total > 0 ? cu_seqlens : nullptr;
  a.dout = dout; a.dfinal = dfinal_states;
  a.back = true;
  a.dq = dq; a.dk = dk; a.dv = dv; a.dg = dg; a.dbeta = dbeta; a.dinit = dinitial_states;
  if (a.total == 0) a.nc_row = a.max_chunks = a.split.slots = 0;
  ssd::delta_layout(a, p->nseq > 0, true, workspace);
  a.split.block = ssd::delta_chain_rows(a);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const int64_t qk = (int64_t)(m.G * m.N * m.e), v_row = (int64_t)(m.H * m.P * m.e), gate = (int64_t)(m.H * m.ge);
  hipError_t e = ssd::launch_delta_plan(
      a, {p->clear_outside ? 5 : 0, {dq, dk, dv, dg, dbeta}, {qk, qk, v_row, gate, gate}}, s);
  if (e == hipSuccess) e = ssd::launch_delta_prep(a, true, s);
  if (e == hipSuccess) e = ssd::launch_delta_chain(a, true, s);
  if (e == hipSuccess) e = ssd::launch_delta_chain_bwd(a, s);
  if (e == hipSuccess) e = ssd::launch_delta_local_bwd(a, s);
  return ssd::status_of(e);
}

ssd_status_t ssd_delta_step(const ssd_delta_step_problem_t* p, const void* q, const void* k,
                            const void* v, const void* g, const void* beta, float* states,
                            const int32_t* slots, void* out, void* stream) {
  const ssd_status_t st = ssd::check_delta_step(p);
  if (st != SSD_OK) return st;
  if (!slots && p->nslots < p->batch) return SSD_ERR_INVALID_ARG;
  if (p->batch > 0 && (!q || !k || !v || !g || !beta || !out || (p->nslots > 0 && !states)))
    return SSD_ERR_INVALID_ARG;
  if (!ssd::elem_aligned(q, p->dtype) || !ssd::elem_aligned(k, p->dtype) ||
      !ssd::elem_aligned(v, p->dtype) || !ssd::elem_aligned(out, p->dtype) ||
      !ssd::elem_aligned(g, p->gate_dtype) || !ssd::elem_aligned(beta, p->gate_dtype) ||
      !ssd::aligned_to(states, 4))
    return SSD_ERR_INVALID_ARG;
  const int64_t HP = p->nheads * p->headdim, GN = p->ngroups * p->dstate;
  ssd::DeltaStepArgs a{};
  a.batch = (int)p->batch; a.H = (int)p->nheads; a.G = (int)p->ngroups;
  a.P = (int)p->headdim; a.N = (int)p->dstate;
  a.nslots = p->nslots;
  a.q_stride = p->q_stride ? p->q_stride : GN;
  a.k_stride = p->k_stride ? p->k_stride : GN;
  a.v_stride = p->v_stride ? p->v_stride : HP;
  a.g_stride = p->g_stride ? p->g_stride : p->nheads;
  a.beta_stride = p->beta_stride ? p->beta_stride : p->nheads;
  a.bf16 = p->dtype == SSD_BF16;
  a.gate_bf16 = p->gate_dtype == SSD_BF16;
  a.scale = p->scale;
  const uint64_t e = ssd::elem_size(p->dtype), ge = ssd::elem_size(p->gate_dtype);
  if (ssd::aliased({ssd::bytes_of(states, ssd::capped((uint64_t)p->nslots, (uint64_t)(HP * p->dstate * 4))),
                    ssd::bytes_of(out, (uint64_t)(p->batch * HP) * e)},
                   {ssd::rows_of(q, p->batch, GN, a.q_stride, e), ssd::rows_of(k, p->batch, GN, a.k_stride, e),
                    ssd::rows_of(v, p->batch, HP, a.v_stride, e),
                    ssd::rows_of(g, p->batch, p->nheads, a.g_stride, ge),
                    ssd::rows_of(beta, p->batch, p->nheads, a.beta_stride, ge),
                    ssd::bytes_of(slots, (uint64_t)p->batch * 4)}))
    return SSD_ERR_INVALID_ARG;
  a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta;
  a.states = states; a.slots = slots; a.out = out;
  return ssd::status_of(ssd::launch_delta_step(a, static_cast<hipStream_t>(stream)));
}

ssd_status_t ssd_qk_norm_fwd(const ssd_qk_norm_problem_t* p, const void* q, const void* k,
                             const float* q_weight, const float* k_weight,
                             const int32_t* positions, const float* inv_freq, void* q_out,
                             void* k_out, void* stream) {
  const ssd_status_t st = ssd::check_qk_norm(p);
  if (st != SSD_OK) return st;
  const bool rot = p->rotary_pairs > 0;
  if (p->tokens > 0 && (!q || !k || !q_out || !k_out || (rot && (!positions || !inv_freq))))
    return SSD_ERR_INVALID_ARG;
  if (!ssd::elem_aligned(q, p->dtype) || !ssd::elem_aligned(k, p->dtype) ||
      !ssd::elem_aligned(q_out, p->dtype) || !ssd::elem_aligned(k_out, p->dtype) ||
      !ssd::aligned_to(positions, 4) || !ssd::aligned_to(inv_freq, 4) ||
      !ssd::aligned_to(q_weight, 4) || !ssd::aligned_to(k_weight, 4))
    return SSD_ERR_INVALID_ARG;
  ssd::QkNormArgs a = ssd::qk_norm_args(p);
  const uint64_t e = ssd::elem_size(p->dtype), D4 = (uint64_t)p->headdim * 4;
  const int64_t qr = p->q_heads * p->headdim, kr = p->k_heads * p->headdim;
  if (ssd::aliased({ssd::rows_of(q_out, p->tokens, qr, qr, e), ssd::rows_of(k_out, p->tokens, kr, kr, e)},
                   {ssd::rows_of(q, p->tokens, qr, a.stride[0], e), ssd::rows_of(k, p->tokens, kr, a.stride[1], e),
                    ssd::bytes_of(q_weight, D4), ssd::bytes_of(k_weight, D4),
                    ssd::bytes_of(rot ? positions : nullptr, (uint64_t)p->tokens * 4),
                    ssd::bytes_of(rot ? inv_freq : nullptr, (uint64_t)p->rotary_pairs * 4)}))
    return SSD_ERR_INVALID_ARG;
  a.x[0] = q; a.x[1] = k; a.w[0] = q_weight; a.w[1] = k_weight;
  a.pos = positions; a.freq = inv_freq;
  a.out[0] = q_out; a.out[1] = k_out;
  return ssd::status_of(ssd::launch_qk_norm_fwd(a, static_cast<hipStream_t>(stream)));
}

size_t ssd_qk_norm_bwd_workspace_size(const ssd_qk_norm_problem_t* p) {
  if (ssd::check_qk_norm(p) != SSD_OK) return 0;
  const size_t b = sizeof(float) * (size_t)ssd::qk_norm_bwd_floats(p->tokens, p->headdim);
  return ssd::align_up(b + 1);
}

ssd_status_t ssd_qk_norm_bwd(const ssd_qk_norm_problem_t* p, const void* q, const void* k,
                             const float* q_weight, const float* k_weight,
                             const int32_t* positions, const float* inv_freq, const void* dq_out,
                             const void* dk_out, void* dq, void* dk, float* dq_weight,
                             float* dk_weight, void* workspace, size_t workspace_bytes,
                             void* stream) {
  const ssd_status_t st = ssd::check_qk_norm(p);
  if (st != SSD_OK) return st;
  const bool rot = p->rotary_pairs > 0;
  if (!q_weight != !dq_weight || !k_weight != !dk_weight) return SSD_ERR_INVALID_ARG;
  if (p->tokens > 0 && (!q || !k || !dq_out || !dk_out || !dq || !dk || (rot && (!positions || !inv_freq))))
    return SSD_ERR_INVALID_ARG;
  if (!ssd::elem_aligned(q, p->dtype) || !ssd::elem_aligned(k, p->dtype) ||
      !ssd::elem_aligned(dq_out, p->dtype) || !ssd::elem_aligned(dk_out, p->dtype) ||
      !ssd::elem_aligned(dq, p->dtype) || !ssd::elem_aligned(dk, p->dtype) ||
      !ssd::aligned_to(positions, 4) || !ssd::aligned_to(inv_freq, 4) ||
      !ssd::aligned_to(q_weight, 4) || !ssd::aligned_to(k_weight, 4) ||
      !ssd::aligned_to(dq_weight, 4) || !ssd::aligned_to(dk_weight, 4))
    return SSD_ERR_INVALID_ARG;
  const bool sums = q_weight || k_weight;
  if (sums && !ssd::workspace_ok(workspace, workspace_bytes, ssd_qk_norm_bwd_workspace_size(p)))
    return SSD_ERR_WORKSPACE;
  ssd::QkNormArgs a = ssd::qk_norm_args(p);
  const uint64_t e = ssd::elem_size(p->dtype), D4 = (uint64_t)p->headdim * 4;
  const int64_t qr = p->q_heads * p->headdim, kr = p->k_heads * p->headdim;
  if (ssd::aliased({ssd::rows_of(dq, p->tokens, qr, a.dstride[0], e), ssd::rows_of(dk, p->tokens, kr, a.dstride[1], e),
                    ssd::bytes_of(dq_weight, D4), ssd::bytes_of(dk_weight, D4),
                    ssd::bytes_of(sums ? workspace : nullptr, ssd_qk_norm_bwd_workspace_size(p))},
                   {ssd::rows_of(q, p->tokens, qr, a.stride[0], e), ssd::rows_of(k, p->tokens, kr, a.stride[1], e),
                    ssd::rows_of(dq_out, p->tokens, qr, qr, e), ssd::rows_of(dk_out, p->tokens, kr, kr, e),
                    ssd::bytes_of(q_weight, D4), ssd::bytes_of(k_weight, D4),
                    ssd::bytes_of(rot ? positions : nullptr, (uint64_t)p->tokens * 4),
                    ssd::bytes_of(rot ? inv_freq : nullptr, (uint64_t)p->rotary_pairs * 4)}))
    return SSD_ERR_INVALID_ARG;
  a.x[0] = q; a.x[1] = k; a.w[0] = q_weight; a.w[1] = k_weight;
  a.pos = positions; a.freq = inv_freq;
  a.dout[0] = dq_out; a.dout[1] = dk_out;
  a.dx[0] = dq; a.dx[1] = dk; a.dw[0] = dq_weight; a.dw[1] = dk_weight;
  a.part = sums ? static_cast<float*>(workspace) : nullptr;
  return ssd::status_of(ssd::launch_qk_norm_bwd(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

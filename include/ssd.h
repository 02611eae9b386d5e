/*
 * ssd.h: C ABI of the Mamba-2 SSD (state-space duality) chunked-scan
 * forward on one AMD Instinct MI355X (gfx950).
 *
 * What the library computes.  A Mamba-2 layer updates a fixed-size hidden
 * state per head with every token, and the chunkwise form processes it
 * chunk by chunk (aiproviderindex.com, item on CUDA Tile Mamba-2 kernels,
 * "Mamba-2 offers a different scaling path").  The pages do not write the
 * update out; this library reads it as the plain Mamba-2 selective
 * state-space update.  For each sequence s, head h (B/C group g =
 * h / (nheads / ngroups)) and token t:
 *
 *   delta_t  = clamp(softplus(dt[t,h] + dt_bias[h]), dt_min, dt_max)
 *   h_t      = exp(delta_t * A[h]) * h_{t-1} + delta_t * x[t,h,:] (outer) B[t,g,:]
 *   y[t,h,:] = h_t . C[t,g,:]  +  D[h] * x[t,h,:]        (h_t is P x N)
 *   h_{-1}   = initial_states[s,h] (or 0);  final_states[s,h] = h after the
 *              sequence's last token.
 *
 * It does so with the chunked scan whose forward stages the pages name
 * (aiproviderindex.com, "Mamba-2 offers a different scaling path":
 * chunk_cumsum, state propagation and output construction; clova.ai, table
 * "Share of compute time by kernel": _chunk_state_fwd, _state_passing_fwd,
 * _chunk_scan_fwd), as hand-written HIP kernels:
 *
 *   stage 0  plan            logical chunk table (chunks never straddle a
 *                            sequence)
 *   stage 1  chunk_cumsum    delta and its chunk-local running sum of delta*A
 *   stage 2  bmm_chunk       C B^T inside each chunk (lower triangle)
 *   stage 3  chunk_state     per-chunk state from a zero start
 *   stage 4  state_passing   chain over chunks: states entering each chunk
 *                            and the final states; one sequential chain per
 *                            sequence, or, for problems with few state
 *                            elements, blocks of chunks composed as an
 *                            associative scan (clova.ai, "Stage 3. Logic and
 *                            heuristic refinement")
 *   stage 5  chunk_scan      decay-masked (C B^T) x  +  exp(cumsum) C . state
 *                            +  D x, accumulated in fp32
 *
 * Conventions for every entry point:
 *   - All tensor pointers are DEVICE pointers owned by the caller; the
 *     library allocates nothing and keeps no state between calls.  Inputs are
 *     only read; `out`, `final_states` and `workspace` are written.  No
 *     pointer may alias another.
 *   - Layouts are contiguous row-major:
 *       x, out  [batch, seqlen, nheads, headdim]        dtype
 *       dt      [batch, seqlen, nheads]                 fp32 (before softplus)
 *       dt_bias [nheads] fp32 (nullable: 0);  A [nheads] fp32
 *       B, C    [batch, seqlen, ngroups, dstate]        dtype
 *       D       [nheads] fp32 (nullable: no skip term)
 *       initial_states, final_states [nstates, nheads, headdim, dstate] fp32,
 *               nstates = nseq for a packed batch, else batch (nullable)
 *       cu_seqlens [nseq + 1] int32, seq_idx [seqlen] int32 (packed batch)
 *   - `stream` is a hipStream_t (NULL: the null stream).  Work is enqueued
 *     asynchronously; nothing synchronises with the host and nothing is
 *     allocated, so a call can be captured in a HIP graph.  Kernel faults
 *     surface at the caller's next synchronisation.
 *   - Errors: argument checks run on the host before anything is enqueued; a
 *     non-OK status means no work was enqueued, except SSD_ERR_HIP (a launch
 *     failed; earlier stages of that call may have been enqueued).
 *   - Results are deterministic: no atomics, fixed reduction orders.
 */
#ifndef SSD_H_
#define SSD_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  SSD_OK = 0,
  SSD_ERR_INVALID_ARG = 1,  /* a size, pointer or combination is invalid   */
  SSD_ERR_UNSUPPORTED = 2,  /* valid, but (dtype, headdim, dstate, chunk)  */
                            /* has no compiled kernel, or a size is beyond */
                            /* the limits stated at its problem struct     */
  SSD_ERR_WORKSPACE = 3,    /* workspace NULL or smaller than required     */
  SSD_ERR_HIP = 4,          /* a HIP launch or device query failed         */
  SSD_ERR_TOO_LARGE = 5     /* ssd_fwd_noalloc: the problem's workspace is */
                            /* larger than SSD_NOALLOC_SCRATCH_BYTES       */
} ssd_status_t;

typedef enum { SSD_F32 = 0, SSD_BF16 = 1 } ssd_dtype_t;

/* Stage bits for ssd_fwd_stages. */
enum {
  SSD_STAGE_PLAN = 1u << 0,
  SSD_STAGE_CUMSUM = 1u << 1,
  SSD_STAGE_BMM = 1u << 2,
  SSD_STAGE_CHUNK_STATE = 1u << 3,
  SSD_STAGE_STATE_PASSING = 1u << 4,
  SSD_STAGE_CHUNK_SCAN = 1u << 5,
  SSD_STAGE_ALL = 0x3Fu
};

typedef struct {
  int64_t batch;       /* rows; must be 1 for a packed batch               */
  int64_t seqlen;      /* tokens per row (packed batch: total tokens); >= 0 */
  int64_t nheads;      /* H >= 1                                            */
  int64_t headdim;     /* P                                                 */
  int64_t dstate;      /* N                                                 */
  int64_t ngroups;     /* G >= 1, H % G == 0                                */
  int64_t chunk_size;  /* L                                                 */
  int64_t nseq;        /* 0: rows are the sequences; > 0: packed batch of   */
                       /* nseq sequences given by cu_seqlens or seq_idx     */
  int32_t dtype;       /* ssd_dtype_t of x, B, C and out                    */
  float dt_min;        /* clamp of delta after softplus; use 0 and +inf for */
  float dt_max;        /* no clamp                                          */
} ssd_problem_t;

/* Byte offsets into the workspace of the stage intermediates (all 256-byte
 * aligned) and the bound on the number of logical chunks they are sized for.
 *   chunk_table  int32 [max_chunks][4]: first token on the flattened token
 *                axis, valid length (<= L), sequence, index within sequence
 *   seq_chunks   int32 [nstates + 1]: first logical chunk of each sequence;
 *                the last entry is the number of chunks in use
 *   delta, dA_cumsum  fp32 [max_chunks][nheads][L]
 *   cb           dtype [max_chunks][ngroups][L][L] (entries with s <= l of
 *                the valid rows hold C B^T, fp32 accumulation stored in the
 *                dtype of x; entries with s > l in the same 64-token block
 *                as l are 0; the rest are not written)
 *   chunk_states fp32 [max_chunks][nheads][headdim][dstate]
 *   states_in    dtype [max_chunks][nheads][headdim][dstate]: state entering
 *                each chunk
 *   block_states, block_logdecay  fp32 [nstates][sp_blocks][nheads][headdim *
 *                dstate] and [nstates][sp_blocks][nheads]: the blocked
 *                state_passing's per-block end states and log decays
 *                (present, with sp_blocks = 16, only when nstates * nheads *
 *                headdim * dstate < 2^18; else sp_blocks = 1 and both are
 *                empty)
 *   sync         int32 counters of the fused forward (ssd_tuning_t.fused):
 *                max_chunks * nheads + 1                                   */
typedef struct {
  int64_t max_chunks;
  size_t chunk_table, seq_chunks, delta, dA_cumsum, cb, chunk_states, states_in;
  size_t block_states, block_logdecay, sync;
  int64_t sp_blocks;
  size_t total_bytes;
} ssd_workspace_layout_t;

/* Workspace bytes ssd_fwd needs for this problem (0 if the problem is
 * invalid or unsupported): the intermediates the stages above hand to one
 * another, stored in the layout their consumer reads (aiproviderindex.com,
 * "Memory layout is part of the algorithm").  Library bookkeeping: no
 * passage of the pages defines it. */
size_t ssd_fwd_workspace_size(const ssd_problem_t* p);

/* Fills *layout for this problem.  SSD_ERR_INVALID_ARG / SSD_ERR_UNSUPPORTED
 * as for ssd_fwd. */
ssd_status_t ssd_workspace_layout(const ssd_problem_t* p, ssd_workspace_layout_t* layout);

/* 1 if (dtype, headdim, dstate, chunk_size) has compiled kernels, else 0
 * (library bookkeeping, not from the pages). */
int ssd_config_supported(int32_t dtype, int64_t headdim, int64_t dstate, int64_t chunk_size);

/*
 * The whole SSD forward: stages 0..5 above, enqueued on `stream`.
 *
 * x, dt, A, B, C, out are required (they may be NULL only when
 * batch * seqlen == 0).  dt_bias, D, initial_states, final_states are
 * optional.  A packed batch (p->nseq > 0, p->batch == 1) takes exactly one
 * of cu_seqlens (non-decreasing, from 0 to seqlen) or seq_idx (the sequence
 * id of each token, non-decreasing, in [0, nseq)); with seqlen == 0 it may
 * pass neither (every sequence is then empty).  An unpacked problem takes
 * neither.  Malformed packing arrays give unspecified outputs but never an
 * access outside the given buffers.  Tokens that belong to no sequence keep
 * whatever `out` held.
 *
 * The workspace (ssd_fwd_workspace_size bytes, 256-byte aligned) holds the
 * intermediates laid out as ssd_workspace_layout reports; its prior contents
 * do not matter.
 */
ssd_status_t ssd_fwd(const ssd_problem_t* p,
                     const void* x, const float* dt, const float* dt_bias,
                     const float* A, const void* B, const void* C, const float* D,
                     const float* initial_states,
                     const int32_t* cu_seqlens, const int32_t* seq_idx,
                     void* out, float* final_states,
                     void* workspace, size_t workspace_bytes, void* stream);

/*
 * As ssd_fwd, but enqueues only the stages whose SSD_STAGE_* bit is set in
 * `stages`, in stage order, reading the intermediates earlier stages left in
 * the workspace.  Used to time and test stages one by one.
 */
ssd_status_t ssd_fwd_stages(const ssd_problem_t* p,
                            const void* x, const float* dt, const float* dt_bias,
                            const float* A, const void* B, const void* C, const float* D,
                            const float* initial_states,
                            const int32_t* cu_seqlens, const int32_t* seq_idx,
                            void* out, float* final_states,
                            void* workspace, size_t workspace_bytes,
                            uint32_t stages, void* stream);

/*
 * Kernel choices a caller may pin for one call.  0 in a field keeps the
 * library's own choice for the shape.  An offline tuner times the choices
 * per problem shape and records the fastest in a config file; the Python
 * binding reads that file and falls back to 0 (the built-in choice) for
 * shapes it does not list.  None of the choices changes what is computed;
 * they move rounding only where noted.
 *   scan_kernel  chunk_scan for bf16: 1 = one workgroup per (chunk, head)
 *                tile (its rescaled path rounds differently from the
 *                masked one), 2 = the persistent walk over tiles, 3 = one
 *                workgroup of four waves per tile (bitwise the same results
 *                as 1; with 256-token chunks each wave owns four 16-row
 *                groups instead of two, so three workgroups fit on a CU).
 *                Must be 0 for fp32.
 *   sp_vec       consecutive state elements per state_passing thread: 1, 2
 *                or 4 (identical results).
 *   front        bf16 stages 1-3: 1 = one fused launch, 2 = one launch per
 *                stage (identical results).  Must be 0 for fp32.
 *   sp_blocks    state_passing: 1 = one sequential chain per sequence; 2, 4,
 *                8 or 16 = that many blocks per sequence, scanned in two
 *                launches (rounds differently: the blocks' maps are
 *                composed in another order).  Above 1 only when the
 *                workspace layout's sp_blocks is 16.
 *   fused        bf16 with 128- or 256-token chunks: 1 = front,
 *                state_passing and chunk_scan as separate launches, 2 =
 *                the front's launch, then state_passing and chunk_scan in
 *                one persistent launch in which the scan tiles of a chunk
 *                start once the state chain has passed it; bitwise the same
 *                results as 1 with the one-chain state passing and the same
 *                scan tile (scan_kernel 1 or 3, or the library's choice).
 *                2 cannot be combined with sp_blocks > 1, front 2, sp_vec
 *                1 or 2, or scan_kernel 2; it applies when a call runs all
 *                of stages 1-5.
 * A field outside its range, or a choice the dtype does not have, is
 * rejected with SSD_ERR_INVALID_ARG before anything is enqueued.
 */
typedef struct {
  int32_t scan_kernel;
  int32_t sp_vec;
  int32_t front;
  int32_t sp_blocks;
  int32_t fused;
} ssd_tuning_t;

/*
 * As ssd_fwd_stages, with kernel choices pinned by `tuning` (NULL: all 0).
 * Meant for tuners and for callers replaying a tuned configuration.
 */
ssd_status_t ssd_fwd_tuned(const ssd_problem_t* p,
                           const void* x, const float* dt, const float* dt_bias,
                           const float* A, const void* B, const void* C, const float* D,
                           const float* initial_states,
                           const int32_t* cu_seqlens, const int32_t* seq_idx,
                           void* out, float* final_states,
                           void* workspace, size_t workspace_bytes,
                           uint32_t stages, const ssd_tuning_t* tuning, void* stream);

/*
 * The kernel choices ssd_fwd / ssd_fwd_stages (and ssd_fwd_tuned for its
 * fields left 0) make for this problem on the calling thread's current HIP
 * device, in the fields of ssd_tuning_t: scan_kernel 1-3 (0 for fp32),
 * sp_vec 1/2/4, front 1 (bf16) or 0 (fp32), sp_blocks 1-16, fused 1 or 2.  They depend on
 * the shape and on the device's compute-unit count and occupancy only, never
 * on earlier calls, so a tuner or test can pin exactly what the default
 * path runs (clova.ai page, section "Stage 3. Logic and heuristic
 * refinement": launch parameters tied to the GPU's unit count belong with
 * the device, not in the code).  Host only; enqueues nothing.  Errors:
 * SSD_ERR_INVALID_ARG / SSD_ERR_UNSUPPORTED as for ssd_fwd, SSD_ERR_HIP if
 * a device query fails (e.g. no device).
 */
ssd_status_t ssd_fwd_choices(const ssd_problem_t* p, ssd_tuning_t* choices);

/*
 * The backward: gradients of loss = sum(out * dout) + sum(final_states *
 * dfinal_states) with respect to every input of ssd_fwd (the layer's backward
 * kernels are listed next to the forward ones on the clova.ai page, table
 * "Share of compute time by kernel").  Same problem, inputs and conventions
 * as ssd_fwd; the forward's stages 0-4 are recomputed inside, so no forward
 * call needs to precede it.
 *
 *   dout           [batch, seqlen, nheads, headdim] dtype (required)
 *   dfinal_states  [nstates, nheads, headdim, dstate] fp32 (nullable: 0)
 *   dx             like x, dtype          ddt  like dt, fp32
 *   dB, dC         like B and C, dtype    dA   [nheads] fp32
 *   dD, ddt_bias   [nheads] fp32 (nullable: not computed)
 *   dinitial_states [nstates, nheads, headdim, dstate] fp32 (nullable)
 * dD and ddt_bias are the gradients at the given D and dt_bias (also when
 * those are NULL, i.e. 0); dinitial_states likewise for a NULL initial
 * state.  Gradients accumulate in fp32; dx, dB, dC are rounded once to the
 * dtype.  Entries of tokens that belong to no sequence are not written.
 * The workspace is ssd_bwd_workspace_size bytes (256-byte aligned); it
 * begins with the forward's layout (ssd_workspace_layout) followed by the
 * backward's own fp32 buffers.  Errors as for ssd_fwd.
 */
size_t ssd_bwd_workspace_size(const ssd_problem_t* p);

ssd_status_t ssd_bwd(const ssd_problem_t* p,
                     const void* x, const float* dt, const float* dt_bias,
                     const float* A, const void* B, const void* C, const float* D,
                     const float* initial_states,
                     const int32_t* cu_seqlens, const int32_t* seq_idx,
                     const void* dout, const float* dfinal_states,
                     void* dx, float* ddt, float* dA, void* dB, void* dC,
                     float* dD, float* ddt_bias, float* dinitial_states,
                     void* workspace, size_t workspace_bytes, void* stream);

/*
 * As ssd_bwd, without recomputing the forward's stages 0-4: the workspace
 * (ssd_bwd_workspace_size bytes) must hold, unchanged, what a completed
 * ssd_fwd / ssd_fwd_stages / ssd_fwd_tuned call that ran stages 0-4 on the
 * same problem and the same inputs wrote into its leading
 * ssd_workspace_layout part (the steps, running sums, CB and entering
 * states), as in training, where the backward follows its forward.  The
 * gradients are those of that forward's intermediates; with the forward's
 * default kernel choices they equal ssd_bwd's bit for bit.  The library
 * cannot check that the workspace holds them: anything else in it gives
 * wrong gradients without an error.  Arguments and errors as for ssd_bwd.
 */
ssd_status_t ssd_bwd_after_fwd(const ssd_problem_t* p,
                               const void* x, const float* dt, const float* dt_bias,
                               const float* A, const void* B, const void* C, const float* D,
                               const float* initial_states,
                               const int32_t* cu_seqlens, const int32_t* seq_idx,
                               const void* dout, const float* dfinal_states,
                               void* dx, float* ddt, float* dA, void* dB, void* dC,
                               float* dD, float* ddt_bias, float* dinitial_states,
                               void* workspace, size_t workspace_bytes, void* stream);

/*
 * The gated RMS norm that follows the SSD in a Mamba-2 layer, and its
 * backward.  The pages name the layer's norm only through its backward
 * kernel (clova.ai page, table "Share of compute time by kernel":
 * _layer_norm_bwd, the largest share, memory-bound; section "How we fixed
 * it"); the norm read here is the Mamba-2 gated RMS norm.  For every row t
 * (token) and every group of group_size consecutive channels:
 *
 *   g_c   = y[t,c] * silu(z[t,c]),        silu(v) = v / (1 + exp(-v))
 *   r     = 1 / sqrt(mean_{c in group} g_c^2 + eps)
 *   out[t,c] = g_c * r * w[c]
 *
 * y is the SSD output flattened to rows of channels = nheads * headdim
 * ([tokens][channels], the layout of ssd_fwd's out), z the gate of the same
 * layout and dtype, w [channels] fp32.  Accumulation in fp32, one rounding of
 * each output to the dtype.
 *   - group_size divides channels; group_size / (16 / dtype size) is a
 *     power of two up to 64 or a multiple of 64 (else SSD_ERR_UNSUPPORTED);
 *     channels <= 8192 (bf16) or 4096 (fp32); eps >= 0.
 *   - ssd_gated_norm_fwd: out (may be y itself: each element is read before
 *     it is written, by the same thread); rstd [tokens][channels /
 *     group_size] fp32 receives r (nullable).
 *   - ssd_gated_norm_bwd: the gradients of sum(out * dout): dy, dz like y,
 *     dw [channels] fp32 (required); the workspace is
 *     ssd_gated_norm_bwd_workspace_size bytes, 256-byte aligned.  No atomics:
 *     deterministic.
 * Device pointers, asynchronous on `stream`; errors as for ssd_fwd.
 */
typedef struct {
  int64_t tokens;      /* rows                                           */
  int64_t channels;    /* channels per row                               */
  int64_t group_size;  /* consecutive channels normalised together       */
  int32_t dtype;       /* ssd_dtype_t of y, z, out, dout, dy, dz         */
  float eps;
} ssd_norm_problem_t;

ssd_status_t ssd_gated_norm_fwd(const ssd_norm_problem_t* p, const void* y, const void* z,
                                const float* w, void* out, float* rstd, void* stream);

size_t ssd_gated_norm_bwd_workspace_size(const ssd_norm_problem_t* p);

ssd_status_t ssd_gated_norm_bwd(const ssd_norm_problem_t* p, const void* y, const void* z,
                                const float* w, const void* dout, void* dy, void* dz, float* dw,
                                void* workspace, size_t workspace_bytes, void* stream);

/*
 * The forward followed by the gated RMS norm of its output (the same norm as
 * ssd_gated_norm_fwd, over rows of nheads * headdim channels): `out`
 * receives rmsnorm(y * silu(z)) * weight, not y.  Where the norm's groups lie
 * inside a head (group_size divides headdim; bf16) and chunk_scan runs a
 * one-tile-per-workgroup kernel (the library's choice for most shapes), the
 * norm is applied in chunk_scan's store and y never reaches memory;
 * otherwise the forward writes y into `out` and the norm runs over it in
 * place.  Either way the result equals ssd_fwd followed by
 * ssd_gated_norm_fwd bit for bit.  final_states and the workspace are as
 * for ssd_fwd.
 */
typedef struct {
  const void* z;        /* gate, layout and dtype of x and out           */
  const float* weight;  /* [nheads * headdim]                            */
  float eps;
  int64_t group_size;   /* channels normalised together (see ssd_norm_problem_t) */
} ssd_gate_t;

ssd_status_t ssd_fwd_gated(const ssd_problem_t* p,
                           const void* x, const float* dt, const float* dt_bias,
                           const float* A, const void* B, const void* C, const float* D,
                           const float* initial_states,
                           const int32_t* cu_seqlens, const int32_t* seq_idx,
                           const ssd_gate_t* gate, void* out, float* final_states,
                           void* workspace, size_t workspace_bytes, void* stream);

/*
 * For callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc): ssd_fwd
 * without a workspace argument.  The workspace is a static device array of
 * SSD_NOALLOC_SCRATCH_BYTES inside the library, one per device, allocated
 * when the library's code is loaded on that device and held until the
 * process ends; this call allocates nothing and calls no allocating routine.
 * The caller still passes every input and output, as for ssd_fwd.
 *   - Problems whose ssd_fwd_workspace_size exceeds SSD_NOALLOC_SCRATCH_BYTES
 *     are rejected with SSD_ERR_TOO_LARGE before anything is enqueued.
 *   - Every call on one device shares that device's array, whose contents
 *     persist between calls (nothing in it needs to start at zero).  Calls
 *     that overlap on one device, on different streams or from different
 *     threads, race on it and give wrong results: serialise them (e.g. on
 *     one stream).
 * Results are bit for bit those of ssd_fwd on the same problem and inputs.
 * Other errors as for ssd_fwd.
 */
#define SSD_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)

ssd_status_t ssd_fwd_noalloc(const ssd_problem_t* p,
                             const void* x, const float* dt, const float* dt_bias,
                             const float* A, const void* B, const void* C, const float* D,
                             const float* initial_states,
                             const int32_t* cu_seqlens, const int32_t* seq_idx,
                             void* out, float* final_states, void* stream);

/*
 * The short causal convolution in front of the SSD in a Mamba-2 layer: it
 * makes x, B and C from the layer's projection, channel by channel.  The
 * pages do not write it out (they list the layer's kernels, clova.ai page,
 * table "Share of compute time by kernel"); it is read here as the Mamba-2
 * layer's depthwise convolution of `width` K taps over the channels
 * x | B | C side by side.  For sequence s, token t of it and channel c:
 *
 *   pre[t,c] = bias[c] + sum_{k < K} weight[c,k] * in[t - (K-1) + k, c]
 *   out[t,c] = pre * sigmoid(pre)   (activation 1: SiLU)   or   pre (0)
 *   in[t] for -(K-1) <= t < 0 is initial_states[s, K-1 + t] (or 0)
 *   final_states[s] = the last K-1 rows of in, oldest first (a sequence
 *                     shorter than K-1 keeps rows of its initial state)
 *
 * Layouts (C = channels_x + channels_b + channels_c):
 *   xbc      one row of C channels per token, `in_stride` elements from one
 *            token to the next (0: C), so the rows may lie inside wider ones
 *            (the projection's z | x | B | C | dt); batch rows follow one
 *            another, seqlen * in_stride apart                       dtype
 *   weight   [C][K] fp32;  bias [C] fp32 (nullable: 0)
 *   initial_states, final_states  [nstates][K-1][C] dtype (nullable)
 *   out_x, out_b, out_c  [batch][seqlen][channels_*] dtype, each contiguous:
 *            ssd_fwd's x, B and C.  An output with no channels may be NULL.
 * Any channel counts and any alignment of the dtype's size are taken, within
 * these limits (beyond them SSD_ERR_UNSUPPORTED): width 2 to 4, C up to 2^20,
 * sequences (batch, or nseq) up to 65535, tokens (batch * seqlen) up to 2^30,
 * tokens * C up to 2^40, sequences * C up to 2^30, slots (ssd_conv_step) below
 * 2^31.  Strides of up to 2^31 elements (else SSD_ERR_INVALID_ARG).
 * Accumulation in fp32, one rounding of each output to the dtype; final
 * states are copies.  A packed batch (nseq > 0, batch 1) takes cu_seqlens
 * (non-decreasing); tokens before its first entry and from its last entry on
 * belong to no sequence, and their rows of the outputs keep what they held, or
 * with clear_outside become zeros.
 * Malformed cu_seqlens give unspecified outputs but never an access outside
 * the given buffers.  No buffer that a call writes may share memory with another
 * of its buffers (SSD_ERR_INVALID_ARG; final_states are not updated in place),
 * but strided rows may lie beside other rows of the same stride, as columns of one
 * wider tensor.  Errors as for ssd_fwd.
 */
typedef struct {
  int64_t batch;       /* rows, up to 65535; 1 for a packed batch           */
  int64_t seqlen;      /* tokens per row (packed batch: total tokens); >= 0 */
  int64_t nseq;        /* 0: rows are the sequences; > 0: packed batch, up  */
                       /* to 65535 sequences                                */
  int64_t channels_x;  /* nheads * headdim of the SSD that follows; >= 1    */
  int64_t channels_b;  /* ngroups * dstate; >= 0                            */
  int64_t channels_c;  /* ngroups * dstate; >= 0                            */
  int64_t width;       /* taps K, 2 to 4                                    */
  int64_t in_stride;   /* elements between tokens of xbc; 0: contiguous     */
  int64_t din_stride;  /* the same of dxbc (ssd_conv_bwd)                   */
  int32_t dtype;       /* ssd_dtype_t of xbc, the states and the outputs    */
  int32_t activation;  /* 0: none, 1: SiLU                                  */
  int32_t clear_outside; /* packed batch: 1 clears the rows of tokens outside */
                       /* every sequence in what the call writes (the       */
                       /* outputs, or dxbc); 0 leaves them                  */
} ssd_conv_problem_t;

ssd_status_t ssd_conv_fwd(const ssd_conv_problem_t* p, const void* xbc, const float* weight,
                          const float* bias, const void* initial_states,
                          const int32_t* cu_seqlens, void* out_x, void* out_b, void* out_c,
                          void* final_states, void* stream);

/*
 * The backward of ssd_conv_fwd: gradients of sum(out * dout) +
 * sum(final_states * dfinal_states).  With dpre = dout * act'(pre),
 *
 *   dxbc[t]     = sum_{j < K} weight[K-1-j] * dpre[t + j]   (t + j inside the
 *                 sequence) + the row of dfinal_states that holds token t
 *   dweight[k]  = sum_t dpre[t] * in[t - (K-1) + k];   dbias = sum_t dpre[t]
 *   dinitial_states likewise for the rows before a sequence's first token.
 *
 *   dout_x, dout_b, dout_c  like the outputs (ssd_bwd's dx, dB and dC)
 *   dfinal_states           like final_states (nullable: 0)
 *   dxbc                    like xbc, din_stride elements from token to token
 *                           (0: C); what lies between the rows is not written
 *   dweight [C][K] fp32 (required);  dbias [C] fp32 (nullable: not computed)
 *   dinitial_states         like initial_states (nullable: not computed)
 * pre is computed again from xbc.  Tokens outside every sequence add nothing
 * and their rows of dxbc are not written (clear_outside: zeros).  The workspace (no initial contents)
 * is ssd_conv_bwd_workspace_size bytes, 256-byte aligned; calls that may overlap
 * (on different streams, or in graphs replayed side by side) need one each.  No
 * atomics: results are deterministic.
 */
size_t ssd_conv_bwd_workspace_size(const ssd_conv_problem_t* p);

ssd_status_t ssd_conv_bwd(const ssd_conv_problem_t* p, const void* xbc, const float* weight,
                          const float* bias, const void* initial_states,
                          const int32_t* cu_seqlens, const void* dout_x, const void* dout_b,
                          const void* dout_c, const void* dfinal_states, void* dxbc,
                          float* dweight, float* dbias, void* dinitial_states, void* workspace,
                          size_t workspace_bytes, void* stream);

/*
 * ssd_conv_fwd for one new token per sequence, in place on a cache of states:
 * p->seqlen is 1 and p->nseq 0, row b of xbc is the next token of the
 * sequence whose state is conv_states[slots[b]] (slots NULL: conv_states[b]),
 * [nslots][K-1][C] dtype as final_states.  The slot's rows move up by one and
 * the token becomes the last.
 *   - A row whose slot is outside [0, nslots) is padding: its outputs keep
 *     what they held and no state changes.
 *   - A row whose slot an earlier row (a lower b) has is padding as well, so
 *     the same slot twice is well defined: the first row has it.
 * Without slots, nslots >= batch.
 */
ssd_status_t ssd_conv_step(const ssd_conv_problem_t* p, const void* xbc, const float* weight,
                           const float* bias, void* conv_states, int64_t nslots,
                           const int32_t* slots, void* out_x, void* out_b, void* out_c,
                           void* stream);

/*
 * The SSD for one new token per sequence: the recurrence at the top of this
 * file, one update, in place on a cache of states (decoding after ssd_fwd,
 * whose final_states are the first states).  For row b with its state h =
 * states[slots[b]] and head i (group g = i / (nheads / ngroups)):
 *
 *   delta = clamp(softplus(dt[b,i] + dt_bias[i]), dt_min, dt_max)
 *   h[i]  = exp(delta * A[i]) * h[i] + delta * x[b,i,:] (outer) B[b,g,:]
 *   out[b,i,:] = h[i] . C[b,g,:]  +  D[i] * x[b,i,:]
 *
 *   x       [batch][nheads][headdim] dtype, rows x_stride elements apart
 *   dt      [batch][nheads] fp32 or the dtype (dt_dtype), rows dt_stride apart
 *   B, C    [batch][ngroups][dstate] dtype, rows b_stride and c_stride apart
 *           (a stride of 0 is a contiguous tensor's; rows may lie inside
 *           wider ones, as the projection and the convolution leave them)
 *   A       [nheads] fp32;  D, dt_bias [nheads] fp32 (nullable)
 *   states  [nslots][nheads][headdim][dstate] fp32, updated in place
 *   slots   [batch] int32 (nullable: row b has slot b, nslots >= batch);
 *           padding and repeated slots as for ssd_conv_step
 *   out     [batch][nheads][headdim] dtype, contiguous
 * Any headdim and dstate within these limits (beyond them
 * SSD_ERR_UNSUPPORTED), whatever chunk configurations are compiled: dstate up
 * to 256; batch, nheads and headdim up to 65535 each; nslots below 2^31; and
 * batch * nheads * ceil(headdim / r) up to 2^23 with r = 256 / l, l the least
 * power of two of lanes that hold a row of dstate values, four (dstate below
 * four: one) each.  At dstate 128 r is 8, and the last limit 2^26 rows of
 * states, 32 GiB: larger batches take several calls.  Strides as for the
 * convolution.  The state is held and
 * updated in fp32; out is rounded once.  No workspace; `states` is the only
 * buffer that is both read and written, and neither it nor out may share memory
 * with another buffer (SSD_ERR_INVALID_ARG).
 */
typedef struct {
  int64_t batch;      /* rows, 0 to 65535                                   */
  int64_t nheads;     /* H, 1 to 65535                                      */
  int64_t headdim;    /* P, 1 to 65535                                      */
  int64_t dstate;     /* N, 1 to 256                                        */
  int64_t ngroups;    /* G >= 1, H % G == 0                                 */
  int64_t nslots;     /* states in the cache                                */
  int64_t x_stride, dt_stride, b_stride, c_stride;  /* elements; 0: contiguous */
  int32_t dtype;      /* ssd_dtype_t of x, B, C and out                     */
  int32_t dt_dtype;   /* ssd_dtype_t of dt                                  */
  float dt_min;       /* clamp of delta, as in ssd_problem_t                */
  float dt_max;
} ssd_step_problem_t;

ssd_status_t ssd_step(const ssd_step_problem_t* p, const void* x, const void* dt,
                      const float* dt_bias, const float* A, const void* B, const void* C,
                      const float* D, float* states, const int32_t* slots, void* out,
                      void* stream);

/*
 * The norms around a block of the network (around a whole Mamba-2 layer; the
 * gated norm above is the one inside it): the norm after the block with its
 * gate and residual scale, the residual sum, and the norm before the next
 * block, in one pass over the rows.  For every row t of `channels` channels:
 *
 *   p   = x * r1 * post_weight,  r1 = 1 / sqrt(mean(x^2) + eps)   (post_weight)
 *       = x                                                      (NULL)
 *   u   = p * act(gate)                                          (gate NULL: p)
 *   h   = residual + residual_scale * scale * u        (residual NULL: 0,
 *                                                       scale NULL: 1)
 *   out = h * r2 * pre_weight,   r2 = 1 / sqrt(mean(h^2) + eps)
 *
 * act is gate_activation: 0 the gate itself, 1 its sigmoid, 2 its SiLU.
 *   x, gate, out [tokens][channels] dtype;  residual, residual_out the same
 *   shape in residual_dtype (the dtype or fp32);  weights [channels] fp32.
 *   residual_out receives h (nullable).  h is normalised as summed, before
 *   its rounding to residual_dtype.
 * Any channel count up to 8192 and up to 2^40 elements (beyond:
 * SSD_ERR_UNSUPPORTED).  Accumulation in fp32, one rounding of each output.  residual_out may be residual, and out may be x (each element is
 * read before it is written, by the same thread); else no buffer that is written
 * may share memory with another (SSD_ERR_INVALID_ARG).  Errors as for ssd_fwd.
 */
typedef struct {
  int64_t tokens;          /* rows                                          */
  int64_t channels;        /* channels per row, 1 to 8192                   */
  int32_t dtype;           /* ssd_dtype_t of x, gate, out and their gradients */
  int32_t residual_dtype;  /* of residual, residual_out and their gradients */
  int32_t gate_activation; /* 0: the gate itself, 1: sigmoid, 2: SiLU       */
  float residual_scale;
  float eps;
} ssd_block_norm_problem_t;

ssd_status_t ssd_block_norm_fwd(const ssd_block_norm_problem_t* p, const void* x,
                                const void* residual, const void* gate,
                                const float* post_weight, const float* scale,
                                const float* pre_weight, void* out, void* residual_out,
                                void* stream);

/*
 * The backward of ssd_block_norm_fwd: gradients of sum(out * dout) +
 * sum(residual_out * dresidual_out).  With n = h r2 and dn = dout pre_weight:
 *
 *   dh   = r2 (dn - n mean(dn n)) + dresidual_out;      dresidual = dh
 *   du   = dh residual_scale scale;    dgate = du p act'(gate)
 *   dp   = du act(gate);               dx = dp, or with post_weight, m = x r1
 *          and dm = dp post_weight:    dx = r1 (dm - m mean(dm m))
 *   dpre_weight = sum_t dout n,  dscale = sum_t dh residual_scale u,
 *   dpost_weight = sum_t dp m
 *
 * dresidual_out (nullable: 0) and dresidual (nullable: not written) are like
 * residual, dx and dgate like x; dgate is required with a gate, dscale with a
 * scale, dpost_weight with a post_weight, and NULL otherwise; dpre_weight is
 * required.  h is computed again from the inputs.  The workspace (no initial
 * contents) is ssd_block_norm_bwd_workspace_size bytes, 256-byte aligned; calls
 * that may overlap (on different streams, or in graphs replayed side by side)
 * need one each.  No atomics: results are deterministic.
 */
size_t ssd_block_norm_bwd_workspace_size(const ssd_block_norm_problem_t* p);

ssd_status_t ssd_block_norm_bwd(const ssd_block_norm_problem_t* p, const void* x,
                                const void* residual, const void* gate,
                                const float* post_weight, const float* scale,
                                const float* pre_weight, const void* dout,
                                const void* dresidual_out, void* dx, void* dresidual,
                                void* dgate, float* dpost_weight, float* dscale,
                                float* dpre_weight, void* workspace, size_t workspace_bytes,
                                void* stream);

/*
 * The gated delta rule: the layer of a gated delta network, which hybrid models
 * mix with Mamba-2 and attention layers (clova.ai page, "Why optimize Mamba-2?",
 * names it; the formula is read here as the published gated delta rule).  For each
 * sequence s, head h (q/k group i = h / (nheads / ngroups)) and token t, with the
 * state S of headdim x dstate:
 *
 *   a   = exp(g[t,h])
 *   w   = beta[t,h] * (v[t,h,:] - a * S_{t-1} k[t,i,:])
 *   S_t = a * S_{t-1} + w (outer) k[t,i,:]
 *   out[t,h,:] = scale * S_t q[t,i,:]
 *   S_{-1} = initial_states[s,h] (or 0);  final_states[s,h] = S after the last token.
 *
 * It is the SSD's recurrence with a state that first forgets what it holds at k;
 * x, B, C of the SSD are v, k, q here.
 *
 *   q, k    [batch][seqlen][ngroups][dstate] dtype (as ssd_qk_norm_fwd leaves them)
 *   v, out  [batch][seqlen][nheads][headdim] dtype
 *   g       [batch][seqlen][nheads] gate_dtype: log decays, at most 0 as a rule; one
 *           below -512 (also -inf) is one of -512, after which the state is zero
 *   beta    [batch][seqlen][nheads] gate_dtype
 *   initial_states, final_states [nstates][nheads][headdim][dstate] fp32 (nullable)
 * all contiguous; q, k, v, out and their gradients 16-byte aligned.  Packed batches as
 * for ssd_conv_fwd (cu_seqlens, clear_outside; malformed entries never leave the
 * buffers).  The state is carried in fp32; with bf16 inputs whatever enters it does so
 * to 2^-17 or better, while the output's own products round their operands to bf16
 * once, as the output is.  A NaN or infinity in a token's inputs may reach the outputs
 * of earlier tokens of the same 64 (they are computed together), and no others before it.
 * Limits (beyond them SSD_ERR_UNSUPPORTED): dstate 32, 64 or 128; headdim a multiple of
 * 16 up to 256; nheads up to 4096; batch and nseq up to 65535; seqlen and batch * seqlen
 * up to 2^30; chunks (of 64 tokens, a sequence's last one part-filled) * nheads, and
 * sequences * nheads * ceil(headdim / 32), up to 2^22.
 * The workspace (no initial contents) is ssd_delta_fwd_workspace_size bytes, 256-byte
 * aligned; calls that may overlap need one each.  It is 20 KB (fp32: 26) per 64 tokens and
 * head, more in fp32 per group and where long sequences of few heads are cut into segments:
 * 312 MiB for 4 x 8192 tokens of 32 heads.  No buffer that is written may share memory with
 * another (SSD_ERR_INVALID_ARG).  Deterministic: the same call gives the same bits.  Those of
 * one sequence may differ between batches, as a call's sizes and lengths say where its
 * sequences are cut.  Errors as for ssd_fwd.
 */
typedef struct {
  int64_t batch;       /* rows, up to 65535; 1 for a packed batch           */
  int64_t seqlen;      /* tokens per row (packed batch: total tokens); >= 0 */
  int64_t nheads;      /* H, 1 to 4096                                      */
  int64_t headdim;     /* P, 16 to 256 in steps of 16                       */
  int64_t dstate;      /* N, 32, 64 or 128                                  */
  int64_t ngroups;     /* G >= 1, H % G == 0: heads of q and k              */
  int64_t nseq;        /* 0: rows are the sequences; > 0: packed batch      */
  int32_t dtype;       /* ssd_dtype_t of q, k, v, out                       */
  int32_t gate_dtype;  /* ssd_dtype_t of g, beta: fp32 or the dtype         */
  float scale;         /* of the output; dstate^-0.5 as a rule              */
  int32_t clear_outside; /* packed batch: 1 clears the rows of tokens outside */
                       /* every sequence in what the call writes; 0 leaves them */
} ssd_delta_problem_t;

size_t ssd_delta_fwd_workspace_size(const ssd_delta_problem_t* p);

ssd_status_t ssd_delta_fwd(const ssd_delta_problem_t* p, const void* q, const void* k,
                           const void* v, const void* g, const void* beta,
                           const float* initial_states, const int32_t* cu_seqlens, void* out,
                           float* final_states, void* workspace, size_t workspace_bytes,
                           void* stream);

/*
 * The backward of ssd_delta_fwd: gradients of sum(out * dout) + sum(final_states *
 * dfinal_states).  dq, dk, dv, dg, dbeta like q, k, v, g, beta (required);
 * dinitial_states like initial_states (nullable: not computed, also given without an
 * initial state); dfinal_states nullable: 0.  dq and dk sum over the heads of a group.
 * The forward's states are computed again.  The gradient of the state is carried as the
 * state is; with bf16 inputs the other products round their operands to bf16 once.
 * dbeta[t] is w's gradient times w / beta, and dg[t] the sum of the decayed state times its
 * gradient.  fp32 gates' are summed from values kept to 2^-17: relative to the 2-norm of the
 * products that are summed, 1e-5 as a rule.  bf16 gates' are too while tokens * nheads is below
 * 65536.  Above, the state, its gradient and w / beta are rounded to bf16 once before: dbeta is
 * off by 2.4e-3 in the 2-norm, and dg by up to 2^-8 of that of its products, 2.5e-3 to 3.3e-3
 * of dg as a rule.  Where dg is small beside its products it is off by more of its own size (beta
 * 1 and keys 0.02 apart: 1e-2; beta 1, equal keys and no decay: dg is zero but for this error);
 * fp32 gates are for callers to whom that matters.
 * Workspace: ssd_delta_bwd_workspace_size bytes, as for the forward, with the states of all
 * chunks: per 64 tokens and head 38 KB and 4 P N + 384 P bytes (P headdim, N dstate), or
 * 8 P N + 512 P in fp32, with fp32 gates and below those 65536.  4 x 8192 tokens of 32 heads of
 * 128 x 128 take 2.3 GiB, with fp32 gates 3.6 GiB.
 */
size_t ssd_delta_bwd_workspace_size(const ssd_delta_problem_t* p);

ssd_status_t ssd_delta_bwd(const ssd_delta_problem_t* p, const void* q, const void* k,
                           const void* v, const void* g, const void* beta,
                           const float* initial_states, const int32_t* cu_seqlens,
                           const void* dout, const float* dfinal_states, void* dq, void* dk,
                           void* dv, void* dg, void* dbeta, float* dinitial_states,
                           void* workspace, size_t workspace_bytes, void* stream);

/*
 * The gated delta rule for one new token per sequence: the recurrence above, one update,
 * in place on a cache of states (decoding after ssd_delta_fwd, whose final_states are the
 * first states).  Slots, padding and repeated slots as for ssd_conv_step.
 *
 *   q, k    [batch][ngroups][dstate] dtype, rows q_stride and k_stride elements apart
 *   v       [batch][nheads][headdim] dtype, rows v_stride apart
 *   g, beta [batch][nheads] gate_dtype, rows g_stride and beta_stride apart
 *           (a stride of 0 is a contiguous tensor's; rows may lie inside wider ones)
 *   states  [nslots][nheads][headdim][dstate] fp32, updated in place
 *   out     [batch][nheads][headdim] dtype, contiguous
 * Any headdim and dstate within ssd_step's limits, which hold here too.  fp32
 * arithmetic; out is rounded once.  No workspace; neither states nor out may share
 * memory with another buffer (SSD_ERR_INVALID_ARG).
 */
typedef struct {
  int64_t batch;      /* rows, 0 to 65535                                   */
  int64_t nheads;     /* H, 1 to 65535                                      */
  int64_t headdim;    /* P, 1 to 65535                                      */
  int64_t dstate;     /* N, 1 to 256                                        */
  int64_t ngroups;    /* G >= 1, H % G == 0                                 */
  int64_t nslots;     /* states in the cache                                */
  int64_t q_stride, k_stride, v_stride, g_stride, beta_stride; /* elements; 0: contiguous */
  int32_t dtype;      /* ssd_dtype_t of q, k, v and out                     */
  int32_t gate_dtype; /* ssd_dtype_t of g and beta: fp32 or the dtype       */
  float scale;
} ssd_delta_step_problem_t;

ssd_status_t ssd_delta_step(const ssd_delta_step_problem_t* p, const void* q, const void* k,
                            const void* v, const void* g, const void* beta, float* states,
                            const int32_t* slots, void* out, void* stream);

/*
 * The norm of queries and keys in each head, and the rotation by the token's position, in
 * one pass: what stands in front of the gated delta rule (norm 1, no rotation), of an
 * attention layer of a hybrid model, or of an SSD whose B and C are normed and rotated.
 * For every token t and head of `headdim` D channels, x being q or k:
 *
 *   n = x * r * weight,  r = 1 / sqrt(mean(x^2) + eps)   (norm 0)
 *                          = 1 / sqrt(sum(x^2) + eps)    (norm 1)
 *   the rotary_pairs R pairs (a, b) of n become (a cos - b sin, b cos + a sin) of the
 *   angle positions[t] * inv_freq[i]; pair i is channels (i, i + R), or (2i, 2i + 1) with
 *   `interleaved`; channels from 2R on stay.
 *
 *   q, k     [tokens][q_heads or k_heads][headdim] dtype, rows q_stride and k_stride
 *            elements apart (0: contiguous), so they may lie inside the projection's rows
 *   weights  [headdim] fp32, one for all heads of q and one for k's (nullable: 1)
 *   positions [tokens] int32, inv_freq [rotary_pairs] fp32 (with rotary_pairs > 0)
 *   q_out, k_out  contiguous, dtype
 * Accumulation in fp32, one rounding of each output; angles are reduced in fp64, so a
 * far position is as exact as a near one.  Squares are summed in fp32 as well: values beyond
 * 1e18, or with eps 0 rows of values below 1e-18, leave its range.  headdim up to 256, heads up
 * to 4096 each, tokens up to 2^30 (beyond: SSD_ERR_UNSUPPORTED); any alignment of the dtype's
 * size.
 * No buffer that is written may share memory with another (SSD_ERR_INVALID_ARG), but
 * strided rows may lie beside others of the same stride.  Errors as for ssd_fwd.
 */
typedef struct {
  int64_t tokens;         /* rows                                           */
  int64_t q_heads;        /* 1 to 4096                                      */
  int64_t k_heads;
  int64_t headdim;        /* D, 1 to 256                                    */
  int64_t rotary_pairs;   /* R, 2 R <= D; 0: no rotation                    */
  int64_t q_stride, k_stride;    /* elements between tokens; 0: contiguous  */
  int64_t dq_stride, dk_stride;  /* the same of dq and dk (ssd_qk_norm_bwd) */
  int32_t dtype;          /* ssd_dtype_t of q, k, the outputs and gradients */
  int32_t norm;           /* 0: by the mean of squares, 1: by their sum     */
  int32_t interleaved;    /* 0: pairs (i, i + R), 1: (2i, 2i + 1)           */
  float eps;
} ssd_qk_norm_problem_t;

ssd_status_t ssd_qk_norm_fwd(const ssd_qk_norm_problem_t* p, const void* q, const void* k,
                             const float* q_weight, const float* k_weight,
                             const int32_t* positions, const float* inv_freq, void* q_out,
                             void* k_out, void* stream);

/*
 * The backward of ssd_qk_norm_fwd: gradients of sum(q_out * dq_out) + sum(k_out * dk_out).
 * With d the output's gradient turned back, n = x r and dn = d weight:
 *
 *   dx = r (dn - n mean(dn n))   (norm 1: sum);    dweight = sum over tokens and heads of d n
 *
 * dq_out, dk_out like the outputs; dq, dk like q and k, dq_stride and dk_stride elements
 * apart (what lies between the rows is not written); dq_weight is required with a
 * q_weight and NULL without, dk_weight likewise.  The workspace (no initial contents;
 * not needed without weights) is ssd_qk_norm_bwd_workspace_size bytes, 256-byte aligned;
 * calls that may overlap need one each.  No atomics: results are deterministic.
 */
size_t ssd_qk_norm_bwd_workspace_size(const ssd_qk_norm_problem_t* p);

ssd_status_t ssd_qk_norm_bwd(const ssd_qk_norm_problem_t* p, const void* q, const void* k,
                             const float* q_weight, const float* k_weight,
                             const int32_t* positions, const float* inv_freq, const void* dq_out,
                             const void* dk_out, void* dq, void* dk, float* dq_weight,
                             float* dk_weight, void* workspace, size_t workspace_bytes,
                             void* stream);

/* Static description of a status code (library bookkeeping, not from the
 * pages). */
const char* ssd_status_string(ssd_status_t s);

#ifdef __cplusplus
}
#endif

#endif /* SSD_H_ */

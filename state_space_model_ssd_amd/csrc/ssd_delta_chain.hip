// The gated delta rule, the chain of states.  Per sequence, head and chunk, from the
// state S (P x N) entering the chunk and the chunk's T, A and decays (ssd_delta_prep.hip):
//   W = (T beta) (V - E K S^T)
//   O = scale E (Q S^T) + A W
//   S <- E_C S + (D W)^T K,     D_i = exp(G_C - G_i)
// (for the backward R = T' (V - E K S^T), W = beta R: R is kept, also where beta is 0)
// and backward, from the last chunk to the first, with dO the output's gradient, dS that of
// the state leaving the chunk and dR that of beta V - beta E K S^T, which is W's with all that
// later rows make of it:
//   dW = A^T dO + D K dS^T,   dR = T^T dW
//   dS <- E_C dS + dO^T (scale E Q) - dR^T (beta E K)
//
// Rows of S (values of the head) do not meet, so a wave owns 16 of them and carries them
// through the sequence in its registers, in fp32: S^T, W and the products between them
// chain result to operand without LDS (ssd_delta_device.h).  What the products read besides
// is the same for all of a head's rows and lies in LDS as operands.
//
// One token chunk is one step of a dependent chain, and a step is bound by the instructions
// that one wave issues.  So a workgroup has NW state waves, which do only the chain, and four
// helper waves, which move the operands from memory to LDS (through registers, a phase ahead)
// and do what nothing waits for: O, or what the backward keeps.  A step has two phases with
// a barrier after each; each half of the operands is read in one and replaced in the other,
// so one copy in LDS is enough:
//              state waves                         helper waves
//   phase 1    W by K, T, V; S and W as operands   loads of the next chunk's operands; O of the
//              to LDS                              chunk before
//   phase 2    S by K^T                            next K, T, V to LDS
// K^T is read out of K's rows by transposing reads, so bf16's K has two copies; fp32 has no such
// reads, and takes K^T from memory (ssd_delta_prep.hip).
//
// Long sequences of few heads leave most of the device idle for as long as their chains are.  They
// are cut (DeltaSplit), backward too: each segment runs once from zeros, for what it adds to a state (B), and with
// as many more rows as the state has columns from a unit matrix without values, for what becomes of
// a state (M); delta_starts_kernel makes the states that segments start from out of these; then all
// run side by side.  1x8192 tokens, 24 heads of 64 x 128: 233 -> 136 us a forward; 16 heads of 64 x 64,
// backward: 430 -> 231 us.  The packed prompts of 14371 tokens, 24 heads of 64 x 128: B and M 87, the
// states 20, the segments of 16 chunks 83 us.
//
// 4x8192 tokens, 32 heads of 128 x 128, bf16 (256 workgroups, 128 steps): 310 us in a graph, 326 with
// counters, 2.4 to 2.5 us a step.  LDS is busy for 0.47 of it, matrix instructions for 0.25, and 1.39 GB
// are read and written, 4.3 TB/s; half of the waves' time they wait to issue.  2x4096 tokens, backward:
// 129 us for the states, 185 for their gradients (3 TB/s, LDS 0.3).
#include <type_traits>

#include "ssd_delta_device.h"

#pragma clang fp contract(on)

namespace ssd {

int device_cu_count();

namespace {

constexpr int C = kDeltaChunk;
constexpr int HW = 4;                     // helper waves
constexpr int kLdsBytes = 160 * 1024;

int device_cus() { return device_cu_count() > 0 ? device_cu_count() : 256; }

// One helper wave's share of `COUNT` loads of 16 bytes per lane on their way from memory to
// LDS, through registers.  Loads are issued also where there is no next chunk (from an empty
// resource: zeros, no access): behind a branch around loads the compiler does not know how many
// are under way, and waits for all of them.
template <int COUNT> struct Pieces {
  static constexpr int n = (COUNT + HW - 1) / HW;
  uint4 q[n];
  // The i-th load of helper w; the last ones may be made twice.
  __device__ __forceinline__ static int index(int i, int w) {
    return COUNT % HW ? min(i * HW + w, COUNT - 1) : i * HW + w;
  }
};

// Operands that lie in memory as they do in LDS.
template <int COUNT> struct Copied : Pieces<COUNT> {
  __device__ __forceinline__ void load(const char* p, bool some, int w, int lane) {
    const __amdgpu_buffer_rsrc_t r = buf_rsrc(p, some ? COUNT * kPiece : 0);
#pragma unroll
    for (int i = 0; i < this->n; ++i) this->q[i] = buf_load16(r, this->index(i, w) * kPiece + lane * 16);
  }
  __device__ __forceinline__ void store(char* lds, int w, int lane) const {
#pragma unroll
    for (int i = 0; i < this->n; ++i)
      *reinterpret_cast<uint4*>(lds + this->index(i, w) * kPiece + lane * 16) = this->q[i];
  }
};

// The operands of a [C][N] matrix of T in its caller's rows, rows dealt to tiles as tile_row()
// does.  LDS has them in the order [32-block][tile].  A load takes 128 bytes of 8 rows (64 of 16
// where rows have no more): a lane per row, the operands' own order, takes four times as long to
// issue.  The exclusive or in a lane's slot keeps the eight lanes that write LDS together on
// different banks, and the sixteen of a transposing read.
template <typename T, int N> struct Rows : Pieces<4 * (N / 32) * Opnd<T>::PX> {
  static constexpr int LR = N * (int)sizeof(T) >= 128 ? 8 : 4;    // lanes on one row
  static constexpr int RL = 64 / LR, PR = N * (int)sizeof(T) / (16 * LR);
  static constexpr bool FLIP = LR == 8 && sizeof(T) == 2;
  __device__ __forceinline__ static uint32_t slot(int a, int i, int flip) {
    return (uint32_t)(16 * a + (i ^ 4 * a ^ flip)) * 16;
  }
  // A reader's slot; `flip` is 1 for the second of two pieces that share 128 bytes.
  __device__ __forceinline__ static uint32_t read(int lane, int flip) {
    return slot(lane >> 4, lane & 15, FLIP ? flip : 0);
  }
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t pitch, int w, int lane) {
#pragma unroll
    for (int i = 0; i < this->n; ++i) {
      const int x = this->index(i, w), part = x % PR, row = x / PR * RL + lane / LR;   // tile by tile
      this->q[i] = buf_load16(r, tile_row(row / 16, row % 16) * pitch + (part * LR + lane % LR) * 16);
    }
  }
  __device__ __forceinline__ void store(char* lds, int w, int lane) const {
#pragma unroll
    for (int i = 0; i < this->n; ++i) {
      const int x = this->index(i, w), part = x % PR, row = x / PR * RL + lane / LR;
      const int b = (part * LR + lane % LR) * 16;                 // byte of the row
      const int e = b / (int)sizeof(T), kb = e / 32, a = e % 32 / 8, px = e % 8 * (int)sizeof(T) / 16;
      const int flip = FLIP ? b / 64 & 1 : 0;
      const int piece = (kb * 4 + row / 16) * Opnd<T>::PX + px;
      *reinterpret_cast<uint4*>(lds + piece * kPiece + slot(a, row % 16, flip)) = this->q[i];
    }
  }
};

// The operand of the transposed matrix: rows are the channels of dealt tile u, it contracts
// tokens 32 cb + 8 (lane / 16) ...
template <int N>
__device__ __forceinline__ bf16x8 transposed_opnd(const char* lds, int cb, int u, int lane) {
  using R = Rows<bf16, N>;
  const int m = lane & 15;
  const char* p = lds + ((u >> 1) * 4 + 2 * cb) * kPiece +
                  R::slot(m & 3, 4 * (lane >> 4) + (m >> 2), R::FLIP ? u >> 1 & 1 : 0) + 8 * (u & 1);
  const i16x4 lo = lds_tr16_b64(reinterpret_cast<const bf16*>(p));
  const i16x4 hi = lds_tr16_b64(reinterpret_cast<const bf16*>(p + kPiece));
  typedef short i16x8v __attribute__((ext_vector_type(8)));
  const i16x8v v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  return __builtin_bit_cast(bf16x8, v);
}
// All tiles of it: out of the matrix's rows, or of pieces that are laid out so (fp32, for which no
// transposing read is).
template <typename T, int N>
__device__ __forceinline__ void lds_transposed(const char* lds, int cb, int lane, typename Opnd<T>::X (&x)[N / 16]) {
#pragma unroll
  for (int u = 0; u < N / 16; ++u) {
    if constexpr (sizeof(T) == 2) x[u] = transposed_opnd<N>(lds, cb, u, lane);
    else x[u] = piece_x(lds + (cb * (N / 16) + u) * Opnd<T>::PX * kPiece, lane * 16, T{});
  }
}

// A [C][16 NW] block of T, as rows in LDS: the workgroup's columns of V or dO.
template <typename T, int NW> struct Block : Pieces<NW * (int)sizeof(T)> {
  static constexpr int LR = NW * (int)sizeof(T);                  // lanes on one row
  static constexpr int pitch = 16 * NW + 16 / (int)sizeof(T);     // elements
  static constexpr int bytes = C * pitch * (int)sizeof(T);
  // `row`: bytes from token to token; `cols`: columns that there are (a multiple of 16).
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t row, int cols, int w, int lane) {
    const uint32_t at = lane % LR * 16;
#pragma unroll
    for (int i = 0; i < this->n; ++i) {
      const int c = this->index(i, w) * (64 / LR) + lane / LR;
      this->q[i] = buf_load16(r, at < cols * sizeof(T) ? c * row + at : 0xffffff00u);   // else zeros
    }
  }
  __device__ __forceinline__ void store(char* lds, int w, int lane) const {
#pragma unroll
    for (int i = 0; i < this->n; ++i) {
      const int c = this->index(i, w) * (64 / LR) + lane / LR;
      *reinterpret_cast<uint4*>(lds + c * pitch * sizeof(T) + lane % LR * 16) = this->q[i];
    }
  }
};
// Rows 32 cb + 8 (lane / 16) .. + 7 of a block's column tile_row(s, lane % 16).
template <int NW>
__device__ __forceinline__ bf16x8 column_opnd(const char* lds, int s, int cb, int lane, bf16) {
  constexpr int pitch = Block<bf16, NW>::pitch;
  const int m = lane & 15;
  const bf16* p = reinterpret_cast<const bf16*>(lds) + (32 * cb + 8 * (lane >> 4) + (m >> 2)) * pitch +
                  32 * (s >> 1) + 8 * (m & 3) + 4 * (s & 1);
  const i16x4 lo = lds_tr16_b64(p), hi = lds_tr16_b64(p + 4 * pitch);
  typedef short i16x8v __attribute__((ext_vector_type(8)));
  const i16x8v v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  return __builtin_bit_cast(bf16x8, v);
}
template <int NW>
__device__ __forceinline__ F8 column_opnd(const char* lds, int s, int cb, int lane, float) {
  constexpr int pitch = Block<float, NW>::pitch;
  F8 f;
  const float* p = reinterpret_cast<const float*>(lds) + (32 * cb + 8 * (lane >> 4)) * pitch + tile_row(s, lane & 15);
#pragma unroll
  for (int e = 0; e < 8; ++e) f.v[e] = p[e * pitch];
  return f;
}

// M operands in a row from `p` on.
template <int M, typename T>
__device__ __forceinline__ void lds_xs(const char* p, uint32_t slot, typename Opnd<T>::X (&x)[M]) {
#pragma unroll
  for (int m = 0; m < M; ++m) x[m] = piece_x(p + m * Opnd<T>::PX * kPiece, slot, T{});
}
template <int M, typename T>
__device__ __forceinline__ void lds_ss(const char* p, uint32_t slot, typename Opnd<T>::S (&x)[M]) {
#pragma unroll
  for (int m = 0; m < M; ++m) x[m] = piece_s(p + m * Opnd<T>::PS * kPiece, slot, T{});
}

// Values 32 cb + 8 (lane / 16) .. + 7 of a row of C floats.
__device__ __forceinline__ void row8(const float* p, int cb, int lane, float (&f)[8]) {
  p += 32 * cb + 8 * (lane >> 4);
  block8(*reinterpret_cast<const f32x4*>(p), *reinterpret_cast<const f32x4*>(p + 4), f);
}

// Bytes from the first of n rows to the end of the last one's `row` bytes.
__device__ __forceinline__ uint32_t rows_bytes(int n, uint32_t pitch, uint32_t row) {
  return n > 0 ? (uint32_t)(n - 1) * pitch + row : 0u;
}

// Workgroup -> (sequence, head) and its block of P: the blocks of one head, which read the
// same operands, run on the same XCD.
struct ChainTask {
  int seq, h, g, block;
  bool none;
  int first, tokens;      // the tokens of the sequence, or of its segment
  int c0, chunks;         // and chunks
  int slot, part, parts;  // the segment's slot; which of the sequence's it is, and of how many
  __device__ __forceinline__ ChainTask(const DeltaArgs& a, const ChunkMap& cm, int b, int blocks) {
    const int x8 = b & 7, rest = b >> 3, unit = rest / blocks * 8 + x8;
    slot = unit / a.H;
    h = unit % a.H;
    g = h / (a.H / a.G);
    block = rest % blocks;
    const DeltaSplit& sp = a.split;
    none = unit >= (sp.slots ? sp.slots : a.nstates) * a.H;
    if (none) return;
    const int length = sp.slots ? sp.length() : 0;
    const int2 seg = sp.slots ? sp.segment(cm, a.nstates, length, slot) : make_int2(slot, 0);
    seq = seg.x;
    const int2 r = cm.seq_range(seq);
    c0 = r.x;
    chunks = r.y - r.x;
    if (a.cu) {           // as the chunk table's launch reads them
      first = min(max(a.cu[seq], 0), a.total);
      tokens = min(max(a.cu[seq + 1], first), a.total) - first;
    } else {
      first = seq * a.seqlen;
      tokens = a.seqlen;
    }
    part = 0;
    parts = 1;
    if (!sp.slots) return;
    int per;
    DeltaSplit::cut(chunks, length, parts, per);
    part = seg.y;
    none = part >= parts;
    c0 += part * per;
    first += part * per * C;
    tokens = part + 1 < parts ? per * C : tokens - part * per * C;
    chunks = part + 1 < parts ? per : chunks - part * per;
  }
  __device__ __forceinline__ int start(int i) const { return first + i * C; }
  __device__ __forceinline__ int len(int i) const { return i < 0 ? 0 : min(C, tokens - i * C); }
};

// S^T in its tiles from row p of a state, zeros where there is none; of a unit matrix; and back.
template <int N>
__device__ __forceinline__ void load_state(const float* row, bool in, int lane, f32x4 (&S)[N / 16]) {
#pragma unroll
  for (int kb = 0; kb < N / 32; ++kb) {
    const float* r = row + 32 * kb + 8 * (lane >> 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      S[2 * kb][e] = in ? r[e] : 0.f;
      S[2 * kb + 1][e] = in ? r[4 + e] : 0.f;
    }
  }
}
template <int N>
__device__ __forceinline__ void unit_state(int row, int la, f32x4 (&S)[N / 16]) {
#pragma unroll
  for (int i = 0; i < N / 16; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) S[i][e] = 32 * (i / 2) + 8 * la + 4 * (i % 2) + e == row ? 1.f : 0.f;
}
template <int N>
__device__ __forceinline__ void store_state(float* row, int lane, const f32x4 (&S)[N / 16]) {
#pragma unroll
  for (int kb = 0; kb < N / 32; ++kb) {
    float* r = row + 32 * kb + 8 * (lane >> 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      r[e] = S[2 * kb][e];
      r[4 + e] = S[2 * kb + 1][e];
    }
  }
}

// A lane's place in the kb-th operand that a state wave leaves: LeftRows reads one row's
// pieces together, and the exclusive or puts them on different banks.
__device__ __forceinline__ uint32_t left_slot(int a, int i, int kb) {
  return (uint32_t)(16 * a + (i ^ ((a + 4 * kb) & 15))) * 16;
}

// Operands that the state waves left in LDS ([wave][LEFT pieces], from the `from`-th piece on, each
// 32 columns of 16 dealt rows) to rows of a [P][COLS] matrix of T, or of two, one behind the other.
template <typename T, int NW, int LEFT, int COLS, bool PAIR> struct LeftRows {
  static constexpr int PX = Opnd<T>::PX, PL = kPlanes<T, PAIR>, V = 16 / (int)sizeof(T), PR = COLS / V;
  static constexpr int all = 16 * NW * PR, n = (all + 64 * HW - 1) / (64 * HW);
  uint4 q[n][PL];
  __device__ __forceinline__ static int place(int i, int w, int lane) { return (i * HW + w) * 64 + lane; }
  __device__ __forceinline__ void load(const char* x, int from, int w, int lane) {
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const int at = all % (64 * HW) ? min(place(i, w, lane), all - 1) : place(i, w, lane), p = at / PR, c = at % PR * V;
      const int s = 2 * (p / 32) + (p / 4 & 1), l16 = p % 32 / 8 * 4 + p % 4;
      const int kb = c / 32, a = c % 32 / 8, px = c % 8 / V;
#pragma unroll
      for (int pl = 0; pl < PL; ++pl)
        q[i][pl] = *reinterpret_cast<const uint4*>(x + (s * LEFT + from + kb * PX * PL + pl + px) * kPiece + left_slot(a, l16, kb));
    }
  }
  // To the first of `rows` rows at dst; planes `plane` elements apart.
  __device__ __forceinline__ void store(T* dst, int64_t plane, int rows, int w, int lane) const {
#pragma unroll
    for (int pl = 0; pl < PL; ++pl) {
      const __amdgpu_buffer_rsrc_t r = buf_rsrc(dst + pl * plane, rows * COLS * sizeof(T));   // no row past the end
#pragma unroll
      for (int i = 0; i < n; ++i)
        if (all % (64 * HW) == 0 || place(i, w, lane) < all) buf_store16(r, place(i, w, lane) * 16, q[i][pl]);
    }
  }
};

enum class Chain { fwd, keep, ends, bwd, bwd_ends };

// keep: for the backward, S and R are kept (PAIR: as pairs, else rounded) and O is not made.
// ends: neither; what a segment makes of a state of zeros (the first one of the initial state),
// and, by rows of their own past P's, of a unit matrix without values.
template <typename T, int N, int NW, Chain K, bool PAIR>
__global__ __launch_bounds__(64 * (NW + HW)) void delta_chain_kernel(const DeltaArgs a, const ChunkMap cm,
                                                                      int blocks) {
  constexpr bool KEEP = K == Chain::keep, ENDS = K == Chain::ends;
  using O = Opnd<T>;
  using KR = Rows<T, N>;
  using VB = Block<T, NW>;
  constexpr int NK = N / 32, NT = N / 16, PX = O::PX, PS = O::PS, TP = NT * 2 * PX, EX = NK + 2;
  constexpr int PE = PX * kPlanes<T, PAIR>;       // pieces of what is kept
  constexpr int LEFT = EX * PE;                   // and of all that a state wave leaves
  // K is read in both phases where it is transposed on the way: two copies
  constexpr bool TR = sizeof(T) == 2;
  constexpr int kK = 4 * NK * PX * kPiece, oK = 0, oT = oK + (TR ? 2 : 1) * kK, oG = oT + 6 * PS * kPiece;
  constexpr int QS = sizeof(T) == 2 ? NK : 1;     // 32-blocks of Q that a helper's corner takes
  constexpr int oV = oG + kPiece, oKt = oV + VB::bytes, oQ = oKt + (TR ? 0 : TP * kPiece);
  constexpr int oX = oQ + (K == Chain::fwd ? HW * QS * PX * kPiece : 0), kX = ENDS ? 0 : NW * LEFT * kPiece;
  constexpr bool DX = oX + 2 * kX <= kLdsBytes;   // two copies of what the state waves leave
  __shared__ __attribute__((aligned(16))) char lds[oX + (DX ? 2 : 1) * kX];

  if (ENDS && a.split.length() == 0) return;
  const ChainTask t(a, cm, blockIdx.x, blocks);
  if (t.none || (ENDS && t.part + 1 == t.parts)) return;
  // ends: the unit matrix's rows, of all segments but the first
  const int valued = (a.P + 16 * NW - 1) / (16 * NW);
  const bool unit = ENDS && t.block >= valued;
  if (unit && t.part == 0) return;
  const int wave = wave_id(), lane = threadIdx.x & 63, l16 = lane & 15, la = lane >> 4;
  const int h = t.h, p0 = (unit ? t.block - valued : t.block) * 16 * NW;
  const int rows = min(16 * NW, (unit ? N : a.P) - p0);
  const float* gt = reinterpret_cast<const float*>(lds + oG);

  if (wave < NW) {
    const int p = tile_row(wave, l16);
    const int64_t srow = (((int64_t)t.seq * a.H + h) * a.P + p0 + p) * N;
    const uint32_t rs = lane * 16, rk[2] = {KR::read(lane, 0), KR::read(lane, 1)};
    f32x4 S[NT];
    const float* from = a.init + srow;
    bool some = a.init && p < rows;
    if (ENDS && t.part > 0) some = false;
    if (!ENDS && t.part > 0) {
      from = a.split.starts + (((int64_t)t.slot * a.H + h) * a.P + p0 + p) * N;
      some = p < rows;
    }
    load_state<N>(from, some, lane, S);
    if (unit) unit_state<N>(p0 + p, la, S);
    __syncthreads();
    for (int j = 0; j < t.chunks; ++j) {
      // phase 1
      const char* kl = lds + oK + (TR && (j & 1) ? kK : 0);
      typename O::S sf[NK], rf[2];
      typename O::X kf[NK][4];
      float v[2][8], E[2][8], D[2][8];
#pragma unroll
      for (int kb = 0; kb < NK; ++kb) lds_xs<4, T>(kl + kb * 4 * PX * kPiece, rk[kb % 2], kf[kb]);
#pragma unroll
      for (int cb = 0; cb < 2; ++cb) {
        O::get(column_opnd<NW>(lds + oV, wave, cb, lane, T{}), v[cb]);
        row8(gt + C, cb, lane, E[cb]);
        row8(gt + 2 * C, cb, lane, D[cb]);
      }
      const float EC = gt[2 * C - 1];
      f32x4 y[4] = {kZero4, kZero4, kZero4, kZero4};
#pragma unroll
      for (int kb = 0; kb < NK; ++kb) {
        float f[8];
        block8(S[2 * kb], S[2 * kb + 1], f);
        sf[kb] = O::split(f);
        mma_rows(kf[kb], sf[kb], y);
      }
      typename O::S t0[4], t1[2];
      lds_ss<4, T>(lds + oT, rs, t0);
      lds_ss<2, T>(lds + oT + 4 * PS * kPiece, rs, t1);
#pragma unroll
      for (int cb = 0; cb < 2; ++cb) {
        float f[8];
        block8(y[2 * cb], y[2 * cb + 1], f);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = v[cb][e] - E[cb][e] * f[e];
        rf[cb] = O::split(f);
      }
      y[0] = y[1] = y[2] = y[3] = kZero4;
      mma_rows(t0, rf[0], y);
      mma_rows(t1, rf[1], y + 2);
      char* x = lds + oX + ((DX && (j & 1) ? NW : 0) + wave) * LEFT * kPiece;
#pragma unroll
      for (int kb = 0; kb < (ENDS ? 0 : NK); ++kb) put_piece(x + kb * PE * kPiece, left_slot(la, l16, kb), keep<T, PAIR>(sf[kb]));
#pragma unroll
      for (int cb = 0; cb < 2; ++cb) {
        float f[8];
        block8(y[2 * cb], y[2 * cb + 1], f);
        if constexpr (!ENDS) put_piece(x + (NK + cb) * PE * kPiece, left_slot(la, l16, cb), keep<T, PAIR>(f));
        if (KEEP || (ENDS && a.back)) {           // R to W
          float b[8];
          row8(gt, cb, lane, b);
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] *= b[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= D[cb][e];
        rf[cb] = O::split(f);
      }
#pragma unroll
      for (int i = 0; i < NT; ++i) S[i] *= EC;
      __syncthreads();
      // phase 2
#pragma unroll
      for (int cb = 0; cb < 2; ++cb) {
        typename O::X f[NT];
        lds_transposed<T, N>(TR ? kl : lds + oKt, cb, lane, f);
        mma_rows(f, rf[cb], S);
      }
      __syncthreads();
    }
    if (ENDS && p < rows)
      store_state<N>(a.split.ends + (((int64_t)t.slot * a.H + h) * (a.P + N) + (unit ? a.P : 0) + p0 + p) * N, lane, S);
    if (K == Chain::fwd && a.final_states && t.part + 1 == t.parts && p < rows)
      store_state<N>(a.final_states + srow, lane, S);
    return;
  }

  const int w = wave - NW;                        // helper
  const uint32_t qrow = (uint32_t)a.G * N * sizeof(T), vrow = (uint32_t)a.H * a.P * sizeof(T);
  KR cK;
  Copied<6 * PS> cT;
  VB cV;
  uint4 cG;
  Copied<TP> cKt;
  // the next chunk's in memory
  const int64_t jh0 = (int64_t)t.c0 * a.H + h, jg0 = (int64_t)t.c0 * a.G + t.g;
  const char* kp = static_cast<const char*>(a.k) + ((int64_t)t.first * a.G + t.g) * N * sizeof(T);
  const char* qp = static_cast<const char*>(a.q) + ((int64_t)t.first * a.G + t.g) * N * sizeof(T);
  const char* vp = static_cast<const char*>(a.v) + (((int64_t)t.first * a.H + h) * a.P + p0) * sizeof(T);
  const char* Tp = static_cast<const char*>(a.T) + jh0 * (6 * PS * kPiece);
  const char* Ap = static_cast<const char*>(a.A) + jh0 * (6 * PX * kPiece);
  const char* gp = reinterpret_cast<const char*>(a.gates + jh0 * kGateFloats);
  const char* tp = static_cast<const char*>(a.kt) + jg0 * (TP * kPiece);
  auto fetch1 = [&](int j) {                      // no row past the last chunk
    const bool some = j < t.chunks;
    cK.load(buf_rsrc(kp, rows_bytes(t.len(j), qrow, N * sizeof(T))), qrow, w, lane);
    cT.load(Tp, some, w, lane);
    cV.load(buf_rsrc(vp, unit ? 0 : rows_bytes(t.len(j), vrow, rows * sizeof(T))), vrow, rows, w, lane);
    cG = buf_load16(buf_rsrc(gp, some ? kGateFloats * 4 : 0), lane * 16);
    kp += C * (int64_t)qrow;
    vp += C * (int64_t)vrow;
    Tp += a.H * (6 * PS * kPiece);
    gp += a.H * (kGateFloats * 4);
  };
  auto put1 = [&](int j) {
    cK.store(lds + oK + (TR && (j & 1) ? kK : 0), w, lane);
    cT.store(lds + oT, w, lane);
    cV.store(lds + oV, w, lane);
    if (w == 0) *reinterpret_cast<uint4*>(lds + oG + lane * 16) = cG;
  };
  // helper w makes the outputs of tokens 16 w ..: their rows of Q, four lanes on 64 bytes, and
  // of A, as operands
  uint4 cQ[NK * PX], cA[2][PX];
  auto fetch2 = [&](int j) {
    const bool some = j < t.chunks;
    if constexpr (!TR) {
      cKt.load(tp, some, w, lane);
      tp += a.G * (TP * kPiece);
    }
    if constexpr (K == Chain::fwd) {
      const __amdgpu_buffer_rsrc_t qr = buf_rsrc(qp, rows_bytes(t.len(j), qrow, N * sizeof(T)));
      const __amdgpu_buffer_rsrc_t ar = buf_rsrc(Ap, some ? 6 * PX * kPiece : 0);
#pragma unroll
      for (int i = 0; i < NK * PX; ++i) cQ[i] = buf_load16(qr, (16 * w + lane / 4) * qrow + (4 * i + lane % 4) * 16);
      // the second of tokens before 32 is none: past the resource
#pragma unroll
      for (int cb = 0; cb < 2; ++cb)
#pragma unroll
        for (int i = 0; i < PX; ++i)
          cA[cb][i] = buf_load16(ar, cb == 0 || w >= 2 ? (triangle_index(w, cb) * PX + i) * kPiece + lane * 16 : 0xffffff00u);
      qp += C * (int64_t)qrow;
      Ap += a.H * (6 * PX * kPiece);
    }
  };
  typename O::X qf[NK], af[2];
  float sE = 0.f;
  // what chunk j's products with Q need besides S and W; the rows of Q to operand order in the
  // wave's own corner of LDS (the exclusive or as for Rows)
  auto ready = [&]() {
    if constexpr (K == Chain::fwd) {
      char* q = lds + oQ + w * QS * PX * kPiece;
#pragma unroll
      for (int k0 = 0; k0 < NK; k0 += QS) {
        wave_sync();
#pragma unroll
        for (int kb = 0; kb < QS; ++kb)
#pragma unroll
          for (int i = 0; i < PX; ++i) {
            const int e = (4 * i + lane % 4) * 16 / (int)sizeof(T), px = e % 8 * (int)sizeof(T) / 16;
            *reinterpret_cast<uint4*>(q + (kb * PX + px) * kPiece + KR::slot(e / 8, lane / 4, 0)) = cQ[(k0 + kb) * PX + i];
          }
        wave_sync();
#pragma unroll
        for (int kb = 0; kb < QS; ++kb) qf[k0 + kb] = piece_x(q + kb * PX * kPiece, KR::slot(la, l16, 0), T{});
      }
      sE = a.scale * gt[C + 16 * w + l16];
      af[0] = opnd_of(cA[0], T{});
      af[1] = opnd_of(cA[1], T{});
    }
  };
  // O with S and W as first operands: rows are values, the lane's column is a token
  f32x4 o[NW];
  auto product = [&](int j) {
    if constexpr (K == Chain::fwd) {
      const char* x = lds + oX + (DX && (j & 1) ? kX : 0);
#pragma unroll
      for (int s = 0; s < NW; ++s) o[s] = kZero4;
      // all loads from LDS before their first use: one after another each would wait in its queue
      typename O::X f[EX][NW];
#pragma unroll
      for (int kb = 0; kb < EX; ++kb)
#pragma unroll
        for (int s = 0; s < NW; ++s)
          f[kb][s] = piece_x(x + (s * EX + kb) * PX * kPiece, left_slot(la, l16, kb < NK ? kb : kb - NK), T{});
      if constexpr (sizeof(T) == 2) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int kb = 0; kb < NK; ++kb) mma_rows(f[kb], qf[kb], o);
#pragma unroll
      for (int s = 0; s < NW; ++s) o[s] *= sE;
      mma_rows(f[NK], af[0], o);
      if (w >= 2) mma_rows(f[NK + 1], af[1], o);
    }
  };
  auto write = [&](int j) {
    if constexpr (KEEP) {
      const char* x = lds + oX + (DX && (j & 1) ? kX : 0);
      const int64_t jh = jh0 + (int64_t)j * a.H;
      LeftRows<T, NW, LEFT, N, PAIR> ls;
      LeftRows<T, NW, LEFT, C, PAIR> lr;
      constexpr int PL = kPlanes<T, PAIR>;
      ls.load(x, 0, w, lane);
      lr.load(x, NK * PE, w, lane);
      ls.store(static_cast<T*>(a.S0) + (jh * PL * a.P + p0) * N, (int64_t)a.P * N, rows, w, lane);
      lr.store(static_cast<T*>(a.Rt) + (jh * PL * a.P + p0) * C, a.P * C, rows, w, lane);
    } else if constexpr (K == Chain::fwd) {
      const int c = 16 * w + l16;
      T* out = static_cast<T*>(a.out) + ((int64_t)(t.start(j) + c) * a.H + h) * a.P + p0 + 8 * la;
#pragma unroll
      for (int s = 0; s < NW; s += 2) {
        float f[8];
        block8(o[s], o[s + 1], f);
        if (c < t.len(j) && 16 * s + 8 * la < rows) store_opnd(out + 16 * s, O::round(f));
      }
    }
  };
  if (t.chunks > 0) {
    fetch1(0);
    put1(0);
    fetch2(0);
  }
  __syncthreads();
  for (int j = 0; j < t.chunks; ++j) {
    // phase 1; stores come last, as whoever waits for a load waits for the stores before it
    fetch1(j + 1);
    if constexpr (!TR) cKt.store(lds + oKt, w, lane);
    if (DX && j > 0) product(j - 1);
    ready();
    fetch2(j + 1);
    if (DX && j > 0) write(j - 1);
    __syncthreads();
    // phase 2
    if constexpr (!DX) {
      product(j);
      write(j);
    }
    put1(j + 1);
    __syncthreads();
  }
  if (DX && t.chunks > 0) {
    product(t.chunks - 1);
    write(t.chunks - 1);
  }
}

// Backward: dS (before the update; PAIR: as pairs) and dR (as pairs) are kept for ssd_delta_local.hip.
// ENDS: neither; what a segment makes of a gradient of zeros (the last one of the final state's),
// and, by rows past P's, of a unit matrix without outputs' gradients.
template <typename T, int N, int NW, bool ENDS, bool PAIR>
__global__ __launch_bounds__(64 * (NW + HW)) void delta_chain_bwd_kernel(const DeltaArgs a, const ChunkMap cm,
                                                                          int blocks) {
  using O = Opnd<T>;
  using KR = Rows<T, N>;
  using VB = Block<T, NW>;
  constexpr int NK = N / 32, NT = N / 16, PX = O::PX, PS = O::PS, TP = NT * 2 * PX;
  // pieces of an operand of dS and of dR as they are left, and of all that a state wave leaves
  constexpr int ES = PX * kPlanes<T, PAIR>, ER = PX * kPlanes<T, true>, LEFT = NK * ES + 2 * ER;
  // as above; Q, which is read transposed only, lies in rows or transposed
  constexpr bool TR = sizeof(T) == 2;
  constexpr int kK = 4 * NK * PX * kPiece, oK = 0, oA = oK + (TR ? 2 : 1) * kK, oT = oA + 6 * PS * kPiece;
  constexpr int oG = oT + 6 * PS * kPiece, oV = oG + kPiece, oQt = oV + VB::bytes, oKt = oQt + TP * kPiece;
  constexpr int oX = oKt + (TR ? 0 : TP * kPiece);
  constexpr int kX = ENDS ? 0 : NW * LEFT * kPiece;
  constexpr bool DX = oX + 2 * kX <= kLdsBytes;
  __shared__ __attribute__((aligned(16))) char lds[oX + (DX ? 2 : 1) * kX];

  const ChainTask t(a, cm, blockIdx.x, blocks);
  if (t.none || (ENDS && t.part == 0)) return;
  const int valued = (a.P + 16 * NW - 1) / (16 * NW);
  const bool unit = ENDS && t.block >= valued, first = t.part + 1 == t.parts;   // the first to run
  if (unit && first) return;
  const int wave = wave_id(), lane = threadIdx.x & 63, l16 = lane & 15, la = lane >> 4;
  const int h = t.h, p0 = (unit ? t.block - valued : t.block) * 16 * NW;
  const int rows = min(16 * NW, (unit ? N : a.P) - p0);
  const float* gt = reinterpret_cast<const float*>(lds + oG);

  if (wave < NW) {
    const int p = tile_row(wave, l16);
    const int64_t srow = (((int64_t)t.seq * a.H + h) * a.P + p0 + p) * N;
    const uint32_t rs = lane * 16, rk[2] = {KR::read(lane, 0), KR::read(lane, 1)};
    f32x4 S[NT];
    const float* from = a.dfinal + srow;
    bool some = a.dfinal && p < rows;
    if (ENDS && !first) some = false;
    if (!ENDS && !first) {
      from = a.split.starts + (((int64_t)t.slot * a.H + h) * a.P + p0 + p) * N;
      some = p < rows;
    }
    load_state<N>(from, some, lane, S);
    if (unit) unit_state<N>(p0 + p, la, S);
    __syncthreads();
    for (int j = t.chunks - 1; j >= 0; --j) {
      // phase 1
      const char* K = lds + oK + (TR && (j & 1) ? kK : 0);
      typename O::S sf[NK], rf[2], qf[2], t0[2], t1[4];   // t: the upper triangle's tiles of cb 0, of cb 1
      typename O::X kf[NK][4], of[2];
      float D[2][8], E[2][8], bE[2][8];
#pragma unroll
      for (int kb = 0; kb < NK; ++kb) lds_xs<4, T>(K + kb * 4 * PX * kPiece, rk[kb % 2], kf[kb]);
#pragma unroll
      for (int cb = 0; cb < 2; ++cb) {
        of[cb] = column_opnd<NW>(lds + oV, wave, cb, lane, T{});
        row8(gt + 2 * C, cb, lane, D[cb]);
        row8(gt + C, cb, lane, E[cb]);
        row8(gt + 3 * C, cb, lane, bE[cb]);
      }
      const float EC = gt[2 * C - 1];
      f32x4 y[4] = {kZero4, kZero4, kZero4, kZero4};
#pragma unroll
      for (int kb = 0; kb < NK; ++kb) {
        float f[8];
        block8(S[2 * kb], S[2 * kb + 1], f);
        sf[kb] = O::split(f);
        mma_rows(kf[kb], sf[kb], y);
      }
      lds_ss<2, T>(lds + oA, rs, t0);
      lds_ss<4, T>(lds + oA + 2 * PS * kPiece, rs, t1);
#pragma unroll
      for (int cb = 0; cb < 2; ++cb) {
        float o[8];
        O::get(of[cb], o);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] *= a.scale * E[cb][e];
        qf[cb] = O::split(o);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          y[2 * cb][e] *= D[cb][e];
          y[2 * cb + 1][e] *= D[cb][4 + e];
        }
      }
      mma_rows(t0, of[0], y);
      mma_rows(t1, of[1], y);
      lds_ss<2, T>(lds + oT, rs, t0);
      lds_ss<4, T>(lds + oT + 2 * PS * kPiece, rs, t1);
#pragma unroll
      for (int cb = 0; cb < 2; ++cb) {
        float f[8];
        block8(y[2 * cb], y[2 * cb + 1], f);
        rf[cb] = O::split(f);
      }
      y[0] = y[1] = y[2] = y[3] = kZero4;
      mma_rows(t0, rf[0], y);
      mma_rows(t1, rf[1], y);
      char* x = lds + oX + ((DX && (j & 1) ? NW : 0) + wave) * LEFT * kPiece;
#pragma unroll
      for (int kb = 0; kb < (ENDS ? 0 : NK); ++kb) put_piece(x + kb * ES * kPiece, left_slot(la, l16, kb), keep<T, PAIR>(sf[kb]));
#pragma unroll
      for (int cb = 0; cb < 2; ++cb) {
        float f[8];
        block8(y[2 * cb], y[2 * cb + 1], f);
        if constexpr (!ENDS) put_piece(x + (NK * ES + cb * ER) * kPiece, left_slot(la, l16, cb), keep<T, true>(f));
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= -bE[cb][e];
        rf[cb] = O::split(f);
      }
#pragma unroll
      for (int i = 0; i < NT; ++i) S[i] *= EC;
      __syncthreads();
      // phase 2
#pragma unroll
      for (int cb = 0; cb < 2; ++cb) {
        typename O::X f[NT];
        lds_transposed<T, N>(lds + oQt, cb, lane, f);
        mma_rows(f, qf[cb], S);
        lds_transposed<T, N>(TR ? K : lds + oKt, cb, lane, f);
        mma_rows(f, rf[cb], S);
      }
      __syncthreads();
    }
    if (ENDS && p < rows)
      store_state<N>(a.split.ends + (((int64_t)t.slot * a.H + h) * (a.P + N) + (unit ? a.P : 0) + p0 + p) * N, lane, S);
    if (!ENDS && a.dinit && t.part == 0 && p < rows) store_state<N>(a.dinit + srow, lane, S);
    return;
  }

  const int w = wave - NW;                        // helper
  const uint32_t qrow = (uint32_t)a.G * N * sizeof(T), vrow = (uint32_t)a.H * a.P * sizeof(T);
  KR cK;
  Copied<6 * PS> cA, cT;
  VB cV;
  uint4 cG;
  std::conditional_t<TR, KR, Copied<TP>> cQt;
  Copied<TP> cKt;
  // the next chunk's in memory (the first one's is the last)
  const int last = t.chunks - 1;
  const int64_t jh0 = (int64_t)t.c0 * a.H + h, jh1 = jh0 + (int64_t)last * a.H;
  const int64_t jg1 = ((int64_t)t.c0 + last) * a.G + t.g, tok = t.first + (int64_t)last * C;
  const char* kp = static_cast<const char*>(a.k) + (tok * a.G + t.g) * N * sizeof(T);
  const char* qp = static_cast<const char*>(a.q) + (tok * a.G + t.g) * N * sizeof(T);
  const char* vp = static_cast<const char*>(a.dout) + ((tok * a.H + h) * a.P + p0) * sizeof(T);
  const char* Ap = static_cast<const char*>(a.At) + jh1 * (6 * PS * kPiece);
  const char* Tp = static_cast<const char*>(a.Tt) + jh1 * (6 * PS * kPiece);
  const char* gp = reinterpret_cast<const char*>(a.gates + jh1 * kGateFloats);
  int64_t tp = jg1 * (TP * kPiece);
  auto fetch1 = [&](int j) {
    const bool some = j >= 0;
    cK.load(buf_rsrc(kp, rows_bytes(t.len(j), qrow, N * sizeof(T))), qrow, w, lane);
    cA.load(Ap, some, w, lane);
    cT.load(Tp, some, w, lane);
    cV.load(buf_rsrc(vp, unit ? 0 : rows_bytes(t.len(j), vrow, rows * sizeof(T))), vrow, rows, w, lane);
    cG = buf_load16(buf_rsrc(gp, some ? kGateFloats * 4 : 0), lane * 16);
    kp -= C * (int64_t)qrow;
    vp -= C * (int64_t)vrow;
    Ap -= a.H * (6 * PS * kPiece);
    Tp -= a.H * (6 * PS * kPiece);
    gp -= a.H * (kGateFloats * 4);
  };
  auto put1 = [&](int j) {
    cK.store(lds + oK + (TR && (j & 1) ? kK : 0), w, lane);
    cA.store(lds + oA, w, lane);
    cT.store(lds + oT, w, lane);
    cV.store(lds + oV, w, lane);
    if (w == 0) *reinterpret_cast<uint4*>(lds + oG + lane * 16) = cG;
  };
  auto fetch2 = [&](int j) {
    if constexpr (TR) {
      cQt.load(buf_rsrc(qp, rows_bytes(t.len(j), qrow, N * sizeof(T))), qrow, w, lane);
      qp -= C * (int64_t)qrow;
    } else {
      cQt.load(static_cast<const char*>(a.qt) + tp, j >= 0, w, lane);
      cKt.load(static_cast<const char*>(a.kt) + tp, j >= 0, w, lane);
      tp -= a.G * (TP * kPiece);
    }
  };
  auto finish = [&](int j) {
    const char* x = lds + oX + (DX && (j & 1) ? kX : 0);
    const int64_t jh = jh0 + (int64_t)j * a.H;
    LeftRows<T, NW, LEFT, N, PAIR> ls;
    LeftRows<T, NW, LEFT, C, true> lr;
    ls.load(x, 0, w, lane);
    lr.load(x, NK * ES, w, lane);
    ls.store(static_cast<T*>(a.dS) + (jh * kPlanes<T, PAIR> * a.P + p0) * N, (int64_t)a.P * N, rows, w, lane);
    lr.store(static_cast<T*>(a.dRt) + (jh * kPlanes<T, true> * a.P + p0) * C, a.P * C, rows, w, lane);
  };
  if (t.chunks > 0) {
    fetch1(last);
    put1(last);
    fetch2(last);
  }
  __syncthreads();
  for (int j = last; j >= 0; --j) {
    // phase 1
    fetch1(j - 1);
    cQt.store(lds + oQt, w, lane);
    if constexpr (!TR) cKt.store(lds + oKt, w, lane);
    fetch2(j - 1);
    if (!ENDS && DX && j < last) finish(j + 1);
    __syncthreads();
    // phase 2
    if constexpr (!ENDS && !DX) finish(j);
    put1(j - 1);
    __syncthreads();
  }
  if (!ENDS && DX && t.chunks > 0) finish(0);
}

// The states entering each segment but the first, from what the segments make of a state of zeros
// (B) and of a unit matrix (M):  S_1 = B_0,  S_(i+1) = S_i M_i + B_i.  BACK: their gradients, from
// the last segment on.
//
// A workgroup has 16 rows of a head's state, a wave 16 columns; by fp32 matrix instructions.
// M and B of the next segment are on their way while one is used.
template <int N, bool BACK>
__global__ __launch_bounds__(4 * N) void delta_starts_kernel(const DeltaArgs a, const ChunkMap cm) {
  constexpr int pitch = N + 4;
  __shared__ float row[2][16 * pitch];
  const int length = a.split.length();
  if (length == 0) return;
  const int nb = a.P / 16, p0 = (int)(blockIdx.x % nb) * 16, sh = blockIdx.x / nb, h = sh % a.H, seq = sh / a.H;
  const int2 r = cm.seq_range(seq);
  int parts, per;
  DeltaSplit::cut(r.y - r.x, length, parts, per);
  if (parts < 2) return;
  const int others = a.split.others(cm, a.nstates, length, seq);
  auto slot = [&](int i) {                        // of the i-th to run
    const int part = BACK ? parts - 1 - i : i;
    return (int64_t)(part == 0 ? seq : others + part - 1);
  };
  const int lane = threadIdx.x & 63, l16 = lane & 15, la = lane >> 4, col = 16 * wave_id() + l16;
  struct Next {
    float m[N / 4], b[4];
  };
  auto load = [&](Next& n, int i) {
    const float* B = a.split.ends + (slot(i) * a.H + h) * (a.P + N) * N + col;
    const float* M = B + (int64_t)a.P * N;
#pragma unroll
    for (int e = 0; e < 4; ++e) n.b[e] = B[(p0 + 4 * la + e) * N];
    if (i == 0) return;                           // of the first one there is no M
#pragma unroll
    for (int k = 0; k < N / 4; ++k) n.m[k] = M[(4 * k + la) * N];
  };
  auto step = [&](Next& now, Next& next, int i) {
    if (i + 2 < parts) load(next, i + 1);
    f32x4 c = {now.b[0], now.b[1], now.b[2], now.b[3]};
    if (i > 0) {
      const float* x = row[i & 1] + l16 * pitch + la;
      f32x4 c1 = kZero4;                          // two sums: a product waits for the one before it
#pragma unroll
      for (int k = 0; k < N / 4; k += 2) {
        c = __builtin_amdgcn_mfma_f32_16x16x4f32(x[4 * k], now.m[k], c, 0, 0, 0);
        c1 = __builtin_amdgcn_mfma_f32_16x16x4f32(x[4 * k + 4], now.m[k + 1], c1, 0, 0, 0);
      }
      c += c1;
    }
    float* to = a.split.starts + ((slot(i + 1) * a.H + h) * a.P + p0) * N + col;
    float* y = row[(i + 1) & 1] + col;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      to[(4 * la + e) * N] = c[e];
      y[(4 * la + e) * pitch] = c[e];
    }
    __syncthreads();
  };
  Next even, odd;
  load(even, 0);
  for (int i = 0; i + 1 < parts; i += 2) {
    step(even, odd, i);
    if (i + 2 < parts) step(odd, even, i + 1);
  }
}

template <Chain K, typename T, int N, int NW, bool PAIR>
hipError_t chain_go(const DeltaArgs& a, hipStream_t s) {
  constexpr bool ends = K == Chain::ends || K == Chain::bwd_ends;
  const int blocks = (a.P + 16 * NW - 1) / (16 * NW) + (ends ? (N + 16 * NW - 1) / (16 * NW) : 0);
  const int64_t units = (int64_t)(a.split.slots ? a.split.slots : a.nstates) * a.H;
  const dim3 grid((unsigned)((units + 7) / 8 * 8 * blocks)), th(64 * (NW + HW));
  if constexpr (K == Chain::bwd || K == Chain::bwd_ends)
    hipLaunchKernelGGL((delta_chain_bwd_kernel<T, N, NW, ends, PAIR>), grid, th, 0, s, a, a.cmap(), blocks);
  else
    hipLaunchKernelGGL((delta_chain_kernel<T, N, NW, K, PAIR>), grid, th, 0, s, a, a.cmap(), blocks);
  return hipGetLastError();
}

// Two state waves where heads have no more rows, where fp32 operands of dstate 128 leave LDS for
// no more, and where four would leave half the device idle (200 tokens of 32 heads of 128 x 128:
// 26.8 us a forward with two, 28.9 with four; 2x4096 tokens, backward 581 and 623; 4x8192 tokens,
// which fill the device with four, 563 and 445).
int state_waves(const DeltaArgs& a) {
  if (a.split.slots && a.split.block) return a.split.block / 16;    // as the estimate of segments has it
  const int64_t units = (int64_t)(a.split.slots ? a.split.slots : a.nstates) * a.H * ((a.P + 63) / 64);
  return a.P <= 32 || (!a.bf16 && a.N == 128) || 2 * units <= device_cus() ? 2 : 4;
}

template <Chain K, typename T, bool PAIR>
hipError_t chain_n(const DeltaArgs& a, hipStream_t s) {
  constexpr int most = sizeof(T) == 4 ? 2 : 4;    // dstate 128
  if (state_waves(a) == 2) {
    switch (a.N) {
      case 32: return chain_go<K, T, 32, 2, PAIR>(a, s);
      case 64: return chain_go<K, T, 64, 2, PAIR>(a, s);
      case 128: return chain_go<K, T, 128, 2, PAIR>(a, s);
    }
  }
  switch (a.N) {
    case 32: return chain_go<K, T, 32, 4, PAIR>(a, s);
    case 64: return chain_go<K, T, 64, 4, PAIR>(a, s);
    case 128: return chain_go<K, T, 128, most, PAIR>(a, s);
  }
  return hipErrorInvalidValue;
}

template <Chain K>
hipError_t chain_type(const DeltaArgs& a, hipStream_t s) {
  if (a.nstates <= 0) return hipSuccess;
  if (!a.bf16) return chain_n<K, float, false>(a, s);
  if constexpr (K == Chain::keep || K == Chain::bwd)
    if (a.pairs) return chain_n<K, bf16, true>(a, s);
  return chain_n<K, bf16, false>(a, s);
}

template <bool BACK>
hipError_t starts(const DeltaArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)(a.nstates * a.H * (a.P / 16))), th(4 * a.N);
  switch (a.N) {
    case 32: hipLaunchKernelGGL((delta_starts_kernel<32, BACK>), grid, th, 0, s, a, a.cmap()); break;
    case 64: hipLaunchKernelGGL((delta_starts_kernel<64, BACK>), grid, th, 0, s, a, a.cmap()); break;
    case 128: hipLaunchKernelGGL((delta_starts_kernel<128, BACK>), grid, th, 0, s, a, a.cmap()); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

// The segments' length of equal rows; a packed batch's is in memory by now.
void settle(DeltaArgs& a) {
  if (!a.split.slots || a.cu) return;
  DeltaSplit::Sums v = {};
  v.add(a.split, a.nc_row, a.nstates);
  a.split.fixed = DeltaSplit::best(a.split, v, a.max_chunks, a.H, a.P, a.N, a.split.block, device_cus());
  int parts, per;
  DeltaSplit::cut(a.nc_row, a.split.fixed, parts, per);
  a.split.per_row = parts;
  a.split.slots = parts > 1 ? a.nstates * parts : 0;
}

}  // namespace

int delta_chain_rows(const DeltaArgs& a) { return 16 * state_waves(a); }

hipError_t launch_delta_chain(const DeltaArgs& given, bool keep, hipStream_t s) {
  DeltaArgs a = given;
  hipError_t e = hipSuccess;
  settle(a);
  if (a.split.slots) {
    e = chain_type<Chain::ends>(a, s);
    if (e == hipSuccess) e = starts<false>(a, s);
  }
  if (e != hipSuccess) return e;
  return keep ? chain_type<Chain::keep>(a, s) : chain_type<Chain::fwd>(a, s);
}
hipError_t launch_delta_chain_bwd(const DeltaArgs& given, hipStream_t s) {
  DeltaArgs a = given;
  hipError_t e = hipSuccess;
  settle(a);
  if (a.split.slots) {
    e = chain_type<Chain::bwd_ends>(a, s);
    if (e == hipSuccess) e = starts<true>(a, s);
  }
  return e == hipSuccess ? chain_type<Chain::bwd>(a, s) : e;
}

}  // namespace ssd

// The gated delta rule's backward inside each chunk, from what the two chains left
// (ssd_delta_chain.hip): the state S entering the chunk, the gradient dS of the state
// leaving it, the rows R and the gradient dR of W = beta R.  With A, D, E as there, and
//   P = tril(dO W^T) * D,   M = -tril(dR W^T, -1) * D   (the gradients of q k^T and, per beta, k k^T)
// the gradients are
//   dq = scale (E dO S + P K)
//   X  = M K - E dR S,    dbeta = dR.R,    dv = beta dR
//   dk = beta X + scale P^T Q + D_C W dS + (beta M)^T K
// (dbeta is dR.v + k.X as well, but that adds what R is the sum of: where keys are alike, each
// of up to 64 rows W brings its own rounding, and dbeta was off by 9.7e-3 for 2.3e-3, 2112 tokens.)
// and that of the log decay of token i sums what crosses it:
//   dg_i = sum over pairs c >= i > c' of (P scale q k^T + M beta k k^T)_cc'
//        + sum_{c >= i} (scale E q.(dO S) - beta E k.(dR S))_c  + sum_{c < i} (k.(D_C W dS))_c
//        + E_C <dS, S>
// (pairs by a running sum of column less row sums).  Spelled as k and q times their own
// gradients it would be shorter, but those cancel: a first token's is exactly zero.
//
// One workgroup per chunk and group; it walks over the group's heads, so dq and dk are
// summed over them in registers.  Waves w and w + 4 have tokens 16 w .. as the second operand's
// columns throughout: their results are columns of their own tokens, dot products with q and k
// are sums over a lane's rows, and P and M go into the next product as they lie.  The first of
// the two makes P and M of its tokens' rows, the second P^T and M^T (products of their own, not
// exchanged over tokens); they swap these through LDS, and each has half of dq's and dk's
// channels.  The axis of values is walked in slabs of 32, whose R, dR, S and dS lie in LDS with
// the values as rows (read transposed) and whose dO as operands; beta joins R in the results; the next slabs' loads are in
// flight meanwhile, also those of the next head.
//
// 2x4096 tokens, 32 heads in 16 groups of 128 x 128, bf16: 244 us for 747 MB (3.1 TB/s); S and dS as
// pairs too 337.  LDS is busy for 0.31 of it, matrix instructions for 0.14; 256 registers and 133 KB
// of LDS leave room for one workgroup on a CU, so nothing else runs while its waves wait.
#include "ssd_delta_device.h"

#pragma clang fp contract(on)

namespace ssd {

namespace {

constexpr int C = kDeltaChunk;
constexpr int kLocalThreads = 512;
constexpr int kSlab = 32;

// [kSlab][COLS] tiles in LDS and the operands that contract their rows.
template <typename T, int COLS> struct Tile;
template <int COLS> struct Tile<bf16, COLS> {
  static constexpr int size = kSlab * COLS;
  __device__ __forceinline__ static bf16* piece(bf16* t, int r, int c) { return t + tile_at<COLS>(r, c); }
  __device__ __forceinline__ static bf16x8 at(const bf16* t, int r, int c) {
    const bf16* p = t + tile_at<COLS>(r, c);
    const i16x4 lo = lds_tr16_b64(p), hi = lds_tr16_b64(p + 4 * COLS);
    typedef short i16x8v __attribute__((ext_vector_type(8)));
    const i16x8v v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_bit_cast(bf16x8, v);
  }
  // columns of dealt tile u; of 16 neighbouring columns from c0
  __device__ __forceinline__ static bf16x8 dealt(const bf16* t, int u, int lane) {
    const int m = lane & 15;
    return at(t, 8 * (lane >> 4) + (m >> 2), 32 * (u >> 1) + 8 * (m & 3) + 4 * (u & 1));
  }
  __device__ __forceinline__ static bf16x8 plain(const bf16* t, int c0, int lane) {
    const int m = lane & 15;
    return at(t, 8 * (lane >> 4) + (m >> 2), c0 + 4 * (m & 3));
  }
};
template <int COLS> struct Tile<float, COLS> {
  static constexpr int pitch = COLS + 4, size = kSlab * pitch;
  __device__ __forceinline__ static float* piece(float* t, int r, int c) { return t + r * pitch + c; }
  __device__ __forceinline__ static F8 at(const float* t, int lane, int c) {
    F8 f;
#pragma unroll
    for (int e = 0; e < 8; ++e) f.v[e] = t[(8 * (lane >> 4) + e) * pitch + c];
    return f;
  }
  __device__ __forceinline__ static F8 dealt(const float* t, int u, int lane) {
    return at(t, lane, tile_row(u, lane & 15));
  }
  __device__ __forceinline__ static F8 plain(const float* t, int c0, int lane) {
    return at(t, lane, c0 + (lane & 15));
  }
};

__device__ __forceinline__ float dot16(uint4 x, uint4 y, bf16) {
  const bf16x8 a = __builtin_bit_cast(bf16x8, x), b = __builtin_bit_cast(bf16x8, y);
  float s = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) s += static_cast<float>(a[e]) * static_cast<float>(b[e]);
  return s;
}
__device__ __forceinline__ float dot16(uint4 x, uint4 y, float) {
  const f32x4 a = __builtin_bit_cast(f32x4, x), b = __builtin_bit_cast(f32x4, y);
  return a[0] * b[0] + a[1] * b[1] + a[2] * b[2] + a[3] * b[3];
}
// The same of a tile kept as two, high parts and low parts.
template <typename T, int COLS, bool PAIR>
__device__ __forceinline__ typename Kept<T, PAIR>::V kept_dealt(const T* t, int u, int lane) {
  using TT = Tile<T, COLS>;
  if constexpr (kPlanes<T, PAIR> == 2) return {TT::dealt(t, u, lane), TT::dealt(t + TT::size, u, lane)};
  else return TT::dealt(t, u, lane);
}
template <typename T, int COLS, bool PAIR>
__device__ __forceinline__ typename Kept<T, PAIR>::V kept_plain(const T* t, int c0, int lane) {
  using TT = Tile<T, COLS>;
  if constexpr (kPlanes<T, PAIR> == 2) return {TT::plain(t, c0, lane), TT::plain(t + TT::size, c0, lane)};
  else return TT::plain(t, c0, lane);
}
template <typename T, bool PAIR>
__device__ __forceinline__ void kept_get(const typename Kept<T, PAIR>::V& v, float (&f)[8]) {
  if constexpr (kPlanes<T, PAIR> == 2) {
    float lo[8];
    Opnd<T>::get(v.hi, f);
    Opnd<T>::get(v.lo, lo);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] += lo[e];
  } else {
    Opnd<T>::get(v, f);
  }
}

// A [kSlab][COLS] tile on its way from memory to LDS, through the registers of THREADS threads;
// zeros in rows that there are not.
template <typename T, int COLS, int THREADS> struct Slab {
  static constexpr int V = 16 / (int)sizeof(T), PR = COLS / V, all = kSlab * PR;
  static constexpr int n = (all + THREADS - 1) / THREADS;
  uint4 q[n];
  __device__ __forceinline__ void load(const T* src, int rows, int tid) {
    const __amdgpu_buffer_rsrc_t r = buf_rsrc(src, (uint32_t)(max(rows, 0) * COLS) * (uint32_t)sizeof(T));
#pragma unroll
    for (int i = 0; i < n; ++i) q[i] = buf_load16(r, (i * THREADS + tid) * 16);
  }
  __device__ __forceinline__ void store(T* t, int tid) const {
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const int at = i * THREADS + tid;
      if (all % THREADS == 0 || at < all)
        *reinterpret_cast<uint4*>(Tile<T, COLS>::piece(t, at / PR, at % PR * V)) = q[i];
    }
  }
};

// Tokens' [C][COLS] values as operands: the four dealt tiles of rows of each 32 columns, in
// Opnd<T>::PX pieces; the exclusive or keeps lanes that write together on different banks.
template <typename T, int COLS, int THREADS> struct Tokens {
  static constexpr int PX = Opnd<T>::PX, PR = COLS / 8 * PX, all = C * PR;
  static constexpr int n = (all + THREADS - 1) / THREADS;
  static constexpr int bytes = COLS / 32 * 4 * PX * kPiece;
  uint4 q[n];
  __device__ __forceinline__ static uint32_t slot(int a, int i) { return (uint32_t)(16 * a + (i ^ 4 * a)) * 16; }
  // A row's first columns, of PR * 16 bytes.
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t pitch, int tid) {
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const int at = i * THREADS + tid;
      q[i] = buf_load16(r, all % THREADS == 0 || at < all ? at / PR * pitch + at % PR * 16 : 0xffffff00u);
    }
  }
  __device__ __forceinline__ void store(char* t, int tid) const {
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const int at = i * THREADS + tid, c = at / PR, x = at % PR, y = x % (4 * PX);
      if (all % THREADS == 0 || at < all)
        *reinterpret_cast<uint4*>(t + ((x / (4 * PX) * 4 + tile_of(c)) * PX + y % PX) * kPiece + slot(y / PX, row_of(c))) = q[i];
    }
  }
  __device__ __forceinline__ static int tile_of(int c) { return 2 * (c / 32) + (c / 4 & 1); }
  __device__ __forceinline__ static int row_of(int c) { return c % 32 / 8 * 4 + c % 4; }
  // 32 columns kb of dealt tile u's rows, or of token c (lane % 16 of 16 neighbours).
  __device__ __forceinline__ static typename Opnd<T>::X dealt(const char* t, int kb, int u, int lane) {
    return piece_x(t + (kb * 4 + u) * PX * kPiece, slot(lane >> 4, lane & 15), T{});
  }
  __device__ __forceinline__ static typename Opnd<T>::X token(const char* t, int kb, int c, int lane) {
    return piece_x(t + (kb * 4 + tile_of(c)) * PX * kPiece, slot(lane >> 4, row_of(c)), T{});
  }
  // Tokens 32 cb + 8 (lane / 16) .. + 7 of the channels of dealt tile u: the transposed operand.
  __device__ __forceinline__ static bf16x8 transposed(const char* t, int cb, int u, int lane) {
    static_assert(sizeof(T) == 2, "reads that transpose are of 16 bits");
    const int m = lane & 15, n = 8 * (m & 3) + 4 * (u & 1);   // of 32 channels u / 2
    const uint32_t at = slot(n / 8, 4 * (lane >> 4) + (m >> 2)) + 2 * (n % 8);
    const char* p = t + ((u >> 1) * 4 + 2 * cb) * kPiece + at;
    const i16x4 lo = lds_tr16_b64(reinterpret_cast<const bf16*>(p));
    const i16x4 hi = lds_tr16_b64(reinterpret_cast<const bf16*>(p + kPiece));
    typedef short i16x8v __attribute__((ext_vector_type(8)));
    const i16x8v v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_bit_cast(bf16x8, v);
  }
};

// An operand's lanes (row l % 16, columns 8 (l / 16) ..) in the order of rows: lane l has row l / 4,
// columns 8 (l % 4) ...
template <typename V>
__device__ __forceinline__ V by_rows(V v, int lane) {
  constexpr int n = sizeof(V) / 4;
  int q[n];
  __builtin_memcpy(q, &v, sizeof(V));
#pragma unroll
  for (int i = 0; i < n; ++i) q[i] = __builtin_amdgcn_ds_bpermute(((lane & 3) * 16 + lane / 4) * 4, q[i]);
  __builtin_memcpy(&v, q, sizeof(V));
  return v;
}

// What a slab needs from memory.  The first waves' threads take R, the others dR.
template <typename T, int N, int PL> struct Loads {
  Slab<T, C, kLocalThreads / 2> r[kPlanes<T, true>];
  Slab<T, N, kLocalThreads> s[PL], d[PL];
  Tokens<T, kSlab, kLocalThreads> o;              // dO
};

__device__ __forceinline__ double buf_load_double(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(double, __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 0));
}

__device__ __forceinline__ void store_gate(void* p, bool b16, int64_t i, float v) {
  if (b16) static_cast<bf16*>(p)[i] = static_cast<bf16>(v);
  else static_cast<float*>(p)[i] = v;
}

// The four of an operand's eight values that lie at the rows of its first tile, or of its second.
template <typename T>
__device__ __forceinline__ f32x4 channels4(const typename Opnd<T>::X& x, bool second) {
  float a[8];
  Opnd<T>::get(x, a);
  const f32x4 lo = {a[0], a[1], a[2], a[3]}, hi = {a[4], a[5], a[6], a[7]};
  return second ? hi : lo;
}

// dR comes as pairs; PAIR: S, dS and R too.
template <typename T, int N, bool PAIR>
__global__ __launch_bounds__(kLocalThreads) void delta_local_bwd_kernel(const DeltaArgs a, const ChunkMap cm) {
  using O = Opnd<T>;
  using X = typename O::X;
  using TC = Tile<T, C>;
  using TN = Tile<T, N>;
  using TS = Tokens<T, kSlab, kLocalThreads>;
  using TK = Tokens<T, N, kLocalThreads>;
  constexpr int NK = N / 32, NH = N / 32, PX = O::PX;   // NH: a wave's tiles of dq and dk
  using KV = typename Kept<T, PAIR>::V;
  using KG = typename Kept<T, true>::V;           // of dR
  constexpr int PL = kPlanes<T, PAIR>, PG = kPlanes<T, true>;
  constexpr int BUF = sizeof(T) == 2 && !PAIR ? 2 : 1;  // slabs in LDS
  // k and q of the chunk lie there too, where the slabs leave room
  constexpr bool KQ = sizeof(T) == 2 || N < 128;
  __shared__ __attribute__((aligned(16))) T Rs[BUF][PL * TC::size], dRs[BUF][PG * TC::size];
  __shared__ __attribute__((aligned(16))) T Ss[BUF][PL * TN::size], Ds[BUF][PL * TN::size];
  __shared__ __attribute__((aligned(16))) char dOs[BUF][TS::bytes], swap[4 * 8 * PX * kPiece];
  __shared__ __attribute__((aligned(16))) char kqs[KQ ? 2 * TK::bytes : 16];
  __shared__ double Gs[C];
  __shared__ float bs[C], left[2][C], mid[2][C], dbs[C], sdots[kLocalThreads / 64];
  const int2 jg = xcd_chunk_head(blockIdx.x, a.G);
  const int j = jg.x, g = jg.y, rep = a.H / a.G;
  if (j >= a.max_chunks) return;
  const ChunkDesc d = cm.desc(j);
  if (d.len <= 0) return;
  const int wave = wave_id(), w = wave & 3, half = wave >> 2;
  const uint32_t qrow = (uint32_t)a.G * N * sizeof(T), vrow = (uint32_t)a.H * a.P * sizeof(T);
  const int64_t qo = ((int64_t)d.start * a.G + g) * N;
  const uint32_t qbytes = (uint32_t)(d.len - 1) * qrow + N * sizeof(T);
  const __amdgpu_buffer_rsrc_t qr = buf_rsrc(static_cast<const T*>(a.q) + qo, qbytes);
  const __amdgpu_buffer_rsrc_t kr = buf_rsrc(static_cast<const T*>(a.k) + qo, qbytes);
  const int64_t tr = ((int64_t)j * a.G + g) * (N / 16 * 2) * PX * kPiece;   // fp32
  const char* kt = static_cast<const char*>(a.kt) + tr;
  const char* qt = static_cast<const char*>(a.qt) + tr;

  if constexpr (KQ) {
    TK sk, sq;
    sk.load(kr, qrow, threadIdx.x);
    sq.load(qr, qrow, threadIdx.x);
    sk.store(kqs, threadIdx.x);
    sq.store(kqs + TK::bytes, threadIdx.x);       // read after the slabs' barriers
  }
  f32x4 dq[NH], dk[NH];
#pragma unroll
  for (int i = 0; i < NH; ++i) dq[i] = dk[i] = kZero4;
  // slabs in flight
  constexpr int AHEAD = sizeof(T) == 2 && !PAIR ? 2 : 1;
  Loads<T, N, PL> next[AHEAD];
  float gates[5];
  double Gt = 0.0;
  float bt = 0.f;
  // head h's slab from p0 (none past the group's last head or the last value)
  auto fetch = [&](Loads<T, N, PL>& q, int h, int p0, int tid) {
    const int rows = h < (g + 1) * rep ? a.P - p0 : 0;
    const int64_t jh = (int64_t)j * a.H + h, vo = ((int64_t)d.start * a.H + h) * a.P;
#pragma unroll
    for (int i = 0; i < PG; ++i)                  // a resource of no bytes where R has no low part
      q.r[i].load(static_cast<const T*>(half ? a.dRt : a.Rt) + ((jh * (half ? PG : PL) + i) * a.P + p0) * C,
                  half || i < PL ? min(rows, kSlab) : 0, tid & (kLocalThreads / 2 - 1));
#pragma unroll
    for (int i = 0; i < PL; ++i) {
      const int64_t at = (jh * PL + i) * a.P + p0;
      q.s[i].load(static_cast<const T*>(a.S0) + at * N, min(rows, kSlab), tid);
      q.d[i].load(static_cast<const T*>(a.dS) + at * N, min(rows, kSlab), tid);
    }
    const __amdgpu_buffer_rsrc_t r = buf_rsrc(static_cast<const T*>(a.dout) + vo, rows > 0 ? (uint32_t)(d.len - 1) * vrow + a.P * (uint32_t)sizeof(T) : 0);
    const uint32_t cols = a.P * (uint32_t)sizeof(T), col = p0 * (uint32_t)sizeof(T);
#pragma unroll
    for (int i = 0; i < TS::n; ++i) {
      const int at = i * kLocalThreads + tid;
      const uint32_t b = col + at % TS::PR * 16;
      q.o.q[i] = buf_load16(r, at < TS::all && b < cols ? at / TS::PR * vrow + b : 0xffffff00u);
    }
  };
  // head h's decays
  auto fetch_gates = [&](int h, int tid) {
    const __amdgpu_buffer_rsrc_t r = buf_rsrc(a.gates + ((int64_t)j * a.H + h) * kGateFloats, h < (g + 1) * rep ? kGateFloats * 4 : 0);
    const uint32_t c = 16 * w + (tid & 15);
    gates[0] = buf_load4(r, 4 * c);
    gates[1] = buf_load4(r, 4 * (C + c));
    gates[2] = buf_load4(r, 4 * (2 * C + c));
    gates[3] = buf_load4(r, 4 * (2 * C - 1));
    gates[4] = buf_load4(r, 4 * (16 * w + (tid & 63) / 4));
    Gt = buf_load_double(r, 4 * 4 * C + 8 * (tid & (C - 1)));
    bt = buf_load4(r, 4 * (tid & (C - 1)));
  };
  {
    const int tid = opaque_tid();
    fetch_gates(g * rep, tid);
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) fetch(next[i], g * rep, i * kSlab, tid);
  }

  for (int h = g * rep; h < (g + 1) * rep; ++h) {
    // through opaque_tid, or every address below would be kept from head to head
    const int tid = opaque_tid(), lane = tid & 63, l16 = lane & 15, la = lane >> 4;
    const int c = 16 * w + l16;                   // the lane's token
    // 32 channels kb of dealt tile u's or of the lane's token's k or q
    auto dealt = [&](bool q, int kb, int u) {
      if constexpr (KQ) return TK::dealt(kqs + (q ? TK::bytes : 0), kb, u, lane);
      else return load_opnd(q ? qr : kr, tile_row(u, l16) * qrow + (32 * kb + 8 * la) * (uint32_t)sizeof(T), T{});
    };
    auto token = [&](bool q, int kb) {
      if constexpr (KQ) return TK::token(kqs + (q ? TK::bytes : 0), kb, c, lane);
      else return load_opnd(q ? qr : kr, c * qrow + (32 * kb + 8 * la) * (uint32_t)sizeof(T), T{});
    };
    const int64_t vo = ((int64_t)d.start * a.H + h) * a.P;
    if (tid < C) {
      Gs[tid] = Gt;
      bs[tid] = bt;
    }
    const float be = gates[0], E = gates[1], bD = be * gates[2], EC = gates[3], br = gates[4];

    f32x4 Px[4], Lx[4];                           // [c'][c] of P's and M's sources, or of their transposes
#pragma unroll
    for (int u = 0; u < 4; ++u) Px[u] = Lx[u] = kZero4;
    f32x4 yq[NH], yx[NH], yd[NH];
#pragma unroll
    for (int i = 0; i < NH; ++i) yq[i] = yx[i] = yd[i] = kZero4;
    float sdot = 0.f, db = 0.f;
    auto slab = [&](Loads<T, N, PL>& q, int p0, int b) {
      if constexpr (BUF == 1) __syncthreads();    // the slab before is read
#pragma unroll
      for (int i = 0; i < PG; ++i)
        if (half || i < PL) q.r[i].store((half ? dRs[b] : Rs[b]) + i * TC::size, tid & (kLocalThreads / 2 - 1));
#pragma unroll
      for (int i = 0; i < PL; ++i) {
        q.s[i].store(Ss[b] + i * TN::size, tid);
        q.d[i].store(Ds[b] + i * TN::size, tid);
      }
      q.o.store(dOs[b], tid);
#pragma unroll
      for (int i = 0; i < Slab<T, N, kLocalThreads>::n; ++i) {
        sdot += dot16(q.s[0].q[i], q.d[0].q[i], T{});
        if constexpr (PL == 2) sdot += dot16(q.s[0].q[i], q.d[1].q[i], T{}) + dot16(q.s[1].q[i], q.d[0].q[i], T{});
      }
      __syncthreads();
      const KV ro = kept_plain<T, C, PAIR>(Rs[b], 16 * w, lane);
      const KG go = kept_plain<T, C, true>(dRs[b], 16 * w, lane);
      const X od = TS::token(dOs[b], 0, c, lane);
      if (half == 0) {
        float r8[8], g8[8];
        kept_get<T, PAIR>(ro, r8);
        kept_get<T, true>(go, g8);
#pragma unroll
        for (int e = 0; e < 8; ++e) db += r8[e] * g8[e];
        // dR in the order of rows, four lanes each, as dv goes: one lane a row would issue four
        // times slower
        kept_get<T, true>(by_rows(go, lane), g8);
#pragma unroll
        for (int e = 0; e < 8; ++e) g8[e] *= br;
        const int at = p0 + 8 * (lane & 3), tok = 16 * w + lane / 4;
        if (at < a.P && tok < d.len) store_opnd(static_cast<T*>(a.dv) + vo + (int64_t)tok * a.H * a.P + at, O::round(g8));
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int cb = 0; cb < 2; ++cb) {
        if (half ? cb < w / 2 : cb > w / 2) continue;   // no pairs there
        if (half) {
          X f[2];
          KG r[2];
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            f[t] = TS::dealt(dOs[b], 0, 2 * cb + t, lane);
            r[t] = kept_dealt<T, C, true>(dRs[b], 2 * cb + t, lane);
          }
          mma_rows(f, ro, Px + 2 * cb);
          mma_rows(r, ro, Lx + 2 * cb);
        } else {
          KV r[2];
#pragma unroll
          for (int t = 0; t < 2; ++t) r[t] = kept_dealt<T, C, PAIR>(Rs[b], 2 * cb + t, lane);
          mma_rows(r, od, Px + 2 * cb);
          mma_rows(r, go, Lx + 2 * cb);
        }
      }
      fetch(q, h, p0 + AHEAD * kSlab, tid);
      __builtin_amdgcn_sched_barrier(0);
      {
        KV f[NH];
#pragma unroll
        for (int i = 0; i < NH; ++i) f[i] = kept_dealt<T, N, PAIR>(Ss[b], half * NH + i, lane);
        mma_rows(f, od, yq);
        mma_rows(f, go, yx);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < NH; ++i) f[i] = kept_dealt<T, N, PAIR>(Ds[b], half * NH + i, lane);
        mma_rows(f, ro, yd);
      }
    };
    for (int p0 = 0; p0 < a.P; p0 += AHEAD * kSlab) {
      slab(next[0], p0, 0);
      if constexpr (AHEAD == 2)
        if (p0 + kSlab < a.P) slab(next[1], p0 + kSlab, BUF - 1);
    }
    __builtin_amdgcn_sched_barrier(0);            // what follows needs the registers of the slabs' loads
    X ko[NK], qn[NK];                             // the token's k and q
#pragma unroll
    for (int kb = 0; kb < NK; ++kb) {
      ko[kb] = token(false, kb);
      qn[kb] = token(true, kb);
    }
    // P and M, or their transposes, and their part of the pairs' sums.  A pair's term is the same
    // number as row and as column, so that what crosses no token cancels.
    float pairs = 0.f;
    {
      char* x = swap + (w * 8 + half * 4) * PX * kPiece;
#pragma unroll
      for (int cb = 0; cb < 2; ++cb) {
        float p8[8] = {}, m8[8] = {};
        // 32 tokens that make no pair with the wave's, later ones or earlier ones: zeros
        if (half ? cb < w / 2 : cb > w / 2) {
          put_piece(x + cb * PX * kPiece, lane * 16, O::round(p8));
          put_piece(x + (2 + cb) * PX * kPiece, lane * 16, O::round(m8));
          continue;
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int u = 2 * cb + t;
          f32x4 qk = kZero4, kk = kZero4;
#pragma unroll
          for (int kb = 0; kb < NK; ++kb) {
            const X k = dealt(false, kb, u), f = half ? dealt(true, kb, u) : k;
            kk = mma(k, ko[kb], kk);
            qk = mma(f, half ? ko[kb] : qn[kb], qk);
          }
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int e = 4 * t + r, o = 32 * cb + 8 * la + e;
            const int hi = half ? o : c, lo = half ? c : o;       // the pair's later and earlier token
            const float bo = bs[o], D = (half ? be : bo) * fexp<T>((float)(Gs[hi] - Gs[lo]));    // of use where lo <= hi
            const float p = lo <= hi ? Px[u][r] * D * a.scale : 0.f;
            const float m = lo < hi ? -Lx[u][r] * D : 0.f, mb = m * (half ? bo : be);
            const float term = lo < hi ? p * qk[r] + mb * kk[r] : 0.f;
            pairs += half ? term : -term;
            p8[e] = p;
            m8[e] = half ? mb : m;
          }
          __builtin_amdgcn_sched_barrier(0);
        }
        put_piece(x + cb * PX * kPiece, lane * 16, O::round(p8));
        put_piece(x + (2 + cb) * PX * kPiece, lane * 16, O::round(m8));
      }
    }
    // the row sums that need the states' products alone
    float ql = 0.f, kx = 0.f, kd = 0.f;
    X kh, qh;
#pragma unroll
    for (int i = 0; i < NH; ++i) {
      // the wave's tiles are half NH + i of the token's channels
      if (i % 2 == 0) {
        kh = token(false, (half * NH + i) / 2);
        qh = token(true, (half * NH + i) / 2);
      }
      const f32x4 k4 = channels4<T>(kh, NH >= 2 ? i % 2 : half), q4 = channels4<T>(qh, NH >= 2 ? i % 2 : half);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        ql += q4[r] * yq[i][r];
        kx += k4[r] * yx[i][r];
        kd += k4[r] * yd[i][r];
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    // the next head's first slabs on their way
    fetch_gates(h + 1, tid);
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) fetch(next[i], h + 1, i * kSlab, tid);
    __syncthreads();
    X pr[2], mr[2], pc[2], mc[2];
    {
      const char* x = swap + w * 8 * PX * kPiece;
#pragma unroll
      for (int cb = 0; cb < 2; ++cb) {
        pr[cb] = piece_x(x + cb * PX * kPiece, lane * 16, T{});
        mr[cb] = piece_x(x + (2 + cb) * PX * kPiece, lane * 16, T{});
        pc[cb] = piece_x(x + (4 + cb) * PX * kPiece, lane * 16, T{});
        mc[cb] = piece_x(x + (6 + cb) * PX * kPiece, lane * 16, T{});
      }
    }
#pragma unroll
    for (int i = 0; i < NH; ++i) {
      f32x4 q = yq[i] * (a.scale * E), x = yx[i] * -E, k = yd[i] * bD;
#pragma unroll
      for (int cb = 0; cb < 2; ++cb) {
        X kf, qf;
        if constexpr (sizeof(T) == 2) {
          kf = TK::transposed(kqs, cb, half * NH + i, lane);
          qf = TK::transposed(kqs + TK::bytes, cb, half * NH + i, lane);
        } else {
          const int at = (cb * (N / 16) + half * NH + i) * PX * kPiece;
          kf = piece_x(kt + at, lane * 16, T{});
          qf = piece_x(qt + at, lane * 16, T{});
        }
        q = mma(kf, pr[cb], q);
        x = mma(kf, mr[cb], x);
        k = mma(qf, pc[cb], k);
        k = mma(kf, mc[cb], k);
      }
      dq[i] += q;
      dk[i] += k + x * be;
      if (i % 2) __builtin_amdgcn_sched_barrier(0);
    }
    db = column_sum(db);
    const float lf = column_sum(a.scale * E * ql - be * E * kx), md = column_sum(bD * kd + pairs);
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) sdot += __shfl_xor(sdot, off);
    if (la == 0) {
      left[half][c] = lf;
      mid[half][c] = md;
      if (half == 0) dbs[c] = db;
    }
    if (lane == 0) sdots[wave] = sdot;
    __syncthreads();
    if (wave == 0) {
      // sums over the tokens from this one on, and over those before it
      double s = (double)left[0][63 - lane] + left[1][63 - lane], b = (double)mid[0][lane] + mid[1][lane];
      const double own = b;
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const double x = __shfl_up(s, off), y = __shfl_up(b, off);
        if (lane >= off) {
          s += x;
          b += y;
        }
      }
      s = __shfl(s, 63 - lane);
      double sd = 0.0;
#pragma unroll
      for (int i = 0; i < kLocalThreads / 64; ++i) sd += sdots[i];
      if (lane < d.len) {
        const int64_t at = (int64_t)(d.start + lane) * a.H + h;
        store_gate(a.dg, a.gate_bf16, at, (float)(s + (b - own) + EC * sd));
        store_gate(a.dbeta, a.gate_bf16, at, dbs[lane]);
      }
    }
  }
  const int la = (threadIdx.x & 63) >> 4, c = 16 * w + (threadIdx.x & 15);
  if (c < d.len) {
    // a lane has channels 8 la .. of a 32-block: all eight in two tiles, or four (dstate 32)
    const int64_t at = qo + (int64_t)c * a.G * N;
    T* pq = static_cast<T*>(a.dq) + at;
    T* pk = static_cast<T*>(a.dk) + at;
    if constexpr (NH >= 2) {
#pragma unroll
      for (int i = 0; i < NH; i += 2) {
        float f[8];
        const int n = 32 * ((half * NH + i) / 2) + 8 * la;
        block8(dq[i], dq[i + 1], f);
        store_opnd(pq + n, O::round(f));
        block8(dk[i], dk[i + 1], f);
        store_opnd(pk + n, O::round(f));
      }
    } else {
      T f[4], e[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        f[r] = from_f32<T>(dq[0][r]);
        e[r] = from_f32<T>(dk[0][r]);
      }
      __builtin_memcpy(pq + 8 * la + 4 * half, f, sizeof(f));
      __builtin_memcpy(pk + 8 * la + 4 * half, e, sizeof(e));
    }
  }
}

template <typename T, bool PAIR>
hipError_t local_type(const DeltaArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)xcd_grid(a.max_chunks, a.G)), th(kLocalThreads);
  switch (a.N) {
    case 32: hipLaunchKernelGGL((delta_local_bwd_kernel<T, 32, PAIR>), grid, th, 0, s, a, a.cmap()); break;
    case 64: hipLaunchKernelGGL((delta_local_bwd_kernel<T, 64, PAIR>), grid, th, 0, s, a, a.cmap()); break;
    case 128: hipLaunchKernelGGL((delta_local_bwd_kernel<T, 128, PAIR>), grid, th, 0, s, a, a.cmap()); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_local_bwd(const DeltaArgs& a, hipStream_t s) {
  if (a.max_chunks <= 0) return hipSuccess;
  if (!a.bf16) return local_type<float, false>(a, s);
  return a.pairs ? local_type<bf16, true>(a, s) : local_type<bf16, false>(a, s);
}

}  // namespace ssd

// How the gated delta rule cuts long sequences (internal; host code may include it too).
#pragma once

#ifdef __HIPCC__
#define SSD_SPLIT_FN __host__ __device__ __forceinline__
#define SSD_SPLIT_UNROLL _Pragma("unroll")
#else
#define SSD_SPLIT_FN inline
#define SSD_SPLIT_UNROLL
#endif

namespace ssd {

// How long sequences are cut where they would keep few CUs busy for long: the chain of a sequence
// is one chunk after another, but its segments' chains run side by side, once each for what the
// segment makes of a state of zeros and of a unit matrix, and once more from the states that
// follow from these (ssd_delta_chain.hip).
struct DeltaCut {
  static constexpr int kLengths = 6;     // segments of least, 2 least, 4 least, .. chunks
  static constexpr int kOverhead = 6;    // what the additional launches take, in chunks' steps
  int least;              // chunks of the shortest segments

  // Segments of `per` chunks, at most `length`, for a sequence of n.
  SSD_SPLIT_FN static void cut(int n, int length, int& parts, int& per) {
    parts = 1;
    per = n;
    if (length <= 0 || n < 2 * length) return;
    parts = (n + length - 1) / length;
    per = (n + parts - 1) / parts;
    parts = (n + per - 1) / per;
  }
  // Slots of a packed batch's segments: sequence seq of n has slot seq for its first (or only) one,
  // and from others() on slots for the rest.  One of c chunks has no more than c / length of these,
  // so there is room for them behind those of the chunks before it, `first` in number.
  SSD_SPLIT_FN static int others(int n, int length, int first) { return n + first / length; }
  // The sequence and segment of a slot; no segment that the sequence has: none has the slot.
  // `first(seq)`: the chunks before a sequence.
  template <typename F> SSD_SPLIT_FN static void segment(int n, int length, int slot, F first, int& seq, int& part) {
    seq = slot < n ? slot : 0;
    part = slot < n ? 0 : 1 << 30;
    if (slot < n || length <= 0) return;
    int hi = n - 1;                      // the last sequence whose others are not behind this slot
    while (seq < hi) {
      const int mid = (seq + hi + 1) >> 1;
      if (others(n, length, first(mid)) <= slot) seq = mid;
      else hi = mid - 1;
    }
    part = 1 + slot - others(n, length, first(seq));
  }
  // Chunks that the first passes have over all sequences, of first segments and of later ones; the
  // longest chain of the second pass, which has sequences in it that are too short to be cut and
  // yet longer than a segment; the longest sequence.
  struct Sums {
    int first[kLengths], later[kLengths], chain[kLengths], longest;
    SSD_SPLIT_FN void add(const DeltaCut& s, int n, int times) {
      longest = n > longest ? n : longest;
      SSD_SPLIT_UNROLL
      for (int i = 0; i < kLengths; ++i) {
        int parts, per;
        cut(n, s.least << i, parts, per);
        chain[i] = per > chain[i] ? per : chain[i];
        if (parts < 2) continue;
        first[i] += per * times;
        later[i] += per * (parts - 2) * times;
      }
    }
  };
  // The length of the least estimated time, in steps of a chunk, or 0 where cutting gains nothing:
  // each pass takes as long as its longest chain or as all its chains over the CUs; the states in
  // between, a step each.  `block`: a workgroup's rows of a state.  (Products below 2^31: at most
  // 2^22 chunks and heads, and 64 workgroups of a sequence.)
  SSD_SPLIT_FN static int best(const DeltaCut& s, const Sums& v, int chunks, int H, int P, int N, int block, int cus) {
    const int rows = (P + block - 1) / block * H, unit = (N + block - 1) / block * H, all = chunks * rows / cus;
    int least = v.longest > all ? v.longest : all, length = 0;
    SSD_SPLIT_UNROLL
    for (int i = 0; i < kLengths; ++i) {
      const int L = s.least << i;
      if (v.longest < 2 * L) continue;
      const int w = (v.first[i] * rows + v.later[i] * (rows + unit)) / cus, second = v.chain[i];
      const int t = (w > L ? w : L) + (all > second ? all : second) + v.longest / L + kOverhead;
      if (t < least) {
        least = t;
        length = L;
      }
    }
    return length;
  }
};

}  // namespace ssd

#undef SSD_SPLIT_FN
#undef SSD_SPLIT_UNROLL

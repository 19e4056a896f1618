// step_plan.cuh -- how the attention of a step is cut into pieces for its CTAs
// (the same code plans on the device and, for inspection, on the host).
#pragma once
#include "step.cuh"

namespace dfl {

constexpr int kKeys = 128;   // keys of a block

// What a CTA's work costs, in units of about 800 cycles: a block of keys for
// two tiles (3250 cycles measured) or for one (1900 from L2, 2700 from HBM, both
// streams together), and an item's start and end, which fills and drains the
// pipeline and writes a partial row of each of its rows (5000 cycles for 8 rows,
// 11000 for 128, 13000 for 256).
constexpr int kPairUnits = 4, kSingleUnits = 3;
__host__ __device__ inline int end_units(int rows) { return 6 + min(rows, 128) / 16; }
struct WideCosts {
  static constexpr int kPair = kPairUnits, kSingle = kSingleUnits;
  __host__ __device__ static int ends(int rows) { return end_units(rows); }
  // tokens of an item, at most
  __host__ __device__ static int tokens(const StepAttnArgs& a) { return 2 * a.tpt; }
};
// The same of items of at most few_rows (8, or kFewRows) query rows over a packed
// cache (step_attn_few.cu), in units of about 450 cycles: a block 900 from HBM, an
// item's ends 3500.
constexpr int kFewRows = 16;
struct FewCosts {
  static constexpr int kPair = 2, kSingle = 2;
  __host__ __device__ static int ends(int) { return 8; }
  __host__ __device__ static int tokens(const StepAttnArgs& a) { return a.few_rows / a.G; }
};
// Which sequences' items (and whether the prefix's) a kernel takes: all, or those of
// more / at most few_rows query rows of a kv head.
enum RowKind { kAnyRows, kManyRows, kOnlyFewRows };

// One piece of an item that a CTA runs: key blocks [b0, b1) of the segment.
struct Frag {
  int seg;             // 0 prefix, 1 own keys, -1: no further piece
  int seq, h;
  int tok0, ntok;      // first row of the step and tokens of the item's tiles
  int keys;            // keys of the segment that its rows see
  int lim0;            // own, causal: keys that token tok0 sees (may be <= 0)
  int b0, b1;
  int first;           // holds the item's first unit
  int last_cta;        // and then: the CTA of the item's last block
};

// All counts of units are 32-bit (the host refuses more work than that): 64-bit
// divisions cost 2 us of a 13 us call here.
//
// The items in order: the prefix's by kv head and tile pair, then every
// sequence's.  An item takes its blocks' units one block after the other, then
// end_units; a CTA runs the blocks that start in its share.  A share holds more
// than a block, so the CTAs of an item are consecutive, and an item of one block
// is whole (with the ends in front, 48 such items were 96 pieces).  On the device
// a converged warp walks (it skips sequences without rows 32 at a time).
template <class Costs, RowKind KIND>
struct WalkT {
  const StepAttnArgs& a;
  int pair_tok;        // tokens of an item: two tiles
  int rows;            // rows of all sequences
  int pre_blocks, pre_tiles;
  int ua, ub;          // this CTA's units
  int n_cta, share, more;   // CTAs that have units, a CTA's at least, and how many have one more
  int pos;             // first unit of the item at (seg, seq, h, tile)
  int seg, seq, h, tile;
  int row0, T, len;    // the sequence's first row, rows and keys

  __host__ __device__ explicit WalkT(const StepAttnArgs& args) : a(args) {
    pair_tok = Costs::tokens(a);
    rows = a.s.start(a.s.n_seq);
    pre_blocks = (a.s.prefix_len + kKeys - 1) / kKeys;
    pre_tiles = pre_blocks && mine(rows) ? (rows + pair_tok - 1) / pair_tok : 0;
  }
  __host__ __device__ bool mine(int T) const { return KIND == kAnyRows || (T <= a.few_rows / a.G) == (KIND == kOnlyFewRows); }
  // rows of sequence i (none where its items are another kernel's)
  __host__ __device__ int tokens(int i) const {
    const int T = max(a.s.start(i + 1) - a.s.start(i), 0);
    return mine(T) ? T : 0;
  }
  // Row starts that decrease make a plan of no units: step_fits bounds the sum
  // of rows that do not, and the sum of others can wrap.
  __host__ __device__ bool falls(int i) const { return a.s.start(i + 1) < a.s.start(i); }
  __host__ __device__ int weight(int ntok) const { return ntok > a.tpt ? Costs::kPair : Costs::kSingle; }
  __host__ __device__ int units(int ntok, int blocks) const { return Costs::ends(ntok * a.G) + blocks * weight(ntok); }
  // tokens of tile pair j out of T
  __host__ __device__ int pair_tokens(int j, int T) const { return min(pair_tok, T - j * pair_tok); }
  // keys that rows of tile pair j see of a sequence with T rows and len keys
  __host__ __device__ int seen(int j, int T, int len) const {
    const int n = a.causal ? len - T + min((j + 1) * pair_tok, T) : len;
    return min(max(n, 0), a.s.room());
  }
  __host__ __device__ int blocks(int j, int T, int len) const { return (seen(j, T, len) + kKeys - 1) / kKeys; }
  // units of one kv head: of the prefix, and of sequence i
  __host__ __device__ int prefix_head() const {
    if (!pre_tiles) return 0;
    return (pre_tiles - 1) * units(pair_tok, pre_blocks) + units(pair_tokens(pre_tiles - 1, rows), pre_blocks);
  }
  __host__ __device__ int prefix_units() const { return a.Hkv * prefix_head(); }
  __host__ __device__ int head_units(int i) const {
    const int T = tokens(i), len = a.s.len(i);
    int u = 0;
    for (int j = 0; j * pair_tok < T; ++j) u += units(pair_tokens(j, T), blocks(j, T, len));
    return u;
  }
  // CTA c's share of `total` units.  At most `most` CTAs, none with much less
  // than a block of one tile for both its streams (one token behind 4001 keys:
  // 14.6 us, 17.7 with half of that, 15.5 with 16 units).
  __host__ __device__ void divide(int total, int most, int c) {
    n_cta = min(most, total > 0 ? max(total / (2 * Costs::kSingle), 1) : 0);
    ua = ub = 0;
    if (n_cta <= 0) return;
    share = total / n_cta;
    more = total - share * n_cta;
    if (c < n_cta) {
      ua = c * share + min(c, more);
      ub = ua + share + (c < more);
    }
  }
  __host__ __device__ int cta_of(int unit) const {
    const int big = more * (share + 1);
    return unit < big ? unit / (share + 1) : more + (unit - big) / share;
  }
  __host__ __device__ void enter(int i) {   // sequence i, or the next one with rows
#ifdef __CUDA_ARCH__
    const int lane = threadIdx.x & 31;
    for (; i < a.s.n_seq; i += 32) {
      const unsigned some = __ballot_sync(0xffffffffu, i + lane < a.s.n_seq && tokens(i + lane) > 0);
      if (some) {
        i += __ffs(some) - 1;
        break;
      }
    }
#else
    while (i < a.s.n_seq && tokens(i) == 0) ++i;
#endif
    seq = i;
    h = tile = 0;
    if (i >= a.s.n_seq) {
      pos = ub;        // nothing left
      return;
    }
    row0 = a.s.start(i);
    T = tokens(i);
    len = a.s.len(i);
  }
  // Go to the item that holds unit ua; `seq0` is its sequence (-1: the
  // prefix) and `base` that sequence's first unit.
  __host__ __device__ void begin(int seq0, int base) {
    if (seq0 < 0 && ua >= prefix_units()) {   // no sequence holds it: arrays written to while the call runs
      pos = ub;
      return;
    }
    seg = seq0 < 0 ? 0 : 1;
    seq = seq0;
    tile = 0;
    if (!seg) {
      const int per_head = prefix_head(), full = units(pair_tok, pre_blocks);
      h = ua / per_head;
      pos = h * per_head;
      tile = min((ua - pos) / full, pre_tiles - 1);   // every pair but the last is full
      pos += tile * full;
      return;
    }
    pos = base;
    enter(seq0);
    if (pos >= ub) return;
    const int per_head = head_units(seq);
    h = min((ua - base) / per_head, a.Hkv - 1);
    pos += h * per_head;
    for (; (tile + 1) * pair_tok < T; ++tile) {
      const int n = units(pair_tokens(tile, T), blocks(tile, T, len));
      if (pos + n > ua) break;
      pos += n;
    }
  }
  // The next fragment, or false behind the last.
  __host__ __device__ bool next(Frag& f) {
    for (;;) {
      if (pos >= ub) return false;
      const int n = seg ? blocks(tile, T, len) : pre_blocks;
      f.seg = seg;
      f.seq = seq;
      f.h = h;
      f.tok0 = tile * pair_tok + (seg ? row0 : 0);
      f.ntok = pair_tokens(tile, seg ? T : rows);
      f.keys = seg ? seen(tile, T, len) : a.s.prefix_len;
      f.lim0 = seg && a.causal ? len - T + tile * pair_tok + 1 : f.keys;
      const int w = weight(f.ntok);
      auto block_at = [&](int unit) {   // the first block that starts at `unit` or behind
        const int u = max(unit - pos, 0) + w - 1;
        return min(w == Costs::kPair ? u / Costs::kPair : u / Costs::kSingle, n);
      };
      f.b0 = block_at(ua);
      f.b1 = block_at(ub);
      f.first = ua <= pos;
      f.last_cta = f.first ? cta_of(pos + max(n - 1, 0) * w) : -1;
      pos += n * w + Costs::ends(f.ntok * a.G);
      ++tile;
      if (seg == 0) {
        if (tile == pre_tiles) {
          tile = 0;
          if (++h == a.Hkv) {
            seg = 1;
            enter(0);
          }
        }
      } else if (tile * pair_tok >= T) {
        tile = 0;
        if (++h == a.Hkv) enter(seq + 1);
      }
      // an item without a block still has its rows written, by its first CTA
      if (f.first || f.b0 < f.b1) return true;
    }
  }
};

using Walk = WalkT<WideCosts, kAnyRows>;

// The units of all sequences' own keys on the host's worst case, and of the
// prefix: an upper bound that fits 31 bits, or more work than is accepted.  (It
// holds for row starts that do not decrease: their rows are at most n_rows.)
template <class Costs = WideCosts>
inline bool step_fits(const StepAttnArgs& a, int max_keys) {
  const int tok = Costs::tokens(a);
  const long pairs = ((long)a.s.n_rows + tok - 1) / tok;
  const long blocks = (max_keys + (long)kKeys - 1) / kKeys, pre = (a.s.prefix_len + (long)kKeys - 1) / kKeys;
  const long most = Costs::ends(tok * a.G) + Costs::kPair;   // and one block more than a share may hold
  return a.Hkv * ((pairs + a.s.n_seq) * (most + blocks * Costs::kPair) + pairs * (most + pre * Costs::kPair)) <
         (1L << 31);
}

}  // namespace dfl

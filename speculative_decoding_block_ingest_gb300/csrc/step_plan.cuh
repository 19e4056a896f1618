// step_plan.cuh -- how the attention of a step is cut into pieces for its CTAs
// (the same code plans on the device and, for inspection, on the host).
#pragma once
#include "step.cuh"

namespace dfl {

constexpr int kKeys = 128;   // keys of a block

// One piece of an item that a CTA runs: key blocks [b0, b1) of the segment.
struct Frag {
  int seg;             // 0 prefix, 1 own keys, -1: no further piece
  int seq, h;
  int tok0, ntok;      // first row of the step and tokens of the item's tiles
  int keys;            // keys of the segment that may be read
  int lim0;            // own, causal: keys that token tok0 sees (may be <= 0)
  int b0, b1;
  int first;           // holds the item's own unit
  int last_cta;        // and then: the CTA of the item's last unit
};

// Units of one sequence's tile pair j, and the walk over a CTA's fragments.
struct Walk {
  const StepAttnArgs& a;
  int pair_tok;        // tokens of two tiles
  int rows;            // rows of all sequences
  int pre_blocks, pre_tiles;
  long ua, ub;         // this CTA's units
  long total, n_cta;   // all units, and the CTAs that have some
  long pos;            // first unit of the item at (seg, seq, h, tile)
  int seg, seq, h, tile;

  __host__ __device__ explicit Walk(const StepAttnArgs& args) : a(args) {
    pair_tok = 2 * a.tpt;
    rows = a.s.start(a.s.n_seq);
    pre_blocks = (a.s.prefix_len + kKeys - 1) / kKeys;
    pre_tiles = pre_blocks ? (rows + pair_tok - 1) / pair_tok : 0;
  }
  __host__ __device__ long prefix_units() const { return (long)a.Hkv * pre_tiles * (pre_blocks + 1); }
  __host__ __device__ int tokens(int i) const { return max(a.s.start(i + 1) - a.s.start(i), 0); }
  // key blocks that tile pair j of sequence i needs
  __host__ __device__ int blocks(int i, int j, int T) const {
    const int len = a.s.len(i);
    const int seen = a.causal ? len - T + min((j + 1) * pair_tok, T) : len;
    return (min(max(seen, 0), a.s.room()) + kKeys - 1) / kKeys;
  }
  __host__ __device__ long head_units(int i) const {   // units of one kv head of sequence i
    const int T = tokens(i);
    long u = 0;
    for (int j = 0; j * pair_tok < T; ++j) u += 1 + blocks(i, j, T);
    return u;
  }
  // Go to the item that holds unit ua; `seq0` is its sequence (-1: the
  // prefix) and `base` that sequence's first unit.
  __host__ __device__ void begin(int seq0, long base) {
    seg = seq0 < 0 ? 0 : 1;
    seq = seq0;
    const long per_head = seg ? head_units(seq) : (long)pre_tiles * (pre_blocks + 1);
    h = per_head ? (int)((ua - base) / per_head) : 0;
    pos = base + h * per_head;
    tile = 0;
    if (!seg) {
      tile = (int)((ua - pos) / (pre_blocks + 1));
      pos += (long)tile * (pre_blocks + 1);
    } else {
      const int T = tokens(seq);
      for (long n; tile * pair_tok < T && pos + (n = 1 + blocks(seq, tile, T)) <= ua; ++tile) pos += n;
    }
  }
  // The next fragment, or false behind the last.
  __host__ __device__ bool next(Frag& f) {
    while (pos < ub) {
      int n, T = rows;
      if (seg == 0) {
        n = 1 + pre_blocks;
      } else {
        T = tokens(seq);
        if (tile * pair_tok >= T) {   // the next head, or sequence
          tile = 0;
          if (T == 0 || ++h == a.Hkv) {
            h = 0;
            if (++seq >= a.s.n_seq) return false;
          }
          continue;
        }
        n = 1 + blocks(seq, tile, T);
      }
      f.seg = seg;
      f.seq = seq;
      f.h = h;
      f.tok0 = tile * pair_tok + (seg ? a.s.start(seq) : 0);
      f.ntok = min(pair_tok, T - tile * pair_tok);
      f.keys = seg ? min(a.s.len(seq), a.s.room()) : a.s.prefix_len;
      f.lim0 = seg && a.causal ? a.s.len(seq) - T + tile * pair_tok + 1 : f.keys;
      f.b0 = (int)max(ua - pos - 1, 0L);
      f.b1 = (int)min((long)n, ub - pos) - 1;
      f.first = ua <= pos;
      f.last_cta = (int)min(((pos + n) * n_cta + total - 1) / total - 1, n_cta - 1);
      pos += n;
      ++tile;
      if (seg == 0 && tile == pre_tiles) {
        tile = 0;
        if (++h == a.Hkv) seg = 1, h = 0, seq = 0;
      }
      return true;
    }
    return false;
  }
};


// CTA c's share [ua, ub) of `total` units over at most `n_cta` CTAs.  No CTA
// in use is without a unit, so the CTAs of an item are consecutive.
__host__ __device__ inline void share_units(Walk& w, long total, int n_cta, int c) {
  w.total = total;
  w.n_cta = min((long)n_cta, total);
  w.ua = w.ub = 0;
  if (c < w.n_cta) {
    w.ua = c * total / w.n_cta;
    w.ub = (c + 1) * total / w.n_cta;
  }
}

}  // namespace dfl

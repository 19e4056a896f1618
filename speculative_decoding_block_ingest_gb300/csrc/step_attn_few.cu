// step_attn_few.cu -- attention of a step over a packed cache where a kv head has
// at most 16 query rows of a sequence (or of the batch, for the prefix): single
// tokens and short drafts.  (More rows than that are right here too, 16 at a time.)
// The formula, the items and their pieces are those of
// step_attn.cu; what is different is that the keys' bytes bound it, and that codes
// have to become f16 on the way: 144 bytes a key, 256 values.
//
// step_attn.cu writes every value as f16 to a tile in shared memory, where its products
// take K and V from: 1600 cycles for a block of 128 keys that HBM delivers in 790, for 128
// query rows of which 16 exist.  Here codes go from shared memory to registers, become f16
// there and are a warp-wide product's operand at once (mma.sync, 16 keys or elements by 8
// query rows).  (Tensor memory can hold one operand of a tcgen05.mma; K or V from there is
// not tried.)
//
// For 16 keys of a warp and N tiles of 8 query rows (keys and elements may come in
// any order, as long as both operands agree):
//   S^T [16 keys x 8 rows] += K [16 x 16 elements] Q^T    d / 16 times
//   P^T = 2^(S^T - m), to f16, transposed in registers (movmatrix)
//   O^T [16 elements x 8 rows] += V^T [16 x 16 keys] P^T  d / 16 times
// A lane's codes of K are 32 elements in a row of two keys (one 16-byte load each),
// those of V 16 elements of four keys, whose nibbles are paired key by key before
// they become f16.
//
// A CTA has 15 such warps for 8 rows (N = 1), or 11 with the registers that 16 need,
// each with every fifteenth (eleventh) 32 keys and a running maximum of its own; at a
// piece's end their parts are summed in a fixed order.  A further warp plans the pieces
// and loads their blocks, ahead into the next ones.  (Smaller loads for a warp each are
// too many: 64 decoding sequences took 231 us with TMA boxes of 16 keys, 247 with 32,
// 220 with cp.async; 185 with 11 warps for 8 rows too.)
#include <float.h>

#include <atomic>

#include "../../include/dflash.h"
#include "fp4.cuh"
#include "kernels.cuh"
#include "ptx.cuh"
#include "step_attn.cuh"
#include "step_plan.cuh"

namespace dfl {
namespace {

constexpr int kGroup = 16;                  // keys of a product
constexpr int kUnit = 2 * kGroup;           // and of a warp at a time
constexpr int kFewFrags = 4;                // pieces described ahead
constexpr int kBarParts = 1;                // named barrier of those warps
constexpr float kFewBias = 7.f;             // weights are 2^7 times as large (see pack2)
constexpr float kNoMax = FLT_MAX;           // bias minus a maximum below any

template <int D, int NT>
struct Few {
  static constexpr int kWarps = NT == 1 ? 15 : 11, kThreads = (kWarps + 1) * 32;
  static constexpr int kTile = 8 * NT;                   // query rows of an item
  static constexpr int kCode = D / 2, kScale = D / 16;   // bytes of a head row
  // of a block: by page (of 128 rows at most) K's codes and V's, then by page their scales
  static constexpr int kCodes = 2 * kKeys * kCode;
  static constexpr int kStage = kCodes + 2 * 1024;
  // a page's scales take 128 bytes at least: a TMA copy starts on such a boundary
  static __device__ __forceinline__ int scale_pitch(int rows) { return max(rows * kScale, 128); }
  static constexpr int kAhead = D == 64 ? 13 : NT == 1 ? 8 : 7;   // blocks in flight
  static constexpr int kRow = D + 4;                     // floats of a partial row
};
template <int WARPS, int TILE>
struct FewShared {
  uint64_t ffull[kFewFrags], fempty[kFewFrags];
  uint64_t full[13], empty[13];
  Frag frag[kFewFrags];
  float2 ml[WARPS][TILE];
  int bad[8];            // first own key whose scale is NaN, by block
  int any_bad, abort;
};
template <int D, int NT>
using FewState = FewShared<Few<D, NT>::kWarps, Few<D, NT>::kTile>;
template <int D, int NT>
constexpr size_t few_smem() {
  using F = Few<D, NT>;
  return (size_t)F::kAhead * F::kStage + (size_t)F::kWarps * F::kTile * F::kRow * 4 + sizeof(FewState<D, NT>);
}
static_assert(few_smem<128, 1>() <= 227 * 1024 && few_smem<128, 2>() <= 227 * 1024 && few_smem<64, 1>() <= 227 * 1024 &&
              few_smem<64, 2>() <= 227 * 1024, "shared memory of the kernel for few rows");

__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, const uint32_t* b) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// The key that row n of a product's operand is: with rows of 64 bytes swizzled like
// this, the loads below take all banks.
__device__ __forceinline__ int key_of(int n) { return (n & ~3) | ((0x9C >> (2 * (n & 3))) & 3); }
template <int D>
__device__ __forceinline__ int flip(int row) { return D == 128 ? row >> 1 & 3 : row >> 2 & 1; }

__device__ __forceinline__ void tma_load_5d(void* dst, const void* map, uint64_t* bar, int x, int y, int z, int w, int v) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6, %7}], "
      "[%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(v)
      : "memory");
}

// The loading warp: a piece's blocks into the ring.  A box has a page's rows of K and
// of V where one tensor map can reach both: issuing boxes is what takes this warp's
// time (8 for a block of 64-row pages instead of 4: 187 us for 64 decoding sequences,
// not 181).
template <int D, int NT>
struct BlockLoader {
  using F = Few<D, NT>;
  const StepAttnArgs& a;
  const PairMaps& maps;
  FewState<D, NT>& sh;
  uint8_t* ring;
  const int lane;
  uint32_t issued = 0;

  __device__ __forceinline__ void piece(const Frag& f) {
    const int* table = f.seg ? a.s.block_table + f.seq * a.s.table_stride : a.s.prefix_pages;
    const int shift = __ffs(a.box_rows) - 1, n_box = (f.keys + a.box_rows - 1) >> shift;
    // page ids: one lane per box of the next 32, the following 32 in flight
    auto page_of = [&](int box) -> int {
      return box < n_box ? table[(int)(((long)box << shift) >> a.s.page_shift)] : 0;
    };
    int win = f.b0 * a.boxes, cur = page_of(win + lane), nxt = page_of(win + 32 + lane);
    const int sc = lane & 1, second = lane >> 1 & 1, bi = lane >> 2;
    const bool pair = maps.pair[sc], mine = !(second && pair);
    const int to = (sc ? F::kCodes : 0) + (2 * bi + second) * (sc ? F::scale_pitch(a.box_rows) : a.box_rows * F::kCode);
    const CUtensorMap* map = sc ? &maps.scales[second] : &maps.codes[second];
    for (int b = f.b0; b < f.b1; ++b, ++issued) {
      const int box0 = b * a.boxes, n = min(a.boxes, n_box - box0);
      if (box0 >= win + 32) {                             // boxes of a block never straddle a window
        cur = nxt;
        win += 32;
        nxt = page_of(win + 32 + lane);
      }
      const uint32_t slot = issued % F::kAhead;
      if (!__all_sync(0xffffffffu, pipe_wait(&sh.empty[slot], ((issued / F::kAhead) & 1) ^ 1, &sh.abort))) {
        sh.abort = 1;
        return;
      }
      if (lane == 0) mbar_arrive_expect_tx(&sh.full[slot], (uint32_t)(n * a.box_rows * 2 * (F::kCode + F::kScale)));
      __syncwarp();
      const int page = __shfl_sync(0xffffffffu, cur, min(box0 - win + bi, 31));
      const int at = (int)(((long)(box0 + bi) << shift) & (a.s.page_size - 1));
      uint8_t* dst = ring + slot * F::kStage + to;
      if (bi < n && mine) {
        if (sc && pair) tma_load_4d(dst, map, &sh.full[slot], at, f.h, page, 0);
        else if (sc) tma_load_3d(dst, map, &sh.full[slot], at, f.h, page);
        else if (pair) tma_load_5d(dst, map, &sh.full[slot], 0, f.h, at, page, 0);
        else tma_load_4d(dst, map, &sh.full[slot], 0, f.h, at, page);
      }
      __syncwarp();
    }
  }
  __device__ __forceinline__ void drain() {   // leave no copy in flight behind
    int none = 0;
    for (uint32_t i = issued > (uint32_t)F::kAhead ? issued - F::kAhead : 0; i < issued; ++i)
      pipe_wait(&sh.full[i % F::kAhead], (i / F::kAhead) & 1, &none);
  }
};

// One piece's rows of a warp: NT tiles of 8.
template <int D, bool BF16, int NT>
struct Rows {
  using F = Few<D, NT>;
  static constexpr int kSteps = D / 16;
  uint32_t q[NT][kSteps][2];     // Q^T operands, every row times a power of two
  float o[NT][kSteps][4];
  float sc[NT][2], nm[NT][2], l[NT][2];   // of rows 8 nt + 2 t, + 1; nm: 7 minus the running maximum
  int lim[NT][2], least;         // keys those see, and the fewest that one sees

  __device__ __forceinline__ void start(const StepAttnArgs& a, const Frag& f, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = 8 * nt + g, tok = r / a.G, head = r - tok * a.G;
      uint32_t w[D / 8];          // D / 4 16-bit elements: 4-element runs a quarter each
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + (f.tok0 + tok) * a.q_stride +
                                                        (long)(f.h * a.G + head) * D + t * (D / 4));
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint4 x = tok < f.ntok ? src[i] : make_uint4(0, 0, 0, 0);
        w[4 * i] = x.x, w[4 * i + 1] = x.y, w[4 * i + 2] = x.z, w[4 * i + 3] = x.w;
      }
      float up = 1.f;             // what the row's scores are to be multiplied by
      if constexpr (BF16) {
        // bf16's range in f16: the row times 2^-e, its largest element in [2^14, 2^15); an
        // element is off by half of f16's smallest step, 2^-24, which is 2^-39 of the largest
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) top = max(top, max(w[i] & 0x7FFFu, w[i] >> 16 & 0x7FFFu));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int e = max((int)(top >> 7), 1) - 127 - 14;             // (127 + 14 - e stays within 1 .. 254)
        const int ec = min(max(e, -126), 113);
        const float down = __uint_as_float((uint32_t)(127 - ec) << 23);
        up = __uint_as_float((uint32_t)(127 + ec) << 23);
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          const float2 v = __bfloat1622float2(reinterpret_cast<const __nv_bfloat162&>(w[i]));
          w[i] = __float_as_uint(pack2<false>(make_float2(v.x * down, v.y * down)));
        }
      }
#pragma unroll
      for (int j = 0; j < kSteps; ++j) q[nt][j][0] = w[2 * j], q[nt][j][1] = w[2 * j + 1];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        // (a normal float: times 0 a masked score, -inf, would be NaN, and a score of 0 times
        // infinity.  Scores that the lower bound changes are less than 2^-92.)
        sc[nt][c] = fminf(fmaxf(a.scale_log2 * __shfl_sync(0xffffffffu, up, (2 * t + c) * 4), FLT_MIN), FLT_MAX);
        const int at = (8 * nt + 2 * t + c) / a.G;
        lim[nt][c] = at < f.ntok && f.seg == 1 && a.causal ? min(max(f.lim0 + at, 0), f.keys) : f.keys;
        nm[nt][c] = kNoMax;
        l[nt][c] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < kSteps; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[nt][j][c] = 0.f;
    }
    least = f.seg == 1 && a.causal ? min(max(f.lim0, 0), f.keys) : f.keys;
  }

  // 32 keys, from key0 and row r0 of a block on; rows of a box (their
  // logarithm), and whether V's codes (scales)
  // lie first in it.
  __device__ __forceinline__ void keys(const uint8_t* st, int r0, int key0, int n_keys, int box_shift, const int* v_first,
                                       FewState<D, NT>& sh, int lane) {
    constexpr int kCode = F::kCode, kScale = F::kScale;
    const int g = lane >> 2, t = lane & 3, rows = 1 << box_shift;
    float s[2][NT][4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      // K: a quarter of two keys' elements
      const int r = r0 + u * kGroup, box = r >> box_shift, in = r & (rows - 1);
      const uint8_t* codes = st + ((2 * box + v_first[0]) * rows + in) * kCode;
      const uint8_t* scales = st + F::kCodes + (2 * box + v_first[1]) * F::scale_pitch(rows) + in * kScale;
      constexpr int kWords = D / 32;
      uint32_t x[2][kWords];
      __half2 f[2][2];           // scales of the words' blocks
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = key_of(g) + 8 * i;
        if constexpr (D == 128) {
          const uint4 v = *reinterpret_cast<const uint4*>(codes + row * kCode + (t ^ flip<D>(row)) * 16);
          x[i][0] = v.x, x[i][1] = v.y, x[i][2] = v.z, x[i][3] = v.w;
          const __half2 two = e4m3_to2(*reinterpret_cast<const uint16_t*>(scales + row * kScale + 2 * t));
          f[i][0] = __low2half2(two), f[i][1] = __high2half2(two);
        } else {
          const uint2 v = *reinterpret_cast<const uint2*>(codes + row * kCode + ((t >> 1) ^ flip<D>(row)) * 16 + (t & 1) * 8);
          x[i][0] = v.x, x[i][1] = v.y;
          f[i][0] = f[i][1] = __low2half2(e4m3_to2(scales[row * kScale + t]));
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 4; ++c) s[u][nt][c] = 0.f;
#pragma unroll
      for (int w = 0; w < kWords; ++w) {
        uint32_t p[4], r[4];
        e2m1_to8(x[0][w], p);
        e2m1_to8(x[1][w], r);
        const __half2 f0 = f[0][w * 2 / kWords], f1 = f[1][w * 2 / kWords];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          p[i] = as_u32(__hmul2(as_half2(p[i]), f0));
          r[i] = as_u32(__hmul2(as_half2(r[i]), f1));
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t op[4] = {p[2 * i], r[2 * i], p[2 * i + 1], r[2 * i + 1]};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16816(s[u][nt], op, q[nt][2 * w + i]);
        }
      }
    }
    if (key0 + kUnit > least) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (key0 + u * kGroup + key_of(g) + 8 * (c >> 1) >= lim[nt][c & 1]) s[u][nt][c] = -INFINITY;
    }
    // the running maximum moves only when it grows by more than 2^8 (kGrow), as in step_attn.cu
    float x[2][NT][4];
    bool grow = false;
    auto shift = [&]() {
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c) x[u][nt][c] = fmaf(s[u][nt][c], sc[nt][c & 1], nm[nt][c & 1]);
    };
    shift();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
      grow |= max3(max3(fmaxf(x[0][nt][0], x[0][nt][1]), x[0][nt][2], x[0][nt][3]),
                   max3(x[1][nt][0], x[1][nt][1], x[1][nt][2]), x[1][nt][3]) > kGrow + kFewBias;
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float mx = fmaxf(fmaxf(s[0][nt][c], s[0][nt][c + 2]), fmaxf(s[1][nt][c], s[1][nt][c + 2])) * sc[nt][c];
#pragma unroll
          for (int i = 4; i < 32; i <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, i));
          if (mx + nm[nt][c] > kGrow + kFewBias) {
            const float to = kFewBias - mx, f = ex2_fast(to - nm[nt][c]);
            nm[nt][c] = to;
            l[nt][c] *= f;
#pragma unroll
            for (int j = 0; j < kSteps; ++j) o[nt][j][c] *= f, o[nt][j][c + 2] *= f;
          }
        }
      shift();
    }
    uint32_t p[2][NT][2];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float w[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) w[c] = ex2_fast(x[u][nt][c]);
        l[nt][0] += w[0] + w[2];
        l[nt][1] += w[1] + w[3];
        p[u][nt][0] = transpose8(__float_as_uint(pack2<false>(make_float2(w[0], w[1]))));
        p[u][nt][1] = transpose8(__float_as_uint(pack2<false>(make_float2(w[2], w[3]))));
      }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      // V: an eighth of the elements of four keys
      const int k[4] = {key_of(2 * t), key_of(2 * t + 1), key_of(2 * t) + 8, key_of(2 * t + 1) + 8};
      const int r = r0 + u * kGroup, box = r >> box_shift, in = r & (rows - 1);
      const uint8_t* codes = st + ((2 * box + 1 - v_first[0]) * rows + in) * kCode;
      const uint8_t* scales = st + F::kCodes + (2 * box + 1 - v_first[1]) * F::scale_pitch(rows) + in * kScale;
      constexpr int kWords = D / 64;
      uint32_t y[4][kWords], sv[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint8_t* row = codes + k[i] * kCode;
        if constexpr (D == 128) {
          const uint2 v = *reinterpret_cast<const uint2*>(row + ((g >> 1) ^ flip<D>(k[i])) * 16 + (g & 1) * 8);
          y[i][0] = v.x, y[i][1] = v.y;
          sv[i] = scales[k[i] * kScale + g];
        } else {
          y[i][0] = *reinterpret_cast<const uint32_t*>(row + ((g >> 2) ^ flip<D>(k[i])) * 16 + (g & 3) * 4);
          sv[i] = scales[k[i] * kScale + (g >> 1)];
        }
      }
      // behind the last key lies anything; NaN scales of the step's own rows that some row
      // must not see are remembered
      if (key0 + kUnit > least) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = key0 + u * kGroup + k[i];
          if (key >= n_keys) {
            sv[i] = 0;
          } else if ((sv[i] & 0x7F) == kScaleNaN && key >= least) {
            sv[i] = 0;
            atomicMin(&sh.bad[D == 128 ? g : g >> 1], key);
            sh.any_bad = 1;
          }
        }
      }
      const __half2 f0 = e4m3_to2(sv[0] | sv[1] << 8), f1 = e4m3_to2(sv[2] | sv[3] << 8);
#pragma unroll
      for (int w = 0; w < kWords; ++w) {
        // two keys' nibbles side by side: the even elements, then the odd ones
        uint32_t v[4][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t lo = y[2 * i][w], hi = y[2 * i + 1][w];
          e2m1_to8((lo & 0x0F0F0F0Fu) | (hi << 4 & 0xF0F0F0F0u), v[2 * i]);
          e2m1_to8((lo >> 4 & 0x0F0F0F0Fu) | (hi & 0xF0F0F0F0u), v[2 * i + 1]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t op[4] = {as_u32(__hmul2(as_half2(v[0][j]), f0)), as_u32(__hmul2(as_half2(v[1][j]), f0)),
                                  as_u32(__hmul2(as_half2(v[2][j]), f1)), as_u32(__hmul2(as_half2(v[3][j]), f1))};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma16816(o[nt][4 * w + j], op, p[u][nt]);
        }
      }
    }
  }

  // This warp's part into shared memory.
  __device__ __forceinline__ void finish(float* part, float2* ml, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float sum = l[nt][c];
#pragma unroll
        for (int i = 4; i < 32; i <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, i);
        // (the sum and O are 2^7 times theirs, and so go with a maximum less 7)
        if (g == 0) ml[8 * nt + 2 * t + c] = make_float2(nm[nt][c] == kNoMax ? -INFINITY : -nm[nt][c], sum);
        float* to = part + (8 * nt + 2 * t + c) * F::kRow + g * (D / 8);
#pragma unroll
        for (int j = 0; j < kSteps; j += 2)
          *reinterpret_cast<float4*>(to + 2 * j) =
              make_float4(o[nt][j][c], o[nt][j][c + 2], o[nt][j + 1][c], o[nt][j + 1][c + 2]);
      }
  }
};

template <int D, bool BF16, int NT>
__global__ void __launch_bounds__(Few<D, NT>::kThreads, 1)
    step_attn_few_kernel(const __grid_constant__ PairMaps maps, const __grid_constant__ StepAttnArgs a,
                         const bool wide_ran) {
  extern __shared__ __align__(1024) uint8_t smem[];
  using F = Few<D, NT>;
  constexpr int kWarps = F::kWarps;
  float* parts = reinterpret_cast<float*>(smem + F::kAhead * F::kStage);
  auto& sh = *reinterpret_cast<FewState<D, NT>*>(parts + kWarps * F::kTile * F::kRow);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kFewFrags; ++i) {
      mbar_init(&sh.ffull[i], 1);
      mbar_init(&sh.fempty[i], kWarps);
    }
    for (int i = 0; i < F::kAhead; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], kWarps);
    }
    for (int i = 0; i < 2; ++i) {
      if (i == 0 || !maps.pair[0]) tma_prefetch_map(&maps.codes[i]);
      if (i == 0 || !maps.pair[1]) tma_prefetch_map(&maps.scales[i]);
    }
    sh.abort = sh.any_bad = 0;
    for (int i = 0; i < 8; ++i) sh.bad[i] = INT_MAX;
    fence_barrier_init();
  }
  __syncthreads();
  pdl_wait();
  pdl_launch_dependents();

  if (warp == kWarps) {
    // ------------------------------------------------------------------ plan and loads
    BlockLoader<D, NT> loader{a, maps, sh, smem, lane};
    auto plan = [&](auto w) {
      plan_pieces(w, a.n_cta - a.n_wide, sh.frag, sh.ffull, sh.fempty, kFewFrags, lane,
                  [&](const Frag& f) { loader.piece(f); });
    };
    if (wide_ran) plan(WalkT<FewCosts, kOnlyFewRows>(a));
    else plan(WalkT<FewCosts, kAnyRows>(a));
    loader.drain();
  } else {
    int slot = 0, mine = warp;                           // this warp's next unit, from the next block on
    uint32_t parity = 0;
    const int box_shift = __ffs(a.box_rows) - 1;
    bool ok = true;
    int4 split = make_int4(0, 0, 0, 0);
    auto all = [&]() { asm volatile("barrier.sync %0, %1;" ::"n"(kBarParts), "n"(kWarps * 32) : "memory"); };
    const int cta = a.n_wide + blockIdx.x;
    for (uint32_t nf = 0;; ++nf) {
      if (!__all_sync(0xffffffffu, ring_wait(&sh.ffull[nf % kFewFrags], (nf / kFewFrags) & 1))) {
        sh.abort = 1;      // (the others' waits on this piece fail alike)
        break;
      }
      const Frag f = sh.frag[nf % kFewFrags];
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.fempty[nf % kFewFrags]);
      if (f.seg < 0) break;
      const int rows = f.ntok * a.G;
      float* part = parts + warp * F::kTile * F::kRow;
      Rows<D, BF16, NT> r;
      r.start(a, f, lane);
      for (int b = f.b0; b < f.b1; ++b) {
        // (every warp waits for every block, so a barrier's parity is read in turn)
        if (ok) ok = __all_sync(0xffffffffu, pipe_wait(&sh.full[slot], parity, &sh.abort));
        if (mine < kKeys / kUnit) {
          const int key0 = b * kKeys + mine * kUnit;
          if (ok && key0 < f.keys) r.keys(smem + slot * F::kStage, mine * kUnit, key0, f.keys, box_shift, maps.v_first, sh, lane);
          mine += kWarps;
        }
        mine -= kKeys / kUnit;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.empty[slot]);
        if (++slot == F::kAhead) slot = 0, parity ^= 1;
      }
      if (!ok) sh.abort = 1;
      r.finish(part, sh.ml[warp], lane);
      all();
      // ---- the warps' parts, in order; four elements a thread
      const bool whole = f.first && f.last_cta == (int)blockIdx.x && a.s.prefix_len == 0;
      const bool poisoned = sh.any_bad;
      if (*(volatile int*)&sh.abort) ok = false;
      for (int e = tid; e < rows * (D / 4); e += kWarps * 32) {
        const int i = e / (D / 4), c = e % (D / 4) * 4, tok = i / a.G, head = f.h * a.G + i - tok * a.G;
        float mx = -INFINITY, l = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, sh.ml[w][i].x);
        float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float2 ml = sh.ml[w][i];
          // a part without a maximum is left out, unless its sum is NaN
          const float wt = ml.x == -INFINITY ? (ml.y == 0.f ? 0.f : 1.f) : ex2_fast(ml.x - mx);
          if (ml.x == -INFINITY && ml.y == 0.f) continue;
          const float4 x = *reinterpret_cast<const float4*>(parts + (w * F::kTile + i) * F::kRow + c);
          l = fmaf(ml.y, wt, l);
          o[0] = fmaf(x.x, wt, o[0]), o[1] = fmaf(x.y, wt, o[1]), o[2] = fmaf(x.z, wt, o[2]), o[3] = fmaf(x.w, wt, o[3]);
        }
        const int lim = f.seg == 1 && a.causal ? min(max(f.lim0 + tok, 0), f.keys) : f.keys;
        if (poisoned && sh.bad[c / 16] < lim) o[0] = o[1] = o[2] = o[3] = __int_as_float(0x7fc00000);
        const long row = f.tok0 + tok, item = row * a.Hq + head;
        if (whole) {
          const float inv = !ok ? __int_as_float(0x7fc00000) : l == 0.f ? 0.f : a.out_scale / l;
          uint32_t y[2];
#pragma unroll
          for (int v = 0; v < 2; ++v)
            y[v] = __float_as_uint(pack2<BF16>(make_float2(o[2 * v] * inv, o[2 * v + 1] * inv)));
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + row * a.out_stride + (long)head * D + c) =
              make_uint2(y[0], y[1]);
          if (c == 0 && a.lse) a.lse[item] = ok ? log_sum(mx, l) : inv;
        } else {
          const long at = f.first ? item : cta_row(a, cta, i);
          *reinterpret_cast<float4*>((f.first ? a.seg_o[f.seg] : a.cta_o) + at * D + c) =
              make_float4(o[0], o[1], o[2], o[3]);
          if (c == 0) (f.first ? a.seg_ml[f.seg] : a.cta_ml)[at] = make_float2(mx, l);
        }
        if (c == 0 && f.first && i == tok * a.G && !a.by_cta)
          a.meta[((long)f.seg * a.s.n_rows + row) * a.Hkv + f.h] = make_int4(cta, a.n_wide + f.last_cta, tok, whole);
      }
      if (tid == 0 && f.first && !whole) split = make_int4(f.tok0, f.ntok, f.h, a.n_wide + f.last_cta);
      all();
      if (poisoned) {
        if (tid < 8) sh.bad[tid] = INT_MAX;
        if (tid == 8) sh.any_bad = 0;
        all();
      }
    }
    if (tid == 0 && a.by_cta) a.split[cta] = split;
  }
  __syncthreads();
  if (tid == 0) {
    const int bad = sh.abort ? DERR_TIMEOUT : 0;
    a.status[blockIdx.x] = wide_ran && a.status[blockIdx.x] ? a.status[blockIdx.x] : bad;
  }
}

template <int D, bool BF16, int NT>
cudaError_t launch(const StepAttnArgs& a, const PairMaps& m, bool wide_ran, cudaStream_t s) {
  auto* kernel = step_attn_few_kernel<D, BF16, NT>;
  // the kernel's shared memory is raised once on every device
  static std::atomic<uint64_t> raised{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(raised.load(std::memory_order_relaxed) >> dev & 1)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)few_smem<D, NT>());
    if (e != cudaSuccess) return e;
    if (dev < 64) raised.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
  }
  return launch_pdl(kernel, dim3(a.n_cta - a.n_wide), dim3(Few<D, NT>::kThreads), few_smem<D, NT>(), s, m, a, wide_ran);
}

}  // namespace

cudaError_t launch_step_attention_few(const StepAttnArgs& a, const PairMaps& m, bool wide_ran, cudaStream_t s) {
  auto* run = a.few_rows == 8 ? a.d == 128 ? (a.bf16 ? launch<128, true, 1> : launch<128, false, 1>)
                                           : (a.bf16 ? launch<64, true, 1> : launch<64, false, 1>)
              : a.d == 128    ? (a.bf16 ? launch<128, true, 2> : launch<128, false, 2>)
                              : (a.bf16 ? launch<64, true, 2> : launch<64, false, 2>);
  return run(a, m, wide_ran, s);
}

}  // namespace dfl

// step_append.cu -- a step's queries, keys and values: per-head RMSNorm, RoPE
// and the paged-cache rows, in one pass.
//
// For a query or key head row x of d elements at position p:
//   y = x * rsqrt(mean(x^2) + eps) * gain          (where there is a gain)
//   y_j, y_{j+h} = y_j c_j - y_{j+h} s_j, y_{j+h} c_j + y_j s_j,  h = rot / 2,
//   c_j, s_j = mscale * cos, sin(p inv_freq_j)
// (or on y_{2j}, y_{2j+1} where pairs are interleaved)
// and values pass through.  Everything is read once and written once, a few
// flops an element: bytes bound it, for one token the launch and a chain of
// dependent loads (row -> sequence -> length -> page).
//
// A warp takes a whole row, or (few rows) an eighth of its heads: d / 16 lanes
// hold a head row, each the two 8-element chunks that RoPE pairs, so the
// rotation needs no exchange, the norm three shuffles and no warp waits for
// another.  Sequence, cache row and angles are found while the first head
// rows' loads are in flight; the 8 (cos, sin) pairs a lane needs are the same
// for all heads and stay in registers.
//
// Angles are counted in turns modulo 1 as 64-bit integers: position times
// frequency wraps around by itself, exactly, where f32 would leave 2^-7 of a
// radian at position 10^5 and f64 runs at 1/64 of the f32 rate.
#include "../../include/dflash.h"
#include "kernels.cuh"
#include "ptx.cuh"
#include "step.cuh"
#include "step_rows.cuh"

namespace dfl {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kFewWarps = 8;      // warps of a row when there are few rows
constexpr int kManyWarps = 1;     // and when there are many

// Resident CTAs of an SM.  Many rows: four, each lane 2 head rows deep (1 in
// f32): 34912 rows of 48 f16 heads in 148 us (6.2 TB/s), 32000 normed bf16 rows in
// 145; three CTAs, two warps a row and 3 deep 148 and 152, deeper ones spill.
// Few rows: one to four waves at any occupancy.
constexpr int append_ctas(int warps) { return warps == kManyWarps ? 4 : 2; }

template <typename In, typename Out, int D, int WARPS, bool INTER>
__global__ void __launch_bounds__(kAppendThreads, append_ctas(WARPS))
    step_append_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int kLanes = D / 16;               // lanes of a head row
  constexpr int kGroups = 32 / kLanes;         // head rows of a warp at once
  constexpr int kDepth = WARPS == kManyWarps && sizeof(In) == 4 ? 1 : 2;   // of those, in flight
  constexpr int kStep = WARPS * kGroups;       // heads between a lane's
  __shared__ __align__(16) float2 cs_all[kAppendThreads / 32][D / 2];
  pdl_wait();
  pdl_launch_dependents();
  const StepView& s = a.s;
  const int lane = threadIdx.x & 31, l = lane % kLanes;
  const int id = blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
  const int first = id % WARPS * kGroups + lane / kLanes;   // this lane's first head
  const int Hq = a.n_heads, Hkv = a.c.n_kv_heads, heads = Hq + 2 * Hkv;
  float2* cs = cs_all[threadIdx.x >> 5];
  // the two chunks of a head row this lane holds: a RoPE pair, or two of the
  // chunks behind the rotated ones
  const int pairs = a.rot / 16;
  const bool rot = l < pairs;
  const int c0 = 8 * (rot ? l : 2 * pairs + (l - pairs));
  const int c1 = rot ? c0 + 8 * pairs : c0 + 8 * (kLanes - pairs);
  // turns per position of the angles this lane forms
  uint64_t turn[D / 64];
#pragma unroll
  for (int i = 0; i < D / 64; ++i) turn[i] = a.turns[lane + 32 * i];

  const int stride = gridDim.x * (kAppendThreads / 32) / WARPS;
  for (int row = id / WARPS; row < s.n_rows; row += stride) {
    Raw<In> x0[kDepth], x1[kDepth];
    auto fetch = [&](int h0) {
#pragma unroll
      for (int i = 0; i < kDepth; ++i) {
        const int h = h0 + i * kStep;
        if (h < heads) {
          const In* p = h < Hq ? static_cast<const In*>(a.q) + row * a.q_stride + (long)h * D
                        : h < Hq + Hkv ? static_cast<const In*>(a.k) + row * a.k_stride + (long)(h - Hq) * D
                                       : static_cast<const In*>(a.v) + row * a.v_stride + (long)(h - Hq - Hkv) * D;
          x0[i].load(p + c0);
          x1[i].load(p + c1);
        }
      }
    };
    // many rows: other warps cover these loads' latency, and held through the
    // look-ups below their registers spill
    if constexpr (WARPS == kFewWarps) fetch(first);
    // the row's sequence: as many end at or before the row as lie below it
    // (each lane looks at the end of one 32nd of what is left)
    int seq = 0;
    for (int left = s.n_seq; left > 0;) {
      const int step = (left + 31) / 32;
      const int end = seq + min((lane + 1) * step, left);
      const int below = __popc(__ballot_sync(0xffffffffu, s.start(end) <= row)) * step;
      seq += min(below, left);
      left = below >= left ? 0 : min(step, left - below) - 1;
    }
    if (seq >= s.n_seq) break;   // rows behind the last sequence stay as they are
    const int own = s.len(seq) - s.start(seq + 1) + row;   // this row's own key index
    long dst = -1;                                         // its row in the cache
    if (own >= 0 && (own >> s.page_shift) < s.table_cols) {
      const int page = s.block_table[seq * s.table_stride + (own >> s.page_shift)];
      if (page >= 0 && page < s.n_pages)
        dst = page * a.c.page_stride + (long)(own & (s.page_size - 1)) * a.c.row_stride;
    }
    if constexpr (WARPS == kManyWarps) fetch(first);
    float2 w[8];
    if (a.rot) {
      const long pos = a.positions ? (long)a.positions[row] : (long)s.prefix_len + own;
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        // a signed fraction of a turn, times 2: sin and cos of pi x
        const float x = __ll2float_rn((long long)((uint64_t)pos * turn[i])) * 0x1p-63f;
        float sn, cn;
        sincospif(x, &sn, &cn);
        cs[lane + 32 * i] = make_float2(cn * a.mscale, sn * a.mscale);
      }
      __syncwarp();
      if (rot) {
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          const float4 v = *reinterpret_cast<const float4*>(pair_angles<INTER>(cs, j, c0, c1));
          w[j] = make_float2(v.x, v.y);
          w[j + 1] = make_float2(v.z, v.w);
        }
      }
      __syncwarp();
    }
    for (int h0 = first; __any_sync(0xffffffffu, h0 < heads); h0 += kDepth * kStep) {
      if (h0 != first) fetch(h0);
#pragma unroll
      for (int i = 0; i < kDepth; ++i) {
        const int h = h0 + i * kStep;
        const bool is_q = h < Hq, is_v = h >= Hq + Hkv;
        const float* gain = is_q ? a.q_gain : (is_v ? nullptr : a.k_gain);
        Chunk y0 = x0[i].get(), y1 = x1[i].get();
        if (a.q_gain || a.k_gain) {
          float ss = 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) ss += y0.v[j] * y0.v[j] + y1.v[j] * y1.v[j];
#pragma unroll
          for (int o = kLanes / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          if (h < heads && gain) {
            const float r = rsqrtf(ss * (1.f / D) + a.eps);
            Raw<float> g;
            g.load(gain + c0);
            Chunk x = g.get();
#pragma unroll
            for (int j = 0; j < 8; ++j) y0.v[j] *= r * x.v[j];
            g.load(gain + c1);
            x = g.get();
#pragma unroll
            for (int j = 0; j < 8; ++j) y1.v[j] *= r * x.v[j];
          }
        }
        if (h >= heads || (!is_q && dst < 0)) continue;
        if (rot && !is_v) rotate<INTER>(y0, y1, w);
        Out* o = is_q   ? static_cast<Out*>(a.q_out) + row * a.q_out_stride + (long)h * D
                 : is_v ? static_cast<Out*>(a.c.v) + dst + (h - Hq - Hkv) * a.c.head_stride
                        : static_cast<Out*>(a.c.k) + dst + (h - Hq) * a.c.head_stride;
        store8(o + c0, y0);
        store8(o + c1, y1);
      }
    }
  }
}

template <bool INTER, typename In, typename Out>
cudaError_t launch(const AppendArgs& a, int n_sm, cudaStream_t s) {
  // Eight warps a row up to four waves of them (bf16, 48 normed heads: 300 rows
  // 4.9 us against 11.0 with one warp, 1200 rows 10.9 against 11.3, 1600 rows 14.5
  // against 14.0): beyond, the repeated look-ups cost more than short rows save.
  const bool few = (long)a.s.n_rows * kFewWarps <= 64L * n_sm;
  const long warps = (long)a.s.n_rows * (few ? kFewWarps : kManyWarps);
  const long ctas = (warps + kAppendThreads / 32 - 1) / (kAppendThreads / 32);
  const long most = (long)append_ctas(few ? kFewWarps : kManyWarps) * n_sm;
  const dim3 grid((unsigned)(ctas < most ? ctas : most)), block(kAppendThreads);
  auto* kernel = few ? (a.c.d == 128 ? step_append_kernel<In, Out, 128, kFewWarps, INTER>
                                     : step_append_kernel<In, Out, 64, kFewWarps, INTER>)
                     : (a.c.d == 128 ? step_append_kernel<In, Out, 128, kManyWarps, INTER>
                                     : step_append_kernel<In, Out, 64, kManyWarps, INTER>);
  return launch_pdl(kernel, grid, block, 0, s, a);
}

template <bool INTER>
cudaError_t launch(const AppendArgs& a, int in_dtype, int out_dtype, int n_sm, cudaStream_t s) {
  if (out_dtype == DFLASH_BF16)
    return in_dtype == DFLASH_F32 ? launch<INTER, float, __nv_bfloat16>(a, n_sm, s)
                                  : launch<INTER, __nv_bfloat16, __nv_bfloat16>(a, n_sm, s);
  return in_dtype == DFLASH_F32 ? launch<INTER, float, __half>(a, n_sm, s) : launch<INTER, __half, __half>(a, n_sm, s);
}

}  // namespace

cudaError_t launch_step_append(const AppendArgs& a, int in_dtype, int out_dtype, int n_sm, cudaStream_t s) {
  return a.interleaved ? launch<true>(a, in_dtype, out_dtype, n_sm, s) : launch<false>(a, in_dtype, out_dtype, n_sm, s);
}

}  // namespace dfl

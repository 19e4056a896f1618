// step_append4.cu -- a step's queries, keys and values into a packed cache:
// per-head RMSNorm and RoPE as in step_append.cu, then the key and value rows
// rounded to 4 bits, in one pass.
//
// A head row goes in blocks of 16 elements.  With u the cache's unit,
//   s = e4m3(max |y| / (6 u)),  c_j = e2m1(y_j / (s u))    (nearest, ties to even)
// and the row stands for c_j s u.  A block with a NaN or an infinity gets s = NaN.
//
// The codes are those of y in exact arithmetic, so that a row's bits do not
// depend on how a kernel adds its squares, or on which kernel wrote it.  Values
// that pass through (and 16-bit ones times a power of two) are exact: their
// quotients by s are taken so that a tie stays one.  Normed or rotated keys
// carry an f32 error of at most `slack` times their pair: a row with a code or a
// scale that changes within it (one warp pass in fifty of normal rows) is
// computed again in 64 bits.
//
// Bytes bound it as in step_append.cu, whose division of rows among warps and
// lanes it shares.
#include "../../include/dflash.h"
#include "fp4.cuh"
#include "kernels.cuh"
#include "ptx.cuh"
#include "step.cuh"
#include "step_rows.cuh"

namespace dfl {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kFewWarps = 8;      // warps of a row when there are few rows
constexpr int kManyWarps = 1;     // and when there are many

// x to f32 towards zero, its last bit set where that is not exact: rounded
// again to a few bits it gives what x itself would.
__device__ __forceinline__ float odd_float(double x) {
  const float f = __double2float_rz(x);
  return (double)f == x ? f : __uint_as_float(__float_as_uint(f) | 1u);
}
// The same of a / b, b with few significant bits, r = 1 / b rounded.  EXACT16: a
// has at most 11 bits, and a quotient that is no tie is further from one than f32's
// step.
template <bool EXACT16>
__device__ __forceinline__ float odd_quotient(float a, float b, float r) {
  const float q0 = a * r;
  const float q = fmaf(fmaf(-q0, b, a), r, q0);   // a / b to the nearest; exact where that is
  if (EXACT16 || a == 0.f) return a == 0.f ? a : q;
  const float rest = fmaf(-q, b, a);
  if (rest == 0.f) return q;
  const bool below = (rest < 0.f) != (q < 0.f);   // the quotient is nearer to zero than q
  return __uint_as_float((__float_as_uint(q) - below) | 1u);
}

// What the rounded blocks of a lane's two chunks come to.
struct Codes {
  uint32_t code[2];   // eight codes each
  uint32_t scale;     // their blocks' scales, the first chunk's in the low byte
};

// A lane's two chunks once more, in 64 bits (all lanes of a warp come here).
struct Again {
  float x[16];
  const float* gain;
  int c0, c1;
  int lanes;          // of a head row
  bool rot, inter;
  int from0, from1;   // lane that holds the other chunk of each chunk's block
  bool second0, second1;   // as its second chunk
  float inv_unit;
};

__device__ __forceinline__ double max16(const double* y) {
  double m = 0.0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = fabs(y[j]) > m || isnan(y[j]) ? fabs(y[j]) : m;
  return m;
}

__device__ __noinline__ Codes code_again(const Again& g, const Append4Args& p, uint64_t pos, double2* cs) {
  const AppendArgs& a = p.a;
  const int lane = threadIdx.x & 31;
  double y[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) y[j] = g.x[j];
  double ss = 0.0;
#pragma unroll
  for (int j = 0; j < 16; ++j) ss += y[j] * y[j];
  for (int o = g.lanes / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  if (g.gain) {
    const double r = 1.0 / sqrt(ss / (16 * g.lanes) + p.eps);
#pragma unroll
    for (int j = 0; j < 16; ++j) y[j] *= r * (double)g.gain[(j < 8 ? g.c0 : g.c1 - 8) + j];
  }
  if (a.rot) {
    for (int i = lane; i < a.rot / 2; i += 32) {
      double sn, cn;
      sincospi((double)(long long)(pos * a.turns[i]) * 0x1p-63, &sn, &cn);
      cs[i] = make_double2(cn * p.mscale, sn * p.mscale);
    }
    __syncwarp();
    if (g.rot) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const double2 w = g.inter ? *pair_angles<true>(cs, j, g.c0, g.c1) : *pair_angles<false>(cs, j, g.c0, g.c1);
        const int at = (j < 4 ? 0 : 8) + 2 * (j & 3), ia = g.inter ? at : j, ib = g.inter ? at + 1 : j + 8;
        double ya = 0, yb = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) ya = i == ia ? y[i] : ya, yb = i == ib ? y[i] : yb;
        const double na = ya * w.x - yb * w.y, nb = yb * w.x + ya * w.y;
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] = i == ia ? na : i == ib ? nb : y[i];
      }
    }
    __syncwarp();
  }
#pragma unroll
  for (int j = 0; j < 16; ++j) y[j] *= g.inv_unit;
  const double m0 = max16(y), m1 = max16(y + 8);
  const double a0 = __shfl_sync(0xffffffffu, m0, g.from0), a1 = __shfl_sync(0xffffffffu, m1, g.from0);
  const double b0 = __shfl_sync(0xffffffffu, m0, g.from1), b1 = __shfl_sync(0xffffffffu, m1, g.from1);
  const double o[2] = {g.second0 ? a1 : a0, g.second1 ? b1 : b0}, m[2] = {m0, m1};
  Codes c;
  c.scale = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const double top = m[i] > o[i] || isnan(m[i]) ? m[i] : o[i];
    const bool fine = isfinite(top);
    const uint32_t sc = fine ? e4m3_of2(odd_float(fmin(top / 6.0, 448.0)), 0.f) & 0xFF : kScaleNaN;
    const float s = fine ? e4m3_to1(sc) : 0.f;
    float q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = s > 0.f ? odd_float(y[8 * i + j] / s) : fine ? copysignf(0.f, (float)y[8 * i + j]) : 0.f;
    c.code[i] = e2m1_of8(q);
    c.scale |= sc << (8 * i);
  }
  return c;
}

// Resident CTAs of an SM (the same as in step_append.cu).
constexpr int append_ctas(int warps) { return warps == kManyWarps ? 4 : 2; }

template <typename In, typename Out, int D, int WARPS, bool INTER>
__global__ void __launch_bounds__(kAppendThreads, append_ctas(WARPS))
    step_append4_kernel(const __grid_constant__ Append4Args p) {
  constexpr int kLanes = D / 16;               // lanes of a head row
  constexpr int kGroups = 32 / kLanes;         // head rows of a warp at once
  constexpr int kStep = WARPS * kGroups;       // heads between a lane's
  constexpr bool kExact16 = sizeof(In) == 2;
  __shared__ __align__(16) double2 cs_all[kAppendThreads / 32][D / 2];   // in f32, and in 64 bits where that is wanted
  pdl_wait();
  pdl_launch_dependents();
  const AppendArgs& a = p.a;
  const StepView& s = a.s;
  const int lane = threadIdx.x & 31, l = lane % kLanes;
  const int id = blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
  const int first = id % WARPS * kGroups + lane / kLanes;   // this lane's first head
  const int Hq = a.n_heads, Hkv = a.c.n_kv_heads, heads = Hq + 2 * Hkv;
  double2* cs64 = cs_all[threadIdx.x >> 5];
  float2* cs = reinterpret_cast<float2*>(cs64);
  // the two chunks of a head row this lane holds: a RoPE pair, or two of the
  // chunks behind the rotated ones
  const int pairs = a.rot / 16;
  const bool rot = l < pairs;
  const int c0 = 8 * (rot ? l : 2 * pairs + (l - pairs));
  const int c1 = rot ? c0 + 8 * pairs : c0 + 8 * (kLanes - pairs);
  // who holds the other chunk of a chunk's block, and as its second one
  auto holder = [&](int chunk, bool& second) {
    const int n = chunk < 2 * pairs ? pairs : kLanes - pairs, at = chunk < 2 * pairs ? chunk : chunk - 2 * pairs;
    second = at >= n;
    return (lane & ~(kLanes - 1)) + (chunk < 2 * pairs ? 0 : pairs) + at - (second ? n : 0);
  };
  bool second0, second1;
  const int from0 = holder((c0 / 8) ^ 1, second0), from1 = holder((c1 / 8) ^ 1, second1);
  const bool across = pairs & 1;               // else both are the neighbour's chunk of the same place
  // turns per position of the angles this lane forms
  uint64_t turn[D / 64];
#pragma unroll
  for (int i = 0; i < D / 64; ++i) turn[i] = a.turns[lane + 32 * i];
  // The f32 error of a key element, as a part of |y| + |other of its pair|, in
  // units of 2^-24: the norm's 21 (sum of squares 20 halved, its root 2, two
  // products and the rest), the rotation's 7 (angle 1.6, sine and cosine 1 of
  // themselves, mscale 1, the sum 2) times sqrt 2 for a pair seen after its
  // rotation, and the quotient's 2.
  const float slack = (a.k_gain ? (rot ? 42.f : 23.f) : rot ? 12.f : 0.f) * 0x1p-24f;

  const int stride = gridDim.x * (kAppendThreads / 32) / WARPS;
  for (int row = id / WARPS; row < s.n_rows; row += stride) {
    Raw<In> x0, x1;
    auto fetch = [&](int h) {
      if (h < heads) {
        const In* src = h < Hq ? static_cast<const In*>(a.q) + row * a.q_stride + (long)h * D
                        : h < Hq + Hkv ? static_cast<const In*>(a.k) + row * a.k_stride + (long)(h - Hq) * D
                                       : static_cast<const In*>(a.v) + row * a.v_stride + (long)(h - Hq - Hkv) * D;
        x0.load(src + c0);
        x1.load(src + c1);
      }
    };
    fetch(first);
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
    long dst = -1, sdst = -1;                              // its codes and scales in the cache
    if (own >= 0 && (own >> s.page_shift) < s.table_cols) {
      const int page = s.block_table[seq * s.table_stride + (own >> s.page_shift)];
      if (page >= 0 && page < s.n_pages) {
        dst = page * a.c.page_stride + (long)(own & (s.page_size - 1)) * a.c.row_stride;
        sdst = page * p.sc.page_stride + (long)(own & (s.page_size - 1)) * p.sc.row_stride;
      }
    }
    const uint64_t pos = (uint64_t)(a.positions ? (long)a.positions[row] : (long)s.prefix_len + own);
    float2 w[8];
    auto angles = [&]() {
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        // a signed fraction of a turn, times 2: sin and cos of pi x
        const float x = __ll2float_rn((long long)(pos * turn[i])) * 0x1p-63f;
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
    };
    if (a.rot) angles();
    for (int h = first; __any_sync(0xffffffffu, h < heads); h += kStep) {
      if (h != first) fetch(h);
      const bool is_q = h < Hq, is_v = h >= Hq + Hkv;
      const float* gain = is_q ? a.q_gain : (is_v ? nullptr : a.k_gain);
      Chunk y0 = x0.get(), y1 = x1.get();
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
      if (rot && !is_v) rotate<INTER>(y0, y1, w);
      if (h < heads && is_q) {
        Out* o = static_cast<Out*>(a.q_out) + row * a.q_out_stride + (long)h * D;
        store8(o + c0, y0);
        store8(o + c1, y1);
      }
      if (!__any_sync(0xffffffffu, h >= Hq && h < heads)) continue;
      // ---- 4 bits
      const float inv_unit = is_v ? p.v_inv_unit : p.k_inv_unit;
      const float eps = is_v ? 0.f : slack;
      float d0[8], d1[8];                     // what each element can be off by
      float hi[2], lo[2];                     // of the chunks' largest
      {
        uint32_t top[2] = {0, 0};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          // (beyond any code all the same, and still finite)
          top[0] = max(top[0], __float_as_uint(fabsf(y0.v[j])));
          top[1] = max(top[1], __float_as_uint(fabsf(y1.v[j])));
          y0.v[j] = fminf(fmaxf(y0.v[j] * inv_unit, -0x1p100f), 0x1p100f);
          y1.v[j] = fminf(fmaxf(y1.v[j] * inv_unit, -0x1p100f), 0x1p100f);
        }
        float m[2] = {0.f, 0.f}, n[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float u0 = INTER ? y0.v[j ^ 1] : y1.v[j], u1 = INTER ? y1.v[j ^ 1] : y0.v[j];
          d0[j] = eps * (fabsf(y0.v[j]) + fabsf(u0));
          d1[j] = eps * (fabsf(y1.v[j]) + fabsf(u1));
          m[0] = fmaxf(m[0], fabsf(y0.v[j]) + d0[j]);
          m[1] = fmaxf(m[1], fabsf(y1.v[j]) + d1[j]);
          n[0] = fmaxf(n[0], fabsf(y0.v[j]) - d0[j]);
          n[1] = fmaxf(n[1], fabsf(y1.v[j]) - d1[j]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (top[i] >= 0x7F800000u) m[i] = INFINITY;
          const float mo = __shfl_sync(0xffffffffu, m[i], i ? from1 : from0);
          const float no = __shfl_sync(0xffffffffu, n[i], i ? from1 : from0);
          hi[i] = fmaxf(m[i], mo);
          lo[i] = fmaxf(n[i], no);
        }
        if (across) {                          // (the block's other chunk may lie in another place)
          const float mo0 = __shfl_sync(0xffffffffu, m[1], from0), no0 = __shfl_sync(0xffffffffu, n[1], from0);
          const float mo1 = __shfl_sync(0xffffffffu, m[0], from1), no1 = __shfl_sync(0xffffffffu, n[0], from1);
          if (second0) hi[0] = fmaxf(m[0], mo0), lo[0] = fmaxf(n[0], no0);
          if (!second1) hi[1] = fmaxf(m[1], mo1), lo[1] = fmaxf(n[1], no1);
        }
      }
      Codes c;
      c.scale = 0;
      bool border = false;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const Chunk& y = i ? y1 : y0;
        const float* d = i ? d1 : d0;
        const bool fine = hi[i] < INFINITY;
        float q[8];
        uint32_t sc;
        if (eps == 0.f) {
          sc = e4m3_of2(odd_quotient<kExact16>(fminf(hi[i], 0x1p20f), 6.f, 1.f / 6.f), 0.f) & 0xFF;
        } else {
          const uint32_t two = e4m3_of2(lo[i] * (1.f / 6.f) * (1.f - 0x1p-22f), hi[i] * (1.f / 6.f) * (1.f + 0x1p-22f));
          sc = two & 0xFF;
          border |= fine && sc != two >> 8;
        }
        const float sf = e4m3_to1(sc), r = fine && sf > 0.f ? __frcp_rn(sf) : 0.f;
        if (eps == 0.f) {
#pragma unroll
          for (int j = 0; j < 8; ++j) q[j] = r > 0.f ? odd_quotient<kExact16>(y.v[j], sf, r) : fine ? y.v[j] * 0.f : 0.f;
          c.code[i] = e2m1_of8(q);
        } else {
          float t[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float e = d[j] * r;
            q[j] = fine ? fmaf(y.v[j], r, -e) : 0.f;
            t[j] = fine ? fmaf(y.v[j], r, e) : 0.f;
          }
          c.code[i] = e2m1_of8(q);
          border |= c.code[i] != e2m1_of8(t);
        }
        c.scale |= (fine ? sc : kScaleNaN) << (8 * i);
      }
      border &= h >= Hq && h < heads;
      if (__any_sync(0xffffffffu, border)) {
        Again g;
        const Chunk z0 = x0.get(), z1 = x1.get();
#pragma unroll
        for (int j = 0; j < 8; ++j) g.x[j] = h < heads ? z0.v[j] : 0.f, g.x[8 + j] = h < heads ? z1.v[j] : 0.f;
        g.gain = h < heads ? gain : nullptr;
        g.c0 = c0, g.c1 = c1, g.lanes = kLanes, g.rot = rot, g.inter = INTER;
        g.from0 = from0, g.from1 = from1, g.second0 = second0, g.second1 = second1;
        g.inv_unit = inv_unit;
        const Codes b = code_again(g, p, pos, cs64);
        if (eps != 0.f) c = b;
      }
      if (h < Hq || h >= heads || dst < 0) continue;
      const int kv = h - Hq - (is_v ? Hkv : 0);
      uint8_t* o = static_cast<uint8_t*>(is_v ? a.c.v : a.c.k) + dst + kv * a.c.head_stride;
      *reinterpret_cast<uint32_t*>(o + c0 / 2) = c.code[0];
      *reinterpret_cast<uint32_t*>(o + c1 / 2) = c.code[1];
      uint8_t* so = static_cast<uint8_t*>(is_v ? p.sc.v : p.sc.k) + sdst + kv * p.sc.head_stride;
      if (!(c0 & 8)) so[c0 / 16] = (uint8_t)c.scale;
      if (!(c1 & 8)) so[c1 / 16] = (uint8_t)(c.scale >> 8);
      Out* vo = static_cast<Out*>(is_v ? p.v_values : p.k_values);
      if (vo) {
        vo += row * (is_v ? p.v_values_stride : p.k_values_stride) + (long)kv * D;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float f = e4m3_to1(c.scale >> (8 * i)) * (is_v ? p.v_unit : p.k_unit);
          uint32_t e[4];
          e2m1_to8(c.code[i], e);
          Chunk y;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 t = __half22float2(as_half2(e[j]));
            y.v[2 * j] = t.x * f;
            y.v[2 * j + 1] = t.y * f;
          }
          store8(vo + (i ? c1 : c0), y);
        }
      }
    }
  }
}

template <bool INTER, typename In, typename Out>
cudaError_t launch(const Append4Args& p, int n_sm, cudaStream_t s) {
  const AppendArgs& a = p.a;
  // eight warps a row up to four waves of them, as in step_append.cu
  const bool few = (long)a.s.n_rows * kFewWarps <= 64L * n_sm;
  const long warps = (long)a.s.n_rows * (few ? kFewWarps : kManyWarps);
  const long ctas = (warps + kAppendThreads / 32 - 1) / (kAppendThreads / 32);
  const long most = (long)append_ctas(few ? kFewWarps : kManyWarps) * n_sm;
  const dim3 grid((unsigned)(ctas < most ? ctas : most)), block(kAppendThreads);
  auto* kernel = few ? (a.c.d == 128 ? step_append4_kernel<In, Out, 128, kFewWarps, INTER>
                                     : step_append4_kernel<In, Out, 64, kFewWarps, INTER>)
                     : (a.c.d == 128 ? step_append4_kernel<In, Out, 128, kManyWarps, INTER>
                                     : step_append4_kernel<In, Out, 64, kManyWarps, INTER>);
  return launch_pdl(kernel, grid, block, 0, s, p);
}

template <bool INTER>
cudaError_t launch(const Append4Args& p, int in_dtype, int out_dtype, int n_sm, cudaStream_t s) {
  if (out_dtype == DFLASH_BF16)
    return in_dtype == DFLASH_F32 ? launch<INTER, float, __nv_bfloat16>(p, n_sm, s)
                                  : launch<INTER, __nv_bfloat16, __nv_bfloat16>(p, n_sm, s);
  return in_dtype == DFLASH_F32 ? launch<INTER, float, __half>(p, n_sm, s) : launch<INTER, __half, __half>(p, n_sm, s);
}

}  // namespace

cudaError_t launch_step_append4(const Append4Args& p, int in_dtype, int out_dtype, int n_sm, cudaStream_t s) {
  return p.a.interleaved ? launch<true>(p, in_dtype, out_dtype, n_sm, s)
                         : launch<false>(p, in_dtype, out_dtype, n_sm, s);
}

}  // namespace dfl

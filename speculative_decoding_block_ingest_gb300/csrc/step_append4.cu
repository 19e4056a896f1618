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
// scale that changes within it (one pass of a warp in fifty over normal rows) is
// computed again in two floats, and if that is not enough (2^-38 of a pair) in 64
// bits.  64 bits at once took 18 us for one such row.
//
// 34912 rows of 32 query and 16 other heads take 195 us (4.1 TB/s; instructions, 58% of
// the issue slots of 16 warps an SM); step_append.cu, whose division of rows among
// warps and lanes it shares, is bound by the bytes.  The later computations are inline:
// a call among them cost every row 40 us of the 250 it took then.
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
// The same of a / b, b with few significant bits, r = 1 / b rounded; large ones as
// they come.  EXACT16: a has at most 11 bits, and a quotient that is no tie is further
// from one than f32's step.
template <bool EXACT16>
__device__ __forceinline__ float odd_quotient(float a, float b, float r) {
  const float q0 = a * r;
  if (!(fabsf(q0) < 0x1p20f) || q0 == 0.f) return q0;
  const float q = fmaf(fmaf(-q0, b, a), r, q0);   // a / b to the nearest; exact where that is
  if (EXACT16) return q;
  const float rest = fmaf(-q, b, a);
  if (rest == 0.f) return q;
  const bool below = (rest < 0.f) != (q < 0.f);   // the quotient is nearer to zero than q
  return __uint_as_float((__float_as_uint(q) - below) | 1u);
}

// The reciprocal of a scale, rounded down, and what that leaves: with both, fmaf(a, h, a l)
// of a 16-bit a is a tie where a / s is one (49 products of a scale's bits with a tie's,
// each checked: one float alone misses 11), and keeps a zero's sign.
struct Reciprocal {
  float h, l;
  __device__ __forceinline__ Reciprocal(float s, float inv_unit) : h(0.f), l(0.f) {
    if (s > 0.f) {
      const float r = __frcp_rd(s);
      h = r * inv_unit;
      l = fmaf(-r, s, 1.f) * h;
    }
  }
};
// The larger, or NaN where one is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}

// What the rounded blocks of a lane's two chunks come to.
struct Codes {
  uint32_t code[2];   // eight codes each
  uint32_t scale;     // their blocks' scales, the first chunk's in the low byte
};

// Which elements of a head row a lane has: the two chunks that RoPE pairs, or two of
// the chunks behind the rotated ones; and who has the other chunk of each one's block.
template <int D>
struct Lane {
  static constexpr int kLanes = D / 16;        // lanes of a head row
  int c0, c1;                                  // the chunks' first elements
  int from0, from1;                            // lanes that hold the other chunk
  bool rot, second0, second1;                  // (as their second one)
  __device__ __forceinline__ Lane(int rot_dim, int lane) {
    const int pairs = rot_dim / 16, l = lane % kLanes;
    rot = l < pairs;
    c0 = 8 * (rot ? l : 2 * pairs + (l - pairs));
    c1 = rot ? c0 + 8 * pairs : c0 + 8 * (kLanes - pairs);
    auto holder = [&](int chunk, bool& second) {
      const int n = chunk < 2 * pairs ? pairs : kLanes - pairs, at = chunk < 2 * pairs ? chunk : chunk - 2 * pairs;
      second = at >= n;
      return (lane & ~(kLanes - 1)) + (chunk < 2 * pairs ? 0 : pairs) + at - (second ? n : 0);
    };
    from0 = holder((c0 / 8) ^ 1, second0);
    from1 = holder((c1 / 8) ^ 1, second1);
  }
};

// Codes and scales of a lane's chunks of a key or value row into the cache, and the
// values they stand for to where they are wanted.
template <typename Out, int D>
__device__ __forceinline__ void store_codes(const Append4Args& p, int c0, int c1, const Codes& c, long row, int h, long dst,
                                            long sdst) {
  const AppendArgs& a = p.a;
  const bool is_v = h >= a.n_heads + a.c.n_kv_heads;
  const int kv = h - a.n_heads - (is_v ? a.c.n_kv_heads : 0);
  uint8_t* o = static_cast<uint8_t*>(is_v ? a.c.v : a.c.k) + dst + kv * a.c.head_stride;
  *reinterpret_cast<uint32_t*>(o + c0 / 2) = c.code[0];
  *reinterpret_cast<uint32_t*>(o + c1 / 2) = c.code[1];
  uint8_t* so = static_cast<uint8_t*>(is_v ? p.sc.v : p.sc.k) + sdst + kv * p.sc.head_stride;
  if (!(c0 & 8)) so[c0 / 16] = (uint8_t)c.scale;
  if (!(c1 & 8)) so[c1 / 16] = (uint8_t)(c.scale >> 8);
  Out* vo = static_cast<Out*>(is_v ? p.v_values : p.k_values);
  if (!vo) return;
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

__device__ __forceinline__ double largest8(const double* y) {
  double m = 0.0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = fabs(y[j]) > m || isnan(y[j]) ? fabs(y[j]) : m;
  return m;
}

// A warp's key rows (head h of each lane's group) in 64 bits.
template <typename In, typename Out, int D, bool INTER>
__device__ __forceinline__ void code_exactly(const Append4Args& p, long row, int h, long dst, long sdst, uint64_t pos,
                                        double2* cs) {
  const AppendArgs& a = p.a;
  const int lane = threadIdx.x & 31;
  const Lane<D> at(a.rot, lane);
  const bool mine = h >= a.n_heads && h < a.n_heads + a.c.n_kv_heads;
  double y[16];
  {
    Raw<In> x0, x1;
    const In* src = static_cast<const In*>(a.k) + row * a.k_stride + (long)(mine ? h - a.n_heads : 0) * D;
    x0.load(src + at.c0);
    x1.load(src + at.c1);
    const Chunk z0 = x0.get(), z1 = x1.get();
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = z0.v[j], y[8 + j] = z1.v[j];
  }
  if (a.k_gain) {
    double ss = 0.0;
#pragma unroll
    for (int j = 0; j < 16; ++j) ss += y[j] * y[j];
    for (int o = Lane<D>::kLanes / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const double r = 1.0 / sqrt(ss / D + p.eps);
#pragma unroll
    for (int j = 0; j < 16; ++j) y[j] *= r * (double)a.k_gain[(j < 8 ? at.c0 : at.c1 - 8) + j];
  }
  if (a.rot) {
    for (int i = lane; i < a.rot / 2; i += 32) {
      double sn, cn;
      sincospi((double)(long long)(pos * a.turns[i]) * 0x1p-63, &sn, &cn);
      cs[i] = make_double2(cn * p.mscale, sn * p.mscale);
    }
    __syncwarp();
    if (at.rot) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const double2 w = *pair_angles<INTER>(cs, j, at.c0, at.c1);
        const int first = (j < 4 ? 0 : 8) + 2 * (j & 3);
        double &ya = y[INTER ? first : j], &yb = y[INTER ? first + 1 : j + 8];
        const double u = ya, t = yb;
        ya = u * w.x - t * w.y;
        yb = t * w.x + u * w.y;
      }
    }
    __syncwarp();
  }
#pragma unroll
  for (int j = 0; j < 16; ++j) y[j] *= p.k_inv_unit;
  const double m0 = largest8(y), m1 = largest8(y + 8);
  const double a0 = __shfl_sync(0xffffffffu, m0, at.from0), a1 = __shfl_sync(0xffffffffu, m1, at.from0);
  const double b0 = __shfl_sync(0xffffffffu, m0, at.from1), b1 = __shfl_sync(0xffffffffu, m1, at.from1);
  const double o[2] = {at.second0 ? a1 : a0, at.second1 ? b1 : b0}, m[2] = {m0, m1};
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
    for (int j = 0; j < 8; ++j)
      q[j] = s > 0.f ? odd_float(y[8 * i + j] / s) : fine ? copysignf(0.f, (float)y[8 * i + j]) : 0.f;
    c.code[i] = e2m1_of8(q);
    c.scale |= sc << (8 * i);
  }
  if (mine && dst >= 0) store_codes<Out, D>(p, at.c0, at.c1, c, row, h, dst, sdst);
}

// Resident CTAs of an SM (34912 rows of 32 and 16 heads: 195 us; three, whose registers
// spill, 293).
constexpr int kAppendCtas = 2;

// Numbers of two floats (the second at most half a step of the first), with Knuth's error-free
// sum, Dekker's for an ordered pair, and the product's error by fma (Ogita, Rump and Oishi,
// "Accurate sum and dot product", 2005): about 2^-46 of a sum's or product's terms is lost.
struct Two {
  float h, l;
};
__device__ __forceinline__ Two quick(float a, float b) {   // |a| >= |b|
  const float s = __fadd_rn(a, b);
  return {s, __fsub_rn(b, __fsub_rn(s, a))};
}
__device__ __forceinline__ Two sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Two product(float a, float b) {
  const float p = __fmul_rn(a, b);
  return {p, __fmaf_rn(a, b, -p)};
}
__device__ __forceinline__ Two operator+(Two a, Two b) {
  const Two s = sum(a.h, b.h);
  return quick(s.h, __fadd_rn(s.l, __fadd_rn(a.l, b.l)));
}
__device__ __forceinline__ Two operator*(Two a, Two b) {
  const Two p = product(a.h, b.h);
  return quick(p.h, __fadd_rn(p.l, __fmaf_rn(a.h, b.l, __fmul_rn(a.l, b.h))));
}
__device__ __forceinline__ Two operator*(Two a, float b) {
  const Two p = product(a.h, b);
  return quick(p.h, __fmaf_rn(a.l, b, p.l));
}
__device__ __forceinline__ Two operator-(Two a) { return {-a.h, -a.l}; }
// (sums above lose the sign of a zero, which one float's arithmetic gives)
__device__ __forceinline__ Two zero_as(Two a, float z) { return a.h == 0.f ? Two{z, 0.f} : a; }
__device__ __forceinline__ Two two(double x) {
  const float h = (float)x;
  return {h, (float)(x - h)};
}

// Sine and cosine of u / 2^64 turns: quarters off, then the Taylor series, whose terms
// from the fifth on are small enough for one float (up to 4e-7 of the sum: 2^-45).
__device__ __forceinline__ void sine_cosine(uint64_t u, Two& sn, Two& cn) {
  const uint64_t quarter = (u + (1ull << 61)) >> 62;
  const long long r = (long long)(u - (quarter << 62));
  const float rh = __ll2float_rn(r), rl = __ll2float_rn(r - (long long)rh);
  const Two x = quick(rh, rl) * Two{0x1.921fb6p-62f, -0x1.777a5cp-87f};   // 2 pi / 2^64
  const Two z = x * x;
  const float zh = z.h;
  // sin x = x (1 - z/3! + z^2/5! - ...), cos x = 1 - z/2! + z^2/4! - ...
  const float s4 = fmaf(zh, fmaf(zh, fmaf(zh, -7.6471637e-13f, 1.6059044e-10f), -2.5052108e-8f), 2.7557319e-6f);
  const float c4 = fmaf(zh, fmaf(zh, fmaf(zh, fmaf(zh, 4.7794773e-14f, -1.1470746e-11f), 2.0876757e-9f), -2.7557319e-7f),
                        2.4801587e-5f);
  Two s = z * s4 + Two{-0x1.a01a02p-13f, 0x1.7f97fap-39f};
  Two c = z * c4 + Two{-0x1.6c16c2p-10f, 0x1.27d27ep-35f};
  s = z * s, c = z * c;
  s = s + Two{0x1.111112p-7f, -0x1.dddddep-32f};
  c = c + Two{0x1.555556p-5f, -0x1.555556p-30f};
  s = z * s + Two{-0x1.555556p-3f, 0x1.555556p-28f};
  c = z * c + Two{-0.5f, 0.f};
  s = x * (z * s + Two{1.f, 0.f});
  c = z * c + Two{1.f, 0.f};
  sn = quarter & 1 ? c : s;
  cn = quarter & 1 ? s : c;
  if (quarter & 2) sn = -sn;
  if ((quarter + 1) & 2) cn = -cn;
}

// a / b as odd_quotient has it; unsure where a is nearer than `off` to a tie.
__device__ __forceinline__ float odd_quotient(Two a, float b, float r, float off, bool& unsure) {
  const float q0 = a.h * r;
  if (!(fabsf(q0) < 0x1p20f) || q0 == 0.f) return q0;
  const float q = fmaf(fmaf(-q0, b, a.h) + a.l, r, q0);
  const float rest = fmaf(-q, b, a.h) + a.l;
  unsure |= fabsf(rest) <= off && !(__float_as_uint(q) & 0xFFFFu);   // (ties have 7 bits at most)
  const bool below = (rest < 0.f) != (q < 0.f);
  return rest == 0.f ? q : __uint_as_float((__float_as_uint(q) - below) | 1u);
}

// A warp's key rows (head h of each lane's group) once more, in two floats.
template <typename In, typename Out, int D, bool INTER>
__device__ __forceinline__ void code_again(const Append4Args& p, long row, int h, long dst, long sdst, uint64_t pos,
                                        double2* cs64) {
  const AppendArgs& a = p.a;
  const int lane = threadIdx.x & 31;
  const Lane<D> at(a.rot, lane);
  const bool mine = h >= a.n_heads && h < a.n_heads + a.c.n_kv_heads;
  float4* cs = reinterpret_cast<float4*>(cs64);
  bool unsure = false;
  float x[16];
  {
    Raw<In> x0, x1;
    const In* src = static_cast<const In*>(a.k) + row * a.k_stride + (long)(mine ? h - a.n_heads : 0) * D;
    x0.load(src + at.c0);
    x1.load(src + at.c1);
    const Chunk z0 = x0.get(), z1 = x1.get();
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = z0.v[j], x[8 + j] = z1.v[j];
  }
  Two y[16];
  if (a.k_gain) {
    Two ss{0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 16; ++j) ss = ss + product(x[j], x[j]);
    for (int o = Lane<D>::kLanes / 2; o; o >>= 1)
      ss = ss + Two{__shfl_xor_sync(0xffffffffu, ss.h, o), __shfl_xor_sync(0xffffffffu, ss.l, o)};
    const Two m = ss * (1.f / D) + two(p.eps);
    unsure = !(m.h < INFINITY && m.h > 0.f);
    // 1 / sqrt m = r + r (1 - m r^2) / 2 to the square of the first one's error
    const float r0 = rsqrtf(m.h);
    const Two one = m * product(r0, r0);
    const float miss = (1.f - one.h) - one.l;
    const Two r = quick(r0, 0.5f * r0 * miss);
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const Two g = r * a.k_gain[(j < 8 ? at.c0 : at.c1 - 8) + j];
      y[j] = zero_as(g * x[j], g.h * x[j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j) y[j] = {x[j], 0.f};
  }
  if (a.rot) {
    const Two ms = two(p.mscale);
    for (int i = lane; i < a.rot / 2; i += 32) {
      Two sn, cn;
      sine_cosine(pos * a.turns[i], sn, cn);
      sn = sn * ms, cn = cn * ms;
      cs[i] = make_float4(cn.h, cn.l, sn.h, sn.l);
    }
    __syncwarp();
    if (at.rot) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float4 w = *pair_angles<INTER>(cs, j, at.c0, at.c1);
        const int first = (j < 4 ? 0 : 8) + 2 * (j & 3);
        Two &ya = y[INTER ? first : j], &yb = y[INTER ? first + 1 : j + 8];
        const Two u = ya, t = yb, cn{w.x, w.y}, sn{w.z, w.w};
        ya = zero_as(u * cn + -(t * sn), u.h * cn.h - t.h * sn.h);
        yb = zero_as(t * cn + u * sn, t.h * cn.h + u.h * sn.h);
      }
    }
    __syncwarp();
  }
  // a chunk's largest, and its largest pair (as its error goes)
  Two top[2] = {{0.f, 0.f}, {0.f, 0.f}};
  float wide[2] = {0.f, 0.f};
  uint32_t bits[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const int i = j / 8;
    const Two v = y[j].h < 0.f ? -y[j] : y[j];
    if (v.h > top[i].h || (v.h == top[i].h && v.l > top[i].l)) top[i] = v;
    bits[i] = max(bits[i], __float_as_uint(fabsf(y[j].h)));
    wide[i] = fmaxf(wide[i], fabsf(y[j].h) + fabsf(y[INTER ? j ^ 1 : j ^ 8].h));
  }
  Codes c;
  c.scale = 0;
  const Two t0 = top[0], t1 = top[1];
  const float w0 = wide[0], w1 = wide[1];
  const uint32_t b0 = bits[0], b1 = bits[1];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int from = i ? at.from1 : at.from0;
    const bool second = i ? at.second1 : at.second0;
    auto other = [&](auto v0, auto v1) {
      const auto x0 = __shfl_sync(0xffffffffu, v0, from), x1 = __shfl_sync(0xffffffffu, v1, from);
      return second ? x1 : x0;
    };
    const Two o{other(t0.h, t1.h), other(t0.l, t1.l)};
    Two big = i ? t1 : t0;
    if (o.h > big.h || (o.h == big.h && o.l > big.l)) big = o;
    const float off = 0x1p-38f * fmaxf(i ? w1 : w0, other(w0, w1));
    const bool fine = max(i ? b1 : b0, other(b0, b1)) < 0x7F800000u;
    bool open = false;
    const uint32_t sc = e4m3_of2(odd_quotient(big * p.k_inv_unit, 6.f, 1.f / 6.f, off * p.k_inv_unit, open), 0.f) & 0xFF;
    const float sf = e4m3_to1(sc), r = sf > 0.f ? __frcp_rn(sf) * p.k_inv_unit : 0.f;
    float q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = odd_quotient(y[8 * i + j], sf * p.k_unit, r, off, open);
    c.code[i] = fine ? e2m1_of8(q) : 0;
    c.scale |= (fine ? sc : kScaleNaN) << (8 * i);
    unsure |= fine && open;
  }
  if (__any_sync(0xffffffffu, mine && unsure)) return code_exactly<In, Out, D, INTER>(p, row, h, dst, sdst, pos, cs64);
  if (mine && dst >= 0) store_codes<Out, D>(p, at.c0, at.c1, c, row, h, dst, sdst);
}

template <typename In, typename Out, int D, int WARPS, bool INTER>
__global__ void __launch_bounds__(kAppendThreads, kAppendCtas)
    step_append4_kernel(const __grid_constant__ Append4Args p) {
  constexpr int kLanes = D / 16;               // lanes of a head row
  constexpr int kGroups = 32 / kLanes;         // head rows of a warp at once
  constexpr int kStep = WARPS * kGroups;       // heads between a lane's
  constexpr bool kExact16 = sizeof(In) == 2;
  constexpr int kCtaRows = kAppendThreads / 32 / WARPS;   // rows of a CTA at a time
  __shared__ __align__(16) double2 cs_all[kAppendThreads / 32][D / 2];   // in f32, and in 64 bits where that is wanted
  pdl_wait();
  pdl_launch_dependents();
  const AppendArgs& a = p.a;
  const StepView& s = a.s;
  const int lane = threadIdx.x & 31;
  const int id = blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
  const int Hq = a.n_heads, Hkv = a.c.n_kv_heads, heads = Hq + 2 * Hkv;
  const int first = id % WARPS * kGroups + lane / kLanes;   // this lane's first head
  double2* cs64 = cs_all[threadIdx.x >> 5];
  float2* cs = reinterpret_cast<float2*>(cs64);
  const Lane<D> at(a.rot, lane);
  const int c0 = at.c0, c1 = at.c1, from0 = at.from0, from1 = at.from1;
  const bool rot = at.rot;
  const bool across = a.rot / 16 & 1;          // else both are the neighbour's chunk of the same place
  // turns per position of the angles this lane forms
  uint64_t turn[D / 64];
#pragma unroll
  for (int i = 0; i < D / 64; ++i) turn[i] = a.turns[lane + 32 * i];
  // The f32 error of a key element, as a part of |y| + |other of its pair|, in
  // units of 2^-24: the norm's 17 (20 of the sum of squares halved, its root 4, the
  // products with the gain and with the quotient's factor), the rotation's 8 (angle 1.6,
  // sine and cosine 2, mscale 1 and its product 1, the sum 2) times sqrt 2 for a pair seen
  // after its rotation, and the quotient's 3.
  const float slack = (a.k_gain ? (rot ? 39.f : 21.f) : rot ? 15.f : 0.f) * 0x1p-24f;

  // A CTA's rows: each warp takes the next one where a row is a warp's, because some are
  // computed again.
  __shared__ int taken;
  if (WARPS == 1) {
    if (threadIdx.x == 0) taken = kCtaRows;
    __syncthreads();
  }
  const int stride = gridDim.x * (kAppendThreads / 32) / WARPS;
  auto behind = [&](int row) -> int {
    if (WARPS > 1) return row + stride;
    int k = 0;
    if (lane == 0) k = atomicAdd(&taken, 1);
    k = __shfl_sync(0xffffffffu, k, 0);
    return k / kCtaRows * stride + (int)blockIdx.x * kCtaRows + k % kCtaRows;
  };
  Raw<In> x0, x1;   // the next head's chunks
  auto fetch = [&](int row, int h) {
    if (h < heads) {
      const In* src = h < Hq ? static_cast<const In*>(a.q) + row * a.q_stride + (long)h * D
                      : h < Hq + Hkv ? static_cast<const In*>(a.k) + row * a.k_stride + (long)(h - Hq) * D
                                     : static_cast<const In*>(a.v) + row * a.v_stride + (long)(h - Hq - Hkv) * D;
      x0.load(src + c0);
      x1.load(src + c1);
    }
  };
  for (int row = id / WARPS; row < s.n_rows; row = behind(row)) {
    fetch(row, first);
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
    uint32_t again = 0;                                    // passes over heads with a border
    for (int h = first; __any_sync(0xffffffffu, h < heads); h += kStep) {
      const bool is_q = h < Hq, is_v = h >= Hq + Hkv;
      const float* gain = h >= heads || is_v ? nullptr : is_q ? a.q_gain : a.k_gain;
      Chunk y0 = x0.get(), y1 = x1.get();
      fetch(row, h + kStep);   // (on its way under this one's arithmetic)
      float rn = 1.f;        // the norm's factor, which the rotation lets pass
      const bool only_v = __all_sync(0xffffffffu, is_v);
      if (!only_v && (a.q_gain || a.k_gain)) {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) ss += y0.v[j] * y0.v[j] + y1.v[j] * y1.v[j];
#pragma unroll
        for (int o = kLanes / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (gain) {
          rn = rsqrtf(ss * (1.f / D) + a.eps);
          Raw<float> g;
          g.load(gain + c0);
          Chunk x = g.get();
#pragma unroll
          for (int j = 0; j < 8; ++j) y0.v[j] *= x.v[j];
          g.load(gain + c1);
          x = g.get();
#pragma unroll
          for (int j = 0; j < 8; ++j) y1.v[j] *= x.v[j];
        }
      }
      if (rot && !is_v) rotate<INTER>(y0, y1, w);
      if (is_q) {
#pragma unroll
        for (int j = 0; j < 8; ++j) y0.v[j] *= rn, y1.v[j] *= rn;
        Out* o = static_cast<Out*>(a.q_out) + row * a.q_out_stride + (long)h * D;
        store8(o + c0, y0);
        store8(o + c1, y1);
      }
      if (!__any_sync(0xffffffffu, h >= Hq && h < heads)) continue;
      // ---- 4 bits
      // the chunks' largest element (NaN is above all) and largest pair, then their blocks'
      float t0 = 0.f, t1 = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        t0 = max_nan(t0, fabsf(y0.v[j]));
        t1 = max_nan(t1, fabsf(y1.v[j]));
      }
      // a lane's two values to its blocks' (whose other chunk may lie in another place)
      auto of_blocks = [&](float x0, float x1, auto larger, float* to) {
        to[0] = larger(x0, __shfl_sync(0xffffffffu, x0, from0));
        to[1] = larger(x1, __shfl_sync(0xffffffffu, x1, from1));
        if (across) {
          const float o0 = __shfl_sync(0xffffffffu, x1, from0), o1 = __shfl_sync(0xffffffffu, x0, from1);
          if (at.second0) to[0] = larger(x0, o0);
          if (!at.second1) to[1] = larger(x1, o1);
        }
      };
      float top[2], wide[2] = {0.f, 0.f}, both[8];
      of_blocks(t0, t1, [](float x, float y) { return max_nan(x, y); }, top);
      if (!only_v && (a.k_gain || a.rot)) {
        float w0 = 0.f, w1 = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int at = (j < 4 ? 0 : 1), k = 2 * (j & 3);
          both[j] = INTER ? fabsf((at ? y1 : y0).v[k]) + fabsf((at ? y1 : y0).v[k + 1]) : fabsf(y0.v[j]) + fabsf(y1.v[j]);
          if (!INTER || j < 4) w0 = fmaxf(w0, both[j]);
          else w1 = fmaxf(w1, both[j]);
        }
        of_blocks(w0, INTER ? w1 : w0, [](float x, float y) { return fmaxf(x, y); }, wide);
      }
      Codes c;
      c.scale = 0;
      bool border = false;
      if (is_v || slack == 0.f) {
        const float inv_unit = is_v ? p.v_inv_unit : p.k_inv_unit, unit = is_v ? p.v_unit : p.k_unit;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const Chunk& y = i ? y1 : y0;
          const uint32_t sc = e4m3_of2(odd_quotient<kExact16>(top[i] * inv_unit, 6.f, 1.f / 6.f), 0.f) & 0xFF;
          const float sf = e4m3_to1(sc);
          const Reciprocal r(sf, inv_unit);
          float q[8];
#pragma unroll
          for (int j = 0; j < 8; ++j)
            q[j] = kExact16 ? fmaf(y.v[j], r.h, y.v[j] * r.l) : odd_quotient<false>(y.v[j], sf * unit, r.h);
          const bool fine = top[i] < INFINITY;
          c.code[i] = fine ? e2m1_of8(q) : 0;
          c.scale |= (fine ? sc : kScaleNaN) << (8 * i);
        }
      } else {
        border = !(rn < INFINITY);             // (a sum of squares that is 0 or not finite is looked at again)
        const float scaled = p.k_inv_unit * rn, six = scaled * (1.f / 6.f);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const Chunk& y = i ? y1 : y0;
          const float off = slack * wide[i];
          const uint32_t two = e4m3_of2((top[i] - off) * six * (1.f - 0x1p-22f), (top[i] + off) * six * (1.f + 0x1p-22f));
          const uint32_t sc = two & 0xFF;
          const float sf = e4m3_to1(sc), r = sf > 0.f ? __frcp_rn(sf) * scaled : 0.f, er = slack * r;
          float q[8], t[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float e = er * both[INTER ? 4 * i + j / 2 : j];
            q[j] = fmaf(y.v[j], r, -e);
            t[j] = fmaf(y.v[j], r, e);
          }
          const bool fine = top[i] < INFINITY;
          const uint32_t code = e2m1_of8(q);
          border |= fine && (sc != two >> 8 || code != e2m1_of8(t));
          c.code[i] = fine ? code : 0;
          c.scale |= (fine ? sc : kScaleNaN) << (8 * i);
        }
        border |= !(rn > 0.f);
      }
      const bool mine = h >= Hq && h < heads;
      if (__any_sync(0xffffffffu, border && mine)) again |= 1u << min((h - first) / kStep, 31);
      if (mine && dst >= 0) store_codes<Out, D>(p, c0, c1, c, row, h, dst, sdst);
    }
    // those with a border, when nothing else is held (bit 31: all from there on)
    for (int i = 0; again; ++i) {
      if (!(again >> min(i, 31) & 1)) continue;
      if (i < 31) again &= ~(1u << i);
      const int h = first + i * kStep;
      if (!__any_sync(0xffffffffu, h < heads)) break;
      code_again<In, Out, D, INTER>(p, row, h, dst, sdst, pos, cs64);
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
  const long most = (long)kAppendCtas * n_sm;
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

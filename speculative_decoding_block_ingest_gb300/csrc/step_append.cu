// step_append.cu -- a step's queries, keys and values: per-head RMSNorm, RoPE
// and the paged-cache rows, in one pass.
//
// For a query or key head row x of d elements at position p:
//   y = x * rsqrt(mean(x^2) + eps) * gain          (where there is a gain)
//   y_j, y_{j+h} = y_j c_j - y_{j+h} s_j, y_{j+h} c_j + y_j s_j,  h = rot / 2,
//   c_j, s_j = mscale * cos, sin(p inv_freq_j)
// and values pass through.  Everything is read once and written once, a few
// flops an element: bytes bound it, for one token the launch and a chain of
// dependent loads (row -> sequence -> length -> page).
//
// One CTA per row of the step.  A group of d / 16 threads takes one head row,
// each thread the two 8-element chunks that RoPE pairs, so the rotation needs
// no exchange and the norm three shuffles.  The row's angles are shared by
// all of its heads: they are formed once per CTA while the first head rows'
// loads are in flight.  An angle is reduced in f64 (p * turns, minus its
// nearest integer): in f32 a position of 10^5 would leave 2^-7 of a radian.
#include "../../include/dflash.h"
#include "kernels.cuh"
#include "ptx.cuh"
#include "step.cuh"

namespace dfl {
namespace {

constexpr int kAppendThreads = 256;
constexpr int kAppendDepth = 2;   // head rows a thread group has in flight

struct Chunk {
  float v[8];
};

__device__ __forceinline__ Chunk load8(const float* p) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  return {{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}
__device__ __forceinline__ Chunk load8(const __nv_bfloat16* p) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  Chunk c;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __bfloat1622float2(reinterpret_cast<const __nv_bfloat162&>(w[i]));
    c.v[2 * i] = f.x;
    c.v[2 * i + 1] = f.y;
  }
  return c;
}
__device__ __forceinline__ Chunk load8(const __half* p) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  Chunk c;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(reinterpret_cast<const __half2&>(w[i]));
    c.v[2 * i] = f.x;
    c.v[2 * i + 1] = f.y;
  }
  return c;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const Chunk& c) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(c.v[2 * i], c.v[2 * i + 1]);
    w[i] = reinterpret_cast<const uint32_t&>(b);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(__half* p, const Chunk& c) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 b = __floats2half2_rn(c.v[2 * i], c.v[2 * i + 1]);
    w[i] = reinterpret_cast<const uint32_t&>(b);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename In, typename Out, int D>
__global__ void __launch_bounds__(kAppendThreads) step_append_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int kLanes = D / 16;                     // threads of a head row
  constexpr int kGroups = kAppendThreads / kLanes;   // head rows of one sweep
  __shared__ float2 cs[D / 2];
  pdl_wait();
  pdl_launch_dependents();
  const StepView& s = a.s;
  const int row = blockIdx.x, tid = threadIdx.x;
  const int lane = tid % kLanes, group = tid / kLanes;
  const int Hq = a.n_heads, Hkv = a.c.n_kv_heads, heads = Hq + 2 * Hkv;
  // the two chunks of a head row this thread holds: a RoPE pair, or two of
  // the chunks behind the rotated ones
  const int pairs = a.rot / 16;
  const bool rot = lane < pairs;
  const int c0 = rot ? lane : 2 * pairs + (lane - pairs);
  const int c1 = rot ? lane + pairs : c0 + (kLanes - pairs);

  // rows behind the last sequence stay as they are
  int before = 0;
  for (int i = tid; i < s.n_seq; i += kAppendThreads) before += s.start(i + 1) <= row;
  int seq = __syncthreads_count(before > 0);
  if (s.n_seq > kAppendThreads) {   // more than one sequence a thread: sum the counts
    __shared__ int total;
    if (tid == 0) total = 0;
    __syncthreads();
    if (before) atomicAdd(&total, before);
    __syncthreads();
    seq = total;
  }
  if (seq >= s.n_seq) return;

  auto source = [&](int h) -> const In* {
    if (h < Hq) return static_cast<const In*>(a.q) + row * a.q_stride + (long)h * D;
    if (h < Hq + Hkv) return static_cast<const In*>(a.k) + row * a.k_stride + (long)(h - Hq) * D;
    return static_cast<const In*>(a.v) + row * a.v_stride + (long)(h - Hq - Hkv) * D;
  };
  Chunk x0[kAppendDepth], x1[kAppendDepth];
  auto fetch = [&](int h0) {
#pragma unroll
    for (int i = 0; i < kAppendDepth; ++i) {
      const int h = h0 + i * kGroups + group;
      if (h < heads) {
        const In* p = source(h);
        x0[i] = load8(p + 8 * c0);
        x1[i] = load8(p + 8 * c1);
      }
    }
  };
  fetch(0);

  const int own = s.len(seq) - s.start(seq + 1) + row;   // this row's own key index
  long dst = -1;                                          // its row in the cache
  if (own >= 0 && (own >> s.page_shift) < s.table_cols) {
    const int page = s.block_table[seq * s.table_stride + (own >> s.page_shift)];
    if (page >= 0 && page < s.n_pages)
      dst = page * a.c.page_stride + (long)(own & (s.page_size - 1)) * a.c.row_stride;
  }
  if (tid < a.rot / 2) {
    const long pos = a.positions ? (long)a.positions[row] : (long)s.prefix_len + own;
    const double t = (double)pos * a.turns[tid];
    float sn, cn;
    sincospif(2.f * (float)(t - rint(t)), &sn, &cn);
    cs[tid] = make_float2(cn * a.mscale, sn * a.mscale);
  }
  __syncthreads();

  for (int h0 = 0; h0 < heads; h0 += kAppendDepth * kGroups) {
    if (h0) fetch(h0);
#pragma unroll
    for (int i = 0; i < kAppendDepth; ++i) {
      const int h = h0 + i * kGroups + group;
      const bool is_q = h < Hq, is_v = h >= Hq + Hkv;
      const float* gain = is_q ? a.q_gain : (is_v ? nullptr : a.k_gain);
      Chunk y0 = x0[i], y1 = x1[i];
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) ss += y0.v[j] * y0.v[j] + y1.v[j] * y1.v[j];
#pragma unroll
      for (int o = kLanes / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (h >= heads) continue;
      if (gain) {
        const float r = rsqrtf(ss * (1.f / D) + a.eps);
        const Chunk g0 = load8(gain + 8 * c0), g1 = load8(gain + 8 * c1);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          y0.v[j] *= r * g0.v[j];
          y1.v[j] *= r * g1.v[j];
        }
      }
      if (rot && !is_v) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 w = cs[8 * lane + j];
          const float u = y0.v[j], t = y1.v[j];
          y0.v[j] = u * w.x - t * w.y;
          y1.v[j] = t * w.x + u * w.y;
        }
      }
      Out* o;
      if (is_q) {
        o = static_cast<Out*>(a.q_out) + row * a.q_out_stride + (long)h * D;
      } else {
        if (dst < 0) continue;
        o = is_v ? static_cast<Out*>(a.c.v) + dst + (h - Hq - Hkv) * a.c.head_stride
                 : static_cast<Out*>(a.c.k) + dst + (h - Hq) * a.c.head_stride;
      }
      store8(o + 8 * c0, y0);
      store8(o + 8 * c1, y1);
    }
  }
}

template <typename In, typename Out>
cudaError_t launch(const AppendArgs& a, cudaStream_t s) {
  auto* kernel = a.c.d == 128 ? step_append_kernel<In, Out, 128> : step_append_kernel<In, Out, 64>;
  return launch_pdl(kernel, dim3(a.s.n_rows), dim3(kAppendThreads), 0, s, a);
}

}  // namespace

cudaError_t launch_step_append(const AppendArgs& a, int in_dtype, int out_dtype, cudaStream_t s) {
  if (out_dtype == DFLASH_BF16)
    return in_dtype == DFLASH_F32 ? launch<float, __nv_bfloat16>(a, s) : launch<__nv_bfloat16, __nv_bfloat16>(a, s);
  return in_dtype == DFLASH_F32 ? launch<float, __half>(a, s) : launch<__half, __half>(a, s);
}

}  // namespace dfl

// step_rows.cuh -- a head row's elements on their way through the append
// kernels: loads that stay packed while in flight, f32 values, 16-byte stores,
// and which elements of a row a lane holds.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <type_traits>

namespace dfl {

struct Chunk {
  float v[8];
};

// Eight elements as loaded (16-bit ones stay packed while in flight).
template <typename T>
struct Raw {
  uint4 u;
  __device__ __forceinline__ void load(const T* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ Chunk get() const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    Chunk c;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 f;
      if constexpr (std::is_same_v<T, __nv_bfloat16>)
        f = __bfloat1622float2(reinterpret_cast<const __nv_bfloat162&>(w[i]));
      else
        f = __half22float2(reinterpret_cast<const __half2&>(w[i]));
      c.v[2 * i] = f.x;
      c.v[2 * i + 1] = f.y;
    }
    return c;
  }
};
template <>
struct Raw<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ Chunk get() const { return {{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}}; }
};
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

// RoPE of a lane's two 8-element chunks: elements j of both are a pair (halves),
// or elements 2j, 2j + 1 of each (interleaved).  w holds the (cos, sin) of the
// lane's 8 pairs: of the first chunk's elements, or four of each chunk.
template <bool INTER>
__device__ __forceinline__ void rotate(Chunk& y0, Chunk& y1, const float2* w) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float& a = INTER ? (j < 4 ? y0 : y1).v[2 * (j & 3)] : y0.v[j];
    float& b = INTER ? (j < 4 ? y0 : y1).v[2 * (j & 3) + 1] : y1.v[j];
    const float u = a, t = b;
    a = u * w[j].x - t * w[j].y;
    b = t * w[j].x + u * w[j].y;
  }
}
// A lane's 8 pairs out of a row's; c0 and c1: its chunks' first elements.
template <bool INTER, typename T>
__device__ __forceinline__ const T* pair_angles(const T* cs, int j, int c0, int c1) {
  return INTER ? cs + (j < 4 ? c0 / 2 : c1 / 2 - 4) + j : cs + c0 + j;
}

}  // namespace dfl

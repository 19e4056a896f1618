// step_attn.cuh -- what the attention kernels of a step share: tensor-memory
// access, packed arithmetic, descriptors and bounded waits.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ptx.cuh"
#include "step_plan.cuh"

namespace dfl {

constexpr int kAtomBytes = kKeys * 128;  // 128 rows x 128 bytes

// A packed cache's tiles in shared memory: codes and scales of 128 head rows.  A
// copy ends on a 128-byte boundary, and 16 rows' scales at d = 64 are 64 bytes: those
// of a page take 128.
constexpr int scale_bytes(int d) { return d == 128 ? kKeys * 8 : kKeys / 16 * 128; }
constexpr int code_tile(int d) { return kKeys * (d / 2) + scale_bytes(d); }
template <int D>
__device__ __forceinline__ int scale_place(int r, int box_rows) {
  return r * (D / 16) + (D == 64 && box_rows == 16 ? (r >> 4) * 64 : 0);
}
static_assert(code_tile(128) % 512 == 0 && code_tile(64) % 512 == 0, "swizzled tiles");

constexpr float kGrow = 8.f;             // O is rescaled when a row's max grows by more than 2^8
constexpr int kFrags = 2;                // fragments described ahead
constexpr int kBarPair = 3;              // named barrier of the 256 softmax threads

// ---------------------------------------------------------------- TMEM access
// 128 columns of a row are loaded at once and waited for once; the wait takes
// the registers as operands so that no use of them can move above it.
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
        "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
        "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_wait32(float* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]),
                 "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]),
                 "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]),
                 "+f"(v[30]), "+f"(v[31])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(taddr),
      "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]),
      "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// 32 aligned bytes at once: rows of a tile lie far apart, so a lane's store
// fills whole sectors by itself.
__device__ __forceinline__ void store_sector(float* p, const float* v) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
               "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float m;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
  return m;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)), "l"(reinterpret_cast<uint64_t&>(c)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return d;
}
// Two softmax weights (the lower key in the low half) or results in the
// cache's type: the product with V takes both operands in one 16-bit type.  The
// row sums add the unrounded weights, so the rounding (half a step, either way)
// does not add up in the quotient.  f16 rounds to zero, always downward, below
// 2^-25, and loses bits below 2^-14: its weights are taken times 2^7, the most
// that keeps them (2^8 and less, see kGrow) in its range, so that what is lost
// of a weight is at most 2^-32 of the row's maximum's.
template <bool BF16>
__device__ __forceinline__ float pack2(float2 p) {
  if constexpr (BF16) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(p.x, p.y);
    return __uint_as_float(reinterpret_cast<const uint32_t&>(b));
  } else {
    const __half2 b = __floats2half2_rn(p.x, p.y);
    return __uint_as_float(reinterpret_cast<const uint32_t&>(b));
  }
}

// log of a row's sum of exponentials from its maximum (in log2 units) and sum
__device__ __forceinline__ float log_sum(float m, float l) {
  return l == 0.f ? -INFINITY : 0.69314718055994531f * (m + log2f(l));
}

// Descriptor of an MN-major tile in the 128-byte swizzle: rows are K (keys)
// of 128 B (64 MN elements), 8-key atoms 1024 B apart along K, the next 64
// MN elements one tile of 128 keys further.
__device__ __forceinline__ uint64_t desc_sw128_mn(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(kAtomBytes >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

__device__ __forceinline__ void tma_load_4d(void* dst, const void* map, uint64_t* bar, int x, int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], "
      "[%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}

// One lane of a converged warp, the same in every call.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}

// Wait for the phase of `parity` of a pipeline barrier; false once `abort` is
// raised or kWaitNs have passed (the clock is read once in 64 tries).
__device__ __forceinline__ bool pipe_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  if (mbar_try_wait(bar, parity)) return true;
  uint64_t t0 = 0;
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63) == 0) {
      if (*abort) return false;
      const uint64_t t = globaltimer();
      if (t0 == 0) t0 = t;
      else if (t - t0 > kWaitNs) return false;
    }
  }
}

// Place of a K (kv = 0) or V (1) tile of a fragment's block among its 2 n
// tiles.  A single item's two streams each hold a V tile while its softmax
// runs, so the K tiles of both blocks go first: the next pair's keys land
// meanwhile.
__device__ __forceinline__ uint32_t tile_of(bool pair, int block, int n, int kv) {
  if (pair) return 2 * block + kv;
  const int first = block & ~1;
  return 2 * first + (block & 1) + kv * min(2, n - first);
}

// The inverse: block (and kv) of tile t of a fragment of n blocks.
__device__ __forceinline__ int block_of(bool pair, int t, int n, int& kv) {
  if (pair) {
    kv = t & 1;
    return t >> 1;
  }
  const int first = t >> 2 << 1, m = min(2, n - first), w = t & 3;
  kv = w >= m;
  return first + w - kv * m;
}

// Waits on the fragment ring outlast any one fragment; a failed wait
// elsewhere ends the others within kWaitNs, so this limit is not met.
__device__ __forceinline__ bool ring_wait(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = globaltimer();
  while (!mbar_try_wait(bar, parity))
    if (globaltimer() - t0 > 10 * kWaitNs) return false;
  return true;
}

// This CTA's pieces of n_cta CTAs' work, described in a ring (and then given to
// `each`); seg -1 ends them.  A warp's work.
template <class AnyWalk, class Each>
__device__ __forceinline__ void plan_pieces(AnyWalk& w, int n_cta, Frag* frag, uint64_t* ffull, uint64_t* fempty,
                                            uint32_t n_frags, int lane, Each&& each) {
  // The warp counts all units, 32 sequences at a time, then looks for the
  // sequence that holds this CTA's first.
  const StepAttnArgs& a = w.a;
  const int n = a.s.n_seq, prefix = w.prefix_units();
  auto units_of = [&](int i) { return i < n ? a.Hkv * w.head_units(i) : 0; };
  const int mine = units_of(lane);
  bool falls = lane < n && w.falls(lane);
  unsigned total = prefix + __reduce_add_sync(0xffffffffu, (unsigned)mine);
#pragma unroll 4
  for (int i = 32; i < n; i += 32) {
    total += __reduce_add_sync(0xffffffffu, (unsigned)units_of(i + lane));
    falls |= i + lane < n && w.falls(i + lane);
  }
  w.divide(__any_sync(0xffffffffu, falls) ? 0 : (int)total, n_cta, blockIdx.x);
  int seq0 = -1, base = 0;
  if (w.ua < w.ub && w.ua >= prefix) {
    base = prefix;
    for (int i = 0; i < n; i += 32) {
      const int u = i ? units_of(i + lane) : mine;
      int inc = u;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
      }
      const unsigned holds = __ballot_sync(0xffffffffu, w.ua < base + inc);
      if (holds) {
        const int l = __ffs(holds) - 1;
        seq0 = i + l;
        base += __shfl_sync(0xffffffffu, inc - u, l);
        break;
      }
      base += __shfl_sync(0xffffffffu, inc, 31);
    }
  }
  if (w.ua < w.ub) w.begin(seq0, base);
  else w.pos = w.ub;
  bool more = true;
  for (uint32_t i = 0; more; ++i) {
    Frag f;
    more = w.next(f);
    if (!more) f.seg = -1;
    if (!__all_sync(0xffffffffu, ring_wait(&fempty[i % n_frags], ((i / n_frags) & 1) ^ 1))) break;
    if (lane == 0) {
      frag[i % n_frags] = f;
      mbar_arrive(&ffull[i % n_frags]);
    }
    __syncwarp();
    if (more) each(f);
  }
}

}  // namespace dfl

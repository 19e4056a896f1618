// step_attn.cu -- attention of a step's rows over [shared prefix ; own keys]
// of a paged cache, on the 5th-generation tensor cores.
//
// For row t, head h of kv head g = h / G, with M its largest scaled score:
//   l = sum_j exp(s_j - M),  o = sum_j exp(s_j - M) v_j / l,  s_j = scale q.k_j
// over its keys, computed block by block (128 keys) with a running M and l.
//
// Items.  The G query heads of a kv head and consecutive tokens fill query
// tiles of 128 rows (floor(128 / G) tokens).  The prefix is attended by tiles
// that run over the rows of the whole batch, so its keys are read once per
// kv head and 256 rows instead of once per sequence; own keys by tiles of one
// sequence.  Item = (segment, sequence, kv head, two tiles).  Partial results
// (o, max, sum) of the segments and pieces are merged by a second kernel; an
// item that one CTA ran whole, without a prefix, is finished where it is.
//
// Balance.  One CTA per SM; the items' key blocks form one line of units that
// is cut into equal pieces (step_plan.cuh), so a single long sequence, many
// short ones and any mixture load the SMs alike, with lengths known only on
// the device.  A CTA continues at most one item begun by another (its first),
// which bounds the partials: one per row and segment plus one tile per CTA.
//
// A CTA runs two streams of 128 query rows each:
//   pair   (an item with rows for both tiles)  both streams take every key
//          block, so a K/V tile feeds 256 rows;
//   single (at most one tile of rows: decoding)  stream 0 takes the even
//          blocks and stream 1 the odd ones of the same rows, and their
//          results are merged in tensor memory.
// Either way one stream's products run under the other's softmax.  What bounds
// it: a pair's block takes 2830 cycles of which the tensor pipe works 2048 (the
// issue path between them; 32 sequences of 16 rows behind 16384 keys: 111 us, 1.28
// PFLOP/s with the merge); a single's 2700 are HBM's (one sequence, 131016 keys:
// 6.7 TB/s in the loop, 93 us in all).
//   warps 0..3, 4..7  softmax of stream 0 / 1, one thread per query row
//   warp 8            TMA: query tiles (ring of 2), K and V tiles (ring)
//   warp 10           the pieces of items this CTA runs, described in a ring
//   warp 11           waits for the tiles that the MMA warp's next products read
//   warp 9            tcgen05.mma: S = Q K^T into TMEM, O += P V with P (in the
//                     cache's type, over S) read from TMEM
// V tiles are used as they lie in the cache (rows are keys), as the MN-major
// operand of the second product.
#include <atomic>

#include "../../include/dflash.h"
#include "kernels.cuh"
#include "ptx.cuh"
#include "step_plan.cuh"

namespace dfl {
namespace {

constexpr int kStepThreads = 384;
// registers of a softmax / other thread: 2 x 208 + 88 = 3 x 168, the launch's own
constexpr int kSoftRegs = 208, kOtherRegs = 88;
constexpr int kSoftThreads = 256;        // warps 0..7
constexpr int kAtomBytes = kKeys * 128;  // 128 rows x 128 bytes
constexpr int kMaxStages = 11;
constexpr int kSharedBytes = 3 * 1024;   // control block
constexpr size_t step_smem(int d, int stages) { return (size_t)(2 + stages) * (d / 64) * kAtomBytes + kSharedBytes; }
// as many K and V tiles as shared memory holds beside two query tiles: 5 at d = 128, 11 at 64
constexpr int step_stages(int d) {
  int n = kMaxStages;
  while (step_smem(d, n) > 227 * 1024) --n;
  return n;
}
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

struct Shared {
  uint64_t kvfull[kMaxStages], kvempty[kMaxStages];
  uint64_t qfull[2], qempty[2], sfull[2], pfull[2][2], pvdone[2], kfirst[2];
  uint64_t drained;
  uint32_t tmem;
  int abort;
  // this CTA's fragments, in a ring
  uint64_t ffull[kFrags], fempty[kFrags];
  Frag frag[kFrags];
  float2 ml[2][128];   // merge of the two streams of a single item
  // first own key whose value element is not finite, per element
  int bad[128];
  int any_bad;
};
static_assert(sizeof(Shared) <= kSharedBytes, "control block of the attention kernel");

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

// Waits on the fragment ring outlast any one fragment; a failed wait
// elsewhere ends the others within kWaitNs, so this limit is not met.
__device__ __forceinline__ bool ring_wait(uint64_t* bar, uint32_t parity) {
  const uint64_t t0 = globaltimer();
  while (!mbar_try_wait(bar, parity))
    if (globaltimer() - t0 > 10 * kWaitNs) return false;
  return true;
}

// ---------------------------------------------------------------- the kernel
template <int D, bool BF16>
__global__ void __launch_bounds__(kStepThreads, 1)
    step_attn_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ StepAttnArgs a) {
  constexpr int kDAtoms = D / 64;
  constexpr int kTile = kDAtoms * kAtomBytes;          // a Q, K or V tile
  constexpr int kStages = step_stages(D);              // K and V tiles in flight
  constexpr uint32_t kFmt = BF16 ? (1u << 7) | (1u << 10) : 0u;
  constexpr uint32_t kIdescS = (1u << 4) | kFmt | ((128u >> 3) << 17) | ((128u >> 4) << 24);
  constexpr uint32_t kIdescO = (1u << 4) | kFmt | (1u << 16) | ((uint32_t)(D >> 3) << 17) | ((128u >> 4) << 24);
  constexpr float kBias = BF16 ? 0.f : 7.f;            // weights, their sums and products are 2^kBias times as large
  constexpr uint32_t kColO = 256;                      // TMEM: S / P of the streams at 0 and 128, O at 256 and 384
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sQ = smem;
  uint8_t* sKV = smem + 2 * kTile;
  Shared& sh = *reinterpret_cast<Shared*>(sKV + kStages * kTile);
  volatile int* abort = &sh.abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sh.kvfull[i], 1);
      mbar_init(&sh.kvempty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.qfull[i], 1);
      mbar_init(&sh.qempty[i], 1);
      mbar_init(&sh.sfull[i], 1);
      mbar_init(&sh.pfull[i][0], 129);   // and warp 11
      mbar_init(&sh.pfull[i][1], 128);
      mbar_init(&sh.pvdone[i], 1);
      mbar_init(&sh.kfirst[i], 1);
    }
    mbar_init(&sh.drained, 1);
    for (int i = 0; i < kFrags; ++i) {
      mbar_init(&sh.ffull[i], 1);
      mbar_init(&sh.fempty[i], 11);   // warps 8, 9 and 11 and eight softmax warps
    }
    sh.abort = 0;
    sh.any_bad = 0;
    fence_barrier_init();
    tma_prefetch_map(&tmQ);
    tma_prefetch_map(&tmK);
    tma_prefetch_map(&tmV);
  }
  if (tid < 128) sh.bad[tid] = INT_MAX;
  if (warp == 9) tmem_alloc(&sh.tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  pdl_wait();   // the step's arrays, queries and cache may come from the kernel before
  pdl_launch_dependents();

  // Every role takes every fragment, also after a failed wait (it then skips
  // the work), so the ring and the named barriers never starve.
  uint32_t nf = 0;
  auto take = [&](Frag& f) -> bool {
    const int i = nf % kFrags;
    if (!__all_sync(0xffffffffu, ring_wait(&sh.ffull[i], (nf / kFrags) & 1))) {
      sh.abort = 1;
      return false;
    }
    f = sh.frag[i];
    ++nf;
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.fempty[i]);
    return f.seg >= 0;
  };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == 8) {
      // ------------------------------------------------------------------ TMA
      bool ok = true;
      uint32_t nq = 0, nkv = 0;                       // query tiles and K/V tiles so far
      const uint32_t q_bytes = (uint32_t)(kDAtoms * a.tpt * a.G * 128);
      const uint32_t box_bytes = (uint32_t)a.box_rows * 128;
      const int box_shift = __ffs(a.box_rows) - 1;
      Frag f;
      while (take(f)) {
        if (!ok || f.b0 >= f.b1) continue;
        const int tiles = f.ntok > a.tpt ? 2 : 1;
        for (int i = 0; i < tiles && ok; ++i, ++nq) {
          const int slot = nq & 1;
          ok = __all_sync(0xffffffffu, pipe_wait(&sh.qempty[slot], ((nq >> 1) & 1) ^ 1, abort));
          if (!ok) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(&sh.qfull[slot], q_bytes);
            for (int at = 0; at < kDAtoms; ++at)
              tma_load_3d(sQ + slot * kTile + at * kAtomBytes, &tmQ, &sh.qfull[slot], at * 64, f.h * a.G,
                          f.tok0 + i * a.tpt);
          }
          __syncwarp();
        }
        // page ids: one lane per box of the next 32, the following 32 in flight
        const int* table = f.seg ? a.s.block_table + f.seq * a.s.table_stride : a.s.prefix_pages;
        const int n_box = (f.keys + a.box_rows - 1) >> box_shift;
        auto page_of = [&](int box) -> int {
          return box < n_box ? table[(int)(((long)box << box_shift) >> a.s.page_shift)] : 0;
        };
        const int first_box = f.b0 * a.boxes;
        int cur = page_of(first_box + lane), nxt = page_of(first_box + 32 + lane), win = first_box;
        const int step = tiles == 2 ? 1 : 2;           // blocks whose K tiles go before their V tiles
        for (int b = f.b0; b < f.b1 && ok; b += step) {
          if (b * a.boxes >= win + 32) {               // boxes of a step never straddle a window
            cur = nxt;
            win += 32;
            nxt = page_of(win + 32 + lane);
          }
          const int blocks = min(step, f.b1 - b);
          for (int i = 0; i < 2 * blocks && ok; ++i, ++nkv) {
            const int kv = i >= blocks, box0 = (b + i - kv * blocks) * a.boxes, n = min(a.boxes, n_box - box0);
            const int st = (int)(nkv % kStages);
            ok = __all_sync(0xffffffffu, pipe_wait(&sh.kvempty[st], ((nkv / kStages) & 1) ^ 1, abort));
            if (!ok) break;
            if (lane == 0) mbar_arrive_expect_tx(&sh.kvfull[st], (uint32_t)n * kDAtoms * box_bytes);
            __syncwarp();
            const int bi = lane / kDAtoms, at = lane % kDAtoms;
            const int page = __shfl_sync(0xffffffffu, cur, min(box0 - win + bi, 31));
            if (bi < n)
              tma_load_4d(sKV + st * kTile + at * kAtomBytes + bi * box_bytes, kv ? &tmV : &tmK, &sh.kvfull[st],
                          at * 64, f.h, (int)(((long)(box0 + bi) << box_shift) & (a.s.page_size - 1)), page);
            __syncwarp();
          }
        }
      }
      if (!ok) {   // leave no copy in flight behind
        sh.abort = 1;
        int none = 0;
        for (uint32_t i = nkv > (uint32_t)kStages ? nkv - kStages : 0; i < nkv; ++i)
          pipe_wait(&sh.kvfull[i % kStages], (i / kStages) & 1, &none);
        for (uint32_t i = nq > 2 ? nq - 2 : 0; i < nq; ++i) pipe_wait(&sh.qfull[i & 1], (i >> 1) & 1, &none);
      }
    } else if (warp == 9) {
      // ------------------------------------------------------------------ MMA
      // The warp runs converged and elects a lane only around the tensor
      // instructions: their descriptors then stay in uniform registers (issued
      // from one lane's branch, each cost about 110 cycles).  One warp issues
      // both streams' products in turn, which keeps the streams half a period
      // apart (with a warp each they fall into step, softmax against softmax
      // and product against product: 4140 cycles a pair block).
      bool ok = true;
      uint32_t nq = 0, nb = 0;                         // query tiles and key blocks before this fragment
      uint32_t np[2] = {0, 0};                         // P tiles used by each stream
      const uint64_t q_desc = desc_sw128(smem_u32(sQ)), k_desc = desc_sw128(smem_u32(sKV));
      const uint64_t v_desc = desc_sw128_mn(smem_u32(sKV));
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (ok) ok = __all_sync(0xffffffffu, pipe_wait(bar, parity, abort));
        return ok;
      };
      uint32_t nfirst[2] = {0, 0};                     // fragments each stream had a part in
      Frag f;
      while (take(f)) {
        const int n = f.b1 - f.b0;
        if (!ok || n <= 0) continue;
        const bool pair = f.ntok > a.tpt;
        const int cnt[2] = {pair ? n : (n + 1) / 2, pair ? n : n / 2};
        auto tile = [&](int s, int j, int kv) { return 2 * nb + tile_of(pair, pair ? j : 2 * j + s, n, kv); };
        const int slot0 = nq & 1;
        // S of a stream's block j (one elected lane)
        auto issue_s = [&](int s, int j) {
          const int st = tile(s, j, 0) % kStages, slot = pair ? slot0 ^ s : slot0;
          const uint64_t qd = q_desc + (uint64_t)(slot * (kTile >> 4)), kd = k_desc + (uint64_t)(st * (kTile >> 4));
#pragma unroll
          for (int kk = 0; kk < 4 * kDAtoms; ++kk) {
            const uint64_t at = (uint64_t)((kk >> 2) * (kAtomBytes >> 4) + (kk & 3) * 2);
            mma_bf16(tmem + 128u * s, qd + at, kd + at, kIdescS, kk > 0);
          }
          mma_commit(&sh.sfull[s]);
          if (!pair || s == 1) mma_commit(&sh.kvempty[st]);
          // the last product on a query tile frees its slot
          if (j + 1 == cnt[s] && (pair || s == ((n - 1) & 1))) mma_commit(&sh.qempty[slot]);
        };
        wait(&sh.qfull[slot0], (nq >> 1) & 1);
        if (pair) wait(&sh.qfull[slot0 ^ 1], ((nq + 1) >> 1) & 1);
#pragma unroll
        for (int s = 0; s < 2; ++s)
          if (cnt[s] && wait(&sh.kfirst[s], nfirst[s]++ & 1)) {
            if (elect_one()) issue_s(s, 0);
            __syncwarp();
          }
        for (int j = 0; j < cnt[0] && ok; ++j) {
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            if (j >= cnt[s]) continue;
            const uint32_t t = tile(s, j, 1), parity = np[s]++ & 1;
            const int st = t % kStages;
            const uint64_t vd = v_desc + (uint64_t)(st * (kTile >> 4));
            // P arrives in two halves of 64 keys; warp 11 holds the first one
            // back until this product's V and the next scores' K have landed
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              if (!wait(&sh.pfull[s][half], parity)) break;
              tc_fence_after();
              if (elect_one()) {
#pragma unroll
                for (int kk = 4 * half; kk < 4 * half + 4; ++kk)
                  mma_f16_ts(tmem + kColO + 128u * s, tmem + 128u * s + (uint32_t)(kk * 8),
                             vd + (uint64_t)(kk * (2048 >> 4)), kIdescO, (j > 0 || kk > 0) ? 1u : 0u);
                if (half == 1) {
                  mma_commit(&sh.pvdone[s]);
                  if (!pair || s == 1) mma_commit(&sh.kvempty[st]);
                  if (j + 1 < cnt[s]) issue_s(s, j + 1);
                }
              }
              __syncwarp();
            }
          }
        }
        nq += pair ? 2 : 1;
        nb += (uint32_t)n;
      }
      if (!ok) sh.abort = 1;
      // every product is done before tensor memory is freed
      if (elect_one()) mma_commit(&sh.drained);
      __syncwarp();
      int none = 0;
      pipe_wait(&sh.drained, 0, &none);
    } else if (warp == 11) {
      // ------------------------------------------------------------------ tiles landed
      // Waits for the tiles in the MMA warp's place: that warp's instructions
      // bound a pair's blocks, and a wait that is over already costs it 200
      // cycles.  It waits for every tile, none before the one that had its
      // slot before, so a barrier's parity is never read a turn early; and it
      // goes on to a stream's next block only when the last P is complete,
      // because its arrival would count for that one.
      bool ok = true;
      uint32_t nb = 0, np[2] = {0, 0};
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (ok) ok = __all_sync(0xffffffffu, pipe_wait(bar, parity, abort));
      };
      auto landed = [&](uint32_t tile) { wait(&sh.kvfull[tile % kStages], (tile / kStages) & 1); };
      Frag f;
      while (take(f)) {
        const int n = f.b1 - f.b0;
        if (!ok || n <= 0) continue;
        const bool pair = f.ntok > a.tpt;
        const int cnt[2] = {pair ? n : (n + 1) / 2, pair ? n : n / 2};
        auto tile = [&](int s, int j, int kv) { return 2 * nb + tile_of(pair, pair ? j : 2 * j + s, n, kv); };
        for (int j = -1; j < cnt[0] && ok; ++j) {   // -1: the first scores' K tiles
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            if (j >= cnt[s] || cnt[s] == 0) continue;
            if (!pair || s == 0) {                  // a pair shares its tiles
              if (j >= 0) landed(tile(s, j, 1));
              if (j + 1 < cnt[s]) landed(tile(s, j + 1, 0));
            }
            if (np[s] > 0) wait(&sh.pfull[s][0], (np[s] - 1) & 1);
            if (j >= 0) ++np[s];
            if (ok && lane == 0) mbar_arrive(j < 0 ? &sh.kfirst[s] : &sh.pfull[s][0]);
          }
        }
        nb += (uint32_t)n;
      }
      if (!ok) sh.abort = 1;
    } else if (warp == 10) {
      // ------------------------------------------------------------------ fragments
      // The warp counts all units, 32 sequences at a time, then looks for the
      // sequence that holds this CTA's first.
      Walk w(a);
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
      w.divide(__any_sync(0xffffffffu, falls) ? 0 : (int)total, a.n_cta, blockIdx.x);
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
        if (!__all_sync(0xffffffffu, ring_wait(&sh.fempty[i % kFrags], ((i / kFrags) & 1) ^ 1))) break;
        if (lane == 0) {
          sh.frag[i % kFrags] = f;
          mbar_arrive(&sh.ffull[i % kFrags]);
        }
        __syncwarp();
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));
    // ------------------------------------------------------------------ softmax
    const int st = warp >> 2;                        // stream
    const int r = tid & 127;                         // row of its tile
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t s_addr = tmem + lanes + 128u * st;
    const int tok = r / a.G, head = r - tok * a.G;
    bool ok = true;
    uint32_t np = 0, nb = 0;
    int4 split = make_int4(0, 0, 0, 0);              // the item that goes on in another CTA, if any
    auto both = [&]() { asm volatile("barrier.sync %0, %1;" ::"r"(kBarPair), "r"(kSoftThreads) : "memory"); };
    Frag f;
    while (take(f)) {
      const int n = f.b1 - f.b0;
      const bool pair = f.ntok > a.tpt;
      const int cnt = pair ? n : (n + 1 - st) / 2;
      const int t = (pair ? st * a.tpt : 0) + tok;   // token within the item
      const bool live = tok < a.tpt && t < f.ntok;
      const bool causal = f.seg == 1 && a.causal;
      // keys this row sees; rows without a token skip the mask
      const int lim = !live ? INT_MAX : min(causal ? max(f.lim0 + t, 0) : f.keys, f.keys);
      const bool any_live = __any_sync(0xffffffffu, live);
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < cnt; ++j, ++np) {
        const int bi = pair ? j : 2 * j + st;        // block of the fragment
        const int key0 = (f.b0 + bi) * kKeys;
        if (ok && !__all_sync(0xffffffffu, pipe_wait(&sh.sfull[st], np & 1, abort))) ok = false;
        tc_fence_after();
        // V rows behind the last key hold anything: zero them.  Own keys that
        // some row of the step must not see may hold anything too: their
        // elements that are not finite are taken out and remembered.
        const int own0 = causal && f.lim0 < f.keys ? max(f.lim0, 0) : INT_MAX;   // first key not seen by all rows
        if (ok && (st == 0 || !pair) && (key0 + kKeys > f.keys || key0 + kKeys > own0)) {
          // (a pair shares the tile and its streams' products come in turn, so
          // stream 0 does it for both; the slot's use before this one is over,
          // because the scores just read were issued behind its product)
          const uint32_t tile = 2 * nb + tile_of(pair, bi, n, 1), stage = tile % kStages;
          if (!__all_sync(0xffffffffu, pipe_wait(&sh.kvfull[stage], (tile / kStages) & 1, abort))) ok = false;
          uint8_t* v = sKV + stage * kTile + r * 128;
          const int key = key0 + r;
          if (key >= f.keys) {
#pragma unroll
            for (int c = 0; c < 8 * kDAtoms; ++c)
              *reinterpret_cast<uint4*>(v + (c >> 3) * kAtomBytes + ((c & 7) ^ (r & 7)) * 16) = make_uint4(0, 0, 0, 0);
          } else if (key >= own0) {
            // an exponent of ones carries into the sign's place
            constexpr uint32_t kExp = BF16 ? 0x7F807F80u : 0x7C007C00u, kOne = BF16 ? 0x00800080u : 0x04000400u;
            auto odd = [&](uint32_t x) { return ((x & kExp) + kOne) & 0x80008000u; };
#pragma unroll 4
            for (int c = 0; c < 8 * kDAtoms; ++c) {
              uint4* e = reinterpret_cast<uint4*>(v + (c >> 3) * kAtomBytes + (((c & 7) ^ (r & 7)) * 16));
              const uint4 x = *e;
              if (odd(x.x) | odd(x.y) | odd(x.z) | odd(x.w)) {
                uint32_t y[4] = {x.x, x.y, x.z, x.w};
                for (int i = 0; i < 8; ++i)
                  if (odd(y[i >> 1]) & (i & 1 ? 0x80000000u : 0x8000u)) atomicMin(&sh.bad[c * 8 + i], key);
                sh.any_bad = 1;
                for (int i = 0; i < 4; ++i)
                  y[i] &= (odd(y[i]) & 0x80000000u ? 0u : 0xFFFF0000u) | (odd(y[i]) & 0x8000u ? 0u : 0xFFFFu);
                *e = make_uint4(y[0], y[1], y[2], y[3]);
              }
            }
          }
          fence_proxy_async_smem();
        }
        if (ok && any_live) {
          float x[kKeys];
          const int seen = lim - key0;
          const bool whole = __all_sync(0xffffffffu, seen >= kKeys);
          auto scores = [&]() {
#pragma unroll
            for (int i = 0; i < kKeys; i += 32) tmem_ld32_async(s_addr + i, x + i);
#pragma unroll
            for (int i = 0; i < kKeys; i += 32) tmem_ld_wait32(x + i);
            if (!whole) {
#pragma unroll
              for (int i = 0; i < kKeys; ++i) x[i] = i < seen ? x[i] : -INFINITY;
            }
          };
          scores();
          float mx[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) mx[i] = fmaxf(x[i], x[i + 4]);
#pragma unroll
          for (int i = 8; i < kKeys; i += 8)
#pragma unroll
            for (int v = 0; v < 4; ++v) mx[v] = max3(mx[v], x[i + v], x[i + v + 4]);
          const float mj = a.scale_log2 * fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
          // the running maximum moves only when it grows by more than 2^8:
          // weights stay below 2^8 and the final division uses the same one
          const bool grow = mj > m + kGrow;
          if (j > 0 && __any_sync(0xffffffffu, grow)) {
            // O holds the products through this stream's block j - 1
            if (!__all_sync(0xffffffffu, pipe_wait(&sh.pvdone[st], (np - 1) & 1, abort))) ok = false;
            tc_fence_after();
            const float f0 = grow ? ex2_fast(m - mj) : 1.f;
            for (int c = 0; c < D; c += 32) {
              float o[32];
              const uint32_t oa = tmem + lanes + kColO + 128u * st + c;
              tmem_ld32_async(oa, o);
              tmem_ld_wait32(o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] *= f0;
              tmem_st32(oa, o);
            }
            l *= f0;
            scores();   // read again rather than kept beside O
          }
          if (grow) m = mj;
          const float nm = m == -INFINITY ? 0.f : kBias - m;
          const float2 neg = make_float2(nm, nm), sc = make_float2(a.scale_log2, a.scale_log2);
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int i = 0; i < kKeys; i += 32) {
            float pw[16];
#pragma unroll
            for (int v = 0; v < 16; ++v) {
              float2 p = fma2(make_float2(x[i + 2 * v], x[i + 2 * v + 1]), sc, neg);
              p.x = ex2_fast(p.x);
              p.y = ex2_fast(p.y);
              sum[v & 1] = add2(sum[v & 1], p);
              pw[v] = pack2<BF16>(p);
            }
            tmem_st16(s_addr + i / 2, pw);
            if (i % 64 == 32) {
              tmem_st_wait();
              tc_fence_before();
              mbar_arrive(&sh.pfull[st][i / 64]);
            }
          }
          const float2 tot = add2(sum[0], sum[1]);
          l += tot.x + tot.y;
        } else {
          tc_fence_before();
          mbar_arrive(&sh.pfull[st][0]);
          mbar_arrive(&sh.pfull[st][1]);
        }
      }
      nb += (uint32_t)n;
      // ---- the fragment's result
      if (ok && cnt > 0 && !__all_sync(0xffffffffu, pipe_wait(&sh.pvdone[st], (np - 1) & 1, abort))) ok = false;
      tc_fence_after();
      const long row = f.tok0 + t;                   // row of the step
      float* po;
      float2* pml;
      if (f.first) {
        const long at = row * a.Hq + f.h * a.G + head;
        po = a.seg_o[f.seg] + at * D;
        pml = a.seg_ml[f.seg] + at;
      } else {
        const long at = (long)blockIdx.x * 256 + (pair ? st * 128 : 0) + r;
        po = a.cta_o + at * D;
        pml = a.cta_ml + at;
      }
      m -= kBias;                                    // the maximum that the sum and O go with
      float m0 = m, l0 = l, w0 = 1.f, w1 = 0.f;      // this stream's part, or the merge of both
      if (!pair) sh.ml[st][r] = make_float2(m, l);
      if (!ok) sh.abort = 1;
      // a single item's streams read each other's products, which only their
      // own stream has waited for
      tc_fence_before();
      both();
      tc_fence_after();
      if (*abort) ok = false;
      if (!pair) {
        const float2 e0 = sh.ml[0][r], e1 = sh.ml[1][r];
        m0 = fmaxf(e0.x, e1.x);
        w0 = e0.x == -INFINITY ? 0.f : ex2_fast(e0.x - m0);
        w1 = e1.x == -INFINITY ? 0.f : ex2_fast(e1.x - m0);
        l0 = e0.y * w0 + e1.y * w1;
        // a row whose every score is NaN has no maximum but a NaN sum
        if (e0.x == -INFINITY && e0.y != 0.f) l0 = e0.y, w0 = 1.f;
        if (e1.x == -INFINITY && e1.y != 0.f) l0 = e1.y, w1 = 1.f;
      }
      // a row whose every key was here needs no merge: its result as it stands
      const bool whole = f.first && f.last_cta == (int)blockIdx.x && a.s.prefix_len == 0;
      const float inv = !ok ? __int_as_float(0x7fc00000) : (l0 == 0.f ? 0.f : 1.f / l0);
      const bool empty = pair ? cnt == 0 : n == 0;
      const bool poisoned = sh.any_bad;
      // a pair's streams write their own rows; of a single item each writes
      // half of the elements
      const int c_lo = pair ? 0 : st * (D / 2), c_hi = pair ? D : c_lo + D / 2;
      if (any_live) {
        for (int c = c_lo; c < c_hi; c += 32) {
          float o[32];
          if (empty || !ok) {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0.f;   // (times inv)
          } else {
            const uint32_t oa = tmem + lanes + kColO + c;
            tmem_ld32_async(oa + (pair ? 128u * st : 0u), o);
            tmem_ld_wait32(o);
            if (!pair) {
              float o1[32];
              tmem_ld32_async(oa + 128u, o1);
              tmem_ld_wait32(o1);
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                o[i] = w0 != 0.f ? o[i] * w0 : 0.f;
                o[i] = w1 != 0.f ? fmaf(o1[i], w1, o[i]) : o[i];
              }
            }
          }
          if (poisoned) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (sh.bad[c + i] < lim) o[i] = __int_as_float(0x7fc00000);
          }
          if (live && whole) {
            uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + row * a.out_stride +
                                                  (long)(f.h * a.G + head) * D + c);
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
              uint32_t y[4];
#pragma unroll
              for (int v = 0; v < 4; ++v)
                y[v] = __float_as_uint(pack2<BF16>(make_float2(o[i + 2 * v] * inv, o[i + 2 * v + 1] * inv)));
              dst[i / 8] = make_uint4(y[0], y[1], y[2], y[3]);
            }
          } else if (live) {
#pragma unroll
            for (int i = 0; i < 32; i += 8) store_sector(po + c + i, o + i);
          }
        }
      }
      if (live && (pair || st == 0)) {
        if (!whole) *pml = make_float2(m0, l0);
        else if (a.lse) a.lse[row * a.Hq + f.h * a.G + head] = ok ? log_sum(m0, l0) : inv;
        if (f.first && head == 0 && !a.by_cta)
          a.meta[((long)f.seg * a.s.n_rows + row) * a.Hkv + f.h] = make_int4(blockIdx.x, f.last_cta, t, whole);
      }
      if (tid == 0 && f.first && !whole) split = make_int4(f.tok0, f.ntok, f.h, f.last_cta);
      tc_fence_before();
      both();                                        // both streams have read O, and the notes on bad values
      if (poisoned) {
        if (tid < 128) sh.bad[tid] = INT_MAX;
        if (tid == 0) sh.any_bad = 0;
        both();
      }
      tc_fence_after();
    }
    if (tid == 0 && a.by_cta) a.split[blockIdx.x] = split;
    if (!ok) sh.abort = 1;
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (tid == 0) a.status[blockIdx.x] = sh.abort ? DERR_TIMEOUT : 0;
  if (warp == 9) {
    __syncwarp();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------- merge
// o = sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i over a row's fragments, one
// per segment and CTA that worked on it.  Few bytes, so latency bounds it: what
// does not depend on an earlier load is loaded at once, and a (row, head) has
// the four warps of a block where all of those run at once (19 short sequences
// behind 15769 keys of one kv head, 100 fragments a row: the call 16.9 us, 24.3
// with a warp; 128 rows x 32 heads 28.2 and 25.0), else a warp (64 rows x 32: the
// call 191.4 us, 192.7 with half a warp), and half a warp where there are more
// than run at once (32 verifying sequences, 512 rows x 32 of 5 fragments: 111.6 us,
// 114.0 with a warp; four prompts of 2000 rows 168.6 and 175.2).
constexpr int kMergeThreads = 128, kMergeWarps = kMergeThreads / 32;
constexpr int kSplitBlocks = 16;   // blocks for the rows of a CTA's last item

// A segment's fragments of one row: CTAs first .. first + n - 1, of which the
// first left its part in the row's own place and the others in tile row `trow`
// of theirs.
struct Parts {
  int first, n, trow;
  float2 ml;   // the first one's max and sum
};
// place of (token t of an item, head of its kv head) among a CTA's 256 tile
// rows: those of a pair's second tile lie behind the first's 128
__device__ __forceinline__ int tile_row(const StepAttnArgs& a, int t, int head) {
  return (t < a.tpt ? t * a.G : 128 + (t - a.tpt) * a.G) + head;
}

// LANES lanes merge a row (all groups of a warp come here, `live` or not), or
// WARPS > 1 warps a part of its fragments each.
template <int D, typename Out, int WARPS, int LANES>
__device__ __forceinline__ void merge_row(const StepAttnArgs& a, bool live, long row, int head, const Parts& pre,
                                          const Parts& own, int lane, int warp) {
  constexpr int kPer = D / LANES;                // elements of a lane
  constexpr int kAhead = LANES == 32 ? 4 : 2;    // partial rows in flight
  const long item = row * a.Hq + head;
  const int all = pre.n + own.n, share = (all + WARPS - 1) / WARPS;
  const int begin = warp * share, total = live ? min(begin + share, all) : 0;
  const int most = LANES == 32 ? total : __reduce_max_sync(0xffffffffu, total);
  float m = -INFINITY, l = 0.f, o[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) o[i] = 0.f;
  bool bad = false;
  for (int i0 = begin; i0 < most; i0 += LANES) {
    // lane i: fragment i's max, sum and partial row
    const int i = i0 + lane, seg = i >= pre.n, k = i - (seg ? pre.n : 0);
    float2 ml = make_float2(-INFINITY, 0.f);
    const float* src = nullptr;
    if (i < total) {
      const int cta = (seg ? own.first : pre.first) + k;
      const long at = (long)cta * 256 + (seg ? own.trow : pre.trow);
      ml = k == 0 ? (seg ? own.ml : pre.ml) : a.cta_ml[at];
      src = k == 0 ? (seg ? a.seg_o[1] : a.seg_o[0]) + item * D : a.cta_o + at * D;
      bad |= a.status[cta] != 0;
    }
    float mx = ml.x;
#pragma unroll
    for (int s = LANES / 2; s; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
    const float mn = fmaxf(m, mx);
    // a part without a maximum is left out (< 0), unless its sum is NaN; one
    // that weighs nothing is not: it can hold NaN
    const float wt = ml.x == -INFINITY ? (ml.y == 0.f ? -1.f : 1.f) : ex2_fast(ml.x - mn);
    float add = wt < 0.f ? 0.f : wt * ml.y;
#pragma unroll
    for (int s = LANES / 2; s; s >>= 1) add += __shfl_xor_sync(0xffffffffu, add, s);
    if (i0 > begin) {
      const float keep = m == -INFINITY ? (l == 0.f ? 0.f : 1.f) : ex2_fast(m - mn);
      l *= keep;
#pragma unroll
      for (int v = 0; v < kPer; ++v) o[v] *= keep;
    }
    m = mn;
    l += add;
    const int cnt = min(LANES, most - i0);
    for (int f0 = 0; f0 < cnt; f0 += kAhead) {
      float x[kAhead][kPer], g[kAhead];
#pragma unroll
      for (int f = 0; f < kAhead; ++f) {
        g[f] = -1.f;
        if (f0 + f >= cnt) continue;
        g[f] = __shfl_sync(0xffffffffu, wt, f0 + f, LANES);
        const float* p = reinterpret_cast<const float*>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), f0 + f, LANES)) + lane * kPer;
        if (LANES < 32 && g[f] < 0.f) continue;
        if constexpr (kPer >= 4) {
#pragma unroll
          for (int v = 0; v < kPer; v += 4) {
            const float4 q = *reinterpret_cast<const float4*>(p + v);
            x[f][v] = q.x, x[f][v + 1] = q.y, x[f][v + 2] = q.z, x[f][v + 3] = q.w;
          }
        } else {
          const float2 q = *reinterpret_cast<const float2*>(p);
          x[f][0] = q.x, x[f][1] = q.y;
        }
      }
#pragma unroll
      for (int f = 0; f < kAhead; ++f)
        if (!(g[f] < 0.f))
#pragma unroll
          for (int v = 0; v < kPer; ++v) o[v] = fmaf(x[f][v], g[f], o[v]);
    }
  }
  const unsigned any = __ballot_sync(0xffffffffu, bad);
  bad = LANES == 32 ? any != 0 : (any >> (threadIdx.x & 31 & ~(LANES - 1)) & ((1ull << LANES) - 1)) != 0;
  if (!live) return;
  if constexpr (WARPS > 1) {
    __shared__ float part[WARPS][D];
    __shared__ float3 mlb[WARPS];
#pragma unroll
    for (int v = 0; v < kPer; ++v) part[warp][lane * kPer + v] = o[v];
    if (lane == 0) mlb[warp] = make_float3(m, l, bad);
    __syncthreads();
    if (warp > 0) return;
    float mn = m;
#pragma unroll
    for (int w = 1; w < WARPS; ++w) mn = fmaxf(mn, mlb[w].x);
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const float3 p = mlb[w];
      const float wt = p.x == -INFINITY ? (p.y == 0.f ? 0.f : 1.f) : ex2_fast(p.x - mn);
      if (w == 0) {
        l *= wt;
#pragma unroll
        for (int v = 0; v < kPer; ++v) o[v] *= wt;
      } else {
        l = fmaf(p.y, wt, l);
#pragma unroll
        for (int v = 0; v < kPer; ++v) o[v] = fmaf(part[w][lane * kPer + v], wt, o[v]);
      }
      bad |= p.z != 0.f;
    }
    m = mn;
  }
  const float inv = bad ? __int_as_float(0x7fc00000) : (l == 0.f ? 0.f : 1.f / l);
  Out* dst = static_cast<Out*>(a.out) + row * a.out_stride + (long)head * D + lane * kPer;
  uint32_t y[kPer / 2];
#pragma unroll
  for (int v = 0; v < kPer; v += 2)
    y[v / 2] = __float_as_uint(pack2<std::is_same_v<Out, __nv_bfloat16>>(make_float2(o[v] * inv, o[v + 1] * inv)));
  if constexpr (kPer == 8) *reinterpret_cast<uint4*>(dst) = make_uint4(y[0], y[1], y[2], y[3]);
  else if constexpr (kPer == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(y[0], y[1]);
  else *reinterpret_cast<uint32_t*>(dst) = y[0];
  if (a.lse && lane == 0)
    a.lse[item] = bad ? inv : log_sum(m, l);
}

template <int D, typename Out, int WARPS, int LANES>
__global__ void __launch_bounds__(kMergeThreads, 8) step_merge_kernel(const __grid_constant__ StepAttnArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  constexpr int kRows = kMergeThreads / LANES;   // rows of a block at once
  const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES;
  const Parts none{0, 0, 0, {-INFINITY, 0.f}};
  if (LANES == 16 && a.by_cta) {
    // only rows of an item that goes on in another CTA: at most one a CTA
    const int cta = blockIdx.x / kSplitBlocks, part = blockIdx.x % kSplitBlocks;
    const int4 s = a.split[cta];   // its first row, tokens, kv head and last CTA
    const int n = s.y * a.G;
    for (int r0 = part * kRows; r0 < n; r0 += kSplitBlocks * kRows) {
      const bool live = r0 + group < n;
      const int r = live ? r0 + group : 0, t = r / a.G, sub = r - t * a.G, head = s.z * a.G + sub;
      const long row = s.x + t;
      const Parts own{cta, s.w - cta + 1, tile_row(a, t, sub), a.seg_ml[1][row * a.Hq + head]};
      merge_row<D, Out, 1, LANES>(a, live, row, head, none, own, lane, 0);
    }
    return;
  }
  const unsigned item = WARPS == 1 ? blockIdx.x * kRows + group : blockIdx.x;   // at most 2^31
  const unsigned row = item / (unsigned)a.Hq;
  bool live = row < (unsigned)a.s.n_rows;
  const int head = (int)(item - row * a.Hq), h = head / a.G;
  const int rows = a.s.start(a.s.n_seq);
  Parts p[2] = {none, none};
  bool whole = false;
#pragma unroll
  for (int seg = 0; seg < 2; ++seg)
    if (live && (seg == 1 || a.s.prefix_len > 0)) {
      const int4 meta = a.meta[((long)seg * a.s.n_rows + row) * a.Hkv + h];
      p[seg].ml = a.seg_ml[seg][item];
      p[seg].first = min(max(meta.x, 0), a.n_cta - 1);
      p[seg].n = min(max(meta.y, p[seg].first), a.n_cta - 1) - p[seg].first + 1;
      p[seg].trow = tile_row(a, min(max(meta.z, 0), 2 * a.tpt - 1), head - h * a.G);
      whole = meta.w != 0;
    }
  // written already, or behind the last sequence: left as it is
  if ((whole && a.s.prefix_len == 0) || row >= (unsigned)rows) live = false;
  if (!__any_sync(0xffffffffu, live)) return;
  merge_row<D, Out, WARPS, LANES>(a, live, row, head, p[0], p[1], lane, WARPS == 1 ? 0 : group);
}

template <int D, bool BF16>
cudaError_t launch(const StepAttnArgs& a, const CUtensorMap& q, const CUtensorMap& k, const CUtensorMap& v,
                   cudaStream_t s) {
  auto* attn = step_attn_kernel<D, BF16>;
  const size_t smem = step_smem(D, step_stages(D));
  // the kernel's shared memory is raised once on every device
  static std::atomic<uint64_t> raised{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(raised.load(std::memory_order_relaxed) >> dev & 1)) {
    e = cudaFuncSetAttribute(attn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    if (dev < 64) raised.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
  }
  e = launch_pdl(attn, dim3(a.n_cta), dim3(kStepThreads), smem, s, q, k, v, a);
  if (e != cudaSuccess) return e;
  // items of at most one block are whole: nothing to merge (48 single tokens 11.8 -> 10.5 us,
  // 56 short verifications 32.0 -> 23.7)
  if (a.s.prefix_len == 0 && a.s.room() <= kKeys) return cudaSuccess;
  // a block, a warp or half a warp for every (row, head), as many as run at
  // once; or sixteen blocks for every CTA's last item
  using Out = std::conditional_t<BF16, __nv_bfloat16, __half>;
  const long items = (long)a.s.n_rows * a.Hq, resident = 8L * a.n_cta;
  auto merge = [&](auto* kernel, long blocks) {
    return launch_pdl(kernel, dim3((unsigned)blocks), dim3(kMergeThreads), 0, s, a);
  };
  if (a.by_cta) return merge(step_merge_kernel<D, Out, 1, 16>, (long)a.n_cta * kSplitBlocks);
  if (items <= resident) return merge(step_merge_kernel<D, Out, kMergeWarps, 32>, items);
  if (items <= resident * kMergeWarps)
    return merge(step_merge_kernel<D, Out, 1, 32>, (items + kMergeWarps - 1) / kMergeWarps);
  return merge(step_merge_kernel<D, Out, 1, 16>, (items + 2 * kMergeWarps - 1) / (2 * kMergeWarps));
}

}  // namespace

cudaError_t launch_step_attention(const StepAttnArgs& a, const CUtensorMap& q, const CUtensorMap& k,
                                  const CUtensorMap& v, cudaStream_t s) {
  if (a.d == 128) return a.bf16 ? launch<128, true>(a, q, k, v, s) : launch<128, false>(a, q, k, v, s);
  return a.bf16 ? launch<64, true>(a, q, k, v, s) : launch<64, false>(a, q, k, v, s);
}

}  // namespace dfl

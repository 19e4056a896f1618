// verify.cu -- verification of drafted tokens against the target's
// probabilities (dflash_verify_tokens).
//
// Draft x_j is accepted while u_j q_j(x_j) < p_j(x_j).  Behind the accepted
// ones the next token comes from w = max(p_j - q_j, 0) (after a rejection) or
// w = p_n (after none), by inversion: the lowest index whose cumulative sum
// exceeds u * total.  So of the k + 1 rows of a sequence only the one behind
// the accepted drafts is read: 4 (V + V) bytes a sequence bound it, and for
// one sequence the latency of two gathers, one sweep and a search.
//
// One cluster of up to 8 CTAs per sequence.  The row is cut into runs, one per
// warp of the cluster; each warp sums its run, the sums are exchanged through
// distributed shared memory, every CTA finds the run where u * total falls,
// and the CTA that holds it searches it (its entries are in L1 / L2).  Small
// CTAs, four to an SM, hide one sequence's gathers and search behind another's
// sweep: 256 sequences x 262144 f32 in 91 us (5.9 TB/s) against 103 with CTAs of
// 512 threads, two to an SM.
//
// A cumulative sum is compared with a number, and a vocabulary has 10^5
// boundaries, so f32 sums (2^-24) would move one draw in a few hundred to a
// neighbouring token.  The f64 unit issues one warp instruction in 64 cycles
// here (a search in f64 took 9 us of a 16 us call), so every sum is kept in
// two floats: p - q and every addition are split into result and rounding
// error without loss, and the errors are summed beside: 2^-44 or better.
//
// The same sum taken in another order can differ in its last bits, so next to
// the threshold two levels of the search may disagree.  Each level therefore
// looks only among parts that have weight, and where none of them passes the
// threshold the last entry with weight stands.
#include <cooperative_groups.h>

#include <type_traits>

#include "../../include/dflash.h"
#include "kernels.cuh"
#include "ptx.cuh"
#include "step.cuh"

namespace dfl {
namespace {

namespace cg = cooperative_groups;

constexpr int kVerifyThreads = 256;   // four CTAs to an SM
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kMaxCluster = 8;        // the portable limit
constexpr int kMaxRuns = kMaxCluster * kVerifyWarps;

__device__ __forceinline__ float as_f32(float x) { return x; }
__device__ __forceinline__ float as_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float as_f32(__half x) { return __half2float(x); }

// NaN, infinite and negative probabilities count as zero: the positive finite
// floats are the bit patterns 1 .. 0x7f7fffff.
__device__ __forceinline__ float weight(float x) {
  return __float_as_uint(x) - 1u < 0x7f7fffffu ? x : 0.f;
}

// a + b = s + e exactly
__device__ __forceinline__ void two_sum(float a, float b, float& s, float& e) {
  s = __fadd_rn(a, b);
  const float t = __fsub_rn(s, a);
  e = __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t));
}

// A sum in two floats, |lo| at most half a step of hi once normal.
struct Sum {
  float hi = 0.f, lo = 0.f;
  // + x + err, errors gathered in lo
  __device__ __forceinline__ void add(float x, float err) {
    float s, e;
    two_sum(hi, x, s, e);
    hi = s;
    lo += e + err;
  }
  __device__ __forceinline__ Sum normal() const {
    Sum r;
    r.hi = __fadd_rn(hi, lo);
    r.lo = __fsub_rn(lo, __fsub_rn(r.hi, hi));
    return r;
  }
  __device__ __forceinline__ Sum operator+(const Sum& b) const {
    Sum r = *this;
    r.add(b.hi, b.lo);
    return r.normal();
  }
  __device__ __forceinline__ bool operator>(const Sum& b) const { return hi > b.hi || (hi == b.hi && lo > b.lo); }
  __device__ __forceinline__ Sum operator*(float u) const {
    Sum r;
    r.hi = __fmul_rn(hi, u);
    r.lo = fmaf(lo, u, fmaf(hi, u, -r.hi));
    return r.normal();
  }
};
__device__ __forceinline__ Sum shfl_xor(const Sum& s, int o) {
  Sum r;
  r.hi = __shfl_xor_sync(0xffffffffu, s.hi, o);
  r.lo = __shfl_xor_sync(0xffffffffu, s.lo, o);
  return r;
}
__device__ __forceinline__ Sum shfl(const Sum& s, int lane) {
  Sum r;
  r.hi = __shfl_sync(0xffffffffu, s.hi, lane);
  r.lo = __shfl_sync(0xffffffffu, s.lo, lane);
  return r;
}
// Sum over this and the lower lanes (inclusive); `before`: over the lower ones.
__device__ __forceinline__ Sum scan(Sum s, int lane, Sum& before) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    Sum x;
    x.hi = __shfl_up_sync(0xffffffffu, s.hi, o);
    x.lo = __shfl_up_sync(0xffffffffu, s.lo, o);
    if (lane >= o) s = x + s;
  }
  before.hi = __shfl_up_sync(0xffffffffu, s.hi, 1);
  before.lo = __shfl_up_sync(0xffffffffu, s.lo, 1);
  if (lane == 0) before = Sum{};
  return s;
}

// The weights of the row that the token is drawn from: p, or max(p - q, 0).
template <typename T>
struct Row {
  const T* p;
  const T* q;     // subtracted, or null
  int skip;       // index without weight (a rejected greedy draft), or -1
};
__device__ __forceinline__ void add_weight(Sum& s, bool diff, float p, float q) {
  p = weight(p);
  if (!diff) {
    s.add(p, 0.f);
    return;
  }
  float d, e;
  two_sum(p, -weight(q), d, e);
  s.add(fmaxf(d, 0.f), d > 0.f ? e : 0.f);
}

// Two sums side by side (an instruction adds both).
struct Sum2 {
  float2 hi = {0.f, 0.f}, lo = {0.f, 0.f};
};
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return d;
}
__device__ __forceinline__ float2 sub2(float2 a, float2 b) {
  float2 d;
  asm("sub.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t&>(d))
      : "l"(reinterpret_cast<uint64_t&>(a)), "l"(reinterpret_cast<uint64_t&>(b)));
  return d;
}
// s + max(p - q, 0) of two entries, exact but for lo's roundings.  Negative
// and NaN entries count as zero by the maxima; an infinite one leaves the sum
// infinite or NaN, and the run is then summed entry by entry.
template <bool DIFF>
__device__ __forceinline__ void add_pair(Sum2& s, float2 p, float2 q) {
  float2 x, e;
  if constexpr (DIFF) {
    q = make_float2(fmaxf(q.x, 0.f), fmaxf(q.y, 0.f));
    p = make_float2(fmaxf(p.x, q.x), fmaxf(p.y, q.y));
    x = sub2(p, q);
    const float2 t = sub2(x, p);                       // -(the part of q taken)
    e = sub2(sub2(p, sub2(x, t)), add2(q, t));
  } else {
    x = make_float2(fmaxf(p.x, 0.f), fmaxf(p.y, 0.f));
  }
  const float2 h = add2(s.hi, x), t = sub2(h, s.hi);
  float2 err = add2(sub2(s.hi, sub2(h, t)), sub2(x, t));
  if constexpr (DIFF) err = add2(err, e);
  s.hi = h;
  s.lo = add2(s.lo, err);
}

// 16 bytes of a row as pairs of floats.
template <typename T>
struct Pack {
  static constexpr int kEntries = 16 / sizeof(T);
  uint4 u;
  __device__ __forceinline__ void load(const T* p) { u = *reinterpret_cast<const uint4*>(p); }
  // entry i, if it is one of these, becomes 0
  __device__ __forceinline__ void clear(int i) {
    if (i < 0 || i >= kEntries) return;
    const uint32_t keep = sizeof(T) == 4 ? 0u : (i & 1 ? 0x0000ffffu : 0xffff0000u);
    const int w = sizeof(T) == 4 ? i : i / 2;
    if (w == 0) u.x &= keep;
    else if (w == 1) u.y &= keep;
    else if (w == 2) u.z &= keep;
    else u.w &= keep;
  }
  __device__ __forceinline__ float2 pair(int i) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    if constexpr (sizeof(T) == 4) return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    else if constexpr (std::is_same_v<T, __nv_bfloat16>)
      return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    else return __half22float2(reinterpret_cast<const __half2&>(w[i]));
  }
};

// The 16 bytes that start `shift` bytes into lo (a multiple of the type's size).
template <typename T>
__device__ __forceinline__ uint4 shifted(const uint4& lo, const uint4& hi, int shift) {
  uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
  for (int i = 0; i < 6; ++i) w[i] = shift & 8 ? w[i + 2] : w[i];
#pragma unroll
  for (int i = 0; i < 5; ++i) w[i] = shift & 4 ? w[i + 1] : w[i];
  if (sizeof(T) == 2 && (shift & 2))
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Adds entries i, i + 1, ... in steps of 32 lanes x DEPTH x 16 bytes while they
// end at or before b; p + i is aligned, and q + i `shift` bytes behind a
// 16-byte boundary (entries next to the step, inside the run, are read too).
template <typename T, bool DIFF, bool SHIFT, int DEPTH>
__device__ __forceinline__ void add_steps(Sum2 (&s)[2], const Row<T>& r, int& i, int b, int lane, int shift) {
  constexpr int kVec = Pack<T>::kEntries, kStep = 32 * kVec * DEPTH;
  for (; i + kStep + (SHIFT ? kVec : 0) <= b; i += kStep) {
    Pack<T> p[DEPTH], q[DEPTH];
    uint4 next[DEPTH];
#pragma unroll
    for (int u = 0; u < DEPTH; ++u) {
      const int at = i + (u * 32 + lane) * kVec;
      p[u].load(r.p + at);
      if (DIFF) {
        const uint4* src = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(r.q + at) - shift);
        q[u].u = src[0];
        if (SHIFT) next[u] = src[1];
      }
    }
    if (!DIFF && r.skip >= i && r.skip < i + kStep)
#pragma unroll
      for (int u = 0; u < DEPTH; ++u) p[u].clear(r.skip - (i + (u * 32 + lane) * kVec));
#pragma unroll
    for (int u = 0; u < DEPTH; ++u) {
      if (DIFF && SHIFT) q[u].u = shifted<T>(q[u].u, next[u], shift);
#pragma unroll
      for (int v = 0; v < kVec / 2; ++v)
        add_pair<DIFF>(s[v & 1], p[u].pair(v), DIFF ? q[u].pair(v) : make_float2(0.f, 0.f));
    }
  }
}

// Sum of entries [a, b) over the warp's lanes (every lane gets lane 0's: a sum's
// last bits depend on the order of its terms, and the CTAs have to agree).
template <typename T, bool DIFF>
__device__ __forceinline__ Sum run_total(const Row<T>& r, int a, int b, int lane) {
  constexpr int kVec = Pack<T>::kEntries, kScalar = 4;
  Sum2 s[2];
  const T zero = T(0.f);
  auto add_entries = [&](int i, int end) {   // one by one
    for (; i < end; i += 32 * kScalar) {
      T p[kScalar], q[kScalar];
#pragma unroll
      for (int u = 0; u < kScalar; ++u) {
        const int at = i + u * 32 + lane;
        p[u] = at < end && at != r.skip ? r.p[at] : zero;
        q[u] = DIFF && at < end ? r.q[at] : zero;
      }
#pragma unroll
      for (int u = 0; u < kScalar; u += 2)
        add_pair<DIFF>(s[u / 2 & 1], make_float2(as_f32(p[u]), as_f32(p[u + 1])),
                       make_float2(as_f32(q[u]), as_f32(q[u + 1])));
    }
  };
  // from the first aligned entry of p; rows of p and q are seldom aligned
  // alike, so q's are put together from two aligned loads
  int i = a + (int)((16 - (reinterpret_cast<uintptr_t>(r.p + a) & 15)) & 15) / (int)sizeof(T);
  const int shift = DIFF ? (int)(reinterpret_cast<uintptr_t>(r.q + i) & 15) : 0;
  if (i - shift / (int)sizeof(T) < a) i += kVec;
  i = min(i, b);
  add_entries(a, i);
  if (DIFF && shift) {
    add_steps<T, DIFF, DIFF, 2>(s, r, i, b, lane, shift);
  } else {
    add_steps<T, DIFF, false, 4>(s, r, i, b, lane, 0);
    add_steps<T, DIFF, false, 1>(s, r, i, b, lane, 0);
  }
  add_entries(i, b);
  Sum t[4];
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    t[v].hi = v & 1 ? s[v / 2].hi.y : s[v / 2].hi.x;
    t[v].lo = v & 1 ? s[v / 2].lo.y : s[v / 2].lo.x;
    t[v] = t[v].normal();
  }
  Sum c = (t[0] + t[1]) + (t[2] + t[3]);
  if (__any_sync(0xffffffffu, !(c.hi < INFINITY))) {
    c = Sum{};
    for (int k = a + lane; k < b; k += 32)
      if (k != r.skip) add_weight(c, DIFF, as_f32(r.p[k]), DIFF ? as_f32(r.q[k]) : 0.f);
    c = c.normal();
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) c = c + shfl_xor(c, o);
  return shfl(c, 0);
}

template <typename T>
__global__ void __launch_bounds__(kVerifyThreads, 4) verify_kernel(const __grid_constant__ VerifyArgs a) {
  __shared__ Sum run_sum[kMaxRuns];       // every run's sum, written by the whole cluster
  __shared__ Sum warp_sum[kVerifyWarps];
  __shared__ Sum sh_base, sh_th;
  __shared__ int sh_acc, sh_run, sh_token;
  cg::cluster_group cl = cg::this_cluster();
  const int rank = (int)cl.block_rank(), ctas = (int)cl.num_blocks(), seq = blockIdx.x / ctas;
  const int runs = ctas * kVerifyWarps;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_launch_dependents();
  const int nd = a.n_draft ? min(max(a.n_draft[seq], 0), a.k) : a.k;
  const int* draft = a.draft + seq * a.draft_stride;
  const T* P = static_cast<const T*>(a.p) + seq * a.p_seq;
  const T* Q = a.q ? static_cast<const T*>(a.q) + seq * a.q_seq : nullptr;
  const float u0 = a.u_token[seq];

  if (warp == 0) {   // accepted drafts, the same in every CTA of the cluster
    int acc = 0;
    for (int j0 = 0; j0 < nd; j0 += 32) {
      const int j = j0 + lane;
      bool take = false;
      if (j < nd) {
        const int x = draft[j];
        float u = a.u_accept[seq * a.u_stride + j];
        if (x >= 0 && x < a.vocab) {
          float p = weight(as_f32(P[j * a.p_row + x]));
          const float q = Q ? weight(as_f32(Q[j * a.q_row + x])) : 1.f;
          // u q < p, the product with its rounding error; next to a tiny p
          // both sides times 2^64, where that error still is a float
          if (p < 0x1p-60f) {
            p *= 0x1p64f;
            u *= 0x1p64f;
          }
          const float h = __fmul_rn(u, q);
          take = h < p || (h == p && fmaf(u, q, -h) < 0.f);
        }
      }
      const unsigned refused = ~__ballot_sync(0xffffffffu, take);
      acc += refused ? __ffs(refused) - 1 : 32;
      if (refused) break;
    }
    if (lane == 0) sh_acc = min(acc, nd);
  }
  __syncthreads();
  const int acc = sh_acc;
  const float u = u0 > 0.f ? fminf(u0, 1.f) : 0.f;
  const int V = a.vocab;
  // runs start on multiples of 16 entries
  const int len = ((V + runs - 1) / runs + 15) & ~15;
  Row<T> r{P + acc * a.p_row, nullptr, -1};
  if (acc < nd) {
    if (Q) r.q = Q + acc * a.q_row;
    else r.skip = draft[acc];
  }
  for (bool retry = true;; retry = false) {
    const int my = rank * kVerifyWarps + warp;
    const int lo = min(my * len, V), hi = min((my + 1) * len, V);
    const Sum t = r.q ? run_total<T, true>(r, lo, hi, lane) : run_total<T, false>(r, lo, hi, lane);
    cl.sync();   // every CTA runs, and has read the sums of a first try
    if (lane < ctas) *cl.map_shared_rank(&run_sum[my], lane) = t;
    cl.sync();
    if (warp == 0) {   // where u * total falls among the runs: a few neighbours per lane
      constexpr int kPer = kMaxRuns / 32;
      Sum v[kPer], c;
      int last = -1;       // last run with weight
      unsigned some = 0;   // which of the lane's runs have any
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int k = lane * kPer + i;
        if (k < runs) {
          c = c + run_sum[k];
          if (run_sum[k].hi > 0.f) {
            last = k;
            some |= 1u << i;
          }
        }
        v[i] = c;
      }
      Sum before;
      const Sum inc = scan(c, lane, before);
      const Sum th = shfl(inc, 31) * u;
      int run = kMaxRuns;   // first run past th
      Sum base;
#pragma unroll
      for (int i = kPer - 1; i >= 0; --i)
        if (some >> i & 1 && before + v[i] > th) {
          run = lane * kPer + i;
          base = i ? before + v[i - 1] : before;
        }
      const unsigned hit = __ballot_sync(0xffffffffu, run < kMaxRuns);
      const int src = hit ? __ffs(hit) - 1 : 0;
      run = __shfl_sync(0xffffffffu, run, src);
      base = shfl(base, src);
      // u * total at or past the total: the last run that has weight
      last = __reduce_max_sync(0xffffffffu, last);
      if (lane == 0) {
        sh_run = hit ? run : last;
        sh_base = base;
        sh_th = th;
        if (!hit) sh_th.hi = INFINITY;
        sh_token = -1;
      }
    }
    __syncthreads();
    // nothing left of p - q: draw from p
    if (sh_run >= 0 || !retry || (!r.q && r.skip < 0)) break;
    r.q = nullptr;
    r.skip = -1;
  }
  const int run = sh_run;
  int* out = a.tokens + (long)seq * (a.k + 1);
  if (rank == 0) {   // accepted drafts and the padding
    for (int j = tid; j <= a.k; j += kVerifyThreads)
      if (j != acc) out[j] = j < acc ? draft[j] : -1;
    if (tid == 0) {
      a.n_accepted[seq] = acc;
      if (run < 0) out[acc] = 0;
    }
  }
  if (run < 0 || run / kVerifyWarps != rank) return;
  // The entry of the run: each thread takes a few neighbours; the warp, the
  // lane and the entry where the sum passes th follow from the warps' and the
  // lanes' sums.  `fallback` is the last entry with weight so far: the answer
  // at u = 1, or if the sums here round below the run's own.
  constexpr int kPer = 4;
  const Sum th = sh_th;
  Sum base = sh_base;
  const int end = min((run + 1) * len, V);
  int fallback = 0;
  for (int i0 = run * len; i0 < end; i0 += kVerifyThreads * kPer) {
    const int i = i0 + tid * kPer;
    Sum w[kPer], c;
    int last = -1;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (i + j < end && i + j != r.skip) {
        Sum x;
        add_weight(x, r.q != nullptr, as_f32(r.p[i + j]), r.q ? as_f32(r.q[i + j]) : 0.f);
        if (x.hi > 0.f) {
          last = i + j;
          c = c + x;
        }
      }
      w[j] = c;
    }
    Sum before;
    const Sum inc = scan(c, lane, before);
    last = __reduce_max_sync(0xffffffffu, last);
    if (lane == 31) warp_sum[warp] = inc;
    if (lane == 0 && last >= 0) atomicMax(&sh_token, last);
    __syncthreads();
    fallback = max(fallback, sh_token);
    Sum wb;
    const Sum wsum = lane < kVerifyWarps ? warp_sum[lane] : Sum{};
    const Sum winc = scan(wsum, lane, wb);
    const unsigned past = __ballot_sync(0xffffffffu, wsum.hi > 0.f && base + winc > th);
    if (past) {   // the same in every warp
      if (warp != __ffs(past) - 1) return;
      const Sum mine = base + shfl(wb, warp);
      int first = INT_MAX;
#pragma unroll
      for (int j = kPer - 1; j >= 0; --j)
        if (mine + (before + w[j]) > th && w[j] > (j ? w[j - 1] : Sum{})) first = i + j;
      first = __reduce_min_sync(0xffffffffu, first);
      if (lane == 0) out[acc] = first != INT_MAX ? first : last;
      return;
    }
    base = base + shfl(winc, 31);
    __syncthreads();
  }
  if (tid == 0) out[acc] = fallback;
}

template <typename T>
cudaError_t launch(const VerifyArgs& a, int n_sm, cudaStream_t s) {
  // CTAs of a sequence: enough for 40960 entries each (f32: 256 x 262144 91 us
  // with 8 CTAs, 94 with 4; 256 x 160736 52.9 with 8, 46.3 with 4), for 16384
  // while not all the SMs' places are taken (172 x 59277: 4 22.0, 8 26.3, 2 24.6;
  // 256 x 32000: 2 12.9, 4 16.2), and more while half of them are free (100 x
  // 32000: 4 9.1, 2 10.0; one greedy 32768: 8 5.8, 2 7.8).
  unsigned ctas = 1;
  while (ctas < kMaxCluster &&
         (a.vocab > 40960 * (int)ctas || ((long)a.n_seq * ctas < 4L * n_sm && a.vocab > 16384 * (int)ctas) ||
          ((long)a.n_seq * ctas <= 2L * n_sm && a.vocab > 2048 * (int)ctas)))
    ctas *= 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(a.n_seq * ctas);
  cfg.blockDim = dim3(kVerifyThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {ctas, 1, 1};
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, verify_kernel<T>, a);
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& a, int dtype, int n_sm, cudaStream_t s) {
  if (dtype == DFLASH_F32) return launch<float>(a, n_sm, s);
  if (dtype == DFLASH_BF16) return launch<__nv_bfloat16>(a, n_sm, s);
  return launch<__half>(a, n_sm, s);
}

}  // namespace dfl

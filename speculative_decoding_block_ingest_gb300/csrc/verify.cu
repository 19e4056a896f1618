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
// One cluster of 8 CTAs per sequence.  The row is cut into 128 runs, one per
// warp of the cluster; each warp sums its run, the sums are exchanged through
// distributed shared memory, every CTA scans all 128, and the CTA that holds
// the run where u * total falls searches it (its entries are in L1 / L2).
//
// A cumulative sum is compared with a number, and a vocabulary has 10^5
// boundaries, so f32 sums (2^-24) would move one draw in a few hundred to a
// neighbouring token.  f64 adds run at 1/64 of the f32 rate here, so the
// sweep keeps each sum in two floats: p - q and every addition are split into
// result and rounding error without loss, the errors are summed beside, and
// only the lanes' totals and the search work in f64.
#include <cooperative_groups.h>

#include "../../include/dflash.h"
#include "kernels.cuh"
#include "ptx.cuh"
#include "step.cuh"

namespace dfl {
namespace {

namespace cg = cooperative_groups;

constexpr int kVerifyCtas = 8;      // CTAs of a cluster (the portable limit)
constexpr int kVerifyThreads = 512;
constexpr int kVerifyWarps = kVerifyThreads / 32;
constexpr int kRuns = kVerifyCtas * kVerifyWarps;

__device__ __forceinline__ float as_f32(float x) { return x; }
__device__ __forceinline__ float as_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float as_f32(__half x) { return __half2float(x); }

// NaN, infinite and negative probabilities count as zero.
__device__ __forceinline__ float weight(float x) { return x > 0.f && x < INFINITY ? x : 0.f; }

// a + b = s + e exactly
__device__ __forceinline__ void two_sum(float a, float b, float& s, float& e) {
  s = __fadd_rn(a, b);
  const float t = __fsub_rn(s, a);
  e = __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t));
}

struct Sum {
  float hi = 0.f, lo = 0.f;
  __device__ __forceinline__ void add(float x, float err) {
    float s, e;
    two_sum(hi, x, s, e);
    hi = s;
    lo += e + err;
  }
  // max(p - q, 0)
  __device__ __forceinline__ void add_diff(float p, float q) {
    p = weight(p);
    q = weight(q);
    if (p > q) {
      float d, e;
      two_sum(p, -q, d, e);
      add(d, e);
    }
  }
};

// The weights of the row that the token is drawn from.
template <typename T>
struct Row {
  const T* p;
  const T* q;     // subtracted, or null
  int skip;       // index without weight (a rejected greedy draft), or -1
  __device__ __forceinline__ double at(int i) const {
    if (i == skip) return 0.0;
    const double x = weight(as_f32(p[i]));
    return q ? fmax(x - (double)weight(as_f32(q[i])), 0.0) : x;
  }
};

// Sum of entries [a, b) over the warp's lanes (every lane gets it).
template <typename T>
__device__ double warp_sum(const Row<T>& r, int a, int b, int lane) {
  constexpr int kVec = 16 / sizeof(T), kDepth = 4;
  Sum s[2];
  auto take = [&](Sum& t, int i, T p, T q) { t.add_diff(i == r.skip ? 0.f : as_f32(p), r.q ? as_f32(q) : 0.f); };
  const T zero = T(0.f);
  const bool vec = ((reinterpret_cast<uintptr_t>(r.p + a) | (r.q ? reinterpret_cast<uintptr_t>(r.q + a) : 0)) & 15) == 0;
  int i = a;
  if (vec) {
    struct alignas(16) Pack {
      T v[kVec];
    };
    for (; i + 32 * kVec * kDepth <= b; i += 32 * kVec * kDepth) {
      Pack p[kDepth], q[kDepth];
#pragma unroll
      for (int u = 0; u < kDepth; ++u) {
        const int at = i + (u * 32 + lane) * kVec;
        p[u] = *reinterpret_cast<const Pack*>(r.p + at);
        if (r.q) q[u] = *reinterpret_cast<const Pack*>(r.q + at);
      }
#pragma unroll
      for (int u = 0; u < kDepth; ++u)
#pragma unroll
        for (int v = 0; v < kVec; ++v)
          take(s[v & 1], i + (u * 32 + lane) * kVec + v, p[u].v[v], r.q ? q[u].v[v] : zero);
    }
  }
  constexpr int kScalar = 8;
  for (; i < b; i += 32 * kScalar) {
    T p[kScalar], q[kScalar];
#pragma unroll
    for (int u = 0; u < kScalar; ++u) {
      const int at = i + u * 32 + lane;
      p[u] = at < b ? r.p[at] : zero;
      q[u] = r.q && at < b ? r.q[at] : zero;
    }
#pragma unroll
    for (int u = 0; u < kScalar; ++u) take(s[u & 1], i + u * 32 + lane, p[u], q[u]);
  }
  double t = ((double)s[0].hi + (double)s[0].lo) + ((double)s[1].hi + (double)s[1].lo);
#pragma unroll
  for (int o = 16; o; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  return t;
}

template <typename T>
__global__ void __launch_bounds__(kVerifyThreads) verify_kernel(const __grid_constant__ VerifyArgs a) {
  __shared__ double run_sum[kRuns];       // every run's sum, written by the whole cluster
  __shared__ double warp_tot[kVerifyWarps];
  __shared__ double sh_base, sh_th;
  __shared__ int sh_acc, sh_run, sh_first, sh_last;
  cg::cluster_group cl = cg::this_cluster();
  const int rank = (int)cl.block_rank(), seq = blockIdx.x / kVerifyCtas;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_launch_dependents();
  const int nd = a.n_draft ? min(max(a.n_draft[seq], 0), a.k) : a.k;
  const int* draft = a.draft + seq * a.draft_stride;
  const T* P = static_cast<const T*>(a.p) + seq * a.p_seq;
  const T* Q = a.q ? static_cast<const T*>(a.q) + seq * a.q_seq : nullptr;

  if (warp == 0) {   // accepted drafts, the same in every CTA of the cluster
    int acc = 0;
    for (int j0 = 0; j0 < nd; j0 += 32) {
      const int j = j0 + lane;
      bool take = false;
      if (j < nd) {
        const int x = draft[j];
        if (x >= 0 && x < a.vocab) {
          const float p = weight(as_f32(P[j * a.p_row + x]));
          const float q = Q ? weight(as_f32(Q[j * a.q_row + x])) : 1.f;
          take = (double)a.u_accept[seq * a.u_stride + j] * (double)q < (double)p;
        }
      }
      const unsigned refused = ~__ballot_sync(0xffffffffu, take);
      acc += refused ? __ffs(refused) - 1 : 32;
      if (refused) break;
    }
    if (lane == 0) sh_acc = acc;
  }
  __syncthreads();
  const int acc = sh_acc;
  const float u0 = a.u_token[seq];
  const double u = u0 > 0.f ? (double)fminf(u0, 1.f) : 0.0;
  const int V = a.vocab;
  // runs start on multiples of 16 entries
  const int len = ((V + kRuns - 1) / kRuns + 15) & ~15;
  Row<T> r{P + acc * a.p_row, nullptr, -1};
  if (acc < nd) {
    if (Q) r.q = Q + acc * a.q_row;
    else r.skip = draft[acc];
  }
  for (bool retry = true;; retry = false) {
    const int my = rank * kVerifyWarps + warp;
    const double t = warp_sum(r, min(my * len, V), min((my + 1) * len, V), lane);
    cl.sync();   // every CTA runs, and has read the sums of a first try
    if (lane < kVerifyCtas) *cl.map_shared_rank(&run_sum[my], lane) = t;
    cl.sync();
    if (warp == 0) {   // where u * total falls among the runs
      double v[kRuns / 32], c = 0.0;
#pragma unroll
      for (int i = 0; i < kRuns / 32; ++i) v[i] = c += run_sum[lane * (kRuns / 32) + i];
      double inc = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
      }
      double base = __shfl_up_sync(0xffffffffu, inc, 1);
      if (lane == 0) base = 0.0;
      const double th = u * __shfl_sync(0xffffffffu, inc, 31);
      int run = kRuns, last = -1;   // first run past th; last run with weight
      double before = 0.0;
#pragma unroll
      for (int i = kRuns / 32 - 1; i >= 0; --i) {
        const double prev = base + (i ? v[i - 1] : 0.0);
        if (base + v[i] > th) run = lane * (kRuns / 32) + i, before = prev;
        if (last < 0 && run_sum[lane * (kRuns / 32) + i] > 0.0) last = lane * (kRuns / 32) + i;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, run < kRuns);
      const int src = hit ? __ffs(hit) - 1 : 0;
      run = __shfl_sync(0xffffffffu, run, src);
      before = __shfl_sync(0xffffffffu, before, src);
      // u * total at or past the total: the last run that has weight
      last = __reduce_max_sync(0xffffffffu, last);
      if (lane == 0) {
        sh_run = hit ? run : last;
        sh_base = before;
        sh_th = hit ? th : INFINITY;
        sh_first = INT_MAX;
        sh_last = -1;
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
  // the entry of the run: each thread takes a few neighbours, the CTA scans
  const double th = sh_th;
  double base = sh_base;
  const int end = min((run + 1) * len, V);
  for (int i0 = run * len; i0 < end; i0 += kVerifyThreads * 4) {
    const int i = i0 + tid * 4;
    double w[4], c = 0.0;
    int last = -1;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const double x = i + j < end ? r.at(i + j) : 0.0;
      if (x > 0.0) last = i + j;
      w[j] = c += x;
    }
    double inc = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    if (lane == 31) warp_tot[warp] = inc;
    __syncthreads();
    double before = base;
    for (int v = 0; v < kVerifyWarps; ++v) {
      if (v < warp) before += warp_tot[v];
      base += warp_tot[v];
    }
    before += inc - c;
    int first = INT_MAX;
#pragma unroll
    for (int j = 3; j >= 0; --j)
      if (before + w[j] > th && w[j] > (j ? w[j - 1] : 0.0)) first = i + j;
    first = __reduce_min_sync(0xffffffffu, first);
    last = __reduce_max_sync(0xffffffffu, last);
    if (lane == 0) {
      if (first != INT_MAX) atomicMin(&sh_first, first);
      if (last >= 0) atomicMax(&sh_last, last);
    }
    __syncthreads();
    if (sh_first != INT_MAX) break;
  }
  // the scan may round below the run's own sum: then its last entry with weight
  if (tid == 0) out[acc] = sh_first != INT_MAX ? sh_first : max(sh_last, 0);
}

template <typename T>
cudaError_t launch(const VerifyArgs& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(a.n_seq * kVerifyCtas);
  cfg.blockDim = dim3(kVerifyThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {kVerifyCtas, 1, 1};
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, verify_kernel<T>, a);
}

}  // namespace

cudaError_t launch_verify(const VerifyArgs& a, int dtype, cudaStream_t s) {
  if (dtype == DFLASH_F32) return launch<float>(a, s);
  if (dtype == DFLASH_BF16) return launch<__nv_bfloat16>(a, s);
  return launch<__half>(a, s);
}

}  // namespace dfl

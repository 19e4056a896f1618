// next_step.cu -- the tables of a step from what stands of the last one and
// what is asked for: lengths, row starts, pages, and the place of every row.
//
// For sequence i with n_i keys, T_i of them the last step's rows, of which the
// first and a_i accepted drafts stand, and t_i rows asked for:
//   kept_i = min(keep_i, n_i)  or  n_i - T_i + min(T_i, 1 + a_i)  or  n_i
//   new_i  = kept_i + t_i, while pages and rows last (in order), else kept_i
// Pages behind the new length go on the free stack, the last sequence's last page
// first; then each sequence takes what it needs off its top, the first sequence
// first.  Both are prefix sums over the sequences: page a that is taken is the
// a-th that was given in ascending order, as long as there is one, and else
// comes from the old stack.  Giving back what was just taken restores the stack.
//
// A few hundred bytes a sequence at the most: latency bounds it, a chain of
// loads, two scans, a search and a look-up (3.4 us for 8 sequences, 6.3 for 256).  Every CTA scans all sequences (at
// most 4096: four a thread) and takes its part of the rows and of the pages that
// move, so there is one launch; lengths may be written where they were read
// because the CTA that comes last does it.
#include <atomic>

#include "kernels.cuh"
#include "ptx.cuh"
#include "step.cuh"

namespace dfl {
namespace {

constexpr int kMostSeqs = 4096;
constexpr int kMostThreads = 1024;
constexpr int kPer = kMostSeqs / kMostThreads;   // sequences of a thread

struct Sums {
  long long give, take, rows;
};
__device__ __forceinline__ Sums operator+(const Sums& a, const Sums& b) {
  return {a.give + b.give, a.take + b.take, a.rows + b.rows};
}
__device__ __forceinline__ Sums from_lane(const Sums& a, int lane) {
  return {__shfl_sync(0xffffffffu, a.give, lane), __shfl_sync(0xffffffffu, a.take, lane),
          __shfl_sync(0xffffffffu, a.rows, lane)};
}
// Sums of the threads before this one; *all: of every thread.
__device__ __forceinline__ Sums before(const Sums& mine, Sums* part, Sums* all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = blockDim.x >> 5;
  auto scan = [&](Sums inc) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const Sums x = from_lane(inc, max(lane - o, 0));
      if (lane >= o) inc = inc + x;
    }
    return inc;
  };
  const Sums inc = scan(mine);
  __syncthreads();           // the array's readers of an earlier call are done
  if (lane == 31) part[warp] = inc;
  __syncthreads();
  const Sums warps = scan(lane < n ? part[lane] : Sums{0, 0, 0});   // (by every warp; 32 adds in turn took 2 us)
  *all = from_lane(warps, 31);
  Sums base = from_lane(warps, max(warp - 1, 0));
  if (warp == 0) base = {0, 0, 0};
  return {base.give + inc.give - mine.give, base.take + inc.take - mine.take, base.rows + inc.rows - mine.rows};
}

// The last i with start[i] <= x, x < start[n]: who holds item x.
__device__ __forceinline__ int holder(const int* start, int n, int x) {
  int lo = 0, hi = n;        // start[lo] <= x < start[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kMostThreads) next_step_kernel(const __grid_constant__ NextArgs a) {
  extern __shared__ int shared[];
  __shared__ Sums part[kMostThreads / 32];
  __shared__ bool last;
  const int n = a.n_seq, tid = threadIdx.x, threads = blockDim.x;
  int* kept = shared;                 // [n]
  int* have = kept + n;               // [n] pages of the sequence before
  int* row0 = have + n;               // [n + 1] first row, page taken and page given
  int* take0 = row0 + n + 1;
  int* give0 = take0 + n + 1;
  pdl_wait();
  pdl_launch_dependents();
  const int shift = a.page_shift;
  const long long room = min((long long)a.table_cols << shift, (long long)INT_MAX - 256);
  auto pages = [&](long long len) { return (int)((len + (1 << shift) - 1) >> shift); };
  const int n_free = min(max(*a.n_free, 0), a.n_pages);
  const int per = (n + threads - 1) / threads, i0 = tid * per;

  int old[kPer], keep[kPer], want[kPer];
  Sums mine{0, 0, 0}, all;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int i = i0 + k;
    old[k] = keep[k] = want[k] = 0;
    if (k >= per || i >= n) continue;
    const int len = (int)min((long long)max(a.kv_len[i], 0), room);
    const int t = a.rows[i], acc = a.n_accepted ? a.n_accepted[i] : -1, given = a.keep ? a.keep[i] : -1;
    const int T = acc >= 0 ? min(max(a.row_start[i + 1] - a.row_start[i], 0), len) : 0;
    old[k] = len;
    keep[k] = given >= 0 ? min(given, len) : acc >= 0 ? len - T + (acc < T ? acc + 1 : T) : len;
    if (t > 0 && (long long)keep[k] + t <= room) want[k] = t;
    const int need = pages(keep[k] + want[k]) - pages(old[k]);
    mine = mine + Sums{max(-need, 0), max(need, 0), want[k]};
  }
  Sums run = before(mine, part, &all);
  const long long most = n_free + all.give;
  // rows for the sequences in order while pages and rows last
  mine = {0, 0, 0};
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    if (k >= per || i0 + k >= n) continue;
    const int need = pages(keep[k] + want[k]) - pages(old[k]);
    run.take += max(need, 0);
    run.rows += want[k];
    if (run.take > most || run.rows > a.n_rows) want[k] = 0;
    const int now = pages(keep[k] + want[k]) - pages(old[k]);
    mine = mine + Sums{max(-now, 0), max(now, 0), want[k]};
  }
  run = before(mine, part, &all);
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int i = i0 + k;
    if (k >= per || i >= n) continue;
    kept[i] = keep[k];
    have[i] = pages(old[k]);
    row0[i] = (int)run.rows;
    take0[i] = (int)run.take;
    give0[i] = (int)run.give;
    const int now = pages(keep[k] + want[k]) - have[i];
    run = run + Sums{max(-now, 0), max(now, 0), want[k]};
  }
  const int n_give = (int)all.give, n_take = (int)all.take, n_rows = (int)all.rows;
  const long long top = (long long)n_free + n_give;   // of the stack, once all are given (may pass 31 bits)
  if (tid == 0) {
    row0[n] = n_rows;
    take0[n] = n_take;
    give0[n] = n_give;
  }
  __syncthreads();

  // page x of those given, in ascending order
  auto given = [&](int x) {
    const int j = holder(give0, n, x);
    const int col = pages(kept[j] + row0[j + 1] - row0[j]) + x - give0[j];
    return a.block_table[j * a.table_stride + col];
  };
  auto taken = [&](int x) { return x < n_give ? given(x) : a.free[top - 1 - x]; };
  const int at = blockIdx.x * threads + tid, stride = gridDim.x * threads;
  for (int r = at; r < n_rows; r += stride) {
    const int i = holder(row0, n, r), own = kept[i] + r - row0[i], col = own >> shift;
    if (a.slots) {
      const int page = col < have[i] ? a.block_table[i * a.table_stride + col] : taken(take0[i] + col - have[i]);
      a.slots[r] = ((long long)page << shift) + (own & ((1 << shift) - 1));
    }
    if (a.positions) a.positions[r] = a.prefix_len + own;
    if (a.sequences) a.sequences[r] = i;
  }
  for (int x = at; x < n_take; x += stride) {           // (a row takes a page at most: far from 31 bits)
    const int i = holder(take0, n, x);
    a.block_table[i * a.table_stride + have[i] + x - take0[i]] = taken(x);
  }
  for (long long x = at; x < n_give; x += stride)
    if (top - 1 - x < a.n_pages) a.free[top - 1 - x] = given((int)x);

  // nobody reads the old lengths any more
  if (gridDim.x > 1) {
    __syncthreads();
    if (tid == 0) {
      __threadfence();
      last = atomicAdd(a.ticket, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!last) return;
    if (tid == 0) *a.ticket = 0;
  }
  for (int i = tid; i < n; i += threads) {
    a.kv_len_out[i] = kept[i] + row0[i + 1] - row0[i];
    a.row_start_out[i] = row0[i];
  }
  if (tid == 0) {
    a.row_start_out[n] = n_rows;
    *a.n_free_out = (int)min(top - n_take, (long long)a.n_pages);
  }
}

}  // namespace

cudaError_t launch_next_step(const NextArgs& a, int n_sm, cudaStream_t s) {
  // Up to four sequences a thread: smaller CTAs scan sooner (1245 sequences 6.9 us, with
  // 1024 threads 9.3), and a row a thread (256 sequences 6.3, with four 7.3).
  const int threads = a.n_seq <= kMostSeqs / 4 ? kMostThreads / 4 : a.n_seq <= kMostSeqs / 2 ? kMostThreads / 2 : kMostThreads;
  const size_t smem = (5 * (size_t)a.n_seq + 3) * sizeof(int);
  static std::atomic<uint64_t> raised{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(raised.load(std::memory_order_relaxed) >> dev & 1)) {
    e = cudaFuncSetAttribute(next_step_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)((5 * kMostSeqs + 3) * sizeof(int)));
    if (e != cudaSuccess) return e;
    if (dev < 64) raised.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
  }
  // (and a page, were a sixteenth of the table to move)
  const long work = a.n_rows + (long)a.n_seq * a.table_cols / 16;
  const long ctas = (work + threads - 1) / threads;
  const dim3 grid((unsigned)(ctas < 1 ? 1 : ctas < n_sm ? ctas : n_sm));
  return launch_pdl(next_step_kernel, grid, dim3(threads), smem, s, a);
}

}  // namespace dfl

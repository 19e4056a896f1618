// step.cuh -- device-side view of a target step (include/dflash.h,
// dflash_step and dflash_paged_cache) and the launches of its operators.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <limits.h>
#include <stdint.h>

namespace dfl {

// The step's lengths live on the device and are bounded where they are read:
// rows stay inside [0, n_rows], the keys that are read inside the block table.
struct StepView {
  int n_seq, n_rows;
  const int* row_start;
  const int* kv_len;
  const int* block_table;
  int table_cols;
  long table_stride;
  int prefix_len;
  const int* prefix_pages;
  int page_size, page_shift, n_pages;

  __host__ __device__ int start(int i) const { return min(max(row_start[i], 0), n_rows); }
  // own keys as given, and the rows the block table has room for
  __host__ __device__ int len(int i) const { return max(kv_len[i], 0); }
  __host__ __device__ int room() const {
    return (int)min((long)table_cols << page_shift, (long)INT_MAX);
  }
};

struct CacheView {
  void* k;
  void* v;
  long page_stride, row_stride, head_stride;   // elements
  int n_kv_heads, d;
};

struct AppendArgs {
  StepView s;
  CacheView c;
  const void* q;
  const void* k;
  const void* v;
  long q_stride, k_stride, v_stride;
  int n_heads;
  const float* q_gain;
  const float* k_gain;
  float eps;
  int rot;
  int interleaved;        // pairs (2j, 2j + 1) instead of (j, j + rot / 2)
  float mscale;
  const int* positions;
  void* q_out;
  long q_out_stride;
  uint64_t turns[64];   // turns per position modulo 1, times 2^64
};
// in_dtype / out_dtype: dflash_dtype values of q, k, v and of the cache
cudaError_t launch_step_append(const AppendArgs& a, int in_dtype, int out_dtype, int n_sm, cudaStream_t s);

// The same into a packed cache (fp4.cuh): a.c and sc give the codes' and the
// scales' places in bytes.
struct Append4Args {
  AppendArgs a;
  CacheView sc;
  double eps, mscale;   // as given, for what is computed again in 64 bits
  float k_unit, v_unit, k_inv_unit, v_inv_unit;
  void* k_values;       // the rounded rows in the queries' type, or null
  void* v_values;
  long k_values_stride, v_values_stride;
};
cudaError_t launch_step_append4(const Append4Args& a, int in_dtype, int out_dtype, int n_sm, cudaStream_t s);

struct VerifyArgs {
  int n_seq, k, vocab;
  const int* draft;
  long draft_stride;
  const int* n_draft;
  const void* p;
  long p_seq, p_row;
  const void* q;        // null: greedy drafts
  long q_seq, q_row;
  const float* u_accept;
  long u_stride;
  const float* u_token;
  int* tokens;
  int* n_accepted;
};
cudaError_t launch_verify(const VerifyArgs& a, int dtype, int n_sm, cudaStream_t s);

struct NextArgs {
  int n_seq, page_shift, table_cols, n_pages, n_rows, prefix_len;
  long table_stride;
  const int* kv_len;
  const int* row_start;
  const int* n_free;
  const int* rows;
  const int* n_accepted;   // or null
  const int* keep;         // or null
  int* block_table;
  int* free;
  int* kv_len_out;
  int* row_start_out;
  int* n_free_out;
  long long* slots;        // or null, like the next two
  int* positions;
  int* sequences;
  unsigned* ticket;        // 0 between calls
};
cudaError_t launch_next_step(const NextArgs& a, int n_sm, cudaStream_t s);

// Boxes of a packed cache: codes [rows of a page][head_dim / 2 bytes],
// swizzled by their length, and the scales of as many rows.
struct PackedMaps {
  CUtensorMap k, v, k_scale, v_scale;
};
// The same of K and V in one box, the one that lies lower in memory first, or of K
// and of V where they lie too far apart; of codes and of scales.
struct PairMaps {
  CUtensorMap codes[2], scales[2];
  int pair[2], v_first[2];
};

// Attention of a step (step_attn.cu; how it is cut into pieces: step_plan.cuh).
constexpr int kStepStatusWords = 1024;   // most CTAs (one status word each)
struct StepAttnArgs {
  StepView s;
  int Hq, Hkv, G, d;
  int tpt;             // tokens of a 128-row tile: floor(128 / G)
  int causal;
  float scale_log2;    // scale * log2(e)
  int bf16;            // else f16
  int box_rows, boxes; // rows of one cache box (a page, at most 128) and boxes of a 128-key tile
  void* out;
  long out_stride;
  float* lse;
  // workspace
  int* status;         // [n_cta]
  int by_cta;          // the merge goes by CTA (split), else by row (meta)
  int4* meta;          // [2][n_rows][Hkv]: segment's first and last CTA, row's token within its tiles,
                       // whether the row's result is written
  int4* split;         // [n_cta]: first row, tokens, kv head and last CTA of the item that
                       // begins in a CTA and goes on in others (no tokens: none)
  float* seg_o[2];     // [n_rows][Hq][d]: a segment's first fragment (prefix, own), unnormalised
  float2* seg_ml[2];   // [n_rows][Hq]: its (max, sum)
  float* cta_o;        // [cta_row][d]: the fragment a CTA continues
  float2* cta_ml;      // [cta_row]
  int n_cta;           // CTAs that leave partial results: n_wide of step_attn.cu, whose rows come
  int n_wide;          // first, then those of step_attn_few.cu (16 rows each)
  int n_sm;
  // (of a packed cache, behind the others: among them they cost the 16-bit kernel 0.7 us of 111)
  int few_rows;        // most query rows of an item of step_attn_few.cu: 8 or kFewRows
  float out_scale;     // of the results
  const void* q;       // (step_attn_few.cu; the other kernel loads boxes)
  long q_stride;
};
// Partial rows of a CTA, and one of them among all CTAs'.
__host__ __device__ inline int cta_rows(const StepAttnArgs& a, int cta) { return cta < a.n_wide ? 256 : 16; }
__host__ __device__ inline long cta_row(const StepAttnArgs& a, int cta, int row) {
  return cta < a.n_wide ? cta * 256L + row : a.n_wide * 256L + (cta - a.n_wide) * 16L + row;
}
cudaError_t launch_step_attention(const StepAttnArgs& a, const CUtensorMap& q, const CUtensorMap& k,
                                  const CUtensorMap& v, cudaStream_t s);
cudaError_t launch_step_attention4(const StepAttnArgs& a, const CUtensorMap& q, const PackedMaps& m, cudaStream_t s);
// wide_ran: launch_step_attention4 went before with the items of many rows, and has
// set the status words; else this does all of them.
cudaError_t launch_step_attention_few(const StepAttnArgs& a, const PairMaps& m, bool wide_ran, cudaStream_t s);
// o = out_scale sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i over the fragments of every row that is not whole.
cudaError_t launch_step_merge(const StepAttnArgs& a, cudaStream_t s);

// The calling thread's error message (dflash_last_error); returns code.
int report_error(int code, const char* message);
// Tiled tensor map of 16-bit elements, 128-byte swizzle; false on failure.
bool encode_tiled_map(CUtensorMap* m, int dtype, uint32_t rank, const void* base, const uint64_t* dims,
                      const uint64_t* strides, const uint32_t* box);
// The same of bytes in rows of 32 or 64 (swizzled by that) or of 4- or 8-byte
// elements that lie as they are.
bool encode_packed_map(CUtensorMap* m, int element_bytes, uint32_t rank, const void* base, const uint64_t* dims,
                       const uint64_t* strides, const uint32_t* box);

}  // namespace dfl

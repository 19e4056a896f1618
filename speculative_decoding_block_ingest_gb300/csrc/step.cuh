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
  float mscale;
  const int* positions;
  void* q_out;
  long q_out_stride;
  uint64_t turns[64];   // turns per position modulo 1, times 2^64
};
// in_dtype / out_dtype: dflash_dtype values of q, k, v and of the cache
cudaError_t launch_step_append(const AppendArgs& a, int in_dtype, int out_dtype, int n_sm, cudaStream_t s);

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
  float* cta_o;        // [n_cta][256][d]: the fragment a CTA continues
  float2* cta_ml;      // [n_cta][256]
  int n_cta;
};
cudaError_t launch_step_attention(const StepAttnArgs& a, const CUtensorMap& q, const CUtensorMap& k,
                                  const CUtensorMap& v, cudaStream_t s);

// The calling thread's error message (dflash_last_error); returns code.
int report_error(int code, const char* message);
// Tiled tensor map of 16-bit elements, 128-byte swizzle; false on failure.
bool encode_tiled_map(CUtensorMap* m, int dtype, uint32_t rank, const void* base, const uint64_t* dims,
                      const uint64_t* strides, const uint32_t* box);

}  // namespace dfl

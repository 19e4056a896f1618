// target.cu -- C ABI of the target model's side of a speculative step
// (include/dflash.h): argument checks, tensor maps and launches.
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "../../include/dflash.h"
#include "dflash_internal.cuh"
#include "step_plan.cuh"

using namespace dfl;

namespace {

constexpr int kMaxSeqs = 4096;
constexpr int kMaxGroup = 64;      // query heads of a kv head
constexpr int kMaxHeads = 1024;
constexpr int kMaxRows = 1 << 24;

int fail(int code, const char* fmt, ...) {
  char buf[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return report_error(code, buf);
}
int invalid(const char* what) { return fail(DFLASH_ERR_INVALID_ARG, "%s", what); }

int launched(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return DFLASH_OK;
  return fail(DFLASH_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

int check_cache_shape(const dflash_paged_cache* c) {
  if (!c) return invalid("cache is null");
  if (c->dtype != DFLASH_BF16 && c->dtype != DFLASH_F16)
    return fail(DFLASH_ERR_UNSUPPORTED, "cache dtype must be DFLASH_BF16 or DFLASH_F16");
  if (c->head_dim != 64 && c->head_dim != 128) return fail(DFLASH_ERR_UNSUPPORTED, "head_dim must be 64 or 128");
  if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1)))
    return fail(DFLASH_ERR_UNSUPPORTED, "page_size must be 16, 32, 64, 128 or 256");
  if (c->n_kv_heads < 1 || c->n_kv_heads > kMaxHeads) return invalid("n_kv_heads out of range");
  return DFLASH_OK;
}

int check_cache(const dflash_paged_cache* c) {
  if (int rc = check_cache_shape(c)) return rc;
  if (!c->k || !c->v) return invalid("cache pointer is null");
  if (c->n_pages < 1) return invalid("n_pages must be positive");
  if (!aligned(c->k, 16) || !aligned(c->v, 16)) return invalid("caches must start on a 16-byte boundary");
  for (long st : {(long)c->page_stride, (long)c->row_stride, (long)c->head_stride})
    if (st < 8 || st % 8 || st >= (1L << 38)) return invalid("cache strides must be positive multiples of 8 elements");
  if (c->head_stride < c->head_dim || c->row_stride < c->head_dim || c->page_stride < c->head_dim)
    return invalid("cache strides must not be shorter than a head row");
  return DFLASH_OK;
}

int check_step(const dflash_paged_cache* c, const dflash_step* s) {
  if (!s) return invalid("step is null");
  if (s->n_seq < 1 || s->n_seq > kMaxSeqs) return fail(DFLASH_ERR_INVALID_ARG, "n_seq must be 1..%d", kMaxSeqs);
  if (s->n_rows < 0 || s->n_rows > kMaxRows) return invalid("n_rows out of range");
  if (!s->row_start || !s->kv_len || (!s->block_table && s->table_cols > 0)) return invalid("step array is null");
  if (s->table_cols < 0 || (s->table_stride < s->table_cols && s->table_stride != 0)) return invalid("block table shape");
  if (s->prefix_len < 0 || (s->prefix_len > 0 && !s->prefix_pages)) return invalid("prefix");
  // the ends of the last block of keys and of the last page have 32-bit indices too
  if ((long)s->prefix_len + (long)s->table_cols * c->page_size >= (1L << 31) - 256)
    return invalid("more than 2^31 - 257 keys");
  return DFLASH_OK;
}

StepView view(const dflash_paged_cache* c, const dflash_step* s) {
  StepView v{};
  v.n_seq = s->n_seq;
  v.n_rows = s->n_rows;
  v.row_start = s->row_start;
  v.kv_len = s->kv_len;
  v.block_table = s->block_table;
  v.table_cols = s->table_cols;
  v.table_stride = s->table_stride;
  v.prefix_len = s->prefix_len;
  v.prefix_pages = s->prefix_pages;
  v.page_size = c->page_size;
  v.page_shift = __builtin_ctz(c->page_size);
  v.n_pages = c->n_pages;
  return v;
}

// SMs of the current device (asked once for each).
int sm_count(int* n) {
  static std::atomic<int> known[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && dev < 64 && (*n = known[dev].load(std::memory_order_relaxed)) > 0) return DFLASH_OK;
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return launched(e, "device SM count");
  if (dev < 64) known[dev].store(*n, std::memory_order_relaxed);
  return DFLASH_OK;
}

// CTAs of the attention: one per SM (each takes all of an SM's tensor memory).
int step_ctas(int* n) {
  if (int rc = sm_count(n)) return rc;
  if (*n > kStepStatusWords) *n = kStepStatusWords;
  return DFLASH_OK;
}

int check_heads(const dflash_paged_cache* c, int32_t n_heads) {
  if (n_heads < 1 || n_heads > kMaxHeads || n_heads % c->n_kv_heads)
    return invalid("n_heads must be a multiple of n_kv_heads");
  if (n_heads / c->n_kv_heads > kMaxGroup)
    return fail(DFLASH_ERR_UNSUPPORTED, "more than %d query heads per kv head", kMaxGroup);
  return DFLASH_OK;
}

int check_rows(int32_t n_rows, int32_t n_heads) {
  if (n_rows < 0 || n_rows > kMaxRows || (long)n_rows * n_heads > (1L << 31)) return invalid("n_rows out of range");
  return DFLASH_OK;
}

// Workspace: status words, where rows' fragments are (by row, by CTA), first
// fragments of both segments, one continued tile pair per CTA.
size_t carve(StepAttnArgs& a, char* base) {
  size_t off = 0;
  auto take = [&](size_t bytes) {
    char* p = base + off;
    off += up256(bytes);
    return p;
  };
  const size_t rows = a.s.n_rows;
  a.status = reinterpret_cast<int*>(take(kStepStatusWords * 4));
  a.meta = reinterpret_cast<int4*>(take(2 * rows * a.Hkv * sizeof(int4)));
  a.split = reinterpret_cast<int4*>(take((size_t)a.n_cta * sizeof(int4)));
  for (int i = 0; i < 2; ++i) {
    a.seg_o[i] = reinterpret_cast<float*>(take(rows * a.Hq * a.d * 4));
    a.seg_ml[i] = reinterpret_cast<float2*>(take(rows * a.Hq * 8));
  }
  a.cta_o = reinterpret_cast<float*>(take((size_t)a.n_cta * 256 * a.d * 4));
  a.cta_ml = reinterpret_cast<float2*>(take((size_t)a.n_cta * 256 * 8));
  return off;
}

void set_shape(StepAttnArgs& a, const dflash_paged_cache* c, int n_heads) {
  a.Hq = n_heads;
  a.Hkv = c->n_kv_heads;
  a.G = a.Hq / a.Hkv;
  a.d = c->head_dim;
  a.tpt = 128 / a.G;
}

}  // namespace

extern "C" {

int dflash_step_append(const dflash_paged_cache* cache, const dflash_step* step, const dflash_append_args* p,
                       void* stream) {
  report_error(DFLASH_OK, "");
  if (int rc = check_cache(cache)) return rc;
  if (int rc = check_step(cache, step)) return rc;
  if (!p) return invalid("args is null");
  if (p->dtype != DFLASH_F32 && p->dtype != cache->dtype)
    return fail(DFLASH_ERR_UNSUPPORTED, "rows must be DFLASH_F32 or of the cache's dtype");
  if (p->n_heads < 0 || p->n_heads > kMaxHeads) return invalid("n_heads out of range");
  if (p->rot_dim < 0 || p->rot_dim > cache->head_dim || p->rot_dim % 16)
    return invalid("rot_dim must be a multiple of 16 up to head_dim");
  if (p->rot_dim > 0 && (!p->inv_freq || !std::isfinite((float)p->mscale))) return invalid("RoPE frequencies");
  if ((p->q_gain || p->k_gain) && !((float)p->eps > 0)) return invalid("eps must be > 0 in f32");
  if (step->n_rows == 0) return DFLASH_OK;
  if (!p->k || !p->v || (p->n_heads > 0 && (!p->q || !p->q_out))) return invalid("row pointer is null");
  const int d = cache->head_dim;
  const long vec = p->dtype == DFLASH_F32 ? 4 : 8;
  auto rows_ok = [&](const void* ptr, long stride, long heads, long v) {
    return aligned(ptr, 16) && stride >= heads * d && stride % v == 0;
  };
  if (!rows_ok(p->k, p->k_stride, cache->n_kv_heads, vec) || !rows_ok(p->v, p->v_stride, cache->n_kv_heads, vec) ||
      (p->n_heads > 0 &&
       (!rows_ok(p->q, p->q_stride, p->n_heads, vec) || !rows_ok(p->q_out, p->q_out_stride, p->n_heads, 8))))
    return invalid("rows must start on 16-byte boundaries and strides hold a row");
  if (!aligned(p->q_gain, 16) || !aligned(p->k_gain, 16)) return invalid("gains must start on a 16-byte boundary");
  AppendArgs a{};
  a.s = view(cache, step);
  a.c = {cache->k, cache->v, cache->page_stride, cache->row_stride, cache->head_stride, cache->n_kv_heads, d};
  a.q = p->q;
  a.k = p->k;
  a.v = p->v;
  a.q_stride = p->q_stride;
  a.k_stride = p->k_stride;
  a.v_stride = p->v_stride;
  a.n_heads = p->n_heads;
  a.q_gain = p->q_gain;
  a.k_gain = p->k_gain;
  a.eps = (float)p->eps;
  a.rot = p->rot_dim;
  a.mscale = (float)p->mscale;
  a.positions = p->positions;
  a.q_out = p->q_out;
  a.q_out_stride = p->q_out_stride;
  for (int i = 0; i < p->rot_dim / 2; ++i) {
    const double t = p->inv_freq[i] / (2.0 * M_PI);
    if (!std::isfinite(t)) return invalid("RoPE frequencies");
    a.turns[i] = (uint64_t)std::ldexp(t - std::floor(t), 64);
  }
  int n_sm = 0;
  if (int rc = sm_count(&n_sm)) return rc;
  return launched(launch_step_append(a, p->dtype, cache->dtype, n_sm, static_cast<cudaStream_t>(stream)),
                  "step append");
}

int dflash_step_attention_workspace(const dflash_paged_cache* cache, int32_t n_rows, int32_t n_heads, size_t* bytes) {
  report_error(DFLASH_OK, "");
  if (!bytes) return invalid("bytes is null");
  if (int rc = check_cache_shape(cache)) return rc;
  if (int rc = check_heads(cache, n_heads)) return rc;
  if (int rc = check_rows(n_rows, n_heads)) return rc;
  StepAttnArgs a{};
  set_shape(a, cache, n_heads);
  a.s.n_rows = n_rows;
  if (int rc = step_ctas(&a.n_cta)) return rc;
  *bytes = carve(a, nullptr);
  return DFLASH_OK;
}

int dflash_step_attention(const dflash_paged_cache* cache, const dflash_step* step, const dflash_attention_args* p,
                          void* workspace, size_t workspace_bytes, void* stream) {
  report_error(DFLASH_OK, "");
  if (int rc = check_cache(cache)) return rc;
  if (int rc = check_step(cache, step)) return rc;
  if (!p) return invalid("args is null");
  if (int rc = check_heads(cache, p->n_heads)) return rc;
  if (int rc = check_rows(step->n_rows, p->n_heads)) return rc;
  if (!std::isfinite(p->scale) || p->scale < 0) return invalid("scale must be finite and not negative");
  if (!workspace || !aligned(workspace, 256)) return invalid("workspace must start on a 256-byte boundary");
  const int d = cache->head_dim;
  if (step->n_rows > 0) {
    if (!p->q || !p->out) return invalid("row pointer is null");
    if (!aligned(p->q, 16) || !aligned(p->out, 16) || p->q_stride % 8 || p->out_stride % 8 ||
        p->q_stride < (long)p->n_heads * d || p->out_stride < (long)p->n_heads * d || p->q_stride >= (1L << 38))
      return invalid("rows must start on 16-byte boundaries and strides hold a row");
  }
  StepAttnArgs a{};
  a.s = view(cache, step);
  set_shape(a, cache, p->n_heads);
  if (int rc = step_ctas(&a.n_cta)) return rc;
  a.causal = p->causal != 0;
  if (!step_fits(a, a.s.room())) return fail(DFLASH_ERR_UNSUPPORTED, "more work than one call takes: fewer rows");
  const float scale = p->scale > 0 ? p->scale : 1.f / std::sqrt((float)d);
  a.scale_log2 = scale * 1.4426950408889634f;
  a.bf16 = cache->dtype == DFLASH_BF16;
  a.box_rows = cache->page_size < kKeys ? cache->page_size : kKeys;
  a.boxes = kKeys / a.box_rows;
  a.out = p->out;
  a.out_stride = p->out_stride;
  a.lse = p->lse;
  // Without a prefix only the rows of items that go on in another CTA have
  // something to merge, at most 256 a CTA: worth looking for them there where
  // there are many more (four prompts of 2000 rows: 178 us against 223; 32
  // single tokens 24.9 against 22.8).
  a.by_cta = step->prefix_len == 0 && (long)step->n_rows * p->n_heads > 256L * a.n_cta;
  const size_t need = carve(a, static_cast<char*>(workspace));
  if (workspace_bytes < need)
    return fail(DFLASH_ERR_CAPACITY, "workspace holds %zu bytes, %zu needed", workspace_bytes, need);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (step->n_rows == 0) return launched(cudaMemsetAsync(a.status, 0, kStepStatusWords * 4, s), "step attention");
  CUtensorMap mq, mk, mv;
  const uint64_t qdims[3] = {(uint64_t)d, (uint64_t)p->n_heads, (uint64_t)step->n_rows};
  const uint64_t qstr[2] = {(uint64_t)d * 2, (uint64_t)p->q_stride * 2};
  const uint32_t qbox[3] = {64, (uint32_t)a.G, (uint32_t)a.tpt};
  const uint64_t cdims[4] = {(uint64_t)d, (uint64_t)cache->n_kv_heads, (uint64_t)cache->page_size,
                             (uint64_t)cache->n_pages};
  const uint64_t cstr[3] = {(uint64_t)cache->head_stride * 2, (uint64_t)cache->row_stride * 2,
                            (uint64_t)cache->page_stride * 2};
  const uint32_t cbox[4] = {64, 1, (uint32_t)a.box_rows, 1};
  if (!encode_tiled_map(&mq, cache->dtype, 3, p->q, qdims, qstr, qbox) ||
      !encode_tiled_map(&mk, cache->dtype, 4, cache->k, cdims, cstr, cbox) ||
      !encode_tiled_map(&mv, cache->dtype, 4, cache->v, cdims, cstr, cbox))
    return fail(DFLASH_ERR_CUDA, "tensor map of the queries or the cache was refused");
  return launched(launch_step_attention(a, mq, mk, mv, s), "step attention");
}

int dflash_step_attention_status(const void* workspace, void* stream) {
  report_error(DFLASH_OK, "");
  if (!workspace) return invalid("workspace is null");
  int n = 0;
  if (int rc = step_ctas(&n)) return rc;
  static thread_local int words[kStepStatusWords];
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaMemcpyAsync(words, workspace, n * sizeof(int), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return launched(e, "step attention status");
  for (int i = 0; i < n; ++i)
    if (words[i]) return fail(DFLASH_ERR_TIMEOUT, "a device-side wait of the step attention gave up (CTA %d)", i);
  return DFLASH_OK;
}

int dflash_step_attention_plan(const dflash_paged_cache* cache, const dflash_step* step, int32_t n_heads,
                               int32_t causal, int32_t n_cta, int32_t* n_pieces, dflash_step_piece* pieces,
                               int32_t max_pieces) {
  report_error(DFLASH_OK, "");
  if (int rc = check_cache_shape(cache)) return rc;
  if (int rc = check_step(cache, step)) return rc;
  if (int rc = check_heads(cache, n_heads)) return rc;
  if (!n_pieces || (max_pieces > 0 && !pieces)) return invalid("null argument");
  if (n_cta < 1 || n_cta > kStepStatusWords) return invalid("n_cta out of range");
  StepAttnArgs a{};
  a.s = view(cache, step);
  set_shape(a, cache, n_heads);
  a.causal = causal != 0;
  if (!step_fits(a, a.s.room())) return fail(DFLASH_ERR_UNSUPPORTED, "more work than one call takes: fewer rows");
  Walk w(a);
  int total = w.prefix_units();
  for (int i = 0; i < step->n_seq; ++i) {
    if (w.falls(i)) {
      total = 0;
      break;
    }
    total += a.Hkv * w.head_units(i);
  }
  int n = 0;
  for (int c = 0; c < n_cta; ++c) {
    w.divide(total, n_cta, c);
    if (w.ua >= w.ub) continue;
    int seq0 = -1, base = 0;
    if (w.ua >= w.prefix_units()) {
      base = w.prefix_units();
      for (seq0 = 0;; ++seq0) {
        const int u = a.Hkv * w.head_units(seq0);
        if (w.ua < base + u) break;
        base += u;
      }
    }
    w.begin(seq0, base);
    for (Frag f; w.next(f); ++n)
      if (n < max_pieces)
        pieces[n] = {c, f.seg, f.seg ? f.seq : -1, f.h, f.tok0, f.ntok, f.b0, f.b1, f.first, f.last_cta};
  }
  *n_pieces = n;
  return n > max_pieces ? fail(DFLASH_ERR_CAPACITY, "%d pieces, room for %d", n, max_pieces) : DFLASH_OK;
}

int dflash_verify_tokens(const dflash_verify_args* p, void* stream) {
  report_error(DFLASH_OK, "");
  if (!p) return invalid("args is null");
  if (p->n_seq < 1 || p->n_seq > (1 << 20)) return invalid("n_seq out of range");
  if (p->k < 0 || p->k > (1 << 16)) return invalid("k out of range");
  if (p->vocab < 1 || p->vocab > (1 << 30)) return invalid("vocab out of range");
  if (p->dtype != DFLASH_F32 && p->dtype != DFLASH_BF16 && p->dtype != DFLASH_F16)
    return fail(DFLASH_ERR_UNSUPPORTED, "probabilities must be DFLASH_F32, DFLASH_BF16 or DFLASH_F16");
  if (!p->target_probs || !p->u_token || !p->tokens || !p->n_accepted || (p->k > 0 && (!p->draft || !p->u_accept)))
    return invalid("null argument");
  if (p->target_row_stride < p->vocab || (p->draft_probs && p->k > 0 && p->draft_row_stride < p->vocab))
    return invalid("probability rows must hold the vocabulary");
  if (p->target_seq_stride < 0 || p->draft_seq_stride < 0 || p->draft_stride < 0 || p->u_accept_stride < 0)
    return invalid("strides must not be negative");
  const size_t es = p->dtype == DFLASH_F32 ? 4 : 2;
  if (!aligned(p->target_probs, es) || !aligned(p->draft_probs, es)) return invalid("misaligned probabilities");
  VerifyArgs a{};
  a.n_seq = p->n_seq;
  a.k = p->k;
  a.vocab = p->vocab;
  a.draft = p->draft;
  a.draft_stride = p->draft_stride;
  a.n_draft = p->n_draft;
  a.p = p->target_probs;
  a.p_seq = p->target_seq_stride;
  a.p_row = p->target_row_stride;
  a.q = p->draft_probs;
  a.q_seq = p->draft_seq_stride;
  a.q_row = p->draft_row_stride;
  a.u_accept = p->u_accept;
  a.u_stride = p->u_accept_stride;
  a.u_token = p->u_token;
  a.tokens = p->tokens;
  a.n_accepted = p->n_accepted;
  int n_sm = 0;
  if (int rc = sm_count(&n_sm)) return rc;
  return launched(launch_verify(a, p->dtype, n_sm, static_cast<cudaStream_t>(stream)), "verify tokens");
}

}  // extern "C"

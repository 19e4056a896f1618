// target.cu -- C ABI of the target model's side of a speculative step
// (include/dflash.h): argument checks, tensor maps and launches.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <utility>

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

void set_shape(StepAttnArgs& a, const dflash_paged_cache* c, int n_heads) {
  a.Hq = n_heads;
  a.Hkv = c->n_kv_heads;
  a.G = a.Hq / a.Hkv;
  a.d = c->head_dim;
  a.tpt = 128 / a.G;
}

// CTAs of an attention kernel: one per SM (each takes all of an SM's tensor memory).
int step_ctas(int* n) {
  if (int rc = sm_count(n)) return rc;
  if (*n > kStepStatusWords) *n = kStepStatusWords;
  return DFLASH_OK;
}
// Those of all kernels of a call; over a packed cache few rows have one of their own.
int set_ctas(StepAttnArgs& a, bool packed) {
  if (int rc = step_ctas(&a.n_sm)) return rc;
  a.n_wide = a.n_sm;
  a.n_cta = packed && a.G <= kFewRows ? 2 * a.n_sm : a.n_sm;
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
  const size_t parts = cta_row(a, a.n_cta, 0);
  a.cta_o = reinterpret_cast<float*>(take(parts * a.d * 4));
  a.cta_ml = reinterpret_cast<float2*>(take(parts * 8));
  return off;
}

bool rows_ok(const void* ptr, long stride, long elements, long v) {
  return aligned(ptr, 16) && stride >= elements && stride % v == 0;
}

int check_append(const dflash_paged_cache* cache, const dflash_step* step, const dflash_append_args* p) {
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
  const long v = p->dtype == DFLASH_F32 ? 4 : 8, kv = (long)cache->n_kv_heads * cache->head_dim,
             q = (long)p->n_heads * cache->head_dim;
  if (!rows_ok(p->k, p->k_stride, kv, v) || !rows_ok(p->v, p->v_stride, kv, v) ||
      (p->n_heads > 0 && (!rows_ok(p->q, p->q_stride, q, v) || !rows_ok(p->q_out, p->q_out_stride, q, 8))))
    return invalid("rows must start on 16-byte boundaries and strides hold a row");
  if (!aligned(p->q_gain, 16) || !aligned(p->k_gain, 16)) return invalid("gains must start on a 16-byte boundary");
  return DFLASH_OK;
}

// f / (2 pi) modulo 1, times 2^64, to the nearest: f's 53 bits times the first 192 bits of
// 1 / (2 pi), enough for |f| below 2^120 (others get 0).  A quotient of doubles has 53 bits, which
// is 2^-32 of a turn at position 2^24 for a frequency of 1.
uint64_t turns_of(double f) {
  static const uint64_t inverse[3] = {0x36d8a5664f10e410, 0x7f09d5f47d4d3770, 0x28be60db9391054a};   // low word first
  int e = 0;
  const uint64_t m = (uint64_t)std::ldexp(std::frexp(std::fabs(f), &e), 53);   // |f| = m 2^(e - 53)
  if (e > 120) return 0;
  uint64_t w[5] = {};               // m / (2 pi) times 2^192
  unsigned __int128 carry = 0;
  for (int i = 0; i < 3; ++i) {
    carry += (unsigned __int128)m * inverse[i];
    w[i] = (uint64_t)carry;
    carry >>= 64;
  }
  w[3] = (uint64_t)carry;
  const int down = 181 - e;         // bits of w below the result's
  if (down > 256) return 0;
  auto bits = [&](int at) {         // 64 of them from bit `at` on (0: below the first)
    const int i = at >> 6, s = at & 63;
    if (i > 3) return (uint64_t)0;
    return s ? w[i] >> s | w[i + 1] << (64 - s) : w[i];
  };
  const uint64_t t = bits(down) + (bits(down - 1) & 1);
  return f < 0 ? 0 - t : t;
}

// All of an append's arguments but the cache's.
int append_args(AppendArgs& a, const dflash_paged_cache* cache, const dflash_step* step,
                const dflash_append_args* p, bool interleaved) {
  a.s = view(cache, step);
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
  a.interleaved = interleaved;
  a.mscale = (float)p->mscale;
  a.positions = p->positions;
  a.q_out = p->q_out;
  a.q_out_stride = p->q_out_stride;
  for (int i = 0; i < p->rot_dim / 2; ++i) {
    if (!std::isfinite(p->inv_freq[i])) return invalid("RoPE frequencies");
    a.turns[i] = turns_of(p->inv_freq[i]);
  }
  return DFLASH_OK;
}

int step_append(const dflash_paged_cache* cache, const dflash_step* step, const dflash_append_args* p,
                bool interleaved, void* stream) {
  report_error(DFLASH_OK, "");
  if (int rc = check_cache(cache)) return rc;
  if (int rc = check_step(cache, step)) return rc;
  if (int rc = check_append(cache, step, p)) return rc;
  if (step->n_rows == 0) return DFLASH_OK;
  AppendArgs a{};
  if (int rc = append_args(a, cache, step, p, interleaved)) return rc;
  a.c = {cache->k, cache->v, cache->page_stride, cache->row_stride, cache->head_stride, cache->n_kv_heads,
         cache->head_dim};
  int n_sm = 0;
  if (int rc = sm_count(&n_sm)) return rc;
  return launched(launch_step_append(a, p->dtype, cache->dtype, n_sm, static_cast<cudaStream_t>(stream)),
                  "step append");
}

// A packed cache's shape, for the checks that know the other kind.
dflash_paged_cache shape_of(const dflash_packed_cache* c) {
  dflash_paged_cache s{};
  s.dtype = c->dtype;
  s.n_pages = c->n_pages;
  s.page_size = c->page_size;
  s.n_kv_heads = c->n_kv_heads;
  s.head_dim = c->head_dim;
  return s;
}

int check_packed_shape(const dflash_packed_cache* c) {
  if (!c) return invalid("cache is null");
  const dflash_paged_cache s = shape_of(c);
  return check_cache_shape(&s);
}

// a power of two whose products and quotients with codes stay floats
bool is_unit(float u) {
  int e = 0;
  return std::isfinite(u) && u > 0 && std::frexp(u, &e) == 0.5f && e > -60 && e < 60;
}

int check_packed(const dflash_packed_cache* c) {
  if (int rc = check_packed_shape(c)) return rc;
  if (!c->k || !c->v || !c->k_scale || !c->v_scale) return invalid("cache pointer is null");
  if (c->n_pages < 1) return invalid("n_pages must be positive");
  const long row = c->head_dim / 2, sc = c->head_dim / 16;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 16) || !aligned(c->v_scale, 16))
    return invalid("codes and scales must start on 16-byte boundaries");
  for (long st : {(long)c->page_stride, (long)c->row_stride, (long)c->head_stride})
    if (st < row || st % 16 || st >= (1L << 38))
      return invalid("code strides must be multiples of 16 bytes that hold a head row");
  if (c->scale_row_stride != sc) return fail(DFLASH_ERR_UNSUPPORTED, "the scales of a head's rows of a page must lie together");
  for (long st : {(long)c->scale_page_stride, (long)c->scale_head_stride})
    if (st < sc * c->page_size || st % 16 || st >= (1L << 38))
      return invalid("scale strides must be multiples of 16 bytes that hold a page's rows");
  if (!is_unit(c->k_unit) || !is_unit(c->v_unit)) return invalid("units must be powers of two between 2^-60 and 2^58");
  return DFLASH_OK;
}

int check_attention(const dflash_paged_cache* cache, const dflash_step* step, const dflash_attention_args* p,
                    const void* workspace) {
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
  return DFLASH_OK;
}

// All of an attention's arguments but the cache's.
int attention_args(StepAttnArgs& a, const dflash_paged_cache* cache, const dflash_step* step,
                   const dflash_attention_args* p, bool packed) {
  a.s = view(cache, step);
  set_shape(a, cache, p->n_heads);
  if (int rc = set_ctas(a, packed)) return rc;
  a.causal = p->causal != 0;
  if (!step_fits(a, a.s.room())) return fail(DFLASH_ERR_UNSUPPORTED, "more work than one call takes: fewer rows");
  const float scale = p->scale > 0 ? p->scale : 1.f / std::sqrt((float)cache->head_dim);
  a.scale_log2 = scale * 1.4426950408889634f;
  a.out_scale = 1.f;
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
  a.by_cta = step->prefix_len == 0 && (long)step->n_rows * p->n_heads > 256L * a.n_sm;
  return DFLASH_OK;
}

int attention_workspace(const dflash_paged_cache* cache, int32_t n_rows, int32_t n_heads, size_t* bytes, bool packed) {
  if (!bytes) return invalid("bytes is null");
  if (int rc = check_cache_shape(cache)) return rc;
  if (int rc = check_heads(cache, n_heads)) return rc;
  if (int rc = check_rows(n_rows, n_heads)) return rc;
  StepAttnArgs a{};
  set_shape(a, cache, n_heads);
  a.s.n_rows = n_rows;
  if (int rc = set_ctas(a, packed)) return rc;
  *bytes = carve(a, nullptr);
  return DFLASH_OK;
}

int has_workspace(size_t bytes, size_t need) {
  if (bytes < need) return fail(DFLASH_ERR_CAPACITY, "workspace holds %zu bytes, %zu needed", bytes, need);
  return DFLASH_OK;
}

// Maps of boxes of `rows` rows of a page.
bool encode_packed(PackedMaps* m, const dflash_packed_cache* c, int rows) {
  const uint64_t heads = c->n_kv_heads, page = c->page_size, n_pages = c->n_pages;
  const uint64_t dims[4] = {(uint64_t)c->head_dim / 2, heads, page, n_pages}, sdims[3] = {page, heads, n_pages};
  const uint64_t strides[3] = {(uint64_t)c->head_stride, (uint64_t)c->row_stride, (uint64_t)c->page_stride};
  const uint64_t sstrides[2] = {(uint64_t)c->scale_head_stride, (uint64_t)c->scale_page_stride};
  const uint32_t box[4] = {(uint32_t)c->head_dim / 2, 1, (uint32_t)rows, 1}, sbox[3] = {(uint32_t)rows, 1, 1};
  const int sc = c->head_dim / 16;   // a row's scales are one element
  return encode_packed_map(&m->k, 1, 4, c->k, dims, strides, box) &&
         encode_packed_map(&m->v, 1, 4, c->v, dims, strides, box) &&
         encode_packed_map(&m->k_scale, sc, 3, c->k_scale, sdims, sstrides, sbox) &&
         encode_packed_map(&m->v_scale, sc, 3, c->v_scale, sdims, sstrides, sbox);
}

// And of K and V together, where their distance is one that a tensor map can hold.
bool encode_pair(PairMaps* m, const dflash_packed_cache* c, int rows) {
  const uint64_t heads = c->n_kv_heads, page = c->page_size, n_pages = c->n_pages;
  auto encode = [&](CUtensorMap* maps, int* pair, int* v_first, const void* k, const void* v, int element, uint32_t rank,
                    const uint64_t* dims, const uint64_t* strides, const uint32_t* box) {
    const long apart = static_cast<const char*>(v) - static_cast<const char*>(k);
    // (boxes of fewer than 128 bytes lie 128 apart, and so by themselves)
    *pair = apart != 0 && std::abs(apart) < (1L << 40) && (element == 1 || rows * element >= 128);
    *v_first = *pair && apart < 0;
    uint64_t st[4];
    std::copy(strides, strides + rank - 1, st);
    st[rank - 1] = (uint64_t)std::abs(apart);
    if (*pair) return encode_packed_map(maps, element, rank + 1, *v_first ? v : k, dims, st, box);
    return encode_packed_map(maps, element, rank, k, dims, st, box) &&
           encode_packed_map(maps + 1, element, rank, v, dims, st, box);
  };
  const uint64_t dims[5] = {(uint64_t)c->head_dim / 2, heads, page, n_pages, 2}, sdims[4] = {page, heads, n_pages, 2};
  const uint64_t strides[3] = {(uint64_t)c->head_stride, (uint64_t)c->row_stride, (uint64_t)c->page_stride};
  const uint64_t sstrides[2] = {(uint64_t)c->scale_head_stride, (uint64_t)c->scale_page_stride};
  const uint32_t box[5] = {(uint32_t)c->head_dim / 2, 1, (uint32_t)rows, 1, 2}, sbox[4] = {(uint32_t)rows, 1, 1, 2};
  return encode(m->codes, m->pair, m->v_first, c->k, c->v, 1, 4, dims, strides, box) &&
         encode(m->scales, m->pair + 1, m->v_first + 1, c->k_scale, c->v_scale, c->head_dim / 16, 3, sdims, sstrides,
                sbox);
}

bool encode_queries(CUtensorMap* m, const StepAttnArgs& a, const dflash_attention_args* p, int dtype) {
  const uint64_t dims[3] = {(uint64_t)a.d, (uint64_t)p->n_heads, (uint64_t)a.s.n_rows};
  const uint64_t strides[2] = {(uint64_t)a.d * 2, (uint64_t)p->q_stride * 2};
  const uint32_t box[3] = {64, (uint32_t)a.G, (uint32_t)a.tpt};
  return encode_tiled_map(m, dtype, 3, p->q, dims, strides, box);
}

}  // namespace

extern "C" {

int dflash_step_append(const dflash_paged_cache* cache, const dflash_step* step, const dflash_append_args* p,
                       void* stream) {
  return step_append(cache, step, p, false, stream);
}
int dflash_step_append_interleaved(const dflash_paged_cache* cache, const dflash_step* step,
                                   const dflash_append_args* p, void* stream) {
  return step_append(cache, step, p, true, stream);
}

int dflash_step_append_packed(const dflash_packed_cache* cache, const dflash_step* step,
                              const dflash_packed_append_args* p, void* stream) {
  report_error(DFLASH_OK, "");
  if (int rc = check_packed(cache)) return rc;
  const dflash_paged_cache shape = shape_of(cache);
  if (int rc = check_step(&shape, step)) return rc;
  if (!p) return invalid("args is null");
  if (int rc = check_append(&shape, step, &p->rows)) return rc;
  if (step->n_rows == 0) return DFLASH_OK;
  for (auto [ptr, stride] : {std::pair<const void*, long>{p->k_values, p->k_values_stride},
                             {p->v_values, p->v_values_stride}})
    if (ptr && !rows_ok(ptr, stride, (long)cache->n_kv_heads * cache->head_dim, 8))
      return invalid("rows must start on 16-byte boundaries and strides hold a row");
    else if (ptr && (ptr == p->rows.k || ptr == p->rows.v))   // (keys may be read again behind the first codes)
      return invalid("rounded rows go elsewhere than to k and v");
  Append4Args a{};
  if (int rc = append_args(a.a, &shape, step, &p->rows, p->interleaved != 0)) return rc;
  a.a.c = {cache->k, cache->v, cache->page_stride, cache->row_stride, cache->head_stride, cache->n_kv_heads,
           cache->head_dim};
  a.sc = {cache->k_scale, cache->v_scale, cache->scale_page_stride, cache->scale_row_stride,
          cache->scale_head_stride, cache->n_kv_heads, cache->head_dim};
  a.eps = p->rows.eps;
  a.mscale = p->rows.mscale;
  a.k_unit = cache->k_unit;
  a.v_unit = cache->v_unit;
  a.k_inv_unit = 1.f / cache->k_unit;
  a.v_inv_unit = 1.f / cache->v_unit;
  a.k_values = p->k_values;
  a.v_values = p->v_values;
  a.k_values_stride = p->k_values_stride;
  a.v_values_stride = p->v_values_stride;
  int n_sm = 0;
  if (int rc = sm_count(&n_sm)) return rc;
  return launched(launch_step_append4(a, p->rows.dtype, cache->dtype, n_sm, static_cast<cudaStream_t>(stream)),
                  "packed step append");
}

int dflash_step_attention_workspace(const dflash_paged_cache* cache, int32_t n_rows, int32_t n_heads, size_t* bytes) {
  report_error(DFLASH_OK, "");
  return attention_workspace(cache, n_rows, n_heads, bytes, false);
}

int dflash_step_attention(const dflash_paged_cache* cache, const dflash_step* step, const dflash_attention_args* p,
                          void* workspace, size_t workspace_bytes, void* stream) {
  report_error(DFLASH_OK, "");
  if (int rc = check_cache(cache)) return rc;
  if (int rc = check_step(cache, step)) return rc;
  if (int rc = check_attention(cache, step, p, workspace)) return rc;
  StepAttnArgs a{};
  if (int rc = attention_args(a, cache, step, p, false)) return rc;
  if (int rc = has_workspace(workspace_bytes, carve(a, static_cast<char*>(workspace)))) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (step->n_rows == 0) return launched(cudaMemsetAsync(a.status, 0, kStepStatusWords * 4, s), "step attention");
  CUtensorMap mq, mk, mv;
  const uint64_t cdims[4] = {(uint64_t)a.d, (uint64_t)cache->n_kv_heads, (uint64_t)cache->page_size,
                             (uint64_t)cache->n_pages};
  const uint64_t cstr[3] = {(uint64_t)cache->head_stride * 2, (uint64_t)cache->row_stride * 2,
                            (uint64_t)cache->page_stride * 2};
  const uint32_t cbox[4] = {64, 1, (uint32_t)a.box_rows, 1};
  if (!encode_queries(&mq, a, p, cache->dtype) ||
      !encode_tiled_map(&mk, cache->dtype, 4, cache->k, cdims, cstr, cbox) ||
      !encode_tiled_map(&mv, cache->dtype, 4, cache->v, cdims, cstr, cbox))
    return fail(DFLASH_ERR_CUDA, "tensor map of the queries or the cache was refused");
  return launched(launch_step_attention(a, mq, mk, mv, s), "step attention");
}

int dflash_step_attention_packed_workspace(const dflash_packed_cache* cache, int32_t n_rows, int32_t n_heads,
                                           size_t* bytes) {
  report_error(DFLASH_OK, "");
  if (int rc = check_packed_shape(cache)) return rc;
  const dflash_paged_cache shape = shape_of(cache);
  return attention_workspace(&shape, n_rows, n_heads, bytes, true);
}

int dflash_step_attention_packed(const dflash_packed_cache* cache, const dflash_step* step,
                                 const dflash_attention_args* p, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  report_error(DFLASH_OK, "");
  if (int rc = check_packed(cache)) return rc;
  const dflash_paged_cache shape = shape_of(cache);
  if (int rc = check_step(&shape, step)) return rc;
  if (int rc = check_attention(&shape, step, p, workspace)) return rc;
  StepAttnArgs a{};
  if (int rc = attention_args(a, &shape, step, p, true)) return rc;
  a.scale_log2 *= cache->k_unit;
  if (!std::isfinite(a.scale_log2) || a.scale_log2 < 1e-37f) return invalid("scale times the keys' unit must be a normal float");
  a.out_scale = cache->v_unit;
  a.q = p->q;
  a.q_stride = p->q_stride;
  if (int rc = has_workspace(workspace_bytes, carve(a, static_cast<char*>(workspace)))) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (step->n_rows == 0) return launched(cudaMemsetAsync(a.status, 0, kStepStatusWords * 4, s), "step attention");
  // Which kernels: where a sequence has few rows on average, the one for that, alone
  // where there is no prefix that many rows share (64 single tokens behind a prefix of 4096
  // 364 us without it); else the other one for all (with a launch more that finds
  // nothing to do, 8 ragged verifications 16 -> 25 us).  The mean sends a batch of both
  // kinds to one of them: 32 tokens (88 us) and a piece of 2048 rows (130) take 308 together.
  const long mean = ((long)step->n_rows * a.G + step->n_seq - 1) / step->n_seq;
  // (Among others few rows are one item a head, which the other kernel's bound on units
  // holds too; alone they may be more.)
  const bool some = a.n_cta > a.n_wide && mean <= kFewRows;
  a.few_rows = mean <= 8 && a.G <= 8 ? 8 : kFewRows;
  const bool alone = some && (step->prefix_len == 0 || (long)step->n_rows * a.G <= a.few_rows) && !a.by_cta &&
                     step_fits<FewCosts>(a, a.s.room());
  if (!some) a.n_cta = a.n_wide;
  CUtensorMap mq;
  PackedMaps m;
  PairMaps pair;
  if ((!alone && (!encode_queries(&mq, a, p, cache->dtype) || !encode_packed(&m, cache, a.box_rows))) ||
      (some && !encode_pair(&pair, cache, a.box_rows)))
    return fail(DFLASH_ERR_CUDA, "tensor map of the queries or the cache was refused");
  cudaError_t e = alone ? cudaSuccess : launch_step_attention4(a, mq, m, s);
  if (e == cudaSuccess && some) e = launch_step_attention_few(a, pair, !alone, s);
  if (e == cudaSuccess) e = launch_step_merge(a, s);
  return launched(e, "packed step attention");
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

int dflash_next_step(const dflash_next_step_args* p, void* stream) {
  report_error(DFLASH_OK, "");
  if (!p) return invalid("args is null");
  if (p->n_seq < 1 || p->n_seq > kMaxSeqs) return fail(DFLASH_ERR_INVALID_ARG, "n_seq must be 1..%d", kMaxSeqs);
  if (p->page_size < 16 || p->page_size > 256 || (p->page_size & (p->page_size - 1)))
    return fail(DFLASH_ERR_UNSUPPORTED, "page_size must be 16, 32, 64, 128 or 256");
  if (p->n_rows < 0 || p->n_rows > kMaxRows) return invalid("n_rows out of range");
  if (p->n_pages < 0 || p->table_cols < 0 || p->prefix_len < 0) return invalid("sizes must not be negative");
  if ((long)p->prefix_len + (long)p->table_cols * p->page_size >= (1L << 31) - 256)
    return invalid("more than 2^31 - 257 keys");
  if ((long)p->n_seq * p->table_cols >= (1L << 31)) return invalid("block table of 2^31 pages or more");
  if (p->n_seq > 1 && p->table_stride < p->table_cols) return invalid("the rows of the block table overlap");
  if (!p->kv_len || !p->row_start || !p->n_free || !p->rows || !p->kv_len_out || !p->row_start_out ||
      !p->n_free_out || !p->ticket || (p->table_cols > 0 && !p->block_table) || (p->n_pages > 0 && !p->free_pages))
    return invalid("null argument");
  NextArgs a{};
  a.n_seq = p->n_seq;
  a.page_shift = __builtin_ctz(p->page_size);
  a.table_cols = p->table_cols;
  a.n_pages = p->n_pages;
  a.n_rows = p->n_rows;
  a.prefix_len = p->prefix_len;
  a.table_stride = p->table_stride;
  a.kv_len = p->kv_len;
  a.row_start = p->row_start;
  a.n_free = p->n_free;
  a.rows = p->rows;
  a.n_accepted = p->n_accepted;
  a.keep = p->keep;
  a.block_table = p->block_table;
  a.free = p->free_pages;
  a.kv_len_out = p->kv_len_out;
  a.row_start_out = p->row_start_out;
  a.n_free_out = p->n_free_out;
  a.slots = reinterpret_cast<long long*>(p->slots);
  a.positions = p->positions;
  a.sequences = p->sequences;
  a.ticket = p->ticket;
  int n_sm = 0;
  if (int rc = sm_count(&n_sm)) return rc;
  return launched(launch_next_step(a, n_sm, static_cast<cudaStream_t>(stream)), "next step");
}

}  // extern "C"

// C ABI of the attention operators: argument checks and launches. Declared in include/engram.h.
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "attn.h"
#include "engram.h"
#include "kernels.h"
#include "strided.h"

namespace engram {

namespace {

int fail(int code, const char* fmt, ...) {
  char msg[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof(msg), fmt, ap);
  va_end(ap);
  return set_last_error(code, msg);
}

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

constexpr int32_t kMaxTokens = 1 << 24;     // attn_plan.cuh's sums stay in their types
constexpr int64_t kMaxPositions = 1 << 30;

int check_desc(const engram_attn_desc_t* d) {
  if (d == nullptr) return fail(ENGRAM_EINVAL, "desc is NULL");
  if (d->n_heads <= 0 || d->n_kv_heads <= 0 || d->n_heads % d->n_kv_heads != 0)
    return fail(ENGRAM_EINVAL, "n_heads must be a multiple of n_kv_heads, both > 0");
  if (d->head_dim <= 0) return fail(ENGRAM_EINVAL, "head_dim must be > 0");
  if (d->dtype != ENGRAM_BF16 && d->dtype != ENGRAM_F16)
    return fail(ENGRAM_EINVAL, "dtype must be ENGRAM_BF16 or ENGRAM_F16");
  if (!(d->scale > 0.f) || !std::isfinite(d->scale))
    return fail(ENGRAM_EINVAL, "scale must be finite and > 0");
  if (d->head_dim > 128 || d->head_dim % 8 != 0)
    return fail(ENGRAM_EUNSUPPORTED, "head_dim must be a multiple of 8 up to 128");
  if (d->n_heads / d->n_kv_heads > 128)
    return fail(ENGRAM_EUNSUPPORTED, "at most 128 query heads per key-value head");
  return ENGRAM_OK;
}

// Tensor maps take strides below 2^40 bytes; a tensor that reaches further than an address does not
// exist, and would overflow the sums of strided.h.
bool good_stride(int64_t n, int64_t stride) {
  return n <= 1 || (stride > 0 && stride % 8 == 0 && stride < (int64_t(1) << 38) &&
                    stride <= (int64_t(1) << 56) / (n - 1));
}

int check_view(const engram_attn_view_t* t, const char* name, int32_t tokens, int32_t heads) {
  if (t == nullptr || t->ptr == nullptr) return fail(ENGRAM_EINVAL, "%s is NULL", name);
  if (!aligned(t->ptr, 16)) return fail(ENGRAM_EINVAL, "%s must be 16-byte aligned", name);
  if (!good_stride(tokens, t->token_stride) || !good_stride(heads, t->head_stride))
    return fail(ENGRAM_EINVAL, "%s: strides must be multiples of 8 elements, > 0", name);
  return ENGRAM_OK;
}

int check_tokens(const int32_t* cu, int32_t n_seqs, int32_t total) {
  if (n_seqs < 0 || total < 0) return fail(ENGRAM_EINVAL, "n_seqs and total must be >= 0");
  if (total >= kMaxTokens || n_seqs >= kMaxTokens)
    return fail(ENGRAM_EUNSUPPORTED, "n_seqs and total must be below 2^24");
  if (n_seqs == 0 || total == 0) return ENGRAM_OK;
  if (cu == nullptr || !aligned(cu, 4))
    return fail(ENGRAM_EINVAL, "cu_seqlens must be a 4-byte aligned array");
  return ENGRAM_OK;
}

int check_cache(const engram_attn_desc_t* d, const engram_kv_cache_t* c, const int32_t* kv_len) {
  if (c == nullptr) return fail(ENGRAM_EINVAL, "cache is NULL");
  if (!c->k || !c->v || !c->block_table || !kv_len)
    return fail(ENGRAM_EINVAL, "cache, block_table or kv_len is NULL");
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->block_table, 4) ||
      !aligned(kv_len, 4))
    return fail(ENGRAM_EINVAL, "the cache must be 16-byte aligned, int32 arrays 4-byte aligned");
  if (c->n_pages <= 0 || c->table_width <= 0 || c->page_size <= 0)
    return fail(ENGRAM_EINVAL, "n_pages, page_size and table_width must be > 0");
  if (c->page_size % 8 != 0) return fail(ENGRAM_EUNSUPPORTED, "page_size must be a multiple of 8");
  if (int64_t(c->table_width) * c->page_size >= kMaxPositions)
    return fail(ENGRAM_EUNSUPPORTED, "a sequence may have fewer than 2^30 positions");
  if (!good_stride(c->n_pages, c->k_page_stride) || !good_stride(c->page_size, c->k_slot_stride) ||
      !good_stride(d->n_kv_heads, c->k_head_stride) || !good_stride(c->n_pages, c->v_page_stride) ||
      !good_stride(c->page_size, c->v_slot_stride) || !good_stride(d->n_kv_heads, c->v_head_stride))
    return fail(ENGRAM_EINVAL, "cache: strides must be multiples of 8 elements, > 0");
  return ENGRAM_OK;
}

Strided strided(const engram_attn_view_t* t, int32_t tokens, int32_t heads, int32_t dim) {
  return Strided(t->ptr, int64_t(dim) * 2, tokens, t->token_stride * 2, heads, t->head_stride * 2);
}

Strided strided_keys(const engram_attn_desc_t* d, const engram_kv_cache_t* c) {
  return Strided(c->k, int64_t(d->head_dim) * 2, c->n_pages, c->k_page_stride * 2, c->page_size,
                 c->k_slot_stride * 2, d->n_kv_heads, c->k_head_stride * 2);
}
Strided strided_values(const engram_attn_desc_t* d, const engram_kv_cache_t* c) {
  return Strided(c->v, int64_t(d->head_dim) * 2, c->n_pages, c->v_page_stride * 2, c->page_size,
                 c->v_slot_stride * 2, d->n_kv_heads, c->v_head_stride * 2);
}

// What a call reads and writes, by name. Parts of one buffer may interleave (a projection's q, k and v,
// and an output beside them); what is written may share no byte with anything else, nor two rows of it
// with each other.
struct Operand {
  const char* name;
  Strided at;
};

int check_overlap(const Operand* written, int n_written, const Operand* read, int n_read) {
  for (int i = 0; i < n_written; ++i) {
    const Operand& w = written[i];
    for (int j = 0; j < n_read; ++j)
      if (shares_memory(w.at, read[j].at))
        return fail(ENGRAM_EINVAL, "%s overlaps %s", w.name, read[j].name);
    for (int j = 0; j < i; ++j)
      if (shares_memory(w.at, written[j].at))
        return fail(ENGRAM_EINVAL, "%s overlaps %s", w.name, written[j].name);
    if (rows_share_memory(w.at))
      return fail(ENGRAM_EINVAL, "%s: its rows overlap each other", w.name);
  }
  return ENGRAM_OK;
}

// out, the workspace and lse (of no width where it is NULL) against `read`.
template <int N>
int check_written(const engram_attn_desc_t* d, const engram_attn_view_t* out, int32_t total,
                  const float* lse, const void* workspace, const Operand (&read)[N]) {
  const Operand written[] = {
      {"out", strided(out, total, d->n_heads, d->head_dim)},
      {"workspace", Strided(workspace, static_cast<int64_t>(engram_attn_workspace_size(d)))},
      {"lse", Strided(lse, lse ? int64_t(total) * d->n_heads * 4 : 0)}};
  return check_overlap(written, 3, read, N);
}

int check_workspace(const engram_attn_desc_t* d, void* ws, size_t bytes, const float* lse) {
  if (ws == nullptr || !aligned(ws, 256))
    return fail(ENGRAM_EINVAL, "workspace must be 256-byte aligned");
  if (bytes < engram_attn_workspace_size(d))
    return fail(ENGRAM_EINVAL, "workspace too small: %zu bytes, engram_attn_workspace_size is %zu",
                bytes, engram_attn_workspace_size(d));
  if (!aligned(lse, 4)) return fail(ENGRAM_EINVAL, "lse must be 4-byte aligned");
  return ENGRAM_OK;
}

AttnArgs make_args(const engram_attn_desc_t* d, const engram_attn_view_t* q,
                   const engram_attn_view_t* out, float* lse, const int32_t* cu, int32_t n_seqs,
                   int32_t total, void* workspace, uint32_t* err) {
  AttnArgs a{};
  a.plan.cu = cu;
  a.plan.n_seqs = n_seqs;
  a.plan.total = total;
  a.plan.kv_heads = d->n_kv_heads;
  a.bf16 = d->dtype == ENGRAM_BF16;
  a.heads = d->n_heads;
  a.group = d->n_heads / d->n_kv_heads;
  a.head_dim = d->head_dim;
  a.scale_log2 = d->scale * 1.4426950408889634f;
  a.q = static_cast<const uint16_t*>(q->ptr);
  a.q_token = q->token_stride;
  a.q_head = q->head_stride;
  a.out = static_cast<uint16_t*>(const_cast<void*>(out->ptr));
  a.o_token = out->token_stride;
  a.o_head = out->head_stride;
  a.lse = lse;
  a.workspace = workspace;
  a.err = err;
  return a;
}

// Keys per copy of a paged tile: the largest power of two that divides the page, so that a copy
// never crosses a page and a tile is a whole number of copies.
int32_t granule_of(int32_t page_size) {
  const int32_t g = page_size & -page_size;
  return g < kTileKeys ? g : kTileKeys;
}

int report(cudaError_t e, const char* who) {
  if (e == cudaSuccess) return ENGRAM_OK;
  return fail(ENGRAM_ECUDA, "%s: %s", who, cudaGetErrorString(e));
}

}  // namespace

}  // namespace engram

using namespace engram;

extern "C" {

ENGRAM_API size_t engram_attn_workspace_size(const engram_attn_desc_t* desc) {
  if (check_desc(desc) != ENGRAM_OK) return 0;
  return attn_pieces_bytes(device_sm_count(), kAttnItemRows, attn_width(desc->head_dim));
}

ENGRAM_API int engram_attn_prompt(const engram_attn_desc_t* desc, const engram_attn_view_t* q,
                                  const engram_attn_view_t* k, const engram_attn_view_t* v,
                                  const int32_t* cu_seqlens, int32_t n_seqs, int32_t total,
                                  const engram_attn_view_t* out, float* lse, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  set_last_error(ENGRAM_OK, "");
  int rc = check_desc(desc);
  if (rc) return rc;
  if ((rc = check_tokens(cu_seqlens, n_seqs, total)) != 0) return rc;
  if (n_seqs == 0 || total == 0) return ENGRAM_OK;
  if ((rc = check_view(q, "q", total, desc->n_heads)) != 0 ||
      (rc = check_view(k, "k", total, desc->n_kv_heads)) != 0 ||
      (rc = check_view(v, "v", total, desc->n_kv_heads)) != 0 ||
      (rc = check_view(out, "out", total, desc->n_heads)) != 0 ||
      (rc = check_workspace(desc, workspace, workspace_bytes, lse)) != 0)
    return rc;
  const Operand read[] = {{"q", strided(q, total, desc->n_heads, desc->head_dim)},
                          {"k", strided(k, total, desc->n_kv_heads, desc->head_dim)},
                          {"v", strided(v, total, desc->n_kv_heads, desc->head_dim)},
                          {"cu_seqlens", Strided(cu_seqlens, (int64_t(n_seqs) + 1) * 4)}};
  if ((rc = check_written(desc, out, total, lse, workspace, read)) != 0) return rc;
  cudaError_t e;
  uint32_t* err = device_error_word(&e);
  if (!err) return report(e, "engram_attn_prompt");
  AttnArgs a = make_args(desc, q, out, lse, cu_seqlens, n_seqs, total, workspace, err);
  a.k = static_cast<const uint16_t*>(k->ptr);
  a.v = static_cast<const uint16_t*>(v->ptr);
  a.k_token = k->token_stride;
  a.k_head = k->head_stride;
  a.v_token = v->token_stride;
  a.v_head = v->head_stride;
  a.granule = kTileKeys;
  return report(launch_attn_tiles(a, static_cast<cudaStream_t>(stream)), "engram_attn_prompt");
}

ENGRAM_API int engram_attn_paged(const engram_attn_desc_t* desc, const engram_attn_view_t* q,
                                 const int32_t* cu_seqlens, int32_t n_seqs, int32_t total,
                                 int32_t max_q, const int32_t* kv_len,
                                 const engram_kv_cache_t* cache, const engram_attn_view_t* out,
                                 float* lse, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  set_last_error(ENGRAM_OK, "");
  int rc = check_desc(desc);
  if (rc) return rc;
  if ((rc = check_tokens(cu_seqlens, n_seqs, total)) != 0) return rc;
  if (max_q < 0) return fail(ENGRAM_EINVAL, "max_q must be >= 0");
  if (n_seqs == 0 || total == 0) return ENGRAM_OK;
  if ((rc = check_view(q, "q", total, desc->n_heads)) != 0 ||
      (rc = check_view(out, "out", total, desc->n_heads)) != 0 ||
      (rc = check_cache(desc, cache, kv_len)) != 0 ||
      (rc = check_workspace(desc, workspace, workspace_bytes, lse)) != 0)
    return rc;
  const Operand read[] = {
      {"q", strided(q, total, desc->n_heads, desc->head_dim)},
      {"the cache", strided_keys(desc, cache)},
      {"the cache", strided_values(desc, cache)},
      {"cu_seqlens", Strided(cu_seqlens, (int64_t(n_seqs) + 1) * 4)},
      {"kv_len", Strided(kv_len, int64_t(n_seqs) * 4)},
      {"block_table", Strided(cache->block_table, int64_t(n_seqs) * cache->table_width * 4)}};
  if ((rc = check_written(desc, out, total, lse, workspace, read)) != 0) return rc;
  cudaError_t e;
  uint32_t* err = device_error_word(&e);
  if (!err) return report(e, "engram_attn_paged");
  AttnArgs a = make_args(desc, q, out, lse, cu_seqlens, n_seqs, total, workspace, err);
  a.plan.kv_len = kv_len;
  a.plan.kv_cap = cache->table_width * cache->page_size;
  a.k = static_cast<const uint16_t*>(cache->k);
  a.v = static_cast<const uint16_t*>(cache->v);
  a.k_page = cache->k_page_stride;
  a.k_token = cache->k_slot_stride;
  a.k_head = cache->k_head_stride;
  a.v_page = cache->v_page_stride;
  a.v_token = cache->v_slot_stride;
  a.v_head = cache->v_head_stride;
  a.table = cache->block_table;
  a.table_width = cache->table_width;
  a.page_size = cache->page_size;
  a.n_pages = cache->n_pages;
  a.granule = granule_of(cache->page_size);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int64_t rows = int64_t(max_q > 1 ? max_q : 1) * a.group;
  return report(rows <= kAttnFewRows ? launch_attn_rows(a, static_cast<int32_t>(rows), st)
                                     : launch_attn_tiles(a, st),
                "engram_attn_paged");
}

ENGRAM_API int engram_kv_append(const engram_attn_desc_t* desc, const engram_attn_view_t* k,
                                const engram_attn_view_t* v, const int32_t* cu_seqlens,
                                int32_t n_seqs, int32_t total, const int32_t* kv_len,
                                const engram_kv_cache_t* cache, void* stream) {
  set_last_error(ENGRAM_OK, "");
  int rc = check_desc(desc);
  if (rc) return rc;
  if ((rc = check_tokens(cu_seqlens, n_seqs, total)) != 0) return rc;
  if (n_seqs == 0 || total == 0) return ENGRAM_OK;
  if ((rc = check_view(k, "k", total, desc->n_kv_heads)) != 0 ||
      (rc = check_view(v, "v", total, desc->n_kv_heads)) != 0 ||
      (rc = check_cache(desc, cache, kv_len)) != 0)
    return rc;
  cudaError_t e;
  uint32_t* err = device_error_word(&e);
  if (!err) return report(e, "engram_kv_append");
  KvAppendArgs a{};
  a.cu = cu_seqlens;
  a.kv_len = kv_len;
  a.table = cache->block_table;
  a.n_seqs = n_seqs;
  a.total = total;
  a.table_width = cache->table_width;
  a.page_size = cache->page_size;
  a.n_pages = cache->n_pages;
  a.kv_heads = desc->n_kv_heads;
  a.head_dim = desc->head_dim;
  a.k = static_cast<const uint16_t*>(k->ptr);
  a.v = static_cast<const uint16_t*>(v->ptr);
  a.k_token = k->token_stride;
  a.k_head = k->head_stride;
  a.v_token = v->token_stride;
  a.v_head = v->head_stride;
  a.k_cache = static_cast<uint16_t*>(const_cast<void*>(cache->k));
  a.v_cache = static_cast<uint16_t*>(const_cast<void*>(cache->v));
  a.k_page = cache->k_page_stride;
  a.k_slot = cache->k_slot_stride;
  a.k_chead = cache->k_head_stride;
  a.v_page = cache->v_page_stride;
  a.v_slot = cache->v_slot_stride;
  a.v_chead = cache->v_head_stride;
  a.err = err;
  return report(launch_kv_append(a, static_cast<cudaStream_t>(stream)), "engram_kv_append");
}

}  // extern "C"

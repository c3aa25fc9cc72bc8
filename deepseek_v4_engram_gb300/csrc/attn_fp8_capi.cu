// C ABI of the operators on an 8-bit cache: argument checks and launches. Declared in include/engram.h.
#include "attn_checks.h"
#include "kv_fp8.h"

namespace engram {

namespace {

int check_fp8_desc(const engram_attn_desc_t* d) {
  const int rc = check_desc(d);
  if (rc) return rc;
  if (d->head_dim % 16 != 0) return fail(ENGRAM_EUNSUPPORTED, "an fp8 cache has a head_dim that is a multiple of 16");
  return ENGRAM_OK;
}

// Strides in bytes: copies move 16 of them at a time.
bool good_bytes(int64_t n, int64_t stride) {
  return n <= 1 || (stride > 0 && stride % 16 == 0 && stride < (int64_t(1) << 39) &&
                    stride <= (int64_t(1) << 56) / (n - 1));
}

int check_fp8_cache(const engram_attn_desc_t* d, const engram_kv_cache_fp8_t* c, const int32_t* kv_len) {
  if (c == nullptr) return fail(ENGRAM_EINVAL, "cache is NULL");
  if (!c->k || !c->v || !c->k_scale || !c->v_scale || !c->block_table || !kv_len)
    return fail(ENGRAM_EINVAL, "cache, scales, block_table or kv_len is NULL");
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 16) || !aligned(c->v_scale, 16) ||
      !aligned(c->block_table, 4) || !aligned(kv_len, 4))
    return fail(ENGRAM_EINVAL, "the cache must be 16-byte aligned, int32 arrays 4-byte aligned");
  if (c->n_pages <= 0 || c->table_width <= 0 || c->page_size <= 0)
    return fail(ENGRAM_EINVAL, "n_pages, page_size and table_width must be > 0");
  if (c->page_size % 16 != 0)
    return fail(ENGRAM_EUNSUPPORTED, "an fp8 cache has a page_size that is a multiple of 16");
  if (int64_t(c->table_width) * c->page_size >= kMaxPositions)
    return fail(ENGRAM_EUNSUPPORTED, "a sequence may have fewer than 2^30 positions");
  if (!good_bytes(c->n_pages, c->k_page_stride) || !good_bytes(c->page_size, c->k_slot_stride) ||
      !good_bytes(d->n_kv_heads, c->k_head_stride) || !good_bytes(c->n_pages, c->v_page_stride) ||
      !good_bytes(c->page_size, c->v_slot_stride) || !good_bytes(d->n_kv_heads, c->v_head_stride) ||
      !good_bytes(c->n_pages, c->k_scale_page_stride) || !good_bytes(d->n_kv_heads, c->k_scale_head_stride) ||
      !good_bytes(c->n_pages, c->v_scale_page_stride) || !good_bytes(d->n_kv_heads, c->v_scale_head_stride))
    return fail(ENGRAM_EINVAL, "cache: strides must be multiples of 16 bytes, > 0");
  return ENGRAM_OK;
}

Strided strided_codes(const engram_attn_desc_t* d, const engram_kv_cache_fp8_t* c, bool v) {
  return Strided(v ? c->v : c->k, d->head_dim, c->n_pages, v ? c->v_page_stride : c->k_page_stride, c->page_size,
                 v ? c->v_slot_stride : c->k_slot_stride, d->n_kv_heads, v ? c->v_head_stride : c->k_head_stride);
}
Strided strided_scales(const engram_attn_desc_t* d, const engram_kv_cache_fp8_t* c, bool v) {
  return Strided(v ? c->v_scale : c->k_scale, c->page_size, c->n_pages,
                 v ? c->v_scale_page_stride : c->k_scale_page_stride, d->n_kv_heads,
                 v ? c->v_scale_head_stride : c->k_scale_head_stride);
}

KvFp8Part part(const engram_kv_cache_fp8_t* c, bool v) {
  KvFp8Part p{};
  p.codes = static_cast<uint8_t*>(const_cast<void*>(v ? c->v : c->k));
  p.scales = static_cast<uint8_t*>(const_cast<void*>(v ? c->v_scale : c->k_scale));
  p.page = v ? c->v_page_stride : c->k_page_stride;
  p.slot = v ? c->v_slot_stride : c->k_slot_stride;
  p.head = v ? c->v_head_stride : c->k_head_stride;
  p.scale_page = v ? c->v_scale_page_stride : c->k_scale_page_stride;
  p.scale_head = v ? c->v_scale_head_stride : c->k_scale_head_stride;
  return p;
}

// What append and read have in common: `k` and `v` are the 16-bit side, `reading` whether they are written.
int move(const engram_attn_desc_t* desc, const engram_attn_view_t* k, const engram_attn_view_t* v,
         const int32_t* cu_seqlens, int32_t n_seqs, int32_t total, const int32_t* kv_len,
         const engram_kv_cache_fp8_t* cache, void* stream, bool reading) {
  set_last_error(ENGRAM_OK, "");
  int rc = check_fp8_desc(desc);
  if (rc) return rc;
  if ((rc = check_tokens(cu_seqlens, n_seqs, total)) != 0) return rc;
  if (n_seqs == 0 || total == 0) return ENGRAM_OK;
  const char* names[2] = {reading ? "k_out" : "k", reading ? "v_out" : "v"};
  if ((rc = check_view(k, names[0], total, desc->n_kv_heads)) != 0 ||
      (rc = check_view(v, names[1], total, desc->n_kv_heads)) != 0 ||
      (rc = check_fp8_cache(desc, cache, kv_len)) != 0)
    return rc;
  const Operand rows[2] = {{names[0], strided(k, total, desc->n_kv_heads, desc->head_dim)},
                           {names[1], strided(v, total, desc->n_kv_heads, desc->head_dim)}};
  const Operand pages[4] = {{"the cache", strided_codes(desc, cache, false)},
                            {"the cache", strided_codes(desc, cache, true)},
                            {"the cache's scales", strided_scales(desc, cache, false)},
                            {"the cache's scales", strided_scales(desc, cache, true)}};
  const Operand lists[3] = {
      {"cu_seqlens", Strided(cu_seqlens, (int64_t(n_seqs) + 1) * 4)},
      {"kv_len", Strided(kv_len, int64_t(n_seqs) * 4)},
      {"block_table", Strided(cache->block_table, int64_t(n_seqs) * cache->table_width * 4)}};
  const Operand* written = reading ? rows : pages;
  const Operand* read = reading ? pages : rows;
  if ((rc = check_overlap(written, reading ? 2 : 4, read, reading ? 4 : 2)) != 0 ||
      (rc = check_overlap(written, reading ? 2 : 4, lists, 3)) != 0)
    return rc;
  const char* who = reading ? "engram_kv_read_fp8" : "engram_kv_append_fp8";
  cudaError_t e;
  uint32_t* err = device_error_word(&e);
  if (!err) return report(e, who);
  KvFp8Args a{};
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
  a.bf16 = desc->dtype == ENGRAM_BF16;
  a.k = part(cache, false);
  a.v = part(cache, true);
  a.k16 = static_cast<uint16_t*>(const_cast<void*>(k->ptr));
  a.v16 = static_cast<uint16_t*>(const_cast<void*>(v->ptr));
  a.k_token = k->token_stride;
  a.k_head = k->head_stride;
  a.v_token = v->token_stride;
  a.v_head = v->head_stride;
  a.err = err;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return report(reading ? launch_kv_read_fp8(a, st) : launch_kv_append_fp8(a, st), who);
}

}  // namespace

}  // namespace engram

using namespace engram;

extern "C" {

ENGRAM_API int engram_kv_append_fp8(const engram_attn_desc_t* desc, const engram_attn_view_t* k,
                                    const engram_attn_view_t* v, const int32_t* cu_seqlens, int32_t n_seqs,
                                    int32_t total, const int32_t* kv_len, const engram_kv_cache_fp8_t* cache,
                                    void* stream) {
  return move(desc, k, v, cu_seqlens, n_seqs, total, kv_len, cache, stream, false);
}

ENGRAM_API int engram_kv_read_fp8(const engram_attn_desc_t* desc, const int32_t* cu_seqlens, int32_t n_seqs,
                                  int32_t total, const int32_t* kv_len, const engram_kv_cache_fp8_t* cache,
                                  const engram_attn_view_t* k_out, const engram_attn_view_t* v_out, void* stream) {
  return move(desc, k_out, v_out, cu_seqlens, n_seqs, total, kv_len, cache, stream, true);
}

ENGRAM_API int engram_attn_paged_fp8(const engram_attn_desc_t* desc, const engram_attn_view_t* q,
                                     const int32_t* cu_seqlens, int32_t n_seqs, int32_t total, int32_t max_q,
                                     const int32_t* kv_len, const engram_kv_cache_fp8_t* cache,
                                     const engram_attn_view_t* out, float* lse, void* workspace,
                                     size_t workspace_bytes, void* stream) {
  set_last_error(ENGRAM_OK, "");
  int rc = check_fp8_desc(desc);
  if (rc) return rc;
  if ((rc = check_tokens(cu_seqlens, n_seqs, total)) != 0) return rc;
  if (max_q < 0) return fail(ENGRAM_EINVAL, "max_q must be >= 0");
  if (n_seqs == 0 || total == 0) return ENGRAM_OK;
  if ((rc = check_view(q, "q", total, desc->n_heads)) != 0 ||
      (rc = check_view(out, "out", total, desc->n_heads)) != 0 ||
      (rc = check_fp8_cache(desc, cache, kv_len)) != 0 ||
      (rc = check_workspace(desc, workspace, workspace_bytes, lse)) != 0)
    return rc;
  const Operand read[] = {
      {"q", strided(q, total, desc->n_heads, desc->head_dim)},
      {"the cache", strided_codes(desc, cache, false)},
      {"the cache", strided_codes(desc, cache, true)},
      {"the cache's scales", strided_scales(desc, cache, false)},
      {"the cache's scales", strided_scales(desc, cache, true)},
      {"cu_seqlens", Strided(cu_seqlens, (int64_t(n_seqs) + 1) * 4)},
      {"kv_len", Strided(kv_len, int64_t(n_seqs) * 4)},
      {"block_table", Strided(cache->block_table, int64_t(n_seqs) * cache->table_width * 4)}};
  if ((rc = check_written(desc, out, total, lse, workspace, read)) != 0) return rc;
  cudaError_t e;
  uint32_t* err = device_error_word(&e);
  if (!err) return report(e, "engram_attn_paged_fp8");
  AttnArgs a = make_args(desc, q, out, lse, cu_seqlens, n_seqs, total, workspace, err);
  a.plan.kv_len = kv_len;
  a.plan.kv_cap = cache->table_width * cache->page_size;
  a.table = cache->block_table;
  a.table_width = cache->table_width;
  a.page_size = cache->page_size;
  a.n_pages = cache->n_pages;
  a.granule = granule_of(cache->page_size);
  const int64_t rows = int64_t(max_q > 1 ? max_q : 1) * a.group;
  const KvFp8Part k = part(cache, false), v = part(cache, true);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool few = rows <= attn_fp8_few_rows(desc->head_dim);
  return report(few ? launch_attn_fp8_rows(a, k, v, static_cast<int32_t>(rows), st) : launch_attn_fp8_tiles(a, k, v, st),
                "engram_attn_paged_fp8");
}

}  // extern "C"

// C ABI of the attention operators: argument checks and launches. Declared in include/engram.h.
#include "attn_checks.h"

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

// A paged cache in eight bits: what the C ABI (attn_fp8_capi.cu) hands to the kernels. Host-only
// launch declarations; pointers are device pointers already validated.
#pragma once

#include "attn.h"

namespace engram {

// Codes [pages, page_size, heads, D] and scales [pages, heads, page_size] of the keys or the values,
// with the byte strides of a page, a slot and a head.
struct KvFp8Part {
  uint8_t* codes;
  uint8_t* scales;
  int64_t page, slot, head;
  int64_t scale_page, scale_head;
};

struct KvFp8Args {
  const int32_t* cu;
  const int32_t* kv_len;
  const int32_t* table;
  int32_t n_seqs, total, table_width, page_size, n_pages, kv_heads, head_dim;
  bool bf16;                 // else f16
  KvFp8Part k, v;
  uint16_t* k16;             // the 16-bit side: element strides of a token and of a head follow
  uint16_t* v16;
  int64_t k_token, k_head, v_token, v_head;
  uint32_t* err;
};
cudaError_t launch_kv_append_fp8(const KvFp8Args& a, cudaStream_t st);   // 16 bits to the pages
cudaError_t launch_kv_read_fp8(const KvFp8Args& a, cudaStream_t st);     // the pages to 16 bits

// Attention over such a cache, `a` as for a paged cache of 16 bits, but for its keys and values.
// Items of up to attn_fp8_few_rows rows (attn_fp8_rows_sm103.cu); `rows`: of the longest chunk, at least
// the heads that share a key-value head.
constexpr int32_t attn_fp8_few_rows(int32_t head_dim) { return attn_width(head_dim) == 64 ? 64 : 48; }
cudaError_t launch_attn_fp8_rows(const AttnArgs& a, const KvFp8Part& k, const KvFp8Part& v, int32_t rows,
                                 cudaStream_t st);

// Items of up to 256 rows (attn_fp8_tiles_sm103.cu).
cudaError_t launch_attn_fp8_tiles(const AttnArgs& a, const KvFp8Part& k, const KvFp8Part& v, cudaStream_t st);

// Tensor map (capi.cu) of an 8-bit cache's codes, element (d, head, slot, page) in boxes of `width` (64 or 128)
// columns by `box_heads` heads by `granule` slots with the swizzle of that width; columns past `dim` read as
// zero.
bool tensor_map_fp8_codes(void* map_out, const KvFp8Part& p, int32_t dim, int32_t heads, int32_t page_size,
                          int32_t n_pages, int32_t width, int32_t box_heads, int32_t granule);

// Those of the keys and the values, for items of `item_heads` heads (1 or 2), of which the call has
// a.plan.kv_heads. Two heads of 64 columns are one of 128: they have to lie beside each other.
inline bool attn_fp8_tensor_maps(const AttnArgs& a, const KvFp8Part& k, const KvFp8Part& v, int32_t item_heads,
                                 CUtensorMap (&tm)[2]) {
  const int32_t width = attn_width(a.head_dim);
  const bool merged = item_heads == 2 && width == 64;
  for (int i = 0; i < 2; ++i) {
    KvFp8Part p = i == 0 ? k : v;
    if (merged) p.head *= 2;
    if (!tensor_map_fp8_codes(&tm[i], p, merged ? 128 : a.head_dim,
                              merged ? a.plan.kv_heads : a.plan.kv_heads * item_heads, a.page_size, a.n_pages,
                              merged ? 128 : width, merged ? 1 : item_heads, a.granule))
      return false;
  }
  return true;
}

}  // namespace engram

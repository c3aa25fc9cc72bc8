// Attention over packed prompts and over a paged cache: what the C ABI (attn_capi.cu) hands to the
// kernels. Host-only launch declarations; pointers are device pointers already validated.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "attn_plan.cuh"

namespace engram {

struct AttnArgs {
  AttnPlan plan;             // tokens, workers and extra are the launcher's
  bool bf16;                 // else f16
  int32_t heads;             // query heads
  int32_t group;             // query heads per key-value head
  int32_t head_dim;
  float scale_log2;          // softmax scale * log2(e): scores go straight to exp2
  const uint16_t* q;         // element strides of a token and of a head follow each pointer
  int64_t q_token, q_head;
  uint16_t* out;
  int64_t o_token, o_head;
  float* lse;                // [total, heads] or null
  const uint16_t* k;         // packed: [total, kv_heads, D]; paged: [pages, page_size, kv_heads, D]
  const uint16_t* v;
  int64_t k_token, k_head, v_token, v_head;
  int64_t k_page, v_page;    // paged only
  const int32_t* table;      // [n_seqs, table_width], null: packed
  int32_t table_width, page_size, n_pages;
  int32_t granule;           // keys per copy: a power of two that divides page_size; 128 if packed
  void* workspace;
  uint32_t* err;
};

// The pieces of cut items. A worker continues at most one item that another began and begins at
// most one that another ends: for each of the two, in this order, it has an AttnMeta and a slot of
// `rows` rows.
struct AttnMeta {
  int32_t token0, ntok, h;
  int32_t pieces;            // of workers owner, owner + 1, ...; 0: the worker has no such item
  int32_t owner;             // the worker that begins it
  int32_t unused[3];
};
struct AttnPieces {
  AttnMeta* meta;            // [workers * 2]
  float* ml;                 // [workers * 2, rows, 2]: base of the exponentials (log2) and their sum
  float* o;                  // [workers * 2, rows, width]: sum of 2^(x - base) v
};

constexpr size_t attn_round256(size_t n) { return (n + 255) & ~size_t(255); }

inline size_t attn_pieces_bytes(int32_t workers, int32_t rows, int32_t width) {
  return attn_round256(size_t(workers) * 2 * sizeof(AttnMeta)) +
         attn_round256(size_t(workers) * 2 * rows * 2 * 4) + size_t(workers) * 2 * rows * width * 4;
}

inline AttnPieces attn_pieces_at(void* workspace, int32_t workers, int32_t rows) {
  uint8_t* p = static_cast<uint8_t*>(workspace);
  AttnPieces r;
  r.meta = reinterpret_cast<AttnMeta*>(p);
  p += attn_round256(size_t(workers) * 2 * sizeof(AttnMeta));
  r.ml = reinterpret_cast<float*>(p);
  p += attn_round256(size_t(workers) * 2 * rows * 2 * 4);
  r.o = reinterpret_cast<float*>(p);
  return r;
}

// Width of a row in the kernels: 64 or 128 columns, those past head_dim zero.
constexpr int32_t attn_width(int32_t head_dim) { return head_dim <= 64 ? 64 : 128; }

// Items of up to kAttnFewRows rows (attn_rows_sm103.cu): decoding and short chunks. `rows`: of the
// longest chunk, at least the heads that share a key-value head. Over 16 caches of 3000-4665
// positions in pages of 48, 4 key-value heads of 128: 8 rows 32.0 us, 24 rows 36.3 us (on tcgen05
// 39.0), 32 rows 37.2 us (38.9); 40 rows take 38.5 us on tcgen05 and took 49.5 in a form for 64 rows
// made like these.
constexpr int32_t kAttnFewRows = 32;
cudaError_t launch_attn_rows(const AttnArgs& a, int32_t rows, cudaStream_t st);

// Items of up to 256 rows on tcgen05 (attn_tiles_sm103.cu): prompts and long chunks.
constexpr int32_t kAttnItemRows = 256;
cudaError_t launch_attn_tiles(const AttnArgs& a, cudaStream_t st);

// Joins the pieces of items of `rows` rows.
cudaError_t launch_attn_combine(const AttnArgs& a, int32_t rows, cudaStream_t st);

struct KvAppendArgs {
  const int32_t* cu;
  const int32_t* kv_len;
  const int32_t* table;
  int32_t n_seqs, total, table_width, page_size, n_pages, kv_heads, head_dim;
  const uint16_t* k;
  const uint16_t* v;
  int64_t k_token, k_head, v_token, v_head;
  uint16_t* k_cache;
  uint16_t* v_cache;
  int64_t k_page, k_slot, k_chead, v_page, v_slot, v_chead;
  uint32_t* err;
};
cudaError_t launch_kv_append(const KvAppendArgs& a, cudaStream_t st);

// Device address of the current device's error word (capi.cu), or null with the reason in *e.
uint32_t* device_error_word(cudaError_t* e);

// Tensor map of queries, keys or values (capi.cu): element (d, head, token, page) of a 16-bit tensor
// with the given strides in elements, boxes of 64 columns of `box_heads` heads by `box_tokens`
// tokens, with the 128-byte swizzle; columns past `dim` read as zero.
bool tensor_map_attn(void* map_out, const void* base, bool bf16, uint64_t dim, uint64_t heads,
                     uint64_t tokens, uint64_t pages, int64_t head_stride, int64_t token_stride,
                     int64_t page_stride, uint32_t box_heads, uint32_t box_tokens);

// The tensor maps of a call's keys and values.
inline bool attn_tensor_maps(const AttnArgs& a, void* k_map, void* v_map) {
  const bool paged = a.table != nullptr;
  const uint64_t tokens = paged ? a.page_size : a.plan.total, pages = paged ? a.n_pages : 1;
  return tensor_map_attn(k_map, a.k, a.bf16, a.head_dim, a.plan.kv_heads, tokens, pages, a.k_head,
                         a.k_token, a.k_page, 1, a.granule) &&
         tensor_map_attn(v_map, a.v, a.bf16, a.head_dim, a.plan.kv_heads, tokens, pages, a.v_head,
                         a.v_token, a.v_page, 1, a.granule);
}

}  // namespace engram

// Writes a chunk's keys and values into a paged cache: token t of sequence b, the last n of whose
// kv_len positions are the chunk's, goes to position kv_len - n + t, that is slot p % page_size of
// page table[b, p / page_size]. A copy: 16 bytes of K and of V per thread, both loads issued before
// the place is looked up. Bound by the launch for a decoding batch (64 tokens: 3.1 us) and by memory
// for long chunks (8192 and 5003 tokens with 8 key-value heads of 128: 16.3 us, 6.6 TB/s of reading
// and writing).
#include "attn_device.cuh"
#include "kernels.h"

namespace engram {

namespace {

constexpr int kThreads = 256;

__global__ void __launch_bounds__(kThreads) kv_append_kernel(const KvAppendArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int32_t chunks = a.head_dim / 8;
  const int32_t per_token = a.kv_heads * chunks;
  const int64_t n = static_cast<int64_t>(a.total) * per_token;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int32_t t = static_cast<int32_t>(i / per_token);
    const int32_t in = static_cast<int32_t>(i - static_cast<int64_t>(t) * per_token);
    const int32_t h = in / chunks, c = (in - h * chunks) * 8;
    const uint4 k = *reinterpret_cast<const uint4*>(a.k + t * a.k_token + h * a.k_head + c);
    const uint4 v = *reinterpret_cast<const uint4*>(a.v + t * a.v_token + h * a.v_head + c);
    // the sequence that holds token t: the last b with cu[b] <= t
    int32_t lo = 0, hi = a.n_seqs;
    while (hi - lo > 1) {
      const int32_t mid = lo + (hi - lo) / 2;
      if (a.cu[mid] <= t) lo = mid;
      else hi = mid;
    }
    const int32_t end = attn_clamp(a.cu[lo + 1], 0, a.total);
    if (t < a.cu[lo] || t >= end) continue;   // a token of no sequence
    const int32_t len = a.kv_len[lo];
    const int32_t p = (len > 0 ? len : 0) - (end - t);   // a negative length is an empty cache
    if (p < 0) continue;   // before the cache's first position: such a token is not kept
    const int32_t col = p / a.page_size;
    if (col >= a.table_width) {
      set_error(a.err, kErrCacheCapacity);
      continue;
    }
    const int32_t page = a.table[static_cast<int64_t>(lo) * a.table_width + col];
    if (page < 0 || page >= a.n_pages) {
      set_error(a.err, kErrPageRange);
      continue;
    }
    const int64_t slot = p - col * a.page_size;
    *reinterpret_cast<uint4*>(a.k_cache + page * a.k_page + slot * a.k_slot + h * a.k_chead + c) = k;
    *reinterpret_cast<uint4*>(a.v_cache + page * a.v_page + slot * a.v_slot + h * a.v_chead + c) = v;
  }
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs& a, cudaStream_t st) {
  const int64_t n = static_cast<int64_t>(a.total) * a.kv_heads * (a.head_dim / 8);
  int64_t blocks = (n + kThreads - 1) / kThreads;
  if (blocks > (1 << 20)) blocks = 1 << 20;   // grid-stride beyond
  return launch_ex(kv_append_kernel, dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, st,
                   true, a);
}

}  // namespace engram

// Attention for items of many query rows over an 8-bit cache (the kernel: attn_tiles.cuh). TMA brings the
// codes; four warps write them out as 16-bit tiles, times their scales, which is what engram_kv_read_fp8
// gives, and all else is as over a cache of 16 bits.
#include "attn_tiles.cuh"

namespace engram {

cudaError_t launch_attn_fp8_tiles(const AttnArgs& in, const KvFp8Part& k, const KvFp8Part& v, cudaStream_t st) {
  AttnArgs a = in;
  alignas(64) CUtensorMap tmQ, tm[2];
  if (!attn_fp8_tensor_maps(a, k, v, 1, tm) || !plan_tiles(a, tmQ)) return cudaErrorInvalidValue;
  const cudaError_t e = launch_tiles_any(a, tmQ, tm[0], tm[1], KvFp8{k, v}, st);
  return e != cudaSuccess ? e : launch_attn_combine(a, kItemRows, st);
}

}  // namespace engram

// Attention for items of many query rows over keys and values of 16 bits: packed prompts and a paged cache
// (the kernel: attn_tiles.cuh).
#include "attn_tiles.cuh"

namespace engram {

cudaError_t launch_attn_tiles(const AttnArgs& in, cudaStream_t st) {
  AttnArgs a = in;
  alignas(64) CUtensorMap tmQ, tmK, tmV;
  if (!attn_tensor_maps(a, &tmK, &tmV) || !plan_tiles(a, tmQ)) return cudaErrorInvalidValue;
  const cudaError_t e = launch_tiles_any(a, tmQ, tmK, tmV, Kv16{}, st);
  // prompts of at most one key tile are never cut
  const bool cut = a.table != nullptr || a.plan.total > kTileKeys;
  return e != cudaSuccess || !cut ? e : launch_attn_combine(a, kItemRows, st);
}

}  // namespace engram

// Joins the pieces of the items that a worker's range cut (attn_plan.cuh): for each row
//   M = max_i M_i,  o = sum_i 2^(M_i - M) o_i / sum_i 2^(M_i - M) l_i.
// Every worker that holds a piece of an item joins its share of the item's rows, so that an item
// that many workers share (one long cache) is joined by as many. A row is read by 1, 2, 4 or 8
// warps, each with kAtOnce pieces in flight at a time, so that even the most pieces (one per SM) are
// a handful of reads one after the other; the warps' parts meet in shared memory. Always in the
// same order. What bounds it is the latency of those reads, from L2, and the launch: 2-4 us. (With
// an item's rows all joined by one worker, a cache of 47 k positions with one key-value head took
// 45 us instead of 25. Joining by the last worker to arrive, without this kernel, was slower too.)
#include "attn_device.cuh"
#include "kernels.h"

namespace engram {

namespace {

constexpr int kWarps = 8;
constexpr int kAtOnce = 4;   // pieces

template <int DH, bool kBf16>
__global__ void __launch_bounds__(kWarps * 32)
    attn_combine_kernel(const AttnArgs a, const AttnPieces pieces, const int32_t rows) {
  constexpr int kVec = DH / 32;   // columns per lane
  __shared__ float part_o[kWarps][DH];
  __shared__ float2 part_ml[kWarps];
  pdl_wait();
  pdl_launch_dependents();
  // z = 0: the item that this worker continues; 1: the one that it begins
  const AttnMeta meta = pieces.meta[blockIdx.x * 2 + blockIdx.z];
  if (meta.pieces == 0) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int per_row = 1;   // warps
  while (per_row < kWarps && per_row * kAtOnce < meta.pieces) per_row *= 2;
  const int part = warp % per_row, at_once = kWarps / per_row;
  const int32_t first = static_cast<int32_t>(blockIdx.x) - meta.owner;   // row of this worker
  const int32_t all = meta.ntok * a.group;
  for (int32_t n0 = blockIdx.y * at_once; first + meta.pieces * n0 < all;
       n0 += gridDim.y * at_once) {
    const int32_t r = first + meta.pieces * (n0 + warp / per_row);
    const bool real = r < all;
    // a running maximum over groups of pieces whose loads are in flight together
    float m = -INFINITY, l = 0.f, acc[kVec] = {};
    for (int32_t i0 = part * kAtOnce; real && i0 < meta.pieces; i0 += per_row * kAtOnce) {
      float2 ml[kAtOnce], v[kAtOnce][kVec / 2];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const int32_t k = i0 + i;
        if (k >= meta.pieces) {
          ml[i].x = -INFINITY;
          continue;
        }
        const int64_t at = ((static_cast<int64_t>(meta.owner) + k) * 2 + (k == 0)) * rows + r;
        ml[i] = *reinterpret_cast<const float2*>(pieces.ml + at * 2);
        const float* o = pieces.o + at * DH + lane * kVec;
        if constexpr (kVec == 4) {
          const float4 x = *reinterpret_cast<const float4*>(o);
          v[i][0] = make_float2(x.x, x.y);
          v[i][1] = make_float2(x.z, x.w);
        } else {
          v[i][0] = *reinterpret_cast<const float2*>(o);
        }
      }
      float top = m;
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) top = fmaxf(top, ml[i].x);
      const float base = top == -INFINITY ? 0.f : top, f0 = exp2_fast(m - base);
      m = top;
      l *= f0;
#pragma unroll
      for (int c = 0; c < kVec; ++c) acc[c] *= f0;
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        if (i0 + i >= meta.pieces) continue;
        const float f = exp2_fast(ml[i].x - base);
        l += f * ml[i].y;
#pragma unroll
        for (int c = 0; c < kVec; c += 2) {
          acc[c] += f * v[i][c / 2].x;
          acc[c + 1] += f * v[i][c / 2].y;
        }
      }
    }
    if (per_row > 1) {   // the same for every warp of the block
      if (lane == 0) part_ml[warp] = make_float2(m, l);
#pragma unroll
      for (int c = 0; c < kVec; ++c) part_o[warp][lane * kVec + c] = acc[c];
      __syncthreads();
      if (part == 0) {
        float top = m;
        for (int i = 1; i < per_row; ++i) top = fmaxf(top, part_ml[warp + i].x);
        const float base = top == -INFINITY ? 0.f : top, f0 = exp2_fast(m - base);
        l *= f0;
#pragma unroll
        for (int c = 0; c < kVec; ++c) acc[c] *= f0;
        for (int i = 1; i < per_row; ++i) {
          const float f = exp2_fast(part_ml[warp + i].x - base);
          l += f * part_ml[warp + i].y;
#pragma unroll
          for (int c = 0; c < kVec; ++c) acc[c] += f * part_o[warp + i][lane * kVec + c];
        }
        m = top;
      }
      __syncthreads();
    }
    if (!real || part != 0) continue;
    const int32_t tok = meta.token0 + r / a.group;
    const int32_t head = meta.h * a.group + r % a.group;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint16_t* op = a.out + static_cast<int64_t>(tok) * a.o_token +
                   static_cast<int64_t>(head) * a.o_head + lane * kVec;
#pragma unroll
    for (int c = 0; c < kVec; c += 2)
      if (lane * kVec + c < a.head_dim)
        *reinterpret_cast<uint32_t*>(op + c) = pack16x2<kBf16>(acc[c] * inv, acc[c + 1] * inv);
    if (a.lse != nullptr && lane == 0)
      a.lse[static_cast<int64_t>(tok) * a.heads + head] = (m + log2f(l)) * 0.69314718055994531f;
  }
}

}  // namespace

cudaError_t launch_attn_combine(const AttnArgs& a, int32_t rows, cudaStream_t st) {
  // a worker has at most half of an item's rows to join
  const int32_t y = rows / 2 / kWarps < 1 ? 1 : rows / 2 / kWarps > 8 ? 8 : rows / 2 / kWarps;
  const dim3 grid(a.plan.workers, y, 2), block(kWarps * 32);
  const AttnPieces p = attn_pieces_at(a.workspace, a.plan.workers, rows);
  if (attn_width(a.head_dim) == 64)
    return a.bf16 ? launch_ex(attn_combine_kernel<64, true>, grid, block, 0, st, true, a, p, rows)
                  : launch_ex(attn_combine_kernel<64, false>, grid, block, 0, st, true, a, p, rows);
  return a.bf16 ? launch_ex(attn_combine_kernel<128, true>, grid, block, 0, st, true, a, p, rows)
                : launch_ex(attn_combine_kernel<128, false>, grid, block, 0, st, true, a, p, rows);
}

}  // namespace engram

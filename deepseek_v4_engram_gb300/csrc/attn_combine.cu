// Joins the pieces of the items that a worker's range cut (attn_plan.cuh): for each row
//   M = max_i M_i,  o = sum_i 2^(M_i - M) o_i / sum_i 2^(M_i - M) l_i,
// pieces in the order of the keys. One warp per row; a worker that begins no cut item has nothing
// to join and its blocks leave at once. It reads what the attention kernel has just written (at
// most two slots per SM), mostly from L2.
#include "attn_device.cuh"
#include "kernels.h"

namespace engram {

namespace {

constexpr int kThreads = 256;
constexpr int kAtOnce = 4;   // pieces

template <int DH, bool kBf16>
__global__ void __launch_bounds__(kThreads)
    attn_combine_kernel(const AttnArgs a, const AttnPieces pieces, const int32_t rows) {
  pdl_wait();
  pdl_launch_dependents();
  const int32_t w = blockIdx.x;
  const AttnMeta meta = pieces.meta[w];
  if (meta.pieces == 0) return;
  const int lane = threadIdx.x & 31;
  constexpr int kVec = DH / 32;   // columns per lane
  for (int32_t r = blockIdx.y * (kThreads / 32) + (threadIdx.x >> 5); r < meta.ntok * a.group;
       r += gridDim.y * (kThreads / 32)) {
    // a running maximum over groups of pieces whose loads are in flight together
    float m = -INFINITY, l = 0.f, acc[kVec] = {};
    for (int32_t i0 = 0; i0 < meta.pieces; i0 += kAtOnce) {
      float2 ml[kAtOnce], v[kAtOnce][kVec / 2];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const int32_t k = i0 + i < meta.pieces ? i0 + i : i0;
        const int64_t at = ((static_cast<int64_t>(w) + k) * 2 + (k == 0)) * rows + r;
        ml[i] = *reinterpret_cast<const float2*>(pieces.ml + at * 2);
        const float* o = pieces.o + at * DH + lane * kVec;
#pragma unroll
        for (int c = 0; c < kVec; c += 2) v[i][c / 2] = *reinterpret_cast<const float2*>(o + c);
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
  const dim3 grid(a.plan.workers, rows / 16 < 8 ? (rows + 7) / 8 : 8), block(kThreads);
  const AttnPieces p = attn_pieces_at(a.workspace, a.plan.workers, rows);
  if (attn_width(a.head_dim) == 64)
    return a.bf16 ? launch_ex(attn_combine_kernel<64, true>, grid, block, 0, st, true, a, p, rows)
                  : launch_ex(attn_combine_kernel<64, false>, grid, block, 0, st, true, a, p, rows);
  return a.bf16 ? launch_ex(attn_combine_kernel<128, true>, grid, block, 0, st, true, a, p, rows)
                : launch_ex(attn_combine_kernel<128, false>, grid, block, 0, st, true, a, p, rows);
}

}  // namespace engram

// Joins the pieces of the items that a worker's range cut (attn_plan.cuh): for each row
//   M = max_i M_i,  o = sum_i 2^(M_i - M) o_i / sum_i 2^(M_i - M) l_i.
// Every worker that holds a piece of an item joins its share of the item's rows, so that an item
// that many workers share (one long cache) is joined by as many. A row is read by teams of lanes
// (as many as a block has, for the most pieces), each with kAtOnce pieces in flight at a time, so
// that even one piece per SM is a handful of reads one after the other; the teams' parts meet in
// shared memory. Always in the same order. What bounds it is the latency of those reads, from L2,
// and the launch: 2-4 us. (With an item's rows all joined by one worker, a cache of 47 k positions
// with one key-value head took 45 us instead of 25. Joining by the last worker to arrive, without
// this kernel, was slower too.)
// After the tiled kernel there are many rows and few pieces, and the arithmetic of places and
// factors counts: teams of 16 lanes share it between two rows (a prompt of 1024 tokens 26.1 us instead
// of 27.3, with 32; five drafted tokens over 16 caches 38.6 instead of 38.2). After the few-row
// kernel a row's reads count: teams of 32 lanes where a row has 128 columns (one token over 511
// positions 9.2 us instead of 9.5, with 16).
#include "attn_device.cuh"
#include "kernels.h"

namespace engram {

namespace {

constexpr int kThreads = 256;
constexpr int kAtOnce = 4;   // pieces

// kLanes: of a team, which takes one row at a time.
template <int DH, int kLanes, bool kBf16>
__global__ void __launch_bounds__(kThreads)
    attn_combine_kernel(const AttnArgs a, const AttnPieces pieces, const int32_t rows) {
  constexpr int kTeams = kThreads / kLanes;
  constexpr int kVec = DH / (4 * kLanes);   // per lane, of four columns each, 4 kLanes apart
  __shared__ float4 part_o[kTeams][DH / 4];
  __shared__ float2 part_ml[kTeams];
  pdl_wait();
  pdl_launch_dependents();
  // z = 0: the item that this worker continues; 1: the one that it begins
  const AttnMeta meta = pieces.meta[blockIdx.x * 2 + blockIdx.z];
  if (meta.pieces == 0) return;
  const int lane = threadIdx.x % kLanes, team = threadIdx.x / kLanes;
  int per_row = 1;   // teams
  while (per_row < kTeams && per_row * kAtOnce < meta.pieces) per_row *= 2;
  const int part = team % per_row, at_once = kTeams / per_row;
  const int32_t first = static_cast<int32_t>(blockIdx.x) - meta.owner;   // row of this worker
  const int32_t all = meta.ntok * a.group;
  for (int32_t n0 = blockIdx.y * at_once; first + meta.pieces * n0 < all;
       n0 += gridDim.y * at_once) {
    const int32_t r = first + meta.pieces * (n0 + team / per_row);
    const bool real = r < all;
    // a running maximum over groups of pieces whose loads are in flight together
    float m = -INFINITY, l = 0.f;
    float4 acc[kVec] = {};
    auto add = [&](float f, const float4 (&v)[kVec]) {
#pragma unroll
      for (int c = 0; c < kVec; ++c) {
        acc[c].x += f * v[c].x;
        acc[c].y += f * v[c].y;
        acc[c].z += f * v[c].z;
        acc[c].w += f * v[c].w;
      }
    };
    auto scale = [&](float f) {
      l *= f;
#pragma unroll
      for (int c = 0; c < kVec; ++c)
        acc[c] = make_float4(acc[c].x * f, acc[c].y * f, acc[c].z * f, acc[c].w * f);
    };
    for (int32_t i0 = part * kAtOnce; real && i0 < meta.pieces; i0 += per_row * kAtOnce) {
      float2 ml[kAtOnce];
      float4 v[kAtOnce][kVec];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const int32_t k = i0 + i;
        ml[i].x = -INFINITY;
        if (k >= meta.pieces) continue;
        const int64_t at = ((static_cast<int64_t>(meta.owner) + k) * 2 + (k == 0)) * rows + r;
        ml[i] = *reinterpret_cast<const float2*>(pieces.ml + at * 2);
#pragma unroll
        for (int c = 0; c < kVec; ++c)
          v[i][c] =
              *reinterpret_cast<const float4*>(pieces.o + at * DH + c * 4 * kLanes + lane * 4);
      }
      float top = m;
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) top = fmaxf(top, ml[i].x);
      const float base = top == -INFINITY ? 0.f : top;
      scale(exp2_fast(m - base));
      m = top;
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        if (i0 + i >= meta.pieces) continue;
        const float f = exp2_fast(ml[i].x - base);
        l += f * ml[i].y;
        add(f, v[i]);
      }
    }
    if (per_row > 1) {   // the same for every team of the block
      if (lane == 0) part_ml[team] = make_float2(m, l);
#pragma unroll
      for (int c = 0; c < kVec; ++c) part_o[team][c * kLanes + lane] = acc[c];
      __syncthreads();
      if (part == 0) {
        float top = m;
        for (int i = 1; i < per_row; ++i) top = fmaxf(top, part_ml[team + i].x);
        const float base = top == -INFINITY ? 0.f : top;
        scale(exp2_fast(m - base));
        for (int i = 1; i < per_row; ++i) {
          const float f = exp2_fast(part_ml[team + i].x - base);
          l += f * part_ml[team + i].y;
          float4 v[kVec];
#pragma unroll
          for (int c = 0; c < kVec; ++c) v[c] = part_o[team + i][c * kLanes + lane];
          add(f, v);
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
                   static_cast<int64_t>(head) * a.o_head + lane * 4;
#pragma unroll
    for (int c = 0; c < kVec; ++c)
      if (c * 4 * kLanes + lane * 4 < a.head_dim)
        *reinterpret_cast<uint2*>(op + c * 4 * kLanes) =
            make_uint2(pack16x2<kBf16>(acc[c].x * inv, acc[c].y * inv),
                       pack16x2<kBf16>(acc[c].z * inv, acc[c].w * inv));
    if (a.lse != nullptr && lane == 0)
      a.lse[static_cast<int64_t>(tok) * a.heads + head] = (m + log2f(l)) * 0.69314718055994531f;
  }
}

template <int DH, int kLanes, bool kBf16>
cudaError_t launch(const AttnArgs& a, int32_t rows, cudaStream_t st) {
  // a worker has at most half of an item's rows to join
  const int32_t y = rows / 2 / (kThreads / kLanes);
  return launch_ex(attn_combine_kernel<DH, kLanes, kBf16>, dim3(a.plan.workers, y < 1 ? 1 : y, 2),
                   dim3(kThreads), 0, st, true, a,
                   attn_pieces_at(a.workspace, a.plan.workers, rows), rows);
}

template <bool kBf16>
cudaError_t launch_any(const AttnArgs& a, int32_t rows, cudaStream_t st) {
  if (attn_width(a.head_dim) == 64) return launch<64, 16, kBf16>(a, rows, st);
  return rows <= kAttnFewRows ? launch<128, 32, kBf16>(a, rows, st)
                              : launch<128, 16, kBf16>(a, rows, st);
}

}  // namespace

cudaError_t launch_attn_combine(const AttnArgs& a, int32_t rows, cudaStream_t st) {
  return a.bf16 ? launch_any<true>(a, rows, st) : launch_any<false>(a, rows, st);
}

}  // namespace engram

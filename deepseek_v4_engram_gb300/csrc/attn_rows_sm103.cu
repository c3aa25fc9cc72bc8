// Attention for items of at most 16 or 32 query rows: decoding, a few drafted tokens, any chunk
// of a sequence whose rows (tokens x heads that share a key-value head) are few.
//
//   o_r = sum_j 2^(x_rj - M_r) v_j / sum_j 2^(x_rj - M_r),   x_rj = scale log2(e) q_r . k_j
//
// in one pass over the keys with a running maximum M and sum. What bounds it is the cache's bytes:
// 32 rows make 32 multiply-adds of each key or value element, below what the tensor cores do in the
// time that the element takes to arrive. So the work is shared out by key tiles alone
// (attn_plan.cuh), one CTA per SM streams its tiles through a ring of two 64 KB stages (five of 32 KB
// where heads have up to 64 columns; three and six are no faster), and the ring runs on across the
// ends of items.
//
// Roles (288 threads): warp 8 requests the tiles by TMA, one page granule per lane; warps 0-7 each
// take 16 rows and some of a tile's keys (with kGroups groups of rows, 16 kGroups of the 128), 16
// at a time, so every warp has its own maximum, sum and output and no step of the loop waits for
// another warp. The products run on mma.sync m16n8k16: its 16 rows are the whole item of a decoding
// step, its fragments stay in registers (scores come out in the layout in which they go back in as
// probabilities), and a tcgen05 tile would be seven eighths padding.
//
// Measured (8 key-value heads of 128): one token each over 64 caches of 1584-2048 positions 80-82 us,
// 5.9 TB/s (a kernel that only reads as many bytes takes 74.5), and over 4 caches of 70001-131072
// positions 256-263 us, 6.7-6.9 TB/s (260); one token over 511 positions 8.9-9.9 us. What every call
// pays, about 9 us, is a worker's look for its range (2.3), the latency of its first page entry, page
// and tile (3.4), the eight warps' results becoming one (1.1) and the joining kernel (3). A tile takes
// 1.3 us with 16 rows (memory's rate; 1.56 where pages of 48 slots make copies of 16 keys) and 1.65 with
// 32, where a warp has twice the keys and its own chain sets the pace. The warps put their results down side by
// side and each joins a part of the rows; handing them over pairwise, in three steps with less to
// do in each, took 0.6-1.1 us more.
#include "attn_device.cuh"
#include "kernels.h"
#include "wkv_tiles.cuh"

namespace engram {

namespace {

constexpr int kConsumers = 8;
constexpr int kExtraUnits = 1;   // an item's fixed time, in key tiles; with 0 to 3 within 2-5%
constexpr int kThreads = (kConsumers + 1) * 32;

// Probabilities are rounded to the values' type for the product with them, since mma.sync takes both
// operands in one 16-bit type: each by half a unit in its last place, as the result is at the end.
// They are summed as they are, so what rounding takes from a small one is lost. bf16 has the exponents
// of f32; f16 ends at 2^-24, and a long cache may hold much weight in keys below that. So exponentials
// are taken against the maximum less this, and f16 reaches from 2^15 for the largest, half its range,
// to 2^-39 of it. Maxima below are all lower by it; the quotient of outputs and sum is the same.
template <bool kBf16>
constexpr float kLift = kBf16 ? 0.f : 15.f;

template <int DH>
struct Geo {
  static constexpr int kHalves = DH / 64;                          // 64-column boxes per row
  static constexpr int kTensorBytes = kTileKeys * DH * 2;          // K or V of a stage
  static constexpr int kStages = DH == 128 ? 2 : 5;
  static constexpr int kJoinRow = DH + 8;                          // floats: eight rows, all banks
  static constexpr int kJoinBytes = kConsumers * 16 * kJoinRow * 4;   // every warp's outputs
};

template <int DH>
struct Shared {
  uint64_t full[Geo<DH>::kStages];
  uint64_t empty[Geo<DH>::kStages];
  AttnStart start;
  float2 ml[kConsumers][16];   // running maxima and sums
  int abort;
};

template <int DH>
constexpr size_t smem_bytes() {
  return 1024 + size_t(Geo<DH>::kStages) * 2 * Geo<DH>::kTensorBytes + Geo<DH>::kJoinBytes +
         sizeof(Shared<DH>);
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

template <bool kBf16>
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  if constexpr (kBf16) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  } else {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
}

// Byte offset of 16-byte chunk `c` (8 columns) of key `row` in a K or V tile: 64-column boxes of
// 128 rows of 128 bytes, 128-byte swizzle.
__device__ __forceinline__ uint32_t tile_offset(int row, int c) {
  return static_cast<uint32_t>((c >> 3) * (kTileKeys * 128) + row * 128 +
                               (((c & 7) ^ (row & 7)) << 4));
}

template <int DH, int kGroups, bool kBf16>
__global__ void __launch_bounds__(kThreads, 1)
    attn_rows_kernel(const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ AttnArgs a, const AttnPieces pieces) {
  using G = Geo<DH>;
  constexpr int kRows = 16 * kGroups;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_1024(smem_raw);
  float* join = reinterpret_cast<float*>(smem + G::kStages * 2 * G::kTensorBytes);
  Shared<DH>* sh = reinterpret_cast<Shared<DH>*>(reinterpret_cast<uint8_t*>(join) + G::kJoinBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < G::kStages; ++s) {
      mbar_init(&sh->full[s], 1);
      mbar_init(&sh->empty[s], kConsumers);
    }
    sh->abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  pdl_wait();   // queries, lengths and the cache may come from the previous kernel
  pdl_launch_dependents();
  attn_find_start<kThreads>(a.plan, blockIdx.x, &sh->start, a.err);
  volatile int* abort = &sh->abort;
  AttnCursor cur = sh->start.cursor;
  AttnSegment seg;

  if (warp == kConsumers) {
    // ------------------------------------------------------------- TMA producer
    TmaRingT<G::kStages> ring;
    const int gran = lane & 15;                     // lanes 0-15 the keys' granules, 16-31 the values'
    const CUtensorMap* map = lane < 16 ? &tmK : &tmV;
    bool stop = false;
    while (!stop && cur.next(a.plan, seg)) {
      for (int32_t t = seg.tile0; t < seg.tile1 && t * kTileKeys < seg.keys; ++t) {
        const int32_t k0 = t * kTileKeys;
        const int32_t n = seg.keys - k0 < kTileKeys ? seg.keys - k0 : kTileKeys;
        const int32_t grans = (n + a.granule - 1) / a.granule;
        KvPlace at{0, 0};
        if (gran < grans) at = kv_place(a, seg, k0 + gran * a.granule);
        stop = __any_sync(0xFFFFFFFFu, !attn_wait(&sh->empty[ring.stage], ring.phase ^ 1u, abort));
        if (stop) break;
        uint8_t* dst = smem + (ring.stage * 2 + (lane < 16 ? 0 : 1)) * G::kTensorBytes;
        if (lane == 0)
          mbar_arrive_expect_tx(&sh->full[ring.stage],
                                static_cast<uint32_t>(grans * a.granule) * 128 * G::kHalves * 2);
        __syncwarp();
        if (gran < grans) {
#pragma unroll
          for (int hf = 0; hf < G::kHalves; ++hf)
            tma_load_4d(dst + hf * (kTileKeys * 128) + gran * a.granule * 128, map,
                        &sh->full[ring.stage], hf * 64, seg.h, at.z, at.w);
        }
        ring.issued();
      }
    }
    __syncwarp();
    ring.drain(sh->full);
  } else {
    // ------------------------------------------------------------- consumers
    const int gid = lane >> 2, tid = lane & 3;
    const int group = warp % kGroups;                       // of rows
    const int keys_at = warp / kGroups * (16 * kGroups);    // first of this warp's keys in a tile
    uint32_t stage = 0, phase = 0;
    if (threadIdx.x == 0) attn_no_pieces(pieces);
    while (cur.next(a.plan, seg)) {
      // Rows gid and gid + 8 of the group: token row / G of the item, head h * G + row % G.
      int32_t limit[2];
      uint32_t qf[DH / 16][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int32_t r = group * 16 + gid + 8 * i, tok = r / a.group;
        const bool valid = tok < seg.ntok;
        const int32_t lim = seg.first + tok;
        limit[i] = valid && lim > 0 ? lim : 0;
        const uint16_t* qp = a.q + static_cast<int64_t>(seg.token0 + tok) * a.q_token +
                             static_cast<int64_t>(seg.h * a.group + (r - tok * a.group)) * a.q_head;
#pragma unroll
        for (int c = 0; c < DH / 8; ++c) {   // 8-column chunk c: columns 8 c + 2 tid, + 1
          uint32_t w = 0;
          if (valid && c * 8 < a.head_dim)
            w = *reinterpret_cast<const uint32_t*>(qp + c * 8 + tid * 2);
          qf[c / 2][(c & 1) * 2 + i] = w;
        }
      }
      float mx[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};
      float o[DH / 8][4];
#pragma unroll
      for (int n = 0; n < DH / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;

      for (int32_t t = seg.tile0; t < seg.tile1 && t * kTileKeys < seg.keys; ++t) {
        const bool here = !__any_sync(
            0xFFFFFFFFu, !attn_wait(&sh->full[stage], phase, abort));
        const uint32_t sk = smem_u32(smem + stage * 2 * G::kTensorBytes);
        const uint32_t sv = sk + G::kTensorBytes;
#pragma unroll 1
        for (int at = keys_at; at < keys_at + 16 * kGroups; at += 16) {
          const int32_t key0 = t * kTileKeys + at;
          if (!here || key0 >= seg.keys) break;
          // scores of 16 rows by 16 keys
          float s[2][4] = {};
          {
            const int row = at + ((lane >> 4) << 3) + (lane & 7);
#pragma unroll
            for (int kk = 0; kk < DH / 16; ++kk) {
              uint32_t b[4];
              ldmatrix_x4(b, sk + tile_offset(row, kk * 2 + ((lane >> 3) & 1)));
              mma_16816<kBf16>(s[0], qf[kk], b[0], b[1]);
              mma_16816<kBf16>(s[1], qf[kk], b[2], b[3]);
            }
          }
          const bool edge = key0 + 16 > seg.first;   // some row does not see all of them
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float x = s[n][e] * a.scale_log2;
              s[n][e] = edge && key0 + n * 8 + tid * 2 + (e & 1) >= limit[e >> 1] ? -INFINITY : x;
            }
          uint32_t p[4];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float m = fmaxf(fmaxf(s[0][2 * i], s[0][2 * i + 1]), fmaxf(s[1][2 * i], s[1][2 * i + 1]));
            m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
            m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
            m = fmaxf(m - kLift<kBf16>, mx[i]);
            const float base = m == -INFINITY ? 0.f : m;   // nothing seen yet: every term is 0
            const float f = exp2_fast(mx[i] - base);
            mx[i] = m;
            float e[4];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              e[2 * n] = exp2_fast(s[n][2 * i] - base);
              e[2 * n + 1] = exp2_fast(s[n][2 * i + 1] - base);
              p[2 * n + i] = pack16x2<kBf16>(e[2 * n], e[2 * n + 1]);
            }
            sum[i] = sum[i] * f + ((e[0] + e[1]) + (e[2] + e[3]));
#pragma unroll
            for (int n = 0; n < DH / 8; ++n) {
              o[n][2 * i] *= f;
              o[n][2 * i + 1] *= f;
            }
          }
          const int row = at + (lane & 15);
          const int32_t seen = seg.keys - key0;   // keys past it hold whatever the memory held
          if (!edge) {
#pragma unroll
            for (int n = 0; n < DH / 16; ++n) {
              uint32_t b[4];
              ldmatrix_x4_trans(b, sv + tile_offset(row, n * 2 + (lane >> 4)));
              mma_16816<kBf16>(o[2 * n], p, b[0], b[1]);
              mma_16816<kBf16>(o[2 * n + 1], p, b[2], b[3]);
            }
          } else {
            // A probability of 0 does not undo an infinity or NaN that it multiplies: values past
            // the last key are cleared, and if one that only some rows see is not finite, the
            // products of these 16 keys are formed one by one for the rows that see them.
            uint32_t keep[2];   // this lane's key pairs 2 tid, + 1 and 2 tid + 8, + 9
#pragma unroll
            for (int i = 0; i < 2; ++i)
              keep[i] = (tid * 2 + 8 * i < seen ? 0x0000FFFFu : 0u) |
                        (tid * 2 + 8 * i + 1 < seen ? 0xFFFF0000u : 0u);
            bool bad = false;
#pragma unroll
            for (int n = 0; n < DH / 16; ++n) {
              uint32_t b[4];
              ldmatrix_x4_trans(b, sv + tile_offset(row, n * 2 + (lane >> 4)));
#pragma unroll
              for (int e = 0; e < 4; ++e) bad |= nonfinite_bits<kBf16>(b[e] & keep[e & 1]) != 0;
            }
            if (!__any_sync(0xFFFFFFFFu, bad)) {
#pragma unroll
              for (int n = 0; n < DH / 16; ++n) {
                uint32_t b[4];
                ldmatrix_x4_trans(b, sv + tile_offset(row, n * 2 + (lane >> 4)));
                mma_16816<kBf16>(o[2 * n], p, b[0] & keep[0], b[1] & keep[1]);
                mma_16816<kBf16>(o[2 * n + 1], p, b[2] & keep[0], b[3] & keep[1]);
              }
            } else {
              for (int j = 0; j < 16; ++j) {
                // row i's probability of key j sits in lane (row, (j % 8) / 2)
                const int src = gid * 4 + ((j & 7) >> 1);
                float pj[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  const uint32_t lo = __shfl_sync(0xFFFFFFFFu, p[i], src);
                  const uint32_t hi = __shfl_sync(0xFFFFFFFFu, p[2 + i], src);
                  const uint32_t w = j < 8 ? lo : hi;
                  pj[i] = to_f32<kBf16>(static_cast<uint16_t>(j & 1 ? w >> 16 : w));
                }
#pragma unroll
                for (int n = 0; n < DH / 8; ++n) {
                  uint32_t w;
                  asm volatile("ld.shared.u32 %0, [%1];"
                               : "=r"(w)
                               : "r"(sv + tile_offset(at + j, n) + tid * 4)
                               : "memory");
#pragma unroll
                  for (int i = 0; i < 2; ++i)
                    if (key0 + j < limit[i]) {
                      o[n][2 * i] += pj[i] * to_f32<kBf16>(static_cast<uint16_t>(w));
                      o[n][2 * i + 1] += pj[i] * to_f32<kBf16>(static_cast<uint16_t>(w >> 16));
                    }
                }
              }
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->empty[stage]);
        if (++stage == G::kStages) { stage = 0; phase ^= 1u; }
      }

      // ---- the maxima, sums and outputs of a row group's warps become one: each warp puts its own
      // down as they are, and then takes a part of the rows
      named_bar_sync(1, kConsumers * 32);   // the segment before has been read
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        sum[i] += __shfl_xor_sync(0xFFFFFFFFu, sum[i], 1);
        sum[i] += __shfl_xor_sync(0xFFFFFFFFu, sum[i], 2);
        if (tid == 0) sh->ml[warp][gid + 8 * i] = make_float2(mx[i], sum[i]);
        float* to = join + (warp * 16 + gid + 8 * i) * G::kJoinRow + tid * 2;
#pragma unroll
        for (int n = 0; n < DH / 8; ++n)
          *reinterpret_cast<float2*>(to + n * 8) = make_float2(o[n][2 * i], o[n][2 * i + 1]);
      }
      named_bar_sync(1, kConsumers * 32);
      const bool whole = seg.begins() && seg.ends();
      const int64_t slot = static_cast<int64_t>(blockIdx.x) * 2 + (seg.begins() ? 1 : 0);
      constexpr int kLanes = DH / 4;   // of a row
      const int col = lane % kLanes * 4;
#pragma unroll 1
      for (int n = 0; n < kRows * kLanes / (kConsumers * 32); ++n) {
        const int r = (n * kConsumers + warp) * (32 / kLanes) + lane / kLanes, tok = r / a.group;
        if (tok >= seg.ntok) continue;
        float m = -INFINITY, l = 0.f, acc[4] = {};
#pragma unroll
        for (int w = 0; w < kConsumers / kGroups; ++w)
          m = fmaxf(m, sh->ml[w * kGroups + r / 16][r % 16].x);
        const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int w = 0; w < kConsumers / kGroups; ++w) {
          const int from = w * kGroups + r / 16;
          const float2 ml = sh->ml[from][r % 16];
          const float4 v = *reinterpret_cast<const float4*>(
              join + (from * 16 + r % 16) * G::kJoinRow + col);
          const float f = exp2_fast(ml.x - base);
          l += f * ml.y;
          acc[0] += f * v.x;
          acc[1] += f * v.y;
          acc[2] += f * v.z;
          acc[3] += f * v.w;
        }
        if (whole) {
          const float inv = l == 0.f ? 0.f : 1.f / l;
          const int32_t head = seg.h * a.group + (r - tok * a.group);
          const int64_t token = static_cast<int64_t>(seg.token0) + tok;
          if (col < a.head_dim)
            *reinterpret_cast<uint2*>(a.out + token * a.o_token +
                                      static_cast<int64_t>(head) * a.o_head + col) =
                make_uint2(pack16x2<kBf16>(acc[0] * inv, acc[1] * inv),
                           pack16x2<kBf16>(acc[2] * inv, acc[3] * inv));
          if (a.lse != nullptr && col == 0)
            a.lse[token * a.heads + head] = (m + log2f(l)) * 0.69314718055994531f;
        } else {
          *reinterpret_cast<float4*>(pieces.o + (slot * kRows + r) * DH + col) =
              make_float4(acc[0], acc[1], acc[2], acc[3]);
          if (col == 0)
            *reinterpret_cast<float2*>(pieces.ml + (slot * kRows + r) * 2) = make_float2(m, l);
        }
      }
      if (threadIdx.x == 0) attn_piece(pieces, seg);
    }
  }
  __syncwarp();
  cta_sync_all();
  if (threadIdx.x == 0) attn_report(abort, a.err);
}

template <int DH, int kGroups, bool kBf16>
cudaError_t launch(const AttnArgs& a, const CUtensorMap& tmK, const CUtensorMap& tmV,
                   cudaStream_t st) {
  const cudaError_t e = ensure_dynamic_smem(
      reinterpret_cast<const void*>(attn_rows_kernel<DH, kGroups, kBf16>), smem_bytes<DH>());
  if (e != cudaSuccess) return e;
  return launch_ex(attn_rows_kernel<DH, kGroups, kBf16>, dim3(a.plan.workers), dim3(kThreads),
                   smem_bytes<DH>(), st, true, tmK, tmV, a,
                   attn_pieces_at(a.workspace, a.plan.workers, 16 * kGroups));
}

template <int kGroups>
cudaError_t launch_any(AttnArgs a, cudaStream_t st) {
  a.plan.tokens = 16 * kGroups / a.group;
  a.plan.workers = device_sm_count();
  a.plan.extra = kExtraUnits;
  alignas(64) CUtensorMap tmK, tmV;
  if (!attn_tensor_maps(a, &tmK, &tmV)) return cudaErrorInvalidValue;
  cudaError_t e;
  if (attn_width(a.head_dim) == 64)
    e = a.bf16 ? launch<64, kGroups, true>(a, tmK, tmV, st)
               : launch<64, kGroups, false>(a, tmK, tmV, st);
  else
    e = a.bf16 ? launch<128, kGroups, true>(a, tmK, tmV, st)
               : launch<128, kGroups, false>(a, tmK, tmV, st);
  return e != cudaSuccess ? e : launch_attn_combine(a, 16 * kGroups, st);
}

}  // namespace

cudaError_t launch_attn_rows(const AttnArgs& a, int32_t rows, cudaStream_t st) {
  return rows <= 16 ? launch_any<1>(a, st) : launch_any<2>(a, st);
}

}  // namespace engram

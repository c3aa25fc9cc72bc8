// Attention over an 8-bit paged cache for items of at most 8, 16, 32 or 48 query rows (64 too where heads have up
// to 64 columns): decoding, a few drafted tokens, any chunk of a sequence whose rows (tokens x heads that share a
// key-value head) are few.
//
//   x_rj = scale log2(e) 2^k_j q_r . K_j,   y_rj = x_rj + v_j        K_j, V_j: codes; k_j, v_j: scales
//   o_r  = sum_j 2^(y_rj - B_r) V_j / sum_j 2^(y_rj - B_r) 2^-v_j
//
// in one pass over the keys. What bounds it is the cache's bytes, half of a 16-bit cache's, so there is
// half the time for a key: a code must cost little on its way into a product. A scale belongs to a key
// or a value as a whole, so it is a factor of a score and of a probability, and codes become f16 with one
// conversion for two and nothing else, exactly; queries are f16 too (a bf16 row scaled by a power of two).
//
// The products run on mma.sync m16n8k16 turned over: S^T = K Q^T and O^T = V^T P^T, with the codes as the
// 16-row operand and 8 query rows as the narrow one, so that a decoding item of up to 8 rows fills it.
// Which of a lane's elements stand for which index of a contraction is free as long as both operands
// agree, and so codes are read 16 bytes at a time, straight from where TMA puts them: a lane's 16 bytes
// of a key row are the columns of four steps, and 16 bytes of four value rows, their bytes interleaved in
// pairs, are eight tiles of V^T. S^T becomes P^T's operand by two 8 x 8 transposes in registers.
//
// Roles (384 threads): warps 8-10 request the tiles; warps 0-7 each take 16 or 32 of a stage's keys, so every
// warp has its own base, sum and output and no step of the loop waits for another warp. Work is shared out by key
// tiles (attn_plan.cuh).
//
// Two key-value heads make an item where they lie beside each other (the usual [slot, head, column] order): TMA is
// slow per row, not per byte, and memory gives less where 128 bytes of every kilobyte are read. The even warps then
// take one head, the odd ones the other. With more than 16 rows they take one half of a head's rows each instead:
// every code is then converted by two warps, but a warp's rows leave it the registers for 32 keys at once (32 rows:
// two caches of 100003 and 131072 positions with 8 heads 150 us; all the rows in every warp, 16 keys at a time,
// 163-170). 24 rows of 128 columns leave it that room only with the queries in shared memory (40 or 48 rows over
// those caches 197 us; 16 keys at a time with the queries in registers 233), and registers spill all the same: 160
// bytes a thread are stored and 68 loaded (128 and 40 with 32 rows of 64 columns, less than 80 in the other forms).
//
// The base B_r lags behind the maximum: it is found anew only when some y exceeds it by 2^kSlack or more,
// which a warp finds out with one vote instead of the shuffles of a maximum.
//
// Measured (replayed, inputs larger than L2): one token each over 64 caches of 1584-2048 positions, 32 heads of
// 128 over 8, 50-51 us (a 16-bit cache 82), over 4 caches of 70001-131072 140-144 us, 6.2-6.4 TB/s from one GPU to
// another; 24 caches of 100-7061 with 16 heads of 64, f16, 40.7; one token over 511 positions 8.2. A call's fixed time is about 9 us: range, first
// page entry, page and tile, joining warps and pieces. A stage of 32 KB takes 0.75 us where memory alone sets
// the pace (a copy that only reads; 0.73 at the copy rate) and 0.74-0.8 here with 8 rows of a head, 0.82 with 16,
// 1.5 with 32, 2.0 with 48, whose chain of steps is longer than the wait for memory. What brought it there: all copies
// of a tile from one warp 0.92; scales by TMA 100 cycles a copy like codes; L2 fetches of 256 bytes for rows of
// 128 (44% more traffic); one 16-key step of a warp at a time 1105 cycles, two overlapped 1550. Slower: the codes
// by 16-byte asynchronous copies (1.4 us a tile), two chains for a score, value rows read before the keys.
#include <type_traits>

#include "kernels.h"
#include "kv_fp8.cuh"
#include "wkv_tiles.cuh"

namespace engram {

namespace {

constexpr int kConsumers = 8;
// An item's fixed time, in key tiles. With 0, 1, 2: 24 caches with 16 heads of 64 48.8, 42.5, 40.8 us, five drafted
// tokens over 16 caches 45.5, 45.4, 43.3, two long caches with 16 rows 91.0, 89.8, 88.4, others the same.
constexpr int kExtraUnits = 2;
constexpr int kThreads = (kConsumers + 4) * 32;
// 256 * 232 + 128 * 40 = 384 * 168
constexpr int kConsumerRegs = 232, kProducerRegs = 40;

// Probabilities times their values' scales are rounded to f16 for the product with the codes, by half a
// unit in the last place (2^-11); f16 ends at 2^-24. They are taken kLift above the largest one, and up
// to kSlack more until the base is raised: 2^15 at most, and what lies 2^-35 below the largest is lost.
constexpr float kLift = 11.f, kSlack = 4.f;
// Scores beyond 2^24 or so leave no room for kLift between them: a difference may be a whole step of theirs.
constexpr float kMostExponent = 15.5f;
// The sum goes without the values' scales: from a probability times its value's scale, 2^-v of it. With
// scales from 2^-100 on that may be large, so it is taken this much lower and the sum stays finite. (Terms
// whose probability has underflowed in f32 are missing: values 2^100 below the ones that count.)
constexpr int kSumDrop = 6;
// A row of zeros among the values has a scale too, 1 as the append writes it, and adds nothing to the outputs. Were it
// to raise the base by that scale, what smaller values add would be rounded away beside it. So where the base is to rise
// and some scale is 1 or more, such keys are looked for: their probabilities go into the sum at once, and they raise
// the base as values of scale 2^-kZeroReach would, for a sum of 2^30 of them, each up to 2^(kZeroReach + kLift -
// kSumDrop) = 2^97, to stay finite. (Looked for whatever the scales, every rise is longer: five drafted tokens over 16
// caches 44.4 us instead of 43.9, 42.9 without it; 64 rows over 24 caches in f16 144, 142.8, 138; two long caches with
// 16 rows 90.5, 87.8, 86.6.)
constexpr float kZeroReach = 92.f;

// An item's rows are one part, or two that the even and the odd warps take: of a key-value head each (kHeads = 2),
// or of the same one (kGroups = 2). NT: tiles of 8 rows of a part.
template <int DH, int NT, int kHeads, int kGroups>
struct Geo {
  static constexpr int kParts = kHeads * kGroups, kPartRows = 8 * NT, kRows = kParts * kPartRows;
  static constexpr int kTensorBytes = kTileKeys * kHeads * DH;         // codes of K or V of a stage
  static constexpr int kScaleBytes = kTileKeys * kHeads;
  static constexpr int kJoinRow = DH + 4;
  static constexpr int kJoinRows = NT == 2 ? 16 : 8;                   // of a part, joined at a time
  static constexpr int kJoinBytes = kConsumers * kJoinRows * kJoinRow * 4;
  // Queries in shared memory, where registers have no room for them: [part][step][tile][lane]
  static constexpr bool kQueriesShared = DH == 128 && NT == 3;
  static constexpr int kQueryBytes = kQueriesShared ? kParts * (DH / 16) * NT * 32 * 8 : 0;
  static constexpr int kStages = kTensorBytes == 32768 ? 2 : kTensorBytes == 16384 ? (NT == 2 ? 4 : 5) : 8;
};

template <int DH, int NT, int kHeads, int kGroups>
struct Shared {
  using G = Geo<DH, NT, kHeads, kGroups>;
  uint64_t full[G::kStages];
  uint64_t empty[G::kStages];
  AttnStart start;
  float row_scale[G::kQueriesShared ? G::kRows : 1];
  float2 ml[kConsumers][G::kPartRows];   // bases and sums
  // Columns of a row that are NaN by a value's code, and whether there are any. Of a segment and of the next, which
  // a warp may be at while others still write the rows of the first.
  uint32_t poison[2][G::kRows][DH / 32];
  int poisoned[2];
  int abort;
};

template <int DH, int NT, int kHeads, int kGroups>
constexpr size_t smem_bytes() {
  using G = Geo<DH, NT, kHeads, kGroups>;
  return 1024 + size_t(G::kStages) * 2 * (G::kTensorBytes + G::kScaleBytes) + G::kQueryBytes + G::kJoinBytes +
         sizeof(Shared<DH, NT, kHeads, kGroups>);
}

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float min_nan(float a, float b) {
  float d;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

__device__ __forceinline__ uint32_t codes_lo(uint32_t w) {
  return e4m3x2_to_f16x2(static_cast<uint16_t>(w));
}
__device__ __forceinline__ uint32_t codes_hi(uint32_t w) {
  return e4m3x2_to_f16x2(static_cast<uint16_t>(w >> 16));
}

// Which key of 16 (of each half) a lane's row `i` of S^T stands for: chosen so that eight lanes' 16-byte
// reads of a key row (lanes g and g + 1, four chunks each), and of a value row (lanes t, and two or four
// chunks), meet every bank of the swizzle once.
//   128 columns, one head:   keys of g and g + 1 differ in bit 2 (values: see `swapped`)
//   128 columns, two heads:  a key is two rows, so in bit 1; values of lanes t in their low two bits
//   64 columns, one head:    rows of 64 bytes, keys differ in bit 0, values in bits 0 and 2
//   64 columns, two heads:   in bit 2, values in bits 1 and 2
template <int DH, int kHeads>
__device__ __forceinline__ int key_of(int i) {
  const int t = i >> 1, up = i & 1;
  if constexpr (DH == 128) return kHeads == 1 ? (up << 2) | t : (up ? (t ^ 2) + 4 : t);
  if constexpr (kHeads == 2) return up ? (2 * t ^ 4) + 1 : 2 * t;
  return ((t & 1) | ((t & 2) << 1)) ^ (up * 3);
}

template <int DH, int NT, int kHeads, int kGroups, bool kBf16>
__global__ void __launch_bounds__(kThreads, 1)
    attn_fp8_rows_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                         const __grid_constant__ AttnArgs a, const KvFp8Part ks, const KvFp8Part vs,
                         const AttnPieces pieces) {
  using G = Geo<DH, NT, kHeads, kGroups>;
  constexpr int kWarpKeys = kTileKeys * G::kParts / kConsumers;   // of a stage: 16 or 32
  constexpr int U = kWarpKeys / 16;   // times 16 keys at once, whose chains of steps overlap
  constexpr int kSteps = DH / 16;     // of a score's contraction; and tiles of V^T
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_1024(smem_raw);
  uint8_t* scales = smem + G::kStages * 2 * G::kTensorBytes;
  uint2* queries = reinterpret_cast<uint2*>(scales + G::kStages * 2 * G::kScaleBytes);
  float* join = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(queries) + G::kQueryBytes);
  using S = Shared<DH, NT, kHeads, kGroups>;
  S* sh = reinterpret_cast<S*>(reinterpret_cast<uint8_t*>(join) + G::kJoinBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < G::kStages; ++s) {
      mbar_init(&sh->full[s], 2 + 32);   // keys, values, and each lane's scales
      mbar_init(&sh->empty[s], kConsumers);
    }
    sh->abort = 0;
    sh->poisoned[0] = sh->poisoned[1] = 0;
    for (int i = 0; i < 2 * G::kRows * (DH / 32); ++i) (&sh->poison[0][0][0])[i] = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  pdl_wait();   // queries, lengths and the cache may come from the previous kernel
  pdl_launch_dependents();
  attn_find_start<kThreads>(a.plan, blockIdx.x, &sh->start, a.err);
  volatile int* abort = &sh->abort;

  if (warp >= kConsumers) {
    // ------------------------------------------------------------- producers
    // Warp 8 requests the keys, warp 9 the values, a page granule per lane (a warp issues its lanes' copies
    // one after the other: with both in one warp that, not memory, set the pace); warp 10 the scales of both,
    // four slots per lane, with copies of 4 bytes: TMA takes as long for a granule's as for its codes.
    set_max_regs_down<kProducerRegs>();
    const int part = warp - kConsumers;
    AttnCursor cur = sh->start.cursor;
    AttnSegment seg;
    TmaRingT<G::kStages> ring;
    bool stop = part > 2;
    while (!stop && cur.next(a.plan, seg)) {
      const int32_t h0 = seg.h * kHeads;
      for (int32_t k0 = seg.tile0 * kTileKeys; k0 < seg.tile1 * kTileKeys && k0 < seg.keys; k0 += kTileKeys) {
        const int32_t n = seg.keys - k0 < kTileKeys ? seg.keys - k0 : kTileKeys;
        const int32_t grans = (n + a.granule - 1) / a.granule;
        const int32_t mine = part < 2 ? lane * a.granule : lane * 4;   // first slot of the lane's copy
        const bool live = mine < grans * a.granule;
        KvPlace at{0, 0};
        if (live) at = kv_place(a, seg, k0 + mine);
        stop = __any_sync(0xFFFFFFFFu, !attn_wait(&sh->empty[ring.stage], ring.phase ^ 1u, abort));
        if (stop) break;
        uint64_t* full = &sh->full[ring.stage];
        if (part < 2) {
          if (lane == 0) mbar_arrive_expect_tx(full, static_cast<uint32_t>(grans * a.granule) * kHeads * DH);
          __syncwarp();
          if (live)
            tma_load_4d(smem + (ring.stage * 2 + part) * G::kTensorBytes + lane * a.granule * kHeads * DH,
                        part == 0 ? &tmK : &tmV, full, 0, DH == 64 ? seg.h : h0, at.z, at.w);
        } else {
          const bool there = at.w < a.n_pages;
#pragma unroll
          for (int head = 0; head < kHeads; ++head) {
            if (!live) continue;
            const uint32_t to = smem_u32(scales + ring.stage * 2 * G::kScaleBytes + head * kTileKeys + mine);
            copy4(to, ks.scales + (there ? at.w * ks.scale_page + (h0 + head) * ks.scale_head + at.z : 0), there);
            copy4(to + G::kScaleBytes,
                  vs.scales + (there ? at.w * vs.scale_page + (h0 + head) * vs.scale_head + at.z : 0), there);
          }
          arrive_after_copies(full);
        }
        ring.issued();
      }
    }
    __syncwarp();
    ring.drain(sh->full);
  } else {
    // ------------------------------------------------------------- consumers
    set_max_regs_up<kConsumerRegs>();
    AttnCursor cur = sh->start.cursor;
    AttnSegment seg;
    const int g = lane >> 2, t4 = lane & 3;
    const int part = G::kParts == 2 ? warp & 1 : 0;
    const int sub = kHeads == 2 ? part : 0;                     // the warp's key-value head
    const int row0 = kGroups == 2 ? part * G::kPartRows : 0;    // its first row of those of the head
    const int keys_at = warp / G::kParts * kWarpKeys;           // its first key of a stage
    const int group = a.group / kHeads;                         // query heads of a key-value head
    const int kg = key_of<DH, kHeads>(g);                       // rows g and g + 8 of S^T: keys kg and kg + 8
    const int scale0 = sub * kTileKeys + keys_at + kg;
    // Where chunk `c` of 16 bytes of the warp's head in key `key` of a stage lies. Two heads: 128-byte rows of
    // one key and head each, in this order, or of both heads of a key.
    auto row_at = [&](int key, int c) -> uint32_t {
      if constexpr (DH == 128) {
        const int row = key * kHeads + sub;
        return row * 128 + ((c ^ (row & 7)) << 4);
      } else if constexpr (kHeads == 2) {
        return key * 128 + (((c + 4 * sub) ^ (key & 7)) << 4);
      } else {
        return key * 64 + ((c ^ (key >> 1 & 3)) << 4);
      }
    };
    constexpr int kKeyBytes = kHeads * DH;
    // a lane's place in a stage: 16 bytes of columns of two key rows, and of four value rows
    const uint32_t k_off = row_at(keys_at + kg, t4);
    const bool swapped = DH == 128 && kHeads == 1 && (g & 1);   // the first one read is the second of the pair
    const int va = key_of<DH, kHeads>(2 * t4 + swapped), vb = key_of<DH, kHeads>(2 * t4 + !swapped);
    auto v_at = [&](int key) {
      return DH == 128 ? row_at(keys_at + key, g) : row_at(keys_at + key, g >> 1) + (g & 1) * 8;
    };
    const uint32_t va_off = v_at(va), vb_off = v_at(vb);
    const uint32_t sel_lo = swapped ? 0x1504 : 0x5140, sel_hi = swapped ? 0x3726 : 0x7362;
    uint32_t stage = 0, phase = 0;
    int turn = 1;   // which of the two sets of marks is the segment's
    if (threadIdx.x == 0) attn_no_pieces(pieces);
    while (cur.next(a.plan, seg)) {
      turn ^= 1;
      // ---- queries: row n of a head's is token n / group of the item, its query head n % group
      uint2 qf[G::kQueriesShared ? 1 : NT][kSteps];
      float rc[NT][2];       // of rows 2 t4 and + 1: what turns a product into a score, but for the key's scale
      int32_t limit[NT][2];
      auto load_row = [&](int nt, uint32_t (&w)[kSteps][2]) {
        const int32_t r = row0 + nt * 8 + g, tok = r / group;
        const bool valid = tok < seg.ntok;
        const uint16_t* qp = a.q + static_cast<int64_t>(seg.token0 + tok) * a.q_token +
                             static_cast<int64_t>(seg.h * a.group + sub * group + (r - tok * group)) * a.q_head;
#pragma unroll
        for (int half = 0; half < DH / 64; ++half) {   // columns 16 (t4 + 4 half) + 0 .. 15
          const int col = 16 * (t4 + 4 * half);
          uint4 x = make_uint4(0, 0, 0, 0), y = x;
          if (valid && col < a.head_dim) {
            x = *reinterpret_cast<const uint4*>(qp + col);
            y = *reinterpret_cast<const uint4*>(qp + col + 8);
          }
          w[half * 4][0] = x.x;
          w[half * 4][1] = x.y;
          w[half * 4 + 1][0] = x.z;
          w[half * 4 + 1][1] = x.w;
          w[half * 4 + 2][0] = y.x;
          w[half * 4 + 2][1] = y.y;
          w[half * 4 + 3][0] = y.z;
          w[half * 4 + 3][1] = y.w;
        }
      };
      // All the loads before the first shuffle, which no load passes (24 caches with 64 rows, bf16, 176 -> 151 us).
      uint32_t words[NT][kSteps][2];
      if constexpr (!G::kQueriesShared)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) load_row(nt, words[nt]);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (!G::kQueriesShared || warp / G::kParts == nt) {
          uint32_t (&w)[kSteps][2] = words[nt];
          if constexpr (G::kQueriesShared) load_row(nt, w);
          float back = a.scale_log2;
          if constexpr (kBf16) {
            // the largest element goes to 2^14 .. 2^15
            uint32_t top = 0;
#pragma unroll
            for (int kk = 0; kk < kSteps; ++kk)
              top = __vmaxu2(top, __vmaxu2(w[kk][0] & 0x7FFF7FFFu, w[kk][1] & 0x7FFF7FFFu));
            top = __vmaxu2(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
            top = __vmaxu2(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
            top = max(top >> 16, top & 0xFFFFu) >> 7;          // its exponent
            top = top < 15 ? 15 : top;
            const float f = __uint_as_float((268u - top) << 23);
            back *= __uint_as_float((top - 14) << 23);
#pragma unroll
            for (int kk = 0; kk < kSteps; ++kk)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                w[kk][e] = pack16x2<false>(__uint_as_float(w[kk][e] << 16) * f,
                                           __uint_as_float(w[kk][e] & 0xFFFF0000u) * f);
          }
          if constexpr (G::kQueriesShared) {
#pragma unroll
            for (int kk = 0; kk < kSteps; ++kk)
              queries[((part * kSteps + kk) * NT + nt) * 32 + lane] = make_uint2(w[kk][0], w[kk][1]);
            if (t4 == 0) sh->row_scale[part * G::kPartRows + nt * 8 + g] = back;
          } else {
#pragma unroll
            for (int kk = 0; kk < kSteps; ++kk) qf[nt][kk] = make_uint2(w[kk][0], w[kk][1]);
#pragma unroll
            for (int j = 0; j < 2; ++j) rc[nt][j] = __shfl_sync(0xFFFFFFFFu, back, (2 * t4 + j) * 4);
          }
        }
      }
      if constexpr (G::kQueriesShared) named_bar_sync(1, kConsumers * 32);
      float base[NT][2], sum[NT][2];
      float o[NT][kSteps][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int32_t tok = (row0 + nt * 8 + 2 * t4 + j) / group;
          const bool valid = tok < seg.ntok;
          const int32_t lim = seg.first + tok;
          limit[nt][j] = valid && lim > 0 ? lim : 0;
          base[nt][j] = valid ? -INFINITY : 1e30f;   // rows that are not there never ask for a new one
          sum[nt][j] = 0.f;
          if constexpr (G::kQueriesShared) rc[nt][j] = sh->row_scale[part * G::kPartRows + nt * 8 + 2 * t4 + j];
        }
#pragma unroll
        for (int i = 0; i < kSteps; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
      }

      for (int32_t first = seg.tile0 * kTileKeys; first < seg.tile1 * kTileKeys && first < seg.keys;
           first += kTileKeys) {
        const bool here = !__any_sync(0xFFFFFFFFu, !attn_wait(&sh->full[stage], phase, abort));
        const int32_t key0 = first + keys_at;   // of U times 16
        if (here && key0 < seg.keys) {
          const uint8_t* sk = smem + stage * 2 * G::kTensorBytes;
          const uint8_t* sv = sk + G::kTensorBytes;
          const uint8_t* ss = scales + stage * 2 * G::kScaleBytes;
          // ---- scores of 16 U keys by the rows
          float s[U][NT][4] = {};
#pragma unroll
          for (int half = 0; half < DH / 64; ++half) {
            uint32_t wl[U][4], wh[U][4];
#pragma unroll
            for (int u = 0; u < U; ++u) {
              const uint8_t* at = sk + u * 16 * kKeyBytes + (k_off ^ (half * 64));
              const uint4 lo = *reinterpret_cast<const uint4*>(at);
              const uint4 hi = *reinterpret_cast<const uint4*>(at + 8 * kKeyBytes);
              wl[u][0] = lo.x, wl[u][1] = lo.y, wl[u][2] = lo.z, wl[u][3] = lo.w;
              wh[u][0] = hi.x, wh[u][1] = hi.y, wh[u][2] = hi.z, wh[u][3] = hi.w;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint2 q[NT];
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                if constexpr (G::kQueriesShared)
                  q[nt] = queries[((part * kSteps + half * 4 + i) * NT + nt) * 32 + lane];
                else
                  q[nt] = qf[nt][half * 4 + i];
#pragma unroll
              for (int u = 0; u < U; ++u) {
                const uint32_t f[4] = {codes_lo(wl[u][i]), codes_lo(wh[u][i]), codes_hi(wl[u][i]), codes_hi(wh[u][i])};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma_f16(s[u][nt], f, q[nt].x, q[nt].y);
              }
            }
          }
          // ---- values: four rows of 16 (8) columns, pairs of rows to be interleaved
          constexpr int kWords = DH / 32;
          uint32_t v[U][4][kWords];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const uint32_t at[4] = {va_off, vb_off, va_off + 8 * kKeyBytes, vb_off + 8 * kKeyBytes};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint8_t* from = sv + u * 16 * kKeyBytes + at[i];
              if constexpr (DH == 128) {
                const uint4 w = *reinterpret_cast<const uint4*>(from);
                v[u][i][0] = w.x, v[u][i][1] = w.y, v[u][i][2] = w.z, v[u][i][3] = w.w;
              } else {
                const uint2 w = *reinterpret_cast<const uint2*>(from);
                v[u][i][0] = w.x, v[u][i][1] = w.y;
              }
            }
          }
          // ---- scales: a lane's keys are kg and kg + 8 of each 16
          float kf[2 * U];
          uint32_t vb8[2 * U];   // the values' bytes
          bool not_numbers = false;
#pragma unroll
          for (int i = 0; i < 2 * U; ++i) {
            kf[i] = fp8_scale_value(ss[scale0 + 8 * i]);
            vb8[i] = ss[G::kScaleBytes + scale0 + 8 * i];
            not_numbers |= vb8[i] == kNanScale;
          }
          if (__any_sync(0xFFFFFFFFu, not_numbers)) {   // rare: NaN codes instead
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int key = keys_at + u * 16 + (i & 1 ? vb : va) + (i & 2 ? 8 : 0);
                if (ss[G::kScaleBytes + sub * kTileKeys + key] == kNanScale)
#pragma unroll
                  for (int w = 0; w < kWords; ++w) v[u][i][w] = 0x7F7F7F7Fu;
              }
#pragma unroll
            for (int i = 0; i < 2 * U; ++i) vb8[i] = vb8[i] == kNanScale ? 127u : vb8[i];
          }
          float ve[2 * U], unscale[2 * U];   // exponents, and 2^-(v + kSumDrop)
#pragma unroll
          for (int i = 0; i < 2 * U; ++i) {
            ve[i] = static_cast<float>(static_cast<int>(max(vb8[i], kMinScale)) - 127);
            // (below f32's normal numbers from byte 248 on, and exact there too)
            unscale[i] = __uint_as_float((255u - max(vb8[i], kMinScale)) << 23) * (0.5f / (1 << kSumDrop));
          }
          const bool edge = key0 + 16 * U > seg.first;   // some row does not see all of them
          bool over = false;
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int j = e & 1, k = 2 * u + (e >> 1);
                const bool hidden = edge && key0 + kg + 8 * k >= limit[nt][j];
                float& y = s[u][nt][e];
                y = hidden ? -INFINITY : fmaf(y, rc[nt][j] * kf[k], ve[k]);
                over |= y > base[nt][j] + (kLift + kSlack);
              }
          // ---- the base rises; `zeros`: a key's values may be all zeros
          auto raise = [&](auto zeros) {
            constexpr bool kZeros = decltype(zeros)::value;
            uint32_t some = 0;   // the warp's keys whose values are not all zeros
            float lower[2 * U] = {};   // what a key's y counts less
            if constexpr (kZeros) {
#pragma unroll
              for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  uint32_t any = v[u][i][0];
#pragma unroll
                  for (int w = 1; w < kWords; ++w) any |= v[u][i][w];
                  if (any & 0x7F7F7F7Fu) some |= 1u << (u * 16 + (i & 1 ? vb : va) + (i & 2 ? 8 : 0));
                }
              some = __reduce_or_sync(0xFFFFFFFFu, some);
#pragma unroll
              for (int i = 0; i < 2 * U; ++i)
                if (!(some >> (kg + 8 * i) & 1u)) lower[i] = ve[i] + kZeroReach;
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                float m = -INFINITY;
#pragma unroll
                for (int u = 0; u < U; ++u)
                  m = kZeros ? fmaxf(m, fmaxf(s[u][nt][j] - lower[2 * u], s[u][nt][2 + j] - lower[2 * u + 1]))
                             : fmaxf(m, fmaxf(s[u][nt][j], s[u][nt][2 + j]));
                m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 4));
                m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 8));
                m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 16));
                m = fmaxf(m - kLift, base[nt][j]);
                const float f = m == -INFINITY ? 1.f : exp2_fast(base[nt][j] - m);
                base[nt][j] = m;
                sum[nt][j] *= f;
#pragma unroll
                for (int i = 0; i < kSteps; ++i) {
                  o[nt][i][j] *= f;
                  o[nt][i][2 + j] *= f;
                }
                if constexpr (kZeros) {
                  const float b = m == -INFINITY ? 0.f : m;
#pragma unroll
                  for (int i = 0; i < 2 * U; ++i) {
                    if (some >> (kg + 8 * i) & 1u) continue;
                    float& y = s[i / 2][nt][2 * (i & 1) + j];
                    sum[nt][j] += exp2_fast(min_nan(y - ve[i] - b - kSumDrop, kZeroReach + kLift - kSumDrop));
                    y = -INFINITY;
                  }
                }
              }
          };
          if (__any_sync(0xFFFFFFFFu, over)) {
            bool large = false;   // a scale of 1 or more
#pragma unroll
            for (int i = 0; i < 2 * U; ++i) large |= ve[i] >= 0.f;
            if (__any_sync(0xFFFFFFFFu, large)) raise(std::true_type());
            else raise(std::false_type());
          }
          uint32_t p[U][NT][2];
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float e[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float b = base[nt][i & 1] == -INFINITY ? 0.f : base[nt][i & 1];
                e[i] = exp2_fast(min_nan(s[u][nt][i] - b, kMostExponent));
                sum[nt][i & 1] = fmaf(e[i], unscale[2 * u + (i >> 1)], sum[nt][i & 1]);
              }
              p[u][nt][0] = transpose8x8(pack16x2<false>(e[0], e[1]));
              p[u][nt][1] = transpose8x8(pack16x2<false>(e[2], e[3]));
            }
          // ---- a probability of 0 does not undo a NaN that it multiplies: the codes of values past the
          // last key are cleared; NaN codes of values that only some rows see are taken out, and noted for
          // the rows that do see them
          uint32_t poison = 0;
          if (edge) {
            const int32_t pair_key[4] = {va, vb, va + 8, vb + 8};
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
              for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int w = 0; w < kWords; ++w) {
                  if (key0 + u * 16 + pair_key[i] >= seg.keys) v[u][i][w] = 0;
                  poison |= nan_codes(v[u][i][w]);
                }
          }
          if (__any_sync(0xFFFFFFFFu, poison != 0)) {   // rare
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int32_t key = key0 + u * 16 + (i & 1 ? vb : va) + (i & 2 ? 8 : 0);
                uint32_t columns = 0;   // of the lane's 4 kWords
#pragma unroll
                for (int w = 0; w < kWords; ++w) {
                  const uint32_t n = nan_codes(v[u][i][w]) >> 7;   // 1 in such a byte
                  v[u][i][w] &= ~(n * 0xFFu);
                  columns |= ((n | n >> 7 | n >> 14 | n >> 21) & 15u) << (4 * w);
                }
                if (columns == 0) continue;
                sh->poisoned[turn] = 1;
                const int bit = g * (DH / 8);
#pragma unroll 1
                for (int n = 0; n < G::kPartRows; ++n) {
                  const int tok = (row0 + n) / group;
                  if (tok < seg.ntok && key < seg.first + tok)
                    atomicOr(&sh->poison[turn][part * G::kPartRows + n][bit / 32], columns << (bit % 32));
                }
              }
          }
          // ---- products with the values
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int w = 0; w < kWords; ++w) {
              const uint32_t l0 = __byte_perm(v[u][0][w], v[u][1][w], sel_lo);
              const uint32_t h0 = __byte_perm(v[u][0][w], v[u][1][w], sel_hi);
              const uint32_t l1 = __byte_perm(v[u][2][w], v[u][3][w], sel_lo);
              const uint32_t h1 = __byte_perm(v[u][2][w], v[u][3][w], sel_hi);
              const uint32_t fl[4] = {codes_lo(l0), codes_hi(l0), codes_lo(l1), codes_hi(l1)};
              const uint32_t fh[4] = {codes_lo(h0), codes_hi(h0), codes_lo(h1), codes_hi(h1)};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                mma_f16(o[nt][2 * w], fl, p[u][nt][0], p[u][nt][1]);
                mma_f16(o[nt][2 * w + 1], fh, p[u][nt][0], p[u][nt][1]);
              }
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->empty[stage]);
        if (++stage == G::kStages) { stage = 0; phase ^= 1u; }
      }

      // ---- the warps' bases, sums and outputs become one: each puts its own down and then takes a part of
      // the rows. From here on both are relative to base + kSumDrop.
      const bool whole = seg.begins() && seg.ends();
      const int64_t slot = static_cast<int64_t>(blockIdx.x) * 2 + (seg.begins() ? 1 : 0);
      constexpr float drop = 1.f / (1 << kSumDrop);
#pragma unroll
      for (int r0 = 0; r0 < G::kPartRows; r0 += G::kJoinRows) {
        if (r0 >= seg.ntok * group) break;
        named_bar_sync(1, kConsumers * 32);   // what was there has been read
        // so have the marks of the segment before, and the next one begins behind the barrier below
        if (r0 == 0 && threadIdx.x == 0 && sh->poisoned[turn ^ 1]) {
          for (int i = 0; i < G::kRows * (DH / 32); ++i) (&sh->poison[turn ^ 1][0][0])[i] = 0;
          sh->poisoned[turn ^ 1] = 0;
        }
#pragma unroll
        for (int n = 0; n < G::kJoinRows / 8; ++n) {
          const int nt = r0 / 8 + n;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float l = sum[nt][j];
            l += __shfl_xor_sync(0xFFFFFFFFu, l, 4);
            l += __shfl_xor_sync(0xFFFFFFFFu, l, 8);
            l += __shfl_xor_sync(0xFFFFFFFFu, l, 16);
            if (g == 0) sh->ml[warp][nt * 8 + 2 * t4 + j] = make_float2(base[nt][j] + kSumDrop, l);
            float* to = join + (warp * G::kJoinRows + n * 8 + 2 * t4 + j) * G::kJoinRow + g * (DH / 8);
#pragma unroll
            for (int i = 0; i < kSteps; ++i)
              *reinterpret_cast<float2*>(to + 2 * i) = make_float2(o[nt][i][j] * drop, o[nt][i][2 + j] * drop);
          }
        }
        named_bar_sync(1, kConsumers * 32);
        constexpr int kLanes = DH / 4;   // of a row
        const int col = lane % kLanes * 4;
#pragma unroll 1
        for (int at = warp * (32 / kLanes) + lane / kLanes; at < G::kParts * G::kJoinRows;
             at += kConsumers * (32 / kLanes)) {
          const int n = at / G::kParts, of = at % G::kParts;   // a row of one of the parts
          const int r = r0 + n + (kGroups == 2 ? of * G::kPartRows : 0), tok = r / group;
          if (tok >= seg.ntok) continue;
          float m = -INFINITY, l = 0.f, acc[4] = {};
#pragma unroll
          for (int w = 0; w < kConsumers; w += G::kParts) m = fmaxf(m, sh->ml[w + of][r0 + n].x);
          const float b = m == -INFINITY ? 0.f : m;
#pragma unroll
          for (int w = 0; w < kConsumers; w += G::kParts) {
            const float2 ml = sh->ml[w + of][r0 + n];
            const float4 v =
                *reinterpret_cast<const float4*>(join + ((w + of) * G::kJoinRows + n) * G::kJoinRow + col);
            const float f = exp2_fast(ml.x - b);
            l += f * ml.y;
            acc[0] += f * v.x;
            acc[1] += f * v.y;
            acc[2] += f * v.z;
            acc[3] += f * v.w;
          }
          if (sh->poisoned[turn]) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (sh->poison[turn][of * G::kPartRows + r0 + n][col / 32] >> (col % 32 + e) & 1)
                acc[e] = __uint_as_float(0x7FC00000u);
          }
          const int32_t of_token = (kHeads == 2 ? of * group : 0) + (r - tok * group);   // which of a token's rows
          if (whole) {
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const int32_t query = seg.h * a.group + of_token;
            const int64_t token = static_cast<int64_t>(seg.token0) + tok;
            if (col < a.head_dim)
              *reinterpret_cast<uint2*>(a.out + token * a.o_token + static_cast<int64_t>(query) * a.o_head + col) =
                  make_uint2(pack16x2<kBf16>(acc[0] * inv, acc[1] * inv), pack16x2<kBf16>(acc[2] * inv, acc[3] * inv));
            if (a.lse != nullptr && col == 0)
              a.lse[token * a.heads + query] = (m + log2f(l)) * 0.69314718055994531f;
          } else {
            const int64_t to = slot * G::kRows + tok * a.group + of_token;
            *reinterpret_cast<float4*>(pieces.o + to * DH + col) = make_float4(acc[0], acc[1], acc[2], acc[3]);
            if (col == 0) *reinterpret_cast<float2*>(pieces.ml + to * 2) = make_float2(m, l);
          }
        }
      }
      if (threadIdx.x == 0) attn_piece(pieces, seg);
    }
  }
  __syncwarp();
  cta_sync_all();
  if (threadIdx.x == 0) attn_report(abort, a.err);
}

template <int DH, int NT, int kHeads, int kGroups, bool kBf16>
cudaError_t launch(const AttnArgs& a, const KvFp8Part& k, const KvFp8Part& v, const CUtensorMap (&tm)[2],
                   cudaStream_t st) {
  constexpr size_t smem = smem_bytes<DH, NT, kHeads, kGroups>();
  static_assert(smem <= 232448, "shared memory");
  const auto kernel = attn_fp8_rows_kernel<DH, NT, kHeads, kGroups, kBf16>;
  const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kernel), smem);
  if (e != cudaSuccess) return e;
  return launch_ex(kernel, dim3(a.plan.workers), dim3(kThreads), smem, st, true, tm[0], tm[1], a, k, v,
                   attn_pieces_at(a.workspace, a.plan.workers, Geo<DH, NT, kHeads, kGroups>::kRows));
}

template <int NT, int kHeads, int kGroups>
cudaError_t launch_any(AttnArgs a, const KvFp8Part& k, const KvFp8Part& v, cudaStream_t st) {
  constexpr int32_t rows = 8 * NT * kHeads * kGroups;
  // An item's heads are one key-value head to the plan and to the joining kernel.
  a.plan.kv_heads /= kHeads;
  a.group *= kHeads;
  a.plan.tokens = rows / a.group;
  a.plan.workers = device_sm_count();
  a.plan.extra = kExtraUnits;
  alignas(64) CUtensorMap tm[2];
  if (!attn_fp8_tensor_maps(a, k, v, kHeads, tm)) return cudaErrorInvalidValue;
  cudaError_t e = cudaErrorInvalidValue;
  if (attn_width(a.head_dim) == 64)
    e = a.bf16 ? launch<64, NT, kHeads, kGroups, true>(a, k, v, tm, st)
               : launch<64, NT, kHeads, kGroups, false>(a, k, v, tm, st);
  else if constexpr (NT <= 3)
    e = a.bf16 ? launch<128, NT, kHeads, kGroups, true>(a, k, v, tm, st)
               : launch<128, NT, kHeads, kGroups, false>(a, k, v, tm, st);
  return e != cudaSuccess ? e : launch_attn_combine(a, rows, st);
}

}  // namespace

cudaError_t launch_attn_fp8_rows(const AttnArgs& a, const KvFp8Part& k, const KvFp8Part& v, int32_t rows,
                                 cudaStream_t st) {
  // Two key-value heads an item where they lie beside each other in memory: TMA then takes rows twice as long,
  // and memory pieces of 256 bytes. (24 caches of 100-7061 positions with 16 heads of 64: 64 us with one, 40.8
  // with two; 4 of 70001-131072 with 8 heads of 128: 161 and 144; two long caches with 16 rows 104 and 88.5.) But not
  // where even tables that are full leave SMs without a tile of one head: one token over 511 positions 8.2 us with
  // one, 8.6 with two. The lengths are on the device, so that a short cache takes two, and that time, where the
  // table has room for a long one.
  const int64_t width = attn_width(a.head_dim);
  const int64_t most = int64_t(a.plan.n_seqs) * a.plan.kv_heads * ((a.plan.kv_cap + kTileKeys - 1) / kTileKeys);
  const bool two = a.plan.kv_heads % 2 == 0 && a.head_dim == width && k.head == width && v.head == width &&
                   most > device_sm_count();
  if (rows <= 8) return two ? launch_any<1, 2, 1>(a, k, v, st) : launch_any<1, 1, 1>(a, k, v, st);
  if (rows <= 16) return two ? launch_any<2, 2, 1>(a, k, v, st) : launch_any<2, 1, 1>(a, k, v, st);
  if (rows <= 32) return launch_any<2, 1, 2>(a, k, v, st);
  // With three tiles and on tcgen05: 40 or 48 rows over two caches of 100003 and 131072 positions, 8 heads of 128, 197
  // and 212 us, over 16 of 3000-4665 in pages of 48, 4 heads, 43.4 and 46.0; 40 or 48 rows over 24 of 140-6558, 16 heads
  // of 64, f16 and bf16, 117-118, 125 and 156-158, 148. With four, of 64 columns only: 64 rows over the last ones 143,
  // 150 and 154, 148 (bf16 is as fast on either), but of 128 columns over the first ones, where registers spill more,
  // 350 and 209.
  return rows <= 48 ? launch_any<3, 1, 2>(a, k, v, st) : launch_any<4, 1, 2>(a, k, v, st);
}

}  // namespace engram

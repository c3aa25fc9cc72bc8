// Attention for items of many query rows, prompts and long chunks, on tcgen05: over keys and values of
// 16 bits (attn_tiles_sm103.cu) and over an 8-bit cache (attn_fp8_tiles_sm103.cu).
//
// An item is up to 256 rows (tokens x the query heads that share a key-value head), two row tiles
// of 128; key tiles of 128 pass by once:
//   S_t = Q_t K^T                 tcgen05.mma, both operands in shared memory, f32 in TMEM
//   P_t = 2^(c S_t - c M_t)       one thread per row, in registers; M_t the row's maximum
//   O_t = O_t + P_t V             tcgen05.mma, P_t from TMEM (it takes the place of S_t), V as it
//                                 lies: its rows are keys, so it enters transposed (MN-major)
// with c = scale log2(e). Bound by the tensor cores for heads of 128 columns: a pair of row tiles
// costs 4 * 128 * 128 * D multiply-adds there (2048 cycles an SM at D = 128) and 2 * 128 * 128
// exponentials on the special-function units (1024). So the two row tiles take turns: while the
// tensor cores work on one, the other's softmax runs. Both read the same key and value tiles.
//
// Measured (bf16, queries, keys and values in one buffer): 16384 tokens with 16 heads of 128 over
// 4 key-value heads 640-645 us, 1705-1720 TFLOP/s, 89-90% of a large library matrix product's rate;
// 8192 tokens 184-187 us (1470-1490), with heads of 64 columns 157-166 us (830-875). What bounds it
// there, at either width, is the chain from a row tile's scores through its softmax to the product
// and the next scores, of which two row tiles in turn hide most. For scores that run ahead TMEM has no
// columns left at 128; at 64 it has 128, which nothing uses yet. At 8192 tokens the tensor cores are
// busy 69% of the time (39% at 64 columns), the special-function units 35% (39%), and the schedulers
// issue in 39% (42%) of the cycles. Short prompts wait for
// instructions (2.9 stalled warps per issue against 0.3 in a long one): a worker with a handful of
// items runs through most of the kernel a few times only, out of caches that do not hold all of
// it. So loops are rolled where they do not carry the inner work, and one warp walks the work for
// all: with 90 KB of code (94 now) instead of 137 a batch of 14 prompts of 0-801 tokens took 45 us, not 55.
// It takes 43 now: 5 before the first product, 1.3 per key tile, 2.5 per item (its output 1.2-1.8).
// Tried and slower: two threads per row (the barrier between their maxima costs what the shorter
// rows save); scores in blocks of 64 keys, so that a row tile always has the next ones; an MMA warp
// per row tile; P apart from S where heads of 64 columns leave room for it; loading 32 scores while
// the exponentials of the 32 before are taken, in one piece of code with what needs all of them at
// once (9%: the compiler then schedules 32 columns at a time instead of 128) or in two (4%).
//
// The maximum that a row subtracts lags: it is only raised when a tile's probabilities against it
// sum to more than kMostSum, because finding it costs a pass over the scores and raising it means
// rescaling O in TMEM. Probabilities are then up to 512 instead of 1, which f32 sums and both 16-bit
// types hold as exactly, and the result is the same quotient. f16, whose values end at 2^-24, gets
// them another 2^6 larger (kLift), which fills its range: 2^-30 of the largest one is still there.
//
// Roles (384 threads): warps 0-3 and 4-7 softmax and output of row tile 0 and 1 (thread = row =
// TMEM lane); warp 8 issues the MMAs; warp 9 requests key and value tiles by TMA (one page granule
// per lane), warp 10 each item's queries (a box of its tokens by the heads that share its key-value
// head is the item's rows in order, whatever their number); warps 10-11 make the values that some
// row of the item must not see harmless (below). Registers: the softmax warps hold a row of 128
// scores, so they take 192 each and the other four 120.
//
// Over an 8-bit cache there are four warps more, 12-15: TMA brings codes (warp 9; the scales by warp 11), and
// they write them out as 16-bit tiles times their scales, through registers, with the work of warps 10-11 below
// done on the way. All else is the same; so a call takes what it would over 16 bits (378 us for a chunk of 2047 over
// 30000 positions, 16 heads of 128 over 4, f16, on keys of these sizes; 160 for chunks of 1024 and 300 beside six
// single tokens) and 7-18% more: 447 and 171. (On keys of one size, whose maxima hardly grow, 316 and 398, 128 and 166.)
// Registers spill a little: 72 bytes a thread stored and 116 loaded in f16 with 128 columns, 40 and 92 in bf16. What the conversion costs: 64 KB written and 32 read per pair of
// tiles in shared memory, where the MMAs take their operands (without any stores 409 us instead of 468, without
// any arithmetic 389, without the conversion 358), issue slots beside the softmax, and the room of its instructions
// beside the softmax's: its loop takes one row of a team of lanes at a time (with batches of two and of four rows the
// mixed chunks take 176 and 183 us, with twice four unrolled 220, with half a row 203). Not faster: bf16 codes put in
// place bit by bit, three tiles' room for codes and four for tiles, keys and values requested by a warp each (10%
// slower) or converted by two warps each (467 and 199 us), the next row's codes or scale fetched a turn ahead
// (187, 180). Items of one row tile with the even key tiles in one half of the softmax warps and the odd ones in the
// other: 16 chunks of 128 rows 42 us instead of 44.5, but the mixed chunks 10 us more.
//
// A probability of 0 does not undo an infinity or NaN that it multiplies. In the tiles that reach
// past what the item's first row sees, warps 10-11 clear the value rows that no row sees (another
// sequence's, or memory that was never written) and replace infinities and NaN in the others by
// 0; if they replaced any, the rows that do see them get them added at the end, each times the key's
// probability, formed once more: where that has underflowed, the product is NaN, as in a tile that
// every row sees.
#pragma once

#include "attn_device.cuh"
#include "kernels.h"
#include "kv_fp8.cuh"
#include "wkv_tiles.cuh"

namespace engram {

namespace {

// Where keys and values come from: tensors of 16 bits, or an 8-bit cache.
struct Kv16 {
  static constexpr bool kFp8 = false;
};
struct KvFp8 {
  static constexpr bool kFp8 = true;
  KvFp8Part k, v;
};

constexpr int kSoftmaxWarps = 8;
constexpr int kConvertWarps = 4;             // of an 8-bit cache
template <class Kv>
constexpr int kThreads = (kSoftmaxWarps + 4 + (Kv::kFp8 ? kConvertWarps : 0)) * 32;
constexpr int kTileRows = 128;
constexpr int kItemRows = kAttnItemRows;   // two row tiles
// 256 * 192 + 128 * 120 = 384 * 168. With 176 + 152 the softmax warps spill, with 208 + 88 the others
// do: the prompt of 16384 tokens takes 676, 641, 658 us.
// 256 * 184 + 256 * 72 = 512 * 128 with the four warps more that an 8-bit cache takes, 176 + 80 in bf16, whose
// conversion takes more: chunks of 1024 and 300 tokens beside six single ones, bf16, 185, 172, 169, 173 us with 192,
// 184, 176, 168, a chunk of 2047 over 30000, f16, 455, 449, 459, 478.
template <bool kBf16, class Kv>
constexpr int kSoftmaxRegs = !Kv::kFp8 ? 192 : kBf16 ? 176 : 184;
template <bool kBf16, class Kv>
constexpr int kOtherRegs = !Kv::kFp8 ? 120 : kBf16 ? 80 : 72;
constexpr int kSegments = 4;                 // in the ring from warp 9 to the others
template <class Kv>
constexpr int kSegmentReaders = kSoftmaxWarps + 3 + (Kv::kFp8 ? kConvertWarps : 0);
constexpr int kPoisonSlots = 8;
// Of a tile's probabilities against an older maximum. With 1, where nearly every tile looks for its
// maximum, the prompt of 16384 tokens took 1093 us instead of 661.
constexpr float kMostSum = 512.f;
// Over an 8-bit cache in bf16, whose keys' sizes differ more from row to row in the cases measured. With 512 a
// quarter of the tiles find their maximum: chunks of 1024 and 300 tokens beside six single ones 203 us; with this and
// the lift below, where hardly any does, 171 (a chunk of 512 over 16000 positions 96 and 81; on keys of one size
// 165 and 166, 78 and 79). A tile adds up to 2^16 times its largest value to an
// output's sum, which is finite for values up to 2^99 over 2^12 tiles, and 2^88 over 2^23, all that there may be.
constexpr float kMostSumFp8 = 65536.f;
// Probabilities are rounded to the values' type for the product with them, since the MMA takes both
// operands in one 16-bit type: each by half a unit in its last place, as the result is at the end.
// They are summed as they are, so what rounding takes from a small one is lost, and a long cache may
// hold much weight in keys that f16 has no value for beside 1. So they are 2^kLift times larger there,
// kMostSum of it below f16's largest value. bf16 has the exponents of f32.
// (With an 8-bit cache they are lowered instead: a maximum may grow by 2^40 before it is found anew, and
// products with values down to 2^-100 are normal numbers still.)
template <bool kBf16, class Kv>
constexpr float kLift = !kBf16 ? 6.f : Kv::kFp8 ? -24.f : 0.f;
template <bool kBf16, class Kv>
constexpr float kMostLifted = !kBf16 ? kMostSum * 64.f : Kv::kFp8 ? kMostSumFp8 : kMostSum;
// The maximum is subtracted in the multiply-add that scales a score, so the rounding of its product stays in
// the difference: from here on (2^24 in units of log2) it is subtracted first.
constexpr float kFarScore = 16777216.f;
// Tiles of an item whose maximum is found at once: among the first ones it grows, and taking exponentials twice
// costs more. (f16 over an 8-bit cache, where it may grow by no more than kSpare, 2^14 with the lift. With 1, 8, 32:
// 16 chunks of 128 rows over 3000-4665 positions 50.0, 47.9, 45.2 us, chunks of 1024 and 300 tokens beside single ones
// 191, 187, 180, one of 512 over 16000 91, 89, 81, of 2047 over 30000 459, 459, 448, and with all of them 463. Keys of
// one size, whose maxima hardly grow, want few: the mixed chunks 150, 152, 163, the last one 391, 393, 398.)
template <bool kBf16, class Kv>
constexpr int kYoung = Kv::kFp8 && !kBf16 ? 32 : 1;
constexpr float kSpare = 8.f;
// An item's fixed time in key tiles: fetching its queries, filling the pipeline, writing its rows.
// With 1, 2, 3: a prompt of 8192 tokens 210, 194, 194 us, 14 prompts of 0-801 tokens 45.8, 44.5,
// 46.3, chunks of 1024 and 300 tokens beside six single ones 151, 133, 137.
constexpr int kExtraUnits = 2;

template <int DH, class Kv>
struct Geo {
  static constexpr int kHalves = DH / 64;
  static constexpr int kTileBytes = 128 * DH * 2;            // a tile of Q, K or V
  static constexpr int kStages = Kv::kFp8 ? (DH == 128 ? 3 : 6)
                                          : (DH == 128 ? 5 : 10);   // of one K or V tile each: as many
                                                             // as fit (3 / 6 are as fast)
  static constexpr int kCodeBytes = 128 * DH;                // a tile of K or V in eight bits
  static constexpr int kCodeStages = Kv::kFp8 ? (DH == 128 ? 4 : 8) : 0;
  static constexpr uint32_t kO = 256;                        // TMEM columns: S0 S1 O0 O1
};

template <int kCodes>
struct CodeRing {
  uint64_t code_full[kCodes], code_empty[kCodes];
  uint8_t scales[kCodes][kTileKeys];
};
template <>
struct CodeRing<0> {};

template <int DH, class Kv>
struct alignas(16) Shared : CodeRing<Geo<DH, Kv>::kCodeStages> {
  static constexpr int kStages = Geo<DH, Kv>::kStages;
  static constexpr int kGuards = Kv::kFp8 ? kConvertWarps : 2;
  uint64_t full[kStages], empty[kStages], vok[kStages];
  uint64_t qfull, qempty, sfull[2], pfull[2], ofull[2];
  uint64_t drain;
  uint64_t seg_full[kSegments], seg_empty[kSegments];
  AttnSegment seg[kSegments];
  AttnStart start;
  int poison[kGuards][kPoisonSlots];   // of warps 10 and 11 (12-15), by segment
  uint32_t tmem_base;
  int abort;
};

template <int DH, class Kv>
constexpr size_t smem_bytes() {
  using G = Geo<DH, Kv>;
  return 1024 + size_t(2 + G::kStages) * G::kTileBytes + size_t(G::kCodeStages) * G::kCodeBytes +
         sizeof(Shared<DH, Kv>);
}

// Instruction descriptor: f32 accumulator, A and B bf16 or f16, B K-major or (transposed)
// MN-major.
template <bool kBf16>
constexpr uint32_t idesc(int M, int N, bool b_mn) {
  return (1u << 4) | ((kBf16 ? 1u : 0u) << 7) | ((kBf16 ? 1u : 0u) << 10) |
         ((b_mn ? 1u : 0u) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

// The MMA warp runs converged and lets one lane issue, chosen by elect.sync: descriptors that are
// the same in every lane then come from uniform registers. (Issued from a branch that lane 0 takes
// alone, an MMA took 70 cycles to issue, and the issue, not the tensor cores, set the pace.)
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xFFFFFFFFu, v, 0); }

// Low and high words of a shared-memory descriptor: the low one holds the address (in 16-byte
// units, 14 bits) and the leading offset, the high one stride, version and swizzle.
__device__ __forceinline__ uint64_t desc_of(uint32_t lo) {
  constexpr uint32_t hi = (1024u >> 4) | (1u << 14) | (2u << 29);
  return (static_cast<uint64_t>(hi) << 32) | lo;
}
// K-major tile with the 128-byte swizzle (rows of 64 elements, 8-row groups 1 KB apart).
__device__ __forceinline__ uint32_t kmajor_lo(uint32_t saddr) {
  return ((saddr & 0x3FFFFu) >> 4) | ((16u >> 4) << 16);
}
// The same tile read MN-major: its rows are K (keys); boxes of 128 rows by 64 columns 16 KB apart.
__device__ __forceinline__ uint32_t mnmajor_lo(uint32_t saddr) {
  return ((saddr & 0x3FFFFu) >> 4) | (((128u * 128u) >> 4) << 16);
}

__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(r));
  return r != 0;
}

// D[tmem] (+)= A[tmem] * B[smem], A 16-bit pairs in 32-bit columns.
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bd, uint32_t id,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bd), "r"(id), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tc_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tc_st_32x32b_x32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(
          r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
      "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31]), "r"(taddr)
      : "memory");
}
// One column: a value per lane.
__device__ __forceinline__ uint32_t tc_ld_32x32b_x1(uint32_t taddr) {
  uint32_t r;
  __syncwarp();
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=r"(r)
      : "r"(taddr)
      : "memory");
  return r;
}
__device__ __forceinline__ void tc_st_32x32b_x1(uint32_t taddr, uint32_t v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(v) : "memory");
}
__device__ __forceinline__ void tc_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Two multiply-adds or adds per instruction.
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Four lanes transpose their four 16-byte pieces: lane q's piece v becomes lane v's piece q.
__device__ __forceinline__ void exchange4(uint32_t (&w)[4][4], int own) {
#pragma unroll
  for (int mask = 1; mask < 4; mask <<= 1)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      if (v & mask) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool up = own & mask;
        const uint32_t got =
            __shfl_xor_sync(0xFFFFFFFFu, up ? w[v][e] : w[v | mask][e], mask);
        w[v][e] = up ? got : w[v][e];
        w[v | mask][e] = up ? w[v | mask][e] : got;
      }
    }
}

// Key row (`values` false) or value row of position `pos`, for the rare rows that see an infinity or
// NaN; null: the position's page number is not the cache's, its row reads as zeros.
__device__ __forceinline__ const uint16_t* kv_row(const AttnArgs& a, const AttnSegment& s,
                                                  bool values, int32_t pos) {
  const uint16_t* p = values ? a.v : a.k;
  const int64_t token = values ? a.v_token : a.k_token, head = values ? a.v_head : a.k_head;
  if (a.table == nullptr) return p + (int64_t(s.q0) + pos) * token + s.h * head;
  const int32_t col = pos / a.page_size;
  const int32_t page = a.table[int64_t(s.b) * a.table_width + col];
  if (page < 0 || page >= a.n_pages) return nullptr;
  return p + page * (values ? a.v_page : a.k_page) + (pos - int64_t(col) * a.page_size) * token +
         s.h * head;
}

__device__ __forceinline__ uint2 lds64(uint32_t saddr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(saddr) : "memory");
  return v;
}

// Warp-wide: rows [first, first + 32) of a tile of codes (rows of DH bytes with the swizzle of that width) to a
// tile of 16 bits (64-column boxes with the 128-byte swizzle). Value rows from `end` on become zeros, and in
// those from `guard` on a NaN does: returns whether this lane has taken one out.
template <int DH, bool kBf16>
__device__ __forceinline__ bool convert_tile(uint32_t codes, const uint8_t* scales, uint32_t tile, int first,
                                             int32_t end, int32_t guard, bool values) {
  constexpr int kChunks = DH / 16, kAtOnce = 32 / kChunks;   // 16-byte chunks of a row, rows at a time
  const int lane = threadIdx.x & 31, c = lane % kChunks, in = lane / kChunks;
  // A lane takes chunk c of a row as two halves, each 8 codes in and 16 bytes out. Of 128 columns the
  // lanes of the second box begin with the second half, so that eight lanes meet every bank once.
  const int flip = DH == 128 && c >= 4;
  auto from = [&](int r, int half) {
    return codes + r * DH + ((DH == 128 ? c ^ (r & 7) : c ^ (r >> 1 & 3)) << 4) + (half ^ flip) * 8;
  };
  auto to = [&](int r, int half) {
    return tile + (c >> 2) * (kTileKeys * 128) + r * 128 + ((((2 * c & 7) + (half ^ flip)) ^ (r & 7)) << 4);
  };
  const uint32_t own = first + lane < end ? scales[first + lane] : 127u;   // of row `lane`
  if (__all_sync(0xFFFFFFFFu, is_fast<kBf16>(own))) {
    // kAtOnce rows further a 128-byte swizzle has its third bit the other way round, the others are as they were
    uint32_t at[2], put[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      at[h] = from(first + in, h);
      put[h] = to(first + in, h);
    }
    const uint32_t scale = fast_scale<kBf16>(own);
    const bool edge = values && (first + 32 > end || first + 32 > guard);   // the same for all lanes
    uint32_t bad = 0;
#pragma unroll 1
    for (int i = 0; i < 32; i += kAtOnce) {
      uint2 w[2] = {lds64(at[0]), lds64(at[1])};
#pragma unroll
      for (int h = 0; h < 2; ++h) at[h] = (DH == 128 ? at[h] ^ 64u : at[h]) + kAtOnce * DH;
      const uint32_t s = __shfl_sync(0xFFFFFFFFu, scale, in + i);
      if (edge) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (first + in + i >= end) w[h] = make_uint2(0, 0);
          bad |= nan_codes(w[h].x) | nan_codes(w[h].y);
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint4 x;
        scaled16x4<kBf16>(w[h].x, s, x.x, x.y);
        scaled16x4<kBf16>(w[h].y, s, x.z, x.w);
        sts128(put[h], x);
        put[h] = (DH == 128 ? put[h] ^ 64u : put[h]) + kAtOnce * 128;
      }
    }
    if (!__any_sync(0xFFFFFFFFu, bad != 0)) return false;
  }
  bool taken = false;
#pragma unroll 1
  for (int r = first + in; r < first + 32; r += kAtOnce)
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
      const uint2 q = lds64(from(r, h));
      uint32_t w[2] = {q.x, q.y}, byte = scales[r];
      if (r >= end) {
        byte = 127;
        if (values) w[0] = w[1] = 0;
      } else if (r >= guard) {   // some rows must not see it
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t bad = byte == kNanScale ? 0x80808080u : nan_codes(w[e]);
          taken |= bad != 0;
          w[e] &= ~((bad >> 7) * 0xFFu);
        }
        if (byte == kNanScale) byte = 127;
      }
      const float scale = fp8_scale_value(byte);
      sts128(to(r, h), make_uint4(scaled16x2<kBf16>(w[0], scale), scaled16x2<kBf16>(w[0] >> 16, scale),
                                  scaled16x2<kBf16>(w[1], scale), scaled16x2<kBf16>(w[1] >> 16, scale)));
    }
  return taken;
}

// Adds to `columns` those in which the value row of position `pos` is NaN.
template <int N>
__device__ __forceinline__ void fp8_nan_columns(const AttnArgs& a, const KvFp8Part& v, const AttnSegment& s,
                                                int32_t pos, uint32_t (&columns)[N]) {
  const KvPlace at = kv_place(a, s, pos);
  if (at.w >= a.n_pages) return;
  const bool all = v.scales[at.w * v.scale_page + s.h * v.scale_head + at.z] == kNanScale;
  const uint8_t* row = v.codes + at.w * v.page + at.z * v.slot + s.h * v.head;
#pragma unroll
  for (int w = 0; w < N; ++w)
#pragma unroll 1
    for (int d = 0; d < 32 && w * 32 + d < a.head_dim; ++d)
      if (all || (row[w * 32 + d] & 0x7F) == 0x7F) columns[w] |= 1u << d;
}

template <int DH, bool kBf16, class Kv>
__global__ void __launch_bounds__(kThreads<Kv>, 1)
    attn_tiles_kernel(const __grid_constant__ CUtensorMap tmQ,
                      const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV,
                      const __grid_constant__ AttnArgs a, const AttnPieces pieces,
                      const __grid_constant__ Kv source) {
  using G = Geo<DH, Kv>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_1024(smem_raw);
  uint8_t* sQ = smem;                       // 64-column boxes of 256 rows
  uint8_t* sKV = smem + 2 * G::kTileBytes;
  uint8_t* sCodes = sKV + G::kStages * G::kTileBytes;
  Shared<DH, Kv>* sh = reinterpret_cast<Shared<DH, Kv>*>(sCodes + G::kCodeStages * G::kCodeBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < G::kStages; ++s) {
      mbar_init(&sh->full[s], Kv::kFp8 ? kConvertWarps : 1);
      mbar_init(&sh->empty[s], Kv::kFp8 ? 1 : 3);   // the MMAs that read it, and warps 10 and 11
      if constexpr (!Kv::kFp8) mbar_init(&sh->vok[s], 2);
    }
    if constexpr (Kv::kFp8)
      for (int s = 0; s < G::kCodeStages; ++s) {
        mbar_init(&sh->code_full[s], 1 + 32);   // the codes, and each lane's scales
        mbar_init(&sh->code_empty[s], kConvertWarps);
      }
    mbar_init(&sh->qfull, 1);
    mbar_init(&sh->qempty, 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sh->sfull[t], 1);
      mbar_init(&sh->pfull[t], 4);   // a lane of each warp
      mbar_init(&sh->ofull[t], 1);
    }
    mbar_init(&sh->drain, 1);
    for (int i = 0; i < kSegments; ++i) {
      mbar_init(&sh->seg_full[i], 1);
      mbar_init(&sh->seg_empty[i], kSegmentReaders<Kv>);
    }
    sh->abort = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == 8) {
    tmem_alloc(&sh->tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  pdl_wait();   // queries, lengths and the cache may come from the previous kernel
  pdl_launch_dependents();
  attn_find_start<kThreads<Kv>>(a.plan, blockIdx.x, &sh->start, a.err);   // synchronises the CTA
  tc_fence_after();
  const uint32_t tmem = sh->tmem_base;
  volatile int* abort = &sh->abort;
  // Warp 9 walks the worker's segments and passes them on through a ring (each role walking them for
  // itself is more code than the instruction cache has room for); one without pieces ends them.
  uint32_t seg_at = 0, seg_phase = 0;
  auto next_segment = [&]() {
    const bool ok = attn_wait(&sh->seg_full[seg_at], seg_phase, abort);
    return !__any_sync(0xFFFFFFFFu, !ok) && sh->seg[seg_at].pieces != 0;
  };
  auto segment_done = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh->seg_empty[seg_at]);
    if (++seg_at == kSegments) {
      seg_at = 0;
      seg_phase ^= 1u;
    }
  };

  // The item's rows, once the MMAs have read the last ones.
  auto request_queries = [&](const AttnSegment& seg, uint32_t& q_phase, uint32_t& q_loads) {
    const bool ok = !__any_sync(0xFFFFFFFFu, !attn_wait(&sh->qempty, q_phase ^ 1u, abort));
    q_phase ^= 1u;
    if (ok && lane == 0) {
      ++q_loads;
      mbar_arrive_expect_tx(&sh->qfull, static_cast<uint32_t>(a.plan.tokens * a.group) * 128 * G::kHalves);
#pragma unroll
      for (int hf = 0; hf < G::kHalves; ++hf)
        tma_load_4d(sQ + hf * (kItemRows * 128), &tmQ, &sh->qfull, hf * 64, seg.h * a.group, seg.token0, 0);
    }
    __syncwarp();
  };

  if (warp < 8) {
    // ------------------------------------------------------------- softmax and output
    set_max_regs_up<kSoftmaxRegs<kBf16, Kv>>();
    const int t = warp >> 2;
    const int32_t row = t * kTileRows + (warp & 3) * 32 + lane;   // of the item
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lanes + t * 128, tO = tmem + lanes + G::kO + t * DH;
    const float c = a.scale_log2;
    const int32_t tok = row / a.group, sub = row - tok * a.group;
    uint32_t s_phase = 0, o_phase = 0, count = 0;
    if (threadIdx.x == 0) attn_no_pieces(pieces);
#pragma unroll 1
    for (; next_segment(); segment_done()) {
      const AttnSegment& seg = sh->seg[seg_at];
      if (threadIdx.x == 0) attn_piece(pieces, seg);
      const bool tiles = seg.keys > 0;
      const uint32_t slot8 = count % kPoisonSlots;
      if (tiles) ++count;
      if (t * kTileRows >= seg.ntok * a.group) continue;   // this row tile is empty
      const bool valid = tok < seg.ntok;
      const int32_t lim = seg.first + tok;
      const int32_t limit = valid && lim > 0 ? lim : 0;
      float m = -INFINITY, l = 0.f;
      bool far = false;   // some row of the warp has its maximum beyond kFarScore (8-bit cache)
      if (tiles) {
#pragma unroll 1
        for (int32_t j = seg.tile0; j < seg.tile1; ++j) {
          attn_wait(&sh->sfull[t], s_phase, abort);
          s_phase ^= 1u;
          tc_fence_after();
          uint32_t s[4][32];
#pragma unroll
          for (int i = 0; i < 4; ++i) tc_ld_32x32b_x32(tS + i * 32, s[i]);
#pragma unroll
          for (int i = 0; i < 4; ++i) tc_wait_ld(s[i]);
          const int32_t left = limit - j * kTileKeys;   // keys of the tile that this row sees
          if (__any_sync(0xFFFFFFFFu, left < kTileKeys)) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (i * 32 + e >= left) s[i][e] = 0xFF800000u;   // -infinity
          }
          // The maximum of a row's first tile is found first. Later tiles rarely raise it: their
          // exponentials are taken against the one that is there, and only if their sum says that
          // some were far above it (or nothing had been seen), the maximum is found after all, O
          // and l are scaled down to it and the exponentials taken again.
          bool fresh = kYoung<kBf16, Kv> > 1 ? j < seg.tile0 + kYoung<kBf16, Kv> || far : j == seg.tile0 || far;
          float sums;
#pragma unroll 1
          for (;;) {
            if (fresh) {
              float mt[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
              for (int e = 0; e < 32; e += 2)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  mt[i] = max3(mt[i], __uint_as_float(s[i][e]), __uint_as_float(s[i][e + 1]));
              float top = fmaxf(m, fmaxf(fmaxf(mt[0], mt[1]), fmaxf(mt[2], mt[3])));
              // The old maximum will do where no row's has grown by much.
              if (kYoung<kBf16, Kv> > 1 && j > seg.tile0 && !far &&
                  !__any_sync(0xFFFFFFFFu, m == -INFINITY ? top > m : (top - m) * c > kSpare))
                top = m;
              else if (j > seg.tile0) {
                // The score MMA that this tile waited for came after the last product with V, so
                // O is at rest.
                const float f = m == -INFINITY ? 0.f : exp2_fast((m - top) * c);
                l *= f;
#pragma unroll 1
                for (int i = 0; i < DH / 32; ++i) {
                  uint32_t o[32];
                  tc_ld_32x32b_x32(tO + i * 32, o);
                  tc_wait_ld(o);
#pragma unroll
                  for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                  tc_st_32x32b_x32(tO + i * 32, o);
                }
              }
              m = top;
              if constexpr (Kv::kFp8) {
                far = __any_sync(0xFFFFFFFFu, fabsf(m * c) > kFarScore && m > -INFINITY);
                if (far)
#pragma unroll
                  for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                      s[i][e] = __float_as_uint(__uint_as_float(s[i][e]) - (m == -INFINITY ? 0.f : m));
              }
            }
            const float base = m == -INFINITY ? 0.f : far ? kLift<kBf16, Kv> : fmaf(-m, c, kLift<kBf16, Kv>);
            const uint64_t c2 = pair(c, c), b2 = pair(base, base);
            uint64_t sum[4] = {};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t p[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                float x, y;
                unpair(fma2(pair(__uint_as_float(s[i][2 * e]), __uint_as_float(s[i][2 * e + 1])),
                            c2, b2),
                       x, y);
                x = exp2_fast(x);
                y = exp2_fast(y);
                sum[e & 3] = add2(sum[e & 3], pair(x, y));
                p[e] = pack16x2<kBf16>(x, y);
              }
              tc_st_32x32b_x16(tS + i * 16, p);
            }
            float x, y;
            unpair(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), x, y);
            sums = x + y;
            if (fresh || !__any_sync(0xFFFFFFFFu, sums > kMostLifted<kBf16, Kv> || (m == -INFINITY && left > 0)))
              break;
            fresh = true;
          }
          tc_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh->pfull[t]);
          l += sums;
        }
        attn_wait(&sh->ofull[t], o_phase, abort);
        o_phase ^= 1u;
        tc_fence_after();
      }
      const bool whole = seg.begins() && seg.ends();
      const float inv = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
      const int32_t head = seg.h * a.group + sub;
      const int64_t slot =
          (static_cast<int64_t>(blockIdx.x) * 2 + (seg.begins() ? 1 : 0)) * kItemRows + row;
      auto found = [&](int part) { return *static_cast<volatile int*>(&sh->poison[part][slot8]); };
      const bool poison = tiles && (Kv::kFp8 ? found(0) | found(1) | found(2) | found(3) : found(0) | found(1)) != 0;
      // Rows leave in pieces of 16 bytes that four lanes exchange, so that each store writes 64
      // bytes of a row: the lane's own row, and those of its three neighbours.
      const int64_t place = !valid ? -1
                            : whole ? static_cast<int64_t>(seg.token0 + tok) * a.o_token +
                                          static_cast<int64_t>(head) * a.o_head
                                    : slot * DH;
      int64_t to[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        to[e] = __shfl_sync(0xFFFFFFFFu, place, (lane & ~3) + e);
      const int own = lane & 3;
      uint32_t nan_columns[DH / 32] = {};   // of an 8-bit cache
      if constexpr (Kv::kFp8) {
        if (poison) {   // rare: the NaN that warps 12-15 took out
          const int32_t k1 = limit < seg.tile1 * kTileKeys ? limit : seg.tile1 * kTileKeys;
#pragma unroll 1
          for (int32_t k = seg.first > seg.tile0 * kTileKeys ? seg.first : seg.tile0 * kTileKeys; k < k1; ++k)
            fp8_nan_columns(a, source.v, seg, k, nan_columns);
        }
      } else if (poison) {   // rare: what warps 10-11 took out goes back to the rows that see it
        const int32_t k0 = seg.first > seg.tile0 * kTileKeys ? seg.first
                                                                  : seg.tile0 * kTileKeys;
        const int32_t k1 = limit < seg.tile1 * kTileKeys ? limit : seg.tile1 * kTileKeys;
        const int32_t end = seg.keys < seg.tile1 * kTileKeys ? seg.keys : seg.tile1 * kTileKeys;
        const float base = m == -INFINITY ? 0.f : fmaf(-m, c, kLift<kBf16, Kv>);
        const uint16_t* q = a.q + static_cast<int64_t>(seg.token0 + tok) * a.q_token +
                            static_cast<int64_t>(head) * a.q_head;
        // 32 keys at a time, the same for all rows: which of them hold such values, and which of those
        // have no probability left, are found once, not once per column
#pragma unroll 1
        for (int32_t from = k0; from < end; from += 32) {
          uint32_t found = 0, gone = 0;
#pragma unroll 1
          for (int32_t k = from; k < from + 32 && k < k1; ++k) {
            const uint16_t* v = kv_row(a, seg, true, k);
            uint32_t any = 0;
#pragma unroll 1
            for (int d = 0; v != nullptr && d < a.head_dim; d += 8) {
              const uint4 w = *reinterpret_cast<const uint4*>(v + d);
              any |= nonfinite_bits<kBf16>(w.x) | nonfinite_bits<kBf16>(w.y) |
                     nonfinite_bits<kBf16>(w.z) | nonfinite_bits<kBf16>(w.w);
            }
            if (any == 0) continue;
            const uint16_t* key = kv_row(a, seg, false, k);
            float s = 0.f;
#pragma unroll 1
            for (int d = 0; d < a.head_dim; d += 2) {
              const uint32_t x = *reinterpret_cast<const uint32_t*>(q + d);
              const uint32_t y = *reinterpret_cast<const uint32_t*>(key + d);
              s += to_f32<kBf16>(static_cast<uint16_t>(x)) * to_f32<kBf16>(static_cast<uint16_t>(y));
              s += to_f32<kBf16>(static_cast<uint16_t>(x >> 16)) *
                   to_f32<kBf16>(static_cast<uint16_t>(y >> 16));
            }
            const uint32_t p = pack16x2<kBf16>(exp2_fast(fmaf(s, c, base)), 0.f);
            found |= 1u << (k - from);
            if (!(to_f32<kBf16>(static_cast<uint16_t>(p)) > 0.f)) gone |= 1u << (k - from);
          }
          if (!__any_sync(0xFFFFFFFFu, found != 0)) continue;
#pragma unroll 1
          for (int col = 0; col < a.head_dim; ++col) {
            uint32_t o = tc_ld_32x32b_x1(tO + col);
#pragma unroll 1
            for (uint32_t left = found; left != 0; left &= left - 1) {
              const int k = __ffs(left) - 1;
              const float x = to_f32<kBf16>(kv_row(a, seg, true, from + k)[col]);
              if (!(fabsf(x) < INFINITY))
                o = __float_as_uint(__uint_as_float(o) + (gone >> k & 1u ? x * 0.f : x));
            }
            __syncwarp();
            tc_st_32x32b_x1(tO + col, o);
          }
          tc_wait_st();
        }
      }
      // 32 columns at a time; 16 bytes of a row are 8 results or 4 sums
#pragma unroll 1
      for (int i = 0; i < DH; i += 32) {
        uint32_t o[32];
        tc_ld_32x32b_x32(tO + i, o);
        tc_wait_ld(o);
        if constexpr (Kv::kFp8) {
          if (poison) {
            uint32_t mine = 0;
#pragma unroll
            for (int w = 0; w < DH / 32; ++w)
              if (w * 32 == i) mine = nan_columns[w];
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (mine >> e & 1) o[e] = 0x7FC00000u;
          }
        }
        if (whole) {
          uint32_t w[4][4];
#pragma unroll
          for (int v = 0; v < 4; ++v)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[v][e] = tiles ? pack16x2<kBf16>(__uint_as_float(o[8 * v + 2 * e]) * inv,
                                                __uint_as_float(o[8 * v + 2 * e + 1]) * inv)
                              : 0u;
          exchange4(w, own);
          const int col = i + own * 8;
#pragma unroll
          for (int v = 0; v < 4; ++v)
            if (to[v] >= 0 && col < a.head_dim)
              *reinterpret_cast<uint4*>(a.out + to[v] + col) =
                  make_uint4(w[v][0], w[v][1], w[v][2], w[v][3]);
        } else {
#pragma unroll 1
          for (int q = 0; q < 2; ++q) {
            uint32_t w[4][4];
#pragma unroll
            for (int v = 0; v < 4; ++v)
#pragma unroll
              for (int e = 0; e < 4; ++e) w[v][e] = o[4 * v + e];
            exchange4(w, own);
#pragma unroll
            for (int v = 0; v < 4; ++v)
              if (to[v] >= 0)
                *reinterpret_cast<uint4*>(pieces.o + to[v] + i + q * 16 + own * 4) =
                    make_uint4(w[v][0], w[v][1], w[v][2], w[v][3]);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = o[e + 16];   // the other 16 sums
          }
        }
      }
      tc_fence_before();   // the next product into O follows this thread's next P
      if (valid) {
        const float base = fmaf(m, c, -kLift<kBf16, Kv>);   // of the exponentials
        if (!whole)
          *reinterpret_cast<float2*>(pieces.ml + slot * 2) = make_float2(base, l);
        else if (a.lse != nullptr)
          a.lse[static_cast<int64_t>(seg.token0 + tok) * a.heads + head] =
              (base + log2f(l)) * 0.69314718055994531f;
      }
      __syncwarp();
    }
  } else {
    set_max_regs_down<kOtherRegs<kBf16, Kv>>();
    if (warp == 8) {
      // ----------------------------------------------------------- MMA issuer
      constexpr uint32_t kIdS = idesc<kBf16>(128, 128, false), kIdO = idesc<kBf16>(128, DH, true);
      uint32_t stage = 0, phase = 0;           // next K or V tile
      uint32_t vphase = 0;                     // per stage: parity of its next vok
      uint32_t q_phase = 0, p_phase[2] = {0, 0};
      const uint32_t td = uniform(tmem);
      const uint32_t q_lo = uniform(kmajor_lo(smem_u32(sQ))), kv = uniform(smem_u32(sKV));
      // After a wait that gave up, the warp still runs to its end, on whatever shared memory holds.
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        attn_wait(bar, parity, abort);
        tc_fence_after();
      };
      // Scores of a key tile. `done`: for its last reader; `last`: the item's last key tile.
      auto scores = [&](int t, uint32_t ks, bool done, bool last) {
        const uint32_t k_lo = kmajor_lo(kv + ks * G::kTileBytes);
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < DH / 16; ++kk)
            tc_mma_bf16(td + t * 128,
                        desc_of(q_lo + ((t * kTileRows + (kk >> 2) * kItemRows) * 128 >> 4) +
                                2 * (kk & 3)),
                        desc_of(k_lo + ((kk >> 2) * kTileKeys * 128 >> 4) + 2 * (kk & 3)), kIdS,
                        kk != 0);
          tc_commit(&sh->sfull[t]);
          if (done) tc_commit(&sh->empty[ks]);
          if (done && last) tc_commit(&sh->qempty);
        }
        __syncwarp();
      };
#pragma unroll 1
      for (; next_segment(); segment_done()) {
        const AttnSegment& seg = sh->seg[seg_at];
        if (seg.keys == 0) continue;
        const bool two = uniform(seg.ntok * a.group > kTileRows) != 0;
        const int32_t n = uniform(seg.tile1 - seg.tile0);
        const int32_t j_guard =   // from this tile on, warps 10-11 look at the values first
            uniform((seg.first > 0 ? seg.first : 0) / kTileKeys - seg.tile0);
        wait(&sh->qfull, q_phase);
        q_phase ^= 1u;
        wait(&sh->full[stage], phase);
        scores(0, stage, !two, n == 1);
        if (two) scores(1, stage, true, n == 1);
        if (++stage == G::kStages) { stage = 0; phase ^= 1u; }
#pragma unroll 1
        for (int32_t j = 0; j < n; ++j) {
          const uint32_t vs = stage, vph = phase;
          if (++stage == G::kStages) { stage = 0; phase ^= 1u; }
          const uint32_t ks = stage, kph = phase;
          const bool more = j + 1 < n;
          const uint32_t v_lo = mnmajor_lo(kv + vs * G::kTileBytes);
          // what was requested long ago first, so that nothing else stands between P and its MMAs
          if (!Kv::kFp8 && j >= j_guard) {
            wait(&sh->vok[vs], (vphase >> vs) & 1u);
            vphase ^= 1u << vs;
          } else {
            wait(&sh->full[vs], vph);
          }
          auto tile = [&](int t) {
            wait(&sh->pfull[t], p_phase[t]);
            p_phase[t] ^= 1u;
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < kTileKeys / 16; ++kk)
                mma_ts(td + G::kO + t * DH, td + t * 128 + kk * 8,
                       desc_of(v_lo + (kk * 16 * 128 >> 4)), kIdO, (j | kk) != 0);
              if (!more) tc_commit(&sh->ofull[t]);
              if (t == 1 || !two) tc_commit(&sh->empty[vs]);
            }
            __syncwarp();
            if (more) {
              if (t == 0) wait(&sh->full[ks], kph);
              scores(t, ks, t == 1 || !two, j + 2 == n);
            }
          };
          tile(0);
          if (two) tile(1);
          if (more) {
            if (++stage == G::kStages) { stage = 0; phase ^= 1u; }
          }
        }
      }
      // Every MMA this warp issued has finished before TMEM is released.
      if (elect_one()) tc_commit(&sh->drain);
      __syncwarp();
      mbar_wait_drain(&sh->drain, 0);
    } else if (warp == 9) {
      // ----------------------------------------------------------- TMA producer
      // of tiles, or of their codes
      constexpr int kRing = Kv::kFp8 ? G::kCodeStages : G::kStages;
      uint64_t *ring_full = sh->full, *ring_empty = sh->empty;
      if constexpr (Kv::kFp8) {
        ring_full = sh->code_full;
        ring_empty = sh->code_empty;
      }
      TmaRingT<kRing> ring;
      bool stop = false;
      AttnCursor cur = sh->start.cursor;
      for (; !stop; seg_phase ^= ++seg_at == kSegments, seg_at %= kSegments) {
        stop = __any_sync(0xFFFFFFFFu,
                          !attn_wait(&sh->seg_empty[seg_at], seg_phase ^ 1u, abort));
        if (stop) break;
        AttnSegment& seg = sh->seg[seg_at];
        if (lane == 0) {
          if (!cur.next(a.plan, seg)) seg.pieces = 0;
          mbar_arrive(&sh->seg_full[seg_at]);
        }
        __syncwarp();
        if (seg.pieces == 0) break;
        if (seg.keys == 0) continue;
#pragma unroll 1
        for (int32_t j = seg.tile0; j < seg.tile1 && !stop; ++j) {
          const int32_t k0 = j * kTileKeys;
          const int32_t n = seg.keys - k0 < kTileKeys ? seg.keys - k0 : kTileKeys;
          const int32_t grans = (n + a.granule - 1) / a.granule;
          KvPlace at{0, 0};
          if (lane < grans) at = kv_place(a, seg, k0 + lane * a.granule);
#pragma unroll 1
          for (int kv = 0; kv < 2; ++kv) {
            stop = __any_sync(0xFFFFFFFFu,
                              !attn_wait(&ring_empty[ring.stage], ring.phase ^ 1u, abort));
            if (stop) break;
            if (lane == 0)
              mbar_arrive_expect_tx(&ring_full[ring.stage],
                                    static_cast<uint32_t>(grans * a.granule) *
                                        (Kv::kFp8 ? DH : 128 * G::kHalves));
            __syncwarp();
            if (lane < grans) {
              if constexpr (Kv::kFp8) {
                tma_load_4d(sCodes + ring.stage * G::kCodeBytes + lane * a.granule * DH, kv ? &tmV : &tmK,
                            &ring_full[ring.stage], 0, seg.h, at.z, at.w);
              } else {
                uint8_t* dst = sKV + ring.stage * G::kTileBytes;
#pragma unroll
                for (int hf = 0; hf < G::kHalves; ++hf)
                  tma_load_4d(dst + hf * (kTileKeys * 128) + lane * a.granule * 128,
                              kv ? &tmV : &tmK, &ring_full[ring.stage], hf * 64, seg.h, at.z, at.w);
              }
            }
            ring.issued();
          }
        }
      }
      __syncwarp();
      ring.drain(ring_full);
    } else if (Kv::kFp8 && warp == 10) {
      // ----------------------------------------------------------- queries
      uint32_t q_phase = 0, q_loads = 0;
#pragma unroll 1
      for (; next_segment(); segment_done())
        if (sh->seg[seg_at].keys > 0) request_queries(sh->seg[seg_at], q_phase, q_loads);
      if (q_loads > 0) mbar_wait_drain(&sh->qfull, (q_loads - 1) & 1u);
    } else if (Kv::kFp8 && warp == 11) {
      // ----------------------------------------------------------- scales, four slots per lane
      if constexpr (Kv::kFp8) {
        uint32_t stage = 0, phase = 0;
#pragma unroll 1
        for (; next_segment(); segment_done()) {
          const AttnSegment& seg = sh->seg[seg_at];
          if (seg.keys == 0) continue;
          bool stop = false;
#pragma unroll 1
          for (int32_t j = seg.tile0; j < seg.tile1 && !stop; ++j) {
            const int32_t pos = j * kTileKeys + lane * 4;
            KvPlace at{0, a.n_pages};
            if (pos < seg.keys) at = kv_place(a, seg, pos);
            const bool there = at.w < a.n_pages;
#pragma unroll 1
            for (int kv = 0; kv < 2; ++kv) {
              stop = __any_sync(0xFFFFFFFFu, !attn_wait(&sh->code_empty[stage], phase ^ 1u, abort));
              if (stop) break;
              const KvFp8Part& p = kv ? source.v : source.k;
              copy4(smem_u32(&sh->scales[stage][lane * 4]),
                    p.scales + (there ? at.w * p.scale_page + seg.h * p.scale_head + at.z : 0), there);
              arrive_after_copies(&sh->code_full[stage]);
              if (++stage == G::kCodeStages) { stage = 0; phase ^= 1u; }
            }
          }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
      }
    } else if (Kv::kFp8) {
      // ----------------------------------------------------------- codes to 16 bits
      if constexpr (Kv::kFp8) {
        const int part = warp - kSoftmaxWarps - 4;   // 32 rows of a tile
        uint32_t stage = 0, phase = 0, code = 0, code_phase = 0, count = 0;
#pragma unroll 1
        for (; next_segment(); segment_done()) {
          const AttnSegment& seg = sh->seg[seg_at];
          if (seg.keys == 0) continue;
          const uint32_t slot8 = count++ % kPoisonSlots;
          if (lane == 0) sh->poison[part][slot8] = 0;
          __syncwarp();
#pragma unroll 1
          for (int32_t j = seg.tile0; j < seg.tile1; ++j) {
#pragma unroll 1
            for (int kv = 0; kv < 2; ++kv) {
              attn_wait(&sh->empty[stage], phase ^ 1u, abort);
              attn_wait(&sh->code_full[code], code_phase, abort);
              __syncwarp();
              const int32_t end = seg.keys - j * kTileKeys;                        // rows from here on: nobody's
              const int32_t guard = kv == 0 ? kTileKeys : seg.first - j * kTileKeys;   // not everybody's
              if (convert_tile<DH, kBf16>(smem_u32(sCodes + code * G::kCodeBytes), sh->scales[code],
                                          smem_u32(sKV + stage * G::kTileBytes), part * 32, end, guard, kv == 1))
                *static_cast<volatile int*>(&sh->poison[part][slot8]) = 1;
              fence_proxy_async_shared();
              __syncwarp();
              if (lane == 0) {
                mbar_arrive(&sh->full[stage]);
                mbar_arrive(&sh->code_empty[code]);
              }
              if (++stage == G::kStages) { stage = 0; phase ^= 1u; }
              if (++code == G::kCodeStages) { code = 0; code_phase ^= 1u; }
            }
          }
        }
      }
    } else {
      // ----------------------------------------------------------- values nobody may see
      const int part = warp - kSoftmaxWarps - 2;   // of the rows
      uint32_t stage = 0, phase = 0, count = 0, q_phase = 0, q_loads = 0;
#pragma unroll 1
      for (; next_segment(); segment_done()) {
        const AttnSegment& seg = sh->seg[seg_at];
        if (seg.keys == 0) continue;
        const uint32_t slot8 = count++ % kPoisonSlots;
        if (part == 0) request_queries(seg, q_phase, q_loads);
        if (lane == 0) sh->poison[part][slot8] = 0;
        __syncwarp();
#pragma unroll 1
        for (int32_t j = seg.tile0; j < seg.tile1; ++j) {
#pragma unroll 1
          for (int kv = 0; kv < 2; ++kv) {
            attn_wait(&sh->full[stage], phase, abort);
            __syncwarp();
            if (kv == 1 && (j + 1) * kTileKeys > seg.first) {
              // Each lane takes one 16-byte chunk column and every kStep-th row.
              constexpr int kChunks = DH / 8, kStep = 2 * (32 / kChunks);
              const int ch = lane % kChunks;
              const uint32_t v = smem_u32(sKV + stage * G::kTileBytes) +
                                 (ch >> 3) * (kTileKeys * 128);
              auto at = [&](int32_t r) { return v + r * 128 + (((ch & 7) ^ (r & 7)) << 4); };
              const int32_t f = seg.first - j * kTileKeys, e = seg.keys - j * kTileKeys;
              const int32_t r1 = e < kTileKeys ? e : kTileKeys;   // rows from here on: nobody's
              int32_t r = (f > 0 ? f : 0) + part * (32 / kChunks) + lane / kChunks;
              uint32_t any = 0;
              const int32_t r_first = r;
#pragma unroll 1
              for (; r < r1; r += 8 * kStep) {
                uint4 w[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  w[i] = r + i * kStep < r1 ? lds128(at(r + i * kStep)) : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  any |= nonfinite_bits<kBf16>(w[i].x) | nonfinite_bits<kBf16>(w[i].y) |
                         nonfinite_bits<kBf16>(w[i].z) | nonfinite_bits<kBf16>(w[i].w);
              }
              if (any != 0) {   // rare: replace what is not finite
                *static_cast<volatile int*>(&sh->poison[part][slot8]) = 1;
#pragma unroll 1
                for (r = r_first; r < r1; r += kStep) {
                  const uint4 w = lds128(at(r));
                  sts128(at(r), make_uint4(finite_only<kBf16>(w.x), finite_only<kBf16>(w.y),
                                           finite_only<kBf16>(w.z), finite_only<kBf16>(w.w)));
                }
              }
#pragma unroll 1
              for (r = r1 + part * (32 / kChunks) + lane / kChunks; r < kTileKeys; r += kStep)
                sts128(at(r), make_uint4(0, 0, 0, 0));
              fence_proxy_async_shared();
              __syncwarp();
              if (lane == 0) mbar_arrive(&sh->vok[stage]);
            }
            if (lane == 0) mbar_arrive(&sh->empty[stage]);
            if (++stage == G::kStages) { stage = 0; phase ^= 1u; }
          }
        }
      }
      if (q_loads > 0) mbar_wait_drain(&sh->qfull, (q_loads - 1) & 1u);
    }
  }

  tc_fence_before();
  __syncwarp();
  cta_sync_all();   // every role is done with TMEM (each thread counted on its own)
  if (threadIdx.x == 0) attn_report(abort, a.err);
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int DH, bool kBf16, class Kv>
cudaError_t launch_tiles(const AttnArgs& a, const CUtensorMap& tmQ, const CUtensorMap& tmK,
                         const CUtensorMap& tmV, const Kv& source, cudaStream_t st) {
  static_assert(smem_bytes<DH, Kv>() <= 232448, "shared memory");
  const cudaError_t e = ensure_dynamic_smem(
      reinterpret_cast<const void*>(attn_tiles_kernel<DH, kBf16, Kv>), smem_bytes<DH, Kv>());
  if (e != cudaSuccess) return e;
  return launch_ex(attn_tiles_kernel<DH, kBf16, Kv>, dim3(a.plan.workers), dim3(kThreads<Kv>),
                   smem_bytes<DH, Kv>(), st, true, tmQ, tmK, tmV, a,
                   attn_pieces_at(a.workspace, a.plan.workers, kItemRows), source);
}

template <class Kv>
cudaError_t launch_tiles_any(const AttnArgs& a, const CUtensorMap& tmQ, const CUtensorMap& tmK,
                             const CUtensorMap& tmV, const Kv& source, cudaStream_t st) {
  if (attn_width(a.head_dim) == 64)
    return a.bf16 ? launch_tiles<64, true>(a, tmQ, tmK, tmV, source, st)
                  : launch_tiles<64, false>(a, tmQ, tmK, tmV, source, st);
  return a.bf16 ? launch_tiles<128, true>(a, tmQ, tmK, tmV, source, st)
                : launch_tiles<128, false>(a, tmQ, tmK, tmV, source, st);
}

// How items of 256 rows are shared out, and the tensor map of the queries.
inline bool plan_tiles(AttnArgs& a, CUtensorMap& tmQ) {
  a.plan.tokens = kItemRows / a.group;
  a.plan.workers = device_sm_count();
  a.plan.extra = kExtraUnits;
  return tensor_map_attn(&tmQ, a.q, a.bf16, a.head_dim, a.heads, a.plan.total, 1, a.q_head, a.q_token, 0,
                         a.group, a.plan.tokens);
}

}  // namespace

}  // namespace engram

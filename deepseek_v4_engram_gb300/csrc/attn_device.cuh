// What the attention kernels share on the device.
#pragma once

#include <cuda_fp16.h>

#include "attn.h"
#include "device.cuh"

namespace engram {

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two f32 -> packed pair of the 16-bit type (lo in the low half), round to nearest even.
template <bool kBf16>
__device__ __forceinline__ uint32_t pack16x2(float lo, float hi) {
  if constexpr (kBf16) return pack_bf16x2(lo, hi);
  __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}

// Not zero where one of the two 16-bit values in `w` is an infinity or NaN: one added to an
// exponent of all ones carries into the sign's place.
template <bool kBf16>
__device__ __forceinline__ uint32_t nonfinite_bits(uint32_t w) {
  return ((w & 0x7FFF7FFFu) + (kBf16 ? 0x00800080u : 0x04000400u)) & 0x80008000u;
}

// `w` with an infinity or NaN replaced by 0.
template <bool kBf16>
__device__ __forceinline__ uint32_t finite_only(uint32_t w) {
  const uint32_t b = nonfinite_bits<kBf16>(w);
  return w & ((b & 0x8000u ? 0u : 0x0000FFFFu) | (b & 0x80000000u ? 0u : 0xFFFF0000u));
}

template <bool kBf16>
__device__ __forceinline__ float to_f32(uint16_t bits) {
  if constexpr (kBf16) return bf16_bits_to_f32(bits);
  return __half2float(__ushort_as_half(bits));
}

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar,
                                            int32_t x, int32_t y, int32_t z, int32_t w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}

// Where the keys of the granule that starts at position `pos` of the segment's sequence lie: z and w
// coordinates of the tensor maps. A page number that the cache does not have is reported and
// addressed past the end, where a copy reads zeros.
struct KvPlace {
  int32_t z, w;
};
__device__ __forceinline__ KvPlace kv_place(const AttnArgs& a, const AttnSegment& s, int32_t pos) {
  if (a.table == nullptr) return {s.q0 + pos, 0};
  const int32_t col = pos / a.page_size;
  int32_t page = a.table[static_cast<int64_t>(s.b) * a.table_width + col];
  if (page < 0 || page >= a.n_pages) {
    set_error(a.err, kErrPageRange);
    page = a.n_pages;
  }
  return {pos - col * a.page_size, page};
}

// Wait for the phase of `bar` with the given parity, in few instructions: it stands in many places,
// and code that does not fit the instruction cache costs these kernels more than anything else
// where items are short. Looks at the clock every 32 tries; gives up (false) after kWaitLimitNs or
// once another role has: the roles then run to their end without touching memory that was never
// filled in earnest, and the CTA reports it (attn_report).
__device__ __forceinline__ bool attn_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  const uint32_t at = smem_u32(bar);
  uint32_t since = 0;   // in units of 2^20 ns
#pragma unroll 1
  for (uint32_t i = 1; !mbar_try_wait(at, parity); ++i) {
    if ((i & 31u) != 0) continue;
    const uint32_t now = static_cast<uint32_t>(globaltimer_ns() >> 20) | 1u;
    if (since == 0) since = now;
    if (*abort != 0 || now - since > static_cast<uint32_t>(kWaitLimitNs >> 20)) {
      *abort = 1;
      return false;
    }
  }
  return true;
}

// At the end of a kernel, by one thread: whether a wait has given up.
__device__ __forceinline__ void attn_report(volatile int* abort, uint32_t* err) {
  if (*abort) set_error(err, kErrWaitTimeout);
}

// Finds the calling CTA's range: every thread sums a run of sequences, a scan over the CTA finds
// the run that holds the range's first unit, that run's thread walks it, and the first warp finds
// the place in the sequence, 32 token tiles at a time. One pass over the lengths; all kThreads
// threads call it. A worker without work gets a cursor that has nothing left. Worker 0 reports
// lengths beyond the page table.
struct AttnStart {
  int64_t sums[16];   // per warp
  int64_t pos, units, per, head;
  int32_t b;
  AttnCursor cursor;
};

template <int kThreads>
__device__ __forceinline__ void attn_find_start(const AttnPlan& p, int32_t worker, AttnStart* sh,
                                                uint32_t* err) {
  static_assert(kThreads <= 16 * 32, "sums");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t run = p.n_seqs <= kThreads ? 1 : (p.n_seqs + kThreads - 1) / kThreads;
  const int32_t b0 = tid * run;
  const int32_t b1 = b0 + run < p.n_seqs ? b0 + run : p.n_seqs;
  if (tid == 0) sh->units = 0;
  // Pass 0 sums the run; pass 1, in the thread whose run holds the range's first unit, walks it
  // (one loop for both: the code is read from memory once per launch and SM).
  int64_t mine = 0, at = 0, u0 = -1, per = 0, total = 0, head = 0;   // head: of a key-value head
  bool holds = true;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    if (holds) {
#pragma unroll 1
      for (int32_t b = b0; b < b1; ++b) {
        if (pass == 0 || run > 1) head = attn_head_units(p, attn_seq(p, b));
        const int64_t u = head * p.kv_heads;
        if (pass == 1 && u0 < at + u) {
          sh->b = b;
          sh->pos = u0 - at;
          sh->units = total - u0 < per ? total - u0 : per;
          sh->per = per;
          sh->head = head;
          break;
        }
        at += u;
      }
    }
    if (pass == 1) break;
    mine = at;
    int64_t scan = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xFFFFFFFFu, scan, o);
      if (lane >= o) scan += v;
    }
    if (lane == 31) sh->sums[warp] = scan;
    __syncthreads();
    at = scan - mine;
#pragma unroll 1
    for (int w = 0; w < kThreads / 32 && w * 32 * run < p.n_seqs; ++w) {
      if (w < warp) at += sh->sums[w];
      total += sh->sums[w];
    }
    per = attn_share(p, total);
    u0 = per * worker;
    holds = u0 < total && at <= u0 && u0 < at + mine;
  }
  if (worker == 0 && p.kv_len)
#pragma unroll 1
    for (int32_t b = b0; b < b1; ++b)
      if (p.kv_len[b] > p.kv_cap) set_error(err, kErrCacheCapacity);
  __syncthreads();
  if (warp == 0) {
    const int64_t units = sh->units;
    if (units > 0) {
      const AttnSeq s = attn_seq(p, sh->b);
      const int32_t h = static_cast<int32_t>(attn_div(sh->pos, sh->head));
      const int64_t in = sh->pos - h * sh->head;          // units into the key-value head
      int32_t lo = 0, hi = attn_items(p, s);              // the place is in tile lo .. hi - 1
      int64_t begins = 0;                                 // units before lo
#pragma unroll 1
      while (hi - lo > 1) {
        const int32_t step = (hi - lo + 31) / 32, k = lo + step * lane;
        int64_t u = k <= hi ? attn_units_before(p, s, k) : in + 1;
        if (lane == 0) u = begins;
        const int last = 31 - __clz(__ballot_sync(0xFFFFFFFFu, u <= in));   // lane 0 always is
        begins = __shfl_sync(0xFFFFFFFFu, u, last);
        lo += step * last;
        hi = lo + step < hi ? lo + step : hi;
      }
      if (lane == 0)
        sh->cursor.start(p, worker, sh->per, sh->b, h, lo, static_cast<int32_t>(in - begins), units);
    } else if (lane == 0) {
      sh->cursor.left = 0;
      sh->cursor.b = p.n_seqs;
    }
  }
  __syncthreads();
}

// What the joining kernel has to know of a segment that is a piece, written by one thread; the two
// entries of a worker are first cleared by attn_no_pieces.
__device__ __forceinline__ void attn_no_pieces(const AttnPieces& p) {
  p.meta[blockIdx.x * 2].pieces = 0;
  p.meta[blockIdx.x * 2 + 1].pieces = 0;
}
__device__ __forceinline__ void attn_piece(const AttnPieces& p, const AttnSegment& s) {
  if (s.begins() && s.ends()) return;
  p.meta[blockIdx.x * 2 + (s.begins() ? 1 : 0)] =
      AttnMeta{s.token0, s.ntok, s.h, s.pieces, s.owner, {0, 0, 0}};
}

}  // namespace engram

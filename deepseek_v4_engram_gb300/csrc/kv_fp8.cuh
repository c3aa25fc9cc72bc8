// The 8-bit cache's format on the device. A row, the head_dim values of one position and key-value
// head, is e4m3 codes and one e8m0 byte, value = code * 2^(byte - 127). Where the table's rows have a
// scale for every 32 values, a cache row has one: codes are floating point, so that only rows whose
// values span more than 2^15 would gain by more, and a scale that belongs to a key or a value as a
// whole leaves the products to the codes (it is a factor of a score, or of a probability). A power of
// two makes both ways exact but for the one rounding to a code.
#pragma once

#include "attn_device.cuh"
#include "kv_fp8.h"

namespace engram {

// Rows are not scaled up beyond 2^100: sums over a long cache of weights that were divided by a value's
// scale then stay finite in f32. Bytes below it count as it; a page that is not the cache's reads as 0.
constexpr uint32_t kMinScale = 27;
constexpr uint32_t kNanScale = 255;

// The scale of a row whose largest magnitude is `top` (at least 0, infinite or NaN if any value is): the
// smallest power of two that leaves every value within 448 = 1.75 * 2^8, the largest code; 1 for a row
// of zeros. From the bits: top = 1.f * 2^(E - 127) fits under 448 * 2^(E - 135) unless 1.f > 1.75.
__device__ __forceinline__ uint32_t fp8_scale(float top) {
  const uint32_t b = __float_as_uint(top), E = b >> 23;
  if (E == 255) return kNanScale;
  if (b == 0) return 127;
  const uint32_t s = E + ((b & 0x7FFFFFu) > 0x600000u ? 1u : 0u);
  return s < kMinScale + 8 ? kMinScale : s - 8;
}

// 2^(byte - 127), NaN for its byte.
__device__ __forceinline__ float fp8_scale_value(uint32_t byte) {
  return byte == kNanScale ? __uint_as_float(0x7FC00000u)
                           : __uint_as_float((byte < kMinScale ? kMinScale : byte) << 23);
}

// Two f32 -> two codes (lo in the low byte), round to nearest even.
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(lo), "f"(hi));
  return r;
}

// Two codes -> f16 pair, exactly; NaN codes give NaN.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(codes));
  return r;
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Two codes times a scale in the 16-bit type, rounded once. What that cannot hold becomes its largest value:
// rounding to a code may carry a value past it (bf16's largest one becomes 2^128).
template <bool kBf16>
__device__ __forceinline__ uint32_t scaled16x2(uint32_t codes, float scale) {
  const uint32_t h = e4m3x2_to_f16x2(static_cast<uint16_t>(codes));
  float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h));
  const float most = kBf16 ? __uint_as_float(0x7F7F0000u) : 65504.f;
  x.x *= scale;
  x.y *= scale;
  x.x = fabsf(x.x) > most ? copysignf(most, x.x) : x.x;   // NaN stays
  x.y = fabsf(x.y) > most ? copysignf(most, x.y) : x.y;
  return pack16x2<kBf16>(x.x, x.y);
}

// The same for four codes whose scale is from 2^-14 to 2^7 (f16, with one product for two) or from 2^-100 to
// 2^118 (bf16, through f32): nothing goes beyond the type's range. `scale`: what fast_scale gives.
template <bool kBf16>
__device__ __forceinline__ bool is_fast(uint32_t byte) {
  return kBf16 ? byte >= kMinScale && byte <= 245 : byte >= 113 && byte <= 134;
}
template <bool kBf16>
__device__ __forceinline__ uint32_t fast_scale(uint32_t byte) {
  const uint32_t half = (byte - 112) << 10;
  return kBf16 ? byte << 23 : half | half << 16;
}
template <bool kBf16>
__device__ __forceinline__ void scaled16x4(uint32_t codes, uint32_t scale, uint32_t& lo, uint32_t& hi) {
  lo = e4m3x2_to_f16x2(static_cast<uint16_t>(codes));
  hi = e4m3x2_to_f16x2(static_cast<uint16_t>(codes >> 16));
  if constexpr (kBf16) {
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    const uint64_t f = pair(__uint_as_float(scale), __uint_as_float(scale));
    float p, q;
    unpair(mul2(pair(x.x, x.y), f), p, q);
    lo = pack16x2<true>(p, q);
    unpair(mul2(pair(y.x, y.y), f), p, q);
    hi = pack16x2<true>(p, q);
  } else {
    asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(lo) : "r"(scale));
    asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(hi) : "r"(scale));
  }
}

// The bytes of `w` that are NaN codes, by their top bits.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) {
  return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}

// Asynchronous copy of 4 bytes to shared memory, zeros where there is nothing to read; and this thread's
// arrival on `bar` once its copies so far are there.
__device__ __forceinline__ void copy4(uint32_t to, const void* from, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(from), "r"(there ? 4 : 0) : "memory");
}
__device__ __forceinline__ void arrive_after_copies(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Where token t of the packed ones lies in the cache: it is one of the last positions of the sequence
// that holds it. kNone: a token of no sequence; kOutside: before the first position, or (reported) beyond
// the table or on a page that the cache does not have.
struct Fp8Place {
  enum Kind { kInside, kNone, kOutside } kind;
  int32_t page, slot;
};
__device__ __forceinline__ Fp8Place fp8_place(const KvFp8Args& a, int32_t t) {
  int32_t lo = 0, hi = a.n_seqs;   // the last b with cu[b] <= t
  while (hi - lo > 1) {
    const int32_t mid = lo + (hi - lo) / 2;
    if (a.cu[mid] <= t) lo = mid;
    else hi = mid;
  }
  const int32_t end = attn_clamp(a.cu[lo + 1], 0, a.total);
  if (t < a.cu[lo] || t >= end) return {Fp8Place::kNone, 0, 0};
  const int32_t len = a.kv_len[lo];
  const int32_t p = (len > 0 ? len : 0) - (end - t);   // a negative length is an empty cache
  if (p < 0) return {Fp8Place::kOutside, 0, 0};
  const int32_t col = p / a.page_size;
  if (col >= a.table_width) {
    set_error(a.err, kErrCacheCapacity);
    return {Fp8Place::kOutside, 0, 0};
  }
  const int32_t page = a.table[static_cast<int64_t>(lo) * a.table_width + col];
  if (page < 0 || page >= a.n_pages) {
    set_error(a.err, kErrPageRange);
    return {Fp8Place::kOutside, 0, 0};
  }
  return {Fp8Place::kInside, page, p - col * a.page_size};
}

}  // namespace engram

// The two ways between 16-bit keys and values and the pages of an 8-bit cache.
//   append: s = 2^e with the smallest e for which no value exceeds 448 s, codes = e4m3(x / s)
//   read:   x = code * s, rounded to the 16-bit type
// One row (a position and key-value head) per team of lanes, 16 values each, of the keys and of the
// values at once: a team's maximum is a few shuffles, and 16-bit magnitudes are ordered as integers, so
// that it is found before anything is unpacked.
// Measured: 64 tokens with 8 heads of 128 appended in 2.8 us (launch); 13195 tokens in 16.5 us, 4.9 TB/s (latency:
// a row's loads and the lookup of its place, one after the other in some four rounds of blocks); 48 729 positions
// read back in 49 us, 6.1 TB/s, two thirds of it written (53.6 us with a division of 64 bits and a check of
// every value against the type's range). Slower: two or four rows of a team at once in the append (17.0, 20.3
// us), blocks of 256 and 512 threads, keys and values by different threads (22 us).
#include "kernels.h"
#include "kv_fp8.cuh"

namespace engram {

namespace {

constexpr int kThreads = 128;

// row / heads; a division of 64 bits is most of what a row takes.
__device__ __forceinline__ int32_t token_of(int64_t row, int32_t heads) {
  return static_cast<int32_t>(row >> 32 == 0 ? static_cast<uint32_t>(row) / static_cast<uint32_t>(heads)
                                             : row / heads);
}

template <bool kBf16>
__device__ __forceinline__ float low(uint32_t w) {
  return to_f32<kBf16>(static_cast<uint16_t>(w));
}
template <bool kBf16>
__device__ __forceinline__ float high(uint32_t w) {
  return to_f32<kBf16>(static_cast<uint16_t>(w >> 16));
}

// kLanes: of a team, at least head_dim / 16.
template <int kLanes, bool kBf16>
__global__ void __launch_bounds__(kThreads) kv_append_fp8_kernel(const KvFp8Args a) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x % kLanes;
  const bool live = lane * 16 < a.head_dim;
  const int64_t rows = static_cast<int64_t>(a.total) * a.kv_heads;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kThreads / kLanes);
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (kThreads / kLanes) + threadIdx.x / kLanes;
  for (int64_t i = first; i - threadIdx.x / kLanes < rows; i += step) {   // the same for a whole block
    const bool real = live && i < rows;
    const int64_t row = i < rows ? i : rows - 1;
    const int32_t t = token_of(row, a.kv_heads), h = static_cast<int32_t>(row - int64_t(t) * a.kv_heads);
    uint4 w[2][2] = {};
    if (real) {
      const uint4* k = reinterpret_cast<const uint4*>(a.k16 + t * a.k_token + h * a.k_head + lane * 16);
      const uint4* v = reinterpret_cast<const uint4*>(a.v16 + t * a.v_token + h * a.v_head + lane * 16);
      w[0][0] = k[0];
      w[0][1] = k[1];
      w[1][0] = v[0];
      w[1][1] = v[1];
    }
    const Fp8Place at = fp8_place(a, t);
    uint32_t top = 0;   // of the keys in the low half, of the values in the high one
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      uint32_t m = 0;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const uint4& x = w[p][c];
        m = __vmaxu2(m, __vmaxu2(__vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu),
                               __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu)));
      }
      m = __vmaxu2(m, m >> 16) & 0xFFFFu;
      top |= m << (16 * p);
    }
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) top = __vmaxu2(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    if (!real || at.kind != Fp8Place::kInside) continue;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const uint32_t scale = fp8_scale(p == 0 ? low<kBf16>(top) : high<kBf16>(top));
      // a row with an infinity or NaN is marked by its scale, and its codes are zeros
      const float inv = __uint_as_float((254u - (scale == kNanScale ? 127u : scale)) << 23);
      uint32_t codes[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint4& x = w[p][c / 2];
        const uint32_t lo = c % 2 == 0 ? x.x : x.z, hi = c % 2 == 0 ? x.y : x.w;
        codes[c] = pack_e4m3x2(low<kBf16>(lo) * inv, high<kBf16>(lo) * inv) |
                   pack_e4m3x2(low<kBf16>(hi) * inv, high<kBf16>(hi) * inv) << 16;
        if (scale == kNanScale) codes[c] = 0;
      }
      const KvFp8Part& to = p == 0 ? a.k : a.v;
      *reinterpret_cast<uint4*>(to.codes + at.page * to.page + at.slot * to.slot + h * to.head + lane * 16) =
          make_uint4(codes[0], codes[1], codes[2], codes[3]);
      if (lane == 0)
        to.scales[at.page * to.scale_page + h * to.scale_head + at.slot] = static_cast<uint8_t>(scale);
    }
  }
}

template <int kLanes, bool kBf16>
__global__ void __launch_bounds__(kThreads) kv_read_fp8_kernel(const KvFp8Args a) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x % kLanes;
  if (lane * 16 >= a.head_dim) return;
  const int64_t rows = static_cast<int64_t>(a.total) * a.kv_heads;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kThreads / kLanes);
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * (kThreads / kLanes) + threadIdx.x / kLanes; i < rows; i += step) {
    const int32_t t = token_of(i, a.kv_heads), h = static_cast<int32_t>(i - int64_t(t) * a.kv_heads);
    const Fp8Place at = fp8_place(a, t);
    if (at.kind == Fp8Place::kNone) continue;
    uint4 codes[2] = {};
    uint32_t scale[2] = {127u, 127u};
    if (at.kind == Fp8Place::kInside) {
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const KvFp8Part& from = p == 0 ? a.k : a.v;
        codes[p] = *reinterpret_cast<const uint4*>(from.codes + at.page * from.page + at.slot * from.slot +
                                                   h * from.head + lane * 16);
        scale[p] = from.scales[at.page * from.scale_page + h * from.scale_head + at.slot];
      }
    }
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      uint4* to = reinterpret_cast<uint4*>(
          p == 0 ? a.k16 + t * a.k_token + h * a.k_head + lane * 16
                 : a.v16 + t * a.v_token + h * a.v_head + lane * 16);
      const uint32_t c[4] = {codes[p].x, codes[p].y, codes[p].z, codes[p].w};
      uint32_t x[8];
      if (is_fast<kBf16>(scale[p])) {
        const uint32_t s = fast_scale<kBf16>(scale[p]);
#pragma unroll
        for (int e = 0; e < 4; ++e) scaled16x4<kBf16>(c[e], s, x[2 * e], x[2 * e + 1]);
      } else {
        const float s = fp8_scale_value(scale[p]);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = scaled16x2<kBf16>(c[e / 2] >> (16 * (e & 1)), s);
      }
      to[0] = make_uint4(x[0], x[1], x[2], x[3]);
      to[1] = make_uint4(x[4], x[5], x[6], x[7]);
    }
  }
}

template <int kLanes>
dim3 blocks(const KvFp8Args& a) {
  const int64_t n = static_cast<int64_t>(a.total) * a.kv_heads;
  const int64_t b = (n + kThreads / kLanes - 1) / (kThreads / kLanes);
  return dim3(static_cast<unsigned>(b < (1 << 20) ? b : 1 << 20));   // grid-stride beyond
}

}  // namespace

cudaError_t launch_kv_append_fp8(const KvFp8Args& a, cudaStream_t st) {
  if (a.head_dim <= 64)
    return launch_ex(a.bf16 ? kv_append_fp8_kernel<4, true> : kv_append_fp8_kernel<4, false>, blocks<4>(a),
                     dim3(kThreads), 0, st, true, a);
  return launch_ex(a.bf16 ? kv_append_fp8_kernel<8, true> : kv_append_fp8_kernel<8, false>, blocks<8>(a),
                   dim3(kThreads), 0, st, true, a);
}

cudaError_t launch_kv_read_fp8(const KvFp8Args& a, cudaStream_t st) {
  if (a.head_dim <= 64)
    return launch_ex(a.bf16 ? kv_read_fp8_kernel<4, true> : kv_read_fp8_kernel<4, false>, blocks<4>(a),
                     dim3(kThreads), 0, st, true, a);
  return launch_ex(a.bf16 ? kv_read_fp8_kernel<8, true> : kv_read_fp8_kernel<8, false>, blocks<8>(a),
                   dim3(kThreads), 0, st, true, a);
}

}  // namespace engram

// Attention over a paged cache in eight bits.
//
//   x_rj = scale log2(e) 2^k_j q_r . K_j        K_j, V_j: codes; k_j, v_j: exponents of their scales
//   o_r  = sum_j 2^(x_rj - M_r) 2^v_j V_j / sum_j 2^(x_rj - M_r)
//
// The simplest form: a block per token and query head walks the keys 128 at a time with a running
// maximum M and sum; a thread forms one key's score, then one column's sum.
#include "kernels.h"
#include "kv_fp8.cuh"

namespace engram {

namespace {

constexpr int kThreads = 128;

struct Parts {
  KvFp8Part k, v;
};

template <bool kBf16>
__global__ void __launch_bounds__(kThreads) attn_fp8_kernel(const AttnArgs a, const Parts p) {
  __shared__ float sq[128], sp[kThreads], red[kThreads / 32];
  __shared__ int64_t row_v[kThreads];
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t t = blockIdx.x, head = blockIdx.y, h = head / a.group;
  int32_t lo = 0, hi = a.plan.n_seqs;
  while (hi - lo > 1) {
    const int32_t mid = lo + (hi - lo) / 2;
    if (a.plan.cu[mid] <= t) lo = mid;
    else hi = mid;
  }
  const AttnSeq s = attn_seq(a.plan, lo);
  if (t == 0 && head == 0)
    for (int32_t b = tid; b < a.plan.n_seqs; b += kThreads)
      if (a.plan.kv_len[b] > a.plan.kv_cap) set_error(a.err, kErrCacheCapacity);
  if (t < s.q0 || t >= s.q0 + s.n) return;
  const int32_t keys = s.m - s.n + (t - s.q0) + 1;
  sq[tid] = tid < a.head_dim ? to_f32<kBf16>(a.q[t * a.q_token + head * a.q_head + tid]) : 0.f;
  __syncthreads();
  float m = -INFINITY, l = 0.f, o = 0.f;
  for (int32_t j0 = 0; j0 < keys; j0 += kThreads) {
    const int32_t j = j0 + tid;
    float x = -INFINITY, vs = 0.f;
    row_v[tid] = -1;
    if (j < keys) {
      const int32_t col = j / a.page_size, slot = j - col * a.page_size;
      const int32_t page = a.table[static_cast<int64_t>(lo) * a.table_width + col];
      x = 0.f;
      if (page < 0 || page >= a.n_pages) {
        set_error(a.err, kErrPageRange);
      } else {
        const uint4* kp = reinterpret_cast<const uint4*>(p.k.codes + page * p.k.page + slot * p.k.slot + h * p.k.head);
        for (int c = 0; c < a.head_dim / 16; ++c) {
          const uint4 w = kp[c];
          const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t f = e4m3x2_to_f16x2(static_cast<uint16_t>(u[e / 2] >> (16 * (e & 1))));
            const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&f));
            x += sq[c * 16 + 2 * e] * y.x + sq[c * 16 + 2 * e + 1] * y.y;
          }
        }
        x *= fp8_scale_value(p.k.scales[page * p.k.scale_page + h * p.k.scale_head + slot]) * a.scale_log2;
        vs = fp8_scale_value(p.v.scales[page * p.v.scale_page + h * p.v.scale_head + slot]);
        row_v[tid] = page * p.v.page + slot * p.v.slot + h * p.v.head;
      }
    }
    float top = x;
    for (int i = 16; i > 0; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, i));
    if (lane == 0) red[warp] = top;
    __syncthreads();
    for (int i = 0; i < kThreads / 32; ++i) top = fmaxf(top, red[i]);
    top = fmaxf(top, m);
    const float base = top == -INFINITY ? 0.f : top;
    const float f = exp2_fast(m - base), e = exp2_fast(x - base);
    m = top;
    sp[tid] = row_v[tid] < 0 ? 0.f : e * vs;
    float sum = e;
    for (int i = 16; i > 0; i >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, i);
    __syncthreads();
    if (lane == 0) red[warp] = sum;
    __syncthreads();
    sum = 0.f;
    for (int i = 0; i < kThreads / 32; ++i) sum += red[i];
    l = l * f + sum;
    o *= f;
    const int32_t n = keys - j0 < kThreads ? keys - j0 : kThreads;
    if (tid < a.head_dim)
      for (int i = 0; i < n; ++i)
        if (row_v[i] >= 0) {
          const uint32_t c = e4m3x2_to_f16x2(p.v.codes[row_v[i] + tid]);
          o += sp[i] * __half2float(__ushort_as_half(static_cast<uint16_t>(c)));
        }
    __syncthreads();
  }
  if (tid < a.head_dim)
    a.out[t * a.o_token + head * a.o_head + tid] =
        static_cast<uint16_t>(pack16x2<kBf16>(l == 0.f ? 0.f : o / l, 0.f));
  if (a.lse != nullptr && tid == 0)
    a.lse[static_cast<int64_t>(t) * a.heads + head] = (m + log2f(l)) * 0.69314718055994531f;
}

}  // namespace

cudaError_t launch_attn_fp8(const AttnArgs& a, const KvFp8Part& k, const KvFp8Part& v, int32_t rows, cudaStream_t st) {
  if (rows <= kAttnFp8FewRows) return launch_attn_fp8_rows(a, k, v, rows, st);
  return launch_ex(a.bf16 ? attn_fp8_kernel<true> : attn_fp8_kernel<false>, dim3(a.plan.total, a.heads), dim3(kThreads),
                   0, st, true, a, Parts{k, v});
}

}  // namespace engram

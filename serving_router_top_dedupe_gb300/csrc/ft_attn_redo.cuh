// Rows whose sums went wrong because of values that they do not see.
//
// A tile's product with V multiplies every probability with every value, also the zero
// probabilities of tokens that a row does not see (later tokens of its chunk, tokens before its
// window).  Zero times an infinity or a NaN is NaN.  The attention kernels therefore look at
// their results: where a row has a sum that is not finite, and a value that it does not see is
// not finite, one warp forms the row's sums again from the tokens that it does see, one after
// another.  Nothing else pays for this: finite sums are not looked at further, and sums that
// are rightly not finite cost a look at the few tokens of the block that the row does not see.
#pragma once

#include "ft_dot.cuh"
#include "ft_kv_internal.cuh"

namespace ft {
namespace kv {

template <int TYPE, int D>
__device__ __forceinline__ float element(const uint8_t* base, const uint8_t* scales, long long row, int d) {
  if constexpr (TYPE == FT_KV_BF16) {
    return __uint_as_float((uint32_t)__ldg(reinterpret_cast<const uint16_t*>(base) + row * D + d) << 16);
  } else {
    const float s = e8m0(__ldg(scales + row * (D / 32) + d / 32));
    if constexpr (TYPE == FT_KV_MXFP8) {
      return dot::e4m3x2_to_float2((uint16_t)__ldg(base + row * D + d)).x * s;
    } else {
      const uint32_t h2 = dot::e2m1x2_to_f16x2(__ldg(base + row * (D / 2) + d / 2));
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
      return (d & 1 ? f.y : f.x) * s;
    }
  }
}

// Row of the cache of a sequence's token j, -1 for a page that is not there.
__device__ __forceinline__ long long token_row(const AttnParams& p, const Cursor& cur, int j) {
  const int at = j >> p.page_shift;
  const int page = p.staged ? __ldg(p.staged + cur.seq) + at : __ldg(p.page_table + (long long)cur.seq * p.table_stride + at);
  if ((unsigned)page >= (unsigned)p.n_pages) return -1;
  return (((long long)page * p.n_kv_heads + cur.head) << p.page_shift) + (j & (p.page_size - 1));
}

// Whether a value of the tokens [a, b) is not finite (all lanes of a warp; the same answer).
template <int TYPE, int D>
__device__ bool any_not_finite(const AttnParams& p, const Cursor& cur, int a, int b, int lane) {
  float bad = 0.f;
  for (int j = a; j < b; ++j) {
    const long long row = token_row(p, cur, j);
    if (row < 0) continue;
#pragma unroll 1
    for (int i = 0; i < D / 32; ++i) bad = fmaf(element<TYPE, D>(p.v, p.vs, row, lane * (D / 32) + i), 0.f, bad);
  }
  return __any_sync(0xffffffffu, bad != bad);
}

// The sums of one row over its tokens [lo, hi) in [a, b), relative to 2^m: lane l gets columns
// l * D / 32 and on.  False: the row's sums are right as they are.  rr: row of the sequence;
// len: tokens of it that were multiplied.
template <int TYPE, int D>
__device__ bool redo_row(const AttnParams& p, const Cursor& cur, int rr, int lo, int hi, int a, int b, float m, int lane,
                         float* acc) {
  b = min(b, cur.len);
  if (!any_not_finite<TYPE, D>(p, cur, a, min(lo, b), lane) && !any_not_finite<TYPE, D>(p, cur, max(hi, a), b, lane)) return false;
  constexpr int N = D / 32;
  const int tok = div_group(p, rr), hd = cur.head * p.group + rr - tok * p.group;
  const uint16_t* q = p.q + (long long)(cur.q0 + tok) * p.q_stride + (long long)hd * D + lane * N;
#pragma unroll
  for (int i = 0; i < N; ++i) acc[i] = 0.f;
  for (int j = max(lo, a); j < min(hi, b); ++j) {
    const long long row = token_row(p, cur, j);
    float s = 0.f;
    if (row >= 0)
#pragma unroll 1
      for (int i = 0; i < N; ++i)
        s = fmaf(__uint_as_float((uint32_t)__ldg(q + i) << 16), element<TYPE, D>(p.k, p.ks, row, lane * N + i), s);
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (row < 0) continue;  // a page that is not there: values of zero
    const float e = exp2f(s * p.scale_log2 - (m == -INFINITY ? 0.f : m));
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = fmaf(e, element<TYPE, D>(p.v, p.vs, row, lane * N + i), acc[i]);
  }
  return true;
}

}  // namespace kv
}  // namespace ft

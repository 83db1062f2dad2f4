// Values that some rows of a block see and others do not.
//
// A tile's product with V multiplies every probability with every value, also the zero
// probabilities of tokens that a row does not see (later tokens of its chunk, tokens before its
// window).  Zero times an infinity or a NaN is NaN.  So no such value gets into a product: tokens
// that no row of a block sees are cleared when they are loaded, and of those that only some rows
// see (at most the block's own tokens, at either end of what it reads) the elements that are not
// finite are set to zero.  Where there were any, which is noted for the item, the rows that do see
// them get them back at the end, in memory: a sum with p * v, p > 0, is that sum without it plus v.
// Nothing else pays for this than a look at those few tokens.
#pragma once

#include "ft_kv_internal.cuh"

namespace ft {
namespace kv {

// What every row of the item's block of RB rows sees of [cur.lo, cur.hi): [all_lo, all_hi).
template <int RB>
__device__ __forceinline__ void all_see(const AttnParams& p, const Cursor& cur, int& all_lo, int& all_hi) {
  const int r0 = cur.rb * RB, r1 = min(cur.n * p.group, r0 + RB) - 1;
  const int p0 = cur.len - cur.n + div_group(p, r0), p1 = cur.len - cur.n + div_group(p, r1);
  all_hi = p.causal ? max(min(cur.len, p0 + 1), 0) : cur.len;
  all_lo = p.window > 0 ? max(p1 - p.window + 1, 0) : 0;
}

// Eight BF16 elements with zeros in the place of those that are not finite; whether there were any.
__device__ __forceinline__ bool keep_finite(uint4& v) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w}, any = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t bad = __vcmpeq2(w[i] & 0x7f807f80u, 0x7f807f80u);
    w[i] &= ~bad;
    any |= bad;
  }
  v = make_uint4(w[0], w[1], w[2], w[3]);
  return any != 0;
}

// Scale codes with zeros in the place of those that stand for NaN; whether there were any.
__device__ __forceinline__ bool keep_finite(uint32_t& codes) {
  const uint32_t bad = __vcmpeq4(codes, 0xffffffffu);
  codes &= ~bad;
  return bad != 0;
}

// Row of the cache of a sequence's token j, -1 for a page that is not there.
__device__ __forceinline__ int token_row(const AttnParams& p, const Cursor& cur, int j) {
  const int at = j >> p.page_shift;
  const int page = p.staged ? __ldg(p.staged + cur.seq) + at : __ldg(p.page_table + (long long)cur.seq * p.table_stride + at);
  if ((unsigned)page >= (unsigned)p.n_pages) return -1;
  return ((page * p.n_kv_heads + cur.head) << p.page_shift) + (j & (p.page_size - 1));
}

// For a row that sees [lo, hi), over the tokens [a, b) of a part of an item: use(column, value) for
// the values that are not finite of the tokens that only some rows of the block see.
template <int TYPE, int D, typename Use>
__device__ __forceinline__ void not_finite(const AttnParams& p, const Cursor& cur, int all_lo, int all_hi, int lo, int hi, int a, int b,
                                           Use use) {
  a = max(max(a, cur.lo), lo);
  b = min(min(b, cur.hi), hi);
#pragma unroll 1
  for (int j = a; j < b; ++j) {
    if (j >= all_lo && j < all_hi) {  // every row sees these
      j = all_hi - 1;
      continue;
    }
    const int row = token_row(p, cur, j);
    if (row < 0) continue;
    if constexpr (TYPE == FT_KV_BF16) {
      const uint4* v = reinterpret_cast<const uint4*>(p.v + (long long)row * (2 * D));
#pragma unroll 1
      for (int i = 0; i < D / 8; ++i) {
        uint4 w = __ldg(v + i), kept = w;
        if (!keep_finite(kept)) continue;
        const uint32_t words[4] = {w.x ^ kept.x, w.y ^ kept.y, w.z ^ kept.z, w.w ^ kept.w};
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          if (words[x] & 0xffffu) use(8 * i + 2 * x, __uint_as_float(words[x] << 16));
          if (words[x] >> 16) use(8 * i + 2 * x + 1, __uint_as_float(words[x] & 0xffff0000u));
        }
      }
    } else {  // all of a 1x32 block
#pragma unroll 1
      for (int d = 0; d < D; ++d)
        if (__ldg(p.vs + (long long)row * (D / 32) + d / 32) == 255) use(d, __uint_as_float(0x7fc00000u));
    }
  }
}

}  // namespace kv
}  // namespace ft

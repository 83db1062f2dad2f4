// Attention of many rows over the paged cache (prefill chunks) on the 5th-generation tensor
// cores: tcgen05.mma with its accumulators, and the probabilities, in tensor memory.
//
// A CTA takes blocks of 128 (head_dim 256) or 256 rows of one cache head; 128 rows are one
// M = 128 tile.  For every tile of 128 cached tokens
//   S = Q K^T   (Q and K in shared memory, S: 128 TMEM columns, FP32)
//   P = exp2(S * scale - m)  (one thread per row, S read from TMEM, P written back as BF16 over S)
//   O += P V    (P from TMEM, V in shared memory, O: head_dim TMEM columns, FP32)
// With two tiles per CTA the tensor core works on one while the other is in the softmax, and
// each K and V tile in shared memory serves 256 rows; with one (head_dim 256: its O fills half
// of TMEM) S has two buffers, and the scores of the next tile are formed during the softmax.
// Each row's maximum m moves only when a score passes it by 2^8, so O is rarely rescaled; the
// row's thread then does that itself.
//
// Warps 0-3 (and 4-7): softmax, output.  Then one warp that issues every MMA, and the loaders:
// two warps of TMA (K, V) for a BF16 cache, four warps that decode into the same layout for a
// quantised one.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "ft_attn_rows.cuh"
#include "ft_ptx.cuh"

namespace ft {
namespace kv {
namespace chunk {

using rows::e2m1_bits;
using rows::e4m3_bits;
using rows::ex2;
using rows::mul2;
using rows::multiplier;
using rows::pack;

constexpr int KT = 128;           // cached tokens of a tile
constexpr int PANEL = KT * 128;   // bytes of 64 columns of a tile: rows of 128 bytes, 128-byte swizzle
constexpr float kSlack = 8.f;     // log2 units by which scores may pass the running maximum

template <int TYPE, int D>
struct Cfg {
  static constexpr bool q = TYPE != FT_KV_BF16;
  static constexpr int tiles = D <= 128 ? 2 : 1;
  static constexpr int RB = 128 * tiles;
  static constexpr int panels = D / 64;
  static constexpr int stage = panels * PANEL;
  static constexpr int stages = D == 64 ? 4 : D == 128 ? 2 : 1;  // of K, and of V
  static constexpr int soft_warps = 4 * tiles;
  static constexpr int mma_warp = soft_warps, load_warp = q ? soft_warps + 4 : soft_warps + 1;
  static constexpr int threads = 32 * (soft_warps + (q ? 8 : 4));
  static constexpr int qbytes = tiles * stage;
  static constexpr int smem = 1024 + qbytes + 2 * stages * stage + 512;
  static constexpr size_t slot_floats = (size_t)RB * (D + 2);
  static constexpr int o_col = 256;  // TMEM: S (and P) at 0 and 128, O behind
};

__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// Shared-memory matrix descriptor, 128-byte swizzle: 8-row atoms of 1024 bytes (stride byte
// offset); lead: bytes from one 64-column panel to the next, for the operand whose columns
// run along the 128-byte rows (V), unused by the other (Q, K).
__device__ __forceinline__ uint64_t desc(uint32_t saddr, uint32_t lead) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)(lead >> 4) << 16 | (uint64_t)(1024u >> 4) << 32 |
         (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// Instruction descriptor, kind::f16: BF16 operands, FP32 accumulator; bt: B's columns contiguous.
__host__ __device__ constexpr uint32_t idesc(int M, int N, int bt) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)bt << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"(acc)
      : "memory");
}

// 32 consecutive 32-bit columns of this thread's TMEM lane.
__device__ __forceinline__ void tld32(uint32_t a, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(a));
}
__device__ __forceinline__ void tst16(uint32_t a, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(a),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tst32(uint32_t a, const uint32_t* r) {
  tst16(a, r);
  tst16(a + 16, r + 16);
}
// The loaded registers go through the wait, so that nothing reads them earlier.
__device__ __forceinline__ void tld_wait(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(r[i]));
}
__device__ __forceinline__ void tst_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ uint64_t f2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unf2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ void tma2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

// A position in the CTA's sequence of tiles.
template <int TYPE, int D>
struct Walk {
  Cursor cur;
  long long w, w1;
  __device__ __forceinline__ int tile() const { return cur.t0 + (int)(w - cur.start); }
  __device__ __forceinline__ bool first() const { return w == cur.start; }
  // Next tile; true when it is one of another item.
  __device__ __forceinline__ bool next(const AttnParams& p) {
    ++w;
    if (w < w1 && w == cur.start + cur.cost) {
      cursor_next<Cfg<TYPE, D>::RB, KT>(p, cur);
      return true;
    }
    return false;
  }
};

// 16 bytes of codes -> 16 (MXFP8) or 32 (MXFP4) BF16 values in their order.
template <int TYPE>
__device__ __forceinline__ void decode16(uint4 w, uint32_t scale, uint4* out) {
  const uint32_t m = multiplier<TYPE>(scale * 0x01000100u);
  const uint32_t in[4] = {w.x, w.y, w.z, w.w};
  uint32_t o[16];
  if (TYPE == FT_KV_MXFP8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[2 * i] = mul2(e4m3_bits(__byte_perm(in[i], 0, 0x1404)), m);
      o[2 * i + 1] = mul2(e4m3_bits(__byte_perm(in[i], 0, 0x3424)), m);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = in[i] & 0x0F0F0F0Fu, hi = (in[i] >> 4) & 0x0F0F0F0Fu;  // even and odd elements
      // byte j of lo and of hi into the low bytes of the halves (the other bytes are masked off)
      o[4 * i] = mul2(e2m1_bits<0>(__byte_perm(lo, hi, 0x4400)), m);
      o[4 * i + 1] = mul2(e2m1_bits<0>(__byte_perm(lo, hi, 0x5511)), m);
      o[4 * i + 2] = mul2(e2m1_bits<0>(__byte_perm(lo, hi, 0x6622)), m);
      o[4 * i + 3] = mul2(e2m1_bits<0>(__byte_perm(lo, hi, 0x7733)), m);
    }
  }
#pragma unroll
  for (int i = 0; i < (TYPE == FT_KV_MXFP8 ? 2 : 4); ++i)
    out[i] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
}

// 16-byte pieces of a tile's codes that one loader thread holds, and their scale codes.
template <int TYPE, int D>
struct Raw {
  static constexpr int PR = row_bytes(TYPE, D) / 16;  // pieces of a row, and of a thread
  uint4 w[PR];
  uint32_t sc[PR];
};

template <int TYPE, int D>
__device__ __forceinline__ void raw_load(const AttnParams& p, const Cursor& cur, int t, const uint8_t* base,
                                         const uint8_t* scales, int lt, Raw<TYPE, D>& x) {
  constexpr int PR = Raw<TYPE, D>::PR;
  const int32_t* table = p.page_table + (long long)cur.seq * p.table_stride;
#pragma unroll
  for (int i = 0; i < PR; ++i) {
    const int u = lt + 128 * i, tok = t + u / PR, pc = u % PR;
    x.w[i] = make_uint4(0, 0, 0, 0);
    x.sc[i] = 0;
    if (tok < cur.len && tok >= cur.lo) {
      const int page = __ldg(table + (tok >> p.page_shift));
      if ((unsigned)page < (unsigned)p.n_pages) {
        const long long row = (((long long)page * p.n_kv_heads + cur.head) << p.page_shift) + (tok & (p.page_size - 1));
        x.w[i] = __ldg(reinterpret_cast<const uint4*>(base + row * row_bytes(TYPE, D)) + pc);
        x.sc[i] = __ldg(scales + row * (D / 32) + (TYPE == FT_KV_MXFP8 ? pc / 2 : pc));
      } else {
        atomicOr(p.error_word, FT_DEVERR_BAD_INDEX);
      }
    }
  }
}

template <int TYPE, int D>
__device__ __forceinline__ void raw_store(uint8_t* stage, int lt, const Raw<TYPE, D>& x) {
  constexpr int PR = Raw<TYPE, D>::PR, OUT = TYPE == FT_KV_MXFP8 ? 2 : 4;  // 16-byte pieces of BF16 for one of codes
#pragma unroll
  for (int i = 0; i < PR; ++i) {
    const int u = lt + 128 * i, r = u / PR, pc = u % PR;
    uint4 o[OUT];
    decode16<TYPE>(x.w[i], x.sc[i], o);
#pragma unroll
    for (int j = 0; j < OUT; ++j) {
      const int ch = pc * OUT + j;
      *reinterpret_cast<uint4*>(stage + (ch >> 3) * PANEL + r * 128 + (((ch & 7) ^ (r & 7)) << 4)) = o[j];
    }
  }
}

template <int TYPE, int D>
__global__ void __launch_bounds__(Cfg<TYPE, D>::threads, 1)
    attn_chunk_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv, const AttnParams p) {
  using C = Cfg<TYPE, D>;
  constexpr int NS = C::stages, T = C::tiles;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint8_t* ring = smem + C::qbytes;  // K stages, then V stages
  uint64_t* bars = reinterpret_cast<uint64_t*>(ring + 2 * NS * C::stage);
  uint64_t* full = bars;              // [2][NS] a tile of K, of V is in the ring
  uint64_t* empty = bars + 2 * NS;    // [2][NS] its products are done
  uint64_t* q_full = bars + 4 * NS;   // [2] the queries of a row tile are in place
  uint64_t* s_full = q_full + 2;      // [2] scores are in TMEM
  uint64_t* p_full = q_full + 4;      // [2] probabilities are in TMEM
  uint64_t* o_full = q_full + 6;      // [2] a product with V is done
  uint64_t* aux = q_full + 8;         // [2] bytes of a tile whose ends are cleared before it is handed on
  uint64_t* done = q_full + 10;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(q_full + 11);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  auto bar = [](uint64_t* b) { return ptx::smem_u32(b); };

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < 2 * NS; ++s) {
      ptx::mbar_init(bar(full + s), C::q ? 4 : 1);
      ptx::mbar_init(bar(empty + s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(bar(q_full + i), 128);
      ptx::mbar_init(bar(s_full + i), 1);
      ptx::mbar_init(bar(p_full + i), 128);
      ptx::mbar_init(bar(o_full + i), 1);
      ptx::mbar_init(bar(aux + i), 1);
    }
    ptx::mbar_init(bar(done), 1);
    *abort_flag = 0;
    ptx::mbar_fence_init();
  }
  Walk<TYPE, D> wk;
  long long per;
  if (!plan<C::RB, KT, C::threads>(p, *reinterpret_cast<PlanSmem*>(ring), wk.cur, wk.w, wk.w1, per)) return;
  if (warp == C::mma_warp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(ptx::smem_u32(tmem_slot))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_async();  // the ring held the plan: copies may write it now
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = *tmem_slot;
  auto wait = [&](uint64_t* b, uint32_t parity) { return ptx::mbar_wait(bar(b), parity, abort_flag, p.error_word); };
  // for a whole warp: all its lanes go on, or none
  auto wait_all = [&](uint64_t* b, uint32_t parity) { return (bool)__all_sync(0xffffffffu, wait(b, parity)); };
  // rows of row tile x of the item
  auto rows_of = [&](const Cursor& c, int x) { return min(c.n * p.group - c.rb * C::RB - 128 * x, 128); };

  if (warp < C::soft_warps) {
    // ------------------------------------------------------------------ softmax and output
    const int rt = warp >> 2;              // row tile
    const int r = (warp & 3) * 32 + lane;  // row of the tile = TMEM lane
    const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t o_tm = tl + C::o_col + rt * D;
    const float c = fabsf(p.scale_log2) * left_in(TYPE);
    const uint64_t c2 = f2(c, c);
    const uint32_t flip = p.scale_log2 < 0.f ? 0x80008000u : 0u;  // a negative scale turns the queries' signs

    // an item's queries into shared memory, once no product reads the last ones
    auto load_q = [&](const Cursor& cur) {
      const int rows = rows_of(cur, rt);
      if (rows <= 0) return;
      const int rr = cur.rb * C::RB + 128 * rt + r, tok = rr / p.group, hd = rr - tok * p.group;
      const uint4* src = reinterpret_cast<const uint4*>(p.q + (long long)(cur.q0 + tok) * p.q_stride +
                                                        (long long)(cur.head * p.group + hd) * D);
      uint8_t* dst = smem + rt * C::stage + r * 128;
#pragma unroll 8
      for (int i = 0; i < D / 8; ++i) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (r < rows) v = __ldg(src + i);
        *reinterpret_cast<uint4*>(dst + (i >> 3) * PANEL + (((i & 7) ^ (r & 7)) << 4)) =
            r < rows ? make_uint4(v.x ^ flip, v.y ^ flip, v.z ^ flip, v.w ^ flip) : v;
      }
      fence_async();
      ptx::mbar_arrive(bar(q_full + rt));
    };

    uint32_t s_ph = 0, pvs = 0;  // phases of s_full (bit u); products with V so far
    uint32_t step = 0;
    bool ok = true;
    load_q(wk.cur);
    while (ok && wk.w < wk.w1) {  // one item
      const Cursor cur = wk.cur;
      const int rows = rows_of(cur, rt);
      const int rbase = cur.rb * C::RB + 128 * rt;
      int lo = 0, hi = 0, lo_max = 0, hi_min = 0;
      if (rows > 0) {
        auto see = [&](int row, int& a, int& b) {
          const int pos = cur.len - cur.n + row / p.group;
          b = p.causal ? min(cur.len, pos + 1) : cur.len;
          a = p.window > 0 ? max(pos - p.window + 1, 0) : 0;
        };
        int x;
        see(rbase + r, lo, hi);
        see(rbase, x, hi_min);
        see(rbase + rows - 1, lo_max, x);
      }
      float m = -INFINITY, l = 0.f;
      bool first = true;  // no product with V yet
      const long long end = min(cur.start + cur.cost, wk.w1);
      for (; wk.w < end; ++wk.w, ++step) {
        if (rows <= 0) continue;
        const int u = T == 2 ? rt : (int)(step & 1);
        const uint32_t s_tm = tl + 128 * u;
        if (!(ok = wait_all(s_full + u, (s_ph >> u) & 1))) break;
        s_ph ^= 1u << u;
        tc_after();
        const int t = wk.tile() * KT;
        const bool edge = t < lo_max || t + KT > hi_min;
        const int e_lo = lo - t, e_hi = hi - t;  // columns [e_lo, e_hi) are seen
        auto mask = [&](uint32_t* s, int ch) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (32 * ch + i < e_lo || 32 * ch + i >= e_hi) s[i] = 0xff800000u;
        };
        float mx = -INFINITY;
        uint32_t s[2][32];
        tld32(s_tm, s[0]);
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) {
          tld_wait(s[ch & 1]);
          if (ch < 3) tld32(s_tm + 32 * (ch + 1), s[(ch + 1) & 1]);
          if (edge) mask(s[ch & 1], ch);
#pragma unroll
          for (int i = 0; i < 32; ++i) mx = fmaxf(mx, __uint_as_float(s[ch & 1][i]));
        }
        tld32(s_tm, s[0]);
        mx *= c;
        if (__any_sync(0xffffffffu, mx > m + kSlack)) {
          const float mn = fmaxf(m, mx);
          const float al = mn == -INFINITY ? 1.f : ex2(m - mn);
          l *= al;
          m = mn;
          if (!first) {
            if (!(ok = wait_all(o_full + rt, (pvs - 1) & 1))) break;
            tc_after();
            tld_wait(s[0]);
            uint32_t o[32];
#pragma unroll 1
            for (int ch = 0; ch < D / 32; ++ch) {
              tld32(o_tm + 32 * ch, o);
              tld_wait(o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * al);
              tst32(o_tm + 32 * ch, o);
            }
          }
        }
        const float mu = m == -INFINITY ? 0.f : m;
        const uint64_t nm = f2(-mu, -mu);
        uint64_t sum0 = 0, sum1 = 0;
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) {
          tld_wait(s[ch & 1]);
          if (ch < 3) tld32(s_tm + 32 * (ch + 1), s[(ch + 1) & 1]);
          if (edge) mask(s[ch & 1], ch);
          uint32_t pr[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float a, b;
            unf2(fma2(f2(__uint_as_float(s[ch & 1][2 * i]), __uint_as_float(s[ch & 1][2 * i + 1])), c2, nm), a, b);
            a = ex2(a);
            b = ex2(b);
            if (i & 1) sum1 = add2(sum1, f2(a, b));
            else sum0 = add2(sum0, f2(a, b));
            pr[i] = pack(a, b);
          }
          tst16(s_tm + 16 * ch, pr);
        }
        tst_wait();
        // With two S buffers these scores do not tell that the product before last is done.  No
        // phase of o_full may be skipped: a parity tells a phase from its neighbours only.
        if (T == 1 && pvs && !(ok = wait_all(o_full, (pvs - 1) & 1))) break;
        tc_before();
        ptx::mbar_arrive(bar(p_full + u));
        float a0, a1;
        unf2(add2(sum0, sum1), a0, a1);
        l += a0 + a1;
        first = false;
        ++pvs;
      }
      if (!ok) break;
      // on to the next item: its queries first, so that its scores are formed during the output
      if (wk.w < wk.w1) {
        if (wk.w == cur.start + cur.cost) cursor_next<C::RB, KT>(p, wk.cur);
        load_q(wk.cur);
      }
      if (rows <= 0) continue;
      if (!(ok = wait_all(o_full + rt, (pvs - 1) & 1))) break;
      tc_after();
      int ca, cb;
      piece_owners(cur, per, ca, cb);
      const int tok = (rbase + r) / p.group, hd = cur.head * p.group + rbase + r - tok * p.group;
      uint16_t* dst = p.out + (long long)(cur.q0 + tok) * p.out_stride + (long long)hd * D;
      float* lse = p.lse + (long long)(cur.q0 + tok) * p.n_heads + hd;
      if (ca == cb) {
        const float inv = l == 0.f ? 0.f : left_in(TYPE) / l;
#pragma unroll 1
        for (int ch = 0; ch < D / 32; ++ch) {
          uint32_t o[32];
          tld32(o_tm + 32 * ch, o);
          tld_wait(o);
          if (r < rows) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t w[4];
#pragma unroll
              for (int j = 0; j < 4; ++j)
                w[j] = pack(__uint_as_float(o[8 * i + 2 * j]) * inv, __uint_as_float(o[8 * i + 2 * j + 1]) * inv);
              reinterpret_cast<uint4*>(dst + 32 * ch)[i] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        }
        if (p.lse && r < rows) *lse = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
      } else {
        // partial result: columns in groups of four, the rows of a group side by side
        const int me = blockIdx.x, at = 128 * rt + r;
        float* slot = p.partials + (size_t)(2 * me + (me == ca ? 1 : 0)) * C::slot_floats;
#pragma unroll 1
        for (int ch = 0; ch < D / 32; ++ch) {
          uint32_t o[32];
          tld32(o_tm + 32 * ch, o);
          tld_wait(o);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            __stcg(reinterpret_cast<uint4*>(slot) + (8 * ch + i) * C::RB + at,
                   make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]));
        }
        __stcg(slot + C::RB * D + at, m);
        __stcg(slot + C::RB * (D + 1) + at, l);
        // each warp joins its own 32 rows: the last CTA's warp to come, in the parts' order
        uint32_t* counter = p.counters + 8 * ca + warp;
        __threadfence();
        __syncwarp();
        int is_last = 0;
        if (lane == 0) is_last = atomicAdd(counter, 1u) == (uint32_t)(cb - ca);
        if (__shfl_sync(0xffffffffu, is_last, 0)) {
          __threadfence();
          if (lane == 0) *counter = 0u;
          auto part = [&](int x) { return p.partials + (size_t)(2 * x + (x == ca ? 1 : 0)) * C::slot_floats; };
          float mm = -INFINITY, ll = 0.f;
          for (int x = ca; x <= cb; ++x) mm = fmaxf(mm, __ldcg(part(x) + C::RB * D + at));
          for (int x = ca; x <= cb; ++x)
            ll += __ldcg(part(x) + C::RB * (D + 1) + at) *
                  (mm == -INFINITY ? 0.f : ex2(__ldcg(part(x) + C::RB * D + at) - mm));
          const float inv = ll == 0.f ? 0.f : left_in(TYPE) / ll;
#pragma unroll 1
          for (int ch = 0; ch < D / 32; ++ch) {
            float acc[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) acc[i] = 0.f;
#pragma unroll 1
            for (int x = ca; x <= cb; ++x) {
              const float wx = mm == -INFINITY ? 0.f : ex2(__ldcg(part(x) + C::RB * D + at) - mm);
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float4 v = __ldcg(reinterpret_cast<const float4*>(part(x)) + (8 * ch + i) * C::RB + at);
                acc[4 * i] += v.x * wx;
                acc[4 * i + 1] += v.y * wx;
                acc[4 * i + 2] += v.z * wx;
                acc[4 * i + 3] += v.w * wx;
              }
            }
            if (r < rows) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
                reinterpret_cast<uint4*>(dst + 32 * ch)[i] =
                    make_uint4(pack(acc[8 * i] * inv, acc[8 * i + 1] * inv), pack(acc[8 * i + 2] * inv, acc[8 * i + 3] * inv),
                               pack(acc[8 * i + 4] * inv, acc[8 * i + 5] * inv), pack(acc[8 * i + 6] * inv, acc[8 * i + 7] * inv));
            }
          }
          if (p.lse && r < rows) *lse = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * 0.69314718055994530942f;
        }
      }
    }
  } else if (warp == C::mma_warp) {
    // ------------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      const uint32_t q_addr = ptx::smem_u32(smem), ring_addr = ptx::smem_u32(ring);
      uint32_t kst = 0, vst = 0, kph = 0, vph = 0;  // ring positions and phases
      uint32_t q_ph = 0, p_ph = 0;
      auto advance = [&](uint32_t& st, uint32_t& ph) {
        if (++st == (uint32_t)NS) {
          st = 0;
          ph ^= 1u;
        }
      };
      // scores of row tile x into S buffer u, from the K stage at kst
      auto scores = [&](int x, int u) {
        const uint32_t a = q_addr + x * C::stage, b = ring_addr + kst * C::stage;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = (k >> 2) * PANEL + 32 * (k & 3);
          mma_ss(tmem + 128 * u, desc(a + off, 0), desc(b + off, 0), idesc(128, KT, 0), k != 0);
        }
        commit(bar(s_full + u));
      };
      auto product = [&](int x, int u, bool first) {
        const uint32_t b = ring_addr + (NS + vst) * C::stage;
#pragma unroll
        for (int k = 0; k < KT / 16; ++k)
          mma_ts(tmem + C::o_col + x * D, tmem + 128 * u + 8 * k, desc(b + 2048 * k, PANEL), idesc(128, D, 1),
                 !(first && k == 0));
        commit(bar(o_full + x));
      };
      auto wait_q = [&](int x) {
        if (!wait(q_full + x, (q_ph >> x) & 1)) return false;
        q_ph ^= 1u << x;
        return true;
      };
      auto wait_p = [&](int u) {
        if (!wait(p_full + u, (p_ph >> u) & 1)) return false;
        p_ph ^= 1u << u;
        tc_after();
        return true;
      };
      bool first = true;  // of the item's products
      uint32_t step = 0;
      // the scores of the very first tile
      bool ok = wait(full + kst, kph) && wait_q(0);
      bool two = T == 2 && rows_of(wk.cur, 1) > 0;
      if (ok) {
        tc_after();
        scores(0, 0);
        if (two && (ok = wait_q(1))) scores(1, 1);
      }
      if (ok) {
        commit(bar(empty + kst));
        advance(kst, kph);
      }
      while (ok) {
        Walk<TYPE, D> nx = wk;
        const bool new_item = nx.next(p), more = nx.w < nx.w1;
        const bool two_next = T == 2 && rows_of(nx.cur, 1) > 0;
        if (T == 2) {
          // product and next scores of one tile, then of the other; between items both products first
          if (!(ok = wait(full + NS + vst, vph) && wait_p(0))) break;
          product(0, 0, first);
          if (more && !new_item) {
            if (!(ok = wait(full + kst, kph))) break;
            tc_after();
            scores(0, 0);
          }
          if (two) {
            if (!(ok = wait_p(1))) break;
            product(1, 1, first);
          }
          commit(bar(empty + NS + vst));
          advance(vst, vph);
          if (!more) break;
          if (new_item) {
            if (!(ok = wait(full + kst, kph) && wait_q(0))) break;
            tc_after();
            scores(0, 0);
            if (two_next && !(ok = wait_q(1))) break;
          }
          if (two_next) scores(1, 1);
          commit(bar(empty + kst));
          advance(kst, kph);
        } else {
          const int u = step & 1;
          auto next_scores = [&]() {
            if (!wait(full + kst, kph) || (new_item && !wait_q(0))) return false;
            tc_after();
            scores(0, u ^ 1);
            commit(bar(empty + kst));
            advance(kst, kph);
            return true;
          };
          if (more && !new_item && !(ok = next_scores())) break;
          if (!(ok = wait(full + NS + vst, vph) && wait_p(u))) break;
          product(0, u, first);
          commit(bar(empty + NS + vst));
          advance(vst, vph);
          if (!more) break;
          if (new_item && !(ok = next_scores())) break;
        }
        first = new_item;
        two = two_next;
        wk = nx;
        ++step;
      }
      // every MMA issued above has completed once `done` flips
      commit(bar(done));
      for (uint32_t i = 0; i < ptx::kWaitLimit && !ptx::mbar_try_wait(bar(done), 0u); ++i) {
      }
    }
    __syncwarp();
  } else if (!C::q) {
    // ------------------------------------------------------------------ TMA loaders: K, V
    const int kv = warp - C::load_warp;
    if (kv < 2) {
      const CUtensorMap* map = kv ? &tv : &tk;
      const uint32_t ring_addr = ptx::smem_u32(ring) + kv * NS * C::stage;
      const int shift = p.page_shift, ps = p.page_size, npg = KT >> shift;  // pages of a tile
      const int pg = lane & (npg - 1), panel = lane / npg;
      uint32_t st = 0, ph = 0, aux_ph = 0;
      int last_par[NS];
#pragma unroll
      for (int s = 0; s < NS; ++s) last_par[s] = -1;
      bool ok = true;
      while (wk.w < wk.w1) {
        const Cursor& cur = wk.cur;
        const int t = wk.tile() * KT, tok = t + (pg << shift);
        // a page whose tokens are there and may be seen by some row
        const bool there = tok < cur.len && tok + ps > cur.lo;
        int page = there ? __ldg(p.page_table + (long long)cur.seq * p.table_stride + (tok >> shift)) : 0;
        const bool good = there && (unsigned)page < (unsigned)p.n_pages;
        const uint32_t pages = __ballot_sync(0xffffffffu, good) & ((1u << npg) - 1u);
        const bool bad = __any_sync(0xffffffffu, there && !good);
        if (bad && lane == 0) atomicOr(p.error_word, FT_DEVERR_BAD_INDEX);
        // rows to be cleared: of V whatever no row may see or that holds no token (it meets
        // probabilities of zero, and must not be NaN), of K those of a bad page
        const bool clear = kv ? pages != (1u << npg) - 1u || t + KT > cur.len : bad;
        if (!(ok = wait_all(empty + kv * NS + st, ph ^ 1u))) break;
        const uint32_t dst = ring_addr + st * C::stage;
        const uint32_t fb = bar(full + kv * NS + st), lb = clear ? bar(aux + kv) : fb;
        if (lane == 0) ptx::mbar_arrive_expect_tx(lb, __popc(pages) * ps * 128 * C::panels);
        __syncwarp();
        if (good && panel < C::panels)
          tma2d(dst + panel * PANEL + (pg << shift) * 128, map, 64 * panel,
                (page * p.n_kv_heads + cur.head) << shift, lb);
        if (clear) {
          if (!(ok = wait_all(aux + kv, aux_ph))) break;
          aux_ph ^= 1u;
          for (int r = lane; r < KT; r += 32)
            if (!((pages >> (r >> shift)) & 1u) || t + r >= cur.len)
              for (int i = 0; i < 8 * C::panels; ++i)
                *reinterpret_cast<uint4*>(ring + (kv * NS + st) * C::stage + (i >> 3) * PANEL + r * 128 + (i & 7) * 16) =
                    make_uint4(0, 0, 0, 0);
          fence_async();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(fb);
        }
        last_par[st] = (int)ph;
        if (++st == (uint32_t)NS) {
          st = 0;
          ph ^= 1u;
        }
        wk.next(p);
      }
      if (*abort_flag && lane == 0) {  // copies still in flight end before the CTA does
        for (int s = 0; s < NS; ++s)
          if (last_par[s] >= 0)
            for (uint32_t i = 0; i < ptx::kWaitLimit && !ptx::mbar_try_wait(bar(full + kv * NS + s), (uint32_t)last_par[s]); ++i) {
            }
        for (uint32_t i = 0; i < ptx::kWaitLimit && !ok && !ptx::mbar_try_wait(bar(aux + kv), aux_ph); ++i) {
        }
      }
    }
  } else if (warp >= C::load_warp) {
    // ------------------------------------------------------------------ decoding loaders
    // The codes of the next tile are fetched before those of the last one are decoded.  K is
    // one tile ahead of V, as its products are.
    const int lt = tid - 32 * C::load_warp;  // 0..127
    uint32_t st[2] = {0, 0}, ph[2] = {0, 0};
    bool ok = true;
    auto put = [&](int kv, const Raw<TYPE, D>& x) {
      if (!wait_all(empty + kv * NS + st[kv], ph[kv] ^ 1u)) return false;
      raw_store<TYPE, D>(ring + (kv * NS + st[kv]) * C::stage, lt, x);
      fence_async();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar(full + kv * NS + st[kv]));
      if (++st[kv] == (uint32_t)NS) {
        st[kv] = 0;
        ph[kv] ^= 1u;
      }
      return true;
    };
    Raw<TYPE, D> xk, xv;
    raw_load<TYPE, D>(p, wk.cur, wk.tile() * KT, p.k, p.ks, lt, xk);
    raw_load<TYPE, D>(p, wk.cur, wk.tile() * KT, p.v, p.vs, lt, xv);
    ok = put(0, xk);
    while (ok && wk.w < wk.w1) {
      wk.next(p);
      const bool more = wk.w < wk.w1;
      const int t = wk.tile() * KT;
      if (more) raw_load<TYPE, D>(p, wk.cur, t, p.k, p.ks, lt, xk);
      if (T == 1 && more) {  // the next scores come before the product
        if (!(ok = put(0, xk))) break;
        if (!(ok = put(1, xv))) break;
      } else {
        if (!(ok = put(1, xv))) break;
        if (more && !(ok = put(0, xk))) break;
      }
      if (more) raw_load<TYPE, D>(p, wk.cur, t, p.v, p.vs, lt, xv);
    }
  }
  __syncwarp();
  tc_before();
  __syncthreads();
  if (warp == C::mma_warp) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

// ------------------------------------------------------------------------------ host

inline PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  return fn;
}

// The cache's rows as a 2-D tensor [rows][D]: boxes of one page and head, 64 columns wide.
inline cudaError_t page_map(CUtensorMap* m, const void* base, int D, const AttnParams& p) {
  if (!encoder()) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)p.n_pages * p.n_kv_heads * p.page_size};
  const cuuint64_t strides[1] = {(cuuint64_t)D * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)p.page_size}, one[2] = {1, 1};
  const CUresult r = encoder()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, one,
                               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int TYPE, int D>
cudaError_t launch(const AttnParams& p, int n_sm, cudaStream_t s) {
  using C = Cfg<TYPE, D>;
  static_assert(sizeof(PlanSmem) <= 2 * C::stages * C::stage, "the plan fits the ring");
  CUtensorMap tk{}, tv{};
  cudaError_t e = cudaSuccess;
  if (!C::q) {
    e = page_map(&tk, p.k, D, p);
    if (e == cudaSuccess) e = page_map(&tv, p.v, D, p);
  }
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(attn_chunk_kernel<TYPE, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem);
  if (e != cudaSuccess) return e;
  attn_chunk_kernel<TYPE, D><<<n_sm, C::threads, C::smem, s>>>(tk, tv, p);
  return cudaGetLastError();
}

template <int TYPE>
cudaError_t launch_type(const AttnParams& p, int D, int n_sm, cudaStream_t s) {
  return D == 64 ? launch<TYPE, 64>(p, n_sm, s) : D == 128 ? launch<TYPE, 128>(p, n_sm, s) : launch<TYPE, 256>(p, n_sm, s);
}

}  // namespace chunk
}  // namespace kv
}  // namespace ft

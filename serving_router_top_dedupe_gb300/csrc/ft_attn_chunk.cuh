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
// Probabilities are rounded to BF16 for the second product, queries and keys are as they came;
// scores, sums and outputs are FP32 until the end.
//
// Bound by the tensor core together with shared memory: a step of two row tiles is 32 MMAs of 64
// clocks, which read 128 bytes a clock of operands while the next tiles are written, and takes
// about 3500 clocks (84 for an MMA; the rest is between batches of MMAs, whose queue holds three).
// With 64-wide heads the softmax is as long as the products; with 256-wide ones every CTA's row tile
// takes all of K and V out of L2, 128 KB a tile and SM, and that bounds it over long caches.
// Measured, other inputs each time (the same again and again): 8192 new tokens, 32 query heads over 4
// of 128, BF16: 464 us (462) = 1184 TFLOP/s; 2048 over 65536 (MXFP8, decoded once): 1676 us (1646) =
// 1292; 500 over 100001, heads of 256: 744 us (700) = 1098.  Quantised pages decoded where they are
// read, 512 rows over 16 x 8192 tokens of 4 x 128: MXFP8 203 us, MXFP4 181, BF16 144: there the
// decoding warps bound it.
//
// Warps 0-3 (and 4-7): softmax, output.  Then one warp that issues every MMA, and the loaders:
// two warps of TMA (K, V) for a BF16 cache, eight warps that decode into the same layout for a
// quantised one.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "ft_attn_masked.cuh"
#include "ft_attn_rows.cuh"
#include "ft_ptx.cuh"

namespace ft {
namespace kv {
namespace chunk {

using rows::e2m1_bits;
using rows::e4m3_bits;
using rows::ex2;
using rows::pack;

constexpr int KT = 128;           // cached tokens of a tile
constexpr int PANEL = KT * 128;   // bytes of 64 columns of a tile: rows of 128 bytes, 128-byte swizzle
// Tiles' time that a part of an item costs the join: an estimate on which little hangs, as 0 to 2
// measure the same wherever chunks fill the GPU.
constexpr float kJoin = 1.2f;
constexpr float kSlack = 8.f;     // log2 units by which scores may pass the running maximum

template <int TYPE, int D>
struct Cfg {
  static constexpr bool q = TYPE != FT_KV_BF16;
  static constexpr int tiles = D <= 128 ? 2 : 1;
  static constexpr int RB = 128 * tiles;
  // Counts of an item besides its tiles: loading queries, joining and storing outputs (8192 new
  // tokens: 0 746 us, 3 463, 8 476).
  static constexpr int OV = D == 64 ? 5 : 3;
  static constexpr int panels = D / 64;
  static constexpr int stage = panels * PANEL;
  static constexpr int stages = D == 64 ? 4 : D == 128 ? 2 : 1;  // of K, and of V
  static constexpr int soft_warps = 4 * tiles;
  static constexpr int mma_warp = soft_warps, load_warp = soft_warps + 4;
  static constexpr int threads = 32 * (soft_warps + (q ? 12 : 4));
  static constexpr int qbytes = tiles * stage;
  static constexpr int out_bytes = soft_warps * 32 * 128;  // 64 output columns of each warp's rows
  static constexpr int walks = q ? 8 * 112 : 0;            // where the loaders' walks wait
  static constexpr int smem = 1024 + qbytes + 2 * stages * stage + out_bytes + 512 + walks;
  // Registers of the softmax, MMA and loader warps out of those that the block starts with:
  // BF16, two tiles (168 x 384 = 64512): 216 x 256 + 72 x 128 = 64512;
  // quantised, two tiles (96 x 640 = 61440): 136 x 256 + 48 x 128 + 80 x 256 = 61440
  // (64 for the loaders leaves their loads in flight no room: MXFP8, heads of 128, 512 rows over 16 x 8192
  // tokens 265 us, with 72 203, with 80 197);
  // quantised, one tile (128 x 512 = 65536): 192 x 128 + 64 x 128 + 128 x 256 = 65536.
  static constexpr bool split = q || tiles == 2;
  static constexpr int soft_regs = !q ? 216 : tiles == 2 ? 136 : 192;
  static constexpr int mma_regs = !q ? 72 : tiles == 2 ? 48 : 64;
  static constexpr int load_regs = tiles == 2 ? 80 : 128;
  // what the block starts with; the softmax warps raise their share, the others give some up (a
  // warp that asks to give up and names more than it has is an illegal instruction)
  static constexpr int launch_regs = 65536 / threads / 8 * 8 < 256 ? 65536 / threads / 8 * 8 : 255;
  static_assert(!split || (soft_regs >= launch_regs && mma_regs <= launch_regs && (!q || load_regs <= launch_regs) &&
                           32 * (soft_warps * soft_regs + 4 * mma_regs + (q ? 8 * load_regs : 0)) <= launch_regs * threads),
                "shares of the registers");
  static constexpr int batch = !q && tiles == 2 ? 128 : 64;  // score columns that a softmax thread holds
  static constexpr size_t slot_floats = (size_t)RB * (D + 2);
  static constexpr int o_col = 256;  // TMEM: S (and P) at 0 and 128, O behind
};

__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// Whether a phase has passed, without waiting for it.
__device__ __forceinline__ bool passed(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}

// Shared-memory matrix descriptor, 128-byte swizzle: 8-row atoms of 1024 bytes (stride byte
// offset); lead: bytes from one 64-column panel to the next, for the operand whose columns
// run along the 128-byte rows (V), unused by the other (Q, K).  desc_lo is the low word, to
// which offsets / 16 may be added.
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lead) {
  uint32_t lo = ((saddr & 0x3FFFFu) >> 4) | (lead >> 4) << 16;
  asm volatile("" : "+r"(lo));  // formed where it is used: the issuing thread has few registers
  return lo;
}
__device__ __forceinline__ uint64_t desc(uint32_t lo) {
  return (uint64_t)((1024u >> 4) | 1u << 14 | 2u << 29) << 32 | lo;
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

// N consecutive 32-bit columns of this thread's TMEM lane.
template <int N>
__device__ __forceinline__ void tld(uint32_t a, uint32_t* r) {
  static_assert(N == 32, "columns of a load");
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(a));
}
template <int N>
__device__ __forceinline__ void tst(uint32_t a, const uint32_t* r) {
  static_assert(N == 32, "columns of a store");
  asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(a), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
               : "memory");
}
// The loaded registers go through the wait, so that nothing reads them earlier.
template <int N>
__device__ __forceinline__ void tld_wait(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
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

template <int TYPE, int D>
using ChunkWalk = Walk<Cfg<TYPE, D>::RB, KT, Cfg<TYPE, D>::OV>;

__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Scale code -> a pair of BF16 multipliers: 2^e (NaN for code 255) times what the codes' bits lack.
template <int TYPE>
__device__ __forceinline__ uint32_t multiplier(uint32_t code) {
  constexpr uint32_t lack = TYPE == FT_KV_MXFP8 ? 0x7B807B80u   // 2^120
                                                : 0x76807680u;  // 2^110: 2^-16 is left in
  return mul2((code << 7 | (code + 1) >> 8) * 0x00010001u, lack);
}

// 16 bytes of codes -> 16 (MXFP8) or 32 (MXFP4) BF16 values in their order.
template <int TYPE>
__device__ __forceinline__ void decode16(uint4 w, uint32_t scale, uint4* out) {
  const uint32_t m = multiplier<TYPE>(scale);
  const uint32_t in[4] = {w.x, w.y, w.z, w.w};
  uint32_t o[16];
  if (TYPE == FT_KV_MXFP8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[2 * i] = mul2(e4m3_bits<true>(__byte_perm(in[i], 0, 0x1404)), m);
      o[2 * i + 1] = mul2(e4m3_bits<true>(__byte_perm(in[i], 0, 0x3424)), m);
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

// What a loader keeps of an item while it is at it (the rest of its walk waits in shared memory).
struct Part {
  const int32_t* table;  // the sequence's row of the page table
  int lo, hi, head;
  int t, left;           // first token of the next tile, tiles left in this CTA's part of the item
};

// A loader notes, before it hands a tile on, that values that are not finite were left out of the
// item with this number (of the CTA's items).  The place is shared with items 8, 16, ... later, so
// a row that comes late may be told so for nothing, which does no harm, but never misses it.
__device__ __forceinline__ void note(volatile uint32_t* found, uint32_t item) { found[item & 7] = item + 1; }
__device__ __forceinline__ bool noted(const volatile uint32_t* found, uint32_t item) { return found[item & 7] > item; }

// Page ids of a tile: lane i (and i + 8, ...) holds that of tokens [t + 16 i, t + 16 i + 16), or
// -1 where no row sees them.
__device__ __forceinline__ int tile_pages(const AttnParams& p, const Part& it, int t, int lane) {
  const int tok = t + 16 * (lane & 7);
  if (tok >= it.hi || tok + 16 <= it.lo) return -1;
  const int page = __ldg(it.table + (tok >> p.page_shift));
  if ((unsigned)page < (unsigned)p.n_pages) return page;
  atomicOr(p.error_word, FT_DEVERR_BAD_INDEX);
  return -1;
}

// 16-byte pieces of a tile's codes that one loader thread holds: piece lt % PR of rows
// (lt + 128 i) / PR.  A warp's pieces belong to 32 rows, and lane l holds the scale codes of
// the l-th of them (zero where nothing is seen: the codes loaded for such a row, from some
// other place of the cache, then stand for zeros).  some: the tokens outside of which only some
// rows see (of values; NULL for keys).  True: scales that stand for NaN were left out.
template <int TYPE, int D>
struct Raw {
  static constexpr int PR = row_bytes(TYPE, D) / 16;  // pieces of a row, and of a thread
  uint4 w[PR];
  uint32_t sc[D == 256 ? 2 : 1];
};

template <int TYPE, int D>
__device__ __forceinline__ bool raw_load(const AttnParams& p, const Part& it, int t, int pages, const uint8_t* base,
                                         const uint8_t* scales, const int* some, int lt, Raw<TYPE, D>& x) {
  constexpr int PR = Raw<TYPE, D>::PR;
  const int lane = lt & 31, in_page = p.page_size - 1;
  auto row_at = [&](int r, int page) {  // row of the cache; a page that is not there: some row
    return ((max(page, 0) * p.n_kv_heads + it.head) << p.page_shift) + ((t + r) & in_page);
  };
#pragma unroll
  for (int i = 0; i < PR; ++i) {
    const int u = lt + 128 * i, r = u / PR;
    const int row = row_at(r, __shfl_sync(0xffffffffu, pages, r >> 4));
    x.w[i] = __ldg(reinterpret_cast<const uint4*>(base + (size_t)(uint32_t)row * row_bytes(TYPE, D)) + u % PR);
  }
  constexpr int per = 32 / PR;  // rows of a warp's piece i
  const int r = ((lt & ~31) + 128 * (lane / per)) / PR + lane % per;
  const int page = __shfl_sync(0xffffffffu, pages, r >> 4);
  const bool seen = page >= 0 && t + r < it.hi && t + r >= it.lo;
  const uint8_t* src = scales + (size_t)(uint32_t)row_at(r, page) * (D / 32);
  if constexpr (D == 64) {
    const uint32_t s = __ldg(reinterpret_cast<const uint16_t*>(src));
    x.sc[0] = seen ? s : 0u;
  } else if constexpr (D == 128) {
    const uint32_t s = __ldg(reinterpret_cast<const uint32_t*>(src));
    x.sc[0] = seen ? s : 0u;
  } else {
    const uint2 s = __ldg(reinterpret_cast<const uint2*>(src));
    x.sc[0] = seen ? s.x : 0u;
    x.sc[1] = seen ? s.y : 0u;
  }
  bool found = false;
  if (some && (t < some[0] || t + KT > some[1])) {
    if (t + r < some[0] || t + r >= some[1]) {
      found = keep_finite(x.sc[0]);
      if constexpr (D == 256) found |= keep_finite(x.sc[1]);
    }
  }
  return found;
}

template <int TYPE, int D>
__device__ __forceinline__ void raw_store(uint8_t* stage, int lt, const Raw<TYPE, D>& x) {
  constexpr int PR = Raw<TYPE, D>::PR, OUT = TYPE == FT_KV_MXFP8 ? 2 : 4;  // 16-byte pieces of BF16 for one of codes
  constexpr int per = 32 / PR;
  const int lane = lt & 31, pc = lt % PR, blk = TYPE == FT_KV_MXFP8 ? pc / 2 : pc;
#pragma unroll
  for (int i = 0; i < PR; ++i) {
    const int r = (lt + 128 * i) / PR, from = i * per + lane / PR;
    uint32_t s = __shfl_sync(0xffffffffu, x.sc[0], from);
    if constexpr (D == 256) {
      const uint32_t s1 = __shfl_sync(0xffffffffu, x.sc[1], from);
      s = blk < 4 ? s : s1;
    }
    uint4 o[OUT];
    decode16<TYPE>(x.w[i], (s >> (8 * (blk & 3))) & 0xffu, o);
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
  uint8_t* out_stage = ring + 2 * NS * C::stage;
  uint64_t* bars = reinterpret_cast<uint64_t*>(out_stage + C::out_bytes);
  uint64_t* full = bars;              // [2][NS] a tile of K, of V is in the ring
  uint64_t* empty = bars + 2 * NS;    // [2][NS] its products are done
  uint64_t* q_full = bars + 4 * NS;   // [2] the queries of a row tile are in place
  uint64_t* s_full = q_full + 2;      // [2] scores are in TMEM
  uint64_t* p_full = q_full + 4;      // [2] probabilities are in TMEM
  uint64_t* o_full = q_full + 6;      // [2] a product with V is done (two row tiles: the last of an item)
  uint64_t* aux = q_full + 8;         // [2] bytes of a tile whose ends are cleared before it is handed on
  uint64_t* done = q_full + 10;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(q_full + 11);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile uint32_t* found = tmem_slot + 2;  // [8]
  uint8_t* walks = reinterpret_cast<uint8_t*>(bars) + 512;
  static_assert(sizeof(ChunkWalk<TYPE, D>) <= 96, "a walk's place, and two integers");
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
    for (int i = 0; i < 8; ++i) found[i] = 0;
    ptx::mbar_fence_init();
  }
  pdl_wait();
  pdl_trigger();
  if (p.have && __ldg(p.have) != p.want) return;
  ChunkWalk<TYPE, D> wk;
  long long per;
  if (!plan<C::RB, KT, C::OV, C::threads>(p, *reinterpret_cast<PlanSmem*>(ring), blockIdx.x, gridDim.x, kJoin, wk, per)) return;
  if (warp == C::mma_warp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(ptx::smem_u32(tmem_slot))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_async();  // the ring held the plan: copies may write it now
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = *tmem_slot, q_addr = ptx::smem_u32(smem);
  auto wait = [&](uint64_t* b, uint32_t parity) { return ptx::mbar_wait(bar(b), parity, abort_flag, p.error_word); };
  // for a whole warp: all its lanes go on, or none
  auto wait_all = [&](uint64_t* b, uint32_t parity) { return (bool)__all_sync(0xffffffffu, wait(b, parity)); };
  // rows of row tile x of the item
  auto rows_of = [&](const Cursor& c, int x) { return min(c.n * p.group - c.rb * C::RB - 128 * x, 128); };

  if (warp < C::soft_warps) {
    // ------------------------------------------------------------------ softmax and output
    if (C::split) regs_up<C::soft_regs>();
    const int rt = warp >> 2;              // row tile
    const int r = (warp & 3) * 32 + lane;  // row of the tile = TMEM lane
    const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t o_tm = tl + C::o_col + rt * D;
    // never zero: what is masked is -inf before it is scaled
    const float c = fmaxf(fabsf(p.scale_log2) * left_in(TYPE), 1e-30f);
    const uint64_t c2 = f2(c, c);

    // an item's queries into shared memory, once no product reads the last ones
    auto load_q = [&](const Cursor& cur) {
      const int rows = rows_of(cur, rt);
      if (rows <= 0) return;
      constexpr int PQ = D / 8;  // 16-byte pieces of a row
      const int row0 = cur.rb * C::RB + 128 * rt, wt = tid & 127;
      const uint16_t* src = p.q + (long long)cur.q0 * p.q_stride + (long long)cur.head * p.group * D;
      const uint32_t dst = q_addr + rt * C::stage;
      auto at = [&](int u) {
        const int x = u / PQ, pc = u % PQ;
        return (uint32_t)((pc >> 3) * PANEL + x * 128 + (((pc & 7) ^ (x & 7)) << 4));
      };
#pragma unroll 4
      for (int i = 0; i < PQ; ++i) {
        const int u = wt + 128 * i, x = u / PQ, pc = u % PQ;
        const int tok = div_group(p, row0 + x), hd = row0 + x - tok * p.group;
        rows::cp_async16(dst + at(u), x < rows ? src + tok * p.q_stride + hd * D + pc * 8 : p.q, x < rows);
      }
      rows::cp_commit();
      rows::cp_wait<0>();
      if (p.scale_log2 < 0.f)  // a negative scale turns the queries' signs
        for (int i = 0; i < PQ; ++i) {
          uint4* v = reinterpret_cast<uint4*>(smem + rt * C::stage + at(wt + 128 * i));
          *v = make_uint4(v->x ^ 0x80008000u, v->y ^ 0x80008000u, v->z ^ 0x80008000u, v->w ^ 0x80008000u);
        }
      fence_async();
      ptx::mbar_arrive(bar(q_full + rt));
    };
    // 64 normalised output columns of the warp's rows, from the lanes' rows to rows in memory:
    // w: this row's 32 words of BF16 pairs
    uint8_t* stg = out_stage + warp * 4096;
    auto put_out = [&](const Cursor& cur, int rows, int col, const uint32_t* w) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        *reinterpret_cast<uint4*>(stg + lane * 128 + ((i ^ (lane & 7)) << 4)) =
            make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int x = 4 * i + (lane >> 3), row = (warp & 3) * 32 + x, pc = lane & 7;
        if (row < rows) {
          const int rr = cur.rb * C::RB + 128 * rt + row, tok = div_group(p, rr), hd = cur.head * p.group + rr - tok * p.group;
          *reinterpret_cast<uint4*>(p.out + (long long)(cur.q0 + tok) * p.out_stride + (long long)hd * D + col + pc * 8) =
              *reinterpret_cast<const uint4*>(stg + x * 128 + ((pc ^ (x & 7)) << 4));
        }
      }
      __syncwarp();
    };

    uint32_t s_ph = 0, pvs = 0;  // phases of s_full (bit u); products with V so far
    uint32_t items = 0;           // so far, of this row tile
    uint32_t step = 0, item = 0;
    bool ok = true;
    load_q(wk.cur);
    for (; ok && wk.more(); ++item) {  // one item
      const Cursor cur = wk.cur;
      const int rows = rows_of(cur, rt);
      const int rbase = cur.rb * C::RB + 128 * rt;
      // what this row sees: [lo, hi); what every row of the tile sees: [lo_max, hi_min)
      int lo = 0, hi = 1 << 30, lo_max = 0, hi_min = 1 << 30;
      if (rows > 0) {
        auto see = [&](int row, int& a, int& b) {
          const int pos = cur.len - cur.n + div_group(p, row);
          a = p.window > 0 ? max(pos - p.window + 1, 0) : 0;
          b = max(p.causal ? min(cur.len, pos + 1) : cur.len, a);
        };
        if (r < rows) see(rbase + r, lo, hi);  // rows that are not there see everything
        int x;
        see(rbase, x, hi_min);
        see(rbase + rows - 1, lo_max, x);
      }
      float m = -INFINITY, l = 0.f;
      bool first = true;  // no product with V yet
      const int steps = (int)(wk.end() - wk.w);
      int t = wk.tile() * KT;
      const int t_first = t;
      for (int j = 0; j < steps && rows > 0; ++j, ++step, t += KT) {
        const int u = T == 2 ? rt : (int)(step & 1);
        const uint32_t s_tm = tl + 128 * u;
        if (!(ok = wait_all(s_full + u, (s_ph >> u) & 1))) break;
        s_ph ^= 1u << u;
        tc_after();
        const bool edge = t < lo_max || t + KT > hi_min;
        // scores that this row does not see become -inf; a bit for each of 32 columns
        auto mask = [&](uint32_t* s, int col, int n) {
#pragma unroll
          for (int c32 = 0; c32 < n; c32 += 32) {
            const int a = t + col + c32;
            if (a >= lo_max && a + 32 <= hi_min) continue;  // every row of the tile sees these
            const int l0 = min(max(lo - a, 0), 32), h0 = min(max(hi - a, 0), 32);
            const uint32_t seen = (uint32_t)((1ull << h0) - 1ull) & (uint32_t)(~0ull << l0);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!(seen & (1u << i))) s[c32 + i] = 0xff800000u;
          }
        };
        constexpr int BC = C::batch;  // columns read from TMEM at once
        uint32_t pr[64];
        float mx = -INFINITY;
        uint64_t sum0, sum1;
        if (first) {  // a guess at the first maximum: that of 32 columns, the ones behind a window's edge
          const int col = t < lo_max ? KT - 32 : 0;
          uint32_t s[32];
          tld<32>(s_tm + col, s);
          tld_wait<32>(s);
          if (edge) mask(s, col, 32);
#pragma unroll
          for (int i = 0; i < 32; ++i) mx = fmaxf(mx, __uint_as_float(s[i]));
          m = mx * c;
        }
        for (;;) {
          // Probabilities against the running maximum as it is; a score that passes it by too
          // much is found on the way and starts the tile again.
          const float mu = m == -INFINITY ? 0.f : m;
          const uint64_t nm = f2(-mu, -mu);
          sum0 = sum1 = 0;
          mx = -INFINITY;
#pragma unroll
          for (int b = 0; b < KT / BC; ++b) {
            uint32_t s[BC];
#pragma unroll
            for (int i = 0; i < BC; i += 32) tld<32>(s_tm + b * BC + i, s + i);
            tld_wait<BC>(s);
            if (edge) mask(s, b * BC, BC);
#pragma unroll
            for (int i = 0; i < BC / 2; ++i) {
              const float x = __uint_as_float(s[2 * i]), y = __uint_as_float(s[2 * i + 1]);
              mx = fmaxf(mx, fmaxf(x, y));
              float e0, e1;
              unf2(fma2(f2(x, y), c2, nm), e0, e1);
              e0 = ex2(e0);
              e1 = ex2(e1);
              if (i & 1) sum1 = add2(sum1, f2(e0, e1));
              else sum0 = add2(sum0, f2(e0, e1));
              pr[b * BC / 2 + i] = pack(e0, e1);
            }
          }
          mx *= c;
          if (!__any_sync(0xffffffffu, mx > m + kSlack)) break;
          const float mn = fmaxf(m, mx);
          const float al = mn == -INFINITY ? 1.f : ex2(m - mn);
          l *= al;
          m = mn;
          if (!first) {
            // with two row tiles these scores were formed behind the last product
            if (T == 1 && !(ok = wait_all(o_full + rt, (pvs - 1) & 1))) break;
            tc_after();
            uint32_t o[32];
#pragma unroll 1
            for (int ch = 0; ch < D / 32; ++ch) {
              tld<32>(o_tm + 32 * ch, o);
              tld_wait<32>(o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * al);
              tst<32>(o_tm + 32 * ch, o);
            }
          }
        }
        if (!ok) break;
        tst<32>(s_tm, pr);
        tst<32>(s_tm + 32, pr + 32);
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
      wk.next_item(p);
      if (wk.more()) load_q(wk.cur);
      if (rows <= 0) continue;
      if (!(ok = wait_all(o_full + rt, (T == 1 ? pvs - 1 : items++) & 1))) break;
      tc_after();
      int ca, cb;
      piece_owners(cur, per, ca, cb);
      // values that were left out of the row's sums: use(column, value)
      auto left_out = [&](auto use) {
        if (!noted(found, item) || r >= rows) return;
        int all_lo, all_hi;
        all_see<C::RB>(p, cur, all_lo, all_hi);
        not_finite<TYPE, D>(p, cur, all_lo, all_hi, lo, hi, t_first, t, use);
      };
      float* lse = nullptr;
      if (p.lse && r < rows) {
        const int tok = div_group(p, rbase + r), hd = cur.head * p.group + rbase + r - tok * p.group;
        lse = p.lse + (long long)(cur.q0 + tok) * p.n_heads + hd;
      }
      if (ca == cb) {
        const float inv = l == 0.f ? 0.f : left_in(TYPE) / l;
#pragma unroll 1
        for (int ch = 0; ch < D / 64; ++ch) {
          uint32_t w[32];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t o[32];
            tld<32>(o_tm + 64 * ch + 32 * h, o);
            tld_wait<32>(o);
#pragma unroll
            for (int i = 0; i < 16; ++i)
              w[16 * h + i] = pack(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv);
          }
          put_out(cur, rows, 64 * ch, w);
        }
        left_out([&](int d, float v) {  // the warp's rows are in memory: put_out ends with a barrier of the warp
          const int tok = div_group(p, rbase + r), hd = cur.head * p.group + rbase + r - tok * p.group;
          __nv_bfloat16* to = reinterpret_cast<__nv_bfloat16*>(p.out) + (long long)(cur.q0 + tok) * p.out_stride + (long long)hd * D + d;
          *to = __float2bfloat16_rn(__bfloat162float(*to) + v);
        });
        if (lse) *lse = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994530942f;
      } else {
        // partial result: columns in groups of four, the rows of a group side by side
        const int me = blockIdx.x, at = 128 * rt + r;
        float* slot = p.partials + (size_t)(2 * me + (me == ca ? 1 : 0)) * C::slot_floats;
#pragma unroll 1
        for (int ch = 0; ch < D / 32; ++ch) {
          uint32_t o[32];
          tld<32>(o_tm + 32 * ch, o);
          tld_wait<32>(o);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            __stcg(reinterpret_cast<uint4*>(slot) + (8 * ch + i) * C::RB + at,
                   make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]));
        }
        __stcg(slot + C::RB * D + at, m);
        __stcg(slot + C::RB * (D + 1) + at, l);
        left_out([&](int d, float v) {
          float* to = slot + ((d >> 2) * C::RB + at) * 4 + (d & 3);
          __stcg(to, __ldcg(to) + v);
        });
        __syncwarp();
        // each warp joins its own 32 rows: the last CTA's warp to come, in the parts' order
        uint32_t* counter = p.counters + 8 * ca + 4 * rt + (warp & 3);
        __syncwarp();
        int is_last = 0;
        if (lane == 0) {  // with the warp's barriers, one lane's fences order all its accesses
          __threadfence();
          is_last = atomicAdd(counter, 1u) == (uint32_t)(cb - ca);
          if (is_last) {
            *counter = 0u;
            __threadfence();
          }
        }
        if (__shfl_sync(0xffffffffu, is_last, 0)) {
          __syncwarp();
          auto part = [&](int x) { return p.partials + (size_t)(2 * x + (x == ca ? 1 : 0)) * C::slot_floats; };
          float mm = -INFINITY, ll = 0.f;
#pragma unroll 8
          for (int x = ca; x <= cb; ++x) mm = fmaxf(mm, __ldcg(part(x) + C::RB * D + at));
#pragma unroll 8
          for (int x = ca; x <= cb; ++x)
            ll += __ldcg(part(x) + C::RB * (D + 1) + at) *
                  (mm == -INFINITY ? 0.f : ex2(__ldcg(part(x) + C::RB * D + at) - mm));
          const float inv = ll == 0.f ? 0.f : left_in(TYPE) / ll;
#pragma unroll 1
          for (int ch = 0; ch < D / 64; ++ch) {
            uint32_t w[32];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float acc[32];
#pragma unroll
              for (int i = 0; i < 32; ++i) acc[i] = 0.f;
#pragma unroll 2
              for (int x = ca; x <= cb; ++x) {
                const float wx = mm == -INFINITY ? 0.f : ex2(__ldcg(part(x) + C::RB * D + at) - mm);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  const float4 v = __ldcg(reinterpret_cast<const float4*>(part(x)) + (16 * ch + 8 * h + i) * C::RB + at);
                  acc[4 * i] += v.x * wx;
                  acc[4 * i + 1] += v.y * wx;
                  acc[4 * i + 2] += v.z * wx;
                  acc[4 * i + 3] += v.w * wx;
                }
              }
#pragma unroll
              for (int i = 0; i < 16; ++i) w[16 * h + i] = pack(acc[2 * i] * inv, acc[2 * i + 1] * inv);
            }
            put_out(cur, rows, 64 * ch, w);
          }
          if (lse) *lse = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * 0.69314718055994530942f;
        }
      }
    }
  } else if (warp < C::soft_warps + 4) {
    if (C::split) regs_down<C::mma_regs>();
    // ------------------------------------------------------------------ MMA issuer
    if (warp == C::mma_warp && lane == 0) {
      const uint32_t ring_addr = ptx::smem_u32(ring);
      uint32_t kst = 0, vst = 0, kph = 0, vph = 0;  // ring positions and phases
      uint32_t q_ph = 0, p_ph = 0;
      auto advance = [&](uint32_t& st, uint32_t& ph) {
        if (++st == (uint32_t)NS) {
          st = 0;
          ph ^= 1u;
        }
      };
      // scores of row tile x into S buffer u, from the K stage at kst.  mid: what the thread does
      // while the last two MMAs are still to be issued, and the ones before keep the tensor core.
      auto scores = [&](int x, int u, auto mid) {
        const uint32_t a = desc_lo(q_addr + x * C::stage, 0), b = desc_lo(ring_addr + kst * C::stage, 0);
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          if (k == D / 16 - 2) mid();
          const uint32_t off = ((k >> 2) * PANEL + 32 * (k & 3)) >> 4;
          mma_ss(tmem + 128 * u, desc(a + off), desc(b + off), idesc(128, KT, 0), k != 0);
        }
        commit(bar(s_full + u));
      };
      auto product = [&](int x, int u, bool first, bool last, auto mid) {
        const uint32_t b = desc_lo(ring_addr + (NS + vst) * C::stage, PANEL);
#pragma unroll
        for (int k = 0; k < KT / 16; ++k) {
          if (k == KT / 16 - 2) mid();
          mma_ts(tmem + C::o_col + x * D, tmem + 128 * u + 8 * k, desc(b + (2048 >> 4) * k), idesc(128, D, 1),
                 !(first && k == 0));
        }
        if (T == 1 || last) commit(bar(o_full + x));
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
      auto nothing = [] {};
      // The issuing thread must not keep the tensor core waiting, whose queue holds about three
      // MMAs: what changes from item to item is worked out between items, and waits and releases
      // that need not stand between two batches of MMAs are done inside a batch.
      uint32_t u = 0;  // S buffer of the step (one row tile)
      bool ok = true;
      while (ok && wk.more()) {
        const int n = (int)(wk.end() - wk.w);
        const bool two = T == 2 && rows_of(wk.cur, 1) > 0;
        // the first scores of the item
        if (!(ok = wait(full + kst, kph) && wait_q(0))) break;
        tc_after();
        scores(0, T == 2 ? 0 : u, nothing);
        if (two) {
          if (!(ok = wait_q(1))) break;
          scores(1, 1, nothing);
        }
        commit(bar(empty + kst));
        advance(kst, kph);
        bool p_there = false;  // of the second row tile, seen ahead of time
        for (int j = 0; j < n; ++j) {
          const bool more = j + 1 < n;
          if (T == 2) {  // product and next scores of one row tile, then of the other
            if (!(ok = wait(full + NS + vst, vph) && (!more || wait(full + kst, kph)) && wait_p(0))) break;
            product(0, 0, j == 0, !more, nothing);
            auto let_v_go = [&] {
              commit(bar(empty + NS + vst));
              advance(vst, vph);
            };
            if (two) {
              if (more) scores(0, 0, [&] { p_there = passed(bar(p_full + 1), (p_ph >> 1) & 1); });
              if (more && p_there) {
                p_ph ^= 2u;
                tc_after();
              } else if (!(ok = wait_p(1))) {
                break;
              }
              product(1, 1, j == 0, !more, nothing);
            }
            if (more) {
              scores(two, two, let_v_go);
              commit(bar(empty + kst));
              advance(kst, kph);
            } else {
              let_v_go();
            }
          } else {  // the next scores are formed during the softmax
            if (more) {
              if (!(ok = wait(full + kst, kph))) break;
              tc_after();
              scores(0, u ^ 1, nothing);
              commit(bar(empty + kst));
              advance(kst, kph);
            }
            if (!(ok = wait(full + NS + vst, vph) && wait_p(u))) break;
            product(0, u, j == 0, !more, nothing);
            commit(bar(empty + NS + vst));
            advance(vst, vph);
            u ^= 1;
          }
        }
        wk.next_item(p);
      }
      // every MMA issued above has completed once `done` flips
      commit(bar(done));
      for (uint32_t i = 0; i < ptx::kWaitLimit && !ptx::mbar_try_wait(bar(done), 0u); ++i) {
      }
    }
    __syncwarp();
    // ------------------------------------------------------------------ TMA loaders: K, V
    const int kv = warp - C::mma_warp - 1;
    if (!C::q && (kv == 0 || kv == 1)) {
      const CUtensorMap* map = kv ? &tv : &tk;
      const uint32_t ring_addr = ptx::smem_u32(ring) + kv * NS * C::stage;
      const int shift = p.page_shift, ps = p.page_size, npg = KT >> shift;  // pages of a tile
      const int pg = lane & (npg - 1), panel = lane / npg;
      uint32_t st = 0, ph = 0, aux_ph = 0;
      int last_par[NS];
#pragma unroll
      for (int s = 0; s < NS; ++s) last_par[s] = -1;
      bool ok = true;
      uint32_t item = 0;
      int all_lo, all_hi;
      all_see<C::RB>(p, wk.cur, all_lo, all_hi);
      while (wk.more()) {
        const Cursor& cur = wk.cur;
        const int t = wk.tile() * KT, tok = t + (pg << shift);
        // a page whose tokens are there and may be seen by some row
        const bool there = tok < cur.hi && tok + ps > cur.lo;
        int page = 0;
        if (there)
          page = p.staged ? __ldg(p.staged + cur.seq) + (tok >> shift)
                          : __ldg(p.page_table + (long long)cur.seq * p.table_stride + (tok >> shift));
        const bool good = there && (unsigned)page < (unsigned)p.n_pages;
        const uint32_t pages = __ballot_sync(0xffffffffu, good) & ((1u << npg) - 1u);
        const bool bad = __any_sync(0xffffffffu, there && !good);
        if (bad && lane == 0) atomicOr(p.error_word, FT_DEVERR_BAD_INDEX);
        // rows to be cleared: of V whatever no row may see (it meets probabilities of zero, and must
        // not be NaN), the tokens that share a page with those that some row sees among them; of K
        // those of a bad page.  Of V, tokens that only some rows see are looked at.
        const bool clear = kv ? pages != (1u << npg) - 1u || t + KT > min(cur.hi, all_hi) || t < max(cur.lo, all_lo) : bad;
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
          // rows [x0, x1) are as every row of the block sees them, but for pages that are not there
          bool left_out = false;
          const int x0 = max(cur.lo, all_lo) - t, x1 = min(cur.hi, all_hi) - t;
          auto sweep = [&](int ra, int rb) {
            constexpr int P = 8 * C::panels;  // 16-byte pieces of a row
#pragma unroll 2
            for (int u = ra * P + lane; u < rb * P; u += 32) {
              const int r = u / P, i = u % P, j = t + r;
              uint4* at = reinterpret_cast<uint4*>(ring + (kv * NS + st) * C::stage + (i >> 3) * PANEL + r * 128 +
                                                   (((i & 7) ^ (r & 7)) << 4));
              if (!((pages >> (r >> shift)) & 1u) || j >= cur.hi || j < cur.lo) {
                *at = make_uint4(0, 0, 0, 0);
              } else if (kv && (r < x0 || r >= x1)) {
                uint4 v = *at;
                if (keep_finite(v)) *at = v, left_out = true;
              }
            }
          };
          if (bad || x0 >= x1) {
            sweep(0, KT);
          } else {
            sweep(0, min(x0, KT));
            sweep(max(x1, 0), KT);
          }
          if (left_out) note(found, item);
          fence_async();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(fb);
        }
        last_par[st] = (int)ph;
        if (++st == (uint32_t)NS) {
          st = 0;
          ph ^= 1u;
        }
        if (wk.next(p)) {
          ++item;
          all_see<C::RB>(p, wk.cur, all_lo, all_hi);
        }
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
  } else {
    // ------------------------------------------------------------------ decoding loaders
    regs_down<C::load_regs>();
    // Four warps for K, four for V.  The page ids of a tile are fetched two tiles ahead, its
    // codes one tile ahead, while the tile before is decoded.
    const int lt = (tid - 32 * C::load_warp) & 127, kv = (warp - C::load_warp) >> 2;
    const uint8_t* base = kv ? p.v : p.k;
    const uint8_t* scales = kv ? p.vs : p.ks;
    uint8_t* my_ring = ring + kv * NS * C::stage;
    uint32_t st = 0, ph = 0;
    uint8_t* mine = walks + 112 * (warp - C::load_warp);
    ChunkWalk<TYPE, D>* my_walk = reinterpret_cast<ChunkWalk<TYPE, D>*>(mine);
    int* all = reinterpret_cast<int*>(mine + 96);  // what every row of the item's block sees
    const int* some = kv ? all : nullptr;
    uint32_t item = 0;
    Part it;
    auto enter = [&](const ChunkWalk<TYPE, D>& w) {
      it.table = p.page_table + (long long)w.cur.seq * p.table_stride;
      it.lo = w.cur.lo;
      it.hi = w.cur.hi;
      it.head = w.cur.head;
      it.t = w.tile() * KT;
      it.left = w.more() ? (int)(w.end() - w.w) : 0;
      int all_lo, all_hi;
      all_see<C::RB>(p, w.cur, all_lo, all_hi);
      __syncwarp();
      if (lane == 0) {
        *my_walk = w;
        all[0] = all_lo;
        all[1] = all_hi;
      }
      __syncwarp();
    };
    // to the next tile; it.left is 0 behind the last one
    auto next = [&]() {
      it.t += KT;
      if (--it.left == 0) {
        ChunkWalk<TYPE, D> w = *my_walk;
        w.next_item(p);
        enter(w);
        ++item;
      }
    };
    enter(wk);
    Raw<TYPE, D> x;
    if (raw_load<TYPE, D>(p, it, it.t, tile_pages(p, it, it.t, lane), base, scales, some, lt, x)) note(found, item);
    next();
    int pages = it.left ? tile_pages(p, it, it.t, lane) : -1;
    for (bool last = false; !last;) {
      if (!wait_all(empty + kv * NS + st, ph ^ 1u)) break;
      raw_store<TYPE, D>(my_ring + st * C::stage, lt, x);
      last = it.left == 0;
      if (!last) {
        if (raw_load<TYPE, D>(p, it, it.t, pages, base, scales, some, lt, x)) note(found, item);
        next();
        if (it.left) pages = tile_pages(p, it, it.t, lane);
      }
      fence_async();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar(full + kv * NS + st));
      if (++st == (uint32_t)NS) {
        st = 0;
        ph ^= 1u;
      }
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
  static std::atomic<uint64_t> ready{0};  // devices whose limit is set
  if (e == cudaSuccess) e = prepare_kernel(attn_chunk_kernel<TYPE, D>, C::smem, ready);
  if (e != cudaSuccess) return e;
  return launch_k(attn_chunk_kernel<TYPE, D>, dim3(n_sm), dim3(C::threads), C::smem, s, true, tk, tv, p);
}

template <int TYPE>
cudaError_t launch_type(const AttnParams& p, int D, int n_sm, cudaStream_t s) {
  return D == 64 ? launch<TYPE, 64>(p, n_sm, s) : D == 128 ? launch<TYPE, 128>(p, n_sm, s) : launch<TYPE, 256>(p, n_sm, s);
}

}  // namespace chunk
}  // namespace kv
}  // namespace ft

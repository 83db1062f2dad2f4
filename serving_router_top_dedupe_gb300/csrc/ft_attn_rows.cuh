// Attention of few rows over the paged cache: single tokens, a few drafted tokens, and
// (block by block) any number of rows.
//
// Every part of an item keeps, for each row, m (a bound of the scores so far, in units of log 2),
// l = sum 2^(s_j - m) and o = sum 2^(s_j - m) v_j in FP32; parts with other bounds are added
// after multiplying with 2^(m - m').  out = o / l, lse = log 2 * (m + log2 l).
//
// A block is 16 or 32 rows of one cache head (the query heads of the group, times new tokens):
// one or two row tiles of mma.sync.  Each cached byte is used by these rows only, so reading the
// cache bounds this kernel, and next to that the decoding of quantised caches:
//  - a warp streams chunks of 16 or 32 tokens (cp.async into its own ring of stages, several
//    chunks ahead) and never waits for another warp; the four warps of a CTA take the four
//    chunks of a tile, each with its own running maximum, sum and accumulators, and join at the
//    end of the CTA's part of the item;
//  - rows lie in shared memory with their 16-byte pieces permuted by the row, so ldmatrix reads
//    keys and (transposed) values without bank conflicts;
//  - MXFP8 and MXFP4 codes go from ldmatrix to operands in registers.  Their scales stay outside.
//    Keys become FP16 (one conversion for two elements; FP16 holds every E4M3 and E2M1 number),
//    and a 1x32 block of them is a product of its own, added to the scores times its scale in
//    FP32.  The queries become FP16 times a power of two that brings a row's largest to 2^14 (exact
//    for elements down to 2^-28 of it; smaller ones are off by 2^-39 of the largest at most).
//    Values become BF16 (their codes' bits in BF16's places: the numbers times 2^-120 or 2^-126),
//    and probabilities take their scale and most of what the bits lack before they become BF16
//    too: FP32's exponents, so a term is rounded relative to itself, whatever the scales of other
//    tokens and blocks, seen or not, and no exponent is kept beside the running maximum.
//  - The order of the reduction is free, and so is the order of the value columns: keys are
//    taken in the order in which a 32-bit word holds their codes, with the queries arranged to
//    match, and a transposed 16-bit unit holds 2 (4) neighbouring value columns of a token,
//    which become the operands of 2 (4) column tiles.
// The running maximum moves only when a score passes it by 2^8 or more, so the accumulators
// are rarely rescaled.
//
// Roundings: probabilities (times the scale of quantised values) to BF16 for their product with the
// values: one rounding of half a unit in the last of 8 bits of each term, what the tensor core takes.
// Their sum is taken before it, so that it is not off by what rounds in one direction; everything
// summed is FP32.
//
// Measured: 64 single tokens over 16384 tokens each, 4 cache heads of 128, 8 rows of a head: BF16
// 322 us = 6.7 TB/s, bound by memory; MXFP8 211 us = 5.3 TB/s; MXFP4 199 us = 2.9 TB/s, bound by the
// decoding: both take about as many instructions for a chunk, 1090 for MXFP8, and issue one in 54 %
// of the clocks; 32 rows 328 and 317 us.  One sequence of 4001 tokens: 15 us, of which a launch, the plan,
// two tiles' latency and the join are nearly all.
#pragma once

#include "ft_attn_masked.cuh"
#include "ft_kv_internal.cuh"

namespace ft {
namespace kv {
namespace rows {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr float kSlack = 8.f;      // log2 units by which scores may pass the running maximum

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// 16-byte piece c of row r in a tile of rows of RBY bytes: pieces of the same column of eight
// neighbouring rows fall into different banks.
template <int RBY>
__device__ __forceinline__ uint32_t piece(int r, int c) {
  constexpr int per = RBY >= 128 ? 8 : RBY / 16;  // pieces of a 128-byte span that are permuted
  constexpr int rows_per = RBY >= 128 ? 1 : 128 / RBY;
  return (uint32_t)(r * RBY + ((c ^ ((r / rows_per) & (per - 1))) << 4));
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool there) {
  const uint32_t n = there ? 16u : 0u;  // 0: the 16 bytes are set to zero, nothing is read
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldm4(uint32_t* r, uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldm4t(uint32_t* r, uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}

__device__ __forceinline__ void ldm2(uint32_t* r, uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldm2t(uint32_t* r, uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(a) : "memory");
}

__device__ __forceinline__ void mma(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  const __nv_bfloat162 r = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void mma_f16(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Low and high 16 bits of a word: two E4M3 codes each -> FP16 pairs.
__device__ __forceinline__ void e4m3x4_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
// E4M3 codes in the low (HIGH: high) bytes of both halves -> the BF16 numbers they stand for, times
// 2^-120.
template <bool HIGH>
__device__ __forceinline__ uint32_t e4m3_bits(uint32_t w) {
  return ((HIGH ? w >> 4 : w << 4) & 0x07F007F0u) | ((HIGH ? w : w << 8) & 0x80008000u);
}
// Nibble I of both halves -> the BF16 numbers their E2M1 codes stand for, times 2^-126.
template <int I>
__device__ __forceinline__ uint32_t e2m1_bits(uint32_t w) {
  const uint32_t mag = I == 0 ? w << 6 : I == 1 ? w << 2 : I == 2 ? w >> 2 : w >> 6;
  const uint32_t sgn = w << (12 - 4 * I);
  return (mag & 0x01C001C0u) | (sgn & 0x80008000u);
}
// Byte i of a word: two E2M1 codes -> an FP16 pair.
__device__ __forceinline__ void e2m1x8_f16(uint32_t w, uint32_t* r) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

template <int TYPE, int D, int MT>
struct Cfg {
  static constexpr bool q = TYPE != FT_KV_BF16;
  static constexpr int RB = 16 * MT;  // rows of a block
  // Tokens of a warp's step.  Quantised: twice as many independent products in a chain that is long
  // for decoding (32 / 16 tokens: MXFP8 8 rows 211 / 230 us, MXFP4 199 / 224 at the size above; 32 rows
  // 328 / 355 and 317 / 337); 256-wide heads have no registers for that, BF16 has no such chain.
  static constexpr int CHUNK = q && D <= 128 ? 32 : 16;
  static constexpr int UT = CHUNK * kWarps;          // tokens of a tile
  // Counts of an item besides its tiles (64 ragged MXFP8 sequences: 0 92 us, 3 57, 8 65).
  static constexpr int OV = CHUNK == 32 ? 3 : 6;
  // Tiles' time that a part of an item costs the join (the same 57 us, with 2.0 72; one sequence
  // of 4001 tokens 15 and 21 us).
  static constexpr float join_cost = 0.35f;
  static constexpr int rby = row_bytes(TYPE, D), sby = scale_bytes(TYPE, D);
  static constexpr int kv_bytes = CHUNK * rby;
  static constexpr int stage = 2 * kv_bytes + 2 * CHUNK * sby;
  static constexpr int scales = q ? 2 * CHUNK * (D / 32) * 4 : 0;  // a warp's chunk of scales in FP32
  // per SM, as registers allow (MXFP8, 4 CTAs of 128 registers: 341 us in place of 205)
  static constexpr int ctas = D == 256 ? (q ? 2 : 1) : q && MT == 1 ? 3 : 2;
  static constexpr int room = ctas == 1 ? 200 * 1024 : ctas == 2 ? 100 * 1024 : 66 * 1024;
  static constexpr int fit = room / (kWarps * stage);
  static constexpr int stages = fit < 8 ? fit : 8;
  static constexpr int ring = kWarps * stages * stage;
  static constexpr int opitch = D + 8;  // floats of a row where the warps join
  static constexpr int join = kWarps * RB * opitch * 4;
  static constexpr int qfrag = MT * (D / 16) * 512;
  static constexpr int head = 1024 * MT;  // maxima and sums where the warps join, and the rows' query scales
  static constexpr int weights = 160 * ctas * RB * 8;  // and sums of an item's parts where CTAs join (up to 160 SMs)
  static constexpr int max0 = ring > join ? ring : join, max1 = max0 > weights ? max0 : weights;
  static constexpr int body = max1 > (int)sizeof(PlanSmem) ? max1 : (int)sizeof(PlanSmem);
  static constexpr int smem = qfrag + head + body + kWarps * scales;
  static constexpr size_t slot_floats = (size_t)RB * (D + 2);
  // The values' scales are staged times 2^lack, and sums are taken back by 2^taken once at the end:
  // together 2^120 or 2^126, which the values' bits lack.  A probability (2^8 at most) times the
  // largest scale (2^7 or 2^13) and 2^lack stays below 2^126.
  static constexpr int lack = TYPE == FT_KV_MXFP8 ? 108 : TYPE == FT_KV_MXFP4 ? 104 : 0;
  static constexpr int taken = TYPE == FT_KV_MXFP8 ? 12 : TYPE == FT_KV_MXFP4 ? 22 : 0;
  static constexpr bool q_regs = D <= 128 && MT == 1 && !q;  // the queries' operands stay in registers
};

// Column of the values that accumulator half h (columns 2c and 2c+1 of tile nt) stands for.
template <int TYPE>
__device__ __forceinline__ int out_col(int nt, int c, int h) {
  if (TYPE == FT_KV_BF16) return 8 * nt + 2 * c + h;
  if (TYPE == FT_KV_MXFP8) return 16 * (nt >> 1) + 4 * c + 2 * h + (nt & 1);
  return 32 * (nt >> 2) + 8 * c + 4 * h + (nt & 3);
}

// A warp's 16 x D accumulators, times f, into rows of shared memory.
template <int TYPE, int D>
__device__ __forceinline__ void put_rows(float* dst, int pitch, const float (*o)[4], float f, int g, int c) {
#pragma unroll
  for (int hr = 0; hr < 2; ++hr) {
    float* row = dst + (g + 8 * hr) * pitch;
    if (TYPE == FT_KV_BF16) {
#pragma unroll
      for (int nt = 0; nt < D / 8; ++nt)
        *reinterpret_cast<float2*>(row + 8 * nt + 2 * c) = make_float2(o[nt][2 * hr] * f, o[nt][2 * hr + 1] * f);
    } else if (TYPE == FT_KV_MXFP8) {
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
        *reinterpret_cast<float4*>(row + 16 * j + 4 * c) =
            make_float4(o[2 * j][2 * hr] * f, o[2 * j + 1][2 * hr] * f, o[2 * j][2 * hr + 1] * f, o[2 * j + 1][2 * hr + 1] * f);
    } else {
#pragma unroll
      for (int j = 0; j < D / 32; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<float4*>(row + 32 * j + 8 * c + 4 * h) =
              make_float4(o[4 * j][2 * hr + h] * f, o[4 * j + 1][2 * hr + h] * f, o[4 * j + 2][2 * hr + h] * f,
                          o[4 * j + 3][2 * hr + h] * f);
    }
  }
}

template <int TYPE, int D, int MT>
__global__ void __launch_bounds__(kThreads, (Cfg<TYPE, D, MT>::ctas)) attn_rows_kernel(const AttnParams p) {
  using C = Cfg<TYPE, D, MT>;
  constexpr int NT = D / 8, KS = D / 16, S = C::stages, RB = C::RB, NB = D / 32;
  constexpr int CHUNK = C::CHUNK, UT = C::UT, TT = CHUNK / 8;  // TT: column tiles of a chunk's scores
  extern __shared__ __align__(128) uint8_t smem[];
  uint4* qf = reinterpret_cast<uint4*>(smem);                 // [MT][KS][32] query operands
  float* join_m = reinterpret_cast<float*>(smem + C::qfrag);  // [kWarps][RB]
  float* join_l = join_m + kWarps * RB;                       // [kWarps][RB]
  float* q_scale = join_l + kWarps * RB;                      // [RB] scale of a row's scores
  float* row_l = q_scale + RB;                                // [RB] where CTAs join
  int* s_flag = reinterpret_cast<int*>(row_l + RB);
  int* s_found = s_flag + 1;                                  // values that are not finite were left out of the item
  uint8_t* body = smem + C::qfrag + C::head;
  float* join_o = reinterpret_cast<float*>(body);             // [kWarps][RB][opitch]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  pdl_wait();
  pdl_trigger();  // the next launch may take its place; it waits for this one's end before it reads
  Walk<RB, UT, C::OV> wk;
  long long per;
  if (!plan<RB, UT, C::OV, kThreads>(p, *reinterpret_cast<PlanSmem*>(body), blockIdx.x, gridDim.x, C::join_cost, wk, per)) return;
  __syncthreads();

  const uint32_t ring = smem_addr(body) + warp * S * C::stage;
  uint8_t* ring_g = body + warp * S * C::stage;
  float* sc_f = reinterpret_cast<float*>(body + C::body + warp * C::scales);  // [K, V][NB][CHUNK]

  for (;;) {
    // ---------------------------------------------------- this CTA's part of the item
    const Cursor& cur = wk.cur;
    const int ta = (int)(wk.w - cur.start), tb = (int)(wk.end() - cur.start);
    const int rows = min(cur.n * p.group - cur.rb * RB, RB);
    auto q_row = [&](int r) {
      const int rr = cur.rb * RB + r, tok = div_group(p, rr), hd = rr - tok * p.group;
      return p.q + (long long)(cur.q0 + tok) * p.q_stride + (long long)(cur.head * p.group + hd) * D;
    };
    if (tid == 0) *s_found = 0;
    // the first chunks are on their way while the queries are arranged
    const int n = tb - ta;
    const int32_t* table = p.page_table + (long long)cur.seq * p.table_stride;
    const int tok0 = (cur.t0 + ta) * UT + warp * CHUNK;  // the warp's first chunk
    auto wanted = [&](int k) { return k < n && tok0 + k * UT < cur.hi && tok0 + k * UT + CHUNK > cur.lo; };
    // page ids of the next chunk's 16-token halves; -1: no row sees them
    constexpr int HALVES = CHUNK / 16;
    int page_next[HALVES];
    auto fetch_pages = [&](int k) {
#pragma unroll
      for (int h = 0; h < HALVES; ++h) {
        const int t = tok0 + k * UT + 16 * h;
        page_next[h] = wanted(k) && t < cur.hi && t + 16 > cur.lo ? __ldg(table + (t >> p.page_shift)) : -1;
      }
    };
    fetch_pages(0);
    auto issue = [&](int k) {
      int page[HALVES];
#pragma unroll
      for (int h = 0; h < HALVES; ++h) page[h] = page_next[h];
      fetch_pages(k + 1);
      if (wanted(k)) {
        const uint32_t dst = ring + (uint32_t)(k % S) * C::stage;
        constexpr int PR = C::rby / 16, PS = C::sby;  // 16-byte pieces of a row; of 16 rows' scales
#pragma unroll
        for (int h = 0; h < HALVES; ++h) {
          const int t = tok0 + k * UT + 16 * h;
          const bool ok = (unsigned)page[h] < (unsigned)p.n_pages;
          if (!ok && t < cur.hi && t + 16 > cur.lo && lane == 0) atomicOr(p.error_word, FT_DEVERR_BAD_INDEX);
          const int r0 = max(cur.lo - t, 0), r1 = ok ? min(cur.hi - t, 16) : 0;  // rows to read; the others are zeros
          const long long row = (((long long)(ok ? page[h] : 0) * p.n_kv_heads + cur.head) << p.page_shift) +
                                (t & (p.page_size - 1));
          const uint8_t* ksrc = p.k + row * C::rby;
          const uint8_t* vsrc = p.v + row * C::rby;
          if (r0 == 0 && r1 == 16) {
#pragma unroll
            for (int i = 0; i < PR / 2; ++i) {
              const int u = lane + 32 * i;
              cp_async16(dst + piece<C::rby>(16 * h + u / PR, u % PR), ksrc + u * 16);
              cp_async16(dst + C::kv_bytes + piece<C::rby>(16 * h + u / PR, u % PR), vsrc + u * 16);
            }
          } else {
#pragma unroll 2
            for (int i = 0; i < PR / 2; ++i) {
              const int u = lane + 32 * i, r = u / PR, pc = u % PR;
              const bool there = r >= r0 && r < r1;
              cp_async16(dst + piece<C::rby>(16 * h + r, pc), ksrc + u * 16, there);
              cp_async16(dst + C::kv_bytes + piece<C::rby>(16 * h + r, pc), vsrc + u * 16, there);
            }
          }
          if constexpr (C::q) {
            if (lane < 2 * PS) {
              const int i = lane % PS;
              const uint8_t* src = (lane < PS ? p.ks : p.vs) + row * C::sby + i * 16;
              cp_async16(dst + 2 * C::kv_bytes + (lane < PS ? 0 : CHUNK * C::sby) + (h * PS + i) * 16, src, ok);
            }
          }
        }
      }
      cp_commit();
    };
#pragma unroll 1
    for (int k = 0; k < S - 1; ++k) issue(k);

    if (C::q) {  // the power of two that brings a row's largest query element to 2^14
      constexpr int TPR = kThreads / RB;  // threads of a row
      const int r = tid / TPR, sub = tid % TPR;
      uint32_t top = 0;
      if (r < rows) {
        const uint4* src = reinterpret_cast<const uint4*>(q_row(r));
#pragma unroll
        for (int i = sub; i < D / 8; i += TPR) {
          const uint4 v = __ldg(src + i);
          top = __vmaxu2(top, __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu), __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu)));
        }
      }
      top = max(top >> 16, top & 0xffffu);
#pragma unroll
      for (int d = 1; d < TPR; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
      // exponent of the power: 14 - (e - 127), within what an FP32 number can be; NaN and infinity stay
      const int k = top >= 0x7f80u || top < 0x80u ? 0 : 141 - (int)(top >> 7);
      if (sub == 0) q_scale[r] = __uint_as_float((uint32_t)(127 + min(k, 126)) << 23);
      __syncthreads();
    }
    for (int i = tid; i < MT * KS * 32; i += kThreads) {
      const int ks = (i >> 5) % KS, mt = i / (KS * 32), l = i & 31, gg = l >> 2, cc = l & 3;
      uint32_t a[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int r = 16 * mt + gg + 8 * (q & 1), kh = q >> 1;
        const int d = TYPE == FT_KV_BF16 ? 16 * ks + 2 * cc + 8 * kh : TYPE == FT_KV_MXFP8 ? 16 * ks + 4 * cc + 2 * kh
                                                              : 32 * (ks >> 1) + 8 * cc + 4 * (ks & 1) + 2 * kh;
        uint32_t v = r < rows ? __ldg(reinterpret_cast<const uint32_t*>(q_row(r) + d)) : 0u;
        if (C::q) v = pack_f16(__uint_as_float(v << 16) * q_scale[r], __uint_as_float(v & 0xffff0000u) * q_scale[r]);
        a[q] = v;
      }
      qf[i] = make_uint4(a[0], a[1], a[2], a[3]);
    }
    __syncthreads();
    // the cached tokens that this thread's rows g and g + 8 of a row tile see: [lo, hi)
    int lo[MT][2], hi[MT][2];
    float scale[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = 16 * mt + g + 8 * h;
        lo[mt][h] = hi[mt][h] = 0;
        scale[mt][h] = C::q ? p.scale_log2 / q_scale[r] : p.scale_log2;
        if (r < rows) {
          const int pos = cur.len - cur.n + div_group(p, cur.rb * RB + r);
          hi[mt][h] = p.causal ? min(cur.len, pos + 1) : cur.len;
          lo[mt][h] = p.window > 0 ? max(pos - p.window + 1, 0) : 0;
        }
      }
    // what every row of the block sees: chunks inside need no mask
    int all_lo, all_hi;
    all_see<RB>(p, cur, all_lo, all_hi);

    uint32_t qr[KS][4];
    if (C::q_regs) {
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) *reinterpret_cast<uint4*>(qr[ks]) = qf[ks * 32 + lane];
    }
    auto query = [&](int mt, int ks, uint32_t* a) {
      if (C::q_regs) {
#pragma unroll
        for (int q = 0; q < 4; ++q) a[q] = qr[ks][q];
      } else {
        *reinterpret_cast<uint4*>(a) = qf[(mt * KS + ks) * 32 + lane];
      }
    };
    float o[MT][NT][4];
    float m[MT][2], l[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[mt][i][j] = 0.f;
      m[mt][0] = m[mt][1] = -INFINITY;
      l[mt][0] = l[mt][1] = 0.f;
    }

#pragma unroll 1
    for (int k = 0; k < n; ++k) {
      __syncwarp();  // every lane is done with the stage that is filled next
      issue(k + S - 1);
      cp_wait<S - 1>();
      __syncwarp();
      if (!wanted(k)) continue;
      const int t = tok0 + k * UT;
      const uint32_t st = ring + (uint32_t)(k % S) * C::stage;
      const bool inside = t >= all_lo && t + CHUNK <= all_hi;
      if constexpr (C::q) {
        // The chunk's scale codes as FP32 powers of two (those of the values times 2^lack), zero for
        // tokens that are left out.
        const uint8_t* codes = ring_g + (k % S) * C::stage + 2 * C::kv_bytes;
        // Lane l takes the codes of token l % CHUNK: with 16 tokens of K or of V, with 32 of both.
        constexpr int SETS = CHUNK / 16;
        const int tok = lane % CHUNK;
        const bool in = t + tok >= cur.lo && t + tok < cur.hi;
#pragma unroll
        for (int i = 0; i < SETS; ++i) {
          const int set = SETS == 2 ? i : lane / CHUNK;  // 0: K, 1: V
          const uint8_t* src = codes + (set * CHUNK + tok) * NB;
          uint32_t w[NB > 4 ? 2 : 1];
          if constexpr (NB == 2) {
            w[0] = *reinterpret_cast<const uint16_t*>(src);
          } else {
            w[0] = *reinterpret_cast<const uint32_t*>(src);
            if constexpr (NB > 4) w[1] = *reinterpret_cast<const uint32_t*>(src + 4);
          }
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            const uint32_t code = (w[b >> 2] >> (8 * (b & 3))) & 0xffu;
            sc_f[(set * NB + b) * CHUNK + tok] = in ? e8m0(code) * (set ? pow2(C::lack) : 1.f) : 0.f;
          }
        }
        __syncwarp();
      }
      if (!inside && (t < all_lo || min(t + CHUNK, cur.hi) > all_hi)) {  // tokens that only some rows see
        const int tok = lane % CHUNK, j = t + tok;
        bool found = false;
        if (j >= cur.lo && j < cur.hi && (j < all_lo || j >= all_hi)) {
          constexpr int L = 32 / CHUNK;  // lanes of a token
          if constexpr (C::q) {
            for (int b = lane / CHUNK; b < NB; b += L) {
              float& x = sc_f[(NB + b) * CHUNK + tok];
              if (x != x) x = 0.f, found = true;
            }
          } else {
            for (int i = lane / CHUNK; i < C::rby / 16; i += L) {
              uint4* at = reinterpret_cast<uint4*>(ring_g + (k % S) * C::stage + C::kv_bytes + piece<C::rby>(tok, i));
              uint4 v = *at;
              if (keep_finite(v)) *at = v, found = true;
            }
          }
        }
        if (found) *s_found = 1;
        __syncwarp();
      }
      // of a block: this thread's tokens 2c, 2c+1 of column tile nt
      auto scale2 = [&](int set, int blk, int nt) {
        return *reinterpret_cast<const float2*>(sc_f + (set * NB + blk) * CHUNK + 8 * nt + 2 * c);
      };
      // ------------------------------------------------------------ scores
      float s[MT][TT][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int i = 0; i < 4 * TT; ++i) s[mt][i >> 2][i & 3] = 0.f;
      const int mrow = (lane & 7) + ((lane >> 4) << 3), mpc = (lane >> 3) & 1;  // ldmatrix row and piece of this lane
      if constexpr (!C::q) {
        float s2[MT][TT][4];  // even and odd steps apart: each product waits for the one before last
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int i = 0; i < 4 * TT; ++i) s2[mt][i >> 2][i & 3] = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          uint32_t b[4], a[4];
          ldm4(b, st + piece<C::rby>(mrow, 2 * ks + mpc));
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            query(mt, ks, a);
            mma(ks & 1 ? s2[mt][0] : s[mt][0], a, b[0], b[1]);
            mma(ks & 1 ? s2[mt][1] : s[mt][1], a, b[2], b[3]);
          }
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int i = 0; i < 4 * TT; ++i) s[mt][i >> 2][i & 3] += s2[mt][i >> 2][i & 3];
      } else {
#pragma unroll
        for (int blk = 0; blk < NB; ++blk) {  // a 1x32 block: two k steps
          uint32_t f[2][TT][2];               // [k step][column tile] operands
#pragma unroll
          for (int h = 0; h < TT / 2; ++h) {
            uint32_t b[4];
            if (TYPE == FT_KV_MXFP8) {  // (tokens 0-7, piece 2blk), (0-7, 2blk+1), (8-15, 2blk), (8-15, 2blk+1)
              ldm4(b, st + piece<C::rby>(16 * h + mrow, 2 * blk + mpc));
#pragma unroll
              for (int x = 0; x < 4; ++x) e4m3x4_f16(b[x], f[x & 1][2 * h + (x >> 1)][0], f[x & 1][2 * h + (x >> 1)][1]);
            } else {                    // piece blk of tokens 0-7 and 8-15
              ldm2(b, st + piece<C::rby>(16 * h + (lane & 15), blk));
#pragma unroll
              for (int nt = 0; nt < 2; ++nt) {
                uint32_t e[4];
                e2m1x8_f16(b[nt], e);
                f[0][2 * h + nt][0] = e[0];
                f[0][2 * h + nt][1] = e[1];
                f[1][2 * h + nt][0] = e[2];
                f[1][2 * h + nt][1] = e[3];
              }
            }
          }
          uint32_t a[MT][2][4];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            query(mt, 2 * blk, a[mt][0]);
            query(mt, 2 * blk + 1, a[mt][1]);
          }
#pragma unroll
          for (int nt = 0; nt < TT; ++nt) {
            const float2 sc = scale2(0, blk, nt);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              float acc[4] = {0.f, 0.f, 0.f, 0.f};
              mma_f16(acc, a[mt][0], f[0][nt][0], f[0][nt][1]);
              mma_f16(acc, a[mt][1], f[1][nt][0], f[1][nt][1]);
#pragma unroll
              for (int q = 0; q < 4; ++q) s[mt][nt][q] = fmaf(acc[q], q & 1 ? sc.y : sc.x, s[mt][nt][q]);
            }
          }
        }
      }
      // ------------------------------------------------------------ softmax
      float mx[MT][2];
      bool move = false;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
        for (int i = 0; i < 4 * TT; ++i) s[mt][i >> 2][i & 3] *= scale[mt][(i >> 1) & 1];
        if (!inside) {
#pragma unroll
          for (int i = 0; i < 4 * TT; ++i) {
            const int j = t + 8 * (i >> 2) + 2 * c + (i & 1), h = (i >> 1) & 1;
            if (j < lo[mt][h] || j >= hi[mt][h]) s[mt][i >> 2][i & 3] = -INFINITY;
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          mx[mt][h] = fmaxf(s[mt][0][2 * h], s[mt][0][2 * h + 1]);
#pragma unroll
          for (int nt = 1; nt < TT; ++nt) mx[mt][h] = fmaxf(mx[mt][h], fmaxf(s[mt][nt][2 * h], s[mt][nt][2 * h + 1]));
          move |= mx[mt][h] > m[mt][h] + kSlack;
        }
      }
      if (__any_sync(0xffffffffu, move)) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          float al[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float x = mx[mt][h];
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
            const float mn = x > m[mt][h] + kSlack ? x : m[mt][h];
            al[h] = mn == m[mt][h] ? 1.f : ex2(m[mt][h] - mn);
            l[mt][h] *= al[h];
            m[mt][h] = mn;
          }
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            o[mt][i][0] *= al[0];
            o[mt][i][1] *= al[0];
            o[mt][i][2] *= al[1];
            o[mt][i][3] *= al[1];
          }
        }
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float mu = m[mt][h] == -INFINITY ? 0.f : m[mt][h];
          float sum = 0.f;
#pragma unroll
          for (int nt = 0; nt < TT; ++nt)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const float e = ex2(s[mt][nt][2 * h + q] - mu);
              s[mt][nt][2 * h + q] = e;
              sum += e;
            }
          l[mt][h] += sum;
        }
      // ------------------------------------------------------------ values
      const uint32_t vst = st + C::kv_bytes;
      const int vrow = lane & 15, vpc = lane >> 4;  // (tokens 0-7, piece j), (8-15, j), (0-7, j+1), (8-15, j+1)
      if constexpr (!C::q) {
        uint32_t pa[MT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int i = 0; i < 4; ++i) pa[mt][i] = pack(s[mt][i >> 1][2 * (i & 1)], s[mt][i >> 1][2 * (i & 1) + 1]);
#pragma unroll
        for (int j = 0; j < NT / 2; ++j) {
          uint32_t b[4];
          ldm4t(b, vst + piece<C::rby>(vrow, 2 * j + vpc));
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            mma(o[mt][2 * j], pa[mt], b[0], b[1]);
            mma(o[mt][2 * j + 1], pa[mt], b[2], b[3]);
          }
        }
      } else {
#pragma unroll
        for (int blk = 0; blk < NB; ++blk) {  // 32 columns: four column tiles with one scale for a token
#pragma unroll
          for (int h = 0; h < TT / 2; ++h) {
            uint32_t f[4][2];  // [column tile] operands of 16 tokens
            uint32_t b[4];
            if (TYPE == FT_KV_MXFP8) {  // (tokens 0-7, piece 2blk), (8-15, 2blk), (0-7, 2blk+1), (8-15, 2blk+1)
              ldm4t(b, vst + piece<C::rby>(16 * h + vrow, 2 * blk + vpc));
#pragma unroll
              for (int x = 0; x < 4; ++x) {  // bytes t0d0 t0d1 t1d0 t1d1 -> (t0d0, t1d0), (t0d1, t1d1)
                f[2 * (x >> 1)][x & 1] = e4m3_bits<false>(b[x]);
                f[2 * (x >> 1) + 1][x & 1] = e4m3_bits<true>(b[x]);
              }
            } else {                    // piece blk of tokens 0-7 and 8-15
              ldm2t(b, vst + piece<C::rby>(16 * h + vrow, blk));
#pragma unroll
              for (int x = 0; x < 2; ++x) {  // four codes of token 0 (low half) and of token 1
                f[0][x] = e2m1_bits<0>(b[x]);
                f[1][x] = e2m1_bits<1>(b[x]);
                f[2][x] = e2m1_bits<2>(b[x]);
                f[3][x] = e2m1_bits<3>(b[x]);
              }
            }
            const float2 sc[2] = {scale2(1, blk, 2 * h), scale2(1, blk, 2 * h + 1)};
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              uint32_t pa[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {  // rows g, g + 8 of tokens 0-7, then of 8-15
                const float* e = s[mt][2 * h + (i >> 1)] + 2 * (i & 1);
                pa[i] = pack(e[0] * sc[i >> 1].x, e[1] * sc[i >> 1].y);
              }
#pragma unroll
              for (int i = 0; i < 4; ++i) mma(o[mt][4 * blk + i], pa, f[i][0], f[i][1]);
            }
          }
        }
      }
    }
    cp_wait<0>();
    // ---------------------------------------------------- join the four warps
    __syncthreads();
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float x = l[mt][h];
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        x += __shfl_xor_sync(0xffffffffu, x, 2);
        if (c == 0) {
          join_m[warp * RB + 16 * mt + g + 8 * h] = m[mt][h];
          join_l[warp * RB + 16 * mt + g + 8 * h] = x;
        }
      }
      put_rows<TYPE, D>(join_o + (warp * RB + 16 * mt) * C::opitch, C::opitch, o[mt], pow2(C::taken), g, c);
    }
    __syncthreads();
    constexpr int TPR = kThreads / RB, PC = D / 4 / TPR;  // threads of a row, 16-byte pieces of a thread
    const int r = tid / TPR, sub = tid % TPR;
    float mm = -INFINITY, ll = 0.f, wt[kWarps];
#pragma unroll
    for (int x = 0; x < kWarps; ++x) mm = fmaxf(mm, join_m[x * RB + r]);
#pragma unroll
    for (int x = 0; x < kWarps; ++x) {
      wt[x] = mm == -INFINITY ? 0.f : ex2(join_m[x * RB + r] - mm);
      ll += join_l[x * RB + r] * wt[x];
    }
    float4 acc[PC];
#pragma unroll
    for (int i = 0; i < PC; ++i) {
      acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int x = 0; x < kWarps; ++x) {
        const float4 v = *reinterpret_cast<const float4*>(join_o + (x * RB + r) * C::opitch + 4 * (sub + TPR * i));
        acc[i].x += v.x * wt[x];
        acc[i].y += v.y * wt[x];
        acc[i].z += v.z * wt[x];
        acc[i].w += v.w * wt[x];
      }
    }
    if (*s_found) {  // the row's sums are in registers from here on: its first places hold what was left out of them
      __syncthreads();
      float* extra = join_o + r * C::opitch;
      for (int i = sub; i < D; i += TPR) extra[i] = 0.f;
      __syncwarp();
      if (r < rows && sub == 0) {
        const int pos = cur.len - cur.n + div_group(p, cur.rb * RB + r);
        const int see_hi = p.causal ? min(cur.len, pos + 1) : cur.len, see_lo = p.window > 0 ? max(pos - p.window + 1, 0) : 0;
        not_finite<TYPE, D>(p, cur, all_lo, all_hi, see_lo, see_hi, (cur.t0 + ta) * UT, (cur.t0 + tb) * UT,
                            [&](int d, float v) { extra[d] += v; });
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < PC; ++i) {
        const float4 x = *reinterpret_cast<const float4*>(extra + 4 * (sub + TPR * i));
        acc[i].x += x.x, acc[i].y += x.y, acc[i].z += x.z, acc[i].w += x.w;
      }
    }
    auto put = [&](int row, int piece4, float4 v, float inv) {
      const int rr = cur.rb * RB + row, tok = div_group(p, rr), hd = cur.head * p.group + rr - tok * p.group;
      *reinterpret_cast<uint2*>(p.out + (long long)(cur.q0 + tok) * p.out_stride + (long long)hd * D + 4 * piece4) =
          make_uint2(pack(v.x * inv, v.y * inv), pack(v.z * inv, v.w * inv));
    };
    auto put_lse = [&](int row, float mr, float lr) {
      if (!p.lse) return;
      const int rr = cur.rb * RB + row, tok = div_group(p, rr), hd = cur.head * p.group + rr - tok * p.group;
      p.lse[(long long)(cur.q0 + tok) * p.n_heads + hd] = lr == 0.f ? -INFINITY : (mr + log2f(lr)) * 0.69314718055994530942f;
    };
    int first, last;
    piece_owners(cur, per, first, last);
    if (first == last) {
      if (r < rows) {
        const float inv = ll == 0.f ? 0.f : 1.f / ll;
#pragma unroll
        for (int i = 0; i < PC; ++i) put(r, sub + TPR * i, acc[i], inv);
        if (sub == 0) put_lse(r, mm, ll);
      }
    } else {
      const int me = blockIdx.x;
      float* slot = p.partials + (size_t)(2 * me + (me == first ? 1 : 0)) * C::slot_floats;
      if (r < rows) {
#pragma unroll
        for (int i = 0; i < PC; ++i) __stcg(reinterpret_cast<float4*>(slot + r * D + 4 * (sub + TPR * i)), acc[i]);
        if (sub == 0) {
          __stcg(slot + RB * D + r, mm);
          __stcg(slot + RB * D + RB + r, ll);
        }
      }
      __syncthreads();
      if (tid == 0) {  // the barrier and one thread's fences order the whole block's accesses
        __threadfence();
        const bool is_last = atomicAdd(p.counters + first, 1u) == (uint32_t)(last - first);
        if (is_last) p.counters[first] = 0u;
        __threadfence();
        *s_flag = is_last;
      }
      __syncthreads();
      if (*s_flag) {
        // the last one: join the item's parts in their order
        auto part = [&](int x) { return p.partials + (size_t)(2 * x + (x == first ? 1 : 0)) * C::slot_floats; };
        float* weight = reinterpret_cast<float*>(body);  // [parts][RB]
        const int np = last - first + 1;
        // maxima and sums of all parts, one load each; then weights in place of the maxima
        float* part_l = weight + np * RB;
        for (int i = tid; i < np * RB; i += kThreads) {
          const int x = i / RB, row = i % RB;
          weight[i] = row < rows ? __ldcg(part(first + x) + RB * D + row) : -INFINITY;
          part_l[i] = row < rows ? __ldcg(part(first + x) + RB * (D + 1) + row) : 0.f;
        }
        __syncthreads();
        mm = -INFINITY;
        ll = 0.f;
        for (int x = sub; x < np; x += TPR) mm = fmaxf(mm, weight[x * RB + r]);
#pragma unroll
        for (int d = 1; d < TPR; d <<= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, d));
        for (int x = sub; x < np; x += TPR) {
          const float f = mm == -INFINITY ? 0.f : ex2(weight[x * RB + r] - mm);
          weight[x * RB + r] = f;
          ll += part_l[x * RB + r] * f;
        }
#pragma unroll
        for (int d = 1; d < TPR; d <<= 1) ll += __shfl_xor_sync(0xffffffffu, ll, d);
        if (sub == 0 && r < rows) {
          row_l[r] = ll;
          put_lse(r, mm, ll);
        }
        __syncthreads();
        // four 16-byte pieces of a thread at a time, the parts in their order: many loads in flight
        const int pieces = rows * (D / 4);
        for (int i0 = tid; i0 < pieces; i0 += 4 * kThreads) {
          float4 v[4];
          int row[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[e] = make_float4(0.f, 0.f, 0.f, 0.f);
            row[e] = min(i0 + e * kThreads, pieces - 1) / (D / 4);
          }
#pragma unroll 4
          for (int x = 0; x < np; ++x) {
            const float4* src = reinterpret_cast<const float4*>(part(first + x));
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (i0 + e * kThreads < pieces) {
                const float4 u = __ldcg(src + i0 + e * kThreads);
                const float f = weight[x * RB + row[e]];
                v[e].x += u.x * f;
                v[e].y += u.y * f;
                v[e].z += u.z * f;
                v[e].w += u.w * f;
              }
            }
          }
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (i0 + e * kThreads < pieces)
              put(row[e], (i0 + e * kThreads) % (D / 4), v[e], row_l[row[e]] == 0.f ? 0.f : 1.f / row_l[row[e]]);
        }
      }
    }
    wk.next_item(p);
    if (!wk.more()) break;
    __syncthreads();  // the ring and the join buffers are free again
  }
}

template <int TYPE, int D, int MT>
cudaError_t launch(const AttnParams& p, int n_sm, cudaStream_t s) {
  using C = Cfg<TYPE, D, MT>;
  static std::atomic<uint64_t> ready{0};  // devices whose limit is set
  cudaError_t e = prepare_kernel(attn_rows_kernel<TYPE, D, MT>, C::smem, ready);
  if (e != cudaSuccess) return e;
  const int grid = n_sm * C::ctas;
  // an item's parts are at most all CTAs: their weights must fit where the CTAs join
  if ((size_t)grid * C::RB * 8 > (size_t)C::body || grid > kMaxCtas) return cudaErrorInvalidConfiguration;
  return launch_k(attn_rows_kernel<TYPE, D, MT>, dim3(grid), dim3(kThreads), C::smem, s, true, p);
}

// rows: of one cache head of a sequence, at most.  Up to 16 rows take one row tile (the second
// one's products would be for nothing: 211 / 328 us above), more take two, for which a chunk is
// decoded once; 256-wide heads have registers for one.
template <int TYPE>
cudaError_t launch_type(const AttnParams& p, int D, int rows, int n_sm, cudaStream_t s) {
  if (D == 64) return rows <= 16 ? launch<TYPE, 64, 1>(p, n_sm, s) : launch<TYPE, 64, 2>(p, n_sm, s);
  if (D == 128) return rows <= 16 ? launch<TYPE, 128, 1>(p, n_sm, s) : launch<TYPE, 128, 2>(p, n_sm, s);
  return launch<TYPE, 256, 1>(p, n_sm, s);
}

}  // namespace rows
}  // namespace kv
}  // namespace ft

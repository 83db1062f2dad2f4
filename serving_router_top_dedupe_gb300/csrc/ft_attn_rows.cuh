// Attention of few rows over the paged cache: single tokens, a few drafted tokens, and
// (block by block) any number of rows.
//
// A block is 16 rows of one cache head (the query heads of the group, times new tokens), the
// row count of one mma.sync tile.  Each cached byte is used by 16 rows only, so reading the
// cache bounds this kernel and its layout serves that:
//  - a warp streams 16-token chunks (cp.async into its own ring of stages, several chunks ahead)
//    and never waits for another warp; the four warps of a CTA take the four chunks of a
//    64-token tile, each with its own running maximum, sum and accumulators, and join at the
//    end of the CTA's part of the item;
//  - rows lie in shared memory with their 16-byte pieces permuted by the row, so ldmatrix reads
//    keys and (transposed) values without bank conflicts;
//  - MXFP8 and MXFP4 codes go from ldmatrix to BF16 operands in registers.  The order of the
//    reduction is free, and so is the order of the value columns: keys are taken in the order
//    in which a 32-bit word holds its codes, with the queries arranged to match, and a
//    transposed 16-bit unit holds 2 (4) neighbouring value columns of a token, which become
//    the operands of 2 (4) column tiles.  Decoding is then a shift, two masks and one BF16
//    multiplication by the block's scale per two elements, with no element moved.
// The running maximum moves only when a score passes it by 2^8 or more, so the accumulators
// are rarely rescaled.
#pragma once

#include "ft_kv_internal.cuh"

namespace ft {
namespace kv {
namespace rows {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int RB = 16;             // rows of a block
constexpr int CHUNK = 16;          // tokens of a warp's step
constexpr int UT = CHUNK * kWarps; // tokens of a tile
constexpr int OV = 4;              // counts of an item besides its tiles
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

__device__ __forceinline__ void mma(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
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

// Two E4M3 codes in the high bytes of both halves -> the BF16 numbers they stand for, times 2^-120.
__device__ __forceinline__ uint32_t e4m3_bits(uint32_t t) { return ((t >> 4) & 0x07F007F0u) | (t & 0x80008000u); }
// Nibble I of both halves -> the BF16 numbers their E2M1 codes stand for, times 2^-126.
template <int I>
__device__ __forceinline__ uint32_t e2m1_bits(uint32_t w) {
  const uint32_t mag = I == 0 ? w << 6 : I == 1 ? w << 2 : I == 2 ? w >> 2 : w >> 6;
  const uint32_t sgn = w << (12 - 4 * I);
  return (mag & 0x01C001C0u) | (sgn & 0x80008000u);
}

// Scale codes in the high bytes of both halves -> BF16 multipliers: 2^e times what the codes'
// bits lack.  A code above 134 (MXFP8) or 144 (MXFP4) gives infinity, which makes the zero
// codes of a NaN block NaN.
template <int TYPE>
__device__ __forceinline__ uint32_t multiplier(uint32_t t) {
  constexpr uint32_t lack = TYPE == FT_KV_MXFP8 ? 0x7B807B80u   // 2^120
                                                : 0x76807680u;  // 2^110: 2^-16 is left in
  return mul2(t >> 1, lack);
}

template <int TYPE, int D>
struct Cfg {
  static constexpr int rby = row_bytes(TYPE, D), sby = scale_bytes(TYPE, D);
  static constexpr int kv_bytes = CHUNK * rby;
  static constexpr int stage = 2 * kv_bytes + 2 * CHUNK * sby;
  static constexpr int room = TYPE == FT_KV_BF16 && D == 256 ? 200 * 1024 : 100 * 1024;  // one or two CTAs per SM
  static constexpr int fit = room / (kWarps * stage);
  static constexpr int stages = fit < 8 ? fit : 8;
  static constexpr int ctas = TYPE == FT_KV_BF16 && D == 256 ? 1 : 2;
  static constexpr int ring = kWarps * stages * stage;
  static constexpr int opitch = D + 8;  // floats of a row where the warps join
  static constexpr int join = kWarps * RB * opitch * 4;
  static constexpr int qfrag = (D / 16) * 512;
  static constexpr int head = 1024;  // maxima and sums where the warps join
  static constexpr int body0 = ring > join ? ring : join;
  static constexpr int body = body0 > (int)sizeof(PlanSmem) ? body0 : (int)sizeof(PlanSmem);
  static constexpr int smem = qfrag + head + body;
  static constexpr size_t slot_floats = (size_t)RB * (D + 2);
};

// Column of the values that accumulator half h (columns 2c and 2c+1 of tile nt) stands for.
template <int TYPE>
__device__ __forceinline__ int out_col(int nt, int c, int h) {
  if (TYPE == FT_KV_BF16) return 8 * nt + 2 * c + h;
  if (TYPE == FT_KV_MXFP8) return 16 * (nt >> 1) + 4 * c + 2 * h + (nt & 1);
  return 32 * (nt >> 2) + 8 * c + 4 * h + (nt & 3);
}

// A warp's 16 x D accumulators into rows of shared memory.
template <int TYPE, int D>
__device__ __forceinline__ void put_rows(float* dst, int pitch, const float (*o)[4], int g, int c) {
#pragma unroll
  for (int hr = 0; hr < 2; ++hr) {
    float* row = dst + (g + 8 * hr) * pitch;
    if (TYPE == FT_KV_BF16) {
#pragma unroll
      for (int nt = 0; nt < D / 8; ++nt)
        *reinterpret_cast<float2*>(row + 8 * nt + 2 * c) = make_float2(o[nt][2 * hr], o[nt][2 * hr + 1]);
    } else if (TYPE == FT_KV_MXFP8) {
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
        *reinterpret_cast<float4*>(row + 16 * j + 4 * c) =
            make_float4(o[2 * j][2 * hr], o[2 * j + 1][2 * hr], o[2 * j][2 * hr + 1], o[2 * j + 1][2 * hr + 1]);
    } else {
#pragma unroll
      for (int j = 0; j < D / 32; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          *reinterpret_cast<float4*>(row + 32 * j + 8 * c + 4 * h) =
              make_float4(o[4 * j][2 * hr + h], o[4 * j + 1][2 * hr + h], o[4 * j + 2][2 * hr + h], o[4 * j + 3][2 * hr + h]);
    }
  }
}

template <int TYPE, int D>
__global__ void __launch_bounds__(kThreads, (Cfg<TYPE, D>::ctas)) attn_rows_kernel(const AttnParams p) {
  using C = Cfg<TYPE, D>;
  constexpr int NT = D / 8, KS = D / 16, S = C::stages;
  extern __shared__ __align__(128) uint8_t smem[];
  uint4* qf = reinterpret_cast<uint4*>(smem);                                // [KS][32] query operands
  float* join_m = reinterpret_cast<float*>(smem + C::qfrag);                 // [kWarps][RB]
  float* join_l = join_m + kWarps * RB;                                      // [kWarps][RB]
  int* s_flag = reinterpret_cast<int*>(join_l + kWarps * RB);
  uint8_t* body = smem + C::qfrag + C::head;
  float* join_o = reinterpret_cast<float*>(body);                            // [kWarps][RB][opitch]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
  Walk<RB, UT, OV> wk;
  long long per;
  if (!plan<RB, UT, OV, kThreads>(p, *reinterpret_cast<PlanSmem*>(body), 1, wk, per)) return;
  __syncthreads();

  const uint32_t ring = smem_addr(body) + warp * S * C::stage;
  uint8_t* ring_g = body + warp * S * C::stage;
  const float scale = p.scale_log2 * left_in(TYPE);

  for (;;) {
    // ---------------------------------------------------- this CTA's part of the item
    const Cursor& cur = wk.cur;
    const int ta = (int)(wk.w - cur.start), tb = (int)(wk.end() - cur.start);
    const int rows = min(cur.n * p.group - cur.rb * RB, RB);
    {  // query operands in the order in which the keys' words hold their elements
      for (int i = tid; i < KS * 32; i += kThreads) {
        const int ks = i >> 5, l = i & 31, gg = l >> 2, cc = l & 3;
        uint32_t a[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int r = gg + 8 * (q & 1), kh = q >> 1;
          uint32_t v = 0;
          if (r < rows) {
            const int rr = cur.rb * RB + r, tok = div_group(p, rr), hd = rr - tok * p.group;
            const uint16_t* src = p.q + (long long)(cur.q0 + tok) * p.q_stride + (long long)(cur.head * p.group + hd) * D;
            if (TYPE == FT_KV_BF16) {
              v = __ldg(reinterpret_cast<const uint32_t*>(src + 16 * ks + 2 * cc + 8 * kh));
            } else if (TYPE == FT_KV_MXFP8) {
              v = __ldg(reinterpret_cast<const uint32_t*>(src + 16 * ks + 4 * cc + 2 * kh));
            } else {
              const int d = 32 * (ks >> 1) + 8 * cc + 2 * (ks & 1) + kh;
              v = (uint32_t)__ldg(src + d) | ((uint32_t)__ldg(src + d + 4) << 16);
            }
          }
          a[q] = v;
        }
        qf[i] = make_uint4(a[0], a[1], a[2], a[3]);
      }
    }
    __syncthreads();
    // the cached tokens that this thread's rows g and g + 8 see: [lo, hi)
    int lo[2], hi[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = g + 8 * h;
      lo[h] = hi[h] = 0;
      if (r < rows) {
        const int pos = cur.len - cur.n + div_group(p, cur.rb * RB + r);
        hi[h] = p.causal ? min(cur.len, pos + 1) : cur.len;
        lo[h] = p.window > 0 ? max(pos - p.window + 1, 0) : 0;
      }
    }
    uint32_t qr[KS][4];
    if (D <= 128) {
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) *reinterpret_cast<uint4*>(qr[ks]) = qf[ks * 32 + lane];
    }
    float o[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

    const int n = tb - ta;
    const int32_t* table = p.page_table + (long long)cur.seq * p.table_stride;
    const int tok0 = (cur.t0 + ta) * UT + warp * CHUNK;  // the warp's first chunk
    auto wanted = [&](int k) { return k < n && tok0 + k * UT < cur.hi && tok0 + k * UT + CHUNK > cur.lo; };
    int page_next = wanted(0) ? __ldg(table + (tok0 >> p.page_shift)) : 0;
    auto issue = [&](int k) {
      const int page = page_next, t = tok0 + k * UT;
      if (wanted(k + 1)) page_next = __ldg(table + ((t + UT) >> p.page_shift));
      if (wanted(k)) {
        const bool ok = (unsigned)page < (unsigned)p.n_pages;
        if (!ok && lane == 0) atomicOr(p.error_word, FT_DEVERR_BAD_INDEX);
        const int r0 = max(cur.lo - t, 0), r1 = ok ? min(cur.hi - t, CHUNK) : 0;  // rows to read; the others are zeros
        const long long row = (((long long)(ok ? page : 0) * p.n_kv_heads + cur.head) << p.page_shift) +
                              (t & (p.page_size - 1));
        const uint8_t* ksrc = p.k + row * C::rby;
        const uint8_t* vsrc = p.v + row * C::rby;
        const uint32_t dst = ring + (uint32_t)(k % S) * C::stage;
        constexpr int PR = C::rby / 16;
#pragma unroll
        for (int i = 0; i < CHUNK * PR / 32; ++i) {
          const int u = lane + 32 * i, r = u / PR, pc = u % PR;
          const bool there = r >= r0 && r < r1;
          cp_async16(dst + piece<C::rby>(r, pc), ksrc + u * 16, there);
          cp_async16(dst + C::kv_bytes + piece<C::rby>(r, pc), vsrc + u * 16, there);
        }
        if constexpr (TYPE != FT_KV_BF16) {  // scales of all 16 rows
          constexpr int PS = CHUNK * C::sby / 16;
          if (lane < 2 * PS) {
            const int i = lane % PS;
            const uint8_t* src = (lane < PS ? p.ks : p.vs) + row * C::sby + i * 16;
            cp_async16(dst + 2 * C::kv_bytes + (lane < PS ? 0 : CHUNK * C::sby) + i * 16, src, ok);
          }
        }
      }
      cp_commit();
    };
#pragma unroll 1
    for (int k = 0; k < S - 1; ++k) issue(k);
#pragma unroll 1
    for (int k = 0; k < n; ++k) {
      __syncwarp();  // every lane is done with the stage that is filled next
      issue(k + S - 1);
      cp_wait<S - 1>();
      __syncwarp();
      if (!wanted(k)) continue;
      const int t = tok0 + k * UT;
      const uint32_t st = ring + (uint32_t)(k % S) * C::stage;
      uint8_t* sc_g = ring_g + (k % S) * C::stage + 2 * C::kv_bytes;
      if (TYPE != FT_KV_BF16 && (t < cur.lo || t + CHUNK > cur.hi)) {
        // rows left out: their values are zero codes, and a scale that stands for NaN would show
        if (lane < CHUNK && (t + lane < cur.lo || t + lane >= cur.hi))
          for (int i = 0; i < C::sby; ++i) sc_g[CHUNK * C::sby + lane * C::sby + i] = 0;
        __syncwarp();
      }
      // ------------------------------------------------------------ scores
      float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
      const int mrow = (lane & 7) + ((lane >> 4) << 3), mpc = (lane >> 3) & 1;  // ldmatrix row and piece of this lane
      if (TYPE == FT_KV_BF16) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          uint32_t b[4];
          ldm4(b, st + piece<C::rby>(mrow, 2 * ks + mpc));
          uint32_t a[4];
          if (D <= 128) {
#pragma unroll
            for (int q = 0; q < 4; ++q) a[q] = qr[ks][q];
          } else {
            *reinterpret_cast<uint4*>(a) = qf[ks * 32 + lane];
          }
          mma(s[0], a, b[0], b[1]);
          mma(s[1], a, b[2], b[3]);
        }
      } else {
        // scales of tokens g and g + 8, for every 1x32 block
        const uint8_t* ks_g = sc_g;
        constexpr int NB = D / 32, SUB = TYPE == FT_KV_MXFP8 ? 2 : 4;  // ldmatrix pieces of a block: 2 or 1
#pragma unroll
        for (int pb = 0; pb < D * (TYPE == FT_KV_MXFP8 ? 1 : 0) / 32 + (TYPE == FT_KV_MXFP4 ? D / 64 : 0); ++pb) {
          uint32_t b[4];  // (tokens 0-7, piece 2pb), (0-7, 2pb+1), (8-15, 2pb), (8-15, 2pb+1)
          ldm4(b, st + piece<C::rby>(mrow, 2 * pb + mpc));
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // piece 2pb + h
            const int pcs = 2 * pb + h;
            const int blk = TYPE == FT_KV_MXFP8 ? pcs / 2 : pcs;
            const uint32_t m0 = multiplier<TYPE>((uint32_t)ks_g[g * NB + blk] * 0x01000100u);
            const uint32_t m1 = multiplier<TYPE>((uint32_t)ks_g[(g + 8) * NB + blk] * 0x01000100u);
            constexpr int STEPS = SUB / 2;  // k steps of one piece
#pragma unroll
            for (int sp = 0; sp < STEPS; ++sp) {
              const int ks = pcs * STEPS + sp;
              uint32_t a[4];
              if (D <= 128) {
#pragma unroll
                for (int q = 0; q < 4; ++q) a[q] = qr[ks][q];
              } else {
                *reinterpret_cast<uint4*>(a) = qf[ks * 32 + lane];
              }
#pragma unroll
              for (int nt = 0; nt < 2; ++nt) {
                const uint32_t x = b[2 * nt + h], mm = nt ? m1 : m0;
                uint32_t b0, b1;
                if (TYPE == FT_KV_MXFP8) {
                  b0 = e4m3_bits(__byte_perm(x, 0, 0x1404));  // bytes 0, 1 into the high bytes of the halves
                  b1 = e4m3_bits(__byte_perm(x, 0, 0x3424));
                } else {
                  b0 = sp == 0 ? e2m1_bits<0>(x) : e2m1_bits<2>(x);
                  b1 = sp == 0 ? e2m1_bits<1>(x) : e2m1_bits<3>(x);
                }
                mma(s[nt], a, mul2(b0, mm), mul2(b1, mm));
              }
            }
          }
        }
      }
      // ------------------------------------------------------------ softmax
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int j = t + 8 * nt + 2 * c + (q & 1), h = q >> 1;
          s[nt][q] = j >= lo[h] && j < hi[h] ? s[nt][q] * scale : -INFINITY;
        }
      float mx[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        mx[h] = fmaxf(fmaxf(s[0][2 * h], s[0][2 * h + 1]), fmaxf(s[1][2 * h], s[1][2 * h + 1]));
        mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
        mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
      }
      if (__any_sync(0xffffffffu, mx[0] > m[0] + kSlack || mx[1] > m[1] + kSlack)) {
        float al[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float mn = fmaxf(m[h], mx[h]);
          al[h] = mn == -INFINITY ? 1.f : ex2(m[h] - mn);
          l[h] *= al[h];
          m[h] = mn;
        }
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          o[i][0] *= al[0];
          o[i][1] *= al[0];
          o[i][2] *= al[1];
          o[i][3] *= al[1];
        }
      }
      uint32_t pa[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float mu = m[h] == -INFINITY ? 0.f : m[h];
        const float p0 = ex2(s[0][2 * h] - mu), p1 = ex2(s[0][2 * h + 1] - mu);
        const float p2 = ex2(s[1][2 * h] - mu), p3 = ex2(s[1][2 * h + 1] - mu);
        l[h] += (p0 + p1) + (p2 + p3);
        pa[h] = pack(p0, p1);
        pa[2 + h] = pack(p2, p3);
      }
      // ------------------------------------------------------------ values
      const uint32_t vst = st + C::kv_bytes;
      const int vrow = lane & 15, vpc = lane >> 4;  // (tokens 0-7, piece j), (8-15, j), (0-7, j+1), (8-15, j+1)
      if (TYPE == FT_KV_BF16) {
#pragma unroll
        for (int j = 0; j < NT / 2; ++j) {
          uint32_t b[4];
          ldm4t(b, vst + piece<C::rby>(vrow, 2 * j + vpc));
          mma(o[2 * j], pa, b[0], b[1]);
          mma(o[2 * j + 1], pa, b[2], b[3]);
        }
      } else {
        constexpr int NB = D / 32;
        const uint8_t* vs_g = sc_g + CHUNK * C::sby;
#pragma unroll
        for (int pb = 0; pb < C::rby / 32; ++pb) {
          uint32_t b[4];
          ldm4t(b, vst + piece<C::rby>(vrow, 2 * pb + vpc));
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int pcs = 2 * pb + h;
            const int blk = TYPE == FT_KV_MXFP8 ? pcs / 2 : pcs;
            const uint32_t m0 = multiplier<TYPE>((uint32_t)vs_g[(2 * c) * NB + blk] << 8 |
                                                 (uint32_t)vs_g[(2 * c + 1) * NB + blk] << 24);
            const uint32_t m1 = multiplier<TYPE>((uint32_t)vs_g[(2 * c + 8) * NB + blk] << 8 |
                                                 (uint32_t)vs_g[(2 * c + 9) * NB + blk] << 24);
            const uint32_t x0 = b[2 * h], x1 = b[2 * h + 1];
            if (TYPE == FT_KV_MXFP8) {
              mma(o[2 * pcs], pa, mul2(e4m3_bits(__byte_perm(x0, 0, 0x2404)), m0),
                  mul2(e4m3_bits(__byte_perm(x1, 0, 0x2404)), m1));
              mma(o[2 * pcs + 1], pa, mul2(e4m3_bits(__byte_perm(x0, 0, 0x3414)), m0),
                  mul2(e4m3_bits(__byte_perm(x1, 0, 0x3414)), m1));
            } else {
              mma(o[4 * pcs], pa, mul2(e2m1_bits<0>(x0), m0), mul2(e2m1_bits<0>(x1), m1));
              mma(o[4 * pcs + 1], pa, mul2(e2m1_bits<1>(x0), m0), mul2(e2m1_bits<1>(x1), m1));
              mma(o[4 * pcs + 2], pa, mul2(e2m1_bits<2>(x0), m0), mul2(e2m1_bits<2>(x1), m1));
              mma(o[4 * pcs + 3], pa, mul2(e2m1_bits<3>(x0), m0), mul2(e2m1_bits<3>(x1), m1));
            }
          }
        }
      }
    }
    cp_wait<0>();
    // ---------------------------------------------------- join the four warps
    __syncthreads();
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
      if (c == 0) {
        join_m[warp * RB + g + 8 * h] = m[h];
        join_l[warp * RB + g + 8 * h] = l[h];
      }
    }
    put_rows<TYPE, D>(join_o + warp * RB * C::opitch, C::opitch, o, g, c);
    __syncthreads();
    const int r = tid >> 3, sub = tid & 7;  // 16 rows x 8 threads
    float mm = -INFINITY, ll = 0.f, wt[kWarps];
#pragma unroll
    for (int x = 0; x < kWarps; ++x) mm = fmaxf(mm, join_m[x * RB + r]);
#pragma unroll
    for (int x = 0; x < kWarps; ++x) {
      wt[x] = mm == -INFINITY ? 0.f : ex2(join_m[x * RB + r] - mm);
      ll += join_l[x * RB + r] * wt[x];
    }
    float4 acc[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int x = 0; x < kWarps; ++x) {
        const float4 v = *reinterpret_cast<const float4*>(join_o + (x * RB + r) * C::opitch + 4 * (sub + 8 * i));
        acc[i].x += v.x * wt[x];
        acc[i].y += v.y * wt[x];
        acc[i].z += v.z * wt[x];
        acc[i].w += v.w * wt[x];
      }
    }
    bool write = true;
    int first, last;
    piece_owners(cur, per, first, last);
    if (first != last) {
      const int me = blockIdx.x;
      float* slot = p.partials + (size_t)(2 * me + (me == first ? 1 : 0)) * C::slot_floats;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) __stcg(reinterpret_cast<float4*>(slot + r * D + 4 * (sub + 8 * i)), acc[i]);
      if (sub == 0) {
        __stcg(slot + RB * D + r, mm);
        __stcg(slot + RB * D + RB + r, ll);
      }
      __threadfence();
      __syncthreads();
      if (tid == 0) *s_flag = atomicAdd(p.counters + first, 1u) == (uint32_t)(last - first);
      __syncthreads();
      write = *s_flag != 0;
      if (write) {
        // the last one: join the item's parts in their order
        __threadfence();
        if (tid == 0) p.counters[first] = 0u;
        auto part = [&](int x) { return p.partials + (size_t)(2 * x + (x == first ? 1 : 0)) * C::slot_floats; };
        mm = -INFINITY;
        for (int x = first + sub; x <= last; x += 8) mm = fmaxf(mm, __ldcg(part(x) + RB * D + r));
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, d));
        ll = 0.f;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
        for (int x = first; x <= last; ++x) {
          const float* sl = part(x);
          const float mx = __ldcg(sl + RB * D + r), lx = __ldcg(sl + RB * D + RB + r);
          const float wx = mm == -INFINITY ? 0.f : ex2(mx - mm);
          ll += lx * wx;
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            const float4 v = __ldcg(reinterpret_cast<const float4*>(sl + r * D + 4 * (sub + 8 * i)));
            acc[i].x += v.x * wx;
            acc[i].y += v.y * wx;
            acc[i].z += v.z * wx;
            acc[i].w += v.w * wx;
          }
        }
      }
    }
    if (write && r < rows) {
      const int rr = cur.rb * RB + r, tok = div_group(p, rr), hd = cur.head * p.group + rr - tok * p.group;
      const float inv = ll == 0.f ? 0.f : left_in(TYPE) / ll;
      uint16_t* dst = p.out + (long long)(cur.q0 + tok) * p.out_stride + (long long)hd * D;
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
        *reinterpret_cast<uint2*>(dst + 4 * (sub + 8 * i)) =
            make_uint2(pack(acc[i].x * inv, acc[i].y * inv), pack(acc[i].z * inv, acc[i].w * inv));
      if (p.lse && sub == 0)
        p.lse[(long long)(cur.q0 + tok) * p.n_heads + hd] = ll == 0.f ? -INFINITY : (mm + log2f(ll)) * 0.69314718055994530942f;
    }
    wk.next_item(p);
    if (!wk.more()) break;
    __syncthreads();  // the ring and the join buffers are free again
  }
}

template <int TYPE, int D>
cudaError_t launch(const AttnParams& p, int n_sm, cudaStream_t s) {
  using C = Cfg<TYPE, D>;
  cudaError_t e = cudaFuncSetAttribute(attn_rows_kernel<TYPE, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem);
  if (e != cudaSuccess) return e;
  attn_rows_kernel<TYPE, D><<<n_sm * C::ctas, kThreads, C::smem, s>>>(p);
  return cudaGetLastError();
}

template <int TYPE>
cudaError_t launch_type(const AttnParams& p, int D, int n_sm, cudaStream_t s) {
  return D == 64 ? launch<TYPE, 64>(p, n_sm, s) : D == 128 ? launch<TYPE, 128>(p, n_sm, s) : launch<TYPE, 256>(p, n_sm, s);
}

}  // namespace rows
}  // namespace kv
}  // namespace ft

// Paged key/value cache: writing new tokens' rows (quantised on the way), gathering cached rows,
// and decoding whole pages, plus the argument checks of the cache's entry points.
//
// x -> element * 2^e: e the smallest for which max|x| of a block is within m * 2^e (m the format's
// largest), element = x * 2^-e rounded once, to nearest, by the hardware's conversion; reading back
// is exact.  These kernels move each byte once and compute next to nothing, so memory bounds them
// where there is much to move, and a launch where there is not.  A thread takes eight neighbouring
// elements, 16 bytes of BF16, so that every access of a warp covers whole lines; the four threads
// of a 1x32 block find its maximum with two shuffles, and nothing goes through shared memory.
// Measured: 131072 MXFP8 tokens of 4 x 128 read in 72.5 us (5.6 TB/s); 131072 tokens of 8 x 128 at
// slots in no order: BF16 written in 192 us (5.6 TB/s), MXFP8 187 (4.3) and read in 171 (4.8), MXFP4
// 175 (3.9) and 164 (4.1).  Why the quantised ones stay behind has not been found: most of their
// bytes are the dense BF16 rows, which the BF16 form moves at full rate; one-byte stores and loads of
// scales, and rows of 64 or 128 bytes in no order, are what they have besides.
#include <cstdarg>
#include <cstdio>

#include "ft_dot.cuh"
#include "ft_kv_internal.cuh"

namespace ft {
namespace kv {

ft_status check_cache(const char* name, const ft_kv_cache* c) {
  if (!c) return kv_fail(FT_ERR_INVALID, "%s: cache is NULL", name);
  if (c->kv_type != FT_KV_BF16 && c->kv_type != FT_KV_MXFP8 && c->kv_type != FT_KV_MXFP4)
    return kv_fail(FT_ERR_INVALID, "%s: kv_type = %d", name, c->kv_type);
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
    return kv_fail(FT_ERR_INVALID, "%s: head_dim = %d (64, 128 or 256)", name, c->head_dim);
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
    return kv_fail(FT_ERR_INVALID, "%s: page_size = %d (16, 32, 64 or 128)", name, c->page_size);
  if (c->n_kv_heads < 1 || c->n_kv_heads > 1024 || c->n_pages < 1 ||
      (long long)c->n_pages * c->n_kv_heads * c->page_size >= (1ll << 31))
    return kv_fail(FT_ERR_INVALID, "%s: n_kv_heads = %d, n_pages = %d", name, c->n_kv_heads, c->n_pages);
  const bool q = c->kv_type != FT_KV_BF16;
  if (!c->k || !c->v || (q && (!c->k_scale || !c->v_scale)))
    return kv_fail(FT_ERR_INVALID, "%s: a pointer of the cache is NULL", name);
  const uintptr_t bits = reinterpret_cast<uintptr_t>(c->k) | reinterpret_cast<uintptr_t>(c->v) |
                         (q ? reinterpret_cast<uintptr_t>(c->k_scale) | reinterpret_cast<uintptr_t>(c->v_scale) : 0);
  if (bits & 15) return kv_fail(FT_ERR_INVALID, "%s: the cache must be 16-byte aligned", name);
  return FT_OK;
}

namespace {

constexpr int kThreads = 128;

struct RowsParams {
  uint8_t *k, *v, *ks, *vs;
  const uint16_t *k_in, *v_in;
  uint16_t *k_out, *v_out;
  long long k_stride, v_stride;
  const int32_t* slots;
  int n_tokens, n_kv_heads, page_size, page_shift, n_slots;
  uint32_t* error_word;
};

// Scale exponent of a block whose largest magnitude has the FP32 bits `a`: the smallest e with
// value <= m * 2^e, by comparing significands (m = 1.75 * 2^8 or 1.5 * 2^2).
template <int TYPE>
__device__ __forceinline__ int block_exponent(uint32_t a) {
  constexpr uint32_t top = TYPE == FT_KV_MXFP8 ? 0x600000u : 0x400000u;  // fraction bits of m
  constexpr int em = TYPE == FT_KV_MXFP8 ? 8 : 2, cap = TYPE == FT_KV_MXFP8 ? 7 : 13;
  const int e = (int)(a >> 23) - 127 - em + ((a & 0x7fffffu) > top ? 1 : 0);
  return min(max(e, -100), cap);
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

__device__ __forceinline__ uint32_t e2m1x8(const float* f) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
  return r;
}

// Eight BF16 values of a thread, of the block that its group of four lanes holds -> their codes
// (8 or 4 bytes) and the block's scale code.
template <int TYPE>
__device__ __forceinline__ uint32_t quantise(const uint4 in, uint2& codes) {
  const uint32_t w[4] = {in.x, in.y, in.z, in.w};
  uint32_t top = 0;  // of the magnitudes
#pragma unroll
  for (int i = 0; i < 4; ++i) top = max(top, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  const bool nan = top >= 0x7f80u;  // a NaN or an infinity: the whole block reads back as NaN
  const int e = block_exponent<TYPE>(top << 16);
  const float inv = nan ? 0.f : __uint_as_float((uint32_t)(127 - e) << 23);
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16) * inv;
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u) * inv;
  }
  if (TYPE == FT_KV_MXFP8) {
    codes.x = nan ? 0u : e4m3x4(f[0], f[1], f[2], f[3]);
    codes.y = nan ? 0u : e4m3x4(f[4], f[5], f[6], f[7]);
  } else {
    codes.x = nan ? 0u : e2m1x8(f);
  }
  return nan ? 255u : (uint32_t)(e + 127);
}

// What eight codes and their scale stand for, as BF16.
template <int TYPE>
__device__ __forceinline__ uint4 stands_for(const uint2 codes, uint32_t scale) {
  const float s = e8m0(scale);
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 f;
    if (TYPE == FT_KV_MXFP8) {
      f = dot::e4m3x2_to_float2((uint16_t)((i < 2 ? codes.x : codes.y) >> (16 * (i & 1))));
    } else {
      const uint32_t h2 = dot::e2m1x2_to_f16x2((codes.x >> (8 * i)) & 0xffu);
      f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
    }
    const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * s, f.y * s);  // exact
    o[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// Eight elements' codes from and to memory: 8 or 4 bytes.
template <int TYPE>
__device__ __forceinline__ uint2 load_codes(const uint8_t* p) {
  if (TYPE == FT_KV_MXFP8) return __ldg(reinterpret_cast<const uint2*>(p));
  return make_uint2(__ldg(reinterpret_cast<const uint32_t*>(p)), 0u);
}
template <int TYPE>
__device__ __forceinline__ void store_codes(uint8_t* p, uint2 c) {
  if (TYPE == FT_KV_MXFP8) *reinterpret_cast<uint2*>(p) = c;
  else *reinterpret_cast<uint32_t*>(p) = c.x;
}

// Slot of token t: >= 0, or -1 for a row that is not there.
__device__ __forceinline__ int slot_of(const RowsParams& p, int t) {
  const int s = __ldg(p.slots + t);
  if (s < p.n_slots) return s < 0 ? -1 : s;
  if (p.error_word) atomicOr(p.error_word, FT_DEVERR_BAD_INDEX);
  return -1;
}

// Eight elements of a row of K (blockIdx.y 0) or V (1), EACH times.  Rows have a multiple of 32
// elements, so the four lanes of a block are together always.
template <int TYPE, int D, bool WRITE, int EACH>
__global__ void __launch_bounds__(kThreads) rows_kernel(const RowsParams p) {
  constexpr int NP = D / 8;  // pieces of a row
  pdl_wait();
  pdl_trigger();  // the next launch may take its place; it waits for this one's end before it reads
  const bool is_v = blockIdx.y != 0;
  const long long i0 = (long long)blockIdx.x * (kThreads * EACH) + threadIdx.x;
  const uint32_t per = (uint32_t)p.n_kv_heads * NP;
  uint8_t* const codes = is_v ? p.v : p.k;
  uint8_t* const scales = is_v ? p.vs : p.ks;
  int slot[EACH];
  long long dense[EACH], row[EACH];
  int d[EACH];
#pragma unroll
  for (int e = 0; e < EACH; ++e) {
    const long long i = i0 + e * kThreads;
    const long long t = (i >> 32) == 0 ? (long long)((uint32_t)i / per) : i / per;
    const uint32_t r = (uint32_t)(i - t * per), head = r / NP;
    d[e] = (r % NP) * 8;
    slot[e] = t < p.n_tokens ? slot_of(p, (int)t) : -2;  // -1: padding, -2: no such token
    dense[e] = t * (is_v ? p.v_stride : p.k_stride) + head * D + d[e];
    row[e] = (((long long)(slot[e] >> p.page_shift) * p.n_kv_heads + head) << p.page_shift) + (slot[e] & (p.page_size - 1));
  }
  uint4 x[EACH];
  uint2 c[EACH];
  uint32_t sc[EACH];
#pragma unroll
  for (int e = 0; e < EACH; ++e) {
    x[e] = make_uint4(0, 0, 0, 0);
    c[e] = make_uint2(0, 0);
    sc[e] = 0;
    if (slot[e] < 0) continue;
    if (WRITE) {
      x[e] = __ldg(reinterpret_cast<const uint4*>((is_v ? p.v_in : p.k_in) + dense[e]));
    } else if (TYPE == FT_KV_BF16) {
      x[e] = __ldg(reinterpret_cast<const uint4*>(codes + (row[e] * D + d[e]) * 2));
    } else {
      c[e] = load_codes<TYPE>(codes + row[e] * row_bytes(TYPE, D) + d[e] * row_bytes(TYPE, 8) / 8);
      sc[e] = __ldg(scales + row[e] * (D / 32) + d[e] / 32);
    }
  }
#pragma unroll
  for (int e = 0; e < EACH; ++e) {
    if (WRITE) {
      uint32_t scale = 0;
      if constexpr (TYPE != FT_KV_BF16) scale = quantise<TYPE>(x[e], c[e]);  // every lane takes part
      if (slot[e] < 0) continue;
      if constexpr (TYPE == FT_KV_BF16) {
        *reinterpret_cast<uint4*>(codes + (row[e] * D + d[e]) * 2) = x[e];
      } else {
        store_codes<TYPE>(codes + row[e] * row_bytes(TYPE, D) + d[e] * row_bytes(TYPE, 8) / 8, c[e]);
        if (d[e] % 32 == 0) scales[row[e] * (D / 32) + d[e] / 32] = (uint8_t)scale;
      }
    } else {
      if (slot[e] == -2) continue;
      if constexpr (TYPE != FT_KV_BF16)
        if (slot[e] >= 0) x[e] = stands_for<TYPE>(c[e], sc[e]);
      *reinterpret_cast<uint4*>((is_v ? p.v_out : p.k_out) + dense[e]) = x[e];
    }
  }
}

// Decodes every page that a batch's new tokens may see, once, into a BF16 copy.  One warp takes
// one page of one head, of K (blockIdx.y 0) or V, in pieces of eight elements.  Reading the codes
// and writing two or four times their bytes bounds it: 65536 MXFP8 tokens of 4 x 128 take
// 36-38 us (5.5 TB/s), which 1024 rows of a head earn back (attn.cu).
constexpr int kStageThreads = 256;

template <int TYPE, int D>
__global__ void __launch_bounds__(kStageThreads) stage_kernel(const StageParams p) {
  constexpr int NB = D / 32, NW = kStageThreads / 32, PER = kMaxSeqs / kStageThreads;
  __shared__ int before[kMaxSeqs + 1];  // pages of the sequences before
  __shared__ int part[NW];
  pdl_wait();
  pdl_trigger();
  const AttnParams& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int first[PER], count[PER], sum = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int s = tid * PER + i;
    first[i] = count[i] = 0;
    if (s < a.n_seqs) {
      int q0, n, len;
      bool bad;
      seq_range(a, s, q0, n, len, bad);
      if (n > 0 && len > 0) {
        const int lo = a.window > 0 ? max(len - n - a.window + 1, 0) : 0;
        first[i] = lo >> a.page_shift;
        count[i] = ((len + a.page_size - 1) >> a.page_shift) - first[i];
      }
    }
    sum += count[i];  // a sequence has at most 2^26 pages; a sum beyond 2^31 is caught below
    if (sum < 0) sum = 1 << 30;
  }
  int x = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x = min((long long)x + y, (long long)(1 << 30));
  }
  if (lane == 31) part[warp] = x;
  __syncthreads();
  long long run = x - sum;
  long long total = 0;
  for (int i = 0; i < NW; ++i) {
    if (i < warp) run += part[i];
    total += part[i];
  }
  const bool room = total <= p.cap_pages;
  if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) *p.have = room;
  if (!room) return;
  int at = (int)run;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int s = tid * PER + i;
    if (s < a.n_seqs) {
      before[s] = at;
      if (blockIdx.x == 0 && blockIdx.y == 0) p.base[s] = at - first[i];
      at += count[i];
    }
  }
  __syncthreads();
  const bool is_v = blockIdx.y != 0;
  const uint8_t* codes0 = is_v ? a.v : a.k;
  const uint8_t* scales0 = is_v ? a.vs : a.ks;
  uint16_t* out0 = is_v ? p.v : p.k;
  const long long items = total * a.n_kv_heads;
  for (long long it = (long long)blockIdx.x * NW + warp; it < items; it += (long long)gridDim.x * NW) {
    const int sp = (int)(it / a.n_kv_heads), head = (int)(it - (long long)sp * a.n_kv_heads);
    int s = 0;  // the last sequence that begins at or before this page and has any
    for (int lo = 0, hi = a.n_seqs; lo < hi;) {
      const int mid = (lo + hi) >> 1;
      if (before[mid] <= sp) {
        s = mid;
        lo = mid + 1;
      } else {
        hi = mid;
      }
    }
    int q0, n, len;
    bool bad;
    seq_range(a, s, q0, n, len, bad);
    const int lo = a.window > 0 ? max(len - n - a.window + 1, 0) : 0;
    const int j = sp - before[s] + (lo >> a.page_shift);  // page of the sequence
    const int page = __ldg(a.page_table + (long long)s * a.table_stride + j);
    const bool ok = (unsigned)page < (unsigned)a.n_pages;
    if (!ok && lane == 0) atomicOr(a.error_word, FT_DEVERR_BAD_INDEX);
    const long long from = ((long long)(ok ? page : 0) * a.n_kv_heads + head) << a.page_shift;
    const long long to = ((long long)sp * a.n_kv_heads + head) << a.page_shift;
    const uint8_t* codes = codes0 + from * row_bytes(TYPE, D);
    const uint8_t* scales = scales0 + from * NB;
    uint4* dst = reinterpret_cast<uint4*>(out0 + to * D);
    // pieces of eight elements: a multiple of 128 in a page
    for (int b = lane; b < a.page_size * (D / 8); b += 128) {
      uint2 c[4];
      uint32_t sc[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        c[i] = load_codes<TYPE>(codes + (b + 32 * i) * row_bytes(TYPE, 8));
        sc[i] = __ldg(scales + (b + 32 * i) / 4);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) dst[b + 32 * i] = ok ? stands_for<TYPE>(c[i], sc[i]) : make_uint4(0, 0, 0, 0);
    }
  }
}

template <int TYPE, int D>
cudaError_t launch_rows_t(const RowsParams& p, bool write, cudaStream_t s) {
  const long long pieces = (long long)p.n_tokens * p.n_kv_heads * (D / 8);
  // One piece a thread while that fills the GPU's threads no more than about once; then four, so
  // that enough loads are under way.  One / four pieces, BF16 rows of 8 x 128: 512 tokens 6.8 / 8.8 us,
  // 2048 10.9 / 10.9, 8192 23.2 / 20.1, 131072 274 / 192 (MXFP8 274 / 171 and MXFP4 273 / 164 read).
  const bool much = pieces > 1 << 17;
  const int each = kThreads * (much ? 4 : 1);
  const dim3 grid((unsigned)((pieces + each - 1) / each), 2);
  static std::atomic<uint64_t> ready[4];
  const auto kernel = write ? (much ? rows_kernel<TYPE, D, true, 4> : rows_kernel<TYPE, D, true, 1>)
                            : (much ? rows_kernel<TYPE, D, false, 4> : rows_kernel<TYPE, D, false, 1>);
  const cudaError_t e = prepare_kernel(kernel, 0, ready[2 * write + much]);
  return e == cudaSuccess ? launch_k(kernel, grid, dim3(kThreads), 0, s, true, p) : e;
}

template <int TYPE>
cudaError_t launch_rows_d(int D, const RowsParams& p, bool write, cudaStream_t s) {
  return D == 64 ? launch_rows_t<TYPE, 64>(p, write, s) : D == 128 ? launch_rows_t<TYPE, 128>(p, write, s)
                                                                   : launch_rows_t<TYPE, 256>(p, write, s);
}

template <int TYPE, int D>
cudaError_t launch_stage_t(const StageParams& p, int n_sm, cudaStream_t s) {
  static std::atomic<uint64_t> ready{0};
  const cudaError_t e = prepare_kernel(stage_kernel<TYPE, D>, 0, ready);
  return e == cudaSuccess ? launch_k(stage_kernel<TYPE, D>, dim3(n_sm * 4, 2), dim3(kStageThreads), 0, s, true, p) : e;
}

template <int TYPE>
cudaError_t launch_stage(const StageParams& p, int D, int n_sm, cudaStream_t s) {
  return D == 64 ? launch_stage_t<TYPE, 64>(p, n_sm, s) : D == 128 ? launch_stage_t<TYPE, 128>(p, n_sm, s)
                                                                   : launch_stage_t<TYPE, 256>(p, n_sm, s);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

ft_status rows_call(const char* name, const ft_kv_cache* c, int n_tokens, const void* k, const void* v,
                    long long k_stride, long long v_stride, const int32_t* slots, uint32_t* error_word, bool write,
                    void* stream) {
  if (ft_status st = check_cache(name, c)) return st;
  if (n_tokens < 0) return kv_fail(FT_ERR_INVALID, "%s: n_tokens = %d", name, n_tokens);
  if (n_tokens == 0) return FT_OK;
  if (!k || !v || !slots) return kv_fail(FT_ERR_INVALID, "%s: a pointer is NULL", name);
  if (!aligned16(k) || !aligned16(v) || (reinterpret_cast<uintptr_t>(slots) & 3))
    return kv_fail(FT_ERR_INVALID, "%s: rows must be 16-byte aligned, slots 4-byte aligned", name);
  const long long width = (long long)c->n_kv_heads * c->head_dim;
  const bool bad = k_stride % 8 || v_stride % 8 || k_stride < 0 || v_stride < 0;
  if (bad || (!write && n_tokens > 1 && (k_stride < width || v_stride < width)))
    return kv_fail(FT_ERR_INVALID, "%s: strides %lld, %lld (multiples of 8; rows written must not overlap)", name,
                   k_stride, v_stride);
  RowsParams p{};
  p.k = static_cast<uint8_t*>(c->k);
  p.v = static_cast<uint8_t*>(c->v);
  p.ks = c->k_scale;
  p.vs = c->v_scale;
  p.k_in = p.k_out = const_cast<uint16_t*>(static_cast<const uint16_t*>(k));
  p.v_in = p.v_out = const_cast<uint16_t*>(static_cast<const uint16_t*>(v));
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.slots = slots;
  p.n_tokens = n_tokens;
  p.n_kv_heads = c->n_kv_heads;
  p.page_size = c->page_size;
  p.page_shift = page_shift(c->page_size);
  p.n_slots = c->n_pages * c->page_size;
  p.error_word = error_word;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = c->kv_type == FT_KV_BF16    ? launch_rows_d<FT_KV_BF16>(c->head_dim, p, write, s)
                        : c->kv_type == FT_KV_MXFP8 ? launch_rows_d<FT_KV_MXFP8>(c->head_dim, p, write, s)
                                                    : launch_rows_d<FT_KV_MXFP4>(c->head_dim, p, write, s);
  return e == cudaSuccess ? FT_OK : kv_fail(FT_ERR_CUDA, "%s: %s", name, cudaGetErrorString(e));
}

}  // namespace

cudaError_t stage_pages(const StageParams& p, int type, int D, int n_sm, cudaStream_t s) {
  return type == FT_KV_MXFP8 ? launch_stage<FT_KV_MXFP8>(p, D, n_sm, s) : launch_stage<FT_KV_MXFP4>(p, D, n_sm, s);
}

}  // namespace kv
}  // namespace ft

extern "C" ft_status ft_kv_write(const ft_kv_cache* cache, int n_tokens, const void* k_bf16, const void* v_bf16,
                                 long long k_stride, long long v_stride, const int32_t* slots,
                                 uint32_t* error_word_out, void* stream) {
  return ft::kv::rows_call("ft_kv_write", cache, n_tokens, k_bf16, v_bf16, k_stride, v_stride, slots, error_word_out,
                           true, stream);
}

extern "C" ft_status ft_kv_read(const ft_kv_cache* cache, int n_tokens, const int32_t* slots, void* k_out, void* v_out,
                                long long k_stride, long long v_stride, uint32_t* error_word_out, void* stream) {
  return ft::kv::rows_call("ft_kv_read", cache, n_tokens, k_out, v_out, k_stride, v_stride, slots, error_word_out,
                           false, stream);
}

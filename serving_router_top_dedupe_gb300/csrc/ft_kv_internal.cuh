// Shared pieces of the paged key/value cache: the formats' decoding, the swizzled layout of
// rows in shared memory, and how ft_attn's work is cut and joined again.
#pragma once

#include <cuda_bf16.h>

#include <atomic>
#include <cstdint>

#include "ft_internal.cuh"
#include "ft_kv.h"

namespace ft {

// Sets ft_last_error() of this thread (api.cu) and returns s.
ft_status kv_fail(ft_status s, const char* fmt, ...);

namespace kv {

// Bytes of one cached row's elements, and of its scales.
__host__ __device__ constexpr int row_bytes(int type, int D) {
  return type == FT_KV_BF16 ? 2 * D : type == FT_KV_MXFP8 ? D : D / 2;
}
__host__ __device__ constexpr int scale_bytes(int type, int D) { return type == FT_KV_BF16 ? 0 : D / 32; }

// What decoded MXFP4 elements are still to be multiplied with: their codes become BF16 numbers
// with an exponent 126 too small, and one BF16 multiplier cannot hold 2^126 * 2^e for every
// scale, so 2^-16 is left in (the attention takes it out of its scores and sums in FP32).
__host__ __device__ constexpr float left_in(int type) { return type == FT_KV_MXFP4 ? 65536.f : 1.f; }

// The power of two of an E8M0 code, NaN for code 255.
__device__ __forceinline__ float e8m0(uint32_t code) { return __uint_as_float(code << 23 | (code + 1) >> 8); }

inline int page_shift(int page_size) { return page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : 7; }

// Sets a kernel's shared-memory limit on the current device, once.  All of these kernels ask
// for the same split of an SM's memory, the largest for shared memory: launches overlap, and an
// SM that a small kernel had switched to another split would take fewer CTAs of the next.
template <typename K>
cudaError_t prepare_kernel(K kernel, int bytes, std::atomic<uint64_t>& ready) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (ready.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
  if (e == cudaSuccess && bytes > 48 * 1024) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) ready.fetch_or(bit);
  return e;
}

// Argument checks of a cache description (kv_cache.cu).
ft_status check_cache(const char* name, const ft_kv_cache* c);

// --------------------------------------------------------------------------- attention

struct AttnParams {
  const uint8_t* k;
  const uint8_t* v;
  const uint8_t* ks;
  const uint8_t* vs;
  int n_pages, page_size, page_shift, n_kv_heads;
  int n_heads, group;    // group = n_heads / n_kv_heads
  uint32_t group_magic;  // ceil(2^32 / group), for group > 1
  int n_tokens, n_seqs, table_stride, causal, window;
  float scale_log2;  // scale * log2(e)
  const uint16_t* q;
  long long q_stride;
  const int32_t* q_start;
  const int32_t* kv_len;
  const int32_t* page_table;
  uint16_t* out;
  long long out_stride;
  float* lse;
  uint32_t* counters;  // [kMaxCtas], zero between calls
  float* partials;
  uint32_t* error_word;  // never NULL
  int rows_min, rows_max;  // sequences of fewer or more rows of a head are another launch's
  // A copy of the pages that the batch sees, decoded to BF16 (stage_pages): k, v and n_pages are
  // the copy's, and page j of sequence s is its page staged[s] + j.  NULL: the cache itself.
  const int32_t* staged;
  // Whether the copy had room is known on the device only: a kernel whose `want` differs from
  // *have returns at once.  NULL: no such choice.
  const int32_t* have;
  int want;
};

constexpr int kMaxCtas = 4096;                     // CTAs of one attention launch, at most
constexpr size_t kCounterBytes = kMaxCtas * 4;
constexpr int kMaxSeqs = 1024;                     // sequences of one call
constexpr int kMaxRows = 1 << 25;                  // rows of one cache head in one call

// r / group for r < kMaxRows: with m = ceil(2^32 / g) = (2^32 + e) / g, e < g <= 128,
// r * m / 2^32 = r / g + r * e / (g * 2^32), and the second term is below 1 / g.
__device__ __forceinline__ int div_group(const AttnParams& p, int r) {
  return p.group == 1 ? r : (int)__umulhi((uint32_t)r, p.group_magic);
}

// a / b, in 32 bits where both fit.
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// How the work is cut.  The rows of one cache head of a sequence (row r: new token r / group,
// query head r % group of the head's group) form blocks of RB rows.  An item is a block of
// one head over the tiles (UT cached tokens) that its rows may see; items are ordered by
// sequence, block and head.  An item counts its tiles and OV more for what it costs to begin
// and end it, and every CTA takes the same share of consecutive counts.  So every CTA has
// about the same work whatever the lengths, an item whose tiles fall to several CTAs leaves
// one partial result in each (sums without their normalisation, and the maximum they refer
// to), and the CTA that finishes last joins them in order.  Each CTA has at most two such
// items, one that began before it (partial slot 2 * cta) and one that goes on after it
// (2 * cta + 1).
struct Cursor {
  int seq, rb, head;
  int q0, n, len, nb;  // of the sequence: first row of q, new tokens, cached length, row blocks
  int lo, hi;          // cached tokens that any row of the block may see
  int t0, cost;        // the block's first tile, and its tiles (at least 1)
  long long start;     // position of the item's first tile in the order of all counts
};

__device__ __forceinline__ void seq_range(const AttnParams& p, int s, int& q0, int& n, int& len, bool& bad) {
  const int a = __ldg(p.q_start + s), b = __ldg(p.q_start + s + 1), l = __ldg(p.kv_len + s);
  const int cap = p.table_stride << p.page_shift;
  q0 = min(max(a, 0), p.n_tokens);
  n = max(min(max(b, 0), p.n_tokens) - q0, 0);
  len = min(max(l, 0), cap);
  if (n * p.group < p.rows_min || n * p.group > p.rows_max) n = 0;
  bad = a != q0 || b < a || b > p.n_tokens || l != len;
}

// Row blocks of a sequence with n new tokens.
template <int RB>
__device__ __forceinline__ int row_blocks(int n, int group) {
  return (n * group + RB - 1) / RB;
}

// The cached tokens that rows [rb * RB, ...) of the sequence may see, in tiles of UT tokens.
template <int RB, int UT>
__device__ __forceinline__ void block_range(const AttnParams& p, int rb, int n, int len, int& lo, int& hi, int& t0,
                                            int& cost) {
  const int rows = n * p.group, r0 = rb * RB, r1 = min(rows, r0 + RB) - 1;
  const int p0 = len - n + div_group(p, r0), p1 = len - n + div_group(p, r1);
  hi = p.causal ? min(len, p1 + 1) : len;
  hi = max(hi, 0);
  lo = p.window > 0 ? min(max(p0 - p.window + 1, 0), hi) : 0;
  t0 = lo / UT;
  cost = max((hi + UT - 1) / UT - t0, 1);
}

template <int RB, int UT>
__device__ __forceinline__ void cursor_seq(const AttnParams& p, Cursor& c) {
  bool bad;
  seq_range(p, c.seq, c.q0, c.n, c.len, bad);
  c.nb = row_blocks<RB>(c.n, p.group);
}

// To the next item (the caller knows that there is one).
template <int RB, int UT, int OV>
__device__ __forceinline__ void cursor_next(const AttnParams& p, Cursor& c) {
  c.start += c.cost + OV;
  if (++c.head < p.n_kv_heads) return;
  c.head = 0;
  if (++c.rb == c.nb) {
    c.rb = 0;
    do {
      ++c.seq;
      cursor_seq<RB, UT>(p, c);
    } while (c.nb == 0 && c.seq + 1 < p.n_seqs);
  }
  block_range<RB, UT>(p, c.rb, c.n, c.len, c.lo, c.hi, c.t0, c.cost);
}

// A position in a CTA's share: count w of item cur, up to w1.
template <int RB, int UT, int OV>
struct Walk {
  Cursor cur;
  long long w, w1;
  __device__ __forceinline__ int tile() const { return cur.t0 + (int)(w - cur.start); }
  __device__ __forceinline__ bool more() const { return w < w1; }
  // Where this CTA's part of the item ends.
  __device__ __forceinline__ long long end() const { return min(cur.start + cur.cost, w1); }
  // From the end of the CTA's part of an item to its next item, if there is one.
  __device__ __forceinline__ void next_item(const AttnParams& p) {
    if (cur.start + cur.cost + OV >= w1) {
      w = w1;
    } else {
      cursor_next<RB, UT, OV>(p, cur);
      w = cur.start;
    }
  }
  // To the next tile; true when it is one of another item.
  __device__ __forceinline__ bool next(const AttnParams& p) {
    if (++w < end()) return false;
    next_item(p);
    return true;
  }
};

// The decoded copy of a batch's pages.
struct StageParams {
  AttnParams a;        // over the quantised cache
  uint16_t *k, *v;     // [cap_pages][n_kv_heads][page_size][D] BF16
  int cap_pages;
  int32_t* base;       // [kMaxSeqs] staged[] of AttnParams
  int32_t* have;       // 1: the copy holds every page, 0: no room
};
cudaError_t stage_pages(const StageParams& p, int type, int D, int n_sm, cudaStream_t s);

struct PlanSmem {
  long long sum[kMaxSeqs];  // counts of a sequence's blocks (one head), then their prefix sums
  int many[kMaxSeqs];       // sequences of more blocks than one thread counts
  long long part[33];
  Cursor cur;
  long long total;
  int n_many, found, longest;
};

// Counts of a share: the total over the CTAs, but no less than suits the longest item.  An item
// of c tiles cut into n parts takes c / n tiles' time, and then joining the parts takes n times
// what a part costs, `join` tiles: the sum is least for parts of sqrt(c * join) tiles.  Up to
// three tiles are not worth a second part.
__device__ __forceinline__ long long share(long long total, int ctas, int longest, float join) {
  return max(quotient(total + ctas - 1, ctas), (long long)max((int)ceilf(sqrtf((float)longest * join)), 3));
}

// All NT threads of the block (a multiple of 32) find the share of CTA `cta` of `ctas` and its first item.
// per: counts of a share.  Returns false for a CTA without work.  Counts are summed for one head
// and multiplied by the heads at the end.
template <int RB, int UT, int OV, int NT>
__device__ bool plan(const AttnParams& p, PlanSmem& sm, int cta, int ctas, float join, Walk<RB, UT, OV>& wk,
                     long long& per) {
  constexpr int kFew = 4;    // blocks of a sequence that one thread counts
  constexpr int kStrips = 4; // sequences / 32 that a warp counts by itself
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (p.n_seqs <= 32 * kStrips && (p.table_stride << p.page_shift) / UT < 1 << 20) {  // sums below 2^31
    // Few sequences of few blocks each, as in decode: every warp counts them all, and nothing
    // waits for another warp.
    int sum[kStrips], q0, n, len;
    int longest = 0;
    bool alone = true, any_bad = false;
#pragma unroll
    for (int i = 0; i < kStrips; ++i) {
      sum[i] = 0;
      const int s = 32 * i + lane;
      if (s < p.n_seqs) {
        bool bad;
        seq_range(p, s, q0, n, len, bad);
        any_bad |= bad;
        const int nb = row_blocks<RB>(n, p.group);
        alone &= nb <= kFew;
        for (int b = 0; b < min(nb, kFew); ++b) {
          int lo, hi, t0, cost;
          block_range<RB, UT>(p, b, n, len, lo, hi, t0, cost);
          sum[i] += cost + OV;
          longest = max(longest, cost);
        }
      }
    }
    if (__all_sync(0xffffffffu, alone)) {
      if (any_bad && blockIdx.x == 0 && warp == 0) atomicOr(p.error_word, FT_DEVERR_BAD_INDEX);
      int before[kStrips], run = 0;  // counts of one head before a strip's sequences
#pragma unroll
      for (int i = 0; i < kStrips; ++i) {
        if (32 * i < p.n_seqs) {
          int x = sum[i];
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
          }
          before[i] = run + x - sum[i];
          run += __shfl_sync(0xffffffffu, x, 31);
        } else {
          before[i] = run;
        }
      }
      const long long total = (long long)run * p.n_kv_heads;
      per = share(total, ctas, (int)__reduce_max_sync(0xffffffffu, (uint32_t)longest), join);
      wk.w = per * cta;
      wk.w1 = min(wk.w + per, total);
      if (wk.w >= wk.w1) return false;
      const int at = (int)quotient(wk.w, p.n_kv_heads);
      Cursor& c = wk.cur;
      int base = 0;
#pragma unroll
      for (int i = 0; i < kStrips; ++i) {
        const uint32_t hit = __ballot_sync(0xffffffffu, before[i] <= at && at < before[i] + sum[i]);
        if (hit) {
          const int from = __ffs(hit) - 1;
          c.seq = 32 * i + from;
          base = __shfl_sync(0xffffffffu, before[i], from);
        }
      }
      cursor_seq<RB, UT>(p, c);
      for (c.rb = 0;; ++c.rb) {
        block_range<RB, UT>(p, c.rb, c.n, c.len, c.lo, c.hi, c.t0, c.cost);
        if (at < base + c.cost + OV) break;
        base += c.cost + OV;
      }
      const long long first = (long long)base * p.n_kv_heads;
      c.head = (int)quotient(wk.w - first, c.cost + OV);
      c.start = first + (long long)c.head * (c.cost + OV);
      if (wk.w >= wk.end()) wk.next_item(p);
      return wk.more();
    }
  }
  if (tid == 0) sm.n_many = sm.longest = 0;
  __syncthreads();
  bool any_bad = false;
  int longest = 0;
  for (int s = tid; s < p.n_seqs; s += NT) {
    int q0, n, len;
    bool bad;
    seq_range(p, s, q0, n, len, bad);
    any_bad |= bad;
    const int nb = row_blocks<RB>(n, p.group);
    long long sum = 0;
    if (nb > 0) {
      int lo, hi, t0, cost;
      block_range<RB, UT>(p, nb - 1, n, len, lo, hi, t0, cost);  // no block sees more than the last
      longest = max(longest, cost);
    }
    if (nb <= kFew) {
      for (int b = 0; b < nb; ++b) {
        int lo, hi, t0, cost;
        block_range<RB, UT>(p, b, n, len, lo, hi, t0, cost);
        sum += cost + OV;
      }
    } else {
      sm.many[atomicAdd(&sm.n_many, 1)] = s;
    }
    sm.sum[s] = sum;
  }
  if (any_bad && blockIdx.x == 0) atomicOr(p.error_word, FT_DEVERR_BAD_INDEX);
  longest = (int)__reduce_max_sync(0xffffffffu, (uint32_t)longest);
  if (lane == 0) atomicMax(&sm.longest, longest);
  __syncthreads();
  // sequences of many blocks: several warps count a slice of one each, or a warp several of them
  const int n_many = sm.n_many;
  if (n_many) {
    constexpr int NW = NT / 32;
    const int slices = n_many < NW ? NW / n_many : 1;
    for (int i = warp; i < n_many * slices; i += NW) {
      const int s = sm.many[i / slices], slice = i % slices;
      int q0, n, len;
      bool bad;
      seq_range(p, s, q0, n, len, bad);
      const int nb = row_blocks<RB>(n, p.group);
      long long sum = 0;
      for (int b = lane + 32 * slice; b < nb; b += 32 * slices) {
        int lo, hi, t0, cost;
        block_range<RB, UT>(p, b, n, len, lo, hi, t0, cost);
        sum += cost + OV;
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (lane == 0) atomicAdd(reinterpret_cast<unsigned long long*>(&sm.sum[s]), (unsigned long long)sum);
    }
    __syncthreads();
  }
  // prefix sums over the sequences
  if (warp == 0) {
    long long run = 0;
    for (int s0 = 0; s0 < p.n_seqs; s0 += 32) {
      const int s = s0 + lane;
      const long long v = s < p.n_seqs ? sm.sum[s] : 0;
      long long x = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (s < p.n_seqs) sm.sum[s] = run + x - v;
      run += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) sm.total = run;
  }
  __syncthreads();
  const long long one_head = sm.total, total = one_head * p.n_kv_heads;
  per = share(total, ctas, sm.longest, join);
  const long long w0 = per * cta;
  wk.w = w0;
  wk.w1 = min(w0 + per, total);
  if (w0 >= wk.w1) return false;
  // the sequence whose counts hold w0, taken in counts of one head (so inside the same block)
  const long long at = quotient(w0, p.n_kv_heads);
  for (int s = tid; s < p.n_seqs; s += NT) {
    const long long a = sm.sum[s], b = s + 1 < p.n_seqs ? sm.sum[s + 1] : one_head;
    if (a <= at && at < b) sm.found = s;
  }
  __syncthreads();
  Cursor c{};
  c.seq = sm.found;
  cursor_seq<RB, UT>(p, c);
  // its blocks: each thread counts a run of them, and the one that meets w0 walks its run
  const int each = (c.nb + NT - 1) / NT, b0 = min(tid * each, c.nb), b1 = min(b0 + each, c.nb);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) {
    block_range<RB, UT>(p, b, c.n, c.len, c.lo, c.hi, c.t0, c.cost);
    mine += c.cost + OV;
  }
  long long x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sm.part[warp] = x;
  __syncthreads();
  long long run = sm.sum[c.seq] + x - mine;
  for (int i = 0; i < warp; ++i) run += sm.part[i];
  if (run <= at && at < run + mine) {
    for (c.rb = b0;; ++c.rb) {
      block_range<RB, UT>(p, c.rb, c.n, c.len, c.lo, c.hi, c.t0, c.cost);
      if (at < run + c.cost + OV) break;
      run += c.cost + OV;
    }
    const long long first = run * p.n_kv_heads;  // where the block's first head starts
    c.head = (int)quotient(w0 - first, c.cost + OV);
    c.start = first + (long long)c.head * (c.cost + OV);
    sm.cur = c;
  }
  __syncthreads();
  wk.cur = sm.cur;
  if (wk.w >= wk.end()) wk.next_item(p);  // the share begins in the counts behind an item's tiles
  return wk.more();
}

// Pieces of the item at `cur`: the CTAs that hold its first and its last tile.
__device__ __forceinline__ void piece_owners(const Cursor& cur, long long per, int& first, int& last) {
  first = (int)quotient(cur.start, per);
  last = (int)quotient(cur.start + cur.cost - 1, per);
}

}  // namespace kv
}  // namespace ft

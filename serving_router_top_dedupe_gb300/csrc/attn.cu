// ft_attn: argument checks, workspace and the choice of the kernel.
#include <algorithm>
#include <climits>
#include <cmath>

#include "ft_kv_internal.cuh"

namespace ft {
namespace kv {

cudaError_t attn_rows_bf16(const AttnParams& p, int D, int rows, int n_sm, cudaStream_t s);
cudaError_t attn_chunk_bf16(const AttnParams& p, int D, int rows, int n_sm, cudaStream_t s);
cudaError_t attn_rows_mxfp8(const AttnParams& p, int D, int rows, int n_sm, cudaStream_t s);
cudaError_t attn_chunk_mxfp8(const AttnParams& p, int D, int rows, int n_sm, cudaStream_t s);
cudaError_t attn_rows_mxfp4(const AttnParams& p, int D, int rows, int n_sm, cudaStream_t s);
cudaError_t attn_chunk_mxfp4(const AttnParams& p, int D, int rows, int n_sm, cudaStream_t s);

namespace {

constexpr int kMaxDevices = 64;

// SMs of the current device (0: the query failed), looked up once per device.
int sm_count() {
  static int cache[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
  int n = __atomic_load_n(&cache[dev], __ATOMIC_RELAXED);
  if (!n) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    __atomic_store_n(&cache[dev], n, __ATOMIC_RELAXED);
  }
  return n;
}

// Counters, a stand-in for the caller's error word, and two partial results for each CTA: of
// head_dim + 2 floats for 16 rows (few rows: up to three CTAs per SM) or 32 (two), or for 256 or
// 128 rows (chunks: one).
static_assert(kCounterBytes == FT_ATTN_CLEAR_BYTES, "what the caller clears");
size_t partial_bytes(int n_sm, int D) { return (size_t)n_sm * 2 * (D == 256 ? 128 : 256) * (D + 2) * 4; }

// What a call cannot do without; then, for the decoded copy of a quantised cache's pages: where
// each sequence's pages begin in it, whether it had room, and the copy.
size_t workspace_least(int n_sm, int D) { return kCounterBytes + 256 + partial_bytes(n_sm, D); }
constexpr size_t kStageHead = kMaxSeqs * 4 + 256;
constexpr size_t kStageBytes = FT_ATTN_COPY_BYTES - kStageHead;
static_assert(kStageHead == 4352, "the copy's part of the workspace");

// From this many rows of a head on, a quantised cache's pages are decoded once into a BF16 copy;
// below it each block of 256 rows decodes what it reads.  Both sides measured (us, decoded where
// it is read / copied; 16 query heads over 4 cache heads of 128, 16 sequences of 4096 tokens):
// MXFP8 512 rows 119 / 138, 1024 199 / 189, 2048 343 / 296; MXFP4 109 / 128, 187 / 181, 326 / 285.
constexpr int kStageRows = 1024;

// Tokens of the cache that a sequence's new ones may see, at most (its length is not known here).
long long may_see(const AttnParams& p, long long rows) {
  const long long cap = (long long)p.table_stride * p.page_size;
  return p.window > 0 ? std::min(cap, p.window + rows / p.group) : cap;
}

// Whether the few-row kernel takes a batch (rows: of one cache head of a sequence, at most).  It
// re-reads the cache for every 16 or 32 rows; the chunk kernel does so for every 128 or 256, but takes
// 12 us longer to start and to end, and decodes a quantised cache's tokens at about half the
// few-row kernel's rate.  Measured with 16 sequences of 8192 tokens and 4 cache heads (us, few-row
// kernel / chunk kernel, one launch each):
//              16 rows      32 rows      48 rows     64 rows    128 rows
//   BF16  64   44 / 60      62 / 62      79 / 60     97 / 62    158 / 61
//   BF16 128   67 / 83     109 / 83     146 / 83    181 / 83    319 / 85
//   BF16 256  101 / 115    180 / 116    250 / 115   329 / 117   616 / 118
//   MXFP8 64   33 / 81      46 / 81      62 / 81     74 / 81    134 / 81
//   MXFP8 128  48 / 109     70 / 108     97 / 109   118 / 108   216 / 109
//   MXFP8 256  81 / 190    128 / 193    177 / 191   226 / 191   421 / 191
//   MXFP4 64   31 / 74      44 / 74      58 / 74     72 / 74    130 / 74
//   MXFP4 128  42 / 95      64 / 95      89 / 95    109 / 95    201 / 95
//   MXFP4 256  72 / 165    120 / 165    165 / 163   212 / 164   398 / 165
// which is the first rule.  The second: where there is little to do in all, the shorter start
// decides whatever the rows (one sequence of 4096 tokens, 64 rows: BF16 19 / 33, MXFP8 23 / 51,
// MXFP4 23 / 48 with heads of 128; BF16 27 / 42 with heads of 256).  The lengths are not known
// here; what the tables and the window allow bounds them.
bool takes_few(const AttnParams& p, int type, int D, long long rows) {
  if (rows <= (type == FT_KV_BF16 ? 16 : D == 64 ? 64 : 48)) return true;
  const long long tokens = (long long)p.n_tokens * p.group;
  const long long blocks = std::min(p.n_seqs * ((rows + 31) / 32), tokens / 32 + p.n_seqs);  // of 32 rows
  const double work = (double)blocks * p.n_kv_heads * may_see(p, rows) * D;  // the two meet at 0.13 to 0.5 of 2^27
  return work <= (type == FT_KV_BF16 ? 1 << 24 : 1 << 25);
}

// Whether a batch's sequences of few rows (single tokens, mostly) get a launch of the few-row
// kernel of their own, before the one for the others: sequences of different numbers of new tokens,
// and much to read.  Measured (us, one launch / two), one chunk besides single tokens that each see
// 8192 tokens: 15 and a chunk of 64, MXFP8, cache heads x head_dim 8 x 64 146 / 103, 4 x 128 120 / 122,
// 2 x 256 132 / 146; 31 and a chunk of 512 over 2048: MXFP8 342 / 125, 302 / 137, 271 / 152, MXFP4
// 302 / 124, 273 / 125, 245 / 141; 63 and a chunk of 1024 over 8192: MXFP8 600 / 235, 487 / 280,
// 596 / 284, BF16 423 / 282, 339 / 320, 263 / 306: over a BF16 cache of 256-wide heads both kernels
// read a block's tokens at about the same rate, and one launch does.  With little to read the second
// launch costs more than it saves (7 that see 1000 and a chunk of 1024: 57 / 86).
constexpr int kFewRows = 16;
bool splits(const AttnParams& p, int type, int D, long long rows, int max_new) {
  if (type == FT_KV_BF16 && D == 256) return false;
  return p.n_tokens < (long long)p.n_seqs * max_new &&
         (double)p.n_seqs * p.n_kv_heads * may_see(p, rows) * D >= (type == FT_KV_BF16 ? 1 << 28 : 1 << 26);
}

ft_status check_heads(const char* name, int n_heads, int n_kv_heads, int head_dim) {
  if (n_kv_heads < 1 || n_kv_heads > 1024 || n_heads < 1 || n_heads % n_kv_heads || n_heads / n_kv_heads > 128)
    return kv_fail(FT_ERR_INVALID, "%s: n_heads = %d over %d cache heads", name, n_heads, n_kv_heads);
  if (head_dim != 64 && head_dim != 128 && head_dim != 256)
    return kv_fail(FT_ERR_INVALID, "%s: head_dim = %d (64, 128 or 256)", name, head_dim);
  return FT_OK;
}

}  // namespace
}  // namespace kv
}  // namespace ft

using namespace ft;

extern "C" ft_status ft_attn_workspace(int n_heads, int n_kv_heads, int head_dim, size_t* bytes_out) {
  if (!bytes_out) return kv_fail(FT_ERR_INVALID, "ft_attn_workspace: bytes_out is NULL");
  if (ft_status st = kv::check_heads("ft_attn_workspace", n_heads, n_kv_heads, head_dim)) return st;
  const int n_sm = kv::sm_count();
  if (!n_sm) return kv_fail(FT_ERR_CUDA, "ft_attn_workspace: no device");
  *bytes_out = kv::workspace_least(n_sm, head_dim) + kv::kStageHead + kv::kStageBytes;
  return FT_OK;
}

extern "C" ft_status ft_attn(const ft_kv_cache* c, const ft_attn_args* a, void* stream) {
  const char* name = "ft_attn";
  if (ft_status st = kv::check_cache(name, c)) return st;
  if (!a) return kv_fail(FT_ERR_INVALID, "%s: args is NULL", name);
  if (ft_status st = kv::check_heads(name, a->n_heads, c->n_kv_heads, c->head_dim)) return st;
  if (a->n_tokens < 0 || a->n_seqs < 0 || a->n_seqs > kv::kMaxSeqs || a->max_new < 1 ||
      (long long)a->n_tokens * a->n_heads >= (1ll << 31) ||
      (long long)a->n_tokens * (a->n_heads / c->n_kv_heads) >= kv::kMaxRows)
    return kv_fail(FT_ERR_INVALID, "%s: n_tokens = %d, n_seqs = %d, max_new = %d", name, a->n_tokens, a->n_seqs,
                   a->max_new);
  if (a->table_stride < 1 || (long long)a->table_stride * c->page_size > (1ll << 30) || a->window < 0 ||
      (a->causal != 0 && a->causal != 1) || !std::isfinite(a->scale))
    return kv_fail(FT_ERR_INVALID, "%s: table_stride = %d, window = %d, causal = %d, scale = %g", name,
                   a->table_stride, a->window, a->causal, (double)a->scale);
  if (a->n_tokens == 0 || a->n_seqs == 0) return FT_OK;
  if (!a->q || !a->q_start || !a->kv_len || !a->page_table || !a->out || !a->workspace)
    return kv_fail(FT_ERR_INVALID, "%s: a pointer is NULL", name);
  const uintptr_t b16 = reinterpret_cast<uintptr_t>(a->q) | reinterpret_cast<uintptr_t>(a->out);
  const uintptr_t b4 = reinterpret_cast<uintptr_t>(a->q_start) | reinterpret_cast<uintptr_t>(a->kv_len) |
                       reinterpret_cast<uintptr_t>(a->page_table) | reinterpret_cast<uintptr_t>(a->lse) |
                       reinterpret_cast<uintptr_t>(a->error_word_out);
  if ((b16 & 15) || (b4 & 3) || (reinterpret_cast<uintptr_t>(a->workspace) & 255))
    return kv_fail(FT_ERR_INVALID, "%s: q and out must be 16-byte, the workspace 256-byte aligned", name);
  const long long width = (long long)a->n_heads * c->head_dim;
  if (a->q_stride % 8 || a->out_stride % 8 || a->q_stride < 0 || (a->n_tokens > 1 && a->out_stride < width))
    return kv_fail(FT_ERR_INVALID, "%s: strides %lld, %lld (multiples of 8; rows of out must not overlap)", name,
                   a->q_stride, a->out_stride);
  const int n_sm = kv::sm_count();
  if (!n_sm) return kv_fail(FT_ERR_CUDA, "%s: no device", name);
  const size_t least = kv::workspace_least(n_sm, c->head_dim);
  if (a->workspace_bytes < least)
    return kv_fail(FT_ERR_CAPACITY, "%s: the workspace has %zu bytes, %zu are needed", name, a->workspace_bytes, least);

  kv::AttnParams p{};
  p.k = static_cast<const uint8_t*>(c->k);
  p.v = static_cast<const uint8_t*>(c->v);
  p.ks = c->k_scale;
  p.vs = c->v_scale;
  p.n_pages = c->n_pages;
  p.page_size = c->page_size;
  p.page_shift = kv::page_shift(c->page_size);
  p.n_kv_heads = c->n_kv_heads;
  p.n_heads = a->n_heads;
  p.group = a->n_heads / c->n_kv_heads;
  p.group_magic = p.group == 1 ? 0 : (uint32_t)((1ull << 32) / p.group + ((1ull << 32) % p.group != 0));
  p.n_tokens = a->n_tokens;
  p.n_seqs = a->n_seqs;
  p.table_stride = a->table_stride;
  p.causal = a->causal;
  p.window = a->window < (1 << 30) ? a->window : 1 << 30;
  p.scale_log2 = (float)((double)a->scale * 1.4426950408889634074);
  p.q = static_cast<const uint16_t*>(a->q);
  p.q_stride = a->q_stride;
  p.q_start = a->q_start;
  p.kv_len = a->kv_len;
  p.page_table = a->page_table;
  p.out = static_cast<uint16_t*>(a->out);
  p.out_stride = a->out_stride;
  p.lse = a->lse;
  p.counters = static_cast<uint32_t*>(a->workspace);
  p.partials = reinterpret_cast<float*>(static_cast<uint8_t*>(a->workspace) + kv::kCounterBytes + 256);
  p.rows_min = 0;
  p.rows_max = INT_MAX;
  p.error_word = a->error_word_out ? a->error_word_out : p.counters + kv::kMaxCtas;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  using Kernel = cudaError_t (*)(const kv::AttnParams&, int, int, int, cudaStream_t);
  static const Kernel kernels[2][3] = {{kv::attn_rows_bf16, kv::attn_rows_mxfp8, kv::attn_rows_mxfp4},
                                       {kv::attn_chunk_bf16, kv::attn_chunk_mxfp8, kv::attn_chunk_mxfp4}};
  const long long rows = (long long)std::min(a->max_new, a->n_tokens) * p.group;  // of one cache head of a sequence, at most
  cudaError_t e = cudaSuccess;
  if (kv::takes_few(p, c->kv_type, c->head_dim, rows)) {
    e = kernels[0][c->kv_type](p, c->head_dim, (int)(rows < 33 ? rows : 33), n_sm, s);
    return e == cudaSuccess ? FT_OK : kv_fail(FT_ERR_CUDA, "%s: %s", name, cudaGetErrorString(e));
  }
  if (kv::splits(p, c->kv_type, c->head_dim, rows, a->max_new)) {
    p.rows_max = kv::kFewRows;
    e = kernels[0][c->kv_type](p, c->head_dim, kv::kFewRows, n_sm, s);
    if (e != cudaSuccess) return kv_fail(FT_ERR_CUDA, "%s: %s", name, cudaGetErrorString(e));
    p.rows_min = kv::kFewRows + 1;
    p.rows_max = INT_MAX;
  }
  if (c->kv_type != FT_KV_BF16 && rows >= kv::kStageRows && a->workspace_bytes >= least + kv::kStageHead + kv::kStageBytes) {
    // many rows over a quantised cache: its pages are decoded once
    uint8_t* at = static_cast<uint8_t*>(a->workspace) + least;
    const size_t page = (size_t)c->n_kv_heads * c->page_size * c->head_dim * 2;
    kv::StageParams st{};
    st.a = p;
    st.cap_pages = (int)(kv::kStageBytes / 2 / page < (1u << 24) ? kv::kStageBytes / 2 / page : 1u << 24);
    st.base = reinterpret_cast<int32_t*>(at);
    st.have = st.base + kv::kMaxSeqs;
    st.k = reinterpret_cast<uint16_t*>(at + kv::kStageHead);
    st.v = st.k + (size_t)st.cap_pages * page / 2;
    e = kv::stage_pages(st, c->kv_type, c->head_dim, n_sm, s);
    // how many pages the batch has is known on the device; where the tables could hold more than
    // there is room for, both kernels are launched and one of them has nothing to do
    const bool fits = (long long)a->n_seqs * a->table_stride <= st.cap_pages;
    if (e == cudaSuccess && !fits) {
      kv::AttnParams direct = p;
      direct.have = st.have;
      direct.want = 0;
      e = kernels[1][c->kv_type](direct, c->head_dim, 33, n_sm, s);
    }
    if (e == cudaSuccess) {
      p.k = reinterpret_cast<const uint8_t*>(st.k);
      p.v = reinterpret_cast<const uint8_t*>(st.v);
      p.ks = p.vs = nullptr;
      p.n_pages = st.cap_pages;
      p.staged = st.base;
      p.have = fits ? nullptr : st.have;
      p.want = 1;
      e = kernels[1][FT_KV_BF16](p, c->head_dim, 33, n_sm, s);
    }
  } else {
    e = kernels[1][c->kv_type](p, c->head_dim, 33, n_sm, s);
  }
  return e == cudaSuccess ? FT_OK : kv_fail(FT_ERR_CUDA, "%s: %s", name, cudaGetErrorString(e));
}

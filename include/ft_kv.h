/*
 * ft_kv.h -- paged key/value cache and the attention that reads it, on one GB300 (sm_103a).
 *
 * The attention half of a decoder layer whose MoE half ft_moe.h serves.  The calls here keep
 * no state: the caller owns the cache pages, the tables and the workspace, names the stream,
 * and may capture every call into a CUDA graph.  Lengths and tables are read on the device
 * when the work runs, so a captured call follows them as they change.
 *
 * Conventions as in ft_moe.h: a call returns FT_OK or an ft_status (ft_last_error() has the
 * message), argument errors change nothing, work is enqueued on the given stream of the
 * current device (NULL: the legacy default stream) without a host synchronisation, and BF16
 * values are raw 16-bit patterns.  A layer's two halves follow one another on one stream: name it
 * here and in ft_moe_config, where NULL means a stream of the library's own.
 */
#ifndef FT_KV_H
#define FT_KV_H

#include "ft_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* How a cached row (head_dim elements of one token and head) is held.
 *   FT_KV_BF16   BF16 elements as they come.
 *   FT_KV_MXFP8  E4M3 elements, one E8M0 scale (2^(code-127)) per 1x32 block of the row.
 *   FT_KV_MXFP4  E2M1 elements packed two per byte (element 2j in the low nibble), one E8M0
 *                scale per 1x32 block: the layout of FT_W_MXFP4.
 * A block x[0..31] is quantised with the smallest scale 2^e for which max|x| <= m * 2^e
 * (MXFP8: m = 448, MXFP4: m = 6), -100 <= e <= 7 (MXFP8) or 13 (MXFP4); an element is
 * x * 2^-e rounded to nearest, ties to even, limited to +-m (magnitudes beyond 57344 or
 * 49152 saturate).  A block that holds a NaN or an infinity gets scale code 255 and reads
 * back as NaN.  What an element stands for (element * 2^e) is always a BF16 number, so
 * reading back and attention work on exactly the stored values.  Pages filled by other means
 * than ft_kv_write keep to these scales, and hold no NaN element codes (E4M3 0x7f, 0xff). */
typedef enum { FT_KV_BF16 = 0, FT_KV_MXFP8 = 1, FT_KV_MXFP4 = 2 } ft_kv_type;

/* Device error bit of the calls below: a slot, page id, offset or length in a device array
 * lies outside its range (each call says what it does then). */
#define FT_DEVERR_BAD_INDEX 0x10u

/* The cache of one layer.  Pages hold page_size tokens and are caller-owned device memory,
 * row-major; token `off` of page `p` is slot p * page_size + off.
 *   k, v             [n_pages][n_kv_heads][page_size][head_dim] elements, 16-byte aligned
 *   k_scale, v_scale [n_pages][n_kv_heads][page_size][head_dim/32] scale codes, 16-byte
 *                    aligned (MXFP8, MXFP4; NULL for BF16) */
typedef struct {
  int kv_type;      /* ft_kv_type */
  int n_kv_heads;   /* 1 .. 1024 */
  int head_dim;     /* 64, 128 or 256 */
  int page_size;    /* 16, 32, 64 or 128 tokens */
  int n_pages;      /* n_pages * n_kv_heads * page_size < 2^31 */
  void* k;
  void* v;
  uint8_t* k_scale;
  uint8_t* v_scale;
} ft_kv_cache;

/* Write n_tokens rows of keys and values into the cache, quantised as its type says.
 *   k_bf16, v_bf16  dev; token t's rows [n_kv_heads][head_dim] start t * k_stride (v_stride)
 *                   elements after the pointer (parts of a wider projection's rows are
 *                   fine); pointers 16-byte aligned, strides multiples of 8
 *   slots           dev [n_tokens]; a negative slot skips its token (padding).  The others of
 *                   a call are distinct: a row that two tokens name is undefined (parts of
 *                   both, and codes of one with scales of the other), other rows are as they
 *                   should be.
 *   error_word_out  optional dev uint32, into which FT_DEVERR_BAD_INDEX is OR-ed for a slot
 *                   beyond the cache (its token is skipped)
 * n_tokens = 0 does nothing.  Errors: FT_ERR_INVALID, FT_ERR_CUDA. */
ft_status ft_kv_write(const ft_kv_cache* cache, int n_tokens, const void* k_bf16, const void* v_bf16,
                      long long k_stride, long long v_stride, const int32_t* slots, uint32_t* error_word_out,
                      void* stream);

/* Gather cached rows into dense BF16 rows: the exact values that the cache holds.
 *   k_out, v_out  dev, laid out as k_bf16 and v_bf16 above; rows of negative slots and of
 *                 slots beyond the cache (FT_DEVERR_BAD_INDEX) are set to zero
 * Other arguments and errors as ft_kv_write. */
ft_status ft_kv_read(const ft_kv_cache* cache, int n_tokens, const int32_t* slots, void* k_out, void* v_out,
                     long long k_stride, long long v_stride, uint32_t* error_word_out, void* stream);

/* Arguments of ft_attn: a batch of sequences, each with some new tokens (whose keys and
 * values are already in the cache) and a length that counts them.  Sequence s has the new
 * tokens q_start[s] .. q_start[s+1]-1; its cached token j is in page
 * page_table[s * table_stride + j / page_size].  New token i of n, in a sequence of length L,
 * stands at position p = L - n + i and attends to the cached tokens j with
 *   0 <= j < L,  j <= p (when causal),  j > p - window (when window > 0).
 * Query head h reads the cache's head h / (n_heads / n_kv_heads).
 *   out  = sum_j exp(s_j - lse) v_j,  s_j = scale * q . k_j,  lse = log sum_j exp(s_j)
 * A token that attends to nothing (p < 0, or a length of 0) gets out = 0 and lse = -inf.
 * What lies in masked places (pages beyond a length, tokens outside the window, later
 * tokens) does not matter, NaN and infinities included. */
typedef struct {
  int n_heads;              /* query heads, a multiple of n_kv_heads; at most 128 per cache head */
  int n_tokens;             /* new tokens of the batch: rows of q, out and lse; n_tokens * n_heads below 2^31,
                               and n_tokens * (n_heads / n_kv_heads) below 2^25 */
  int n_seqs;               /* sequences, at most 1024 */
  int max_new;              /* new tokens of one sequence, at most: chooses the kernel, and any value >= 1
                               gives the same results within rounding */
  int table_stride;         /* pages of one row of page_table; times page_size at most 2^30 */
  int causal;               /* 1: a token sees no later one; 0: every token sees the whole length */
  int window;               /* 0, or how many tokens up to its own position a token sees */
  float scale;              /* of the scores; finite */
  const void* q;            /* dev BF16, token t's [n_heads][head_dim] at t * q_stride elements */
  long long q_stride;       /* multiple of 8 */
  const int32_t* q_start;   /* dev [n_seqs + 1], ascending */
  const int32_t* kv_len;    /* dev [n_seqs] */
  const int32_t* page_table;/* dev [n_seqs][table_stride] */
  void* out;                /* dev BF16, token t's [n_heads][head_dim] at t * out_stride elements */
  long long out_stride;     /* multiple of 8 */
  float* lse;               /* dev [n_tokens][n_heads] (natural logarithm), or NULL */
  void* workspace;          /* dev, ft_attn_workspace() bytes, 256-byte aligned */
  size_t workspace_bytes;
  uint32_t* error_word_out; /* optional dev uint32, into which FT_DEVERR_* bits are OR-ed */
} ft_attn_args;

/* Bytes of workspace that ft_attn uses on the current device, for any batch.  The caller sets
 * the first FT_ATTN_CLEAR_BYTES of it to zero once, before its first use (what the rest holds does
 * not matter); every call leaves it ready for the next (after FT_DEVERR_TIMEOUT, a wait inside a
 * kernel that ran out, they are to be set to zero again, and the call's outputs are not to be
 * used).  Calls that may overlap on the GPU need workspaces of their own.  The last
 * FT_ATTN_COPY_BYTES hold decoded pages of a quantised cache under chunks of many rows: callers
 * without such chunks (a BF16 cache, or fewer than 1024 rows of a cache head in a call) do not need
 * them.  A workspace without them is taken for any call, and such chunks' pages are then decoded
 * where they are read, for every 256 rows again.
 * Errors: FT_ERR_INVALID, FT_ERR_CUDA. */
#define FT_ATTN_CLEAR_BYTES ((size_t)16384)
#define FT_ATTN_COPY_BYTES (((size_t)512 << 20) + 4352)
ft_status ft_attn_workspace(int n_heads, int n_kv_heads, int head_dim, size_t* bytes_out);

/* Attention of a batch's new tokens over the paged cache: single tokens (decode), a few
 * (checking drafted tokens) or whole chunks (prefill), mixed as they come.  Scores, softmax
 * statistics and sums are FP32; probabilities (times the scale of quantised values) are rounded to
 * BF16 for their product with the values, each term relative to itself.  Few rows over a quantised
 * cache take query elements below 2^-28 of their row's largest to within 2^-39 of it.  Which kernels run
 * follows from n_tokens, n_seqs, max_new, window and table_stride: a table much wider than the
 * lengths makes small batches slower.  The same arguments and inputs give the same bits.  Rows of q that no sequence names are left
 * unwritten in out and lse.  A length beyond table_stride pages, offsets outside
 * [0, n_tokens] or out of order, and page ids beyond the cache set FT_DEVERR_BAD_INDEX: the
 * length or offset is limited to its range, a bad page's tokens count as rows of zeros.
 * n_tokens = 0 or n_seqs = 0 does nothing.
 * Errors: FT_ERR_INVALID (arguments), FT_ERR_CAPACITY (workspace too small), FT_ERR_CUDA. */
ft_status ft_attn(const ft_kv_cache* cache, const ft_attn_args* args, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* FT_KV_H */

/*
 * vattn_serving.h -- C ABI of libvattn for a server of many requests: causal
 * attention over prompts packed into one buffer, a paged cache of keys and
 * values in 8 bits, and attention of new tokens over it, on one NVIDIA GB300
 * (sm_103a).
 *
 * Beside vattn_decoder.h, whose calls take padded batches and a cache of one
 * 16-bit buffer.  Tensors of rows, types, errors, threading, streams,
 * workspace and empty problems: as there.
 *
 * The cache.  A page holds page_size consecutive rows (tokens) of a sequence
 * for every key head; row r of sequence b is row r % page_size of page
 * table[b, r / page_size].  Its elements are e4m3 bytes (4 exponent and 3
 * mantissa bits, largest value 448, no infinities), with one f32 scale for
 * each page and head, of the keys and of the values: a byte x stands for
 * x * scale.  A table entry outside [0, n_pages) (-1, say) is a page that is
 * not there: appends to it are dropped, and its rows are seen by no query.
 * What a window has left behind can so be given back.  Pages may be shared
 * by sequences that read them; a page that an append writes to belongs to one
 * sequence of the call, and no two of its rows to one place.
 */
#ifndef VATTN_SERVING_H_
#define VATTN_SERVING_H_

#include "vattn_decoder.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The paged cache of one layer.  Device memory but for the struct itself. */
typedef struct {
  void* k;              /* e4m3 [n_pages, n_kv_heads, page_size, head_dim], 16-byte aligned: */
  void* v;
  int64_t k_stride[3];  /* bytes from page to page, head to head, row to row, multiples of 16; */
  int64_t v_stride[3];  /* elements are distinct, so either order of heads and rows does */
  float* k_scale;       /* [n_pages, n_kv_heads] contiguous, 2^-32 at least */
  float* v_scale;
  const int32_t* table;  /* [batch, max_pages] contiguous */
  const int32_t* kv_len; /* [batch]: rows of each sequence in use, new ones counted */
  int64_t n_pages;       /* < 2^31 - 1 */
  int64_t page_size;     /* a multiple of 16, 16..1024 */
  int64_t max_pages;     /* pages of a sequence; max_pages * page_size < 2^29 */
} vattn_pages;

/* Arguments of vattn_append_paged. */
typedef struct {
  int64_t batch;      /* sequences, < 2^30 */
  int64_t n_kv_heads;
  int64_t n_tokens;   /* cu_seqlens NULL: new tokens of each sequence; else of all together */
  int64_t head_dim;   /* a multiple of 16, at most 128 */
  int64_t rope_dims;  /* 0..head_dim: leading dims of the keys that are rotated */
  const int32_t* cu_seqlens; /* NULL, or [batch + 1]: sequence b's rows of k and v are [cu[b], cu[b + 1]) */
  const int32_t* positions;  /* NULL (the row in the cache), or of each row of k its position */
  const float* factors;      /* NULL, or rope_dims / 2 finite divisors != 0 of the angles */
  double base;        /* > 0, finite */
  int32_t dtype;      /* of k and v: VATTN_F16 or VATTN_BF16 */
} vattn_append_args;

/*
 * vattn_append_paged -- new keys and values of every sequence into the cache.
 * k, v: [batch, n_kv_heads, n_tokens, head_dim], or with cu_seqlens packed
 * [1, n_kv_heads, n_tokens, head_dim] (positions alike: [batch, n_tokens] or
 * [n_tokens]).  Of n new tokens, token i of sequence b goes to row
 * kv_len[b] - n + i (kv_len counts them already); rows < 0 or behind the
 * table's are dropped.  Keys are rotated on the way as by vattn_qk_norm_rope
 * (NeoX, angles good to about 2^-24 at any position).
 *
 * Scales are powers of two.  For a page and head that the call writes to, need =
 * the smallest 2^e with max |x| <= 448 * 2^e over its new finite values (of
 * rotated keys), 2^-32 at least.  A page whose row 0 is written starts anew,
 * with scale = need; else scale = max(scale, need), and the rows before the
 * new ones are rescaled to it, exactly but for values that leave e4m3's
 * normal range.  New values are x / scale rounded to nearest even, once, from
 * f32; an infinity or NaN becomes NaN.  (bf16 values beyond 448 * 2^100 make
 * scales that vattn_forward_paged does not take.)  Every other byte and scale
 * stays as it was, rows behind kv_len among them.
 *
 * cu_seqlens ascends; its values are held to [0, n_tokens], and a sequence
 * that ends before it begins is empty; if the sequences then have more than
 * n_tokens rows together, nothing is appended.  Rows of k and v in no sequence
 * are not read.  The same call gives the same bits every time, and repeated,
 * leaves what it left.
 */
vattn_status vattn_append_paged(const vattn_rows* k, const vattn_rows* v, const vattn_pages* cache,
                                const vattn_append_args* args, void* stream);

/*
 * vattn_forward_paged -- vattn_forward_cached over the paged cache: attention
 * of the n_queries = T <= VATTN_MAX_NEW_TOKENS newest tokens of each sequence,
 * in a row or as a tree, under a window whose first keys stay visible.
 *
 * args: as for vattn_forward_cached, but kv_len is the cache's (args->kv_len
 * and q_start NULL), n_keys is not used, and head_dim is a multiple of 16.
 * New token t's own key and value are cache row kv_len[b] - T + t, appended
 * before.  Sums and statistics are f32; q and the cache's values enter the
 * products exactly (bf16 q down to 2^-29 of its row's largest), the softmax
 * weights, times the values' scale, as f16.  Scales lie in 2^-100 .. 2^100
 * (powers of two or not), those of one sequence's values within 2^100 of each
 * other; a scale of 0 makes the page's keys zeros, or its values, these
 * whatever the bytes and counted as 2^-100.  What rows that no query sees
 * hold, bytes or scales, does not reach the result; any other NaN byte reaches
 * the queries that see it, and no others.
 * Scores that are not finite: as in vattn_forward_window.
 *
 * q, out [batch, n_q_heads, T, head_dim]; alignment and strides as in
 * vattn_forward_window.
 */
vattn_status vattn_forward_paged(const vattn_rows* q, const vattn_pages* cache,
                                 const vattn_rows* out, const vattn_window_args* args,
                                 void* stream);

/*
 * vattn_forward_packed -- vattn_forward_window for prompts of different
 * lengths that follow each other in one buffer: row i of sequence b is row
 * cu_seqlens[b] + i of q, k, v and out, and sees the rows j <= i of its own
 * sequence with j > i - window or j < n_sinks.
 *
 * cu_seqlens: [n_seqs + 1] on the device, ascending; its values are held to
 * [0, n_queries], and a sequence that ends before it begins is empty; if the
 * sequences then have more than n_queries rows together, none is computed.
 * q, out [1, n_q_heads, n_queries, head_dim], k and v [1, n_kv_heads,
 * n_queries, head_dim]: args->batch is 1, n_keys = n_queries, kv_len, q_start
 * and tree NULL; n_seqs < 2^24.  Rows in no sequence are left as they are, in
 * out and in lse (NULL, or f32 [n_q_heads, n_queries]).  All else as in
 * vattn_forward_window.
 */
vattn_status vattn_forward_packed(const vattn_rows* q, const vattn_rows* k, const vattn_rows* v,
                                  const vattn_rows* out, float* lse, const int32_t* cu_seqlens,
                                  int64_t n_seqs, const vattn_window_args* args, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* VATTN_SERVING_H_ */

/*
 * vattn_decoder.h -- C ABI of libvattn for decoder layers: norm and rotation
 * of q and k, causal attention under a sliding window with its gradients,
 * and attention of new tokens over a cache, on one NVIDIA GB300 (sm_103a).
 *
 * The shaders that vattn.h follows rotate q and k by position and attend
 * without a mask; these calls are this library's own for the layers of a
 * text decoder, in training and in serving.
 *
 * Tensors are [batch, heads, rows, head_dim] with any layout of the first
 * three dimensions (vattn_rows): head-major as in vattn.h, or views of a
 * packed projection [batch, rows, heads, head_dim].  The last dimension is
 * contiguous.  Types: see vattn_dtype.  All sums, softmax statistics and
 * norms are held in f32; a result is rounded to its type once, to nearest
 * even.
 *
 * Errors, threading and streams: as in vattn.h.  Every call is asynchronous
 * on `stream`, checks its arguments on the host before any CUDA call, keeps
 * no reference to the caller's buffers after its work on the stream is done,
 * and takes what workspace it needs stream-ordered from the library's pool,
 * so calls on different streams do not share any.  All pointers are device
 * memory of the device that is current on the calling thread, unless said
 * otherwise.  An empty problem is a successful no-op.
 */
#ifndef VATTN_DECODER_H_
#define VATTN_DECODER_H_

#include "vattn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { VATTN_F32 = 0, VATTN_F16 = 1, VATTN_BF16 = 2 } vattn_dtype;

/*
 * A tensor [batch, heads, rows, head_dim]: element (b, h, i, d) sits at
 * data + (b * stride[0] + h * stride[1] + i * stride[2] + d) elements.
 * Strides are >= 0; an input may have stride 0 (a broadcast), an output's
 * elements are distinct.  Outputs do not overlap inputs or each other (views
 * of one packed buffer with equal strides that interleave without sharing
 * elements are fine).
 */
typedef struct {
  void* data;
  int64_t stride[3];
} vattn_rows;

/* Arguments of vattn_qk_norm_rope and its gradient. */
typedef struct {
  int64_t batch;
  int64_t n_q_heads;
  int64_t n_kv_heads;
  int64_t n_patches;
  int64_t head_dim;  /* 1..128 */
  int64_t rope_dims; /* 0..head_dim: leading dims that are rotated */
  int64_t pos0;      /* position of row 0 when positions is NULL, >= 0 */
  const int32_t* positions; /* NULL, or [batch, n_patches]: each row's position */
  const float* factors;     /* NULL, or rope_dims / 2 finite divisors != 0 of the angles */
  const void* q_weight;     /* NULL (ones), or [head_dim] */
  const void* k_weight;
  double base;              /* > 0, finite */
  float eps;                /* >= 0, finite */
  int32_t dtype;            /* of q, k and their outputs and gradients */
  int32_t weight_dtype;     /* VATTN_F32 or dtype */
} vattn_qk_args;

/*
 * vattn_qk_norm_rope -- RMS norm of every row of q and k and the forward
 * NeoX rotation, in one pass: with r = 1 / sqrt(mean(x^2) + eps),
 * y = x r w, and for i < half = rope_dims / 2 and theta_i = position *
 * base^(-2 i / rope_dims) (/ factors[i]):
 *   out[i] = y[i] cos - y[i + half] sin, out[i + half] = y[i] sin + y[i + half] cos
 * and out = y in the dims from 2 * half on.  Angles are exact to about 2^-24
 * at any 32-bit position (vattn_rope_neox computes them in f32).
 * q_out may be q itself and k_out k itself (same pointer and strides).
 */
vattn_status vattn_qk_norm_rope(const vattn_rows* q, const vattn_rows* k, const vattn_rows* q_out,
                                const vattn_rows* k_out, const vattn_qk_args* args, void* stream);

/*
 * vattn_qk_norm_rope_backward -- gradients of vattn_qk_norm_rope: from those
 * of its outputs (dq_out, dk_out) and its inputs, those of q and k, and with
 * a weight those of the weights (f32 [head_dim] each, summed over all rows
 * in a fixed order; NULL: not wanted, or no weight).  dq may be dq_out or q
 * itself, dk likewise.
 */
vattn_status vattn_qk_norm_rope_backward(const vattn_rows* dq_out, const vattn_rows* dk_out,
                                         const vattn_rows* q, const vattn_rows* k,
                                         const vattn_rows* dq, const vattn_rows* dk,
                                         float* dq_weight, float* dk_weight,
                                         const vattn_qk_args* args, void* stream);

/* Arguments of the attention calls below. */
typedef struct {
  int64_t batch;
  int64_t n_q_heads;   /* a multiple of n_kv_heads: query head h reads */
  int64_t n_kv_heads;  /* key head h / (n_q_heads / n_kv_heads) */
  int64_t n_queries;   /* rows of q */
  int64_t n_keys;      /* rows of k and v */
  int64_t head_dim;    /* a multiple of 8, at most 128 */
  int64_t window;      /* keys a query sees, itself among them; 0: all before it */
  int64_t n_sinks;     /* first keys that every later query sees as well */
  const int32_t* kv_len;    /* NULL (n_keys), or [batch]: keys of each sequence */
  const int32_t* q_start;   /* NULL (kv_len - n_queries), or [batch]: position of query row 0 */
  const uint64_t* tree;     /* vattn_forward_cached only */
  float scale;              /* > 0, finite: factor of the scores */
  int32_t dtype;            /* VATTN_F16 or VATTN_BF16 */
} vattn_window_args;

/*
 * vattn_forward_window -- causal attention under a sliding window whose
 * first keys stay visible:
 *   out[b, h, i] = sum_j softmax_j(scale * q[b, h, i] . k[b, g, j]) v[b, g, j]
 * over the keys j that row i sees.  Key j is at position j; row i at
 * p = q_start[b] + i; with len = kv_len[b] (held to [0, n_keys]) the row sees
 *   j <= p < len  with  j > p - window  or  j < n_sinks.
 * A row that sees nothing (p < 0, p >= len) gets zeros, and lse = -infinity.
 * What k and v hold at keys that a row does not see does not reach the row,
 * infinities and NaN included.  An infinity or NaN of v reaches the rows that
 * see it, at the cost of a second look at a few tiles.  A row all of whose
 * scores are -infinity counts as one that sees nothing.  The sum of the weights
 * times v is divided by that of the weights at its end, and is f32 before: in
 * bf16 |v| beyond 2^120 / keys may overflow it.
 *
 * q [batch, n_q_heads, n_queries, head_dim], k and v [batch, n_kv_heads,
 * n_keys, head_dim], out as q: 16-byte aligned, strides multiples of 8
 * elements, and (here and in vattn_backward_window) a row stride of at least
 * head_dim: broadcast heads and sequences are read as they are, broadcast
 * rows are refused.  lse: NULL or f32 [batch, n_q_heads, n_queries] contiguous, the
 * natural logarithm of the sum of the row's exponentials (for
 * vattn_backward_window).  n_queries, n_keys < 2^29, batch times either
 * number of heads < 2^30; q_start is held to +-2^30.
 */
vattn_status vattn_forward_window(const vattn_rows* q, const vattn_rows* k, const vattn_rows* v,
                                  const vattn_rows* out, float* lse,
                                  const vattn_window_args* args, void* stream);

/*
 * vattn_backward_window -- gradients of vattn_forward_window with respect to
 * q, k and v, from dout, the inputs, out and lse of the forward call.  dk and
 * dv are summed over the query heads of a key head.  Rows that see nothing,
 * and keys that no row sees, get zeros.  The same call gives the same bits
 * every time (no atomics).  k, v behind kv_len and q, dout of rows that see
 * nothing may hold anything; a NaN or infinity elsewhere may reach the
 * gradients of rows within 128 of its own.  The softmax weights p and the
 * score gradients p (dp - delta) are rounded to the tensors' type on the way,
 * in f16 times powers of two: neither overflows, and terms keep their digits
 * down to 2^-29 of the largest that 128 rows or keys can give.
 * dq as q, dk as k, dv as v; dout as out.
 */
vattn_status vattn_backward_window(const vattn_rows* dout, const vattn_rows* q, const vattn_rows* k,
                                   const vattn_rows* v, const vattn_rows* out, const float* lse,
                                   const vattn_rows* dq, const vattn_rows* dk,
                                   const vattn_rows* dv, const vattn_window_args* args,
                                   void* stream);

/* Most new tokens of one vattn_forward_cached call. */
#define VATTN_MAX_NEW_TOKENS 64

/*
 * vattn_forward_cached -- attention of the n_queries = T newest tokens of
 * each sequence over its cache, T <= VATTN_MAX_NEW_TOKENS.
 *
 * k, v: the cache, n_keys rows a sequence of which the first kv_len[b]
 * (required, counting the T new tokens) are in use; new token t's own key
 * and value are row base + t, base = kv_len[b] - T.
 * tree: NULL (each new token follows the one before it), or [batch, T]
 * words: bit u of word t says that new token u is an ancestor of t or t
 * itself (drafted tokens in a tree).  With depth_t = the word's bits - 1,
 * token t is at position base + depth_t, and sees the cache rows j < base
 * and the new tokens of its word whose position is > base + depth_t -
 * window or < n_sinks.  A word without bits sees nothing.  Bits >= T are
 * ignored.  Tokens whose row base + t is negative see nothing and are seen
 * by none; they get zeros.  What other rows hold does not reach the result.
 * Scores and values that are not finite: as in vattn_forward_window.
 *
 * q, out [batch, n_q_heads, T, head_dim]; alignment and strides as in
 * vattn_forward_window; q_start must be NULL.
 */
vattn_status vattn_forward_cached(const vattn_rows* q, const vattn_rows* k, const vattn_rows* v,
                                  const vattn_rows* out, const vattn_window_args* args,
                                  void* stream);

#ifdef __cplusplus
}
#endif

#endif /* VATTN_DECODER_H_ */

// window_host.h -- host side that the attention calls under a window share:
// checks of their arguments and the kernels' sizes.
#pragma once

#include <algorithm>
#include <cmath>

#include "rows_host.h"

namespace vattn {
namespace host {

constexpr int64_t kMaxRows = (int64_t{1} << 30) - 1;
constexpr int64_t kMaxKeys = (int64_t{1} << 29) - 1;  // positions and their differences fit in 32 bits

inline vattn_status check_window_args(const vattn_window_args* a) {
  if (!a) return fail(VATTN_ERR_INVALID_ARG, "null args");
  if (a->batch < 0 || a->n_q_heads < 0 || a->n_kv_heads < 0 || a->n_queries < 0 || a->n_keys < 0)
    return fail(VATTN_ERR_INVALID_ARG,
                "negative size (batch=%lld n_q_heads=%lld n_kv_heads=%lld n_queries=%lld n_keys=%lld)",
                (long long)a->batch, (long long)a->n_q_heads, (long long)a->n_kv_heads,
                (long long)a->n_queries, (long long)a->n_keys);
  if (a->head_dim < 1) return fail(VATTN_ERR_INVALID_ARG, "head_dim must be >= 1");
  if (a->head_dim > VATTN_MAX_HEAD_DIM || a->head_dim % 8 != 0)
    return fail(VATTN_ERR_UNSUPPORTED, "head_dim %lld: a multiple of 8 up to %d is needed (16-byte rows)",
                (long long)a->head_dim, VATTN_MAX_HEAD_DIM);
  if (a->dtype != VATTN_F16 && a->dtype != VATTN_BF16)
    return fail(VATTN_ERR_UNSUPPORTED, "dtype must be VATTN_F16 or VATTN_BF16");
  if (a->n_kv_heads == 0 ? a->n_q_heads != 0 : a->n_q_heads % a->n_kv_heads != 0)
    return fail(VATTN_ERR_INVALID_ARG, "n_q_heads %lld is not a multiple of n_kv_heads %lld",
                (long long)a->n_q_heads, (long long)a->n_kv_heads);
  if (a->n_queries > kMaxKeys || a->n_keys > kMaxKeys)
    return fail(VATTN_ERR_UNSUPPORTED, "n_queries and n_keys must stay below 2^29");
  if (a->n_q_heads > kMaxRows || a->n_kv_heads > kMaxRows || a->batch > kMaxRows ||
      a->batch * std::max(a->n_q_heads, a->n_kv_heads) > kMaxRows)
    return fail(VATTN_ERR_UNSUPPORTED, "batch * n_q_heads and batch * n_kv_heads must stay below 2^30");
  if (a->window < 0) return fail(VATTN_ERR_INVALID_ARG, "window must be >= 0");
  if (a->n_sinks < 0) return fail(VATTN_ERR_INVALID_ARG, "n_sinks must be >= 0");
  if (!(a->scale > 0.0f) || !std::isfinite(a->scale))
    return fail(VATTN_ERR_INVALID_ARG, "scale must be a finite positive number");
  if ((reinterpret_cast<uintptr_t>(a->kv_len) | reinterpret_cast<uintptr_t>(a->q_start)) & 3u)
    return fail(VATTN_ERR_MISALIGNED, "kv_len and q_start must be 4-byte aligned");
  if (reinterpret_cast<uintptr_t>(a->tree) & 7u)
    return fail(VATTN_ERR_MISALIGNED, "tree must be 8-byte aligned");
  return VATTN_OK;
}

inline Tensor window_tensor(const char* name, const vattn_rows* t, const vattn_window_args* a, bool is_q, bool out) {
  return Tensor{name, t, {a->batch, is_q ? a->n_q_heads : a->n_kv_heads, is_q ? a->n_queries : a->n_keys},
                a->head_dim, 2, out};
}

inline WindowParams window_params(const vattn_window_args* a) {
  WindowParams w{};
  w.kv_len = a->kv_len;
  w.q_start = a->q_start;
  w.tree = a->tree;
  w.batch = static_cast<int>(a->batch);
  w.heads = static_cast<int>(a->n_q_heads);
  w.kv_heads = static_cast<int>(a->n_kv_heads);
  w.group = a->n_kv_heads > 0 ? static_cast<int>(a->n_q_heads / a->n_kv_heads) : 0;
  w.n_queries = static_cast<int>(a->n_queries);
  w.n_keys = static_cast<int>(a->n_keys);
  w.dim = static_cast<int>(a->head_dim);
  const int64_t none = kMaxKeys + 1;
  w.window = static_cast<int>(a->window == 0 || a->window > none ? none : a->window);
  w.sinks = static_cast<int>(a->n_sinks > none ? none : a->n_sinks);
  w.scale = a->scale;
  const uint64_t key_tiles = static_cast<uint64_t>(a->n_keys) / kTile + 1;
  const uint64_t row_tiles = static_cast<uint64_t>(w.group) * (static_cast<uint64_t>(a->n_queries) / kTile + 1);
  w.wait_ns = kPipeTimeoutNs + kPipeTileNs * (key_tiles + row_tiles);
  return w;
}

inline vattn_status forward_checks(const vattn_rows* q, const vattn_rows* k, const vattn_rows* v,
                            const vattn_rows* out, const float* lse, const vattn_window_args* a) {
  const Tensor tq = window_tensor("q", q, a, true, false), tk = window_tensor("k", k, a, false, false),
               tv = window_tensor("v", v, a, false, false), to = window_tensor("out", out, a, true, true);
  for (const Tensor* t : {&tq, &tk, &tv, &to}) {
    const vattn_status st = check_tensor(*t, 16);
    if (st != VATTN_OK) return st;
  }
  for (const Tensor* t : {&tq, &tk, &tv}) {
    const vattn_status st = check_apart(to, *t);
    if (st != VATTN_OK) return st;
  }
  if (reinterpret_cast<uintptr_t>(lse) & 3u) return fail(VATTN_ERR_MISALIGNED, "lse must be 4-byte aligned");
  const uint64_t bytes = static_cast<uint64_t>(a->batch) * a->n_q_heads * a->n_queries * 4u;
  for (const Tensor* t : {&tq, &tk, &tv, &to}) {
    const vattn_status st = check_apart_bytes(lse, bytes, "lse", *t);
    if (st != VATTN_OK) return st;
  }
  return VATTN_OK;
}

}  // namespace host
}  // namespace vattn

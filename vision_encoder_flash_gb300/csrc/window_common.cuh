// window_common.cuh -- which keys a query sees, shared by the attention
// kernels of the decoder calls.
#pragma once

#include <cstdint>

#include "elem.cuh"

namespace vattn {

// Window and sizes of one call.
struct WindowParams {
  const int32_t* kv_len;   // [batch] or null: n_keys
  const int32_t* q_start;  // [batch] or null: kv_len - n_queries
  const uint64_t* tree;    // [batch, n_queries] or null (cached form)
  int batch, heads, kv_heads, group;  // group = heads / kv_heads
  int n_queries, n_keys, dim;
  int window;  // >= 1; no limit: 2^30 (positions that matter are < n_keys < 2^30)
  int sinks;
  float scale;
};

// Length of sequence b and position of its query row 0.  Row i at p = start
// + i sees key j iff j <= p < len and (j > p - window or j < sinks).
struct Seq {
  int len, start;
};

__device__ __forceinline__ Seq window_seq(const WindowParams& p, int b) {
  Seq s;
  s.len = p.kv_len != nullptr ? min(max(p.kv_len[b], 0), p.n_keys) : p.n_keys;
  s.start = p.q_start != nullptr ? min(max(p.q_start[b], -(1 << 30)), 1 << 30)
                                 : s.len - p.n_queries;
  return s;
}

__device__ __forceinline__ bool window_sees(const WindowParams& p, const Seq& s, int i, int j) {
  const int pos = s.start + i;
  return j <= pos && pos < s.len && (j > pos - p.window || j < p.sinks);
}

}  // namespace vattn

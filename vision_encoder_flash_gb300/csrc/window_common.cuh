// window_common.cuh -- which keys a query sees, shared by the attention
// kernels of the decoder calls.
#pragma once

#include <cstdint>

#include "elem.cuh"

namespace vattn {

// Division of n < 2^31 by a divisor known on the host, as a multiplication: q
// = hi32(n * m) >> s with m = floor(2^(32 + s) / d) + 1, s = floor(log2(d - 1)),
// exact because n (m d - 2^(32 + s)) < 2^(32 + s).
struct FastDiv {
  uint32_t d, m, s;
  __host__ static FastDiv make(uint32_t d) {
    FastDiv f{d, 0, 0};
    if (d > 1) {
      while ((2u << f.s) < d) ++f.s;
      f.m = static_cast<uint32_t>((uint64_t{1} << (32 + f.s)) / d + 1);
    }
    return f;
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const { return d == 1 ? n : __umulhi(n, m) >> s; }
  __device__ __forceinline__ uint32_t div(uint32_t n, uint32_t* rest) const {
    const uint32_t q = div(n);
    *rest = n - q * d;
    return q;
  }
};

// Window and sizes of one call.
struct WindowParams {
  const int32_t* kv_len;   // [batch] or null: n_keys
  const int32_t* q_start;  // [batch] or null: kv_len - n_queries
  const uint64_t* tree;    // [batch, n_queries] or null (cached form)
  int batch, heads, kv_heads, group;  // group = heads / kv_heads
  int n_queries, n_keys, dim;
  int window;  // >= 1; no limit: 2^29 (positions that matter are < n_keys < 2^29)
  int sinks;
  float scale;
  unsigned long long wait_ns;  // limit of a wait inside the kernels (window_pipe.cuh)
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

// A tensor [batch, heads, rows, dim] with its first three strides.
struct RowsTensor {
  const void* p;
  long long s[3];
};

template <typename T>
__device__ __forceinline__ const T* rows_at(const RowsTensor& t, long long b, long long h, long long i) {
  return static_cast<const T*>(t.p) + b * t.s[0] + h * t.s[1] + i * t.s[2];
}
template <typename T>
__device__ __forceinline__ T* rows_at_mut(const RowsTensor& t, long long b, long long h, long long i) {
  return const_cast<T*>(rows_at<T>(t, b, h, i));
}

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

}  // namespace vattn

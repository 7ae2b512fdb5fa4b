// window_rows_kernel.cuh -- the attention of the decoder calls, one warp per
// row, straight from the formulas (see vattn_decoder.h).
#pragma once

#include "ptx.cuh"
#include "window_common.cuh"

namespace vattn {

constexpr int kRowsWarps = 4;
constexpr int kRowsMaxDim = 128;

struct RowsParams {
  WindowParams w;
  RowsTensor q, k, v, out;
};

template <typename T>
__device__ __forceinline__ float rows_dot(const float* a, const T* b, int D) {
  float s = 0.0f;
  for (int d = 0; d < D; d += 8) {
    float x[8];
    reinterpret_cast<const Vec<T, 8>*>(b + d)->widen(x);
#pragma unroll
    for (int e = 0; e < 8; ++e) s = fmaf(a[d + e], x[e], s);
  }
  return s;
}

// Does new token t (row i of the call) see cache row j?  See vattn_forward_cached.
__device__ __forceinline__ bool cached_sees(const WindowParams& p, const Seq& s, int b, int t, int j) {
  const int T = p.n_queries, base = s.start;
  if (base + t < 0 || j >= s.len || j < 0) return false;
  const uint64_t all = T == 64 ? ~0ull : (1ull << T) - 1;
  const uint64_t* words = p.tree + static_cast<long long>(b) * T;
  const uint64_t mine = words[t] & all;
  if (mine == 0) return false;
  const int pos = base + __popcll(mine) - 1;
  int kpos = j;
  if (j >= base) {
    const int u = j - base;
    if (((mine >> u) & 1) == 0) return false;
    kpos = base + __popcll(words[u] & all) - 1;
  }
  return kpos > pos - p.window || kpos < p.sinks;
}

template <typename T>
__global__ void __launch_bounds__(kRowsWarps * 32)
    vattn_window_rows_kernel(const __grid_constant__ RowsParams p) {
  __shared__ float qs[kRowsWarps][kRowsMaxDim];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * kRowsWarps + warp;
  const WindowParams& w = p.w;
  if (row >= static_cast<long long>(w.batch) * w.heads * w.n_queries) return;
  const int i = static_cast<int>(row % w.n_queries);
  const int h = static_cast<int>(row / w.n_queries % w.heads);
  const int b = static_cast<int>(row / w.n_queries / w.heads);
  const int kh = h / w.group, D = w.dim;
  const Seq s = window_seq(w, b);
  for (int d = lane; d < D; d += 32) qs[warp][d] = Elem<T>::widen(rows_at<T>(p.q, b, h, i)[d]) * w.scale;
  __syncwarp();
  float m = -INFINITY, l = 0.0f, o[kRowsMaxDim / 32] = {};
  const int hi = min(s.len, w.tree != nullptr ? s.len : s.start + i + 1);
  for (int j0 = 0; j0 < hi; j0 += 32) {
    const int j = j0 + lane;
    const bool see = j < hi && (w.tree != nullptr ? cached_sees(w, s, b, i, j) : window_sees(w, s, i, j));
    if (!__any_sync(0xffffffffu, see)) continue;
    const float x = see ? rows_dot(qs[warp], rows_at<T>(p.k, b, kh, j), D) : -INFINITY;
    const float mn = fmaxf(m, warp_max(x));
    const float ref = mn == -INFINITY ? 0.0f : mn;
    const float alpha = __expf(m - ref), e = see ? __expf(x - ref) : 0.0f;
    l = l * alpha + warp_sum(e);
    m = mn;
#pragma unroll
    for (int c = 0; c < kRowsMaxDim / 32; ++c) o[c] *= alpha;
    for (uint32_t left = __ballot_sync(0xffffffffu, see); left != 0; left &= left - 1) {
      const int k = __ffs(left) - 1;
      const float pk = __shfl_sync(0xffffffffu, e, k);
      const T* v = rows_at<T>(p.v, b, kh, j0 + k);
#pragma unroll
      for (int c = 0; c < kRowsMaxDim / 32; ++c)
        if (lane + 32 * c < D) o[c] = fmaf(pk, Elem<T>::widen(v[lane + 32 * c]), o[c]);
    }
  }
  const float inv = l > 0.0f || l != l ? 1.0f / l : 0.0f;
#pragma unroll
  for (int c = 0; c < kRowsMaxDim / 32; ++c)
    if (lane + 32 * c < D)
      rows_at_mut<T>(p.out, b, h, i)[lane + 32 * c] = Elem<T>::narrow(l == 0.0f ? 0.0f : o[c] * inv);
}

}  // namespace vattn

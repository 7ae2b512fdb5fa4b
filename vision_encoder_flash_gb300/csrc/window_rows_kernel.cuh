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
  RowsTensor q, k, v, out, dout, dq, dk, dv;
  float* lse;
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
  if (lane == 0 && p.lse != nullptr) p.lse[row] = l == 0.0f ? -INFINITY : m + logf(l);
}

// dq: one warp per query row.
template <typename T>
__global__ void __launch_bounds__(kRowsWarps * 32)
    vattn_window_rows_dq_kernel(const __grid_constant__ RowsParams p) {
  __shared__ float qs[kRowsWarps][kRowsMaxDim], ds[kRowsWarps][kRowsMaxDim];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * kRowsWarps + warp;
  const WindowParams& w = p.w;
  if (row >= static_cast<long long>(w.batch) * w.heads * w.n_queries) return;
  const int i = static_cast<int>(row % w.n_queries);
  const int h = static_cast<int>(row / w.n_queries % w.heads);
  const int b = static_cast<int>(row / w.n_queries / w.heads);
  const int kh = h / w.group, D = w.dim;
  const Seq s = window_seq(w, b);
  float delta = 0.0f;
  for (int d = lane; d < D; d += 32) {
    qs[warp][d] = Elem<T>::widen(rows_at<T>(p.q, b, h, i)[d]) * w.scale;
    ds[warp][d] = Elem<T>::widen(rows_at<T>(p.dout, b, h, i)[d]);
    delta += ds[warp][d] * Elem<T>::widen(rows_at<T>(p.out, b, h, i)[d]);
  }
  delta = warp_sum(delta);
  __syncwarp();
  const float lse = p.lse[row];
  float o[kRowsMaxDim / 32] = {};
  const int hi = min(s.len, s.start + i + 1);
  for (int j0 = 0; j0 < hi; j0 += 32) {
    const int j = j0 + lane;
    const bool see = j < hi && window_sees(w, s, i, j);
    if (!__any_sync(0xffffffffu, see)) continue;
    float g = 0.0f;
    if (see)
      g = __expf(rows_dot(qs[warp], rows_at<T>(p.k, b, kh, j), D) - lse) *
          (rows_dot(ds[warp], rows_at<T>(p.v, b, kh, j), D) - delta);
    for (uint32_t left = __ballot_sync(0xffffffffu, see); left != 0; left &= left - 1) {
      const int k = __ffs(left) - 1;
      const float pk = __shfl_sync(0xffffffffu, g, k);
      const T* x = rows_at<T>(p.k, b, kh, j0 + k);
#pragma unroll
      for (int c = 0; c < kRowsMaxDim / 32; ++c)
        if (lane + 32 * c < D) o[c] = fmaf(pk, Elem<T>::widen(x[lane + 32 * c]), o[c]);
    }
  }
#pragma unroll
  for (int c = 0; c < kRowsMaxDim / 32; ++c)
    if (lane + 32 * c < D)
      rows_at_mut<T>(p.dq, b, h, i)[lane + 32 * c] = Elem<T>::narrow(o[c] * w.scale);
}

// dk and dv: one warp per key row, over the query rows of its group's heads.
template <typename T>
__global__ void __launch_bounds__(kRowsWarps * 32)
    vattn_window_rows_dkv_kernel(const __grid_constant__ RowsParams p) {
  __shared__ float ks[kRowsWarps][kRowsMaxDim], vs[kRowsWarps][kRowsMaxDim];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * kRowsWarps + warp;
  const WindowParams& w = p.w;
  if (row >= static_cast<long long>(w.batch) * w.kv_heads * w.n_keys) return;
  const int j = static_cast<int>(row % w.n_keys);
  const int kh = static_cast<int>(row / w.n_keys % w.kv_heads);
  const int b = static_cast<int>(row / w.n_keys / w.kv_heads);
  const int D = w.dim;
  const Seq s = window_seq(w, b);
  for (int d = lane; d < D; d += 32) {
    ks[warp][d] = Elem<T>::widen(rows_at<T>(p.k, b, kh, j)[d]) * w.scale;
    vs[warp][d] = Elem<T>::widen(rows_at<T>(p.v, b, kh, j)[d]);
  }
  __syncwarp();
  float ok[kRowsMaxDim / 32] = {}, ov[kRowsMaxDim / 32] = {};
  for (int g = 0; g < w.group; ++g) {
    const int h = kh * w.group + g;
    for (int i0 = 0; i0 < w.n_queries; i0 += 32) {
      const int i = i0 + lane;
      const bool see = i < w.n_queries && window_sees(w, s, i, j);
      if (!__any_sync(0xffffffffu, see)) continue;
      float pij = 0.0f, gij = 0.0f;
      if (see) {
        const T* dr = rows_at<T>(p.dout, b, h, i);
        const T* orow = rows_at<T>(p.out, b, h, i);
        float delta = 0.0f;
        for (int d = 0; d < D; ++d) delta = fmaf(Elem<T>::widen(dr[d]), Elem<T>::widen(orow[d]), delta);
        const float lse = p.lse[(static_cast<long long>(b) * w.heads + h) * w.n_queries + i];
        pij = __expf(rows_dot(ks[warp], rows_at<T>(p.q, b, h, i), D) - lse);
        gij = pij * (rows_dot(vs[warp], dr, D) - delta);
      }
      for (uint32_t left = __ballot_sync(0xffffffffu, see); left != 0; left &= left - 1) {
        const int k = __ffs(left) - 1;
        const float pk = __shfl_sync(0xffffffffu, pij, k), gk = __shfl_sync(0xffffffffu, gij, k);
        const T* x = rows_at<T>(p.q, b, h, i0 + k);
        const T* y = rows_at<T>(p.dout, b, h, i0 + k);
#pragma unroll
        for (int c = 0; c < kRowsMaxDim / 32; ++c)
          if (lane + 32 * c < D) {
            ok[c] = fmaf(gk, Elem<T>::widen(x[lane + 32 * c]), ok[c]);
            ov[c] = fmaf(pk, Elem<T>::widen(y[lane + 32 * c]), ov[c]);
          }
      }
    }
  }
#pragma unroll
  for (int c = 0; c < kRowsMaxDim / 32; ++c)
    if (lane + 32 * c < D) {
      rows_at_mut<T>(p.dk, b, kh, j)[lane + 32 * c] = Elem<T>::narrow(ok[c] * w.scale);
      rows_at_mut<T>(p.dv, b, kh, j)[lane + 32 * c] = Elem<T>::narrow(ov[c]);
    }
}

}  // namespace vattn

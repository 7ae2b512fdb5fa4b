// qk_norm_rope_kernel.cuh -- RMS norm of every q and k row with the NeoX
// rotation in the same pass, and its gradient.
//
// A row is one head of one token, x[0 .. D).  With r = 1 / sqrt(mean(x^2) +
// eps) and w the tensor's weight:
//   y = x r w,   out = R(theta) y,
// where R turns the pairs (y[i], y[i + half]), i < half = rope_dims / 2, by
// theta_i = position * base^(-2 i / rope_dims) (/ factors[i]) as
// rope_kernel.cuh does and leaves dims >= 2 * half alone.  Backward, from g
// = d out:
//   g' = R(-theta) g,   dw += g' x r,   dx = r (g' w) - x r^3 / D sum(g' w x).
//
// Angles: in turns, position * f_i only counts modulo 1, so f_i is held as a
// 64-bit binary fraction (from f64) and position * f_i is one wrapping
// integer product: exact to 2^-33 turns at any 32-bit position, where an f32
// product loses all digits.  sincospif of the remainder does the rest.
//
// Work split: a group of lanes holds one row, lane = slot of V pairs (two
// 16-byte loads where the sizes allow), so the rotation needs no exchange
// and the sums a few shuffles.  A group stays on one token and walks over
// that token's heads of one tensor (a slice of them): the angles are computed
// once per token and slice and stay in registers, and the four rows in flight
// per thread keep the loads ahead of the arithmetic.  Memory bound: each row
// is read once and written once.
#pragma once

#include <cstdint>

#include "elem.cuh"
#include "ptx.cuh"

namespace vattn {

constexpr int kQkThreads = 256;
constexpr int kQkMaxDim = 128;

struct QkTensor {
  const void* x;   // input rows
  const void* g;   // gradient of the output rows (backward)
  void* y;         // output rows, or gradient of the input rows
  const void* w;   // weight or null
  long long xs[3], gs[3], ys[3];  // strides (batch, head, row), elements
  int heads;
  int slices;           // blocks in y that share the heads
  int heads_per_slice;
};

struct QkParams {
  QkTensor t[2];  // q, k
  const int32_t* positions;
  const float* factors;
  float* part;  // backward: [gridDim.y * gridDim.x][D] weight gradient of each block
  long long tokens;
  long long pos0;
  int n;  // rows of a sequence
  int D;
  int half;
  int slots;  // pair slots of a row
  int log_lanes;
  int w_f32;
  float eps;
  double turns[kQkMaxDim / 2];  // turns per position
};

// One lane's place in a row: V pairs (a[ia ..], b[ib ..]).
template <int V>
struct QkSlot {
  int ia, ib;
  bool here, pair, rot;
  __device__ __forceinline__ void set(const QkParams& p, int c) {
    const int i = c * V, rest = p.D - 2 * p.half;
    here = c < p.slots;
    rot = here && i < p.half;
    const int r = i - p.half;
    ia = rot ? i : 2 * p.half + r;
    ib = rot ? i + p.half : 2 * p.half + (rest + 1) / 2 + r;
    pair = here && ib < p.D;  // V == 1 and an odd rest: the last slot has no partner
  }
};

template <int V>
__device__ __forceinline__ void qk_weight(const QkSlot<V>& s, const void* w, int w_f32, bool bf16,
                                          float (&wa)[V], float (&wb)[V]) {
  auto at = [&](int i) -> float {
    if (w == nullptr) return 1.0f;
    if (w_f32) return static_cast<const float*>(w)[i];
    return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i])
                : __half2float(static_cast<const __half*>(w)[i]);
  };
#pragma unroll
  for (int e = 0; e < V; ++e) {
    wa[e] = s.here ? at(s.ia + e) : 0.0f;
    wb[e] = s.pair ? at(s.ib + e) : 0.0f;
  }
}

template <int V>
__device__ __forceinline__ void qk_angles(const QkSlot<V>& s, const uint64_t* turn, int c,
                                          long long pos, float (&cs)[V], float (&sn)[V]) {
#pragma unroll
  for (int e = 0; e < V; ++e) {
    cs[e] = 1.0f;
    sn[e] = 0.0f;
    if (s.rot) {
      const uint64_t phase = static_cast<uint64_t>(pos) * turn[c * V + e];
      // half turns in [-1, 1)
      const float h = static_cast<float>(static_cast<int32_t>(phase >> 32)) * 0x1p-31f;
      sincospif(h, &sn[e], &cs[e]);
    }
  }
}

__device__ __forceinline__ void qk_turns(const QkParams& p, uint64_t* turn) {
  if (static_cast<int>(threadIdx.x) < p.half) {
    double f = p.turns[threadIdx.x];
    if (p.factors != nullptr) f /= static_cast<double>(p.factors[threadIdx.x]);
    f -= floor(f);
    turn[threadIdx.x] = static_cast<uint64_t>(f * 0x1p64);
  }
  __syncthreads();
}

template <typename T, int V>
__device__ __forceinline__ Vec<T, V> qk_load(const T* row, int i, bool here) {
  Vec<T, V> v;
  if (here) {
    v = *reinterpret_cast<const Vec<T, V>*>(row + i);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) v.e[e] = Elem<T>::narrow(0.0f);
  }
  return v;
}

// Sum over the lanes of a group (xor below the group's size stays inside).
__device__ __forceinline__ float qk_group_sum(float x, int lanes) {
  for (int o = lanes >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// SL slots per lane (2 only where V == 1 needs up to 64 slots of a warp).
template <typename T, int V, int SL>
__global__ void __launch_bounds__(kQkThreads)
    vattn_qk_norm_rope_kernel(const __grid_constant__ QkParams p) {
  constexpr int U = SL == 1 ? 4 : 2;  // rows in flight
  __shared__ uint64_t turn[kQkMaxDim / 2];
  qk_turns(p, turn);
  const bool is_q = static_cast<int>(blockIdx.y) < p.t[0].slices;
  const QkTensor& t = p.t[is_q ? 0 : 1];
  const int slice = static_cast<int>(blockIdx.y) - (is_q ? 0 : p.t[0].slices);
  const int h0 = slice * t.heads_per_slice;
  const int h1 = min(t.heads, h0 + t.heads_per_slice);
  const int lanes = 1 << p.log_lanes;
  const int c0 = static_cast<int>(threadIdx.x) & (lanes - 1);
  const long long token = static_cast<long long>(blockIdx.x) * (kQkThreads >> p.log_lanes) +
                          (threadIdx.x >> p.log_lanes);
  const bool valid = token < p.tokens;
  const long long tk = valid ? token : p.tokens - 1;
  const long long b = tk / p.n, n = tk - b * p.n;
  const long long pos = p.positions != nullptr ? p.positions[tk] : p.pos0 + n;
  QkSlot<V> s[SL];
  float cs[SL][V], sn[SL][V], wa[SL][V], wb[SL][V];
#pragma unroll
  for (int k = 0; k < SL; ++k) {
    s[k].set(p, c0 + k * lanes);
    qk_angles<V>(s[k], turn, c0 + k * lanes, pos, cs[k], sn[k]);
    qk_weight<V>(s[k], t.w, p.w_f32, Elem<T>::kBf16, wa[k], wb[k]);
  }
  const T* x0 = static_cast<const T*>(t.x) + b * t.xs[0] + n * t.xs[2];
  T* y0 = static_cast<T*>(t.y) + b * t.ys[0] + n * t.ys[2];
  const float inv_d = 1.0f / static_cast<float>(p.D);
  for (int h = h0; h < h1; h += U) {
    Vec<T, V> a[U][SL], c[U][SL];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const T* row = x0 + (h + u < h1 ? h + u : h) * t.xs[1];
#pragma unroll
      for (int k = 0; k < SL; ++k) {
        a[u][k] = qk_load<T, V>(row, s[k].ia, s[k].here);
        c[u][k] = qk_load<T, V>(row, s[k].ib, s[k].pair);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float xa[SL][V], xb[SL][V], sum = 0.0f;
#pragma unroll
      for (int k = 0; k < SL; ++k) {
        a[u][k].widen(xa[k]);
        c[u][k].widen(xb[k]);
#pragma unroll
        for (int e = 0; e < V; ++e) sum = fmaf(xa[k][e], xa[k][e], fmaf(xb[k][e], xb[k][e], sum));
      }
      const float r = __frsqrt_rn(fmaf(qk_group_sum(sum, lanes), inv_d, p.eps));
      if (!valid || h + u >= h1) continue;
      T* row = y0 + (h + u) * t.ys[1];
#pragma unroll
      for (int k = 0; k < SL; ++k) {
        float ya[V], yb[V];
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float va = xa[k][e] * r * wa[k][e], vb = xb[k][e] * r * wb[k][e];
          ya[e] = va * cs[k][e] - vb * sn[k][e];
          yb[e] = va * sn[k][e] + vb * cs[k][e];
        }
        Vec<T, V> oa, ob;
        oa.narrow(ya);
        ob.narrow(yb);
        if (s[k].here) *reinterpret_cast<Vec<T, V>*>(row + s[k].ia) = oa;
        if (s[k].pair) *reinterpret_cast<Vec<T, V>*>(row + s[k].ib) = ob;
      }
    }
  }
}

// The gradient.  A block walks over the tokens with a stride of the grid and
// keeps its slice's share of dw in registers: lane sums, then the groups of a
// warp by shuffles, the warps through shared memory, and one row of `part`
// per block that vattn_qk_weight_sum_kernel adds in a fixed order.
template <typename T, int V, int SL>
__global__ void __launch_bounds__(kQkThreads)
    vattn_qk_norm_rope_backward_kernel(const __grid_constant__ QkParams p) {
  constexpr int U = SL == 1 ? 2 : 1;  // rows in flight (two tensors are read)
  __shared__ uint64_t turn[kQkMaxDim / 2];
  __shared__ float red[kQkThreads / 32][kQkMaxDim];
  qk_turns(p, turn);
  const bool is_q = static_cast<int>(blockIdx.y) < p.t[0].slices;
  const QkTensor& t = p.t[is_q ? 0 : 1];
  const int slice = static_cast<int>(blockIdx.y) - (is_q ? 0 : p.t[0].slices);
  const int h0 = slice * t.heads_per_slice;
  const int h1 = min(t.heads, h0 + t.heads_per_slice);
  const int lanes = 1 << p.log_lanes;
  const int c0 = static_cast<int>(threadIdx.x) & (lanes - 1);
  const int groups = kQkThreads >> p.log_lanes;
  const float inv_d = 1.0f / static_cast<float>(p.D);
  QkSlot<V> s[SL];
  float wa[SL][V], wb[SL][V], da[SL][V], db[SL][V];
#pragma unroll
  for (int k = 0; k < SL; ++k) {
    s[k].set(p, c0 + k * lanes);
    qk_weight<V>(s[k], t.w, p.w_f32, Elem<T>::kBf16, wa[k], wb[k]);
#pragma unroll
    for (int e = 0; e < V; ++e) da[k][e] = db[k][e] = 0.0f;
  }
  for (long long first = static_cast<long long>(blockIdx.x) * groups; first < p.tokens;
       first += static_cast<long long>(gridDim.x) * groups) {
    const long long token = first + (threadIdx.x >> p.log_lanes);
    const bool valid = token < p.tokens;
    const long long tk = valid ? token : p.tokens - 1;
    const long long b = tk / p.n, n = tk - b * p.n;
    const long long pos = p.positions != nullptr ? p.positions[tk] : p.pos0 + n;
    float cs[SL][V], sn[SL][V];
#pragma unroll
    for (int k = 0; k < SL; ++k) qk_angles<V>(s[k], turn, c0 + k * lanes, pos, cs[k], sn[k]);
    const T* x0 = static_cast<const T*>(t.x) + b * t.xs[0] + n * t.xs[2];
    const T* g0 = static_cast<const T*>(t.g) + b * t.gs[0] + n * t.gs[2];
    T* y0 = static_cast<T*>(t.y) + b * t.ys[0] + n * t.ys[2];
    for (int h = h0; h < h1; h += U) {
      Vec<T, V> xv[U][SL][2], gv[U][SL][2];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int hh = h + u < h1 ? h + u : h;
#pragma unroll
        for (int k = 0; k < SL; ++k) {
          xv[u][k][0] = qk_load<T, V>(x0 + hh * t.xs[1], s[k].ia, s[k].here);
          xv[u][k][1] = qk_load<T, V>(x0 + hh * t.xs[1], s[k].ib, s[k].pair);
          gv[u][k][0] = qk_load<T, V>(g0 + hh * t.gs[1], s[k].ia, s[k].here);
          gv[u][k][1] = qk_load<T, V>(g0 + hh * t.gs[1], s[k].ib, s[k].pair);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float xa[SL][V], xb[SL][V], ga[SL][V], gb[SL][V];
        float sum = 0.0f, dot = 0.0f;
#pragma unroll
        for (int k = 0; k < SL; ++k) {
          xv[u][k][0].widen(xa[k]);
          xv[u][k][1].widen(xb[k]);
          float fa[V], fb[V];
          gv[u][k][0].widen(fa);
          gv[u][k][1].widen(fb);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            ga[k][e] = fa[e] * cs[k][e] + fb[e] * sn[k][e];
            gb[k][e] = fb[e] * cs[k][e] - fa[e] * sn[k][e];
            sum = fmaf(xa[k][e], xa[k][e], fmaf(xb[k][e], xb[k][e], sum));
            dot = fmaf(ga[k][e] * wa[k][e], xa[k][e], fmaf(gb[k][e] * wb[k][e], xb[k][e], dot));
          }
        }
        sum = qk_group_sum(sum, lanes);
        dot = qk_group_sum(dot, lanes);
        if (!valid || h + u >= h1) continue;
        const float r = __frsqrt_rn(fmaf(sum, inv_d, p.eps));
        const float back = dot * inv_d * r * r;  // times x r: the norm's own share
        T* row = y0 + (h + u) * t.ys[1];
#pragma unroll
        for (int k = 0; k < SL; ++k) {
          float oa[V], ob[V];
#pragma unroll
          for (int e = 0; e < V; ++e) {
            da[k][e] = fmaf(ga[k][e], xa[k][e] * r, da[k][e]);
            db[k][e] = fmaf(gb[k][e], xb[k][e] * r, db[k][e]);
            oa[e] = r * (ga[k][e] * wa[k][e] - xa[k][e] * back);
            ob[e] = r * (gb[k][e] * wb[k][e] - xb[k][e] * back);
          }
          Vec<T, V> va, vb;
          va.narrow(oa);
          vb.narrow(ob);
          if (s[k].here) *reinterpret_cast<Vec<T, V>*>(row + s[k].ia) = va;
          if (s[k].pair) *reinterpret_cast<Vec<T, V>*>(row + s[k].ib) = vb;
        }
      }
    }
  }
  if (p.part == nullptr) return;
  const int warp = static_cast<int>(threadIdx.x) >> 5;
#pragma unroll
  for (int k = 0; k < SL; ++k)
#pragma unroll
    for (int e = 0; e < V; ++e) {
      float a = da[k][e], c = db[k][e];
      for (int o = lanes; o < 32; o <<= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        c += __shfl_xor_sync(0xffffffffu, c, o);
      }
      if ((threadIdx.x & 31) < static_cast<unsigned>(lanes)) {
        if (s[k].here) red[warp][s[k].ia + e] = a;
        if (s[k].pair) red[warp][s[k].ib + e] = c;
      }
    }
  __syncthreads();
  for (int d = threadIdx.x; d < p.D; d += kQkThreads) {
    float a = 0.0f;
#pragma unroll
    for (int w = 0; w < kQkThreads / 32; ++w) a += red[w][d];
    p.part[(static_cast<long long>(blockIdx.y) * gridDim.x + blockIdx.x) * p.D + d] = a;
  }
}

// dw of one tensor (blockIdx.y) in 32 columns (blockIdx.x): the rows of
// `part` in order, 32 interleaved partial sums, then their sum.
struct QkWeightSum {
  const float* part;
  float* dw[2];
  long long row0[2], row1[2];
  int D;
};

__global__ void __launch_bounds__(1024) vattn_qk_weight_sum_kernel(const QkWeightSum p) {
  __shared__ float red[32][33];
  ptx::grid_dep_wait();
  const int which = blockIdx.y;
  const int d = blockIdx.x * 32 + threadIdx.x;
  if (p.dw[which] == nullptr) return;
  float a = 0.0f;
  if (d < p.D)
    for (long long r = p.row0[which] + threadIdx.y; r < p.row1[which]; r += 32) a += p.part[r * p.D + d];
  red[threadIdx.y][threadIdx.x] = a;
  __syncthreads();
  if (threadIdx.y == 0 && d < p.D) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) sum += red[i][threadIdx.x];
    p.dw[which][d] = sum;
  }
}

}  // namespace vattn

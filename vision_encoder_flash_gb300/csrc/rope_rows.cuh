// rope_rows.cuh -- rows under the NeoX rotation, lane by lane: which elements a
// lane holds, and the angles' sines and cosines (qk_norm_rope_kernel.cuh says how
// exact and why).
#pragma once

#include <cstdint>

#include "elem.cuh"

namespace vattn {

constexpr int kQkMaxDim = 128;

// One lane's place in a row: V pairs (a[ia ..], b[ib ..]).
template <int V>
struct QkSlot {
  int ia, ib;
  bool here, pair, rot;
  template <typename P>  // a call's sizes: D, half, slots
  __device__ __forceinline__ void set(const P& p, int c) { set(p.D, p.half, p.slots, c); }
  __device__ __forceinline__ void set(int D, int half, int slots, int c) {
    const int i = c * V, rest = D - 2 * half;
    here = c < slots;
    rot = here && i < half;
    const int r = i - half;
    ia = rot ? i : 2 * half + r;
    ib = rot ? i + half : 2 * half + (rest + 1) / 2 + r;
    pair = here && ib < D;  // V == 1 and an odd rest: the last slot has no partner
  }
};

// The rotation's frequency i as a 64-bit fraction of a turn; factors: null, or divisors.
__host__ __device__ __forceinline__ uint64_t qk_turn(const double* turns, const float* turns_rest, const float* factors, int i) {
  double f = turns[i];
  float rest = turns_rest[i];  // 24 of its digits are enough: f64 arithmetic is slow
  if (factors != nullptr) {
    const float by = factors[i];
    const double q = f / by;
    rest = (static_cast<float>(fma(-q, static_cast<double>(by), f)) + rest) / by;
    f = q;
  }
  // the fractions of both, times 2^64; their sum modulo that
  f -= floor(f);
  rest -= rintf(rest);
  return static_cast<uint64_t>(f * 0x1p64) + static_cast<uint64_t>(static_cast<long long>(rest * 0x1p64f));
}
// sin and cos of a 32-bit fraction of a turn, to 1.3 x 2^-24: quadrant and
// remainder y in [-pi/4, pi/4] from the integer, then sin y = y + y^3 A(y^2) and
// cos y = 1 - y^2/2 + y^4 B(y^2) with A and B of degree 2, the interpolation of
// (sin y / y - 1) / y^2 and (cos y - 1 + y^2/2) / y^4 at the Chebyshev points
// of [0, (pi/4)^2].
__device__ __forceinline__ void qk_sincos(uint32_t phase, float& sn, float& cs) {
  const uint32_t k = (phase + 0x20000000u) >> 30;  // quarter turns
  const float y = static_cast<float>(static_cast<int32_t>(phase - (k << 30))) * 0x1.921fb6p-30f;  // 2 pi / 2^32
  const float z = y * y;
  const float a = fmaf(fmaf(-0.000195878909f, z, 0.00833274797f), z, -0.166666642f);
  const float b = fmaf(fmaf(2.45479423e-05f, z, -0.00138883025f), z, 0.0416666642f);
  const float s = fmaf(y * z, a, y);
  const float c = fmaf(z * z, b, fmaf(-0.5f, z, 1.0f));
  const float s1 = (k & 1u) ? c : s, c1 = (k & 1u) ? s : c;
  sn = (k & 2u) ? -s1 : s1;
  cs = ((k + 1u) & 2u) ? -c1 : c1;
}

template <int V>
__device__ __forceinline__ void qk_angles(const QkSlot<V>& s, const uint64_t* turn, int c,
                                          long long pos, float (&cs)[V], float (&sn)[V]) {
#pragma unroll
  for (int e = 0; e < V; ++e) {
    cs[e] = 1.0f;
    sn[e] = 0.0f;
    if (s.rot) qk_sincos(static_cast<uint32_t>((static_cast<uint64_t>(pos) * turn[c * V + e]) >> 32), sn[e], cs[e]);
  }
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

// d = a * b, d = a * b + c over V lanes' worth, in pairs where V is even.
template <int V>
__device__ __forceinline__ void vmul(float (&d)[V], const float (&a)[V], const float (&b)[V]) {
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int e = 0; e < V; e += 2) {
      const float2 r = __fmul2_rn(make_float2(a[e], a[e + 1]), make_float2(b[e], b[e + 1]));
      d[e] = r.x;
      d[e + 1] = r.y;
    }
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) d[e] = a[e] * b[e];
  }
}
template <int V>
__device__ __forceinline__ void vfma(float (&d)[V], const float (&a)[V], const float (&b)[V], const float (&c)[V]) {
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int e = 0; e < V; e += 2) {
      const float2 r = __ffma2_rn(make_float2(a[e], a[e + 1]), make_float2(b[e], b[e + 1]), make_float2(c[e], c[e + 1]));
      d[e] = r.x;
      d[e + 1] = r.y;
    }
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) d[e] = fmaf(a[e], b[e], c[e]);
  }
}
template <int V>
__device__ __forceinline__ void vscale(float (&d)[V], const float (&a)[V], float b) {
  float bb[V];
#pragma unroll
  for (int e = 0; e < V; ++e) bb[e] = b;
  vmul<V>(d, a, bb);
}

}  // namespace vattn

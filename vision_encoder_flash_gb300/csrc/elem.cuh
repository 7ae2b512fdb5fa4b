// elem.cuh -- the element types of the decoder kernels: loads and stores of
// V consecutive elements (V * size <= 16 bytes, aligned to that), widened to
// f32 and rounded back to nearest even.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace vattn {

template <typename T> struct Elem;
template <> struct Elem<float> {
  static constexpr bool kBf16 = false;
  static __device__ __forceinline__ float widen(float x) { return x; }
  static __device__ __forceinline__ float narrow(float x) { return x; }
};
template <> struct Elem<__half> {
  static constexpr bool kBf16 = false;
  static __device__ __forceinline__ float widen(__half x) { return __half2float(x); }
  static __device__ __forceinline__ __half narrow(float x) { return __float2half_rn(x); }
};
template <> struct Elem<__nv_bfloat16> {
  static constexpr bool kBf16 = true;
  static __device__ __forceinline__ float widen(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ __nv_bfloat16 narrow(float x) { return __float2bfloat16_rn(x); }
};

// Two f32 as a packed pair of 16-bit elements, the first in the low half.
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (sizeof(T) != 2) return 0;
  else {
    union { T h[2]; uint32_t u; } x;
    x.h[0] = Elem<T>::narrow(lo);
    x.h[1] = Elem<T>::narrow(hi);
    return x.u;
  }
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// V elements as one access.
template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  T e[V];
  __device__ __forceinline__ void widen(float (&x)[V]) const {
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = Elem<T>::widen(e[i]);
  }
  __device__ __forceinline__ void narrow(const float (&x)[V]) {
    if constexpr (sizeof(T) == 2 && V % 2 == 0) {  // one conversion for two elements
      uint32_t* w = reinterpret_cast<uint32_t*>(e);
#pragma unroll
      for (int i = 0; i < V / 2; ++i) w[i] = pack2<T>(x[2 * i], x[2 * i + 1]);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) e[i] = Elem<T>::narrow(x[i]);
    }
  }
};

}  // namespace vattn

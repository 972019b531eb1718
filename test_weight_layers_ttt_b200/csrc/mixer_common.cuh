// Device helpers of the token-mixer kernels: loads and stores of V consecutive elements as
// floats, and fast sigmoid / silu.
#pragma once

#include "common.cuh"

namespace ttt {

using bf16 = __nv_bfloat16;

// V consecutive elements in one access (V * sizeof(T) in {2, 4, 8, 16} bytes and aligned to
// that).
template <typename T, int V> struct Pack;
template <> struct Pack<bf16, 1> { using U = unsigned short; };
template <> struct Pack<bf16, 2> { using U = unsigned; };
template <> struct Pack<bf16, 4> { using U = uint2; };
template <> struct Pack<bf16, 8> { using U = uint4; };
template <> struct Pack<float, 1> { using U = unsigned; };
template <> struct Pack<float, 2> { using U = uint2; };
template <> struct Pack<float, 4> { using U = uint4; };

template <typename T, int V>
__device__ __forceinline__ typename Pack<T, V>::U load_raw(const T* p) {
  return *reinterpret_cast<const typename Pack<T, V>::U*>(p);
}

template <typename T, int V>
__device__ __forceinline__ void unpack(const typename Pack<T, V>::U& u, float (&f)[V]) {
  union { typename Pack<T, V>::U u; T t[V]; } x;
  x.u = u;
#pragma unroll
  for (int i = 0; i < V; ++i) f[i] = to_f32(x.t[i]);
}

template <typename T, int V>
__device__ __forceinline__ void load_vec(const T* p, float (&f)[V]) {
  if constexpr (V * sizeof(T) > 16) {   // two 16-byte accesses
    float lo[V / 2], hi[V / 2];
    load_vec<T, V / 2>(p, lo);
    load_vec<T, V / 2>(p + V / 2, hi);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      f[i] = lo[i];
      f[V / 2 + i] = hi[i];
    }
  } else {
    unpack<T, V>(load_raw<T, V>(p), f);
  }
}

template <typename T, int V>
__device__ __forceinline__ void store_vec(T* p, const float (&f)[V]) {
  union { typename Pack<T, V>::U u; T t[V]; } x;
#pragma unroll
  for (int i = 0; i < V; ++i) x.t[i] = from_f32<T>(f[i]);
  *reinterpret_cast<typename Pack<T, V>::U*>(p) = x.u;
}

// sigmoid with the hardware exponential and division (relative error some 1e-7 (1 + |a|)):
// the accurate forms cost more instructions than the memory-bound kernels here have to spare.
__device__ __forceinline__ float fast_sigmoid(float a) {
  return __fdividef(1.0f, 1.0f + __expf(-a));
}

}  // namespace ttt

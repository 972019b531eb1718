// Device helpers of the token-mixer kernels: loads and stores of V consecutive elements as
// floats, and fast sigmoid / silu.
#pragma once

#include "common.cuh"

namespace ttt {

using bf16 = __nv_bfloat16;

// Two-wide fp32: one issue slot for two operations.
using f2 = unsigned long long;
__device__ __forceinline__ f2 pack2(float lo, float hi) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(f2 v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 both(float v) { return pack2(v, v); }

// o = a * b (+ c) for V values, pairwise.
template <int V>
__device__ __forceinline__ void mul_v(float (&o)[V], const float (&a)[V], const float (&b)[V]) {
#pragma unroll
  for (int i = 0; i < V; i += 2) {
    if constexpr (V == 1) o[0] = a[0] * b[0];
    else unpack2(mul2(pack2(a[i], a[i + 1]), pack2(b[i], b[i + 1])), o[i], o[i + 1]);
  }
}
template <int V>
__device__ __forceinline__ void mul_v(float (&o)[V], const float (&a)[V], float b) {
#pragma unroll
  for (int i = 0; i < V; i += 2) {
    if constexpr (V == 1) o[0] = a[0] * b;
    else unpack2(mul2(pack2(a[i], a[i + 1]), both(b)), o[i], o[i + 1]);
  }
}
template <int V>
__device__ __forceinline__ void fma_v(float (&o)[V], const float (&a)[V], const float (&b)[V], const float (&c)[V]) {
#pragma unroll
  for (int i = 0; i < V; i += 2) {
    if constexpr (V == 1) o[0] = fmaf(a[0], b[0], c[0]);
    else unpack2(fma2(pack2(a[i], a[i + 1]), pack2(b[i], b[i + 1]), pack2(c[i], c[i + 1])), o[i], o[i + 1]);
  }
}
template <int V>
__device__ __forceinline__ void fma_v(float (&o)[V], const float (&a)[V], float b, const float (&c)[V]) {
#pragma unroll
  for (int i = 0; i < V; i += 2) {
    if constexpr (V == 1) o[0] = fmaf(a[0], b, c[0]);
    else unpack2(fma2(pack2(a[i], a[i + 1]), both(b), pack2(c[i], c[i + 1])), o[i], o[i + 1]);
  }
}

template <int V>
__device__ __forceinline__ float sum_v(const float (&a)[V]) {
  if constexpr (V == 1) return a[0];
  else if constexpr (V == 2) return a[0] + a[1];
  else {
    float h[V / 2];
#pragma unroll
    for (int i = 0; i < V / 2; i += 2)
      unpack2(add2(pack2(a[i], a[i + 1]), pack2(a[V / 2 + i], a[V / 2 + i + 1])), h[i], h[i + 1]);
    return sum_v<V / 2>(h);
  }
}

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

// The same load where it stands, or zero when `on` is false: the compiler may sink a plain load
// behind the arithmetic it is meant to run under, down to the first use of its value, and a
// load in a branch is waited for where the branch ends.
__device__ __forceinline__ void load_here(const void* p, bool on, unsigned short& u) {
  asm volatile("{\n.reg .pred q;\nsetp.ne.u32 q, %2, 0;\nmov.u16 %0, 0;\n@q ld.global.u16 %0, [%1];\n}"
               : "=h"(u) : "l"(p), "r"((unsigned)on));
}
__device__ __forceinline__ void load_here(const void* p, bool on, unsigned& u) {
  asm volatile("{\n.reg .pred q;\nsetp.ne.u32 q, %2, 0;\nmov.u32 %0, 0;\n@q ld.global.u32 %0, [%1];\n}"
               : "=r"(u) : "l"(p), "r"((unsigned)on));
}
__device__ __forceinline__ void load_here(const void* p, bool on, uint2& u) {
  asm volatile("{\n.reg .pred q;\nsetp.ne.u32 q, %3, 0;\nmov.u32 %0, 0;\nmov.u32 %1, 0;\n"
               "@q ld.global.v2.u32 {%0, %1}, [%2];\n}"
               : "=r"(u.x), "=r"(u.y) : "l"(p), "r"((unsigned)on));
}
__device__ __forceinline__ void load_here(const void* p, bool on, uint4& u) {
  asm volatile("{\n.reg .pred q;\nsetp.ne.u32 q, %5, 0;\nmov.u32 %0, 0;\nmov.u32 %1, 0;\n"
               "mov.u32 %2, 0;\nmov.u32 %3, 0;\n@q ld.global.v4.u32 {%0, %1, %2, %3}, [%4];\n}"
               : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "l"(p), "r"((unsigned)on));
}

// Asynchronous copy of BYTES (4, 8 or 16) bytes to shared memory, or zeros when `on` is false.
template <int BYTES>
__device__ __forceinline__ void copy_async(void* dst, const void* src, bool on) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(
                   (unsigned)__cvta_generic_to_shared(dst)), "l"(src), "n"(BYTES), "r"(on ? BYTES : 0)
               : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits for all but the newest N groups of this thread's copies.
template <int N>
__device__ __forceinline__ void copies_wait_but() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

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

// Two values rounded to bf16 in one instruction.
__device__ __forceinline__ unsigned bf16_pair(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const unsigned*>(&v);
}

template <typename T, int V>
__device__ __forceinline__ void store_vec(T* p, const float (&f)[V]) {
  if constexpr (V * sizeof(T) > 16) {
    float lo[V / 2], hi[V / 2];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      lo[i] = f[i];
      hi[i] = f[V / 2 + i];
    }
    store_vec<T, V / 2>(p, lo);
    store_vec<T, V / 2>(p + V / 2, hi);
    return;
  } else {
    union { typename Pack<T, V>::U u; T t[V]; unsigned w[(V * sizeof(T) + 3) / 4]; } x;
    if constexpr (sizeof(T) == 2 && V > 1) {
#pragma unroll
      for (int i = 0; i < V; i += 2) x.w[i / 2] = bf16_pair(f[i], f[i + 1]);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) x.t[i] = from_f32<T>(f[i]);
    }
    *reinterpret_cast<typename Pack<T, V>::U*>(p) = x.u;
  }
}

// V elements of an input that nothing writes while the kernel runs (the read-only path: later
// loads may pass earlier stores).
__device__ __forceinline__ unsigned short ldg(const unsigned short* p) { return __ldg(p); }
__device__ __forceinline__ unsigned ldg(const unsigned* p) { return __ldg(p); }
__device__ __forceinline__ uint2 ldg(const uint2* p) { return __ldg(p); }
__device__ __forceinline__ uint4 ldg(const uint4* p) { return __ldg(p); }

template <typename T, int V>
__device__ __forceinline__ void load_input(const T* p, float (&f)[V]) {
  if constexpr (V * sizeof(T) > 16) {
    float lo[V / 2], hi[V / 2];
    load_input<T, V / 2>(p, lo);
    load_input<T, V / 2>(p + V / 2, hi);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      f[i] = lo[i];
      f[V / 2 + i] = hi[i];
    }
  } else {
    unpack<T, V>(ldg(reinterpret_cast<const typename Pack<T, V>::U*>(p)), f);
  }
}

// sigmoid with the hardware exponential and reciprocal (relative error some 1e-7 (1 + |a|)): the
// accurate forms cost more instructions than these kernels have to spare. exp(-a) past fp32's
// range gives 1 / inf = 0.
__device__ __forceinline__ float fast_sigmoid(float a) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(a * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return r;
}

}  // namespace ttt

// Activation tensors of the training operators: fp32, fp16 or bf16 storage, fp32 arithmetic.
#pragma once

#include <type_traits>

#include "ma_internal.h"

namespace ma {

// Storage types, numbered as ma_dtype in the C ABI.
enum ActType { kActF32 = 0, kActF16 = 1, kActBF16 = 2 };

template <int T>
struct Act;
template <>
struct Act<kActF32> {
  typedef float S;
  static __device__ __forceinline__ float up(S v) { return v; }
  static __device__ __forceinline__ S down(float v) { return v; }
};
template <>
struct Act<kActF16> {
  typedef unsigned short S;
  static __device__ __forceinline__ float up(S v) { return h2f(v); }
  static __device__ __forceinline__ S down(float v) { return f2h(v); }
};
template <>
struct Act<kActBF16> {
  typedef unsigned short S;
  static __device__ __forceinline__ float up(S v) { return bf2f(v); }
  static __device__ __forceinline__ S down(float v) { return f2bf(v); }
};

// N consecutive values.  The vector type is aligned like one value only: rows of odd length
// or stride start anywhere, and global memory takes wide accesses at any element's address,
// so one kernel serves every layout (measured where it matters, at the kernels).
template <typename S, int N>
struct Pack {
  typedef S type __attribute__((ext_vector_type(N), aligned(sizeof(S))));
};
template <typename S>
struct Pack<S, 1> {
  typedef S type;
};

template <int T, int N>
__device__ __forceinline__ void load_act(const typename Act<T>::S* p, float (&v)[N]) {
  typedef typename Pack<typename Act<T>::S, N>::type P;
  const P x = *reinterpret_cast<const P*>(p);
  if constexpr (N == 1) {
    v[0] = Act<T>::up(x);
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = Act<T>::up(x[e]);
  }
}
template <int T, int N>
__device__ __forceinline__ void store_act(typename Act<T>::S* p, const float (&v)[N]) {
  typedef typename Pack<typename Act<T>::S, N>::type P;
  P x;
  if constexpr (N == 1) {
    x = Act<T>::down(v[0]);
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) x[e] = Act<T>::down(v[e]);
  }
  *reinterpret_cast<P*>(p) = x;
}
// The first n of N values (n in 1..N); the others read as `fill`.
template <int T, int N>
__device__ __forceinline__ void load_part(const typename Act<T>::S* p, int n, float fill,
                                          float (&v)[N]) {
  if (n >= N) {
    load_act<T, N>(p, v);
    return;
  }
#pragma unroll
  for (int e = 0; e < N; ++e) v[e] = e < n ? Act<T>::up(p[e]) : fill;
}
template <int T, int N>
__device__ __forceinline__ void store_part(typename Act<T>::S* p, int n, const float (&v)[N]) {
  if (n >= N) {
    store_act<T, N>(p, v);
    return;
  }
#pragma unroll
  for (int e = 0; e < N; ++e)
    if (e < n) p[e] = Act<T>::down(v[e]);
}

// Calls f with the storage type as a compile-time constant.
template <typename F>
inline hipError_t with_act(int type, F f) {
  switch (type) {
    case kActF32: return f(std::integral_constant<int, kActF32>());
    case kActF16: return f(std::integral_constant<int, kActF16>());
    case kActBF16: return f(std::integral_constant<int, kActBF16>());
  }
  return hipErrorInvalidValue;
}

// Sums over a wave; every lane gets the result.
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor(v, d, 64));
  return v;
}

}  // namespace ma

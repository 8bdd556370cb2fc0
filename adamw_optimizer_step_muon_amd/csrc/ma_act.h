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

// N consecutive values (two at least).  The vector type is aligned like one value only: rows of
// odd length or stride start anywhere, and global memory takes wide accesses at any element's
// address, so one kernel serves every layout (measured where it matters, at the kernels).
template <typename S, int N>
struct Pack {
  typedef S type __attribute__((ext_vector_type(N), aligned(sizeof(S))));
};

template <int T, int N>
__device__ __forceinline__ void load_act(const typename Act<T>::S* p, float (&v)[N]) {
  typedef typename Pack<typename Act<T>::S, N>::type P;
  const P x = *reinterpret_cast<const P*>(p);
#pragma unroll
  for (int e = 0; e < N; ++e) v[e] = Act<T>::up(x[e]);
}
template <int T, int N>
__device__ __forceinline__ void store_act(typename Act<T>::S* p, const float (&v)[N]) {
  typedef typename Pack<typename Act<T>::S, N>::type P;
  P x;
#pragma unroll
  for (int e = 0; e < N; ++e) x[e] = Act<T>::down(v[e]);
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

// Vectors of 16 bytes.
template <int T>
struct Vec {
  typedef typename Act<T>::S S;
  static constexpr int kN = 16 / sizeof(S);
  typedef typename Pack<S, kN>::type P;
};

// The first cnt (any sign) of a vector's values; zeros behind them.
template <int T>
__device__ __forceinline__ typename Vec<T>::P load_raw(const typename Act<T>::S* p, int cnt) {
  typedef typename Vec<T>::P P;
  P x;
  if (cnt >= Vec<T>::kN) {
    x = *reinterpret_cast<const P*>(p);
  } else {
#pragma unroll
    for (int e = 0; e < Vec<T>::kN; ++e) x[e] = e < cnt ? p[e] : 0;
  }
  return x;
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

// Reductions over a wave by data-parallel moves within the vector unit: after quad, half-row
// and row exchanges every lane has its row of 16, the two row broadcasts carry the rows'
// results to lane 63, and every lane gets that lane's value.  Six dependent operations
// without the shared memory's latency.  `fill` is the operation's neutral element.
template <int kCtrl, int kRowMask>
__device__ __forceinline__ float lane_move(float fill, float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, fill), __builtin_bit_cast(int, v),
                                                               kCtrl, kRowMask, 0xf, false));
}
template <typename F>
__device__ __forceinline__ float row16_reduce(float v, float fill, F f) {
  v = f(v, lane_move<0xb1, 0xf>(fill, v));   // quads: lanes 1 0 3 2
  v = f(v, lane_move<0x4e, 0xf>(fill, v));   // quads: lanes 2 3 0 1
  v = f(v, lane_move<0x141, 0xf>(fill, v));  // halves of a row mirrored
  return f(v, lane_move<0x140, 0xf>(fill, v));  // rows mirrored
}
template <typename F>
__device__ __forceinline__ float wave_reduce(float v, float fill, F f) {
  v = row16_reduce(v, fill, f);
  v = f(v, lane_move<0x142, 0xa>(fill, v));  // lane 15 of rows 0 and 2 to rows 1 and 3
  v = f(v, lane_move<0x143, 0xc>(fill, v));  // lane 31 to rows 2 and 3
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), 63));
}
struct Add {
  __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
struct Max {
  __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
__device__ __forceinline__ float wave_sum(float v) { return wave_reduce(v, 0.0f, Add()); }
__device__ __forceinline__ float wave_max(float v) { return wave_reduce(v, -INFINITY, Max()); }

}  // namespace ma

// Rows in registers: what the normalisations over the last dimension share.
#pragma once

#include "ma_act.h"

namespace ma {

template <int N>
__device__ __forceinline__ void load_floats(const float* p, int cnt, float fill, float (&v)[N]) {
  if (cnt >= N) {
#pragma unroll
    for (int e = 0; e < N; e += 4) {
      const Pack<float, 4>::type x = *reinterpret_cast<const Pack<float, 4>::type*>(p + e);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[e + k] = x[k];
    }
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = e < cnt ? p[e] : fill;
  }
}

// The sums of kCount values over the kTPR threads of a row; every thread gets them.
// `shared` holds kCount values per wave of the block; callers alternate between two of them,
// so one barrier a call is enough (every thread of the block makes every call).
template <int kTPR, int kCount>
__device__ __forceinline__ void row_sums(float (&v)[kCount], float* shared) {
#pragma unroll
  for (int k = 0; k < kCount; ++k) {
    if constexpr (kTPR >= 64) {
      v[k] = wave_sum(v[k]);
    } else {
      v[k] = row16_reduce(v[k], 0.0f, Add());
      if (kTPR == 32) v[k] += __shfl_xor(v[k], 16, 64);
    }
  }
  if constexpr (kTPR > 64) {
    constexpr int kW = kTPR / 64;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int k = 0; k < kCount; ++k) shared[wave * kCount + k] = v[k];
    __syncthreads();
    const int first = wave / kW * kW;
#pragma unroll
    for (int k = 0; k < kCount; ++k) {
      v[k] = 0.0f;
#pragma unroll
      for (int w = 0; w < kW; ++w) v[k] += shared[(first + w) * kCount + k];
    }
  }
}

// The row layout for rows of dim values of type T: threads per row and vectors per thread
// (two, so that the backward pass keeps x, dy, the next row's and the column sums in
// registers; four only for the longest fp32 rows); false when the row does not fit.
template <int T, typename F>
bool with_row(int64_t dim, F f) {
  const int64_t v = (dim + Vec<T>::kN - 1) / Vec<T>::kN;
  if (v <= 16) f(std::integral_constant<int, 16>(), std::integral_constant<int, 1>());
  else if (v <= 32) f(std::integral_constant<int, 32>(), std::integral_constant<int, 1>());
  else if (v <= 64) f(std::integral_constant<int, 64>(), std::integral_constant<int, 1>());
  else if (v <= 128) f(std::integral_constant<int, 64>(), std::integral_constant<int, 2>());
  else if (v <= 256) f(std::integral_constant<int, 128>(), std::integral_constant<int, 2>());
  else if (v <= 512) f(std::integral_constant<int, 256>(), std::integral_constant<int, 2>());
  else if (v <= 1024) f(std::integral_constant<int, 512>(), std::integral_constant<int, 2>());
  else if (v <= 2048) f(std::integral_constant<int, 1024>(), std::integral_constant<int, 2>());
  else if (T == kActF32 && v <= 4096) f(std::integral_constant<int, 1024>(), std::integral_constant<int, T == kActF32 ? 4 : 2>());
  else return false;
  return true;
}

}  // namespace ma

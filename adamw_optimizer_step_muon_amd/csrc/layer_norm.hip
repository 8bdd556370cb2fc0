// Layer norm over the last dimension, forward and backward.
//
//   mean = sum x / D,  rstd = 1 / sqrt(sum (x - mean)^2 / D + eps),  h = (x - mean) rstd
//   y = h w + b
//   u = dy w,  dx = rstd (u - sum u / D - h sum (u h) / D)
//   dw (+)= sum over rows of dy h,  db (+)= sum over rows of dy
//
// All arithmetic in fp32; the variance is summed from the deviations, not as E x^2 - mean^2,
// which loses everything where the mean is large.
#include "ma_act.h"
#include "ma_internal.h"

namespace ma {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

__device__ __forceinline__ float block_sum(float v, float* shared) {
  v = wave_sum(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) shared[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0.0f;
  for (int w = 0; w < kWaves; ++w) v += shared[w];
  return v;
}

template <int T>
__global__ __launch_bounds__(kThreads) void norm_kernel(NormCall c) {
  typedef typename Act<T>::S S;
  __shared__ float shared[kWaves];
  const int64_t row = blockIdx.x;
  const S* x = static_cast<const S*>(c.x) + row * c.x_stride;
  S* y = static_cast<S*>(c.y) + row * c.y_stride;
  float sum = 0.0f;
  for (int64_t i = threadIdx.x; i < c.dim; i += kThreads) sum += Act<T>::up(x[i]);
  const float mean = block_sum(sum, shared) / c.dim;
  float sq = 0.0f;
  for (int64_t i = threadIdx.x; i < c.dim; i += kThreads) {
    const float d = Act<T>::up(x[i]) - mean;
    sq += d * d;
  }
  const float rstd = 1.0f / __builtin_sqrtf(block_sum(sq, shared) / c.dim + c.eps);
  if (threadIdx.x == 0) {
    c.mean[row] = mean;
    c.rstd[row] = rstd;
  }
  for (int64_t i = threadIdx.x; i < c.dim; i += kThreads) {
    const float h = (Act<T>::up(x[i]) - mean) * rstd;
    y[i] = Act<T>::down(h * (c.weight ? c.weight[i] : 1.0f) + (c.bias ? c.bias[i] : 0.0f));
  }
}

// dx, one block per row.
template <int T>
__global__ __launch_bounds__(kThreads) void norm_dx_kernel(NormGradCall c) {
  typedef typename Act<T>::S S;
  __shared__ float shared[kWaves];
  const int64_t row = blockIdx.x;
  const S* x = static_cast<const S*>(c.x) + row * c.x_stride;
  const S* dy = static_cast<const S*>(c.dy) + row * c.dy_stride;
  S* dx = static_cast<S*>(c.dx) + row * c.dx_stride;
  const float mean = c.mean[row], rstd = c.rstd[row];
  float s1 = 0.0f, s2 = 0.0f;
  for (int64_t i = threadIdx.x; i < c.dim; i += kThreads) {
    const float u = Act<T>::up(dy[i]) * (c.weight ? c.weight[i] : 1.0f);
    s1 += u;
    s2 += u * ((Act<T>::up(x[i]) - mean) * rstd);
  }
  s1 = block_sum(s1, shared) / c.dim;
  s2 = block_sum(s2, shared) / c.dim;
  for (int64_t i = threadIdx.x; i < c.dim; i += kThreads) {
    const float u = Act<T>::up(dy[i]) * (c.weight ? c.weight[i] : 1.0f);
    const float h = (Act<T>::up(x[i]) - mean) * rstd;
    dx[i] = Act<T>::down(rstd * (u - s1 - h * s2));
  }
}

// Rows of one group of the reduction over rows.
constexpr int64_t kMaxGroups = 256;

// Block (columns, group): partial sums of dy h and dy over the group's rows.
template <int T>
__global__ __launch_bounds__(kThreads) void norm_dw_kernel(NormGradCall c, int64_t per_group) {
  typedef typename Act<T>::S S;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= c.dim) return;
  const int64_t lo = static_cast<int64_t>(blockIdx.y) * per_group;
  const int64_t hi = lo + per_group < c.n ? lo + per_group : c.n;
  float w = 0.0f, b = 0.0f;
  for (int64_t r = lo; r < hi; ++r) {
    const float dy = Act<T>::up((static_cast<const S*>(c.dy) + r * c.dy_stride)[i]);
    const float x = Act<T>::up((static_cast<const S*>(c.x) + r * c.x_stride)[i]);
    w += dy * ((x - c.mean[r]) * c.rstd[r]);
    b += dy;
  }
  c.workspace[(2 * static_cast<int64_t>(blockIdx.y)) * c.dim + i] = w;
  c.workspace[(2 * static_cast<int64_t>(blockIdx.y) + 1) * c.dim + i] = b;
}

__global__ __launch_bounds__(kThreads) void norm_join_kernel(NormGradCall c, int64_t groups) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= c.dim) return;
  float w = 0.0f, b = 0.0f;
  for (int64_t g = 0; g < groups; ++g) {
    w += c.workspace[2 * g * c.dim + i];
    b += c.workspace[(2 * g + 1) * c.dim + i];
  }
  if (c.dweight) c.dweight[i] = c.add ? c.dweight[i] + w : w;
  if (c.dbias) c.dbias[i] = c.add ? c.dbias[i] + b : b;
}

}  // namespace

hipError_t launch_layer_norm_forward(const NormCall& c, hipStream_t s) {
  return with_act(c.type, [&](auto t) {
    hipLaunchKernelGGL((norm_kernel<decltype(t)::value>), dim3(static_cast<unsigned>(c.n)), dim3(kThreads), 0, s, c);
    return hipGetLastError();
  });
}

size_t layer_norm_workspace_bytes(int64_t n, int64_t dim) {
  const int64_t groups = n < kMaxGroups ? n : kMaxGroups;
  return static_cast<size_t>(2 * groups * dim * 4);
}

hipError_t launch_layer_norm_backward(const NormGradCall& c, hipStream_t s) {
  return with_act(c.type, [&](auto t) {
    constexpr int T = decltype(t)::value;
    if (c.n > 0) hipLaunchKernelGGL((norm_dx_kernel<T>), dim3(static_cast<unsigned>(c.n)), dim3(kThreads), 0, s, c);
    if (!c.dweight && !c.dbias) return hipGetLastError();
    const unsigned cols = static_cast<unsigned>((c.dim + kThreads - 1) / kThreads);
    const int64_t groups0 = c.n < kMaxGroups ? c.n : kMaxGroups;
    const int64_t per = c.n > 0 ? (c.n + groups0 - 1) / groups0 : 1, groups = (c.n + per - 1) / per;
    if (groups > 0) hipLaunchKernelGGL((norm_dw_kernel<T>), dim3(cols, static_cast<unsigned>(groups)), dim3(kThreads), 0, s, c, per);
    hipLaunchKernelGGL(norm_join_kernel, dim3(cols), dim3(kThreads), 0, s, c, groups);
    return hipGetLastError();
  });
}

}  // namespace ma

// Distillation from a teacher's top logits: loss and gradient of a row of student logits.
//
// Row of V student logits z, k teacher logits a with their vocabulary ids, temperature tau:
//   p = softmax(a / tau) over the live entries (id in [0, V), a above -inf)
//   q = softmax(z / tau) over the vocabulary
//   loss = tau^2 sum_i p_i (log p_i - log q_id_i)
//   dz_j = weight tau (P q_j - sum of p_i with id_i = j),  P = 1 (0: no live entry, loss 0)
// With m = max z and s = sum exp((z - m) / tau): log q_j = (z_j - m) / tau - log s; the pair
// (m, s) is what the forward pass keeps per row.  One live entry makes this the ordinary
// cross entropy of a label.
//
// A row whose weight is zero gets a zero gradient whatever it holds.  Ids may repeat: their
// probabilities add up.  The gradient may be written over the logits.
#include "ma_act.h"
#include "ma_internal.h"

namespace ma {
namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float block_sum(float v, float* shared) {
  v = wave_sum(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) shared[threadIdx.x >> 6] = v;
  __syncthreads();
  v = 0.0f;
  for (int w = 0; w < kWaves; ++w) v += shared[w];
  return v;
}
__device__ __forceinline__ float block_max(float v, float* shared) {
  v = wave_max(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) shared[threadIdx.x >> 6] = v;
  __syncthreads();
  v = shared[0];
  for (int w = 1; w < kWaves; ++w) v = fmaxf(v, shared[w]);
  return v;
}

__device__ __forceinline__ float teacher_at(const DistillCall& c, int64_t i) {
  switch (c.teacher_type) {
    case kActF16: return h2f(static_cast<const unsigned short*>(c.teacher)[i]);
    case kActBF16: return bf2f(static_cast<const unsigned short*>(c.teacher)[i]);
    default: return static_cast<const float*>(c.teacher)[i];
  }
}

// One block per row.
template <int T, int kMode>
__global__ __launch_bounds__(kThreads) void distill_kernel(DistillCall c) {
  typedef typename Act<T>::S S;
  constexpr bool kLoss = kMode != kDistillBackward, kGrad = kMode != kDistillForward;
  __shared__ float shared[kWaves];
  __shared__ float prob[kMaxDistillTop];
  __shared__ int32_t id[kMaxDistillTop];
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x;
  const S* z = static_cast<const S*>(c.logits) + row * c.stride;
  S* dz = kGrad ? static_cast<S*>(c.dlogits) + row * c.dlogits_stride : nullptr;
  const float weight = kGrad ? c.row_weight[row] : 0.0f;
  const float scale = kLog2e / c.temperature;  // exp((z - m) / tau) = 2^((z - m) scale)

  // the teacher: thread i holds entry i (at most kThreads of them)
  int32_t my_id = -1;
  float a = -INFINITY, my_z = 0.0f;
  if (tid < c.top) {
    const int64_t at = row * c.top + tid;
    const int64_t j = c.id_bits == 64 ? static_cast<const int64_t*>(c.ids)[at]
                                      : static_cast<const int32_t*>(c.ids)[at];
    a = teacher_at(c, at);
    if (j >= 0 && j < c.vocab && a != -INFINITY) {
      my_id = static_cast<int32_t>(j);
      my_z = Act<T>::up(z[j]);
    } else {
      a = -INFINITY;
    }
  }
  const bool live = my_id >= 0;
  const float a_max = block_max(a, shared);
  const float a_exp = live ? __builtin_amdgcn_exp2f((a - a_max) * scale) : 0.0f;
  const float a_sum = block_sum(a_exp, shared);
  const bool some = block_max(live ? 1.0f : 0.0f, shared) > 0.0f;
  const float p = live ? a_exp / a_sum : 0.0f;
  if (tid < c.top) {
    prob[tid] = p;
    id[tid] = my_id;
  }

  float m, s;
  if (kLoss) {
    // maximum and sum of exponentials in one sweep; a thread's start of -FLT_MAX keeps
    // 2^(z - m) defined for rows of -inf, whose sum stays 0 and is reported as NaN below
    float tm = -3.402823466e38f, ts = 0.0f;
    for (int64_t i = tid; i < c.vocab; i += kThreads) {
      const float v = Act<T>::up(z[i]);
      const float nm = fmaxf(tm, v);
      ts = ts * __builtin_amdgcn_exp2f((tm - nm) * scale) + __builtin_amdgcn_exp2f((v - nm) * scale);
      tm = nm;
    }
    m = block_max(tm, shared);
    s = block_sum(ts * __builtin_amdgcn_exp2f((tm - m) * scale), shared);
    if (s == 0.0f) {
      m = -INFINITY;
      s = __builtin_nanf("");
    }
    float term = 0.0f;
    if (p > 0.0f || a_sum != a_sum) {
      const float log_p = ((a - a_max) * scale - __builtin_log2f(a_sum)) * kLn2;
      const float log_q = ((my_z - m) * scale - __builtin_log2f(s)) * kLn2;
      term = live ? p * (log_p - log_q) : 0.0f;
    }
    const float loss = block_sum(term, shared);
    if (tid == 0) {
      c.loss[row] = c.temperature * c.temperature * loss;
      if (c.stats) {
        c.stats[2 * row] = m;
        c.stats[2 * row + 1] = s;
      }
    }
  } else {
    m = c.stats[2 * row];
    s = c.stats[2 * row + 1];
  }
  if (!kGrad) return;
  const float g = weight * c.temperature;
  const float gq = g / s;
  const bool zero = weight == 0.0f || !some;
  for (int64_t i = tid; i < c.vocab; i += kThreads) {
    const float v = zero ? 0.0f : gq * __builtin_amdgcn_exp2f((Act<T>::up(z[i]) - m) * scale);
    dz[i] = Act<T>::down(v);
  }
  if (zero) return;
  __syncthreads();
  // the teacher's entries again, from the logits read before: the first of equal ids writes
  if (live) {
    float sum = 0.0f;
    bool first = true;
    for (int i = 0; i < c.top; ++i)
      if (id[i] == my_id) {
        if (i < tid) first = false;
        sum += prob[i];
      }
    if (first) dz[my_id] = Act<T>::down(gq * __builtin_amdgcn_exp2f((my_z - m) * scale) - g * sum);
  }
}

}  // namespace

hipError_t launch_distill(const DistillCall& c, DistillMode mode, hipStream_t s) {
  return with_act(c.type, [&](auto t) {
    constexpr int T = decltype(t)::value;
    const dim3 grid(static_cast<unsigned>(c.n)), block(kThreads);
    switch (mode) {
      case kDistillForward: hipLaunchKernelGGL((distill_kernel<T, kDistillForward>), grid, block, 0, s, c); break;
      case kDistillBackward: hipLaunchKernelGGL((distill_kernel<T, kDistillBackward>), grid, block, 0, s, c); break;
      case kDistillBoth: hipLaunchKernelGGL((distill_kernel<T, kDistillBoth>), grid, block, 0, s, c); break;
    }
    return hipGetLastError();
  });
}

}  // namespace ma

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

// Every multiply-add here is written out: left to the compiler, the instances of one kernel
// fused differently, and the one-pass call's loss was an ulp off the two calls'.
#pragma clang fp contract(off)

namespace ma {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLowest = -3.402823466e38f;

__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

// Sums of exponentials in powers of two.  A set of values v has a maximum m, and s is the sum
// of 2^(v scale - r) for the reference r = m scale, rounded (reference below; never fused
// with what it is used in, so that everybody has the same r).  v scale - r is one fused
// multiply-add: it rounds by its own size only.  The maximum's own exponent is what r was
// rounded by, half a step of r: up to 1/2 while |r| < 2^24, and beyond what exp2 can hold from
// some 2^31 on.  So rows whose maximum lies beyond +-far = 2^23 / scale take the slower
// (v - m) scale, where r = 0 stands for the difference already taken: rows filled with a mask's
// value, or far above zero.  Other rows' smaller values are taken against -2 far at least, which
// bounds their sums too.  (With the test as >= and -far as that bound, the compiler keeps 15 more
// registers in the one-pass kernels, whose blocks of 1024 threads then have a CU to themselves:
// 439 against 430 us for 4096 x 128000 bf16.)
constexpr float kFarProduct = 8388608.0f;
struct Soft {
  float m, s;
};
__device__ __forceinline__ float reference(float m, float scale) { return m * scale; }
template <bool kIsFar>
__device__ __forceinline__ float exponent(float v, float scale, float m, float r) {
  return kIsFar ? (v - m) * scale : __builtin_fmaf(v, scale, -r);
}
template <bool kIsFar>
__device__ __forceinline__ float between(float from, float to, float scale) {
  return kIsFar ? (from - to) * scale : reference(from, scale) - reference(to, scale);
}
// The lanes' sets joined; every lane gets the result.
template <bool kIsFar>
__device__ __forceinline__ Soft wave_join(Soft v, float scale) {
  const float m = wave_max(v.m);
  return Soft{m, wave_sum(v.s * exp2_(between<kIsFar>(v.m, m, scale)))};
}

__device__ __forceinline__ float teacher_at(const DistillCall& c, int64_t i) {
  switch (c.teacher_type) {
    case kActF16: return h2f(static_cast<const unsigned short*>(c.teacher)[i]);
    case kActBF16: return bf2f(static_cast<const unsigned short*>(c.teacher)[i]);
    default: return static_cast<const float*>(c.teacher)[i];
  }
}

// A thread reads the row in batches of kU vectors of 16 bytes, all loaded before the first is
// used.
constexpr int kU = 4;
template <int T>
constexpr int kVec = Vec<T>::kN;

// What a first sweep keeps of its row for the second one: the last kKeep whole batches in the
// block's shared memory (each thread reads back what it wrote itself) and the rest behind
// them in registers (kNothing: not even that).  Almost no second read hits the L2 (a
// row of 128000 bf16 values is 256 KB, 32 CUs share 4 MB; 1596 MB are read for 4096 rows'
// 1049 MB, of which 49 % are kept), so what is kept is traffic saved.
// One batch of 64 KB lets two blocks of 1024 threads share a CU, one sweeping while the other
// waits: loss and gradient of 4096 x 128000 bf16 took 467 us keeping nothing, 430 us (4.9
// TB/s, the rate of a large copy) with one batch, and 489 us with two, which leave one block.
constexpr int kKeepBatches = 1, kNothing = -1;
template <int T, int kThreads, int kKeep>
struct Kept {
  typedef typename Vec<T>::P P;
  P tail[kKeep >= 0 ? kU : 1];
  P* shared;  // kKeep batches, or null
};

// Maximum and sum of a row; the waves' results go to out.
template <int T, int kThreads, bool kIsFar, int kKeep>
__device__ void sweep(const typename Act<T>::S* z, int vocab, float scale, float far, Soft* out, Kept<T, kThreads, kKeep>& kept) {
  typedef typename Kept<T, kThreads, kKeep>::P P;
  constexpr int N = kVec<T>, kBatch = kThreads * kU * N;
  const int tid = threadIdx.x;
  Soft a{kIsFar ? kLowest : -2.0f * far, 0.0f};  // finite, so that differences to it are defined
  const auto take = [&](const P (&x)[kU], int left) {  // values at and behind `left` count as -inf
    float v[kU][N], m = a.m;
#pragma unroll
    for (int u = 0; u < kU; ++u)
#pragma unroll
      for (int e = 0; e < N; ++e) {
        v[u][e] = Act<T>::up(x[u][e]);
        if (left < kBatch && (u * kThreads + tid) * N + e >= left) v[u][e] = -INFINITY;
        m = fmaxf(m, v[u][e]);
      }
    const float r = reference(m, scale);
    float s[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      s[u] = 0.0f;
#pragma unroll
      for (int e = 0; e < N; ++e) s[u] += exp2_(exponent<kIsFar>(v[u][e], scale, m, r));
    }
    a = Soft{m, a.s * exp2_(between<kIsFar>(a.m, m, scale)) + ((s[0] + s[1]) + (s[2] + s[3]))};
  };
  const int whole = vocab / kBatch;
  for (int b = 0; b < whole; ++b) {
    P x[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) x[u] = *reinterpret_cast<const P*>(z + b * kBatch + (u * kThreads + tid) * N);
    if (kKeep > 0 && b >= whole - kKeep) {
#pragma unroll
      for (int u = 0; u < kU; ++u) kept.shared[((whole - 1 - b) * kU + u) * kThreads + tid] = x[u];
    }
    take(x, kBatch);
  }
  const int left = vocab - whole * kBatch;
  if (left > 0) {
    P x[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int at = (u * kThreads + tid) * N;
      x[u] = load_raw<T>(z + whole * kBatch + at, left - at);
      if constexpr (kKeep >= 0) kept.tail[u] = x[u];
    }
    take(x, left);
  }
  a = wave_join<kIsFar>(a, scale);
  if ((tid & 63) == 0) out[tid >> 6] = a;
}

// The waves' results joined, one a lane.
template <int kThreads, bool kIsFar>
__device__ Soft block_join(const Soft* of, float scale, float far) {
  const int lane = threadIdx.x & 63;
  return wave_join<kIsFar>(lane < kThreads / 64 ? of[lane] : Soft{kIsFar ? kLowest : -2.0f * far, 0.0f}, scale);
}

// dz = gq 2^exponent over the row, from its end to its beginning: what the first sweep kept,
// or read last, comes first.  Non-temporal stores: dz is not read here, and what it leaves of
// the cache is the logits' (500 -> 462 us for 4096 x 128000 bf16).
template <int T, int kThreads, bool kIsFar, int kKeep>
__device__ void spread(const typename Act<T>::S* z, typename Act<T>::S* dz, int vocab, float scale, float m,
                       float r, float gq, const Kept<T, kThreads, kKeep>& kept) {
  typedef typename Kept<T, kThreads, kKeep>::P P;
  constexpr int N = kVec<T>, kBatch = kThreads * kU * N;
  const int tid = threadIdx.x;
  const auto give = [&](int at, const P& x) {
    P d;
#pragma unroll
    for (int e = 0; e < N; ++e)
      d[e] = Act<T>::down(gq * exp2_(exponent<kIsFar>(Act<T>::up(x[e]), scale, m, r)));
    if (vocab - at >= N) {
      __builtin_nontemporal_store(d, reinterpret_cast<P*>(dz + at));
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (e < vocab - at) dz[at + e] = d[e];
    }
  };
  const int whole = vocab / kBatch;
  const int left = vocab - whole * kBatch;
  if (left > 0) {
    P x[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int at = (u * kThreads + tid) * N;
      if constexpr (kKeep >= 0) x[u] = kept.tail[u];
      else x[u] = load_raw<T>(z + whole * kBatch + at, left - at);
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int at = (u * kThreads + tid) * N;
      if (at < left) give(whole * kBatch + at, x[u]);
    }
  }
  for (int b = whole - 1; b >= 0; --b) {
    P x[kU];
    if (kKeep > 0 && b >= whole - kKeep) {
#pragma unroll
      for (int u = 0; u < kU; ++u) x[u] = kept.shared[((whole - 1 - b) * kU + u) * kThreads + tid];
    } else {
#pragma unroll
      for (int u = 0; u < kU; ++u) x[u] = *reinterpret_cast<const P*>(z + b * kBatch + (u * kThreads + tid) * N);
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) give(b * kBatch + (u * kThreads + tid) * N, x[u]);
  }
}

// One block per row: a sweep for maximum and sum (forward, both), a sweep for the gradient
// (backward, both).  A thread holds up to kPer of the teacher's entries.
template <int T, int kMode, int kThreads, int kPer, int kKeep>
__global__ __launch_bounds__(kThreads) void distill_kernel(DistillCall c) {
  typedef typename Act<T>::S S;
  constexpr int N = kVec<T>, kWaves = kThreads / 64;
  constexpr bool kLoss = kMode != kDistillBackward, kGrad = kMode != kDistillForward;
  __shared__ Soft joined[2][kWaves];
  __shared__ float terms[kWaves];
  __shared__ float counts[kWaves];
  __shared__ float prob[kThreads * kPer];
  __shared__ int32_t id[kThreads * kPer];
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, top = static_cast<int>(c.top);
  const S* z = static_cast<const S*>(c.logits) + row * c.stride;
  S* dz = kGrad ? static_cast<S*>(c.dlogits) + row * c.dlogits_stride : nullptr;
  const float weight = kGrad ? c.row_weight[row] : 0.0f;
  const float scale = kLog2e / c.temperature;  // exp((v - m) / tau) = 2^((v - m) scale)
  const int vocab = static_cast<int>(c.vocab);

  // the teacher's entries and the logits at their places
  int32_t my_id[kPer];
  float a[kPer], my_z[kPer];
  Soft ta{kLowest, 0.0f};
  int live = 0;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int i = k * kThreads + tid;
    my_id[k] = -1;
    my_z[k] = a[k] = 0.0f;
    if (i >= top) continue;
    const int64_t at = row * c.top + i;
    const int64_t j = c.id_bits == 64 ? static_cast<const int64_t*>(c.ids)[at]
                                      : static_cast<const int32_t*>(c.ids)[at];
    a[k] = teacher_at(c, at);
    if (j < 0 || j >= c.vocab || a[k] == -INFINITY) continue;
    my_id[k] = static_cast<int32_t>(j);
    my_z[k] = Act<T>::up(z[j]);
    ++live;
    const float m = fmaxf(ta.m, a[k]);
    ta = Soft{m, ta.s * exp2_(between<true>(ta.m, m, scale)) + exp2_(exponent<true>(a[k], scale, m, 0.0f))};
  }

  Kept<T, kThreads, kKeep> kept;
  kept.shared = nullptr;
  if constexpr (kKeep > 0) {
    __shared__ typename Kept<T, kThreads, kKeep>::P room[kKeep * kU * kThreads];
    kept.shared = room;
  }
  Soft zs{0.0f, 0.0f};
  if (kLoss) sweep<T, kThreads, false, kKeep>(z, vocab, scale, c.far, joined[0], kept);
  ta = wave_join<true>(ta, scale);
  const float lives = wave_sum(static_cast<float>(live));
  if (lane == 0) {
    joined[1][wave] = ta;
    counts[wave] = lives;
  }
  __syncthreads();
  if (kLoss) {
    zs = block_join<kThreads, false>(joined[0], scale, c.far);
    if (fabsf(zs.m) > c.far) {  // the same for every thread
      __syncthreads();
      sweep<T, kThreads, true, kKeep>(z, vocab, scale, c.far, joined[0], kept);
      __syncthreads();
      zs = block_join<kThreads, true>(joined[0], scale, c.far);
      if (zs.s == 0.0f) zs = Soft{-INFINITY, __builtin_nanf("")};  // nothing above -inf
    } else {
      // from the rounded reference to the maximum itself
      zs.s *= exp2_(-exponent<false>(zs.m, scale, zs.m, reference(zs.m, scale)));
    }
  } else {
    zs = Soft{c.stats[2 * row], c.stats[2 * row + 1]};
  }
  ta = block_join<kThreads, true>(joined[1], scale, c.far);
  const bool some = wave_sum(lane < kWaves ? counts[lane] : 0.0f) > 0.0f;
  // q = 2^(exponent(v) - zc) / zs.s, zc the maximum's own exponent
  const bool far = fabsf(zs.m) > c.far;
  const float zr = far ? 0.0f : reference(zs.m, scale);
  const float zc = far ? 0.0f : exponent<false>(zs.m, scale, zs.m, zr);
  const auto power_of = [&](float v) {
    return far ? exponent<true>(v, scale, zs.m, zr) : exponent<false>(v, scale, zs.m, zr);
  };

  float p[kPer], term = 0.0f;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    p[k] = my_id[k] >= 0 ? exp2_(exponent<true>(a[k], scale, ta.m, 0.0f)) / ta.s : 0.0f;
    if (kLoss && p[k] != 0.0f) {  // NaN included
      const float log2_p = exponent<true>(a[k], scale, ta.m, 0.0f) - __builtin_log2f(ta.s);
      const float log2_q = power_of(my_z[k]) - zc - __builtin_log2f(zs.s);
      term += p[k] * (log2_p - log2_q);
    }
    const int i = k * kThreads + tid;
    if (kGrad && i < top) {
      prob[i] = p[k];
      id[i] = my_id[k];
    }
  }
  if (kLoss) {
    term = wave_sum(term);
    if (lane == 0) terms[wave] = term;
  }
  __syncthreads();
  if (kLoss && tid == 0) {
    float sum = 0.0f;
    for (int w = 0; w < kWaves; ++w) sum += terms[w];
    c.loss[row] = c.temperature * c.temperature / kLog2e * sum;
    if (c.stats) {
      c.stats[2 * row] = zs.m;
      c.stats[2 * row + 1] = zs.s;
    }
  }
  if (!kGrad) return;

  const float g = weight * c.temperature, gq = g / zs.s * exp2_(-zc);
  if (weight == 0.0f || !some) {
    const float d[N] = {};
    for (int at = tid * N; at < vocab; at += kThreads * N) store_part<T, N>(dz + at, vocab - at, d);
    return;
  }
  if (far) spread<T, kThreads, true, kKeep>(z, dz, vocab, scale, zs.m, zr, gq, kept);
  else spread<T, kThreads, false, kKeep>(z, dz, vocab, scale, zs.m, zr, gq, kept);
  // the teacher's entries again, from the logits read before: the first of equal ids writes,
  // after the sweep's stores
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    if (my_id[k] < 0) continue;
    const int mine = k * kThreads + tid;
    float sum = 0.0f;
    bool first = true;
    for (int i = 0; i < top; ++i)
      if (id[i] == my_id[k]) {
        if (i < mine) first = false;
        sum += prob[i];
      }
    if (first) dz[my_id[k]] = Act<T>::down(gq * exp2_(power_of(my_z[k])) - g * sum);
  }
}

template <int T, int kThreads, int kPer>
void launch_rows(const DistillCall& c, DistillMode mode, hipStream_t s) {
  constexpr int kKeep = kThreads == 1024 ? kKeepBatches : 0;
  const dim3 grid(static_cast<unsigned>(c.n)), block(kThreads);
  switch (mode) {
    case kDistillForward: hipLaunchKernelGGL((distill_kernel<T, kDistillForward, kThreads, kPer, kNothing>), grid, block, 0, s, c); break;
    case kDistillBackward: hipLaunchKernelGGL((distill_kernel<T, kDistillBackward, kThreads, kPer, kNothing>), grid, block, 0, s, c); break;
    case kDistillBoth: hipLaunchKernelGGL((distill_kernel<T, kDistillBoth, kThreads, kPer, kKeep>), grid, block, 0, s, c); break;
  }
}

}  // namespace

hipError_t launch_distill(const DistillCall& call, DistillMode mode, hipStream_t s) {
  DistillCall c = call;
  c.far = kFarProduct / (kLog2e / c.temperature);
  return with_act(c.type, [&](auto t) {
    constexpr int T = decltype(t)::value;
    // as few threads as read the row in one batch and hold the teacher's entries: short rows
    // spend their time on the way between load, join and store, so more of them at once helps
    // (16384 rows of 1000 bf16 logits and 50 teacher entries, loss and gradient: 37 us with 64
    // threads a row, 72 us with 256; 16384 x 16000: 220 us with 512, 361 us with 1024)
    const int64_t batch = kU * kVec<T>;  // a thread's
    if (c.vocab <= 64 * batch && c.top <= 64) launch_rows<T, 64, 1>(c, mode, s);
    else if (c.vocab <= 256 * batch && c.top <= 256) launch_rows<T, 256, 1>(c, mode, s);
    else if (c.vocab <= 256 * batch) launch_rows<T, 256, kMaxDistillTop / 256>(c, mode, s);
    else if (c.vocab <= 512 * batch) launch_rows<T, 512, kMaxDistillTop / 512>(c, mode, s);
    else launch_rows<T, 1024, 1>(c, mode, s);
    return hipGetLastError();
  });
}

}  // namespace ma

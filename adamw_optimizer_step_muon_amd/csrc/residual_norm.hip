// The norms after and before a block, with the block's gate and residual scale, in one pass.
//
//   b = (x - mean1) rstd1 w1 + b1          the block's output x, normalised (or b = x)
//   out = residual + scale gate b
//   y = (out - mean2) rstd2 w2 + b2        what the next block reads
// with mean the row's mean, or 0 (root mean square), and rstd = 1 / sqrt(mean square deviation +
// eps).  y is made of out before that is rounded to its type.
//
// Backward, from dout and dy, with h1 and h2 the normalised rows and
// N(u, h, rstd) = rstd (u - mean u - h mean(u h)), without its mean u for root mean squares:
//   d = dout + N(dy w2, h2, rstd2)         the residual's gradient
//   dx = N(d scale gate w1, h1, rstd1)     (or d scale gate)
//   dw2 = sum dy h2, db2 = sum dy
//   dw1 = scale gate S, db1 = scale gate R, dgate = scale (w1 S + b1 R)
// with S = sum d h1 and R = sum d over the rows: two column sums stand for three gradients.
//
// Memory-bound: four streams forward (x, residual in; out, y out), six backward.  Rows are held in
// registers between their sums, as in layer norm, with the next row's loads issued before this
// row's sums are joined; scale, gate, w1 and b1 enter as two vectors.  Measured, bf16: 32768 rows of
// 2048 111 us (4.8 TB/s); gradients of 16384 rows of 8192 300 us (5.4 TB/s; 8 of them join the column
// sums).  Calls of few rows are bound by their latency: gradients of 1023 rows of 1280, fp32, 13 us and 5
// for the join, 8 rows of 768 forward 5 us.
#include "ma_act.h"
#include "ma_internal.h"
#include "row_norm.h"

namespace ma {
namespace {

constexpr int kThreads = 256;

// scale gate w1 and scale gate b1 of N columns from `at` on (cnt of them are there).
template <int N>
__device__ __forceinline__ void load_branch(const ResidualGains& g, int at, int cnt, float (&a)[N], float (&b)[N]) {
#pragma unroll
  for (int e = 0; e < N; ++e) a[e] = 1.0f;
  if (g.gate) load_floats<N>(g.gate + at, cnt, 0.0f, a);
  float w[N];
#pragma unroll
  for (int e = 0; e < N; ++e) {
    a[e] *= g.scale;
    b[e] = 0.0f;
    w[e] = 1.0f;
  }
  if (g.post_bias) {
    load_floats<N>(g.post_bias + at, cnt, 0.0f, b);
#pragma unroll
    for (int e = 0; e < N; ++e) b[e] *= a[e];
  }
  if (g.post_weight) load_floats<N>(g.post_weight + at, cnt, 0.0f, w);
#pragma unroll
  for (int e = 0; e < N; ++e) a[e] *= w[e];
}
template <int N>
__device__ __forceinline__ void load_next(const ResidualGains& g, int at, int cnt, float (&w)[N], float (&b)[N]) {
#pragma unroll
  for (int e = 0; e < N; ++e) {
    w[e] = 1.0f;
    b[e] = 0.0f;
  }
  if (g.weight) load_floats<N>(g.weight + at, cnt, 0.0f, w);
  if (g.bias) load_floats<N>(g.bias + at, cnt, 0.0f, b);
}

template <int T, int kTPR, int kNV, int kBlock>
__global__ __launch_bounds__(kBlock) void residual_rows_kernel(ResidualCall c) {
  typedef typename Act<T>::S S;
  typedef typename Vec<T>::P P;
  constexpr int N = Vec<T>::kN, kRows = kBlock / kTPR;
  // 1024 threads have 128 registers each: their gains are read again for every row
  constexpr bool kLean = kTPR == 1024;
  __shared__ float shared[2][kBlock / 64];
  const int t = threadIdx.x % kTPR, sub = threadIdx.x / kTPR;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
  int64_t base = static_cast<int64_t>(blockIdx.x) * kRows;
  const S* x0 = static_cast<const S*>(c.x) + t * N;
  const S* r0 = static_cast<const S*>(c.residual) + t * N;
  int cnt[kNV];
  float a1[kNV][N], c1[kNV][N], a2[kNV][N], c2[kNV][N];
  P nx[kNV], nr[kNV];
  const auto load_rows = [&](int64_t row) {
#pragma unroll
    for (int v = 0; v < kNV; ++v) {
      nx[v] = load_raw<T>(x0 + row * c.x_stride + v * kTPR * N, cnt[v]);
      nr[v] = load_raw<T>(r0 + row * c.residual_stride + v * kTPR * N, cnt[v]);
    }
  };
#pragma unroll
  for (int v = 0; v < kNV; ++v) cnt[v] = static_cast<int>(c.dim) - (v * kTPR + t) * N;
  if (base + sub < c.n) load_rows(base + sub);
  if constexpr (!kLean) {
#pragma unroll
    for (int v = 0; v < kNV; ++v) {
      load_branch<N>(c.g, (v * kTPR + t) * N, cnt[v], a1[v], c1[v]);
      load_next<N>(c.g, (v * kTPR + t) * N, cnt[v], a2[v], c2[v]);
    }
  }
  const float dim = static_cast<float>(c.dim);
  int turn = 0;
  // (mean, 1 / deviation) of the row in z; every thread of the block takes part
  const auto statistics = [&](const float (&z)[kNV][N], float& mean, float& rstd) {
    mean = 0.0f;
    if (c.g.center) {
      float sum[1] = {0.0f};
#pragma unroll
      for (int v = 0; v < kNV; ++v)
#pragma unroll
        for (int e = 0; e < N; ++e) sum[0] += z[v][e];
      row_sums<kTPR>(sum, shared[turn]);
      turn ^= 1;
      mean = sum[0] / dim;
    }
    float sq[1] = {0.0f};
#pragma unroll
    for (int v = 0; v < kNV; ++v)
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float d = e < cnt[v] ? z[v][e] - mean : 0.0f;
        sq[0] += d * d;
      }
    row_sums<kTPR>(sq, shared[turn]);
    turn ^= 1;
    rstd = 1.0f / __builtin_sqrtf(sq[0] / dim + c.g.eps);
  };
  for (; base < c.n; base += step) {  // the same trips for every thread of the block
    const int64_t row = base + sub;
    float x[kNV][N], r[kNV][N];
#pragma unroll
    for (int v = 0; v < kNV; ++v)
#pragma unroll
      for (int e = 0; e < N; ++e) {
        x[v][e] = Act<T>::up(nx[v][e]);
        r[v][e] = Act<T>::up(nr[v][e]);
      }
    if (row + step < c.n) load_rows(row + step);
    float mean1 = 0.0f, rstd1 = 0.0f, mean2, rstd2;
    if (c.g.post) statistics(x, mean1, rstd1);
    const float by = c.g.post ? rstd1 : 1.0f;
#pragma unroll
    for (int v = 0; v < kNV; ++v) {
      if constexpr (kLean) load_branch<N>(c.g, (v * kTPR + t) * N, cnt[v], a1[0], c1[0]);
      constexpr int k = 0;
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float a = kLean ? a1[k][e] : a1[v][e], b = kLean ? c1[k][e] : c1[v][e];
        // behind the row's end everything stays zero
        r[v][e] = e < cnt[v] ? r[v][e] + ((x[v][e] - mean1) * by * a + b) : 0.0f;
      }
    }
    statistics(r, mean2, rstd2);
    if (row >= c.n) continue;
    if (t == 0) {
      c.stats[row] = mean1;
      c.stats[c.n + row] = rstd1;
      c.stats[2 * c.n + row] = mean2;
      c.stats[3 * c.n + row] = rstd2;
    }
#pragma unroll
    for (int v = 0; v < kNV; ++v) {
      if (cnt[v] <= 0) continue;
      if constexpr (kLean) load_next<N>(c.g, (v * kTPR + t) * N, cnt[v], a2[0], c2[0]);
      const int64_t at = (v * kTPR + t) * N;
      store_part<T, N>(static_cast<S*>(c.out) + row * c.out_stride + at, cnt[v], r[v]);
      float y[N];
#pragma unroll
      for (int e = 0; e < N; ++e)
        y[e] = (r[v][e] - mean2) * rstd2 * (kLean ? a2[0][e] : a2[v][e]) + (kLean ? c2[0][e] : c2[v][e]);
      store_part<T, N>(static_cast<S*>(c.y) + row * c.y_stride + at, cnt[v], y);
    }
  }
}

// Backward with the four rows in registers, and the block's share of the column sums, which the
// threads that own the columns add up over the block's rows: sum dy h2 and sum d h1 and, with
// kBias, sum dy and sum d.
template <int T, int kTPR, int kNV, int kBlock, bool kBias>
__global__ __launch_bounds__(kBlock) void residual_grad_kernel(ResidualGradCall c) {
  typedef typename Act<T>::S S;
  typedef typename Vec<T>::P P;
  constexpr int N = Vec<T>::kN, kRows = kBlock / kTPR, kCols = kBias ? 4 : 2;
  // 1024 threads have 128 registers each: gains are read again for every row, and the next row's
  // loads wait
  constexpr bool kLean = kTPR == 1024;
  __shared__ float shared[2][2 * (kBlock / 64)];
  __shared__ float join[kRows > 1 ? kTPR * kNV * N : 1];
  const int t = threadIdx.x % kTPR, sub = threadIdx.x / kTPR;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
  int64_t base = static_cast<int64_t>(blockIdx.x) * kRows;
  const S* in[4] = {static_cast<const S*>(c.dout), static_cast<const S*>(c.dy), static_cast<const S*>(c.x),
                    static_cast<const S*>(c.out)};
  const int64_t stride[4] = {c.dout_stride, c.dy_stride, c.x_stride, c.out_stride};
  int cnt[kNV];
  float col[kCols][kNV][N];
#pragma unroll
  for (int v = 0; v < kNV; ++v) {
    cnt[v] = static_cast<int>(c.dim) - (v * kTPR + t) * N;
#pragma unroll
    for (int k = 0; k < kCols; ++k)
#pragma unroll
      for (int e = 0; e < N; ++e) col[k][v][e] = 0.0f;
  }
  const auto load_rows = [&](int64_t row, P (&z)[4][kNV]) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int v = 0; v < kNV; ++v) {
        if (k == 0 && !in[0]) z[k][v] = 0;
        else z[k][v] = load_raw<T>(in[k] + row * stride[k] + (v * kTPR + t) * N, cnt[v]);
      }
  };
  const auto load_a1 = [&](int v, float (&a)[N]) {
    float b[N];
    load_branch<N>(c.g, (v * kTPR + t) * N, cnt[v], a, b);
  };
  const auto load_a2 = [&](int v, float (&a)[N]) {
#pragma unroll
    for (int e = 0; e < N; ++e) a[e] = 1.0f;
    if (c.g.weight) load_floats<N>(c.g.weight + (v * kTPR + t) * N, cnt[v], 0.0f, a);
  };
  const float dim = static_cast<float>(c.dim);
  float a1[kLean ? 1 : kNV][N], a2[kLean ? 1 : kNV][N];
  P next[4][kNV];
  float stats[4], next_stats[4];
  const auto load_stats = [&](int64_t row, float (&s)[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) s[k] = c.stats[k * c.n + row];
  };
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    next_stats[k] = 0.0f;
#pragma unroll
    for (int v = 0; v < kNV; ++v) next[k][v] = 0;
  }
  if constexpr (!kLean) {
#pragma unroll
    for (int v = 0; v < kNV; ++v) {
      load_a1(v, a1[v]);
      load_a2(v, a2[v]);
    }
    if (base + sub < c.n) {
      load_rows(base + sub, next);
      load_stats(base + sub, next_stats);
    }
  }
  int turn = 0;
  for (; base < c.n; base += step) {  // the same trips for every thread of the block
    const int64_t row = base + sub;
    const bool live = row < c.n;
    P z[4][kNV];
    if constexpr (kLean) {  // one row a block
      load_rows(row, z);
      load_stats(row, stats);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        stats[k] = next_stats[k];
#pragma unroll
        for (int v = 0; v < kNV; ++v) z[k][v] = next[k][v];
      }
      if (row + step < c.n) {
        load_rows(row + step, next);
        load_stats(row + step, next_stats);
      }
    }
    const float mean1 = stats[0], rstd1 = stats[1], mean2 = stats[2], rstd2 = stats[3];
    float s[2] = {0.0f, 0.0f};
    if (live) {
#pragma unroll
      for (int v = 0; v < kNV; ++v) {
        if constexpr (kLean) load_a2(v, a2[0]);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          // behind the row's end dy is zero, so nothing is added
          const float g = Act<T>::up(z[1][v][e]), h = (Act<T>::up(z[3][v][e]) - mean2) * rstd2;
          const float u = g * a2[kLean ? 0 : v][e];
          s[0] += u;
          s[1] += u * h;
          col[0][v][e] += g * h;
          if constexpr (kBias) col[2][v][e] += g;
        }
      }
    }
    row_sums<kTPR>(s, shared[turn]);
    turn ^= 1;
    const float m1 = c.g.center ? s[0] / dim : 0.0f, m2 = s[1] / dim;
    float d[kNV][N];
    float q[2] = {0.0f, 0.0f};
#pragma unroll
    for (int v = 0; v < kNV; ++v) {
      if constexpr (kLean) {
        load_a2(v, a2[0]);
        load_a1(v, a1[0]);
      }
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float h2 = (Act<T>::up(z[3][v][e]) - mean2) * rstd2;
        const float u2 = Act<T>::up(z[1][v][e]) * a2[kLean ? 0 : v][e];
        d[v][e] = e < cnt[v] && live ? Act<T>::up(z[0][v][e]) + rstd2 * (u2 - m1 - h2 * m2) : 0.0f;
        const float x = Act<T>::up(z[2][v][e]), h1 = c.g.post ? (x - mean1) * rstd1 : x;
        const float u1 = d[v][e] * a1[kLean ? 0 : v][e];
        q[0] += u1;
        q[1] += u1 * h1;
        // (a row behind the last has d = 0, and x = 0)
        col[1][v][e] += d[v][e] * h1;
        if constexpr (kBias) col[3][v][e] += d[v][e];
      }
    }
    if (c.g.post) {  // the same for every thread of the grid
      row_sums<kTPR>(q, shared[turn]);
      turn ^= 1;
    }
    if (!live) continue;
    const float n1 = c.g.center ? q[0] / dim : 0.0f, n2 = q[1] / dim;
#pragma unroll
    for (int v = 0; v < kNV; ++v) {
      if (cnt[v] <= 0) continue;
      if constexpr (kLean) load_a1(v, a1[0]);
      const int64_t at = (v * kTPR + t) * N;
      store_part<T, N>(static_cast<S*>(c.dresidual) + row * c.dresidual_stride + at, cnt[v], d[v]);
      float dx[N];
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float u1 = d[v][e] * a1[kLean ? 0 : v][e];
        dx[e] = u1;
        if (c.g.post) dx[e] = rstd1 * (u1 - n1 - (Act<T>::up(z[2][v][e]) - mean1) * rstd1 * n2);
      }
      store_part<T, N>(static_cast<S*>(c.dx) + row * c.dx_stride + at, cnt[v], dx);
    }
  }
  if (!c.reduce) return;
  float* part = c.workspace + static_cast<int64_t>(blockIdx.x) * kCols * c.dim;
#pragma unroll
  for (int k = 0; k < kCols; ++k) {
    // the block's rows' sums: waves that share columns add theirs in order
    if constexpr (kRows > 1) {
      __syncthreads();
      for (int w = 0; w < kRows; ++w) {
        if (sub == w) {
#pragma unroll
          for (int v = 0; v < kNV; ++v)
#pragma unroll
            for (int e = 0; e < N; ++e) {
              float* j = join + (v * N + e) * kTPR + t;
              if (w > 0) col[k][v][e] += *j;
              *j = col[k][v][e];
            }
        }
        __syncthreads();
      }
      if (sub != kRows - 1) continue;
    }
#pragma unroll
    for (int v = 0; v < kNV; ++v)
      if (cnt[v] > 0) store_part<kActF32, N>(part + k * c.dim + (v * kTPR + t) * N, cnt[v], col[k][v]);
  }
}

// ---------------------------------------------------------------------------
// Rows too long for the registers of 1024 threads: several sweeps, a value at a time.
// ---------------------------------------------------------------------------
template <int kCount>
__device__ __forceinline__ void block_sums(float (&v)[kCount], float* shared) {
  constexpr int kWaves = kThreads / 64;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kCount; ++k) {
    v[k] = wave_sum(v[k]);
    if ((threadIdx.x & 63) == 0) shared[(threadIdx.x >> 6) * kCount + k] = v[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kCount; ++k) {
    v[k] = 0.0f;
    for (int w = 0; w < kWaves; ++w) v[k] += shared[w * kCount + k];
  }
}
__device__ __forceinline__ void branch_at(const ResidualGains& g, int64_t i, float& a, float& b) {
  const float gate = g.scale * (g.gate ? g.gate[i] : 1.0f);
  a = gate * (g.post_weight ? g.post_weight[i] : 1.0f);
  b = g.post_bias ? gate * g.post_bias[i] : 0.0f;
}

template <int T>
__global__ __launch_bounds__(kThreads) void residual_kernel(ResidualCall c) {
  typedef typename Act<T>::S S;
  __shared__ float shared[kThreads / 64];
  const int64_t row = blockIdx.x;
  const S* x = static_cast<const S*>(c.x) + row * c.x_stride;
  const S* r = static_cast<const S*>(c.residual) + row * c.residual_stride;
  S* out = static_cast<S*>(c.out) + row * c.out_stride;
  S* y = static_cast<S*>(c.y) + row * c.y_stride;
  const auto statistics = [&](auto value, float& mean, float& rstd) {
    mean = 0.0f;
    if (c.g.center) {
      float sum[1] = {0.0f};
      for (int64_t i = threadIdx.x; i < c.dim; i += kThreads) sum[0] += value(i);
      block_sums(sum, shared);
      mean = sum[0] / c.dim;
    }
    float sq[1] = {0.0f};
    for (int64_t i = threadIdx.x; i < c.dim; i += kThreads) {
      const float d = value(i) - mean;
      sq[0] += d * d;
    }
    block_sums(sq, shared);
    rstd = 1.0f / __builtin_sqrtf(sq[0] / c.dim + c.g.eps);
  };
  float mean1 = 0.0f, rstd1 = 0.0f, mean2, rstd2;
  if (c.g.post) statistics([&](int64_t i) { return Act<T>::up(x[i]); }, mean1, rstd1);
  const float by = c.g.post ? rstd1 : 1.0f;
  const auto sum_at = [&](int64_t i) {
    float a, b;
    branch_at(c.g, i, a, b);
    return Act<T>::up(r[i]) + ((Act<T>::up(x[i]) - mean1) * by * a + b);
  };
  statistics(sum_at, mean2, rstd2);
  if (threadIdx.x == 0) {
    c.stats[row] = mean1;
    c.stats[c.n + row] = rstd1;
    c.stats[2 * c.n + row] = mean2;
    c.stats[3 * c.n + row] = rstd2;
  }
  for (int64_t i = threadIdx.x; i < c.dim; i += kThreads) {
    const float s = sum_at(i);
    out[i] = Act<T>::down(s);
    y[i] = Act<T>::down((s - mean2) * rstd2 * (c.g.weight ? c.g.weight[i] : 1.0f) + (c.g.bias ? c.g.bias[i] : 0.0f));
  }
}

// d at one place, from the row's statistics and its two means.
template <int T>
__device__ __forceinline__ float residual_d(const ResidualGradCall& c, int64_t row, int64_t i, float mean2, float rstd2,
                                            float m1, float m2) {
  typedef typename Act<T>::S S;
  const float dout = c.dout ? Act<T>::up((static_cast<const S*>(c.dout) + row * c.dout_stride)[i]) : 0.0f;
  const float u = Act<T>::up((static_cast<const S*>(c.dy) + row * c.dy_stride)[i]) * (c.g.weight ? c.g.weight[i] : 1.0f);
  const float h = (Act<T>::up((static_cast<const S*>(c.out) + row * c.out_stride)[i]) - mean2) * rstd2;
  return dout + rstd2 * (u - m1 - h * m2);
}

// d and dx, one block per row; the row's two means are left for the column sums.
template <int T>
__global__ __launch_bounds__(kThreads) void residual_dx_kernel(ResidualGradCall c) {
  typedef typename Act<T>::S S;
  __shared__ float shared[2 * (kThreads / 64)];
  const int64_t row = blockIdx.x;
  const S* x = static_cast<const S*>(c.x) + row * c.x_stride;
  const S* dy = static_cast<const S*>(c.dy) + row * c.dy_stride;
  const S* out = static_cast<const S*>(c.out) + row * c.out_stride;
  S* dx = static_cast<S*>(c.dx) + row * c.dx_stride;
  S* dr = static_cast<S*>(c.dresidual) + row * c.dresidual_stride;
  const float mean1 = c.stats[row], rstd1 = c.stats[c.n + row], mean2 = c.stats[2 * c.n + row], rstd2 = c.stats[3 * c.n + row];
  float s[2] = {0.0f, 0.0f};
  for (int64_t i = threadIdx.x; i < c.dim; i += kThreads) {
    const float u = Act<T>::up(dy[i]) * (c.g.weight ? c.g.weight[i] : 1.0f);
    s[0] += u;
    s[1] += u * ((Act<T>::up(out[i]) - mean2) * rstd2);
  }
  block_sums(s, shared);
  const float m1 = c.g.center ? s[0] / c.dim : 0.0f, m2 = s[1] / c.dim;
  if (threadIdx.x == 0 && c.reduce) {
    c.means[2 * row] = m1;
    c.means[2 * row + 1] = m2;
  }
  float q[2] = {0.0f, 0.0f}, a, b;
  if (c.g.post) {
    for (int64_t i = threadIdx.x; i < c.dim; i += kThreads) {
      branch_at(c.g, i, a, b);
      const float u = residual_d<T>(c, row, i, mean2, rstd2, m1, m2) * a;
      q[0] += u;
      q[1] += u * ((Act<T>::up(x[i]) - mean1) * rstd1);
    }
    block_sums(q, shared);
  }
  const float n1 = c.g.center ? q[0] / c.dim : 0.0f, n2 = q[1] / c.dim;
  for (int64_t i = threadIdx.x; i < c.dim; i += kThreads) {
    branch_at(c.g, i, a, b);
    const float d = residual_d<T>(c, row, i, mean2, rstd2, m1, m2), u = d * a;
    dr[i] = Act<T>::down(d);
    dx[i] = Act<T>::down(c.g.post ? rstd1 * (u - n1 - (Act<T>::up(x[i]) - mean1) * rstd1 * n2) : u);
  }
}

// Block (columns, group): the group's rows' share of the four column sums.
template <int T>
__global__ __launch_bounds__(kThreads) void residual_dw_kernel(ResidualGradCall c, int64_t per_group) {
  typedef typename Act<T>::S S;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= c.dim) return;
  const int64_t lo = static_cast<int64_t>(blockIdx.y) * per_group;
  const int64_t hi = lo + per_group < c.n ? lo + per_group : c.n;
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int64_t r = lo; r < hi; ++r) {
    const float mean2 = c.stats[2 * c.n + r], rstd2 = c.stats[3 * c.n + r];
    const float dy = Act<T>::up((static_cast<const S*>(c.dy) + r * c.dy_stride)[i]);
    const float d = residual_d<T>(c, r, i, mean2, rstd2, c.means[2 * r], c.means[2 * r + 1]);
    const float x = Act<T>::up((static_cast<const S*>(c.x) + r * c.x_stride)[i]);
    s[0] += dy * ((Act<T>::up((static_cast<const S*>(c.out) + r * c.out_stride)[i]) - mean2) * rstd2);
    s[1] += d * (c.g.post ? (x - c.stats[r]) * c.stats[c.n + r] : x);
    s[2] += dy;
    s[3] += d;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) c.workspace[(4 * static_cast<int64_t>(blockIdx.y) + k) * c.dim + i] = s[k];
}

// Sums the groups' shares, and makes the gradients of them: a block takes 16 columns, 64 threads a
// column every 64th group, whose sums are joined in order.  (64 columns a block leave too few
// blocks: 19 us instead of 6 for 256 groups of 1280 columns.)
constexpr int kJoinWaves = 16;
template <int kCols>
__global__ __launch_bounds__(64 * kJoinWaves) void residual_join_kernel(ResidualGradCall c, int64_t groups) {
  __shared__ float shared[kCols][kJoinWaves][16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 16 + col;
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (i < c.dim) {
    const float* in = c.workspace + i;
#pragma unroll 4
    for (int64_t g = threadIdx.x >> 4; g < groups; g += 4 * kJoinWaves)
#pragma unroll
      for (int k = 0; k < kCols; ++k) s[k] += in[(g * kCols + k) * c.dim];
  }
#pragma unroll
  for (int k = 0; k < kCols; ++k) {
    s[k] += __shfl_xor(s[k], 16, 64);
    s[k] += __shfl_xor(s[k], 32, 64);
    if (lane < 16) shared[k][wave][lane] = s[k];
  }
  __syncthreads();
  if (threadIdx.x >= 16 || i >= c.dim) return;
  for (int w = 1; w < kJoinWaves; ++w)
#pragma unroll
    for (int k = 0; k < kCols; ++k) s[k] += shared[k][w][col];
  const float gate = c.g.scale * (c.g.gate ? c.g.gate[i] : 1.0f);
  if (c.dweight) c.dweight[i] = s[0];
  if (c.dbias) c.dbias[i] = s[2];
  if (c.dpost_weight) c.dpost_weight[i] = gate * s[1];
  if (c.dpost_bias) c.dpost_bias[i] = gate * s[3];
  if (c.dgate)
    c.dgate[i] = c.g.scale * (s[1] * (c.g.post_weight ? c.g.post_weight[i] : 1.0f) + (c.g.post_bias ? s[3] * c.g.post_bias[i] : 0.0f));
}

constexpr int64_t kMaxGroups = 256;

// Blocks of the backward kernel: one a compute unit, as its registers allow, fewer when they would
// get less than two rows' worth of work each.
int64_t grad_blocks(int64_t n, int rows) {
  const int64_t want = (n + 2 * rows - 1) / (2 * rows);
  return want < kMaxGroups ? want : kMaxGroups;
}

}  // namespace

hipError_t launch_residual_forward(const ResidualCall& c, hipStream_t s) {
  return with_act(c.type, [&](auto t) {
    constexpr int T = decltype(t)::value;
    const bool done = with_row<T>(c.dim, [&](auto tpr, auto nv) {
      constexpr int kTPR = decltype(tpr)::value, kB = kTPR < 256 ? 256 : kTPR, kRows = kB / kTPR;
      const int64_t all = (c.n + kRows - 1) / kRows, most = 2048 * kThreads / kB;
      hipLaunchKernelGGL((residual_rows_kernel<T, kTPR, decltype(nv)::value, kB>),
                         dim3(static_cast<unsigned>(all < most ? all : most)), dim3(kB), 0, s, c);
    });
    if (!done) hipLaunchKernelGGL((residual_kernel<T>), dim3(static_cast<unsigned>(c.n)), dim3(kThreads), 0, s, c);
    return hipGetLastError();
  });
}

size_t residual_workspace_bytes(int64_t n, int64_t dim) {
  const int64_t groups = n < kMaxGroups ? n : kMaxGroups;
  return static_cast<size_t>(4 * groups * dim * 4 + n * 8);
}

hipError_t launch_residual_backward(const ResidualGradCall& call, hipStream_t s) {
  ResidualGradCall c = call;
  const bool bias = c.dbias || c.dpost_bias || (c.dgate && c.g.post_bias);
  c.reduce = c.dweight || c.dpost_weight || c.dgate || bias;
  c.means = c.workspace + 4 * (c.n < kMaxGroups ? c.n : kMaxGroups) * c.dim;
  return with_act(c.type, [&](auto t) {
    constexpr int T = decltype(t)::value;
    int64_t groups = 0;
    int cols = bias ? 4 : 2;
    if (c.n > 0) {
      const bool done = with_row<T>(c.dim, [&](auto tpr, auto nv) {
        constexpr int kTPR = decltype(tpr)::value, kNV = decltype(nv)::value, kB = kTPR < 512 ? 512 : kTPR, kRows = kB / kTPR;
        groups = grad_blocks(c.n, kRows);
        const dim3 grid(static_cast<unsigned>(groups));
        if (bias) hipLaunchKernelGGL((residual_grad_kernel<T, kTPR, kNV, kB, true>), grid, dim3(kB), 0, s, c);
        else hipLaunchKernelGGL((residual_grad_kernel<T, kTPR, kNV, kB, false>), grid, dim3(kB), 0, s, c);
      });
      if (!done) {
        cols = 4;
        hipLaunchKernelGGL((residual_dx_kernel<T>), dim3(static_cast<unsigned>(c.n)), dim3(kThreads), 0, s, c);
        if (c.reduce) {
          const int64_t most = c.n < kMaxGroups ? c.n : kMaxGroups;
          const int64_t per = (c.n + most - 1) / most;
          groups = (c.n + per - 1) / per;
          hipLaunchKernelGGL((residual_dw_kernel<T>), dim3(static_cast<unsigned>((c.dim + kThreads - 1) / kThreads), static_cast<unsigned>(groups)),
                             dim3(kThreads), 0, s, c, per);
        }
      }
    }
    if (c.reduce) {
      const dim3 grid(static_cast<unsigned>((c.dim + 15) / 16));
      if (cols == 4) hipLaunchKernelGGL(residual_join_kernel<4>, grid, dim3(64 * kJoinWaves), 0, s, c, groups);
      else hipLaunchKernelGGL(residual_join_kernel<2>, grid, dim3(64 * kJoinWaves), 0, s, c, groups);
    }
    return hipGetLastError();
  });
}

}  // namespace ma

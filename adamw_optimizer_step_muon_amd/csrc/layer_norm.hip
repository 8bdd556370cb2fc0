// Layer norm over the last dimension, forward and backward.
//
//   mean = sum x / D,  rstd = 1 / sqrt(sum (x - mean)^2 / D + eps),  h = (x - mean) rstd
//   y = h w + b
//   u = dy w,  dx = rstd (u - sum u / D - h sum (u h) / D)
//   dw (+)= sum over rows of dy h,  db (+)= sum over rows of dy
//
// All arithmetic in fp32; the variance is summed from the deviations, not as E x^2 - mean^2,
// which loses everything where the mean is large.
//
// Memory-bound: 2 bytes read and 2 written per 16-bit value forward, 4 read and 2 written
// backward.  Rows are therefore held in registers between the passes that their sums need.
// Measured: 32768 x 2048 bf16 forward 50 us (5.4 TB/s; 190 us where a block sweeps a row three
// times), 16384 x 8192 bf16 backward with both column sums 162 us (5.0 TB/s; 567 us as a
// kernel by rows and one by columns).  A large device copy reaches 4.8 TB/s.
#include "ma_act.h"
#include "ma_internal.h"

namespace ma {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

// ---------------------------------------------------------------------------
// Rows in registers: kTPR threads (16 to 1024) hold a row, kNV vectors of 16 bytes each, so x is read
// once for mean, variance and output.  Blocks walk over rows (the next row's loads are
// issued before this row's sums are joined) and keep the gains in registers.
// ---------------------------------------------------------------------------
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

template <int T, int kTPR, int kNV, int kBlock>
__global__ __launch_bounds__(kBlock) void norm_rows_kernel(NormCall c) {
  typedef typename Act<T>::S S;
  typedef typename Vec<T>::P P;
  constexpr int N = Vec<T>::kN, kRows = kBlock / kTPR;
  __shared__ float shared[2][kBlock / 64];
  const int t = threadIdx.x % kTPR, sub = threadIdx.x / kTPR;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
  int64_t base = static_cast<int64_t>(blockIdx.x) * kRows;
  int cnt[kNV];
  float w[kNV][N], b[kNV][N];
  P next[kNV];
  const S* x0 = static_cast<const S*>(c.x) + t * N;
#pragma unroll
  for (int v = 0; v < kNV; ++v) {
    const int at = (v * kTPR + t) * N;
    cnt[v] = static_cast<int>(c.dim) - at;
    if (base + sub < c.n) next[v] = load_raw<T>(x0 + (base + sub) * c.x_stride + v * kTPR * N, cnt[v]);
    if (c.weight) {
      load_floats<N>(c.weight + at, cnt[v], 0.0f, w[v]);
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) w[v][e] = 1.0f;
    }
    if (c.bias) {
      load_floats<N>(c.bias + at, cnt[v], 0.0f, b[v]);
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) b[v][e] = 0.0f;
    }
  }
  const float dim = static_cast<float>(c.dim);
  for (; base < c.n; base += step) {  // the same trips for every thread of the block
    const int64_t row = base + sub;
    float x[kNV][N], sum[1] = {0.0f};
#pragma unroll
    for (int v = 0; v < kNV; ++v)
#pragma unroll
      for (int e = 0; e < N; ++e) {
        x[v][e] = Act<T>::up(next[v][e]);
        sum[0] += x[v][e];
      }
    if (row + step < c.n) {
#pragma unroll
      for (int v = 0; v < kNV; ++v)
        next[v] = load_raw<T>(x0 + (row + step) * c.x_stride + v * kTPR * N, cnt[v]);
    }
    row_sums<kTPR>(sum, shared[0]);
    const float mean = sum[0] / dim;
    float sq[1] = {0.0f};
#pragma unroll
    for (int v = 0; v < kNV; ++v)
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float d = e < cnt[v] ? x[v][e] - mean : 0.0f;
        sq[0] += d * d;
      }
    row_sums<kTPR>(sq, shared[1]);
    const float rstd = 1.0f / __builtin_sqrtf(sq[0] / dim + c.eps);
    if (row >= c.n) continue;
    if (t == 0) {
      c.mean[row] = mean;
      c.rstd[row] = rstd;
    }
#pragma unroll
    for (int v = 0; v < kNV; ++v) {
      float y[N];
#pragma unroll
      for (int e = 0; e < N; ++e) y[e] = (x[v][e] - mean) * rstd * w[v][e] + b[v][e];
      if (cnt[v] > 0)
        store_part<T, N>(static_cast<S*>(c.y) + row * c.y_stride + (v * kTPR + t) * N, cnt[v], y);
    }
  }
}

// Backward with x and dy in registers: dx, and the block's share of dw and db, which the
// threads that own the columns add up over the block's rows.  512 blocks at most, two a CU:
// each leaves one partial sum per column, 8 % of the traffic at 16384 x 8192, which
// norm_join_kernel adds in order.
template <int T, int kTPR, int kNV, int kBlock>
__global__ __launch_bounds__(kBlock) void norm_grad_rows_kernel(NormGradCall c) {
  typedef typename Act<T>::S S;
  typedef typename Vec<T>::P P;
  constexpr int N = Vec<T>::kN, kRows = kBlock / kTPR;
  // 1024 threads have 128 registers each: for their longest rows the gains are read again
  // for every row and the next row's loads wait
  constexpr bool kLean = kTPR == 1024 && kNV * N >= 16;
  __shared__ float shared[2][2 * (kBlock / 64)];
  __shared__ float join[kRows > 1 ? 2 * kTPR * kNV * N : 1];
  const int t = threadIdx.x % kTPR, sub = threadIdx.x / kTPR;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
  int64_t base = static_cast<int64_t>(blockIdx.x) * kRows;
  const S* x0 = static_cast<const S*>(c.x) + t * N;
  const S* y0 = static_cast<const S*>(c.dy) + t * N;
  int cnt[kNV];
  float dw[kNV][N], db[kNV][N];
#pragma unroll
  for (int v = 0; v < kNV; ++v) {
    cnt[v] = static_cast<int>(c.dim) - (v * kTPR + t) * N;
#pragma unroll
    for (int e = 0; e < N; ++e) dw[v][e] = db[v][e] = 0.0f;
  }
  const auto load_rows = [&](int64_t row, P (&x)[kNV], P (&y)[kNV]) {
#pragma unroll
    for (int v = 0; v < kNV; ++v) {
      x[v] = load_raw<T>(x0 + row * c.x_stride + v * kTPR * N, cnt[v]);
      y[v] = load_raw<T>(y0 + row * c.dy_stride + v * kTPR * N, cnt[v]);
    }
  };
  const auto load_gains = [&](int v, float (&w)[N]) {
#pragma unroll
    for (int e = 0; e < N; ++e) w[e] = 1.0f;
    if (c.weight) load_floats<N>(c.weight + (v * kTPR + t) * N, cnt[v], 0.0f, w);
  };
  const float dim = static_cast<float>(c.dim);
  // the row's two sums, and its share of the columns'
  const auto gather = [&](int v, const P& x, const P& y, const float (&w)[N], float mean, float rstd, float (&s)[2]) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      // behind the row's end dy is zero, so nothing is added
      const float g = Act<T>::up(y[e]), h = (Act<T>::up(x[e]) - mean) * rstd;
      const float u = g * w[e];
      s[0] += u;
      s[1] += u * h;
      dw[v][e] += g * h;
      db[v][e] += g;
    }
  };
  const auto give = [&](int v, const P& x, const P& y, const float (&w)[N], int64_t row, float mean, float rstd,
                        const float (&s)[2]) {
    const float m1 = s[0] / dim, m2 = s[1] / dim;
    float d[N];
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float h = (Act<T>::up(x[e]) - mean) * rstd;
      d[e] = rstd * (Act<T>::up(y[e]) * w[e] - m1 - h * m2);
    }
    if (cnt[v] > 0)
      store_part<T, N>(static_cast<S*>(c.dx) + row * c.dx_stride + (v * kTPR + t) * N, cnt[v], d);
  };
  int turn = 0;
  if constexpr (kLean) {
    for (int64_t row = base; row < c.n; row += step, turn ^= 1) {  // one row a block
      const float mean = c.mean[row], rstd = c.rstd[row];
      P x[kNV], y[kNV];
      load_rows(row, x, y);
      float s[2] = {0.0f, 0.0f};
#pragma unroll
      for (int v = 0; v < kNV; ++v) {
        float w[N];
        load_gains(v, w);
        gather(v, x[v], y[v], w, mean, rstd, s);
      }
      row_sums<kTPR>(s, shared[turn]);
#pragma unroll
      for (int v = 0; v < kNV; ++v) {
        float w[N];
        load_gains(v, w);
        give(v, x[v], y[v], w, row, mean, rstd, s);
      }
    }
  } else {
    float w[kNV][N];
    P nx[kNV], ny[kNV];
#pragma unroll
    for (int v = 0; v < kNV; ++v) load_gains(v, w[v]);
    float next_mean = 0.0f, next_rstd = 0.0f;
    if (base + sub < c.n) {
      load_rows(base + sub, nx, ny);
      next_mean = c.mean[base + sub];
      next_rstd = c.rstd[base + sub];
    }
    for (; base < c.n; base += step, turn ^= 1) {  // the same trips for every thread of the block
      const int64_t row = base + sub;
      const bool live = row < c.n;
      P x[kNV], y[kNV];
#pragma unroll
      for (int v = 0; v < kNV; ++v) {
        x[v] = nx[v];
        y[v] = ny[v];
      }
      const float mean = next_mean, rstd = next_rstd;
      if (row + step < c.n) {
        next_mean = c.mean[row + step];
        next_rstd = c.rstd[row + step];
        load_rows(row + step, nx, ny);
      }
      float s[2] = {0.0f, 0.0f};
      if (live) {
#pragma unroll
        for (int v = 0; v < kNV; ++v) gather(v, x[v], y[v], w[v], mean, rstd, s);
      }
      row_sums<kTPR>(s, shared[turn]);
      if (!live) continue;
#pragma unroll
      for (int v = 0; v < kNV; ++v) give(v, x[v], y[v], w[v], row, mean, rstd, s);
    }
  }
  if (!c.dweight && !c.dbias) return;
  // the block's rows' sums: waves that share columns add theirs in order
  if constexpr (kRows > 1) {
    for (int k = 0; k < kRows; ++k) {
      if (sub == k) {
#pragma unroll
        for (int v = 0; v < kNV; ++v)
#pragma unroll
          for (int e = 0; e < N; ++e) {
            float* j = join + (v * N + e) * 2 * kTPR + t;
            if (k > 0) {
              dw[v][e] += j[0];
              db[v][e] += j[kTPR];
            }
            j[0] = dw[v][e];
            j[kTPR] = db[v][e];
          }
      }
      __syncthreads();
    }
    if (sub != kRows - 1) return;
  }
  float* part = c.workspace + static_cast<int64_t>(blockIdx.x) * 2 * c.dim;
#pragma unroll
  for (int v = 0; v < kNV; ++v) {
    if (cnt[v] <= 0) continue;
    store_part<kActF32, N>(part + (v * kTPR + t) * N, cnt[v], dw[v]);
    store_part<kActF32, N>(part + c.dim + (v * kTPR + t) * N, cnt[v], db[v]);
  }
}

// ---------------------------------------------------------------------------
// Rows too long for the registers of 1024 threads: several sweeps, a value at a time.
// ---------------------------------------------------------------------------
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

// Groups of rows, at most, of the reduction over rows.
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

// Sums the groups' partial sums: a block takes 64 of the 2 dim columns, each wave every
// kJoinWaves-th group, and joins the waves' sums in order.
constexpr int kJoinWaves = 16;
__global__ __launch_bounds__(64 * kJoinWaves) void norm_join_kernel(NormGradCall c, int64_t groups) {
  __shared__ float shared[kJoinWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * 64 + lane, cols = 2 * c.dim;
  float sum = 0.0f;
  if (i < cols) {
#pragma unroll 8
    for (int64_t g = wave; g < groups; g += kJoinWaves) sum += c.workspace[g * cols + i];
  }
  shared[wave][lane] = sum;
  __syncthreads();
  if (wave != 0 || i >= cols) return;
  for (int w = 1; w < kJoinWaves; ++w) sum += shared[w][lane];
  float* out = i < c.dim ? c.dweight : c.dbias;
  if (!out) return;
  out += i < c.dim ? i : i - c.dim;
  *out = c.add ? *out + sum : sum;
}

}  // namespace

namespace {

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

// Blocks of the backward kernel: two a compute unit, fewer when they would get less than
// two rows' worth of work each (every block writes one partial sum per column).  One, two or four
// rows at least give the same times within 1 us from 16 x 8192 to 16384 x 16384 bf16, but for
// 1024 x 8192, where four take 20.7 us and two 23.6.  At most one block a unit is faster for wide
// rows, whose partial sums are a third of the traffic at 4096 x 16384 (104 us against 112; 16384
// x 8192 156 against 165), and slower for narrow ones (16384 x 768: 25.2 against 23.9 us).
int64_t grad_blocks(int64_t n, int rows) {
  const int64_t want = (n + 2 * rows - 1) / (2 * rows);
  return want < 512 ? want : 512;
}

}  // namespace

hipError_t launch_layer_norm_forward(const NormCall& c, hipStream_t s) {
  return with_act(c.type, [&](auto t) {
    constexpr int T = decltype(t)::value;
    const bool done = with_row<T>(c.dim, [&](auto tpr, auto nv) {
      constexpr int kTPR = decltype(tpr)::value, kB = kTPR < 256 ? 256 : kTPR, kRows = kB / kTPR;
      const int64_t all = (c.n + kRows - 1) / kRows, most = 2048 * kThreads / kB;
      hipLaunchKernelGGL((norm_rows_kernel<T, kTPR, decltype(nv)::value, kB>),
                         dim3(static_cast<unsigned>(all < most ? all : most)), dim3(kB), 0, s, c);
    });
    if (!done) hipLaunchKernelGGL((norm_kernel<T>), dim3(static_cast<unsigned>(c.n)), dim3(kThreads), 0, s, c);
    return hipGetLastError();
  });
}

size_t layer_norm_workspace_bytes(int64_t n, int64_t dim) {
  const int64_t groups = n < 512 ? n : 512;
  return static_cast<size_t>(2 * groups * dim * 4);
}

hipError_t launch_layer_norm_backward(const NormGradCall& c, hipStream_t s) {
  return with_act(c.type, [&](auto t) {
    constexpr int T = decltype(t)::value;
    const bool reduce = c.dweight || c.dbias;
    int64_t groups = 0;
    if (c.n > 0) {
      const bool done = with_row<T>(c.dim, [&](auto tpr, auto nv) {
        constexpr int kTPR = decltype(tpr)::value, kB = kTPR < 512 ? 512 : kTPR, kRows = kB / kTPR;
        groups = grad_blocks(c.n, kRows);
        hipLaunchKernelGGL((norm_grad_rows_kernel<T, kTPR, decltype(nv)::value, kB>),
                           dim3(static_cast<unsigned>(groups)), dim3(kB), 0, s, c);
      });
      if (!done) {
        hipLaunchKernelGGL((norm_dx_kernel<T>), dim3(static_cast<unsigned>(c.n)), dim3(kThreads), 0, s, c);
        if (reduce) {
          const int64_t most = c.n < kMaxGroups ? c.n : kMaxGroups;
          const int64_t per = (c.n + most - 1) / most;
          groups = (c.n + per - 1) / per;
          hipLaunchKernelGGL((norm_dw_kernel<T>), dim3(static_cast<unsigned>((c.dim + kThreads - 1) / kThreads), static_cast<unsigned>(groups)),
                             dim3(kThreads), 0, s, c, per);
        }
      }
    }
    if (reduce)
      hipLaunchKernelGGL(norm_join_kernel, dim3(static_cast<unsigned>((2 * c.dim + 63) / 64)), dim3(64 * kJoinWaves), 0, s, c, groups);
    return hipGetLastError();
  });
}

}  // namespace ma

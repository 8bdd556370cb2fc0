// Embedding lookup with scaling, its table gradient by sorted tokens, and the AdamW step of
// a table taken straight from the tokens.
//
//   out[t]   = s table[tok_t]
//   grad[v] (+)= s sum over t with tok_t = v of dout[t]
//
// A token outside [0, rows) (padding) reads nothing, gives a zero row and no gradient.
//
// The gradient sorts the tokens (stable, least significant digit first), so that each row's
// outputs are summed in one fixed order by the threads that own the row: no atomics on
// floats, the same bits on every run.  Three stages share one workspace:
//   1. sort:     keys (row of each token, `rows` for padding) and the tokens' positions
//   2. segments: [start, end) of each row that occurs; rows with more than kChunk tokens
//                get partial sums, one per chunk of sorted positions, so that a frequent
//                token's row is summed by many blocks
//   3. rows:     every element of the table: its row's sum, then the gradient's store or
//                the AdamW update
// Stage 2 writes start and end of the occurring rows only; stage 3 accepts a row's start
// if the sorted keys confirm it (the key there is the row and the one before is not), so
// nothing has to be cleared, whatever the workspace held.
#include "adamw_elem.h"
#include "ma_act.h"
#include "ma_internal.h"

namespace ma {
namespace {

constexpr int kThreads = 256;
constexpr int kSortThreads = 512;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kMaxBins = 512;  // 9 bits a pass: vocabularies up to 2^18 - 1 take two passes

__device__ __forceinline__ uint32_t key_of(const void* tokens, int bits, int64_t i,
                                           uint32_t rows) {
  const int64_t t = bits == 64 ? static_cast<const int64_t*>(tokens)[i]
                               : static_cast<const int32_t*>(tokens)[i];
  return t >= 0 && t < static_cast<int64_t>(rows) ? static_cast<uint32_t>(t) : rows;
}

// ---------------------------------------------------------------------------
// 1. sort
// ---------------------------------------------------------------------------
// Digit counts of each block's share [b * share, (b + 1) * share) of the n keys.
__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(SortArgs a, int shift, int bins,
                                                                  int first,
                                                                  const uint32_t* keys) {
  __shared__ uint32_t hist[kMaxBins];
  const int tid = threadIdx.x;
  hist[tid] = 0;
  __syncthreads();
  const int64_t lo = static_cast<int64_t>(blockIdx.x) * a.share;
  const int64_t hi = lo + a.share < a.n ? lo + a.share : a.n;
  for (int64_t i = lo + tid; i < hi; i += kSortThreads) {
    const uint32_t k = first ? key_of(a.tokens, a.token_bits, i, a.rows) : keys[i];
    atomicAdd(&hist[(k >> shift) & (bins - 1)], 1u);
  }
  __syncthreads();
  if (tid < bins) a.counts[static_cast<int64_t>(blockIdx.x) * bins + tid] = hist[tid];
}

// Stable scatter of each block's share to its digits' places.
__global__ __launch_bounds__(kSortThreads) void sort_scatter_kernel(
    SortArgs a, int shift, int bins, int first, const uint32_t* keys, const uint32_t* order,
    uint32_t* keys_out, uint32_t* order_out) {
  __shared__ uint32_t base[kMaxBins];
  __shared__ uint32_t count[kSortWaves][kMaxBins];
  __shared__ uint32_t wave_total[kSortWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  // this block's first place for digit tid: all smaller digits, and this digit in earlier
  // blocks
  uint32_t before = 0, total = 0;
  if (tid < bins)
    for (int b = 0; b < static_cast<int>(gridDim.x); ++b) {
      const uint32_t c = a.counts[static_cast<int64_t>(b) * bins + tid];
      if (b < static_cast<int>(blockIdx.x)) before += c;
      total += c;
    }
  uint32_t scan = total;
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t up = __shfl_up(scan, d, 64);
    if (lane >= d) scan += up;
  }
  if (lane == 63) wave_total[wave] = scan;
  __syncthreads();
  for (int w = 0; w < wave; ++w) scan += wave_total[w];
  base[tid] = scan - total + before;
  const int64_t lo = static_cast<int64_t>(blockIdx.x) * a.share;
  const int64_t hi = lo + a.share < a.n ? lo + a.share : a.n;
  for (int64_t t0 = lo; t0 < hi; t0 += kSortThreads) {
    for (int w = 0; w < kSortWaves; ++w) count[w][tid] = 0;
    __syncthreads();
    const int64_t i = t0 + tid;
    const bool in = i < hi;
    uint32_t k = 0, o = 0;
    if (in) {
      k = first ? key_of(a.tokens, a.token_bits, i, a.rows) : keys[i];
      o = first ? static_cast<uint32_t>(i) : order[i];
    }
    const uint32_t d = (k >> shift) & (bins - 1);
    // the lanes of this wave with the same digit
    uint64_t same = __ballot(in);
    for (int bit = 1; bit < bins; bit <<= 1) {
      const uint64_t with = __ballot((d & bit) != 0);
      same &= (d & bit) ? with : ~with;
    }
    const int rank = __popcll(same & ((1ull << lane) - 1));
    if (in && rank == 0) count[wave][d] = static_cast<uint32_t>(__popcll(same));
    __syncthreads();
    uint32_t at = base[tid];
    for (int w = 0; w < kSortWaves; ++w) {
      const uint32_t c = count[w][tid];
      count[w][tid] = at;
      at += c;
    }
    base[tid] = at;
    __syncthreads();
    if (in) {
      const uint32_t place = count[wave][d] + rank;
      keys_out[place] = k;
      order_out[place] = o;
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// 2. segments
// ---------------------------------------------------------------------------
// How many of the keys at [lo, hi) equal k (every thread gets the count).
__device__ __forceinline__ int block_count(const uint32_t* keys, int64_t lo, int64_t hi,
                                           uint32_t k, int* shared) {
  int c = 0;
  for (int64_t i = lo + threadIdx.x; i < hi; i += kThreads) c += keys[i] == k;
  for (int d = 32; d > 0; d >>= 1) c += __shfl_xor(c, d, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) shared[threadIdx.x >> 6] = c;
  __syncthreads();
  c = 0;
  for (int w = 0; w < kThreads / 64; ++w) c += shared[w];
  return c;
}

template <int T>
__device__ void partial_sum(const RowArgs& a, int64_t lo, int64_t hi, int64_t slot, int64_t c) {
  const typename Act<T>::S* dout = static_cast<const typename Act<T>::S*>(a.dout);
  if (c >= a.dim) return;
  float acc = 0.0f;
  for (int64_t i = lo; i < hi; ++i) acc += Act<T>::up(dout[a.order[i] * a.dout_stride + c]);
  a.partial[slot * a.dim + c] = acc;
}

// Block (j, slice): sorted positions [j chunk, (j + 1) chunk).  Slice 0 writes the segments'
// ends; every slice sums kThreads columns of the rows with more than `chunk` tokens.  At
// most two of those meet a chunk: the one at its first position (partial 2 j) and the one
// at its last (2 j + 1, where that is another row).
template <int T>
__global__ __launch_bounds__(kThreads) void segments_kernel(RowArgs a) {
  __shared__ int shared[kThreads / 64];
  const int64_t n = a.n;
  const int64_t lo = static_cast<int64_t>(blockIdx.x) * a.chunk;
  const int64_t hi = lo + a.chunk < n ? lo + a.chunk : n;
  if (blockIdx.y == 0)
    for (int64_t i = lo + threadIdx.x; i < hi; i += kThreads) {
      const uint32_t k = a.keys[i];
      if (k >= a.rows) continue;
      if (i == 0 || a.keys[i - 1] != k) a.start[k] = static_cast<uint32_t>(i);
      if (i == n - 1 || a.keys[i + 1] != k) a.end[k] = static_cast<uint32_t>(i + 1);
    }
  const int64_t c = static_cast<int64_t>(blockIdx.y) * kThreads + threadIdx.x;
  const uint32_t k0 = a.keys[lo], k1 = a.keys[hi - 1];
  if (k0 < a.rows) {
    const int back = block_count(a.keys, lo > a.chunk ? lo - a.chunk : 0, lo, k0, shared);
    const int in = block_count(a.keys, lo, hi, k0, shared);
    const int fwd = block_count(a.keys, hi, hi + a.chunk < n ? hi + a.chunk : n, k0, shared);
    if (back + in + fwd > a.chunk) partial_sum<T>(a, lo, lo + in, 2 * static_cast<int64_t>(blockIdx.x), c);
  }
  if (k1 != k0 && k1 < a.rows) {
    const int in = block_count(a.keys, lo, hi, k1, shared);
    const int fwd = block_count(a.keys, hi, hi + a.chunk < n ? hi + a.chunk : n, k1, shared);
    if (in + fwd > a.chunk) partial_sum<T>(a, hi - in, hi, 2 * static_cast<int64_t>(blockIdx.x) + 1, c);
  }
}

// ---------------------------------------------------------------------------
// 3. rows
// ---------------------------------------------------------------------------
// Tokens of row v: their number, 0 if it does not occur; *s the first sorted position.
__device__ __forceinline__ uint32_t segment_of(const RowArgs& a, uint32_t v, uint32_t* s) {
  if (a.n == 0) return 0;
  const uint32_t b = a.start[v];
  if (b >= a.n || a.keys[b] != v || (b > 0 && a.keys[b - 1] == v)) return 0;
  *s = b;
  return a.end[v] - b;
}

// Column c of the sum over the m tokens at sorted position s.
template <int T>
__device__ __forceinline__ float segment_sum(const RowArgs& a, uint32_t s, uint32_t m, int64_t c) {
  float acc = 0.0f;
  if (m <= static_cast<uint32_t>(a.chunk)) {
    const typename Act<T>::S* dout = static_cast<const typename Act<T>::S*>(a.dout);
    for (uint32_t i = s; i < s + m; ++i) acc += Act<T>::up(dout[a.order[i] * a.dout_stride + c]);
  } else {
    const int64_t j0 = s / a.chunk, j1 = (s + m - 1) / a.chunk;
    acc = a.partial[(2 * j0 + (s % a.chunk != 0)) * a.dim + c];
    for (int64_t j = j0 + 1; j <= j1; ++j) acc += a.partial[2 * j * a.dim + c];
  }
  return acc;
}

// grad = s sum, or grad + s sum (kAdd, occurring rows only).  The product is rounded before
// it is added, so adding gives the bits of a separate gradient's addition.
template <int T, bool kAdd>
__global__ __launch_bounds__(kThreads) void grad_rows_kernel(RowArgs a, float* grad) {
#pragma clang fp contract(off)
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= static_cast<int64_t>(a.rows) * a.dim) return;
  const uint32_t v = static_cast<uint32_t>(i / a.dim);
  uint32_t s = 0;
  const uint32_t m = segment_of(a, v, &s);
  if (kAdd && m == 0) return;
  const float g = m ? a.scale * segment_sum<T>(a, s, m, i - v * a.dim) : 0.0f;
  grad[i] = kAdd ? grad[i] + g : g;
}

template <int T, int kMode>
__global__ __launch_bounds__(kThreads) void step_rows_kernel(RowArgs a, float* p, float* m, float* v,
                                                             AdamWConst c) {
#pragma clang fp contract(off)
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= static_cast<int64_t>(a.rows) * a.dim) return;
  const uint32_t r = static_cast<uint32_t>(i / a.dim);
  uint32_t s = 0;
  const uint32_t cnt = segment_of(a, r, &s);
  const float g = cnt ? a.scale * segment_sum<T>(a, s, cnt, i - r * a.dim) : 0.0f;
  float P = p[i], M = m[i], V = v[i];
  adamw_elem_t<kMode>(P, g, M, V, c);
  p[i] = P;
  m[i] = M;
  v[i] = V;
}

// ---------------------------------------------------------------------------
// lookup
// ---------------------------------------------------------------------------
template <int T>
__global__ __launch_bounds__(kThreads) void lookup_kernel(const float* table, uint32_t rows,
                                                          int64_t dim, const void* tokens,
                                                          int token_bits, int64_t n, float scale,
                                                          typename Act<T>::S* out,
                                                          int64_t out_stride) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= n * dim) return;
  const int64_t t = i / dim, c = i - t * dim;
  const uint32_t v = key_of(tokens, token_bits, t, rows);
  out[t * out_stride + c] = Act<T>::down(v < rows ? scale * table[v * dim + c] : 0.0f);
}

int64_t up256(int64_t x) { return (x + 255) / 256 * 256; }

}  // namespace

// Sort passes for keys 0..rows: digits of at most 9 bits, of equal width.
static void sort_digits(uint32_t rows, int* passes, int* width) {
  int bits = 1;
  while (bits < 32 && (rows >> bits)) ++bits;
  *passes = (bits + 8) / 9;
  *width = (bits + *passes - 1) / *passes;
}

EmbeddingPlan plan_embedding(int64_t rows, int64_t dim, int64_t n) {
  EmbeddingPlan p{};
  if (rows < 1 || dim < 1 || n < 1) return p;
  // at most 128 shares, so that each scatter block can add up every block's counts
  p.share = (n + 127) / 128;
  p.share = (p.share + kSortThreads - 1) / kSortThreads * kSortThreads;
  p.blocks = static_cast<int>((n + p.share - 1) / p.share);
  // at most 1024 partial sums to join for one row
  p.chunk = 64;
  while (n / p.chunk > 1024) p.chunk *= 2;
  p.chunks = (n + p.chunk - 1) / p.chunk;
  int64_t at = 0;
  for (int i = 0; i < 2; ++i) {
    p.keys[i] = at;
    at += up256(n * 4);
    p.order[i] = at;
    at += up256(n * 4);
  }
  p.counts = at;
  at += up256(static_cast<int64_t>(p.blocks) * kMaxBins * 4);
  p.start = at;
  at += up256(rows * 4);
  p.end = at;
  at += up256(rows * 4);
  p.partial = at;
  at += n > p.chunk ? up256(2 * p.chunks * dim * 4) : 0;
  p.bytes = at;
  return p;
}

int64_t embedding_threads(int64_t rows, int64_t dim, int64_t n) {
  const EmbeddingPlan p = plan_embedding(rows, dim, n);
  const int64_t table = rows * dim, out = n * dim, parts = p.chunks * kThreads;
  return (table > out ? (table > parts ? table : parts) : (out > parts ? out : parts)) + kThreads;
}

// Sorts the tokens and finds the segments; fills the arguments of stage 3.
static hipError_t sort_tokens(const EmbeddingCall& e, RowArgs* out, hipStream_t s) {
  *out = RowArgs{};
  out->rows = static_cast<uint32_t>(e.rows);
  out->dim = e.dim;
  if (e.n == 0) return hipSuccess;  // no row occurs
  const EmbeddingPlan p = plan_embedding(e.rows, e.dim, e.n);
  char* ws = static_cast<char*>(e.workspace);
  uint32_t* keys[2] = {reinterpret_cast<uint32_t*>(ws + p.keys[0]), reinterpret_cast<uint32_t*>(ws + p.keys[1])};
  uint32_t* order[2] = {reinterpret_cast<uint32_t*>(ws + p.order[0]), reinterpret_cast<uint32_t*>(ws + p.order[1])};
  SortArgs sa{};
  sa.tokens = e.tokens;
  sa.token_bits = e.token_bits;
  sa.n = e.n;
  sa.rows = static_cast<uint32_t>(e.rows);
  sa.share = p.share;
  sa.counts = reinterpret_cast<uint32_t*>(ws + p.counts);
  int passes, width;
  sort_digits(sa.rows, &passes, &width);
  const dim3 grid(static_cast<unsigned>(p.blocks)), block(kSortThreads);
  for (int pass = 0; pass < passes; ++pass) {
    const int from = (pass + 1) & 1, to = pass & 1;
    hipLaunchKernelGGL(sort_count_kernel, grid, block, 0, s, sa, pass * width, 1 << width, pass == 0, keys[from]);
    hipLaunchKernelGGL(sort_scatter_kernel, grid, block, 0, s, sa, pass * width, 1 << width, pass == 0,
                       keys[from], order[from], keys[to], order[to]);
  }
  RowArgs a{};
  a.keys = keys[(passes - 1) & 1];
  a.order = order[(passes - 1) & 1];
  a.start = reinterpret_cast<uint32_t*>(ws + p.start);
  a.end = reinterpret_cast<uint32_t*>(ws + p.end);
  a.partial = reinterpret_cast<float*>(ws + p.partial);
  a.dout = e.dout;
  a.dout_stride = e.dout_stride;
  a.n = e.n;
  a.dim = e.dim;
  a.rows = sa.rows;
  a.chunk = p.chunk;
  a.scale = e.scale;
  *out = a;
  return with_act(e.dout_type, [&](auto t) {
    const dim3 g(static_cast<unsigned>(p.chunks),
                 e.n > p.chunk ? static_cast<unsigned>((e.dim + kThreads - 1) / kThreads) : 1u);
    hipLaunchKernelGGL((segments_kernel<decltype(t)::value>), g, dim3(kThreads), 0, s, a);
    return hipGetLastError();
  });
}

static dim3 row_grid(const EmbeddingCall& e) {
  return dim3(static_cast<unsigned>((e.rows * e.dim + kThreads - 1) / kThreads));
}

hipError_t launch_embedding_forward(const float* table, int64_t rows, int64_t dim,
                                    const void* tokens, int token_bits, int64_t n, float scale,
                                    void* out, int out_type, int64_t out_stride, hipStream_t s) {
  return with_act(out_type, [&](auto t) {
    typedef typename Act<decltype(t)::value>::S S;
    hipLaunchKernelGGL((lookup_kernel<decltype(t)::value>), dim3(static_cast<unsigned>((n * dim + kThreads - 1) / kThreads)),
                       dim3(kThreads), 0, s, table, static_cast<uint32_t>(rows), dim, tokens,
                       token_bits, n, scale, static_cast<S*>(out), out_stride);
    return hipGetLastError();
  });
}

hipError_t launch_embedding_backward(const EmbeddingCall& e, float* grad, bool add, hipStream_t s) {
  RowArgs a;
  const hipError_t st = sort_tokens(e, &a, s);
  if (st != hipSuccess) return st;
  return with_act(e.dout_type, [&](auto t) {
    if (add) hipLaunchKernelGGL((grad_rows_kernel<decltype(t)::value, true>), row_grid(e), dim3(kThreads), 0, s, a, grad);
    else hipLaunchKernelGGL((grad_rows_kernel<decltype(t)::value, false>), row_grid(e), dim3(kThreads), 0, s, a, grad);
    return hipGetLastError();
  });
}

hipError_t launch_adamw_embedding(const EmbeddingCall& e, float* p, float* m, float* v,
                                  const AdamWConst& c, hipStream_t s) {
  RowArgs a;
  const hipError_t st = sort_tokens(e, &a, s);
  if (st != hipSuccess) return st;
  return with_act(e.dout_type, [&](auto t) {
    constexpr int T = decltype(t)::value;
    switch (decay_mode(c)) {
      case kCoupled: hipLaunchKernelGGL((step_rows_kernel<T, kCoupled>), row_grid(e), dim3(kThreads), 0, s, a, p, m, v, c); break;
      case kDecoupledCautious: hipLaunchKernelGGL((step_rows_kernel<T, kDecoupledCautious>), row_grid(e), dim3(kThreads), 0, s, a, p, m, v, c); break;
      default: hipLaunchKernelGGL((step_rows_kernel<T, kDecoupled>), row_grid(e), dim3(kThreads), 0, s, a, p, m, v, c); break;
    }
    return hipGetLastError();
  });
}

}  // namespace ma

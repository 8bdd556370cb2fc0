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
//   2. segments: [start, end) of each row that occurs; rows with more than a chunk of tokens
//                get partial sums, one per chunk of sorted positions, so that a frequent
//                token's row is summed by many blocks
//   3. rows:     every element of the table: its row's sum, then the gradient's store or
//                the AdamW update
// Up to kDirect tokens need none of this: a block finds the tokens of its rows by itself.
//
// start and end are written for the occurring rows only; stage 3 accepts a row's start if the
// sorted keys confirm it (the key there is the row and the one before is not), so nothing
// has to be cleared, whatever the workspace held.
//
// Threads take units of a few columns of a row.  Where fp32 rows are written (stage 3) a unit
// is four columns, so that a wave's stores cover whole cache lines and can bypass the cache:
// units of eight leave every store half a line, 1.2 times slower with non-temporal stores and
// 1.1 times without.  Elsewhere it is eight, one 16-byte access of a 16-bit row.
#include <algorithm>

#include "adamw_elem.h"
#include "ma_act.h"
#include "ma_internal.h"

namespace ma {
namespace {

constexpr int kThreads = 256;
constexpr int kWide = 8;    // columns of a unit: lookup, partial sums
constexpr int kNarrow = 4;  // rows of the table
constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kMaxBins = 512;      // 9 bits a pass: vocabularies up to 2^18 - 1 take two passes
constexpr int kDirect = 256;       // tokens that every block looks through itself
constexpr int kOneLaunch = 16384;  // tokens sorted in one launch: keys and two orders in 128 KB
constexpr int kLocalBits = 6;      // digits of its passes
constexpr int kLocalBins = 1 << kLocalBits;
static_assert(kLocalBins == 64 && kOneLaunch <= 65536, "a digit a lane, 16-bit places");
static_assert(kSortThreads >= kMaxBins, "a thread per digit");

__device__ __forceinline__ uint32_t key_of(int64_t token, uint32_t rows) {
  return token >= 0 && token < static_cast<int64_t>(rows) ? static_cast<uint32_t>(token) : rows;
}
__device__ __forceinline__ uint32_t key_of(const void* tokens, int bits, int64_t i,
                                           uint32_t rows) {
  return key_of(bits == 64 ? static_cast<const int64_t*>(tokens)[i]
                           : static_cast<int64_t>(static_cast<const int32_t*>(tokens)[i]), rows);
}

// ---------------------------------------------------------------------------
// 1. sort
// ---------------------------------------------------------------------------
// Digit counts of each block's share [b * share, (b + 1) * share) of the n keys.
__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(SortArgs a, int shift, int bins, int first,
                                                                  const uint32_t* keys) {
  __shared__ uint32_t hist[kMaxBins];
  const int tid = threadIdx.x;
  if (tid < kMaxBins) hist[tid] = 0;
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

// What a block needs to give its keys their places.
struct Places {
  uint32_t base[kMaxBins];               // next place of each digit
  uint32_t count[kSortWaves][kMaxBins];  // of a tile: each wave's first place of each digit
  uint32_t wave_total[kSortWaves];
};

// Exclusive scan of one value per digit (thread) over the block.
__device__ __forceinline__ uint32_t digit_scan(uint32_t v, Places& s) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t scan = v;
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t up = __shfl_up(scan, d, 64);
    if (lane >= d) scan += up;
  }
  if (lane == 63) s.wave_total[wave] = scan;
  __syncthreads();
  for (int w = 0; w < wave; ++w) scan += s.wave_total[w];
  return scan - v;
}

// The place of this thread's key in a tile of kSortThreads keys (in: it has one), in the
// order of threads within each digit.  Every thread of the block calls it.
__device__ __forceinline__ uint32_t place_of(bool in, uint32_t digit, int bins, Places& s) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  __syncthreads();  // the last tile's counts have been read
  if (tid < bins) {
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) s.count[w][tid] = 0;
  }
  __syncthreads();
  uint64_t same = __ballot(in);  // the lanes of this wave with the same digit
  for (int bit = 1; bit < bins; bit <<= 1) {
    const uint64_t with = __ballot((digit & bit) != 0);
    same &= (digit & bit) ? with : ~with;
  }
  const int rank = __popcll(same & ((1ull << lane) - 1));
  if (in && rank == 0) s.count[wave][digit] = static_cast<uint32_t>(__popcll(same));
  __syncthreads();
  if (tid < bins) {
    uint32_t at = s.base[tid];
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      const uint32_t c = s.count[w][tid];
      s.count[w][tid] = at;
      at += c;
    }
    s.base[tid] = at;
  }
  __syncthreads();
  return in ? s.count[wave][digit] + rank : 0;
}

// Stable scatter of each block's share to its digits' places.
__global__ __launch_bounds__(kSortThreads) void sort_scatter_kernel(
    SortArgs a, int shift, int bins, int first, const uint32_t* keys, const uint32_t* order,
    uint32_t* keys_out, uint32_t* order_out) {
  __shared__ Places s;
  const int tid = threadIdx.x;
  const int64_t lo = static_cast<int64_t>(blockIdx.x) * a.share;
  const int64_t hi = lo + a.share < a.n ? lo + a.share : a.n;
  // this block's first place for digit tid: all smaller digits, and this digit in earlier
  // blocks
  uint32_t before = 0, total = 0;
  if (tid < bins) {
#pragma unroll 8
    for (int b = 0; b < static_cast<int>(gridDim.x); ++b) {
      const uint32_t c = a.counts[static_cast<int64_t>(b) * bins + tid];
      before += b < static_cast<int>(blockIdx.x) ? c : 0;
      total += c;
    }
  }
  const uint32_t smaller = digit_scan(total, s);
  if (tid < bins) s.base[tid] = smaller + before;
  for (int64_t t0 = lo; t0 < hi; t0 += kSortThreads) {
    const int64_t i = t0 + tid;
    const bool in = i < hi;
    uint32_t k = 0, o = 0;
    if (in) {
      k = first ? key_of(a.tokens, a.token_bits, i, a.rows) : keys[i];
      o = first ? static_cast<uint32_t>(i) : order[i];
    }
    const uint32_t at = place_of(in, (k >> shift) & (bins - 1), bins, s);
    if (in) {
      keys_out[at] = k;
      order_out[at] = o;
    }
  }
}

// The whole sort of at most kOneLaunch tokens in one launch, and the rows' starts and ends.  The
// order of the rows is free, as long as a row's tokens stand together in their own order:
// block b takes the rows with b in their low bits.  Every block reads all tokens (from the
// L2), keeps its own in their order, sorts those by the other bits within its shared memory,
// and knows its first place from the number of tokens of the blocks before it.  8191 tokens
// take 9.7 us here and 23 us in the four kernels of two counted passes, 16384 tokens 18 and 27 us.
struct OneLaunch {
  uint32_t keys[kOneLaunch];      // of all tokens
  uint16_t order[2][kOneLaunch];  // of the block's own
  uint32_t base[kLocalBins];
  uint32_t count[kSortWaves][kLocalBins];
  uint32_t own[kSortWaves], before[kSortWaves];
};
__global__ __launch_bounds__(kSortThreads) void sort_one_launch_kernel(SortArgs a, int block_bits, int key_bits,
                                                                       uint32_t* keys_out, uint32_t* order_out,
                                                                       uint32_t* start, uint32_t* end) {
  __shared__ OneLaunch s;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, n = static_cast<int>(a.n);
  const uint32_t mine = blockIdx.x, low = (1u << block_bits) - 1;
  // a wave's share of the tokens: 64-token steps, in order
  const int steps = (n + kSortThreads - 1) / kSortThreads;
  uint32_t own = 0, before = 0;
  const auto read = [&](const auto* tokens) {
    constexpr int kBatch = 8;  // steps whose loads are issued together (clamped, not skipped)
    for (int k0 = 0; k0 < steps; k0 += kBatch) {
      int64_t t[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int i = (wave * steps + k0 + k) * 64 + lane;
        t[k] = tokens[i < n ? i : n - 1];
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int i = (wave * steps + k0 + k) * 64 + lane;
        if (k0 + k < steps && i < n) {
          const uint32_t key = key_of(t[k], a.rows);
          s.keys[i] = key;
          own += (key & low) == mine;
          before += (key & low) < mine;
        }
      }
    }
  };
  if (a.token_bits == 64) read(static_cast<const int64_t*>(a.tokens));
  else read(static_cast<const int32_t*>(a.tokens));
  for (int d = 32; d > 0; d >>= 1) {
    own += __shfl_xor(own, d, 64);
    before += __shfl_xor(before, d, 64);
  }
  if (lane == 0) {
    s.own[wave] = own;
    s.before[wave] = before;
  }
  __syncthreads();
  uint32_t first = 0, m = 0, at = 0;  // the block's first place and tokens, the wave's first
  for (int w = 0; w < kSortWaves; ++w) {
    first += s.before[w];
    if (w < wave) at += s.own[w];
    m += s.own[w];
  }
  for (int k = 0; k < steps; ++k) {
    const int i = (wave * steps + k) * 64 + lane;
    const bool keep = i < n && (s.keys[i] & low) == mine;
    const uint64_t kept = __ballot(keep);
    if (keep) s.order[0][at + __popcll(kept & ((1ull << lane) - 1))] = static_cast<uint16_t>(i);
    at += static_cast<uint32_t>(__popcll(kept));
  }
  int from = 0;
  for (int shift = block_bits; shift < key_bits; shift += kLocalBits, from ^= 1) {
    // stable scatter by one digit, as sort_scatter_kernel's
    if (tid < kLocalBins) s.base[tid] = 0;
    __syncthreads();
    for (uint32_t i = tid; i < m; i += kSortThreads)
      atomicAdd(&s.base[(s.keys[s.order[from][i]] >> shift) & (kLocalBins - 1)], 1u);
    __syncthreads();
    if (wave == 0) {  // kLocalBins digits, one a lane
      const uint32_t c = s.base[lane];
      uint32_t scan = c;
      for (int d = 1; d < 64; d <<= 1) {
        const uint32_t up = __shfl_up(scan, d, 64);
        if (lane >= d) scan += up;
      }
      s.base[lane] = scan - c;
    }
    for (uint32_t t0 = 0; t0 < m; t0 += kSortThreads) {
      const uint32_t i = t0 + tid;
      const bool in = i < m;
      const uint16_t o = in ? s.order[from][i] : 0;
      const uint32_t digit = in ? (s.keys[o] >> shift) & (kLocalBins - 1) : 0;
      s.count[wave][lane] = 0;  // the wave's own row
      uint64_t same = __ballot(in);
      for (int bit = 1; bit < kLocalBins; bit <<= 1) {
        const uint64_t with = __ballot((digit & bit) != 0);
        same &= (digit & bit) ? with : ~with;
      }
      const int rank = __popcll(same & ((1ull << lane) - 1));
      __builtin_amdgcn_wave_barrier();
      if (in && rank == 0) s.count[wave][digit] = static_cast<uint32_t>(__popcll(same));
      __syncthreads();
      if (tid < kLocalBins) {
        uint32_t next = s.base[tid];
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) {
          const uint32_t c = s.count[w][tid];
          s.count[w][tid] = next;
          next += c;
        }
        s.base[tid] = next;
      }
      __syncthreads();
      if (in) s.order[from ^ 1][s.count[wave][digit] + rank] = o;
      __syncthreads();
    }
  }
  __syncthreads();
  for (uint32_t i = tid; i < m; i += kSortThreads) {
    const uint32_t o = s.order[from][i], k = s.keys[o];
    keys_out[first + i] = k;
    order_out[first + i] = o;
    if (k >= a.rows) continue;
    if (i == 0 || s.keys[s.order[from][i - 1]] != k) start[k] = first + i;
    if (i == m - 1 || s.keys[s.order[from][i + 1]] != k) end[k] = first + i + 1;
  }
}

// ---------------------------------------------------------------------------
// 2. segments
// ---------------------------------------------------------------------------
// acc += the output rows of the tokens at sorted positions [lo, hi), columns [c, c + cnt), in
// order; kAhead rows are loaded before the first is added.
constexpr int kAhead = 8;
template <int T, int kUnit>
__device__ __forceinline__ void add_tokens(const RowArgs& a, uint32_t lo, uint32_t hi, int64_t c, int cnt,
                                           float (&acc)[kUnit]) {
  typedef typename Act<T>::S S;
  typedef typename Pack<S, kUnit>::type P;
  const S* dout = static_cast<const S*>(a.dout) + c;
  uint32_t i = lo;
  if (cnt >= kUnit) {
    // the next batch's positions are on their way while this batch's rows are
    uint32_t at[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) at[k] = i + k < hi ? a.order[i + k] : 0;
    for (; i < hi; i += kAhead) {
      P v[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (i + k < hi) v[k] = *reinterpret_cast<const P*>(dout + at[k] * a.dout_stride);
#pragma unroll
      for (int k = 0; k < kAhead; ++k) at[k] = i + kAhead + k < hi ? a.order[i + kAhead + k] : 0;
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (i + k < hi) {
#pragma unroll
          for (int e = 0; e < kUnit; ++e) acc[e] += Act<T>::up(v[k][e]);
        }
    }
    return;
  }
  for (; i < hi; ++i) {
    float v[kUnit];
    load_part<T, kUnit>(dout + a.order[i] * a.dout_stride, cnt, 0.0f, v);
#pragma unroll
    for (int e = 0; e < kUnit; ++e) acc[e] += v[e];
  }
}

// Block (j, slice): sorted positions [j chunk, (j + 1) chunk).  Slice 0 writes the segments'
// ends (ends: where the sort has not); every slice sums 64 units, one a lane, of the rows with
// more than `chunk` tokens, each wave a quarter of the tokens, joined in order.  At most two
// of those rows meet a chunk: the one at its first position (partial 2 j) and the one at its
// last (2 j + 1, where that is another row).
template <int T>
__global__ __launch_bounds__(kThreads) void segments_kernel(RowArgs a, int ends) {
  constexpr int kWaves = kThreads / 64;
  __shared__ float join[kWaves][kWide][64];
  const uint32_t n = static_cast<uint32_t>(a.n), chunk = static_cast<uint32_t>(a.chunk);
  const uint32_t lo = blockIdx.x * chunk, hi = lo + chunk < n ? lo + chunk : n;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (ends && blockIdx.y == 0)
    for (uint32_t i = lo + threadIdx.x; i < hi; i += kThreads) {
      const uint32_t k = a.keys[i];
      if (k >= a.rows) continue;
      if (i == 0 || a.keys[i - 1] != k) a.start[k] = i;
      if (i == n - 1 || a.keys[i + 1] != k) a.end[k] = i + 1;
    }
  const int64_t c = (static_cast<int64_t>(blockIdx.y) * 64 + lane) * kWide;
  const int cnt = static_cast<int>(a.dim - c);
  const auto sum = [&](uint32_t from, uint32_t to, int64_t slot) {
    const uint32_t part = (to - from + kWaves - 1) / kWaves, at = from + wave * part;
    float acc[kWide] = {};
    if (cnt > 0 && at < to) add_tokens<T, kWide>(a, at, at + part < to ? at + part : to, c, cnt, acc);
    __syncthreads();
#pragma unroll
    for (int e = 0; e < kWide; ++e) join[wave][e][lane] = acc[e];
    __syncthreads();
    if (wave != 0 || cnt <= 0) return;
#pragma unroll
    for (int e = 0; e < kWide; ++e)
      for (int w = 1; w < kWaves; ++w) acc[e] += join[w][e][lane];
    store_part<kActF32, kWide>(a.partial + slot * a.dim + c, cnt, acc);
  };
  // each wave counts on its own: the keys before, in and behind the chunk that are its first
  // or its last, a chunk at most on either side
  const uint32_t k0 = a.keys[lo], k1 = a.keys[hi - 1];
  uint32_t in0 = 0, in1 = 0, more0 = 0, more1 = 0;
  for (uint32_t i = lane; i < chunk; i += 64) {
    const uint32_t here = lo + i < hi ? a.keys[lo + i] : a.rows;
    const uint32_t after = hi + i < n ? a.keys[hi + i] : a.rows;
    const uint32_t before = lo > i ? a.keys[lo - 1 - i] : a.rows;
    in0 += here == k0;
    in1 += here == k1;
    more0 += (before == k0) + (after == k0);
    more1 += after == k1;
  }
  for (int d = 32; d > 0; d >>= 1) {
    in0 += __shfl_xor(in0, d, 64);
    in1 += __shfl_xor(in1, d, 64);
    more0 += __shfl_xor(more0, d, 64);
    more1 += __shfl_xor(more1, d, 64);
  }
  if (k0 < a.rows && in0 + more0 > chunk) sum(lo, lo + in0, 2 * static_cast<int64_t>(blockIdx.x));
  if (k1 != k0 && k1 < a.rows && in1 + more1 > chunk) sum(hi - in1, hi, 2 * static_cast<int64_t>(blockIdx.x) + 1);
}

// ---------------------------------------------------------------------------
// 3. rows
// ---------------------------------------------------------------------------
// Tokens of row v: their number, 0 if it does not occur; *s the first sorted position.
__device__ __forceinline__ uint32_t segment_of(const RowArgs& a, uint32_t v, uint32_t* s) {
  const uint32_t b = a.start[v], e = a.end[v];
  if (b >= a.n || a.keys[b] != v || (b > 0 && a.keys[b - 1] == v)) return 0;
  *s = b;
  return e - b;
}

// scale times the sum over the m tokens from sorted position s on (zeros for none).
template <int T>
__device__ __forceinline__ void row_gradient(const RowArgs& a, uint32_t s, uint32_t m, int64_t c, int cnt,
                                             float (&g)[kNarrow]) {
#pragma clang fp contract(off)
#pragma unroll
  for (int e = 0; e < kNarrow; ++e) g[e] = 0.0f;
  if (m == 0) return;
  if (m <= static_cast<uint32_t>(a.chunk)) {
    add_tokens<T, kNarrow>(a, s, s + m, c, cnt, g);
  } else {
    const int64_t j0 = s / a.chunk, j1 = (s + m - 1) / a.chunk;
    load_part<kActF32, kNarrow>(a.partial + (2 * j0 + (s % a.chunk != 0)) * a.dim + c, cnt, 0.0f, g);
#pragma unroll 4
    for (int64_t j = j0 + 1; j <= j1; ++j) {
      float v[kNarrow];
      load_part<kActF32, kNarrow>(a.partial + 2 * j * a.dim + c, cnt, 0.0f, v);
#pragma unroll
      for (int e = 0; e < kNarrow; ++e) g[e] += v[e];
    }
  }
#pragma unroll
  for (int e = 0; e < kNarrow; ++e) g[e] = a.scale * g[e];
}

// Unit u of a table: row u / units, columns from (u % units) N on.
template <int N>
struct Unit {
  uint32_t row, unit;
  __device__ __forceinline__ Unit(uint32_t u, int64_t dim) {
    const uint32_t units = static_cast<uint32_t>((dim + N - 1) / N);
    row = u / units;
    unit = u - row * units;
  }
  __device__ __forceinline__ int64_t column() const { return static_cast<int64_t>(unit) * N; }
};

// Streaming accesses of fp32 state: not read again before the caches are.
__device__ __forceinline__ void stream_in(const float* p, int cnt, float (&v)[kNarrow]) {
  typedef Pack<float, kNarrow>::type P;
  if (cnt >= kNarrow) {
    const P x = __builtin_nontemporal_load(reinterpret_cast<const P*>(p));
#pragma unroll
    for (int e = 0; e < kNarrow; ++e) v[e] = x[e];
  } else {
    load_part<kActF32, kNarrow>(p, cnt, 0.0f, v);
  }
}
__device__ __forceinline__ void stream_out(float* p, int cnt, const float (&v)[kNarrow]) {
  typedef Pack<float, kNarrow>::type P;
  if (cnt >= kNarrow) {
    P x;
#pragma unroll
    for (int e = 0; e < kNarrow; ++e) x[e] = v[e];
    __builtin_nontemporal_store(x, reinterpret_cast<P*>(p));
  } else {
    store_part<kActF32, kNarrow>(p, cnt, v);
  }
}

// kStore: grad = s sum on every row.  kAddRows, kAddTokens: grad += s sum on the rows that
// occur; a unit's row is a row of the table or that of a sorted position, whichever are
// fewer.  The product is rounded before it is added, so adding gives the bits of a separate
// gradient's addition.
enum GradMode { kStore = 0, kAddRows = 1, kAddTokens = 2 };
// The row of line `line` (a row, or in kAddTokens a sorted position), its first sorted position
// and its number of tokens; false where the line has nothing to do.
template <int kMode>
__device__ __forceinline__ bool line_of(const RowArgs& a, uint32_t line, uint32_t* v, uint32_t* s, uint32_t* m) {
  if (kMode == kAddTokens) {
    *s = line;
    *v = a.keys[line];
    if (*v >= a.rows || (line > 0 && a.keys[line - 1] == *v)) return false;
    *m = a.end[*v] - line;
    return true;
  }
  *v = line;
  *m = segment_of(a, line, s);
  return kMode == kStore || *m > 0;
}
template <int kMode>
__device__ __forceinline__ void put(float* to, int cnt, float (&g)[kNarrow]) {
  if (kMode == kStore) {
    stream_out(to, cnt, g);
    return;
  }
  float old[kNarrow];
  load_part<kActF32, kNarrow>(to, cnt, 0.0f, old);
#pragma unroll
  for (int e = 0; e < kNarrow; ++e) g[e] = old[e] + g[e];
  store_part<kActF32, kNarrow>(to, cnt, g);
}

template <int T, int kMode>
__global__ __launch_bounds__(kThreads) void grad_rows_kernel(RowArgs a, float* grad, uint32_t total) {
  const uint32_t u = blockIdx.x * kThreads + threadIdx.x;
  if (u >= total) return;
  const Unit<kNarrow> t(u, a.dim);
  uint32_t s = 0, m, v;
  if (!line_of<kMode>(a, t.row, &v, &s, &m)) return;
  const int64_t c = t.column();
  const int cnt = static_cast<int>(a.dim - c);
  float g[kNarrow];
  row_gradient<T>(a, s, m, c, cnt, g);
  put<kMode>(grad + v * a.dim + c, cnt, g);
}

// kStore where many rows of a wide table occur: a wave per tile of a row, so that the row's
// lookup is the wave's and each token's loads are two a lane.  65536 tokens by 128000 x 2048:
// 265 us against 336 us with a unit a thread; tiles of 256 columns take 326 us, of 1024 276 us.
// Where nearly all rows only need their zeros, the units' shorter stores are faster (8192 tokens
// by 82000 x 2048: 126 against 141 us), so a table takes this form from kTileTokens tokens per
// kTileRows rows on.  Two waves a block: with four, 274 and 148 us.
constexpr int kTile = 512;
constexpr int kTileThreads = 128;
constexpr int kTileTokens = 1, kTileRows = 4;
template <int T>
__global__ __launch_bounds__(kTileThreads) void grad_tiles_kernel(RowArgs a, float* grad) {
#pragma clang fp contract(off)
  typedef typename Act<T>::S S;
  constexpr int kParts = kTile / (64 * kNarrow);
  const int lane = threadIdx.x & 63;
  const uint32_t w = __builtin_amdgcn_readfirstlane(blockIdx.x * (kTileThreads / 64) + (threadIdx.x >> 6));
  const uint32_t tiles = static_cast<uint32_t>((a.dim + kTile - 1) / kTile);
  const uint32_t v = w / tiles;
  if (v >= a.rows) return;
  const int64_t c = static_cast<int64_t>(w - v * tiles) * kTile + lane * kNarrow;
  uint32_t s = 0;
  const uint32_t m = segment_of(a, v, &s);
  constexpr int64_t kNext = 64 * kNarrow;
  if (m > 0 && m <= static_cast<uint32_t>(a.chunk) && a.dim - c >= (kParts - 1) * kNext + kNarrow) {
    // the parts' loads together, in the order that add_tokens has for each of them
    typedef typename Pack<S, kNarrow>::type P;
    float g[kParts][kNarrow] = {};
    const S* dout = static_cast<const S*>(a.dout) + c;
    for (uint32_t i = s; i < s + m; i += kAhead) {
      P x[kAhead][kParts];
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        if (i + j < s + m) {
          const S* from = dout + a.order[i + j] * a.dout_stride;
#pragma unroll
          for (int k = 0; k < kParts; ++k) x[j][k] = *reinterpret_cast<const P*>(from + k * kNext);
        }
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        if (i + j < s + m) {
#pragma unroll
          for (int k = 0; k < kParts; ++k)
#pragma unroll
            for (int e = 0; e < kNarrow; ++e) g[k][e] += Act<T>::up(x[j][k][e]);
        }
    }
#pragma unroll
    for (int k = 0; k < kParts; ++k) {
#pragma unroll
      for (int e = 0; e < kNarrow; ++e) g[k][e] = a.scale * g[k][e];
      stream_out(grad + v * a.dim + c + k * kNext, kNarrow, g[k]);
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < kParts; ++k) {
    const int64_t ck = c + k * kNext;
    const int cnt = static_cast<int>(a.dim - ck);
    if (cnt <= 0) break;
    float g[kNarrow];
    row_gradient<T>(a, s, m, ck, cnt, g);
    stream_out(grad + v * a.dim + ck, cnt, g);
  }
}

// The AdamW update of every row; 24 bytes of state per value and the output rows of the tokens.
// 65536 x 1280 with 16384 tokens: 328 us of the call's 344 (6.2 TB/s; the AdamW kernel on a
// given gradient runs at 5.7).  The state's loads are issued before the row is looked up
// (359 us behind it); without the streaming accesses the call takes 386 us.
template <int T, int kMode>
__global__ __launch_bounds__(kThreads) void step_rows_kernel(RowArgs a, float* p, float* m, float* v,
                                                             AdamWConst c, uint32_t total) {
  const uint32_t u = blockIdx.x * kThreads + threadIdx.x;
  if (u >= total) return;
  const Unit<kNarrow> t(u, a.dim);
  const int64_t col = t.column(), at = t.row * a.dim + col;
  const int cnt = static_cast<int>(a.dim - col);
  float P[kNarrow], M[kNarrow], V[kNarrow], g[kNarrow];
  stream_in(p + at, cnt, P);
  stream_in(m + at, cnt, M);
  stream_in(v + at, cnt, V);
  uint32_t s = 0;
  const uint32_t count = segment_of(a, t.row, &s);
  row_gradient<T>(a, s, count, col, cnt, g);
#pragma unroll
  for (int e = 0; e < kNarrow; ++e) adamw_elem_t<kMode>(P[e], g[e], M[e], V[e], c);
  stream_out(p + at, cnt, P);
  stream_out(m + at, cnt, M);
  stream_out(v + at, cnt, V);
}

// ---------------------------------------------------------------------------
// Few tokens: no sort.  A block of the table's rows keeps the tokens of those rows, in order,
// in shared memory (most blocks have none), and its threads sum the ones of their row.  One
// launch: a step of 512 x 64 with 100 tokens takes 8 us where sort and step take 12, a dense
// gradient of 128000 x 2048 152 us (6.9 TB/s) where they take 169.
// ---------------------------------------------------------------------------
struct Few {
  uint32_t row[kDirect];
  uint32_t at[kDirect];
  uint32_t count[kThreads / 64];
};
// The tokens whose rows lie in [first, last].
__device__ __forceinline__ uint32_t find_tokens(const RowArgs& a, const void* tokens, int token_bits, uint32_t first,
                                                uint32_t last, Few& s) {
  static_assert(kThreads == kDirect && kDirect % kAhead == 0, "a token a thread");
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  uint32_t k = a.rows;
  if (tid < a.n) k = key_of(tokens, token_bits, tid, a.rows);
  const bool mine = k < a.rows && k >= first && k <= last;
  const uint64_t all = __ballot(mine);
  if (lane == 0) s.count[wave] = static_cast<uint32_t>(__popcll(all));
  s.row[tid] = a.rows;  // no row's, for readers of whole batches
  __syncthreads();
  uint32_t i = 0, found = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) {
    if (w < wave) i += s.count[w];
    found += s.count[w];
  }
  if (mine) {
    i += static_cast<uint32_t>(__popcll(all & ((1ull << lane) - 1)));
    s.row[i] = k;
    s.at[i] = static_cast<uint32_t>(tid);
  }
  __syncthreads();
  return found;
}
// Whether one of the found tokens [0, end) is of row v.
__device__ __forceinline__ bool among(const Few& s, uint32_t end, uint32_t v) {
  bool any = false;
  for (uint32_t b = 0; b < end; b += kAhead) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) any |= (b + k < end) & (s.row[b + k] == v);
  }
  return any;
}
// scale times the sum over the found tokens of row v, of which entry i is the first or one
// before it, in the tokens' order.  A gradient and a step of so few tokens both sum here, so
// they agree bit for bit; row_gradient's order is the same for rows of at most a chunk's tokens.
template <int T>
__device__ __forceinline__ void few_gradient(const RowArgs& a, const Few& s, uint32_t i, uint32_t found, uint32_t v,
                                             int64_t c, int cnt, float (&g)[kNarrow]) {
#pragma clang fp contract(off)
  typedef typename Act<T>::S S;
#pragma unroll
  for (int e = 0; e < kNarrow; ++e) g[e] = 0.0f;
  bool any = false;
  for (uint32_t b = i / kAhead * kAhead; b < found; b += kAhead) {
    uint32_t row[kAhead];
    float x[kAhead][kNarrow];
    bool some = false;
#pragma unroll
    for (int k = 0; k < kAhead; ++k) row[k] = s.row[b + k];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) some |= row[k] == v;
    if (!some) continue;
    any = true;
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (row[k] == v)
        load_part<T, kNarrow>(static_cast<const S*>(a.dout) + s.at[b + k] * a.dout_stride + c, cnt, 0.0f, x[k]);
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (row[k] == v) {
#pragma unroll
        for (int e = 0; e < kNarrow; ++e) g[e] += x[k][e];
      }
  }
  if (any) {
#pragma unroll
    for (int e = 0; e < kNarrow; ++e) g[e] = a.scale * g[e];
  }
}

template <int T, int kMode>
__global__ __launch_bounds__(kThreads) void few_grad_kernel(RowArgs a, const void* tokens, int token_bits, float* grad,
                                                            uint32_t total) {
  __shared__ Few s;
  const uint32_t u0 = blockIdx.x * kThreads, u = u0 + threadIdx.x;
  const uint32_t units = static_cast<uint32_t>((a.dim + kNarrow - 1) / kNarrow);
  uint32_t first = 0, last = a.rows - 1;
  if (kMode != kAddTokens) {
    first = u0 / units;
    last = ((total - u0 > kThreads ? u0 + kThreads : total) - 1) / units;
  }
  const uint32_t found = find_tokens(a, tokens, token_bits, first, last, s);
  if (u >= total) return;
  const Unit<kNarrow> t(u, a.dim);
  uint32_t v = t.row, i = 0;
  if (kMode == kAddTokens) {  // a line is one of the found tokens, the first of its row
    i = t.row;
    if (i >= found) return;
    v = s.row[i];
    if (among(s, i, v)) return;
  } else if (kMode == kAddRows) {
    if (!among(s, found, v)) return;
  }
  const int64_t c = t.column();
  const int cnt = static_cast<int>(a.dim - c);
  float g[kNarrow];
  few_gradient<T>(a, s, i, found, v, c, cnt, g);
  put<kMode>(grad + v * a.dim + c, cnt, g);
}

template <int T, int kMode>
__global__ __launch_bounds__(kThreads) void few_step_kernel(RowArgs a, const void* tokens, int token_bits, float* p,
                                                            float* m, float* v, AdamWConst c, uint32_t total) {
  __shared__ Few s;
  const uint32_t u0 = blockIdx.x * kThreads, u = u0 + threadIdx.x;
  const uint32_t units = static_cast<uint32_t>((a.dim + kNarrow - 1) / kNarrow);
  const Unit<kNarrow> t(u < total ? u : total - 1, a.dim);
  const int64_t col = t.column(), at = t.row * a.dim + col;
  const int cnt = static_cast<int>(a.dim - col);
  float P[kNarrow], M[kNarrow], V[kNarrow], g[kNarrow];
  stream_in(p + at, cnt, P);
  stream_in(m + at, cnt, M);
  stream_in(v + at, cnt, V);
  const uint32_t found = find_tokens(a, tokens, token_bits, u0 / units,
                                     ((total - u0 > kThreads ? u0 + kThreads : total) - 1) / units, s);
  if (u >= total) return;
  few_gradient<T>(a, s, 0, found, t.row, col, cnt, g);
#pragma unroll
  for (int e = 0; e < kNarrow; ++e) adamw_elem_t<kMode>(P[e], g[e], M[e], V[e], c);
  stream_out(p + at, cnt, P);
  stream_out(m + at, cnt, M);
  stream_out(v + at, cnt, V);
}

// ---------------------------------------------------------------------------
// lookup: bound by the rows' reads and writes (16384 tokens of 2048 columns to bf16: 25 us,
// 4.9 TB/s).  Units of eight columns: 25 us, of four 29 us.
// ---------------------------------------------------------------------------
template <int T>
__global__ __launch_bounds__(kThreads) void lookup_kernel(const float* table, uint32_t rows,
                                                          int64_t dim, const void* tokens,
                                                          int token_bits, uint32_t total, float scale,
                                                          typename Act<T>::S* out,
                                                          int64_t out_stride) {
  const uint32_t u = blockIdx.x * kThreads + threadIdx.x;
  if (u >= total) return;
  const Unit<kWide> t(u, dim);
  const int64_t c = t.column();
  const int cnt = static_cast<int>(dim - c);
  const uint32_t v = key_of(tokens, token_bits, t.row, rows);
  float x[kWide] = {};
  if (v < rows) {
    load_part<kActF32, kWide>(table + v * dim + c, cnt, 0.0f, x);
#pragma unroll
    for (int e = 0; e < kWide; ++e) x[e] *= scale;
  }
  store_part<T, kWide>(out + t.row * out_stride + c, cnt, x);
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
  if (rows < 1 || dim < 1 || n <= kDirect) return p;  // few tokens: no workspace
  // shares of two tiles, and at most 128 of them: each scatter block adds up all their counts
  p.share = 2 * kSortThreads;
  while ((n + p.share - 1) / p.share > 128) p.share *= 2;
  p.blocks = static_cast<int>((n + p.share - 1) / p.share);
  // at most 1024 partial sums to join for one row
  p.chunk = 32;
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
  at += up256(2 * p.chunks * dim * 4);
  p.bytes = at;
  return p;
}

static int64_t units_of(int64_t rows, int64_t dim, int unit) { return rows * ((dim + unit - 1) / unit); }

int64_t embedding_threads(int64_t rows, int64_t dim, int64_t n) {
  const EmbeddingPlan p = plan_embedding(rows, dim, n);
  return std::max(std::max(units_of(rows, dim, kNarrow), units_of(n, dim, kNarrow)), p.chunks * kThreads) + kThreads;
}

// Sorts the tokens and finds the segments; fills the arguments of stage 3.
static hipError_t sort_tokens(const EmbeddingCall& e, RowArgs* out, hipStream_t s) {
  *out = RowArgs{};
  out->rows = static_cast<uint32_t>(e.rows);
  out->dim = e.dim;
  out->dout = e.dout;
  out->dout_stride = e.dout_stride;
  out->n = e.n;
  out->scale = e.scale;
  if (e.n <= kDirect) return hipSuccess;
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
  uint32_t* start = reinterpret_cast<uint32_t*>(ws + p.start);
  uint32_t* end = reinterpret_cast<uint32_t*>(ws + p.end);
  const bool small = e.n <= kOneLaunch;  // else counted passes
  int last = 0;
  if (small) {
    // some 32 tokens a block, at most a block per CU (8191 tokens: 64 blocks 1.7 us slower)
    int bits = 1, block_bits = 0;
    while (bits < 32 && (sa.rows >> bits)) ++bits;
    while (block_bits < 8 && block_bits < bits && e.n >> (5 + block_bits)) ++block_bits;
    // and as many more as save a pass over the other bits
    const int spare = (bits - block_bits) % kLocalBits;
    if (block_bits + spare <= 8) block_bits += spare;
    hipLaunchKernelGGL(sort_one_launch_kernel, dim3(1u << block_bits), dim3(kSortThreads), 0, s, sa,
                       block_bits, bits, keys[0], order[0], start, end);
  } else {
    const dim3 grid(static_cast<unsigned>(p.blocks)), block(kSortThreads);
    for (int pass = 0; pass < passes; ++pass) {
      const int from = (pass + 1) & 1, to = pass & 1;
      hipLaunchKernelGGL(sort_count_kernel, grid, block, 0, s, sa, pass * width, 1 << width, pass == 0, keys[from]);
      hipLaunchKernelGGL(sort_scatter_kernel, grid, block, 0, s, sa, pass * width, 1 << width, pass == 0, keys[from],
                         order[from], keys[to], order[to]);
    }
    last = (passes - 1) & 1;
  }
  RowArgs a{};
  a.keys = keys[last];
  a.order = order[last];
  a.start = start;
  a.end = end;
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
    const int64_t slices = (units_of(1, e.dim, kWide) + 63) / 64;
    hipLaunchKernelGGL((segments_kernel<decltype(t)::value>), dim3(static_cast<unsigned>(p.chunks), static_cast<unsigned>(slices)),
                       dim3(kThreads), 0, s, a, small ? 0 : 1);
    return hipGetLastError();
  });
}

static dim3 unit_grid(int64_t units) { return dim3(static_cast<unsigned>((units + kThreads - 1) / kThreads)); }

hipError_t launch_embedding_forward(const float* table, int64_t rows, int64_t dim,
                                    const void* tokens, int token_bits, int64_t n, float scale,
                                    void* out, int out_type, int64_t out_stride, hipStream_t s) {
  return with_act(out_type, [&](auto t) {
    typedef typename Act<decltype(t)::value>::S S;
    const int64_t units = units_of(n, dim, kWide);
    hipLaunchKernelGGL((lookup_kernel<decltype(t)::value>), unit_grid(units), dim3(kThreads), 0, s, table,
                       static_cast<uint32_t>(rows), dim, tokens, token_bits, static_cast<uint32_t>(units), scale,
                       static_cast<S*>(out), out_stride);
    return hipGetLastError();
  });
}

hipError_t launch_embedding_backward(const EmbeddingCall& e, float* grad, bool add, hipStream_t s) {
  RowArgs a;
  const hipError_t st = sort_tokens(e, &a, s);
  if (st != hipSuccess) return st;
  return with_act(e.dout_type, [&](auto t) {
    constexpr int T = decltype(t)::value;
    if (!add && e.n > kDirect && e.dim >= kTile && e.n * kTileRows >= e.rows * kTileTokens) {
      const int64_t threads = e.rows * ((e.dim + kTile - 1) / kTile) * 64;
      hipLaunchKernelGGL((grad_tiles_kernel<T>), dim3(static_cast<unsigned>((threads + kTileThreads - 1) / kTileThreads)),
                         dim3(kTileThreads), 0, s, a, grad);
      return hipGetLastError();
    }
    const bool by_token = add && e.n < e.rows;
    const int64_t units = units_of(by_token ? e.n : e.rows, e.dim, kNarrow);
    const uint32_t total = static_cast<uint32_t>(units);
    if (e.n <= kDirect) {
      const void* tk = e.tokens;
      const int bits = e.token_bits;
      if (by_token) hipLaunchKernelGGL((few_grad_kernel<T, kAddTokens>), unit_grid(units), dim3(kThreads), 0, s, a, tk, bits, grad, total);
      else if (add) hipLaunchKernelGGL((few_grad_kernel<T, kAddRows>), unit_grid(units), dim3(kThreads), 0, s, a, tk, bits, grad, total);
      else hipLaunchKernelGGL((few_grad_kernel<T, kStore>), unit_grid(units), dim3(kThreads), 0, s, a, tk, bits, grad, total);
      return hipGetLastError();
    }
    if (by_token) hipLaunchKernelGGL((grad_rows_kernel<T, kAddTokens>), unit_grid(units), dim3(kThreads), 0, s, a, grad, total);
    else if (add) hipLaunchKernelGGL((grad_rows_kernel<T, kAddRows>), unit_grid(units), dim3(kThreads), 0, s, a, grad, total);
    else hipLaunchKernelGGL((grad_rows_kernel<T, kStore>), unit_grid(units), dim3(kThreads), 0, s, a, grad, total);
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
    const int64_t units = units_of(e.rows, e.dim, kNarrow);
    const dim3 grid = unit_grid(units), block(kThreads);
    const uint32_t total = static_cast<uint32_t>(units);
    const auto launch = [&](auto mode) {
      constexpr int kMode = decltype(mode)::value;
      if (e.n <= kDirect)
        hipLaunchKernelGGL((few_step_kernel<T, kMode>), grid, block, 0, s, a, e.tokens, e.token_bits, p, m, v, c, total);
      else
        hipLaunchKernelGGL((step_rows_kernel<T, kMode>), grid, block, 0, s, a, p, m, v, c, total);
    };
    switch (decay_mode(c)) {
      case kCoupled: launch(std::integral_constant<int, kCoupled>()); break;
      case kDecoupledCautious: launch(std::integral_constant<int, kDecoupledCautious>()); break;
      default: launch(std::integral_constant<int, kDecoupled>()); break;
    }
    return hipGetLastError();
  });
}

}  // namespace ma

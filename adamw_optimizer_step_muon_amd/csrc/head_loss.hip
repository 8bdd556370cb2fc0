// The LM head with its softmax cross entropy, without keeping the logits.
//
//   z = h W^T,  lse_r = log sum_v exp z_rv,  loss_r = lse_r - z_r,label
//   g = w_r (exp(z - lse) - [v = label]),  dh = g W,  dW = g^T h
//
// h: n hidden rows of D values, W: vocab x D, both of one type; labels outside the vocabulary mark
// rows without a target.  The logits of the forward pass live in registers, but where their sums are
// split (below): every tile of 256 rows x 256 vocabulary entries leaves its rows' maxima and sums of
// exponentials, which a second kernel joins.  The backward pass works through pieces of the
// vocabulary: a piece's logits are computed again, its g is written to the workspace in the hidden type
// (n x piece values), and two products take it to dh (a sum over pieces, fp32) and to the piece's rows
// of dW.
// Arithmetic: 2 n vocab D FLOP forward, 6 n vocab D with the gradients; the logits' second product,
// the price of not keeping them, makes it 8.  Both directions in one call keep the logits (fp32)
// where those of all rows take no more than the piece's 512 MiB and the product costs more than
// writing and reading them.
// Each product may have few tiles: its sum (over the hidden size, the piece or the rows) is then split
// over blocks, whose fp32 parts the next kernel adds in order.  Split logits are kept, in the forward pass
// too.
//
// Rows with a target (and, for gradients, a weight that is not zero) are gathered first into a
// padded copy, so the others cost nothing and whatever they hold reaches no result, and tiles need
// no checks along the rows.  Both directions in one call number and gather the rows once where logits
// are kept or one tile holds all rows; a row of weight 0 then goes on as zeros behind its loss.
//
// Rounding: products of 16-bit values are exact and summed in fp32.  g is rounded once to the
// hidden type, as the matrix cores take it, after a scaling by a power of two that takes the largest
// finite row weight to 2^14 or more: fp16 then keeps what is 2^-39 of that weight or more.  Every sum has
// a fixed order: the same inputs give the same bits.
// fp32 operands: up to kSplitRows rows on the fp32 matrix instructions; above as three bf16 planes
// each (x = x0 + x1 + x2 exactly: what two roundings to 8 bits leave of 24 fits the third), whose six
// products of 2^-16 and more run as one sum six times as long, the smallest first: the three that are
// left out are 2^-24 of the product together (2^-8 2^-17 twice, and less).
#include "gemm_tile.h"
#include "ma_act.h"
#include "ma_internal.h"

namespace ma {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;

// ---------------------------------------------------------------------------
// Rows: which of them take part, and their copies
// ---------------------------------------------------------------------------
// Planes of operands that the 16-bit tiles read: one, or three for fp32 values in bf16.
template <int T>
struct Planes {
  static constexpr int kCount = T == kActF32 ? 3 : 1;
  // four values into the planes at out, out + stride, ..
  static __device__ __forceinline__ void store(const float (&v)[4], unsigned short* out, int64_t stride) {
    float rest[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      unsigned short x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = f2bf(rest[e]);
        rest[e] -= bf2f(x[e]);
      }
      u32x2 w;
      w[0] = x[0] | (static_cast<unsigned>(x[1]) << 16);
      w[1] = x[2] | (static_cast<unsigned>(x[3]) << 16);
      *reinterpret_cast<u32x2*>(out + k * stride) = w;
    }
  }
};

// A row of dim values from `in` (null: zeros) to a padded row at `out`, as it is or in planes.  A wave.
template <int T, bool kPlanes>
__device__ __forceinline__ void head_copy_row(const typename Act<T>::S* in, void* out, int64_t at, int64_t plane,
                                              int64_t dim, int64_t dim_pad) {
  typedef typename Act<T>::S S;
  typedef typename Pack<S, 4>::type P;
  for (int64_t i = (threadIdx.x & 63) * 4; i < dim_pad; i += 256) {
    P x = 0;
    if (in) {
      if (i + 4 <= dim) {
        x = *reinterpret_cast<const P*>(in + i);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (i + e < dim) x[e] = in[i + e];
      }
    }
    if constexpr (kPlanes) {
      const float v[4] = {x[0], x[1], x[2], x[3]};
      Planes<T>::store(v, static_cast<unsigned short*>(out) + at + i, plane);
    } else {
      *reinterpret_cast<P*>(static_cast<S*>(out) + at + i) = x;
    }
  }
}

constexpr int kRowThreads = 1024;

// One block: numbers the live rows, and finds the scaling of their weights.  kCopy: gathers them too.
template <int T, bool kCopy>
__global__ __launch_bounds__(kRowThreads) void head_rows_kernel(HeadCall c) {
  constexpr int kWaves = kRowThreads / 64;
  __shared__ int counts[2][kWaves];
  __shared__ float tops[kWaves];
  __shared__ int copied[kCopy ? 64 : 1];
  const int t = threadIdx.x, wave = t >> 6;
  const auto label_of = [&](int64_t r) -> int64_t {
    return c.label_bits == 64 ? static_cast<const int64_t*>(c.labels)[r] : static_cast<const int32_t*>(c.labels)[r];
  };
  const auto in_vocab = [&](int64_t l) { return l >= 0 && l < c.vocab; };
  // the largest finite weight of a row with a target
  float top = 0.0f;
  if (c.row_weight) {
#pragma unroll 4
    for (int64_t r = t; r < c.n; r += kRowThreads)
      if (in_vocab(label_of(r))) {
        const float w = fabsf(c.row_weight[r]);
        top = fmaxf(top, w < INFINITY ? w : 0.0f);
      }
    top = wave_max(top);
    if ((t & 63) == 0) tops[wave] = top;
    __syncthreads();
    for (int w = 0; w < kWaves; ++w) top = fmaxf(top, tops[w]);
  }
  // weights are scaled by the power of two that takes the largest into [2^14, 2^15) (then g of an
  // unlikely label, nearly the weight itself, stays within fp16), or by 2^126, whose inverse is a normal
  // number; fp32 needs no scaling
  const int exponent = static_cast<int>(__builtin_bit_cast(uint32_t, top) >> 23) - 127;
  const int shift = T != kActF32 && top > 0.0f ? (exponent < -112 ? 126 : 14 - exponent) : 0;
  int base = 0, turn = 0;
  for (int64_t first = 0; first < c.n; first += kRowThreads, turn ^= 1) {
    const int64_t r = first + t, label = r < c.n ? label_of(r) : -1;
    const float given = c.row_weight && r < c.n ? c.row_weight[r] : 1.0f;
    // (rows that are numbered once, for the loss too, by the labels alone)
    const bool live = in_vocab(label) && (c.once || given != 0.0f);
    const unsigned long long mask = __ballot(live);
    if ((t & 63) == 0) counts[turn][wave] = __popcll(mask);
    __syncthreads();
    int at = base + __popcll(mask & ((1ull << (t & 63)) - 1));
    for (int w = 0; w < kWaves; ++w) {
      if (w < wave) at += counts[turn][w];
      base += counts[turn][w];
    }
    if (r >= c.n) continue;
    if (!live) {
      c.place[r] = -1;
      if (c.lse_out) c.lse_out[r] = 0.0f;
      if (c.loss) c.loss[r] = 0.0f;
      continue;
    }
    c.place[r] = at;
    c.row_of[at] = static_cast<int>(r);
    c.label[at] = static_cast<int>(label);
    if (c.row_weight) {
      const float w = __builtin_ldexpf(given, shift);
      c.weight[at] = w;
      if (!c.once) {
        // exp(z - top) factor = weight exp(z - lse)
        c.top[at] = c.lse_in ? c.lse_in[r] : c.tops[r];
        c.factor[at] = c.lse_in ? w : w / c.sums[r];
      }
    }
    if constexpr (kCopy) copied[at] = static_cast<int>(r);
  }
  if (t == 0) {
    c.head->live = base;
    c.head->unscale = __builtin_ldexpf(1.0f, -shift);
  }
  if constexpr (kCopy) {
    typedef typename Act<T>::S S;
    typedef typename Pack<S, 4>::type P;
    __syncthreads();
    const int padded = (base + c.row_tile - 1) / c.row_tile * c.row_tile, each = static_cast<int>(c.dim_pad / 4);
#pragma unroll 4
    for (int x = t; x < padded * each; x += kRowThreads) {
      const int row = x / each, i = (x - row * each) * 4, from = row < base ? copied[row] : -1;
      P v = 0;
      if (from >= 0) {
        const S* in = static_cast<const S*>(c.hidden) + from * c.hidden_stride + i;
        if (i + 4 <= c.dim) {
          v = *reinterpret_cast<const P*>(in);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (i + e < c.dim) v[e] = in[e];
        }
      }
      *reinterpret_cast<P*>(static_cast<S*>(c.hidden_pad) + row * c.dim_pad + i) = v;
    }
  }
}

// The live rows' padded copies (dim_pad values, zeros behind dim), and zero rows behind the last up
// to a whole tile.  A wave per row.
template <int T, bool kPlanes>
__global__ __launch_bounds__(256) void head_gather_kernel(HeadCall c) {
  const int64_t at = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  const int live = c.head->live;
  if (at >= (live + c.row_tile - 1) / c.row_tile * static_cast<int64_t>(c.row_tile)) return;
  const auto* in = at < live ? static_cast<const typename Act<T>::S*>(c.hidden) + c.row_of[at] * c.hidden_stride : nullptr;
  head_copy_row<T, kPlanes>(in, c.hidden_pad, at * c.dim_pad, c.hidden_plane, c.dim, c.dim_pad);
}

// W in rows of dim_pad values: rows that are not aligned to 16 bytes, or fp32's planes.  A wave per
// row.
template <int T, bool kPlanes>
__global__ __launch_bounds__(256) void head_weight_kernel(HeadCall c) {
  const int64_t v = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (v >= c.vocab) return;
  head_copy_row<T, kPlanes>(static_cast<const typename Act<T>::S*>(c.weight_in) + v * c.weight_in_stride, c.weight_pad,
                                 v * c.dim_pad, c.weight_plane, c.dim, c.dim_pad);
}

// dW of no rows at all.  A wave per row.
__global__ __launch_bounds__(256) void head_clear_kernel(HeadCall c) {
  const int lane = threadIdx.x & 63;
  const int64_t v = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (v >= c.vocab) return;
  if (c.dweight_type == kActF32) {
    for (int64_t i = lane; i < c.dim; i += 64) static_cast<float*>(c.dweight)[v * c.dweight_stride + i] = 0.0f;
  } else {
    for (int64_t i = lane; i < c.dim; i += 64) static_cast<unsigned short*>(c.dweight)[v * c.dweight_stride + i] = 0;
  }
}

// A row's loss and lse, and what the backward pass takes from its largest logit and its sum: a wave,
// whose lanes have the same values.
__device__ __forceinline__ void head_row_done(const HeadCall& c, int64_t at, float top, float sum, float target) {
  const int lane = threadIdx.x & 63, r = c.row_of[at];
  const float log_sum = logf(sum);
  if (lane == 0) {
    if (c.loss) c.loss[r] = (top - target) + log_sum;
    if (c.lse_out) c.lse_out[r] = top + log_sum;
    if (c.tops) {
      c.tops[r] = top;
      c.sums[r] = sum;
    }
  }
  if (!c.once) return;
  const float w = c.weight[at];
  if (lane == 0) {
    c.top[at] = w == 0.0f ? 0.0f : top;
    c.factor[at] = w == 0.0f ? 0.0f : w / sum;
  }
  if (w != 0.0f) return;
  // a row without a gradient goes on as zeros, whatever it holds
  const int size = c.type == kActF32 && !c.planes ? 4 : 2;
  for (int plane = 0; plane < (c.planes ? 3 : 1); ++plane) {
    char* out = static_cast<char*>(c.hidden_pad) + (plane * c.hidden_plane + at * c.dim_pad) * size;
    for (int64_t i = lane * 4; i < c.dim_pad * size; i += 256) *reinterpret_cast<unsigned*>(out + i) = 0;
  }
}

// Joins the tiles' maxima and sums of a row.  A wave per live row.
__global__ __launch_bounds__(256) void head_join_kernel(HeadCall c) {
  const int lane = threadIdx.x & 63;
  const int64_t at = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (at >= c.head->live) return;
  const float2* part = c.partial + at * c.tiles;
  float top = -INFINITY;
  for (int64_t i = lane; i < c.tiles; i += 64) top = fmaxf(top, part[i].x);
  top = wave_max(top);
  const float base = top == -INFINITY ? 0.0f : top;
  float sum = 0.0f;
  for (int64_t i = lane; i < c.tiles; i += 64) {
    const float2 p = part[i];
    // a tile of -inf alone has no share
    sum += p.x == -INFINITY ? p.y : p.y * __builtin_amdgcn_exp2f((p.x - base) * kLog2e);
  }
  head_row_done(c, at, top, wave_sum(sum), c.target[at]);
}

// The same from logits whose sums are split over blocks.  A block per live row.
__global__ __launch_bounds__(256) void head_stats_kernel(HeadCall c) {
  __shared__ float tops[4], sums[4], target;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t at = blockIdx.x;
  if (at >= c.head->live) return;
  const float* z = c.z + at * c.g_stride;
  const int64_t label = c.label[at];
  float top = -INFINITY, sum = 0.0f;
  for (int64_t col = threadIdx.x * 4; col < c.vocab; col += 1024) {
    f32x4 v = *reinterpret_cast<const f32x4*>(z + col);
#pragma unroll 4
    for (int s = 1; s < c.logit_splits; ++s) v += *reinterpret_cast<const f32x4*>(z + s * c.z_plane + col);
    float most = top;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (col + e < c.vocab) most = fmaxf(most, v[e]);
    const float base = most == -INFINITY ? 0.0f : most;
    if (top != -INFINITY) sum *= __builtin_amdgcn_exp2f((top - base) * kLog2e);
    top = most;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (col + e < c.vocab) sum += __builtin_amdgcn_exp2f((v[e] - base) * kLog2e);
      if (col + e == label) target = v[e];
    }
  }
  const float wave_top = wave_max(top), b = wave_top == -INFINITY ? 0.0f : wave_top;
  // a thread of -inf alone has no share
  sum = wave_sum(top == -INFINITY ? sum : sum * __builtin_amdgcn_exp2f((top - b) * kLog2e));
  if (lane == 0) {
    tops[wave] = wave_top;
    sums[wave] = sum;
  }
  __syncthreads();
  if (wave != 0) return;
  top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
  const float base = top == -INFINITY ? 0.0f : top;
  sum = 0.0f;
  for (int w = 0; w < 4; ++w) sum += tops[w] == -INFINITY ? sums[w] : sums[w] * __builtin_amdgcn_exp2f((tops[w] - base) * kLog2e);
  head_row_done(c, at, top, sum, target);
}

// g from kept logits, 8 values a thread; a block takes 2048 columns of a row.
template <int T, bool kPlanes>
__global__ __launch_bounds__(256) void head_convert_kernel(HeadCall c) {
  const int64_t at = blockIdx.y, col = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 8;
  const int live = c.head->live;
  if (at >= (live + c.row_tile - 1) / c.row_tile * static_cast<int64_t>(c.row_tile) || col >= c.piece) return;
  const bool on = at < live;
  const float top = on ? c.top[at] : 0.0f, factor = on ? c.factor[at] : 0.0f, weight = on ? c.weight[at] : 0.0f;
  const int64_t label = on ? c.label[at] : -1;
  const float* in = c.z + at * c.g_stride + col;
  float g[8];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    f32x4 z = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(in + 4 * h));
#pragma unroll 4
    for (int s = 1; s < c.logit_splits; ++s)
      z += __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(in + s * c.z_plane + 4 * h));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int64_t v = col + 4 * h + e;
      const float p = __builtin_amdgcn_exp2f((z[e] - top) * kLog2e);
      g[4 * h + e] = __builtin_fmaf(p, factor, v == label ? -weight : 0.0f);
      if (v >= c.vocab || weight == 0.0f) g[4 * h + e] = 0.0f;
    }
  }
  const int64_t out = at * c.g_stride + col;
  if constexpr (T == kActF32 && !kPlanes) {
    // in place
    float* p = static_cast<float*>(c.g) + out;
#pragma unroll
    for (int h = 0; h < 2; ++h) *reinterpret_cast<f32x4*>(p + 4 * h) = f32x4{g[4 * h], g[4 * h + 1], g[4 * h + 2], g[4 * h + 3]};
  } else {
#pragma unroll
    for (int plane = 0; plane < (kPlanes ? 3 : 1); ++plane) {
      u32x4 w;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        unsigned short x[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float& v = g[2 * k + e];
          if constexpr (kPlanes) {
            x[e] = f2bf(v);
            v -= bf2f(x[e]);
          } else {
            x[e] = Act<T>::down(v);
          }
        }
        w[k] = x[0] | (static_cast<unsigned>(x[1]) << 16);
      }
      *reinterpret_cast<u32x4*>(static_cast<unsigned short*>(c.g) + plane * c.g_plane + out) = w;
    }
  }
}

// dh from the sums of the splits, a wave per 256 columns of a row; rows without a gradient are zero.
template <int T>
__global__ __launch_bounds__(256) void head_out_kernel(HeadCall c) {
  typedef typename Act<T>::S S;
  const int lane = threadIdx.x & 63;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (r >= c.n) return;
  S* out = static_cast<S*>(c.dhidden) + r * c.dhidden_stride;
  const int at = c.place[r];
  const float unscale = c.head->unscale;
  const int64_t i = static_cast<int64_t>(blockIdx.y) * 256 + lane * 4;
  if (i >= c.dim) return;
  const int cnt = c.dim - i < 4 ? static_cast<int>(c.dim - i) : 4;
  float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (at >= 0 && c.weight[at] != 0.0f) {
#pragma unroll 8
    for (int s = 0; s < c.splits; ++s) {
      const f32x4 x = *reinterpret_cast<const f32x4*>(c.sum + (s * c.rows_pad + at) * c.sum_stride + i);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += x[e];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] *= unscale;
  }
  store_part<T, 4>(out + i, cnt, v);
}

// The piece's rows of dW from the sums of the splits, a wave per 256 columns of a row.
template <int T>
__global__ __launch_bounds__(256) void head_weight_out_kernel(HeadCall c) {
  const int lane = threadIdx.x & 63;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6), v = c.piece_start + row;
  const int64_t i = static_cast<int64_t>(blockIdx.y) * 256 + lane * 4;
  if (row >= c.piece || v >= c.vocab || i >= c.dim) return;
  const float unscale = c.head->unscale;
  const int cnt = c.dim - i < 4 ? static_cast<int>(c.dim - i) : 4;
  float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
  for (int s = 0; s < c.weight_splits; ++s) {
    const f32x4 y = *reinterpret_cast<const f32x4*>(c.weight_sum + (s * c.piece + row) * c.sum_stride + i);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] += y[e];
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] *= unscale;
  const int64_t at = v * c.dweight_stride + i;
  if (T == kActF32 || c.dweight_type == kActF32) {
    float* p = static_cast<float*>(c.dweight) + at;
    if (c.add) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < cnt) x[e] += p[e];
    }
    store_part<kActF32, 4>(p, cnt, x);
  } else {
    store_part<T, 4>(static_cast<typename Act<T>::S*>(c.dweight) + at, cnt, x);
  }
}

// ---------------------------------------------------------------------------
// Tiles
// ---------------------------------------------------------------------------
// What a tile computes: the rows' statistics, g, the sum dh, or rows of dW.
enum HeadMode { kStats = 0, kGrad = 1, kHidden = 2, kWeight = 3 };

// Blocks go round-robin to the 8 XCDs: each XCD takes a contiguous run of tiles, whose operands its
// L2 then shares.  Logits: bands of 4 vocabulary tiles, all rows of a band after each other; the
// others: all columns of a row tile after each other.  False for blocks behind the last tile.
__device__ __forceinline__ bool head_tile(int mode, int mt, int nt, int splits, int& m, int& n, int& split) {
  const int tiles = mt * nt * splits;
  const int per = (tiles + 7) / 8, b = static_cast<int>(blockIdx.x);
  const int t = (b & 7) * per + (b >> 3);
  if ((b >> 3) >= per || t >= tiles) return false;
  // (integer divisions run on the vector unit: taken back to scalars, the operands' addresses are
  // made by scalar instructions)
  split = splits > 1 ? t / (mt * nt) : 0;
  const int here = t - split * mt * nt;
  if (mode == kStats || mode == kGrad) {
    const int band = here / (4 * mt), rest = here - band * 4 * mt, left = nt - band * 4, width = left < 4 ? left : 4;
    m = rest / width;
    n = band * 4 + rest % width;
  } else {
    n = here % nt;
    m = here / nt;
  }
  m = __builtin_amdgcn_readfirstlane(m);
  n = __builtin_amdgcn_readfirstlane(n);
  split = __builtin_amdgcn_readfirstlane(split);
  return true;
}

// Accumulators of a wave: tile i of 32 rows, tile j of 32 columns; the lane holds row (lane & 31)
// and columns 8 q + 4 (lane / 32) + e in element 4 q + e.
template <int T, bool kPlanes, int kMode, int BM, int BN, int WM, int WN, int WTM, int WTN>
__device__ __forceinline__ void head_epilogue(const HeadCall& c, const f32x16 (&acc)[WTM][WTN], int m0, int n0, int split,
                                              int live, char* smem) {
  typedef typename Act<T>::S S;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN, frow = lane & 31, half = lane >> 5;
  const int row0 = wm * (WTM * 32) + frow, col0 = wn * (WTN * 32) + 4 * half;
  if constexpr (kMode == kStats) {
    if (c.logit_splits > 1) {
      float* z = c.z + split * c.z_plane + static_cast<int64_t>(m0 + row0) * c.g_stride + n0 + col0;
#pragma unroll
      for (int i = 0; i < WTM; ++i)
#pragma unroll
        for (int j = 0; j < WTN; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<f32x4*>(z + i * 32 * c.g_stride + j * 32 + 8 * q) =
                f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
      return;
    }
    float2* shared = reinterpret_cast<float2*>(smem);  // [WN][BM]
    const int count = c.vocab - n0 < BN ? static_cast<int>(c.vocab - n0) : BN;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < WTM; ++i) {
      const int row = row0 + i * 32;
      // few waves meet a label among their columns
      const int label = m0 + row < live ? c.label[m0 + row] - n0 - wn * (WTN * 32) : -1;
      if (__any(label >= 0 && label < WTN * 32)) {
#pragma unroll
        for (int j = 0; j < WTN; ++j)
#pragma unroll
          for (int k = 0; k < 16; ++k)
            if (j * 32 + 4 * half + 8 * (k >> 2) + (k & 3) == label) c.target[m0 + row] = acc[i][j][k];
      }
      if (c.kept) {
        float* z = c.z + static_cast<int64_t>(m0 + row) * c.g_stride + n0 + col0;
#pragma unroll
        for (int j = 0; j < WTN; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<f32x4*>(z + j * 32 + 8 * q) =
                f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
      }
      float top = -INFINITY, sum = 0.0f, base;
      const auto gather = [&](auto mask) {  // mask: the vocabulary ends within this tile
        constexpr bool kMask = decltype(mask)::value;
#pragma unroll
        for (int j = 0; j < WTN; ++j)
#pragma unroll
          for (int k = 0; k < 16; ++k)
            if (!kMask || col0 + j * 32 + 8 * (k >> 2) + (k & 3) < count) top = fmaxf(top, acc[i][j][k]);
        base = top == -INFINITY ? 0.0f : top;
#pragma unroll
        for (int j = 0; j < WTN; ++j)
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float e = __builtin_amdgcn_exp2f((acc[i][j][k] - base) * kLog2e);
            sum += !kMask || col0 + j * 32 + 8 * (k >> 2) + (k & 3) < count ? e : 0.0f;
          }
      };
      if (count < BN) gather(std::true_type{});
      else gather(std::false_type{});
      // the other half of the columns
      const float top2 = __shfl_xor(top, 32, 64), sum2 = __shfl_xor(sum, 32, 64);
      const float both = fmaxf(top, top2), b = both == -INFINITY ? 0.0f : both;
      sum = (top == -INFINITY ? sum : sum * __builtin_amdgcn_exp2f((top - b) * kLog2e)) +
            (top2 == -INFINITY ? sum2 : sum2 * __builtin_amdgcn_exp2f((top2 - b) * kLog2e));
      if (half == 0) shared[wn * BM + row] = make_float2(both, sum);
    }
    __syncthreads();
    for (int row = threadIdx.x; row < BM; row += 64 * WM * WN) {
      if (m0 + row >= live) break;
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < WN; ++w) top = fmaxf(top, shared[w * BM + row].x);
      const float b = top == -INFINITY ? 0.0f : top;
      float sum = 0.0f;
#pragma unroll
      for (int w = 0; w < WN; ++w) {
        const float2 p = shared[w * BM + row];
        sum += p.x == -INFINITY ? p.y : p.y * __builtin_amdgcn_exp2f((p.x - b) * kLog2e);
      }
      c.partial[static_cast<int64_t>(m0 + row) * c.tiles + n0 / BN] = make_float2(top, sum);
    }
  } else if constexpr (kMode == kGrad) {
    // n0 counts from the piece's first entry
    const int64_t left = c.vocab - c.piece_start - n0;
    const int count = left < BN ? static_cast<int>(left) : BN;
    constexpr bool kStaged = kPlanes || T != kActF32;
    if constexpr (kStaged) __syncthreads();
#pragma unroll
    for (int i = 0; i < WTM; ++i) {
      const int row = row0 + i * 32;
      // a padded row's logits are zeros, and so is its factor
      const bool on = m0 + row < live;
      const float top = on ? c.top[m0 + row] : 0.0f, factor = on ? c.factor[m0 + row] : 0.0f;
      const int label = on ? static_cast<int>(c.label[m0 + row] - c.piece_start) - n0 - wn * (WTN * 32) : -1;
      float g[WTN][16];
#pragma unroll
      for (int j = 0; j < WTN; ++j)
#pragma unroll
        for (int k = 0; k < 16; ++k) g[j][k] = factor * __builtin_amdgcn_exp2f((acc[i][j][k] - top) * kLog2e);
      if (__any(label >= 0 && label < WTN * 32)) {
        const float weight = on ? c.weight[m0 + row] : 0.0f;
#pragma unroll
        for (int j = 0; j < WTN; ++j)
#pragma unroll
          for (int k = 0; k < 16; ++k)
            if (j * 32 + 4 * half + 8 * (k >> 2) + (k & 3) == label)
              g[j][k] = __builtin_fmaf(__builtin_amdgcn_exp2f((acc[i][j][k] - top) * kLog2e), factor, -weight);
      }
      if (count < BN) {
#pragma unroll
        for (int j = 0; j < WTN; ++j)
#pragma unroll
          for (int k = 0; k < 16; ++k)
            if (col0 + j * 32 + 8 * (k >> 2) + (k & 3) >= count) g[j][k] = 0.0f;
      }
      // nothing comes of a row without a gradient, also where its zeros meet an infinity of W
      const bool none = !on || (factor == 0.0f && c.weight[m0 + row] == 0.0f);
      if (__any(none)) {
#pragma unroll
        for (int j = 0; j < WTN; ++j)
#pragma unroll
          for (int k = 0; k < 16; ++k) g[j][k] = none ? 0.0f : g[j][k];
      }
      if constexpr (!kStaged) {
        float* out = static_cast<float*>(c.g) + static_cast<int64_t>(m0 + row) * c.g_stride + n0 + col0;
#pragma unroll
        for (int j = 0; j < WTN; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<f32x4*>(out + j * 32 + 8 * q) = f32x4{g[j][4 * q], g[j][4 * q + 1], g[j][4 * q + 2], g[j][4 * q + 3]};
      } else {
        // a wave stages its 32 rows of 64 columns, chunks of 16 bytes XOR-ed with the row, so that
        // whole 128-byte lines leave
        static_assert(WTN % 2 == 0, "eight chunks a row");
        char* stage = smem + wave * (32 * 128);
#pragma unroll
        for (int plane = 0; plane < (kPlanes ? 3 : 1); ++plane)
#pragma unroll
          for (int part = 0; part < WTN / 2; ++part) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                unsigned short x[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  float& v = g[2 * part + j][4 * q + e];
                  if constexpr (kPlanes) {
                    x[e] = f2bf(v);
                    v -= bf2f(x[e]);
                  } else {
                    x[e] = Act<T>::down(v);
                  }
                }
                u32x2 w;
                w[0] = x[0] | (static_cast<unsigned>(x[1]) << 16);
                w[1] = x[2] | (static_cast<unsigned>(x[3]) << 16);
                *reinterpret_cast<u32x2*>(stage + frow * 128 + (((j * 4 + q) ^ (frow & 7)) << 4) + half * 8) = w;
              }
            unsigned short* out = static_cast<unsigned short*>(c.g) + plane * c.g_plane + n0 + wn * (WTN * 32) + part * 64;
#pragma unroll
            for (int it = 0; it < 4; ++it) {
              const int r = it * 8 + (lane >> 3), ch = lane & 7;
              const u32x4 x = *reinterpret_cast<const u32x4*>(stage + r * 128 + ((ch ^ (r & 7)) << 4));
              *reinterpret_cast<u32x4*>(out + static_cast<int64_t>(m0 + wm * (WTM * 32) + i * 32 + r) * c.g_stride + ch * 8) = x;
            }
          }
      }
    }
  } else if constexpr (kMode == kHidden) {
    float* out = c.sum + (static_cast<int64_t>(split) * c.rows_pad + m0) * c.sum_stride;
#pragma unroll
    for (int i = 0; i < WTM; ++i)
#pragma unroll
      for (int j = 0; j < WTN; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int col = n0 + col0 + j * 32 + 8 * q;
          if (col >= c.sum_stride) continue;  // a multiple of 4
          f32x4* p = reinterpret_cast<f32x4*>(out + static_cast<int64_t>(row0 + i * 32) * c.sum_stride + col);
          f32x4 x = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
          if (!c.first) x += *p;
          *p = x;
        }
  } else if (c.weight_splits > 1) {
    float* out = c.weight_sum + (split * c.piece + m0) * c.sum_stride;
#pragma unroll
    for (int i = 0; i < WTM; ++i)
#pragma unroll
      for (int j = 0; j < WTN; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int col = n0 + col0 + j * 32 + 8 * q;
          if (col < c.sum_stride)
            *reinterpret_cast<f32x4*>(out + static_cast<int64_t>(row0 + i * 32) * c.sum_stride + col) =
                f32x4{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
        }
  } else if (T != kActF32 && c.weight_lines) {
    // rows of dW that start at multiples of 16 bytes leave in whole lines, as g does
    if constexpr (T != kActF32) {
      const float unscale = c.head->unscale;
      char* stage = smem + wave * (32 * 128);
      __syncthreads();
#pragma unroll
      for (int i = 0; i < WTM; ++i)
#pragma unroll
        for (int part = 0; part < WTN / 2; ++part) {
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              u32x2 w;
#pragma unroll
              for (int e = 0; e < 2; ++e)
                w[e] = Act<T>::down(acc[i][2 * part + j][4 * q + 2 * e] * unscale) |
                       (static_cast<unsigned>(Act<T>::down(acc[i][2 * part + j][4 * q + 2 * e + 1] * unscale)) << 16);
              *reinterpret_cast<u32x2*>(stage + frow * 128 + (((j * 4 + q) ^ (frow & 7)) << 4) + half * 8) = w;
            }
#pragma unroll
          for (int it = 0; it < 4; ++it) {
            const int r = it * 8 + (lane >> 3), ch = lane & 7, col = n0 + wn * (WTN * 32) + part * 64 + ch * 8;
            const int64_t v = c.piece_start + m0 + wm * (WTM * 32) + i * 32 + r;
            const u32x4 x = *reinterpret_cast<const u32x4*>(stage + r * 128 + ((ch ^ (r & 7)) << 4));
            if (v < c.vocab && col < c.dim)
              *reinterpret_cast<u32x4*>(static_cast<S*>(c.dweight) + v * c.dweight_stride + col) = x;
          }
        }
    }
  } else {
    const float unscale = c.head->unscale;
#pragma unroll
    for (int i = 0; i < WTM; ++i) {
      const int64_t v = c.piece_start + m0 + row0 + i * 32;
      if (v >= c.vocab) continue;
#pragma unroll
      for (int j = 0; j < WTN; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int col = n0 + col0 + j * 32 + 8 * q;
          const int cnt = c.dim - col < 4 ? static_cast<int>(c.dim - col) : 4;
          if (cnt <= 0) continue;
          float x[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = acc[i][j][4 * q + e] * unscale;
          const int64_t at = v * c.dweight_stride + col;
          if (T == kActF32 || c.dweight_type == kActF32) {
            float* p = static_cast<float*>(c.dweight) + at;
            if (c.add) {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (e < cnt) x[e] += p[e];
            }
            store_part<kActF32, 4>(p, cnt, x);
          } else {
            store_part<T, 4>(static_cast<S*>(c.dweight) + at, cnt, x);
          }
        }
    }
  }
}

// 16-bit operands (or planes of them): BM x 256 tiles of 8 waves (2 x 4), v_mfma_f32_32x32x16, stages
// of 64 of the summed index, loaded straight into LDS.  Operands are contiguous along that index (hidden rows and
// W in the logits, g in dh) or across it (W in dh; g and the hidden rows in dW), which the
// transposing LDS reads take, so nothing is stored twice.  The accumulators hold a row a lane
// (operands passed to the matrix instruction the other way round), so a row's maximum and sum
// need two lanes and four waves only.
// LDS rings: 3 stages of A and 2 of B for 256 rows (160 KiB), 3 and 3 for 128, 4 and 4 for 64, whose
// short stages are bound by the loads' latency.
// Measured: the logits of 8192 rows, 128000 x 2048, bf16, 3.3-3.5 ms (1.2-1.3 PFLOP/s), of 2730 rows,
// 65536 x 1280, fp16, 446-482 us (1.0; the epilogue's exponentials are some 60 us of it), of 8 rows, 65536 x
// 768, 20 us (4.9 TB/s of W); a piece of 32000 entries of the 8192 rows: g 0.89-0.91 ms, dh 0.80-0.83, dW
// 0.82-0.85.  Power holds the clock at 1.7-1.9 GHz under the large ones; the matrix cores are busy in
// 63-70 % of those cycles in the 8192-row call, in 53-63 % in the shorter ones.  A compute unit has room
// for one block, so that nothing runs beside a tile's epilogue, nor beside its first loads.
template <int BM_, int kMode>
struct HeadCfg {
  static constexpr int BM = BM_, BN = 256, BK = 64, WM = 2, WN = 4, kWaves = WM * WN, kThreads = 64 * kWaves;
  static constexpr int SA = BM == 64 ? 4 : 3, SB = BM == 256 ? 2 : SA, LA = SA - 1;
  static constexpr int WTM = BM / (WM * 32), WTN = BN / (WN * 32);
  static constexpr bool kAT = kMode == kWeight, kBT = kMode == kHidden || kMode == kWeight;
  static constexpr int kDmaA = BM * BK / 512 / kWaves, kDmaB = BN * BK / 512 / kWaves, kDma = kDmaA + kDmaB;
  static constexpr int kAElems = BM * BK, kBElems = BN * BK, kBBase = SA * kAElems;
  static constexpr int kLds = (SA * kAElems + SB * kBElems) * 2;
  static_assert(kLds <= 160 * 1024 && kDmaA >= 1, "LDS");
};

template <int T>
__device__ __forceinline__ f32x16 head_mfma(bf16x8 a, bf16x8 b, f32x16 c) {
  if constexpr (T != kActF16) return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  else return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

template <int T, int BM, int kMode>
__global__ __launch_bounds__((HeadCfg<BM, kMode>::kThreads)) void head_gemm_kernel(HeadCall c) {
  typedef HeadCfg<BM, kMode> C;
  __shared__ __attribute__((aligned(16))) unsigned short smem[C::kLds / 2];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / C::WN, wn = wave % C::WN;
  const int live = c.head->live;
  if (live == 0 && kMode != kWeight) return;
  const int row_tiles = (live + BM - 1) / BM, dim_tiles = static_cast<int>((c.dim + 255) / 256);
  int mi, ni, split;
  {
    int mt, nt, splits = 1;
    if constexpr (kMode == kStats || kMode == kGrad) {
      mt = row_tiles;
      nt = c.piece_tiles;
      if constexpr (kMode == kStats) splits = c.logit_splits;
    } else if constexpr (kMode == kHidden) {
      mt = row_tiles;
      nt = dim_tiles;
      splits = c.splits;
    } else {
      mt = c.piece_tiles;
      nt = dim_tiles;
      splits = c.weight_splits;
    }
    if (!head_tile(kMode, mt, nt, splits, mi, ni, split)) return;
  }
  const int m0 = mi * BM, n0 = ni * C::BN;

  // operands: base at the tile's first element, row stride, bytes that may be read from there
  const unsigned short* W = static_cast<const unsigned short*>(c.weight_use) + c.piece_start * c.weight_stride;
  const int64_t w_left = c.vocab - c.piece_start;  // rows of W from the piece on
  const unsigned short *gA, *gB;
  int lda, ldb, k_from = 0, steps;  // steps: stages along the summed index
  int64_t left_b;  // values of B behind gB
  if constexpr (kMode == kStats || kMode == kGrad) {
    steps = static_cast<int>(c.dim_pad / C::BK);
    if (kMode == kStats && c.logit_splits > 1) {
      const int per = __builtin_amdgcn_readfirstlane((steps + c.logit_splits - 1) / c.logit_splits);
      k_from = split * per;
      steps = steps - k_from < per ? steps - k_from : per;
      steps = steps < 0 ? 0 : steps;
    }
    gA = static_cast<const unsigned short*>(c.hidden_pad) + static_cast<int64_t>(m0) * c.dim_pad + k_from * C::BK;
    lda = static_cast<int>(c.dim_pad);
    gB = W + static_cast<int64_t>(n0) * c.weight_stride + k_from * C::BK;
    ldb = static_cast<int>(c.weight_stride);
    left_b = (w_left - n0 - 1) * c.weight_stride + c.dim_use - k_from * C::BK;
  } else if constexpr (kMode == kHidden) {
    // stages that hold an entry of the vocabulary: none begins behind W's end
    const int64_t entries = w_left < c.piece_tiles * 256 ? w_left : c.piece_tiles * 256;
    const int all = static_cast<int>((entries + C::BK - 1) / C::BK);
    const int per = __builtin_amdgcn_readfirstlane((all + c.splits - 1) / c.splits);
    k_from = split * per;
    steps = all - k_from < per ? all - k_from : per;
    steps = steps < 0 ? 0 : steps;
    gA = static_cast<const unsigned short*>(c.g) + static_cast<int64_t>(m0) * c.g_stride + k_from * C::BK;
    lda = static_cast<int>(c.g_stride);
    gB = W + static_cast<int64_t>(k_from) * C::BK * c.weight_stride + n0;
    ldb = static_cast<int>(c.weight_stride);
    left_b = (w_left - static_cast<int64_t>(k_from) * C::BK - 1) * c.weight_stride + c.dim_use - n0;
  } else {
    const int all = (live + C::BK - 1) / C::BK, per = __builtin_amdgcn_readfirstlane((all + c.weight_splits - 1) / c.weight_splits);
    k_from = split * per;
    steps = all - k_from < per ? all - k_from : per;
    steps = steps < 0 ? 0 : steps;
    gA = static_cast<const unsigned short*>(c.g) + static_cast<int64_t>(k_from) * C::BK * c.g_stride + m0;
    lda = static_cast<int>(c.g_stride);
    gB = static_cast<const unsigned short*>(c.hidden_pad) + static_cast<int64_t>(k_from) * C::BK * c.dim_pad + n0;
    ldb = static_cast<int>(c.dim_pad);
    left_b = static_cast<int64_t>(steps) * C::BK * c.dim_pad - n0;
  }

  // fp32's six products of planes, the smallest first; stage kt of the sum is step kt % steps of
  // product kt / steps
  constexpr int kProducts = T == kActF32 ? 6 : 1;
  const int nk = steps * kProducts;
  const int64_t plane_a = kMode == kStats || kMode == kGrad ? c.hidden_plane : c.g_plane;
  const int64_t plane_b = kMode == kWeight ? c.hidden_plane : c.weight_plane;
  const auto at_a = [&](int kt, int& step) -> const unsigned short* {
    step = kt;
    if constexpr (kProducts == 1) return gA;
    const int product = __builtin_amdgcn_readfirstlane(kt / steps);
    step = kt - product * steps;
    return gA + (0x010210 >> (4 * product) & 15) * plane_a;
  };
  const auto at_b = [&](int kt, int& step) -> const unsigned short* {
    step = kt;
    if constexpr (kProducts == 1) return gB;
    const int product = __builtin_amdgcn_readfirstlane(kt / steps);
    step = kt - product * steps;
    return gB + (0x001012 >> (4 * product) & 15) * plane_b;
  };

  const auto issue_a = [&](int kt, int i) {
    unsigned short* s = smem + (kt % C::SA) * C::kAElems;
    const int q = i * C::kWaves + wave;
    int step;
    const unsigned short* base = at_a(kt, step);
    if constexpr (C::kAT) {
      constexpr int kChunks = BM / 8, kRows = 64 / kChunks;
      const int r0 = q * kRows, r = r0 + lane / kChunks, ch = lane % kChunks;
      dma16<C::kBT, 4>(base + static_cast<int64_t>(step) * C::BK * lda, (r * lda + swz_kn(r, ch) * 8) * 2,
                    static_cast<unsigned>(((C::BK - 1) * lda + BM) * 2), s + r0 * BM);
    } else {
      const int r0 = q * 8, r = r0 + lane / 8;
      dma16<C::kBT, 4>(base + step * C::BK, (r * lda + swz<64>(r, lane % 8) * 8) * 2,
                    static_cast<unsigned>(((BM - 1) * lda + C::BK) * 2), s + r0 * C::BK);
    }
  };
  const auto issue_b = [&](int kt, int i) {
    unsigned short* s = smem + C::kBBase + (kt % C::SB) * C::kBElems;
    const int q = i * C::kWaves + wave;
    int step;
    const unsigned short* base = at_b(kt, step);
    // reads behind the operand's end return zeros: vocabulary entries behind the last, and (below)
    // columns behind the hidden size, where W's next row follows
    if constexpr (C::kBT) {
      constexpr int kChunks = C::BN / 8, kRows = 64 / kChunks;
      const int r0 = q * kRows, r = r0 + lane / kChunks, ch = lane % kChunks;
      const int64_t left = left_b - static_cast<int64_t>(step) * C::BK * ldb;
      const int64_t most = static_cast<int64_t>(C::BK - 1) * ldb + C::BN;
      const int64_t values = left < most ? left : most;
      dma16<C::kBT, 4>(base + static_cast<int64_t>(step) * C::BK * ldb, (r * ldb + swz_kn(r, ch) * 8) * 2,
                    static_cast<unsigned>(values * 2), s + r0 * C::BN);
    } else {
      const int r0 = q * 8, r = r0 + lane / 8, ch = swz<64>(r, lane % 8);
      const int64_t left = left_b - step * C::BK;
      const int64_t most = static_cast<int64_t>(C::BN - 1) * ldb + C::BK;
      const int64_t values = left < most ? left : most;
      const int off = (k_from + step) * C::BK + ch * 8 < c.dim_use ? (r * ldb + ch * 8) * 2 : 0x7ffffff0;
      dma16<C::kBT, 4>(base + step * C::BK, off, static_cast<unsigned>(values * 2), s + r0 * C::BK);
    }
  };
  const auto issue_stage_a = [&](int st) {
#pragma unroll
    for (int i = 0; i < C::kDmaA; ++i) issue_a(st, i);
  };
  const auto issue_stage_b = [&](int st) {
#pragma unroll
    for (int i = 0; i < C::kDmaB; ++i) issue_b(st, i);
  };
  // until stage st has landed: what was issued after it may stay in flight
  const auto wait_stage = [&](int st) {
    if (st + 1 >= nk) {
      wait_vmcnt<0>();
    } else if constexpr (C::SA != C::SB) {
      wait_vmcnt<C::kDmaA>();
    } else {
      if (C::LA >= 3 && st + 2 < nk) wait_vmcnt<(C::LA - 1) * C::kDma>();
      else wait_vmcnt<C::kDma>();
    }
  };
  const int frow = lane & 31, fkh = lane >> 5;
  const auto read_t = [&](const unsigned short* s, int width, int col0, int kk) {
    // rows kk 16 + 8 (lane / 32) + 0..7 of column col0 + lane % 32, two transposing reads of 4 rows
    const int g16 = lane >> 4, sl = lane & 15;
    const int col = col0 + 16 * (g16 & 1) + 4 * (sl & 3), row = kk * 16 + 8 * (g16 >> 1) + (sl >> 2);
    const s16x4 lo = lds_read_tr(s + row * width + swz_kn(row, col >> 3) * 8 + (col & 7));
    const s16x4 hi = lds_read_tr(s + (row + 4) * width + swz_kn(row + 4, col >> 3) * 8 + (col & 7));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  };
  const auto read_k = [&](const unsigned short* s, int r, int kk) {
    return *reinterpret_cast<const bf16x8*>(s + r * C::BK + swz<64>(r, kk * 2 + fkh) * 8);
  };
  const auto load_frags = [&](int kt, int kk, bf16x8 (&fa)[C::WTM], bf16x8 (&fb)[C::WTN]) {
    const unsigned short* as = smem + (kt % C::SA) * C::kAElems;
    const unsigned short* bs = smem + C::kBBase + (kt % C::SB) * C::kBElems;
#pragma unroll
    for (int i = 0; i < C::WTM; ++i) {
      const int r = wm * (C::WTM * 32) + i * 32;
      if constexpr (C::kAT) fa[i] = read_t(as, BM, r, kk);
      else fa[i] = read_k(as, r + frow, kk);
    }
#pragma unroll
    for (int j = 0; j < C::WTN; ++j) {
      const int r = wn * (C::WTN * 32) + j * 32;
      if constexpr (C::kBT) fb[j] = read_t(bs, C::BN, r, kk);
      else fb[j] = read_k(bs, r + frow, kk);
    }
  };

  f32x16 acc[C::WTM][C::WTN];
#pragma unroll
  for (int i = 0; i < C::WTM; ++i)
#pragma unroll
    for (int j = 0; j < C::WTN; ++j)
#pragma unroll
      for (int k = 0; k < 16; ++k) acc[i][j][k] = 0.0f;

  if (nk > 0) {
    constexpr int KK = C::BK / 16;
#pragma unroll
    for (int st = 0; st < C::SB; ++st) {
      if (st < C::LA && st < nk) issue_stage_a(st);
      if (st < nk) issue_stage_b(st);
    }
    bf16x8 fa[2][C::WTM], fb[2][C::WTN];
    if (nk >= C::SA) wait_vmcnt<(C::LA - 1) * C::kDmaA + (C::SB - 1) * C::kDmaB>();
    else wait_vmcnt<0>();
    stage_barrier();
    load_frags(0, 0, fa[0], fb[0]);
    // Stage kt loads A of stage kt + LA between its matrix instructions and, once its own slot of B has
    // been read by all, B of stage kt + SB between the last of them.  (All loads ahead of the stage's
    // first matrix instruction keep the matrix cores waiting.  In turn on one card, that way and this: 8192
    // rows, 128000 x 2048, both directions, 14.55 and 13.95 ms; the gradients of 2048 rows, 65536 x 1280, 1002
    // and 947 us; the forward pass of 4095, 476 and 460.  B spread over the stage comes too late: 9 % slower.
    // Four waves of 128 x 128, whose fragments take two thirds of the LDS reads, but alone on their SIMD:
    // 12 % slower.)
    const auto run_stage = [&](int kt, auto steady) {
      constexpr bool kSteady = decltype(steady)::value;
      constexpr int kSlots = (KK - 1) * C::WTM;
#pragma unroll
      for (int kk = 0; kk < KK; ++kk) {
        const int cur = kk & 1;
        if (kk + 1 < KK) {
          load_frags(kt, kk + 1, fa[cur ^ 1], fb[cur ^ 1]);
        } else if (kSteady || kt + 1 < nk) {
          // stage kt + 1 has landed and every wave's reads of this stage are done
          if constexpr (kSteady) {
            if constexpr (C::SA != C::SB) wait_vmcnt<C::kDmaA>();
            else wait_vmcnt<(C::LA - 1) * C::kDma>();
          } else {
            wait_stage(kt + 1);
          }
          stage_barrier();
          load_frags(kt + 1, 0, fa[cur ^ 1], fb[cur ^ 1]);
        }
#pragma unroll
        for (int i = 0; i < C::WTM; ++i) {
          if (kk + 1 < KK && (kSteady || kt + C::LA < nk)) {
            const int slot = kk * C::WTM + i;
#pragma unroll
            for (int u = slot * C::kDmaA / kSlots; u < (slot + 1) * C::kDmaA / kSlots; ++u) issue_a(kt + C::LA, u);
          }
          if (kk + 1 == KK && (kSteady || kt + C::SB < nk)) {
#pragma unroll
            for (int u = i * C::kDmaB / C::WTM; u < (i + 1) * C::kDmaB / C::WTM; ++u) issue_b(kt + C::SB, u);
          }
#pragma unroll
          for (int j = 0; j < C::WTN; ++j) acc[i][j] = head_mfma<T>(fb[cur][j], fa[cur][i], acc[i][j]);
        }
      }
    };
    int kt = 0;
    for (; kt < nk - C::SA; ++kt) run_stage(kt, std::true_type{});
    for (; kt < nk; ++kt) run_stage(kt, std::false_type{});
  }
  head_epilogue<T, T == kActF32, kMode, BM, C::BN, C::WM, C::WN>(c, acc, m0, n0, split, live, reinterpret_cast<char*>(smem));
}

// fp32 operands: BM x 128 tiles of 4 waves, v_mfma_f32_32x32x2, stages of the summed index that pass
// through registers into LDS rows of one index each, whatever the operand's order.  Few rows are
// bound by memory and its latency: 32- and 64-row tiles, with longer stages.
template <int BM, int kMode>
__global__ __launch_bounds__(256, BM == 128 ? 1 : 3) void head_gemm32_kernel(HeadCall c) {  // (waves per SIMD)
  constexpr int B = 128, BK = BM == 128 ? 16 : 32, LA = BM + (kMode == kWeight ? 4 : 2),
                LB = B + (kMode == kHidden || kMode == kWeight ? 4 : 2);  // vectors along k are stored a value at a time
  constexpr int WM = BM == 32 ? 1 : 2, WN = 4 / WM, WTM = BM / (WM * 32), WTN = B / (WN * 32);
  constexpr int kA = BM * BK / 1024, kB = B * BK / 1024;  // vectors of 4 values a thread and stage
  __shared__ __attribute__((aligned(16))) float smem[2][BK * (LA + LB)];
  constexpr bool kAT = kMode == kWeight, kBT = kMode == kHidden || kMode == kWeight;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int live = c.head->live;
  if (live == 0 && kMode != kWeight) return;
  const int row_tiles = (live + BM - 1) / BM, dim_tiles = static_cast<int>((c.dim + B - 1) / B);
  int mi, ni, split;
  {
    int mt, nt, splits = 1;
    if constexpr (kMode == kStats || kMode == kGrad) {
      mt = row_tiles;
      nt = c.piece_tiles;
      if constexpr (kMode == kStats) splits = c.logit_splits;
    } else if constexpr (kMode == kHidden) {
      mt = row_tiles;
      nt = dim_tiles;
      splits = c.splits;
    } else {
      mt = c.piece_tiles;
      nt = dim_tiles;
    }
    if (!head_tile(kMode, mt, nt, splits, mi, ni, split)) return;
  }
  const int m0 = mi * BM, n0 = ni * B;
  const float* W = static_cast<const float*>(c.weight_use) + c.piece_start * c.weight_stride;
  const int64_t w_left = c.vocab - c.piece_start;
  // operand (row, k): contiguous along k, or along the rows (T)
  const float *gA, *gB;
  int lda, ldb;
  int64_t left_b;  // values of B behind gB: reads behind them return zeros
  int k0 = 0, k1;  // the summed indices k0 .. k1 - 1
  if constexpr (kMode == kStats || kMode == kGrad) {
    gA = static_cast<const float*>(c.hidden_pad) + static_cast<int64_t>(m0) * c.dim_pad;
    lda = static_cast<int>(c.dim_pad);
    gB = W + static_cast<int64_t>(n0) * c.weight_stride;
    ldb = static_cast<int>(c.weight_stride);
    left_b = (w_left - n0 - 1) * c.weight_stride + c.dim_use;
    // no stage begins behind the row's end
    const int all = static_cast<int>((c.dim + BK - 1) / BK), per = kMode == kStats ? (all + c.logit_splits - 1) / c.logit_splits : all;
    k0 = split * per * BK;
    k1 = min(all, (split + 1) * per) * BK;
  } else if constexpr (kMode == kHidden) {
    const int64_t entries = w_left < c.piece_tiles * B ? w_left : c.piece_tiles * B;
    const int all = static_cast<int>((entries + BK - 1) / BK), per = (all + c.splits - 1) / c.splits;
    k0 = split * per * BK;
    k1 = min(all, (split + 1) * per) * BK;
    gA = static_cast<const float*>(c.g) + static_cast<int64_t>(m0) * c.g_stride;
    lda = static_cast<int>(c.g_stride);
    gB = W + n0;
    ldb = static_cast<int>(c.weight_stride);
    left_b = (w_left - 1) * c.weight_stride + c.dim_use - n0;
  } else {
    k1 = (live + BK - 1) / BK * BK;
    gA = static_cast<const float*>(c.g) + m0;
    lda = static_cast<int>(c.g_stride);
    gB = static_cast<const float*>(c.hidden_pad) + n0;
    ldb = static_cast<int>(c.dim_pad);
    left_b = static_cast<int64_t>(k1) * c.dim_pad - n0;
  }
  // a thread's vectors of an operand's stage (A is padded to whole tiles)
  constexpr int D = 3;  // stages in registers on their way
  f32x4 ra[D][kA], rb[D][kB];
  const auto load = [&](int k, f32x4 (&ra)[kA], f32x4 (&rb)[kB]) {
    const float* a = gA + (kAT ? static_cast<int64_t>(k) * lda : k);
#pragma unroll
    for (int u = 0; u < kA; ++u) {
      const int x = tid + u * 256;
      ra[u] = *reinterpret_cast<const f32x4*>(a + (kAT ? x / (BM / 4) * lda + x % (BM / 4) * 4 : x / (BK / 4) * lda + x % (BK / 4) * 4));
    }
    const int64_t from = kBT ? static_cast<int64_t>(k) * ldb : k;
    const int64_t most = kBT ? static_cast<int64_t>(BK - 1) * ldb + B : static_cast<int64_t>(B - 1) * ldb + BK;
    const int64_t values = left_b - from < most ? left_b - from : most;
    const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(gB + from), 0, static_cast<int>(values * 4), 0x00020000);
#pragma unroll
    for (int u = 0; u < kB; ++u) {
      const int x = tid + u * 256;
      const int at = kBT ? x / (B / 4) * ldb + x % (B / 4) * 4 : x / (BK / 4) * ldb + x % (BK / 4) * 4;
      rb[u] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, at * 4, 0, 0));
    }
    if (!kBT && k + BK > c.dim_use) {
      // the row's end: W's next row follows
#pragma unroll
      for (int u = 0; u < kB; ++u) {
        const int kk = k + (tid + u * 256) % (BK / 4) * 4;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (kk + e >= c.dim_use) rb[u][e] = 0.0f;
      }
    }
  };
  const auto store = [&](int buf, const f32x4 (&ra)[kA], const f32x4 (&rb)[kB]) {
    float *a = smem[buf], *b = smem[buf] + BK * LA;
#pragma unroll
    for (int u = 0; u < kA; ++u) {
      const int x = tid + u * 256;
      if constexpr (kAT) {
        *reinterpret_cast<f32x4*>(a + x / (BM / 4) * LA + x % (BM / 4) * 4) = ra[u];
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) a[(x % (BK / 4) * 4 + e) * LA + x / (BK / 4)] = ra[u][e];
      }
    }
#pragma unroll
    for (int u = 0; u < kB; ++u) {
      const int x = tid + u * 256;
      if constexpr (kBT) {
        *reinterpret_cast<f32x4*>(b + x / (B / 4) * LB + x % (B / 4) * 4) = rb[u];
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) b[(x % (BK / 4) * 4 + e) * LB + x / (BK / 4)] = rb[u][e];
      }
    }
  };
  f32x16 acc[WTM][WTN];
#pragma unroll
  for (int i = 0; i < WTM; ++i)
#pragma unroll
    for (int j = 0; j < WTN; ++j)
#pragma unroll
      for (int k = 0; k < 16; ++k) acc[i][j][k] = 0.0f;
  const int steps = k0 < k1 ? (k1 - k0) / BK : 0;
  if (steps > 0) {
#pragma unroll
    for (int u = 0; u < D; ++u)
      if (u < steps) load(k0 + u * BK, ra[u], rb[u]);
    store(0, ra[0], rb[0]);
    __syncthreads();
    for (int first = 0; first < steps; first += D) {
#pragma unroll
      for (int u = 0; u < D; ++u) {
        const int s = first + u;
        if (s >= steps) break;
        if (s + D < steps) load(k0 + (s + D) * BK, ra[u], rb[u]);
        const float* a = smem[s & 1] + (lane >> 5) * LA + wm * (WTM * 32) + (lane & 31);
        const float* b = smem[s & 1] + BK * LA + (lane >> 5) * LB + wn * (WTN * 32) + (lane & 31);
#pragma unroll
        for (int kk = 0; kk < BK; kk += 2) {
          float fa[WTM], fb[WTN];
#pragma unroll
          for (int i = 0; i < WTM; ++i) fa[i] = a[kk * LA + i * 32];
#pragma unroll
          for (int j = 0; j < WTN; ++j) fb[j] = b[kk * LB + j * 32];
#pragma unroll
          for (int i = 0; i < WTM; ++i)
#pragma unroll
            for (int j = 0; j < WTN; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x2f32(fb[j], fa[i], acc[i][j], 0, 0, 0);
        }
        if (s + 1 < steps) store((s + 1) & 1, ra[(u + 1) % D], rb[(u + 1) % D]);
        __syncthreads();
      }
    }
  }
  head_epilogue<kActF32, false, kMode, BM, B, WM, WN>(c, acc, m0, n0, split, live, reinterpret_cast<char*>(&smem[0][0]));
}

// Host: whether fp32 runs on bf16 planes, and the tiles' columns.
bool head_split(int type, int64_t n) { return type == kActF32 && n > kSplitRows; }
int64_t head_tile_size(int type, bool split) { return type == kActF32 && !split ? 128 : 256; }
// The rows that gathered ones are padded to a multiple of, and a tile's at most.
int64_t head_row_tile(int type, int64_t n) {
  if (type == kActF32) return head_split(type, n) ? 256 : n <= 32 ? 32 : n <= 64 ? 64 : 128;
  return n <= 64 ? 64 : n <= 128 ? 128 : 256;
}
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t align_up(int64_t x, int64_t q) { return ceil_div(x, q) * q; }
// Seconds of a product of so many tiles and summed indices: rounds of the chip (256 compute units, a
// block each) by what a tile takes for an index on the full chip.  A tile of half the rows takes more
// than half of it.  Measured, a round of 256 tiles of logits over 256 to 1024 indices, the slope: tiles of
// 256, 128 and 64 rows 27, 17 and 18 ns an index (the last by the rate at which W is read, which the model
// leaves out: 12.5), on the fp32 instructions 75, 47 and 27 for 128, 64 and 32; and 3 to 8 us whatever the
// length, which all choices have.
double head_time(int type, bool split, int64_t tiles, int64_t rows, int64_t length) {
  double tile;
  if (type == kActF32 && !split) tile = rows == 128 ? 80e-9 : rows == 64 ? 46e-9 : 25e-9;
  else tile = (rows == 256 ? 27.9e-9 : rows == 128 ? 17.3e-9 : 12.5e-9) * (split ? 6 : 1);
  return static_cast<double>(ceil_div(tiles, 256)) * length * tile;
}
// A tile's rows, in a product of `cols` tiles beside each other.
int64_t head_best_rows(int type, int64_t n, int64_t cols) {
  const int64_t most = head_row_tile(type, n);
  const bool split = head_split(type, n);
  if (type == kActF32 && !split) return most;
  int64_t best = most;
  for (int64_t rows = most / 2; rows >= 64; rows /= 2)
    if (head_time(type, split, ceil_div(n, rows) * cols, rows, 1) < head_time(type, split, ceil_div(n, best) * cols, best, 1)) best = rows;
  return best;
}

// Host: blocks of a launch over `tiles` tiles at most (see head_tile).
dim3 head_grid(int64_t tiles) { return dim3(static_cast<unsigned>(8 * ((tiles + 7) / 8))); }

// kSplit: fp32 on bf16 planes.
template <int T, bool kSplit, int BM, int kMode>
hipError_t launch_head_gemm(const HeadCall& c, int64_t tiles, hipStream_t s) {
  if constexpr (T == kActF32 && !kSplit)
    hipLaunchKernelGGL((head_gemm32_kernel<BM, kMode>), head_grid(tiles), dim3(256), 0, s, c);
  else
    hipLaunchKernelGGL((head_gemm_kernel<T, BM, kMode>), head_grid(tiles), dim3(HeadCfg<BM, kMode>::kThreads), 0, s, c);
  return hipGetLastError();
}

// A product whose rows are the call's, in tiles of `rows` and `cols` of them beside each other.
template <int T, bool kSplit, int kMode>
hipError_t launch_head_rows(const HeadCall& c, int64_t rows, int64_t cols, hipStream_t s) {
  const int64_t tiles = ceil_div(c.n, rows) * cols;
  if constexpr (T == kActF32 && !kSplit) {
    if (rows == 32) return launch_head_gemm<T, kSplit, 32, kMode>(c, tiles, s);
    if (rows == 64) return launch_head_gemm<T, kSplit, 64, kMode>(c, tiles, s);
    return launch_head_gemm<T, kSplit, 128, kMode>(c, tiles, s);
  } else {
    if (rows == 64) return launch_head_gemm<T, kSplit, 64, kMode>(c, tiles, s);
    if (rows == 128) return launch_head_gemm<T, kSplit, 128, kMode>(c, tiles, s);
    return launch_head_gemm<T, kSplit, 256, kMode>(c, tiles, s);
  }
}

template <int T, bool kSplit>
hipError_t gather(const HeadCall& c, hipStream_t s) {
  if constexpr (!kSplit) {
    // one launch for both where a block's copying takes no longer than a second launch, some 4 us
    if (c.n <= 64 && c.row_tile * c.dim_pad <= 128 * 1024) {  // (at most 64 rows a tile)
      hipLaunchKernelGGL((head_rows_kernel<T, true>), dim3(1), dim3(kRowThreads), 0, s, c);
      return hipGetLastError();
    }
  }
  hipLaunchKernelGGL((head_rows_kernel<T, false>), dim3(1), dim3(kRowThreads), 0, s, c);
  hipLaunchKernelGGL((head_gather_kernel<T, kSplit>), dim3(static_cast<unsigned>(c.rows_pad / 4)), dim3(256), 0, s, c);
  return hipGetLastError();
}

template <int T, bool kSplit>
hipError_t forward(const HeadCall& call, hipStream_t s) {
  HeadCall c = call;
  if (!c.once) c.row_weight = nullptr;
  c.piece_start = 0;
  c.piece_tiles = static_cast<int>(ceil_div(c.vocab, head_tile_size(T, kSplit)));
  c.tiles = c.piece_tiles;
  if (const hipError_t e = gather<T, kSplit>(c, s)) return e;
  if (const hipError_t e = launch_head_rows<T, kSplit, kStats>(c, c.stats_rows, c.piece_tiles * c.logit_splits, s)) return e;
  if (c.logit_splits > 1) {
    hipLaunchKernelGGL(head_stats_kernel, dim3(static_cast<unsigned>(c.n)), dim3(256), 0, s, c);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(head_join_kernel, dim3(static_cast<unsigned>(ceil_div(c.n, 4))), dim3(256), 0, s, c);
  return hipGetLastError();
}

template <int T, bool kSplit>
hipError_t backward(const HeadCall& call, hipStream_t s) {
  HeadCall c = call;
  c.loss = nullptr;
  c.lse_out = nullptr;
  const int64_t tile = head_tile_size(T, kSplit), dim_tiles = ceil_div(c.dim, tile);
  if (!c.once)
    if (const hipError_t e = gather<T, kSplit>(c, s)) return e;
  for (int64_t v = 0; v < c.vocab; v += c.piece) {
    c.piece_start = v;
    c.first = v == 0;
    const int64_t here = c.vocab - v < c.piece ? c.vocab - v : c.piece;
    c.piece_tiles = static_cast<int>(ceil_div(here, tile));
    if (c.kept && c.lse_in)  // the backward pass alone
      if (const hipError_t e = launch_head_rows<T, kSplit, kStats>(c, c.stats_rows, c.piece_tiles * c.logit_splits, s)) return e;
    if (c.kept) {
      const dim3 grid(static_cast<unsigned>(ceil_div(c.piece, 2048)), static_cast<unsigned>(align_up(c.n, c.row_tile)));
      hipLaunchKernelGGL((head_convert_kernel<T, kSplit>), grid, dim3(256), 0, s, c);
      if (const hipError_t e = hipGetLastError()) return e;
    } else if (const hipError_t e = launch_head_rows<T, kSplit, kGrad>(c, c.grad_rows, c.piece_tiles, s)) {
      return e;
    }
    if (c.dhidden)
      if (const hipError_t e = launch_head_rows<T, kSplit, kHidden>(c, c.hidden_rows, dim_tiles * c.splits, s)) return e;
    if (c.dweight)
      if (const hipError_t e = launch_head_gemm<T, kSplit, T == kActF32 && !kSplit ? 128 : 256, kWeight>(c, c.piece_tiles * dim_tiles * c.weight_splits, s)) return e;
    if (c.dweight && c.weight_splits > 1) {
      const dim3 grid(static_cast<unsigned>(ceil_div(here, 4)), static_cast<unsigned>(ceil_div(c.dim, 256)));
      hipLaunchKernelGGL((head_weight_out_kernel<T>), grid, dim3(256), 0, s, c);
      if (const hipError_t e = hipGetLastError()) return e;
    }
  }
  if (c.dhidden)
    hipLaunchKernelGGL((head_out_kernel<T>), dim3(static_cast<unsigned>(ceil_div(c.n, 4)), static_cast<unsigned>(ceil_div(c.dim, 256))),
                       dim3(256), 0, s, c);
  return hipGetLastError();
}

template <int T, bool kSplit>
hipError_t run_work(const HeadCall& c, HeadWork work, hipStream_t s) {
  if (c.weight_pad) {
    hipLaunchKernelGGL((head_weight_kernel<T, kSplit>), dim3(static_cast<unsigned>(ceil_div(c.vocab, 4))), dim3(256), 0, s, c);
    if (const hipError_t e = hipGetLastError()) return e;
  }
  if (work != kHeadBackward)
    if (const hipError_t e = forward<T, kSplit>(c, s)) return e;
  return work != kHeadForward ? backward<T, kSplit>(c, s) : hipSuccess;
}

}  // namespace

bool head_weight_copied(int type, int64_t dim, const void* weight, int64_t stride) {
  // (offsets inside a tile of 256 rows have 31 bits)
  if (type == kActF32) return stride > (1 << 21);
  return (reinterpret_cast<uintptr_t>(weight) & 15u) || stride % 8 || dim % 8 || stride > (1 << 22);
}

int64_t head_threads(int type, int64_t n, int64_t dim, int64_t vocab, const HeadPlan& p) {
  const int64_t tile = head_tile_size(type, p.split), dim_tiles = ceil_div(dim, tile);
  int64_t tiles = ceil_div(n, p.stats_rows) * ceil_div(vocab, tile) * p.logit_splits;
  const int64_t others[] = {ceil_div(n, p.hidden_rows) * dim_tiles * p.splits, ceil_div(n, p.grad_rows) * (p.piece / tile),
                            p.piece / tile * dim_tiles * p.weight_splits};
  for (const int64_t t : others) tiles = t > tiles ? t : tiles;
  // the kernels with a wave for each vocabulary entry
  const int64_t waves = p.weight_pad || p.weight_splits > 1 ? vocab * 64 + 256 : 0;
  return (tiles + 8) * 512 > waves ? (tiles + 8) * 512 : waves;
}

HeadPlan plan_head(int type, int64_t n, int64_t dim, int64_t vocab, bool copied, HeadWork work) {
  HeadPlan p{};
  const bool gradients = work != kHeadForward;
  p.split = head_split(type, n);
  // bytes of a value of the gathered rows, g and a copied W
  const int64_t size = p.split ? 6 : type == kActF32 ? 4 : 2, tile = head_tile_size(type, p.split);
  // memory is taken for the rows of whole tiles; pieces and splits are chosen for rows padded to
  // kHeadTile
  p.rows_pad = align_up(n, head_row_tile(type, n));
  const int64_t full_rows = align_up(n, kHeadTile);
  p.dim_pad = align_up(dim, 64);
  int64_t at = 0;
  const auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at = align_up(at + bytes, 256);
    return here;
  };
  p.head = take(sizeof(HeadInfo));
  p.place = take(n * 4);
  p.row_of = take(n * 4);
  p.label = take(n * 4);
  p.target = take(n * 4);
  p.weight = take(n * 4);
  p.top = take(n * 4);
  p.factor = take(n * 4);
  p.tops = take(n * 4);
  p.sums = take(n * 4);
  // (fp32: a tile's columns behind the hidden size are read, and dropped, up to a whole tile)
  p.hidden = take(p.rows_pad * p.dim_pad * size + tile * 4);
  p.weight_pad = copied || p.split ? take(vocab * p.dim_pad * size) : 0;
  // the statistics of the forward pass lie where the backward pass has g
  const int64_t tiles = ceil_div(vocab, tile), dim_tiles = ceil_div(dim, tile);
  int64_t piece = kHeadPieceBytes / (full_rows * size) / tile;
  piece = piece < 1 ? 1 : piece;
  p.piece = ceil_div(tiles, ceil_div(tiles, piece)) * tile;
  // rows a power of two apart would meet in the same memory channels (the gradients of 2048 rows, 65536 x
  // 1280: 1042 us, 1020 with 64 values more)
  p.g_stride = p.piece + 64;
  const int64_t logits = p.rows_pad * p.g_stride * 4;
  const bool fits = p.piece >= vocab && full_rows * p.piece * 4 <= kHeadPieceBytes && full_rows <= 65535;
  p.stats_rows = head_best_rows(type, n, tiles);
  p.grad_rows = head_best_rows(type, n, p.piece / tile);
  p.hidden_rows = head_row_tile(type, n);
  p.logit_splits = p.splits = p.weight_splits = 1;
  // kept logits: the logits' second product, and where rows are numbered once two launches of 10 us,
  // against 8 bytes of traffic each, at a large copy's 4.8 TB/s (fp32: g takes their place).  Rows that
  // fill one tile at most are numbered once anyhow: leaving some out would save nothing.
  const int64_t padded = align_up(n, head_row_tile(type, n));
  p.kept = work == kHeadBoth && fits &&
           8.0 * padded * p.piece / 4.8e12 < head_time(type, p.split, ceil_div(n, p.grad_rows) * (p.piece / tile), p.grad_rows, p.dim_pad) +
                                          (n > head_row_tile(type, n) ? 10e-6 : 0.0);
  // Products of few tiles: their sums are split over blocks where the fuller chip saves more than the
  // sums' traffic (8 bytes a value, 4.8 TB/s) and another launch, if any, cost.
  const int64_t most = head_row_tile(type, n), least = type == kActF32 && !p.split ? most : 64;
  // the logits, over the hidden size (by 256 at least): they are kept then
  if (fits) {
    // (a tenth less does not count: 192 rows of fp32, 30758 x 1896, took 730 us in two parts, 687 whole;
    // the backward pass alone has a launch more: 2 rows of bf16, 9756 x 1046, 68 us in parts, 63 whole.
    // 89 rows of fp32, 1980 x 2421: 95 us in parts, 270 whole)
    double best = 0.8 * head_time(type, p.split, ceil_div(n, p.stats_rows) * tiles, p.stats_rows, p.dim_pad);
    for (int64_t rows = most; rows >= least; rows /= 2)
      for (int64_t splits = 2; splits <= 32 && splits * 256 <= dim && splits * full_rows * p.piece * 4 <= kHeadPieceBytes; ++splits) {
        const double time = head_time(type, p.split, ceil_div(n, rows) * tiles * splits, rows, ceil_div(p.dim_pad, splits)) +
                            8.0 * splits * padded * p.piece / 4.8e12 + (gradients ? 8e-6 : 2e-6);
        if (time < best) {
          best = time;
          p.stats_rows = rows;
          p.logit_splits = static_cast<int>(splits);
        }
      }
    if (p.logit_splits > 1) p.kept = gradients;
  }
  // (fp32's g takes the place of kept logits)
  const bool in_place = p.kept && type == kActF32 && !p.split;
  const int64_t stats = n * tiles * 8, g = gradients && !in_place ? p.rows_pad * p.g_stride * size : 0;
  p.partial = take(stats > g ? stats : g);
  p.logits = p.kept || p.logit_splits > 1 ? take(p.logit_splits * logits) : 0;
  p.sum_stride = align_up(dim, 4);
  if (gradients) {
    // dh, over the piece (by 256 vocabulary entries at least)
    double best = 0.0;
    for (int64_t rows = most; rows >= least; rows /= 2) {
      const int64_t blocks = ceil_div(n, rows) * dim_tiles;
      for (int64_t splits = 1; splits <= 64 && (splits == 1 || splits * 256 <= p.piece); ++splits) {
        const double time = head_time(type, p.split, blocks * splits, rows, ceil_div(p.piece, splits)) + 8.0 * splits * n * dim / 4.8e12;
        if (best == 0.0 || time < best) {
          best = time;
          p.hidden_rows = rows;
          p.splits = static_cast<int>(splits);
        }
      }
    }
    p.sum = take(p.splits * p.rows_pad * p.sum_stride * 4);
    // dW, over the rows (by 128 at least)
    if (type != kActF32 || p.split) {
      const int64_t blocks = p.piece / tile * dim_tiles;
      best = head_time(type, p.split, blocks, 256, n);
      for (int64_t splits = 2; splits <= 64 && splits * 128 <= n; ++splits) {
        const double time = head_time(type, p.split, blocks * splits, 256, ceil_div(n, splits)) + 8.0 * splits * p.piece * dim / 4.8e12 + 4e-6;
        if (time < best) {
          best = time;
          p.weight_splits = static_cast<int>(splits);
        }
      }
      if (p.weight_splits > 1) p.weight_sum = take(p.weight_splits * p.piece * p.sum_stride * 4);
    }
  }
  p.bytes = at;
  return p;
}

hipError_t launch_head_clear(const HeadCall& c, hipStream_t s) {
  hipLaunchKernelGGL(head_clear_kernel, dim3(static_cast<unsigned>(ceil_div(c.vocab, 4))), dim3(256), 0, s, c);
  return hipGetLastError();
}

hipError_t launch_head(const HeadCall& call, const HeadPlan& p, void* workspace, HeadWork work, hipStream_t s) {
  HeadCall c = call;
  char* ws = static_cast<char*>(workspace);
  c.head = reinterpret_cast<HeadInfo*>(ws + p.head);
  c.place = reinterpret_cast<int*>(ws + p.place);
  c.row_of = reinterpret_cast<int*>(ws + p.row_of);
  c.label = reinterpret_cast<int*>(ws + p.label);
  c.target = reinterpret_cast<float*>(ws + p.target);
  c.weight = reinterpret_cast<float*>(ws + p.weight);
  c.top = reinterpret_cast<float*>(ws + p.top);
  c.factor = reinterpret_cast<float*>(ws + p.factor);
  c.tops = work == kHeadBoth ? reinterpret_cast<float*>(ws + p.tops) : nullptr;
  c.sums = work == kHeadBoth ? reinterpret_cast<float*>(ws + p.sums) : nullptr;
  c.hidden_pad = ws + p.hidden;
  c.partial = reinterpret_cast<float2*>(ws + p.partial);
  c.logit_splits = p.logit_splits;
  c.z_plane = p.rows_pad * p.g_stride;
  c.kept = p.kept;
  c.once = work == kHeadBoth && (p.kept || c.n <= head_row_tile(c.type, c.n));
  c.planes = p.split;
  c.z = reinterpret_cast<float*>(ws + p.logits);
  c.g = c.kept && c.type == kActF32 && !p.split ? ws + p.logits : ws + p.partial;
  c.sum = reinterpret_cast<float*>(ws + p.sum);
  c.rows_pad = p.rows_pad;
  c.dim_pad = p.dim_pad;
  c.sum_stride = p.sum_stride;
  c.piece = p.piece;
  c.splits = p.splits;
  c.row_tile = static_cast<int>(head_row_tile(c.type, c.n));
  c.stats_rows = p.stats_rows;
  c.grad_rows = p.grad_rows;
  c.hidden_rows = p.hidden_rows;
  c.weight_splits = p.weight_splits;
  c.weight_sum = reinterpret_cast<float*>(ws + p.weight_sum);
  c.weight_lines = c.dweight && c.dweight_type != kActF32 && reinterpret_cast<uintptr_t>(c.dweight) % 16 == 0 &&
                   c.dweight_stride % 8 == 0 && c.dim % 8 == 0;
  c.weight_use = c.weight_in;
  c.weight_stride = c.weight_in_stride;
  c.dim_use = c.dim;
  c.hidden_plane = p.rows_pad * p.dim_pad;
  c.weight_plane = c.vocab * p.dim_pad;
  c.g_plane = p.rows_pad * p.g_stride;
  c.g_stride = p.g_stride;
  c.weight_pad = nullptr;
  if (p.weight_pad) {
    c.weight_pad = ws + p.weight_pad;
    c.weight_use = c.weight_pad;
    c.weight_stride = c.dim_use = p.dim_pad;
  }
  return with_act(c.type, [&](auto t) {
    constexpr int T = decltype(t)::value;
    if constexpr (T == kActF32)
      if (p.split) return run_work<T, true>(c, work, s);
    return run_work<T, false>(c, work, s);
  });
}

}  // namespace ma

// AdamW over many tensors with both moments held in 8 bits.
//
// A moment is a value of 8 bits per element and a power of two per block of 64 elements (in the
// tensor's flattened order; the last block may be short):
//   exp_avg     OCP e4m3, the block's largest finite magnitude scaled into [2^7, 2^8)
//   exp_avg_sq  OCP e5m2, the block's largest finite value scaled into [2^14, 2^15)
//   scale       e8m0: the byte b stands for 2^(b - 127)
// The step widens them to fp32 (exact), runs the AdamW update on them, writes the parameter
// from the moments before they are rounded, and rounds the moments back.
//
// Rounding is stochastic: y between two neighbours of its type a < b becomes b with probability
// (y - a) / (b - a), so the expected value is y.  Rounding to nearest would never let a slow
// average move: with beta2 = 0.999 a zero gradient lowers exp_avg_sq by a thousandth, and the
// nearest 8-bit value is the old one.  The scales are powers of two for the same reason: while
// the block's largest value stays within its binade the grid stays where it was, and an element
// that lies on the grid is not rounded at all; a scale that followed the largest value exactly
// would round every element of the block anew in every step, and the noise of some 500 steps
// (1 / (2 (1 - beta2))) would add up.  A positive second moment never rounds to zero, which its
// first moment could be divided by in the next step.
// The random bits are a hash of the element's number and a key of seed and step, 16 for each
// moment: the same inputs give the same bits on every call, and no state is kept.
//
// Bound by memory: 16 bytes per element with a 16-bit gradient and a 16-bit copy of the parameter,
// and 1/16 byte of scales (28 bytes with moments in 32 bits).  Measured, card to card: 168 M elements with
// fp32 gradients 434-460 us, 262 M with bf16 gradients and copies 705-745 us, 5.7-6.2 TB/s.  Four elements
// a lane make a scale's block one row of 16 lanes, whose maximum needs no shared memory; four groups of
// loads in flight a thread.  With library root and division, and a hash a moment, it was bound by
// arithmetic (501 and 811 us).
#include "adamw_elem.h"
#include "ma_act.h"
#include "ma_internal.h"

namespace ma {
namespace {

constexpr int kThreads = 256;
// 64 elements of a scale's block are the 4 elements of 16 lanes: a row of data-parallel moves.
constexpr int kEach = 4;
constexpr int kGroups = 4;  // groups of kEach elements a thread, all loaded before any arithmetic
constexpr int kChunk = kThreads * kEach * kGroups;
static_assert(kAdamWByteBlock == 16 * kEach && kChunk % kAdamWByteBlock == 0, "a block of a scale is a row of lanes");

typedef Pack<unsigned char, 4>::type Bytes;
typedef float f32x2 __attribute__((ext_vector_type(2)));

// The finalizer of MurmurHash3 (A. Appleby, public domain): every input bit reaches every
// output bit.
__device__ __forceinline__ uint32_t mix(uint32_t x) {
  x = (x ^ (x >> 16)) * 0x85ebca6bu;
  x = (x ^ (x >> 13)) * 0xc2b2ae35u;
  return x ^ (x >> 16);
}

// The value of a scale byte (e8m0: 0 is 2^-127, 255 is NaN).
__device__ __forceinline__ float scale_of(unsigned b) {
  const uint32_t bits = b == 0 ? 0x00400000u : b == 255 ? 0x7fc00000u : b << 23;
  return __builtin_bit_cast(float, bits);
}

struct E4M3 {
  static constexpr int kBits = 3, kLow = -6, kTop = 7;
  static constexpr bool kFloor = false;
  static __device__ __forceinline__ void up(int x, float (&v)[4]) {
    const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(x, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(x, true);
    v[0] = lo[0]; v[1] = lo[1]; v[2] = hi[0]; v[3] = hi[1];
  }
  static __device__ __forceinline__ int down(const float (&v)[4]) {
    return __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false), true);
  }
};
struct E5M2 {
  static constexpr int kBits = 2, kLow = -14, kTop = 14;
  static constexpr bool kFloor = true;  // a positive value stays positive
  static __device__ __forceinline__ void up(int x, float (&v)[4]) {
    const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_bf8(x, false), hi = __builtin_amdgcn_cvt_pk_f32_bf8(x, true);
    v[0] = lo[0]; v[1] = lo[1]; v[2] = hi[0]; v[3] = hi[1];
  }
  static __device__ __forceinline__ int down(const float (&v)[4]) {
    return __builtin_amdgcn_cvt_pk_bf8_f32(v[2], v[3], __builtin_amdgcn_cvt_pk_bf8_f32(v[0], v[1], 0, false), true);
  }
};

// The 8-bit values of this lane's four elements of a block, and the block's scale byte (in every
// lane of its row).  random: 16 bits per element.
template <typename F>
__device__ __forceinline__ int round8(const float (&x)[4], const uint32_t (&random)[4], unsigned& scale) {
  float big = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));  // (NaN drops out)
  big = row16_reduce(big, 0.0f, Max());
  // infinities leave the scale to the others, which they would take to zero (looked at when there is
  // one: 444 and 715 us as without it, a select for every element takes 450 and 728)
  if (__builtin_expect(__any(big == INFINITY), 0)) {
    big = 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k) big = fmaxf(big, fabsf(x[k]) < INFINITY ? fabsf(x[k]) : 0.0f);
    big = row16_reduce(big, 0.0f, Max());
  }
  // the exponent of the largest magnitude (0 and subnormal numbers end at the lowest scale)
  const int top = static_cast<int>(__builtin_bit_cast(uint32_t, big) >> 23) - 127;
  int e = top - F::kTop;
  e = e < -126 ? -126 : e;
  scale = static_cast<unsigned>(e + 127);
  float q[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float y = __builtin_ldexpf(x[k], -e), a = fabsf(y);
    // the distance of the type's neighbours around y is 2^unit
    int unit = static_cast<int>(__builtin_bit_cast(uint32_t, a) >> 23) - 127;
    unit = (unit < F::kLow ? F::kLow : unit) - F::kBits;
    // up where the place between the neighbours and the random fraction make one or more; nothing
    // here rounds (a sum of the two would)
    const float at = __builtin_ldexpf(a, -unit);
    float t = __builtin_floorf(at);
    t += at - t >= 1.0f - static_cast<float>(random[k]) * 0x1p-16f ? 1.0f : 0.0f;
    if (F::kFloor) t = y > 0.0f && t == 0.0f ? 1.0f : t;
    q[k] = __builtin_copysignf(__builtin_ldexpf(t, unit), y);
  }
  return F::down(q);
}

// The update of one element.  The moments' products and sums round one by one (no multiply-add):
// a last bit decides now and then which 8-bit value is taken, and this way any implementation of
// the formula in fp32 takes the same.
template <int kMode>
__device__ __forceinline__ void element(float& p, float g, float& m, float& v, const AdamWConst& c) {
#pragma clang fp contract(off)
  if (kMode == kCoupled) g = __builtin_fmaf(c.wd, p, g);
  m = c.beta1 * m + c.one_m_beta1 * g;
  v = c.beta2 * v + c.one_m_beta2 * g * g;
  // the update is not rounded into the state: root and reciprocal within one unit of the last place
  // (scaled where v is subnormal, which the instruction takes for zero)
  const float vhat = v * c.inv_bc2;
  const bool tiny = vhat < 0x1p-96f;
  const float root = __builtin_amdgcn_sqrtf(tiny ? vhat * 0x1p32f : vhat) * (tiny ? 0x1p-16f : 1.0f);
  const float upd = (m * c.inv_bc1) * __builtin_amdgcn_rcpf(root + c.eps);
  if (kMode != kCoupled) {
    const float keep = 1.0f - c.lr * c.wd;
    p = p * ((kMode == kDecoupledCautious && !(upd * p > 0.0f)) ? 1.0f : keep);
  }
  p = __builtin_fmaf(-c.lr, upd, p);
}

template <int kMode>
__global__ __launch_bounds__(kThreads) void adamw_byte_kernel(AdamWByteTable table) {
  const AdamWByteTable* kt = (const AdamWByteTable*)__builtin_amdgcn_kernarg_segment_ptr();
  (void)table;
  const uint32_t b = blockIdx.x;
  int s = 0;
  for (int i = 1; i < kt->nseg; ++i)
    if (b >= kt->block_start[i]) s = i;
  const AdamWConst& c = kt->c;
  const AdamWByteSegment& seg = kt->seg[s];
  const int64_t n = seg.n;
  const int64_t base = static_cast<int64_t>(b - kt->block_start[s]) * kChunk + threadIdx.x * kEach;
  const int grad_type = seg.types & 3, copy_type = seg.types >> 2;

  Pack<float, 4>::type P[kGroups], G[kGroups];
  Pack<unsigned short, 4>::type H[kGroups];
  int M[kGroups], V[kGroups];
  unsigned ms[kGroups], vs[kGroups];
  int cnt[kGroups];
#pragma unroll
  for (int u = 0; u < kGroups; ++u) {
    const int64_t i = base + static_cast<int64_t>(u) * (kThreads * kEach);
    cnt[u] = n - i >= kEach ? kEach : n - i > 0 ? static_cast<int>(n - i) : 0;
    P[u] = 0.0f;
    M[u] = V[u] = 0;
    ms[u] = vs[u] = 127;
    if (cnt[u] == kEach) {
      P[u] = __builtin_nontemporal_load(reinterpret_cast<const Pack<float, 4>::type*>(seg.p + i));
      M[u] = __builtin_bit_cast(int, __builtin_nontemporal_load(reinterpret_cast<const Bytes*>(seg.m + i)));
      V[u] = __builtin_bit_cast(int, __builtin_nontemporal_load(reinterpret_cast<const Bytes*>(seg.v + i)));
    } else {
#pragma unroll
      for (int k = 0; k < kEach; ++k)
        if (k < cnt[u]) {
          P[u][k] = seg.p[i + k];
          M[u] |= seg.m[i + k] << (8 * k);
          V[u] |= seg.v[i + k] << (8 * k);
        }
    }
    if (cnt[u] > 0) {
      ms[u] = seg.ms[i / kAdamWByteBlock];
      vs[u] = seg.vs[i / kAdamWByteBlock];
    }
  }
  if (grad_type == kActF32) {
    const float* g = static_cast<const float*>(seg.g);
#pragma unroll
    for (int u = 0; u < kGroups; ++u) {
      const int64_t i = base + static_cast<int64_t>(u) * (kThreads * kEach);
      G[u] = 0.0f;
      if (cnt[u] == kEach) {
        G[u] = __builtin_nontemporal_load(reinterpret_cast<const Pack<float, 4>::type*>(g + i));
      } else {
#pragma unroll
        for (int k = 0; k < kEach; ++k)
          if (k < cnt[u]) G[u][k] = g[i + k];
      }
    }
  } else {
    const unsigned short* g = static_cast<const unsigned short*>(seg.g);
#pragma unroll
    for (int u = 0; u < kGroups; ++u) {
      const int64_t i = base + static_cast<int64_t>(u) * (kThreads * kEach);
      H[u] = 0;
      if (cnt[u] == kEach) {
        H[u] = __builtin_nontemporal_load(reinterpret_cast<const Pack<unsigned short, 4>::type*>(g + i));
      } else {
#pragma unroll
        for (int k = 0; k < kEach; ++k)
          if (k < cnt[u]) H[u][k] = g[i + k];
      }
    }
#pragma unroll
    for (int u = 0; u < kGroups; ++u)
#pragma unroll
      for (int k = 0; k < kEach; ++k) G[u][k] = grad_type == kActBF16 ? bf2f(H[u][k]) : h2f(H[u][k]);
  }

#pragma unroll
  for (int u = 0; u < kGroups; ++u) {
    const int64_t i = base + static_cast<int64_t>(u) * (kThreads * kEach);
    float m[kEach], v[kEach];
    E4M3::up(M[u], m);
    E5M2::up(V[u], v);
    const float mscale = scale_of(ms[u]), vscale = scale_of(vs[u]);
    const int64_t number = seg.first * kAdamWByteBlock + i;
    const uint32_t key = kt->key + static_cast<uint32_t>(number >> 32) * 0x9e3779b1u;
    const uint32_t spread = static_cast<uint32_t>(number) * 0x9e3779b1u;
    uint32_t mr[kEach], vr[kEach];
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      m[k] *= mscale;
      v[k] *= vscale;
      float p = P[u][k];
      element<kMode>(p, G[u][k], m[k], v[k], c);
      P[u][k] = p;
      // elements behind the end must not enter their block's scale
      if (k >= cnt[u]) m[k] = v[k] = 0.0f;
      // (a group of four never passes a multiple of 2^32)
      const uint32_t bits = mix((spread + k * 0x9e3779b1u) ^ key);
      mr[k] = bits & 0xffffu;
      vr[k] = bits >> 16;
    }
    M[u] = round8<E4M3>(m, mr, ms[u]);
    V[u] = round8<E5M2>(v, vr, vs[u]);
    if (cnt[u] == kEach) {
      __builtin_nontemporal_store(P[u], reinterpret_cast<Pack<float, 4>::type*>(seg.p + i));
      __builtin_nontemporal_store(__builtin_bit_cast(Bytes, M[u]), reinterpret_cast<Bytes*>(seg.m + i));
      __builtin_nontemporal_store(__builtin_bit_cast(Bytes, V[u]), reinterpret_cast<Bytes*>(seg.v + i));
    } else {
#pragma unroll
      for (int k = 0; k < kEach; ++k)
        if (k < cnt[u]) {
          seg.p[i + k] = P[u][k];
          seg.m[i + k] = static_cast<unsigned char>(M[u] >> (8 * k));
          seg.v[i + k] = static_cast<unsigned char>(V[u] >> (8 * k));
        }
    }
    if ((threadIdx.x & 15) == 0 && cnt[u] > 0) {
      seg.ms[i / kAdamWByteBlock] = static_cast<unsigned char>(ms[u]);
      seg.vs[i / kAdamWByteBlock] = static_cast<unsigned char>(vs[u]);
    }
    if (copy_type != kActF32) {
      Pack<unsigned short, 4>::type x;
#pragma unroll
      for (int k = 0; k < kEach; ++k) x[k] = copy_type == kActBF16 ? f2bf(P[u][k]) : f2h(P[u][k]);
      if (cnt[u] == kEach) {
        __builtin_nontemporal_store(x, reinterpret_cast<Pack<unsigned short, 4>::type*>(seg.copy + i));
      } else {
#pragma unroll
        for (int k = 0; k < kEach; ++k)
          if (k < cnt[u]) seg.copy[i + k] = x[k];
      }
    }
  }
}

// The same on the host.
uint32_t mix_host(uint32_t x) {
  x = (x ^ (x >> 16)) * 0x85ebca6bu;
  x = (x ^ (x >> 13)) * 0xc2b2ae35u;
  return x ^ (x >> 16);
}

}  // namespace

int64_t adamw_byte_blocks(int64_t n) { return (n + kChunk - 1) / kChunk; }

uint32_t adamw_byte_key(uint64_t seed, int64_t step) {
  const uint32_t a = mix_host(static_cast<uint32_t>(seed)) ^ static_cast<uint32_t>(seed >> 32);
  return mix_host(mix_host(a) ^ static_cast<uint32_t>(step));
}

hipError_t launch_adamw_byte(const AdamWByteTable& t, hipStream_t s) {
  const uint32_t blocks = t.block_start[t.nseg];
  if (blocks == 0) return hipSuccess;
  switch (decay_mode(t.c)) {
    case kCoupled: hipLaunchKernelGGL(adamw_byte_kernel<kCoupled>, dim3(blocks), dim3(kThreads), 0, s, t); break;
    case kDecoupledCautious:
      hipLaunchKernelGGL(adamw_byte_kernel<kDecoupledCautious>, dim3(blocks), dim3(kThreads), 0, s, t);
      break;
    default: hipLaunchKernelGGL(adamw_byte_kernel<kDecoupled>, dim3(blocks), dim3(kThreads), 0, s, t); break;
  }
  return hipGetLastError();
}

}  // namespace ma

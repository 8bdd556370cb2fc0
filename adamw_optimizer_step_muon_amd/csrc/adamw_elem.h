// The AdamW update of one element, shared by every kernel that steps AdamW state.
#pragma once

#include "ma_internal.h"

namespace ma {

// Decay variants, fixed per launch so the vector kernel's body has no branches.
enum DecayMode { kDecoupled = 0, kDecoupledCautious = 1, kCoupled = 2 };

// The multiply-adds are explicit (fmaf) and nothing else is contracted: every kernel
// (flat vector, flat scalar, multi-tensor) rounds the same operations, so an element's
// result does not depend on which kernel updated it (left to the compiler, p keep -
// lr upd was fused differently in different kernels).  g + wd p (coupled decay) keeps a
// single rounding, which matters where the two terms cancel.
template <int kMode>
__device__ __forceinline__ void adamw_elem_t(float& p, float g, float& m, float& v,
                                             const AdamWConst& c) {
#pragma clang fp contract(off)
  if (kMode == kCoupled) g = __builtin_fmaf(c.wd, p, g);
  m = __builtin_fmaf(c.beta1, m, c.one_m_beta1 * g);
  v = __builtin_fmaf(c.beta2, v, c.one_m_beta2 * (g * g));
  const float mhat = m * c.inv_bc1;
  const float vhat = v * c.inv_bc2;
  const float upd = mhat / (__builtin_sqrtf(vhat) + c.eps);
  if (kMode != kCoupled) {
    const float keep = 1.0f - c.lr * c.wd;
    p = p * ((kMode == kDecoupledCautious && !(upd * p > 0.0f)) ? 1.0f : keep);
  }
  p = __builtin_fmaf(-c.lr, upd, p);
}

__device__ __forceinline__ void adamw_elem(float& p, float g, float& m, float& v,
                                           const AdamWConst& c) {
  if (!c.decoupled) adamw_elem_t<kCoupled>(p, g, m, v, c);
  else if (c.cautious) adamw_elem_t<kDecoupledCautious>(p, g, m, v, c);
  else adamw_elem_t<kDecoupled>(p, g, m, v, c);
}

inline int decay_mode(const AdamWConst& c) {
  return !c.decoupled ? kCoupled : c.cautious ? kDecoupledCautious : kDecoupled;
}

}  // namespace ma

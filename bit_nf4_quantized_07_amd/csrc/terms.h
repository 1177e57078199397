// fp32 values as sums of bf16 terms, for MFMA operands.
#pragma once
#include "device_common.h"

namespace qlk {

// x as two bf16 terms, hi + mid2, and as three, hi + mid3 + lo.  A product with
// an infinity has to be what x's own would be, so every term has x's sign and is
// zero only where x is:
//  * hi and mid3 are cut toward zero, which also keeps them finite where x lies
//    above bf16's largest value.  Cut, three terms hold all 24 bits of x; of two
//    the last is rounded (within 2^-16 of x; a first term rounded either way
//    would save one bit more but leave a rest of either sign).
//  * a term that would be zero is 2^-40 of hi, far below the others' rounding (a
//    normal number for |x| down to 2^-86).
//  * all terms of an infinity or NaN are x.
__device__ __forceinline__ uint16_t cut_to_bf16(float x) { return (uint16_t)(__float_as_uint(x) >> 16); }
struct Terms {
  uint16_t hi, mid2, mid3, lo;
};
__device__ __forceinline__ Terms split(float x) {
  if (!__builtin_isfinite(x)) {
    const uint16_t v = f32_to_bf16(x);   // a NaN stays one
    return {v, v, v, v};
  }
  Terms t;
  t.hi = cut_to_bf16(x);
  const float hi = bf16_to_f32(t.hi), rest = x - hi;
  t.mid2 = f32_to_bf16(rest);
  t.mid3 = cut_to_bf16(rest);
  t.lo = f32_to_bf16(rest - bf16_to_f32(t.mid3));   // exact
  const uint16_t tiny = f32_to_bf16(hi * 0x1p-40f);
  if ((t.mid2 & 0x7fffu) == 0) t.mid2 = tiny;
  if ((t.mid3 & 0x7fffu) == 0) t.mid3 = tiny;
  if ((t.lo & 0x7fffu) == 0) t.lo = tiny;
  return t;
}

}  // namespace qlk

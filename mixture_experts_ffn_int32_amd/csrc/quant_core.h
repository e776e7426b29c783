// The E4M3 quantisation rule, shared by the quantisers and the products that quantise their own rows.
#pragma once

#include "device.h"

namespace hmm {

// 448 / max|x| in float32; an all-zero row or group gets 1.  Below a largest
// value of about 1.3e-36 (bf16 holds values down to ~9e-41) the quotient
// overflows: it is clamped to the largest finite float32, so the codes stay
// finite (x * scale is then at most ~448) and the descale 1 / scale is a
// subnormal float32 (about 2.9e-39) instead of 0.
__device__ __forceinline__ float scale_of(float absmax) {
  return absmax > 0.f ? fminf(448.f / absmax, 3.40282347e38f) : 1.f;
}

// The rule of the 128 x 128 block products (both operands): 448 times the reciprocal of
// max|x|, each rounded to float32, as tensor code evaluates 448 / max; it may differ from
// scale_of's quotient in the last bit.  The same clamp (1 / max overflows below 2.9e-39).
__device__ __forceinline__ float block_scale_of(float absmax) {
  return absmax > 0.f ? fminf((1.f / absmax) * 448.f, 3.40282347e38f) : 1.f;
}

// 8 floats * scale -> 8 E4M3 bytes
__device__ __forceinline__ uint2 to_e4m3x8(const float (&v)[8], const float (&s)[8]) {
  int lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * s[0], v[1] * s[1], 0, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2] * s[2], v[3] * s[3], lo, true);
  int hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4] * s[4], v[5] * s[5], 0, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6] * s[6], v[7] * s[7], hi, true);
  return make_uint2((unsigned)lo, (unsigned)hi);
}

}  // namespace hmm

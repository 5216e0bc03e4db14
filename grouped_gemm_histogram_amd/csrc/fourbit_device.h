// fourbit_device.h -- 4-bit codes to bf16 MFMA operands, shared by the 4-bit products and the layer for few tokens.
#pragma once

#include "device_common.h"

namespace moe {

typedef __attribute__((__vector_size__(4 * sizeof(uint32_t)))) uint32_t u32x4;
typedef __attribute__((__vector_size__(2 * sizeof(__bf16)))) __bf16 bf16x2;

__device__ __forceinline__ bf16x8 as_bf16x8(uint4 v) { return __builtin_bit_cast(bf16x8, v); }

// 4 x 4 transpose of words between the four 16-lane rows of a wave: word j of row q becomes
// word q of row j
__device__ __forceinline__ void transpose4(uint32_t (&r)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {   // upper half of r[i] with lower half of r[i + 2]
    const auto s = __builtin_amdgcn_permlane32_swap(r[i], r[i + 2], false, false);
    r[i] = s[0];
    r[i + 2] = s[1];
  }
#pragma unroll
  for (int i = 0; i < 4; i += 2) {   // odd rows of r[i] with even rows of r[i + 1]
    const auto s = __builtin_amdgcn_permlane16_swap(r[i], r[i + 1], false, false);
    r[i] = s[0];
    r[i + 1] = s[1];
  }
}

// eight int4 codes -> bf16 0 to 15, in the channel order 0 2 4 6 1 3 5 7: as an e4m3 byte a code
// is code * 2^-9 (subnormal below 8, and the first binade goes on in the same steps)
__device__ __forceinline__ uint4 unpack_int4(uint32_t v) {
  const uint32_t even = v & 0x0f0f0f0fu, odd = (v >> 4) & 0x0f0f0f0fu;
  uint4 r;
  r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(even, 512.0f, false));
  r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(even, 512.0f, true));
  r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(odd, 512.0f, false));
  r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(odd, 512.0f, true));
  return r;
}

// the same in channel order, at two more moves
__device__ __forceinline__ uint4 unpack_int4_ordered(uint32_t v) {
  const uint32_t even = v & 0x0f0f0f0fu, odd = (v >> 4) & 0x0f0f0f0fu;
  const uint32_t lo = __builtin_amdgcn_perm(odd, even, 0x05010400u), hi = __builtin_amdgcn_perm(odd, even, 0x07030602u);
  uint4 r;
  r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, false));
  r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 512.0f, true));
  r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, false));
  r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 512.0f, true));
  return r;
}

// eight activations into unpack_int4's order
__device__ __forceinline__ uint4 order_int4(uint4 a) {
  return make_uint4(__builtin_amdgcn_perm(a.y, a.x, 0x05040100u), __builtin_amdgcn_perm(a.w, a.z, 0x05040100u),
                    __builtin_amdgcn_perm(a.y, a.x, 0x07060302u), __builtin_amdgcn_perm(a.w, a.z, 0x07060302u));
}

// eight e2m1 codes -> bf16 code * 2^(e8m0 - 127), in channel order; the conversion takes its scale
// from an f32's exponent bits
__device__ __forceinline__ uint4 unpack_mxfp4(uint32_t v, uint32_t e8m0) {
  const float scale = __uint_as_float(e8m0 << 23);
  uint4 r;
  r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, 0));
  r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, 1));
  r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, 2));
  r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, 3));
  return r;
}

}  // namespace moe

// One block of the MXFP4 conversion (FORMAT F29), on one lane: shared by the quantizer and by the
// decode batches that convert their rows on the way.
#pragma once

#include "tq_device.h"

namespace tq {

struct Fp4Block {
  u32x4 codes;     // 32 E2M1 codes, the even element in the low nibble
  uint32_t scale;  // the E8M0 byte
};

// The E8M0 byte of a block whose largest magnitude has the bf16 bits m (m < 0x8000): the
// smallest power of two 2^k, k >= -127, with max <= 7 * 2^k (7 = 1.75 * 2^2); 127 for a zero
// block, 255 for one with an infinity or NaN.
__device__ __forceinline__ uint32_t fp4_scale_byte(uint32_t m) {
  const int b = (int)(m >> 7) - 2 + ((m & 0x7Fu) > 0x60u ? 1 : 0);
  return m >= 0x7F80u ? 255u : m == 0u ? 127u : (uint32_t)max(b, 0);
}

// 32 bf16 values. The hardware conversion divides by the scale (a power of two, so exactly),
// rounds to the nearest E2M1 value, ties to the even code, and keeps 6 for what lies above it.
__device__ __forceinline__ Fp4Block fp4_block(const u32x4 (&x)[4]) {
  u16x2 top = {0, 0};
#pragma unroll
  for (int j = 0; j < 16; ++j)
    top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, x[j >> 2][j & 3] & 0x7FFF7FFFu));
  const uint32_t b = fp4_scale_byte(max((uint32_t)top.x, (uint32_t)top.y));
  // 2^(b - 127) as fp32: the byte is the exponent field, 0 the subnormal 2^-127
  const float scale = __uint_as_float(b == 0u ? 0x00400000u : b << 23);
  Fp4Block r;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t v[4] = {x[j].x, x[j].y, x[j].z, x[j].w};  // (a vector's element cannot be bit-cast)
    uint32_t c = 0;
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, v[0]), scale, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, v[1]), scale, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, v[2]), scale, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, v[3]), scale, 3);
    r.codes[j] = b == 255u ? 0u : c;
  }
  r.scale = b;
  return r;
}

}  // namespace tq

// bf16 rows in MXFP4 (gfx950; FORMAT F29): one thread per block of 32 inputs. The largest
// magnitude's exponent and mantissa give the scale byte; the hardware conversion divides by
// the scale (a power of two, so exactly), rounds to the nearest E2M1 value, ties to the even
// code, and keeps 6 for what lies above it. Bound by memory: 2 bytes read and 17 / 32 written
// per element.
#include "tq_device.h"
#include "tq_internal.h"

namespace tq {

namespace {

// The E8M0 byte of a block whose largest magnitude has the bf16 bits m (m < 0x8000): the
// smallest power of two 2^k, k >= -127, with max <= 7 * 2^k (7 = 1.75 * 2^2); 127 for a zero
// block, 255 for one with an infinity or NaN.
__device__ __forceinline__ uint32_t fp4_scale_byte(uint32_t m) {
  const int b = (int)(m >> 7) - 2 + ((m & 0x7Fu) > 0x60u ? 1 : 0);
  return m >= 0x7F80u ? 255u : m == 0u ? 127u : (uint32_t)max(b, 0);
}

__global__ __launch_bounds__(256) void mxfp4_quantize_kernel(const uint4* __restrict__ x,
                                                             int64_t nblocks,
                                                             uint4* __restrict__ codes,
                                                             uint8_t* __restrict__ scales) {
  const int64_t blk = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (blk >= nblocks) return;
  uint32_t v[16];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint4 u = x[4 * blk + q];
    v[4 * q] = u.x;
    v[4 * q + 1] = u.y;
    v[4 * q + 2] = u.z;
    v[4 * q + 3] = u.w;
  }
  u16x2 top = {0, 0};
#pragma unroll
  for (int j = 0; j < 16; ++j)
    top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, v[j] & 0x7FFF7FFFu));
  const uint32_t b = fp4_scale_byte(max((uint32_t)top.x, (uint32_t)top.y));
  // 2^(b - 127) as fp32: the byte is the exponent field, 0 the subnormal 2^-127
  const float scale = __uint_as_float(b == 0u ? 0x00400000u : b << 23);
  uint32_t c[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t* p = v + 4 * j;
    uint32_t r = 0;
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2, p[0]), scale, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2, p[1]), scale, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2, p[2]), scale, 2);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2, p[3]), scale, 3);
    c[j] = b == 255u ? 0u : r;
  }
  codes[blk] = make_uint4(c[0], c[1], c[2], c[3]);
  scales[blk] = (uint8_t)b;
}

}  // namespace

hipError_t launch_mxfp4_quantize(const uint16_t* x, int64_t rows, int n, uint8_t* codes,
                                 uint8_t* scales, hipStream_t s) {
  const int64_t nblocks = rows * (n / 32);
  if (nblocks == 0) return hipSuccess;
  hipLaunchKernelGGL(mxfp4_quantize_kernel, dim3((unsigned)((nblocks + 255) / 256)), dim3(256), 0,
                     s, reinterpret_cast<const uint4*>(x), nblocks,
                     reinterpret_cast<uint4*>(codes), scales);
  return hipGetLastError();
}

}  // namespace tq

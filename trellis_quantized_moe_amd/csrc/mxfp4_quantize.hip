// bf16 rows in MXFP4 (gfx950; FORMAT F29): one thread per block of 32 inputs (mxfp4_quant.h).
// Bound by memory: 2 bytes read and 17 / 32 written per element (49,152 x 5,120: 135 us, 4.7 TB/s; 64 x
// 5,120: 2.6 us, latency). Four lanes to a block, which load and store whole lines, took 138 and 2.9.
#include "mxfp4_quant.h"
#include "tq_internal.h"

namespace tq {

namespace {

__global__ __launch_bounds__(256) void mxfp4_quantize_kernel(const u32x4* __restrict__ x,
                                                             int64_t nblocks,
                                                             u32x4* __restrict__ codes,
                                                             uint8_t* __restrict__ scales) {
  const int64_t blk = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (blk >= nblocks) return;
  u32x4 v[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) v[q] = x[4 * blk + q];
  const Fp4Block r = fp4_block(v);
  codes[blk] = r.codes;
  scales[blk] = (uint8_t)r.scale;
}

}  // namespace

hipError_t launch_mxfp4_quantize(const uint16_t* x, int64_t rows, int n, uint8_t* codes,
                                 uint8_t* scales, hipStream_t s) {
  const int64_t nblocks = rows * (n / 32);
  if (nblocks == 0) return hipSuccess;
  hipLaunchKernelGGL(mxfp4_quantize_kernel, dim3((unsigned)((nblocks + 255) / 256)), dim3(256), 0,
                     s, reinterpret_cast<const u32x4*>(x), nblocks,
                     reinterpret_cast<u32x4*>(codes), scales);
  return hipGetLastError();
}

}  // namespace tq

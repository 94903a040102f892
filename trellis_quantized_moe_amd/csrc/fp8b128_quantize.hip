// fp8b128_quantize (FORMAT F23): bf16 rows to E4M3 codes with one power-of-two scale per 128
// inputs of a row.
//
// A block is 16 lanes of 8 inputs: each lane takes the largest magnitude of its eight bf16
// patterns (as integers: the order of non-negative floats is that of their bits), four
// exchanges give the block's, and the exponent of the scale follows from the pattern alone:
// magnitude (1 + m / 128) 2^(E - 127) is at most 448 * 2^k = 1.75 * 2^(8 + k) for k = E - 135
// if m <= 96, else for k = E - 134. x * 2^-k is exact, so each code is one rounding of x.
// Bound by memory: 2 bytes read and 1 written per input, 8,192 x 5,120 in 22 to 23 us (5.6 TB/s).
#include "fp8b128.h"

namespace tq {

namespace {

constexpr int FQ_THREADS = 256;

__global__ __launch_bounds__(FQ_THREADS) void fp8b128_quantize_kernel(
    const uint16_t* __restrict__ x, int64_t blocks, int n, int nb, uint8_t* __restrict__ codes,
    float* __restrict__ scales) {
  const int64_t blk = (int64_t)blockIdx.x * (FQ_THREADS / 16) + (threadIdx.x >> 4);
  if (blk >= blocks) return;  // whole groups of 16 lanes
  const int lane = threadIdx.x & 15;
  const int64_t row = blk / nb;
  const int b = (int)(blk % nb);
  const int col = b * FB_BLOCK + 8 * lane;
  const bool in = col < n;  // n is a multiple of 16: a lane is inside or outside
  const u32x4 v = in ? *reinterpret_cast<const u32x4*>(x + row * n + col) : (u32x4){0, 0, 0, 0};
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    top = max(top, v[j] & 0x7FFFu);
    top = max(top, (v[j] >> 16) & 0x7FFFu);
  }
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) top = max(top, (uint32_t)__shfl_xor((int)top, d, 16));
  const int E = (int)(top >> 7), m = (int)(top & 127u);
  int k = max(m <= 96 ? E - 135 : E - 134, -126);
  if (top == 0) k = 0;
  const bool finite = top < 0x7F80u;
  const float inv = finite ? __uint_as_float((uint32_t)(127 - k) << 23) : 0.0f;
  u32x2 out = (u32x2){0, 0};
  if (finite) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(bf16_lo_to_f32(v[2 * j]) * inv,
                                                     bf16_hi_to_f32(v[2 * j]) * inv, 0, false);
      out[j] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(bf16_lo_to_f32(v[2 * j + 1]) * inv,
                                                         bf16_hi_to_f32(v[2 * j + 1]) * inv, lo,
                                                         true);
    }
  }
  if (in) *reinterpret_cast<u32x2*>(codes + row * n + col) = out;
  if (lane == 0)
    scales[row * nb + b] = finite ? __uint_as_float((uint32_t)(k + 127) << 23)
                                  : __uint_as_float(0x7FC00000u);
}

}  // namespace

hipError_t launch_fp8b128_quantize(const uint16_t* x, int64_t rows, int n, uint8_t* codes,
                                   float* scales, hipStream_t s) {
  const int nb = (n + FB_BLOCK - 1) / FB_BLOCK;
  const int64_t blocks = rows * nb;
  const int per = FQ_THREADS / 16;
  hipLaunchKernelGGL(fp8b128_quantize_kernel, dim3((unsigned)((blocks + per - 1) / per)),
                     dim3(FQ_THREADS), 0, s, x, blocks, n, nb, codes, scales);
  return hipGetLastError();
}

}  // namespace tq

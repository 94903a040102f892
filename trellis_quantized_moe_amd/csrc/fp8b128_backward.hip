// The gradients of a product over the fp8b128 store (FORMAT F26), on the bf16 matrix cores:
//   dx[t][i] = sum over o of dy[t][o] * W[o][i],    W = scale of the block * code
//   dw[o][i] = sum over t of dy[t][o] * X[t][i],    X = scale of the token's block * code
// Inputs are the A operand, so a lane ends with four consecutive inputs of a token or channel.
#include "fp8b128.h"

namespace tq {

namespace {

__device__ __forceinline__ u32x4 pack8(const uint16_t v[8]) {
  return (u32x4){(uint32_t)v[0] | (uint32_t)v[1] << 16, (uint32_t)v[2] | (uint32_t)v[3] << 16,
                 (uint32_t)v[4] | (uint32_t)v[5] << 16, (uint32_t)v[6] | (uint32_t)v[7] << 16};
}

// One 16 x 16 tile per wave; the sums over each 128 outputs are scaled by their block's scale.
__global__ __launch_bounds__(256) void fp8b128_dx_kernel(Fp8b128BackwardArgs a) {
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int64_t tile = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int cols = a.in / 16;
  const int64_t t = tile / cols * 16 + r;
  const int i0 = (int)(tile % cols) * 16;
  if (tile / cols * 16 >= a.T) return;
  f32x4 acc = (f32x4){0.f, 0.f, 0.f, 0.f};
  for (int ob = 0; ob * 128 < a.out; ++ob) {
    f32x4 p = (f32x4){0.f, 0.f, 0.f, 0.f};
    for (int o0 = ob * 128; o0 < min(ob * 128 + 128, a.out); o0 += 32) {
      const int o = o0 + 8 * q;
      uint32_t c[2] = {0, 0};
      u32x4 b = (u32x4){0, 0, 0, 0};
      if (o < a.out) {
        for (int j = 0; j < 8; ++j)
          c[j / 4] |= (uint32_t)a.w[(int64_t)(o + j) * a.in + i0 + r] << (8 * (j % 4));
        if (t < a.T) b = *reinterpret_cast<const u32x4*>(a.dy + t * a.out + o);
      }
      p = mfma_bf16(fb_bf16_of8(c[0], c[1]), b, p);
    }
    const float s = a.ws[(int64_t)ob * a.nb + i0 / 128];
    for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(p[i], s, acc[i]);
  }
  if (t < a.T)
    *reinterpret_cast<u32x2*>(a.dx + t * a.in + i0 + 4 * q) =
        (u32x2){fb_pack_bf16(acc[0], acc[1]), fb_pack_bf16(acc[2], acc[3])};
}

// One 16 x 16 tile per wave. X is rounded to bf16 (exact for scales that are powers of two,
// which fp8b128_quantize writes).
__global__ __launch_bounds__(256) void fp8b128_dw_kernel(Fp8b128BackwardArgs a) {
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int64_t tile = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int cols = a.in / 16;
  const int o = (int)(tile / cols) * 16 + r;
  const int i0 = (int)(tile % cols) * 16;
  if (tile / cols * 16 >= a.out) return;
  f32x4 acc = (f32x4){0.f, 0.f, 0.f, 0.f};
  for (int64_t t0 = 0; t0 < a.T; t0 += 32) {
    uint16_t x[8], d[8];
    for (int j = 0; j < 8; ++j) {
      const int64_t t = t0 + 8 * q + j;
      x[j] = d[j] = 0;
      if (t < a.T) {
        const uint32_t c = a.x[t * a.in + i0 + r];
        const float v = bf16_lo_to_f32(fb_bf16_of4(c).x) * a.xs[t * a.nb + i0 / 128];
        x[j] = (uint16_t)fb_pack_bf16(v, 0.0f);
        d[j] = a.dy[t * a.out + o];
      }
    }
    acc = mfma_bf16(pack8(x), pack8(d), acc);
  }
  *reinterpret_cast<u32x2*>(a.dw + (int64_t)o * a.in + i0 + 4 * q) =
      (u32x2){fb_pack_bf16(acc[0], acc[1]), fb_pack_bf16(acc[2], acc[3])};
}

}  // namespace

hipError_t launch_fp8b128_dx(const Fp8b128BackwardArgs& a, hipStream_t s) {
  const int64_t tiles = (a.T + 15) / 16 * (a.in / 16);
  return launch_timed(fp8b128_dx_kernel, dim3((unsigned)((tiles + 3) / 4)), dim3(256), s, a);
}

hipError_t launch_fp8b128_dw(const Fp8b128BackwardArgs& a, hipStream_t s) {
  const int64_t tiles = (int64_t)(a.out / 16) * (a.in / 16);
  hipLaunchKernelGGL(fp8b128_dw_kernel, dim3((unsigned)((tiles + 3) / 4)), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace tq

// Device pieces shared by the kernels of the fp8b128 store (FORMAT F22-F25): E4M3 codes with
// one fp32 scale per 128 x 128 block of a weight and per 128 inputs of an activation row.
#pragma once

#include "gemm_core.h"

namespace tq {

typedef int32_t i32x8 __attribute__((ext_vector_type(8)));

constexpr int FB_BLOCK = 128;         // inputs (and outputs) per scale
constexpr uint32_t FB_OOB = 0x80000000u;  // a buffer offset past every resource: loads give 0

// Four E4M3 codes as four bf16 values (exact: bf16 holds every E4M3 value).
__device__ __forceinline__ u32x2 fb_bf16_of4(uint32_t c) {
  u32x2 r;
  r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.0f, false));
  r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.0f, true));
  return r;
}
// Eight E4M3 codes as one bf16 matrix-core operand.
__device__ __forceinline__ u32x4 fb_bf16_of8(uint32_t c0, uint32_t c1) {
  const u32x2 a = fb_bf16_of4(c0), b = fb_bf16_of4(c1);
  return (u32x4){a.x, a.y, b.x, b.y};
}

// Two fp32 values rounded to bf16 (nearest, ties to even), packed.
__device__ __forceinline__ uint32_t fb_pack_bf16(float lo, float hi) {
  const bf16x2 h = __builtin_convertvector((f32x2){lo, hi}, bf16x2);
  return __builtin_bit_cast(uint32_t, h);
}

// The sum over one block of 128 inputs of the products of two rows' codes, for a 16 x 16 tile:
// lane (r = l % 16, q = l / 16) holds bytes 16 q .. 16 q + 15 and 64 + 16 q .. 64 + 16 q + 15
// of row r of A and of row r of B; result element i is D[4 q + i][r].
//
// EXACT: the codes become bf16 (exactly) and four v_mfma_f32_16x16x32_bf16 add the exact
// products in fp32. Else one v_mfma_f32_16x16x128_f8f6f4, at twice the rate: the fp8 matrix
// cores align the products of an instruction to the largest one and drop bits below about
// 2^-17 of it (measured on block-scaled normal data: 1.5e-5 to 5e-5 of a block's sum in the
// 2-norm, unbiased, against 1e-8 with bf16), which is far below half a step of a bf16
// result (2^-9) and is used only where the result is rounded to bf16.
template <bool EXACT>
struct FbOperand;  // 32 codes of a row, as the matrix cores take them
template <>
struct FbOperand<true> {
  u32x4 v[4];
  __device__ __forceinline__ void set(u32x4 lo, u32x4 hi) {
    v[0] = fb_bf16_of8(lo.x, lo.y);
    v[1] = fb_bf16_of8(lo.z, lo.w);
    v[2] = fb_bf16_of8(hi.x, hi.y);
    v[3] = fb_bf16_of8(hi.z, hi.w);
  }
};
template <>
struct FbOperand<false> {
  i32x8 v;
  __device__ __forceinline__ void set(u32x4 lo, u32x4 hi) {
    v = __builtin_bit_cast(i32x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  }
};

__device__ __forceinline__ f32x4 fb_block_product(const FbOperand<true>& a, const FbOperand<true>& b) {
  f32x4 p = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < 4; ++j) p = mfma_bf16(a.v[j], b.v[j], p);
  return p;
}
__device__ __forceinline__ f32x4 fb_block_product(const FbOperand<false>& a, const FbOperand<false>& b) {
  // scale operands of zero select the instruction without block scales
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.v, b.v, (f32x4){0.f, 0.f, 0.f, 0.f}, 0,
                                                          0, 0, 0, 0, 0);
}

// The tile of this workgroup: the grid is read as 8 interleaved streams, one per XCD, each a
// contiguous range of tiles in an order that walks 4 channel tiles per token tile, so that the
// tiles an XCD works on at one time share rows of both operands in its L2.
__device__ inline bool fb_tile_of(int tt, int tc, int* t, int* c) {
  const int n = tt * tc, per = (n + 7) >> 3, j = blockIdx.x >> 3;
  const int u = (blockIdx.x & 7) * per + j;
  if (j >= per || u >= n) return false;
  const int band = u / (4 * tt), first = 4 * band, width = min(4, tc - first);
  const int v = u - first * tt;
  *c = first + v % width;
  *t = v / width;
  return true;
}

// ---- epilogues ------------------------------------------------------------------------------
// What a forward kernel does with the sums of four consecutive channels o .. o + 3 of one
// token (gated forms: g and u are the sums of gate and up channels o .. o + 3).
__device__ __forceinline__ float fb_sigmoid(float g) { return 1.0f / (1.0f + expf(-g)); }

template <int EPI>
__device__ __forceinline__ void fb_store(const Fp8b128GemmArgs& a, int64_t t, int o, f32x4 g,
                                         f32x4 u) {
  if constexpr (EPI == FB_F32) {
    *reinterpret_cast<f32x4*>(static_cast<float*>(a.y) + t * a.out + o) = g;
  } else if constexpr (EPI == FB_BF16) {
    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.y) + t * a.out + o) =
        (u32x2){fb_pack_bf16(g[0], g[1]), fb_pack_bf16(g[2], g[3])};
  } else if constexpr (EPI == FB_GATED) {
    float h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = g[i] * fb_sigmoid(g[i]) * u[i];
    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a.y) + t * (a.out / 2) + o) =
        (u32x2){fb_pack_bf16(h[0], h[1]), fb_pack_bf16(h[2], h[3])};
  } else {
    // d silu(g) / dg = s + g s (1 - s) with s = sigmoid(g); the two gradients are rounded to
    // bf16, the operand type of the two products that read them
    const u32x2 d2 = *reinterpret_cast<const u32x2*>(a.dh + t * (a.out / 2) + o);
    const float dh[4] = {bf16_lo_to_f32(d2.x), bf16_hi_to_f32(d2.x), bf16_lo_to_f32(d2.y),
                         bf16_hi_to_f32(d2.y)};
    float dg[4], du[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float s = fb_sigmoid(g[i]);
      dg[i] = dh[i] * u[i] * s * (1.0f + g[i] * (1.0f - s));
      du[i] = dh[i] * g[i] * s;
    }
    uint16_t* row = static_cast<uint16_t*>(a.y) + t * a.out + o;
    *reinterpret_cast<u32x2*>(row) = (u32x2){fb_pack_bf16(dg[0], dg[1]), fb_pack_bf16(dg[2], dg[3])};
    *reinterpret_cast<u32x2*>(row + a.out / 2) =
        (u32x2){fb_pack_bf16(du[0], du[1]), fb_pack_bf16(du[2], du[3])};
  }
}

constexpr bool fb_gated(int epi) { return epi == FB_GATED || epi == FB_GATED_GRAD; }

}  // namespace tq

// Device pieces shared by the kernels of the fp8b128 store (FORMAT F22-F25): E4M3 codes with
// one fp32 scale per 128 x 128 block of a weight and per 128 inputs of an activation row.
#pragma once

#include "gemm_core.h"

namespace tq {

typedef int32_t i32x8 __attribute__((ext_vector_type(8)));

constexpr int FB_BLOCK = 128;         // inputs (and outputs) per scale
constexpr uint32_t FB_OOB = 0x80000000u;  // a buffer offset past every resource: loads give 0

// A value at the same address for the whole wave, that the kernel does not write, through the
// scalar cache.
__device__ __forceinline__ float fb_uniform_load(const float* p) {
  return *reinterpret_cast<const __attribute__((address_space(4))) float*>(
      reinterpret_cast<uintptr_t>(p));
}

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

// Sixteen codes times their scale as bf16 (exact for a scale that is a power of two).
__device__ __forceinline__ void fb_widen(u32x4 c, float s, u32x4 (&out)[2]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const u32x2 v = fb_bf16_of4(c[j]);
    out[j / 2][j % 2 * 2] = fb_pack_bf16(bf16_lo_to_f32(v.x) * s, bf16_hi_to_f32(v.x) * s);
    out[j / 2][j % 2 * 2 + 1] = fb_pack_bf16(bf16_lo_to_f32(v.y) * s, bf16_hi_to_f32(v.y) * s);
  }
}

// The sum over one block of 128 inputs of the products of two rows' codes, for a 16 x 16 tile:
// lane (r = l % 16, q = l / 16) holds bytes 16 q .. 16 q + 15 and 64 + 16 q .. 64 + 16 q + 15
// of row r of A and of row r of B; result element i is D[4 q + i][r].
//
// EXACT: the codes become bf16 (exactly) and four v_mfma_f32_16x16x32_bf16 add the exact
// products in fp32 (1e-8 of a block's sum in the 2-norm on block-scaled normal data). Else one
// v_mfma_f32_16x16x128_f8f6f4, at twice the rate, for results that are rounded to bf16. It adds
// the products of 8 consecutive inputs at a time, each cut towards zero at 2^-13 of 2^(e + f), e
// and f the exponents of the two codes with the largest e + f among the eight (a code below the
// smallest normal, 2^-6, has that one's; products with a zero do not count), and the sums of
// eight in fp32. At most seven of the eight are cut, so a block's sum is off by less than 2^-10 of
// the sum of its products' magnitudes (codes below 2^-6 taken as that); on the same data it is
// 1.5e-5 to 5e-5 in the 2-norm. Beside bf16's half step of 2^-8 of the result that counts only
// where a sum's large terms cancel, and there a caller has the fp32 result.
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

constexpr int FB_CUS = 256;  // compute units

// The work items of a grid over tt x tc tiles. It is read as 8 interleaved streams, one per XCD
// (workgroup b belongs to stream b % 8 and starts with the stream's item b / 8), each a contiguous
// range of tiles in an order that walks 4 channel tiles per token tile, so that the tiles an XCD
// works on at one time share rows of both operands in its L2. Where the last round of a stream
// has tiles for half of its 32 compute units at most, each of them is two items, halves along
// the first side, so that the round lasts little over half as long.
struct FbItems {
  int tt, tc, per, full, items;  // tiles of a stream, items that are whole tiles, all items
  __host__ __device__ FbItems(int tt_, int tc_) : tt(tt_), tc(tc_), per((tt_ * tc_ + 7) >> 3) {
    const int rest = per % (FB_CUS / 8);
    full = rest <= FB_CUS / 16 ? per - rest : per;
    items = full + 2 * (per - full);
  }
  // Item j of stream x: its tile and which half of it (-1: all); false past the last.
  __device__ bool at(int x, int j, int* t, int* c, int* half) const {
    if (j >= items) return false;
    const int u = x * per + (j < full ? j : full + (j - full) / 2);
    if (u >= tt * tc) return false;
    *half = j < full ? -1 : (j - full) & 1;
    const int band = u / (4 * tt), first = 4 * band, width = min(4, tc - first);
    const int v = u - first * tt;
    *c = first + v % width;
    *t = v / width;
    return true;
  }
};

// ---- epilogues ------------------------------------------------------------------------------
// What a forward kernel does with the sums of four consecutive channels o .. o + 3 of one
// token (gated forms: g and u are the sums of gate and up channels o .. o + 3).
//
// 1 / (1 + e^-g) by the hardware's 2^x and reciprocal (an ulp each) of -g log2 e, whose rounding
// makes a relative error of at most |g| 2^-24: for every g whose sigmoid is a normal fp32 number
// below 2^-17, far under half a step of the bf16 result (2^-8). The full-precision exponential
// and division took a fifth of the gated tile kernel's time at 1,280 inputs.
__device__ __forceinline__ float fb_sigmoid(float g) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.44269504f));
}

// silu(g) * u of four channels, in bf16.
__device__ __forceinline__ u32x2 fb_gate4(f32x4 g, f32x4 u) {
  float h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = g[i] * fb_sigmoid(g[i]) * u[i];
  return (u32x2){fb_pack_bf16(h[0], h[1]), fb_pack_bf16(h[2], h[3])};
}
// The gradients of four gate sums (*dg) and up sums (*du) from dh (bf16), in bf16, the operand
// type of the two products that read them: d silu(g) / dg = s + g s (1 - s), s = sigmoid(g).
__device__ __forceinline__ void fb_gate_grad4(f32x4 g, f32x4 u, u32x2 d, u32x2* dg, u32x2* du) {
  const float dh[4] = {bf16_lo_to_f32(d.x), bf16_hi_to_f32(d.x), bf16_lo_to_f32(d.y),
                       bf16_hi_to_f32(d.y)};
  float a[4], b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float s = fb_sigmoid(g[i]);
    a[i] = dh[i] * u[i] * s * (1.0f + g[i] * (1.0f - s));
    b[i] = dh[i] * g[i] * s;
  }
  *dg = (u32x2){fb_pack_bf16(a[0], a[1]), fb_pack_bf16(a[2], a[3])};
  *du = (u32x2){fb_pack_bf16(b[0], b[1]), fb_pack_bf16(b[2], b[3])};
}

// Straight from registers to memory (the strip kernel).
template <int EPI>
__device__ __forceinline__ void fb_store(const Fp8b128GemmArgs& a, int64_t t, int o, f32x4 g,
                                         f32x4 u) {
  uint16_t* y = static_cast<uint16_t*>(a.y);
  if constexpr (EPI == FB_F32) {
    *reinterpret_cast<f32x4*>(static_cast<float*>(a.y) + t * a.out + o) = g;
  } else if constexpr (EPI == FB_BF16) {
    *reinterpret_cast<u32x2*>(y + t * a.out + o) =
        (u32x2){fb_pack_bf16(g[0], g[1]), fb_pack_bf16(g[2], g[3])};
  } else if constexpr (EPI == FB_GATED) {
    *reinterpret_cast<u32x2*>(y + t * (a.out / 2) + o) = fb_gate4(g, u);
  } else {
    u32x2 dg, du;
    fb_gate_grad4(g, u, *reinterpret_cast<const u32x2*>(a.dh + t * (a.out / 2) + o), &dg, &du);
    *reinterpret_cast<u32x2*>(y + t * a.out + o) = dg;
    *reinterpret_cast<u32x2*>(y + t * a.out + a.out / 2 + o) = du;
  }
}

// The lane, as a value that the compiler does not know to be the same in every tile: what a kernel
// that walks tiles derives from it between two tiles would otherwise be computed once and held
// in registers through the products.
__device__ __forceinline__ int fb_fresh_lane() {
  int lane = threadIdx.x & 63;
  asm volatile("" : "+v"(lane));
  return lane;
}

// N of a wave's rows of ROW bytes (64, 128 or 256) on their way to memory: written to LDS by pieces of a
// row, 16-byte chunk c of row k at position c ^ (k % chunks) so that the rows of one piece meet
// different banks, and stored by whole rows, 16 bytes a lane.
template <int ROW, int N>
struct FbRows {
  static constexpr int CHUNKS = ROW / 16;
  uint8_t* lds;  // N * ROW bytes of this wave's own
  template <class V>
  __device__ __forceinline__ void put(int k, int byte, V v) {
    *reinterpret_cast<V*>(lds + k * ROW + 16 * ((byte >> 4) ^ (k & (CHUNKS - 1))) + (byte & 15)) = v;
  }
  // rows 0 .. rows - 1 to dst + row * stride, their first `bytes` bytes
  __device__ __forceinline__ void store(uint8_t* dst, int64_t stride, int rows, int bytes, int lane) {
#pragma unroll
    for (int j = 0; j < N * CHUNKS / 64; ++j) {
      const int k = j * (64 / CHUNKS) + lane / CHUNKS;
      const int c = (lane & (CHUNKS - 1)) ^ (k & (CHUNKS - 1));
      const u32x4 v = *reinterpret_cast<const u32x4*>(lds + k * ROW + 16 * (lane & (CHUNKS - 1)));
      if (k < rows && 16 * c < bytes) *reinterpret_cast<u32x4*>(dst + k * stride + 16 * c) = v;
    }
  }
};

constexpr bool fb_gated(int epi) { return epi == FB_GATED || epi == FB_GATED_GRAD; }

}  // namespace tq

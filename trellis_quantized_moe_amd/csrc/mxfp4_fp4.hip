// The routed product of MXFP4 activations with MXFP4 experts on gfx950's fp4 matrix cores
// (FORMAT F30): both operands are their E2M1 codes with their E8M0 scales as stored, nothing is
// decoded.
//
// A work item is up to 128 routed rows of one expert times one group of 128 output channels, on
// four waves, wave w owning channels 32 w .. 32 w + 31 for all rows. A step is 128 inputs:
// lane (n, q) supplies the 32 codes of block q of the step of its row or channel (16 bytes) and
// that block's scale byte to v_mfma_scale_f32_16x16x128_f8f6f4.
#include "gemm_core.h"
#include "mx_unit.h"

namespace tq {

namespace {

typedef int32_t i32x8 __attribute__((ext_vector_type(8)));

constexpr int F4_THREADS = 256;

__device__ __forceinline__ i32x8 fp4_operand(u32x4 c) {
  return (i32x8){(int)c.x, (int)c.y, (int)c.z, (int)c.w, 0, 0, 0, 0};
}

__global__ __launch_bounds__(F4_THREADS) void fp4_gemm_kernel(Fp4GemmArgs a) {
  using U = MxUnit<MX_FP4>;
  int item, grp;
  if (!gemm_unit(a.n_items, a.groups, &item, &grp)) return;
  const int4 itd = reinterpret_cast<const int4*>(a.items)[item];
  const int e = itd.x, nrows = itd.z;
  const int lane = threadIdx.x & 63, q = lane >> 4, n = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ns = min(8, a.out / 16 - grp * 8);
  if (2 * w >= ns) return;
  const uint8_t* unit = a.units + (size_t)e * U::unit_bytes(a.out, a.in);
  // rows past the item load from beyond the buffers' ends and read zeros
  const GemmRsrc ra = gemm_rsrc(a.xa, a.xa_bytes), rs = gemm_rsrc(a.xs, a.xs_bytes);
  const GemmRsrc rb = gemm_rsrc(unit, (uint32_t)U::unit_bytes(a.out, a.in));
  uint32_t avo[8], svo[8];
#pragma unroll
  for (int mb = 0; mb < 8; ++mb) {
    const int r = 16 * mb + n;
    const uint32_t row = r < nrows ? (uint32_t)(a.pairs[itd.y + r] / a.topk) : 0u;
    avo[mb] = r < nrows ? row * (uint32_t)(a.in / 2) + 16u * q : 0x80000000u;
    svo[mb] = r < nrows ? row * (uint32_t)(a.in / 32) + q : 0x80000000u;
  }
  uint32_t bvo[2], bso[2];
#pragma unroll
  for (int nb = 0; nb < 2; ++nb) {
    const int oc = 32 * w + 16 * nb + n;
    const int o = grp * 128 + (oc < 16 * ns ? oc : 16 * ns - 1);
    bvo[nb] = a.layout ? U::packed_at(a.out, a.in, o, q) : U::stored_at(a.in, o, q);
    bso[nb] = U::scale_at(a.out, a.in, o, q);
  }
  const uint32_t bstep = a.layout ? U::packed_at(a.out, a.in, grp * 128, 4) -
                                        U::packed_at(a.out, a.in, grp * 128, 0)
                                  : 64u;
  f32x4 acc[8][2];
#pragma unroll
  for (int mb = 0; mb < 8; ++mb)
#pragma unroll
    for (int nb = 0; nb < 2; ++nb) acc[mb][nb] = (f32x4){0.f, 0.f, 0.f, 0.f};
  const int mblocks = (nrows + 15) / 16;
  for (int k = 0; k < a.in / 128; ++k) {
    i32x8 bv[2];
    int sb[2];
#pragma unroll
    for (int nb = 0; nb < 2; ++nb) {
      bv[nb] = fp4_operand(__builtin_amdgcn_raw_buffer_load_b128(rb, bvo[nb], k * bstep, 0));
      sb[nb] = __builtin_amdgcn_raw_buffer_load_b8(rb, bso[nb], 4 * k, 0);
    }
#pragma unroll
    for (int mb = 0; mb < 8; ++mb) {
      if (mb < mblocks) {
        const i32x8 av = fp4_operand(__builtin_amdgcn_raw_buffer_load_b128(ra, avo[mb], 64 * k, 0));
        const int sa = __builtin_amdgcn_raw_buffer_load_b8(rs, svo[mb], 4 * k, 0);
#pragma unroll
        for (int nb = 0; nb < 2; ++nb)
          acc[mb][nb] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              av, bv[nb], acc[mb][nb], 4, 4, 0, sa, 0, sb[nb]);
      }
    }
  }
#pragma unroll
  for (int mb = 0; mb < 8; ++mb) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 16 * mb + 4 * q + i;
      if (r < nrows) {
        const int slot = a.pairs[itd.y + r];
        const float gate = a.gates ? a.gates[slot] : 1.0f;
#pragma unroll
        for (int nb = 0; nb < 2; ++nb) {
          const int oc = 32 * w + 16 * nb + n;
          if (oc < 16 * ns) a.y[(size_t)slot * a.out + grp * 128 + oc] = acc[mb][nb][i] * gate;
        }
      }
    }
  }
}

}  // namespace

hipError_t launch_fp4_gemm(const Fp4GemmArgs& a, hipStream_t s) {
  const int blocks = gemm_grid(a.max_items, a.groups);
  if (blocks == 0) return hipSuccess;
  return launch_timed(fp4_gemm_kernel, dim3(blocks), dim3(F4_THREADS), s, a);
}

}  // namespace tq

// The products over the fp8b128 store (FORMAT F24, F25):
//   y[t][o] = sum over blocks b of 128 inputs of xs[t][b] * ws[o / 128][b] * P_b[t][o],
//   P_b[t][o] = sum over the block's inputs of x code * w code,
// P_b by the matrix cores from zero, then one fp32 multiply-add per block into the sum, since
// a scale belongs to a block. Weights are the A operand and activations the B operand, so a
// lane ends with four consecutive channels of one token.
#include "fp8b128.h"

namespace tq {

namespace {

// ---- few tokens: one strip of 16 channels per workgroup, the inputs split over its waves ----
//
// A workgroup owns 16 channels (gated: 16 gate and 16 up channels) of up to 16 * TT tokens.
// Its eight waves take the blocks of 128 inputs in turn, each straight from memory to
// registers, D blocks ahead, and their sums are added through LDS in wave order (so the result
// does not depend on timing). One launch, no workspace.
constexpr int FS_WAVES = 8;
constexpr int FS_THREADS = 64 * FS_WAVES;

template <int EPI, int TT>
__global__ __launch_bounds__(FS_THREADS) void fp8b128_strip_kernel(Fp8b128GemmArgs a) {
  constexpr int NS = fb_gated(EPI) ? 2 : 1;
  constexpr bool EXACT = EPI == FB_F32;
  constexpr int D = TT == 1 ? 4 : 2;
  __shared__ f32x4 red[FS_WAVES][TT * NS][64];
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int strips = a.out / 16 / NS;
  const int strip = blockIdx.x % strips;
  const int64_t t0 = (int64_t)(blockIdx.x / strips) * (16 * TT);
  const int rows = (int)min((int64_t)(16 * TT), a.T - t0);

  const GemmRsrc rw = gemm_rsrc(a.w, (uint32_t)a.out * (uint32_t)a.in);
  const GemmRsrc rws = gemm_rsrc(a.ws, (uint32_t)(((a.out + 127) / 128) * a.nb) * 4u);
  const GemmRsrc rx = gemm_rsrc(a.x + t0 * a.in, (uint32_t)rows * (uint32_t)a.in);
  const GemmRsrc rxs = gemm_rsrc(a.xs + t0 * a.nb, (uint32_t)(rows * a.nb) * 4u);
  uint32_t wo[NS], wso[NS], xo[TT], xso[TT];
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    const int o = 16 * strip + s * (a.out / 2);
    wo[s] = (uint32_t)(o + r) * (uint32_t)a.in + 16u * q;
    wso[s] = (uint32_t)(o / 128) * (uint32_t)a.nb * 4u;
  }
#pragma unroll
  for (int t = 0; t < TT; ++t) {
    const int row = 16 * t + r;
    xo[t] = row < rows ? (uint32_t)row * (uint32_t)a.in + 16u * q : FB_OOB;
    xso[t] = row < rows ? (uint32_t)(row * a.nb) * 4u : FB_OOB;
  }

  u32x4 wf[D][NS][2], xf[D][TT][2];
  float ss[D][NS], sx[D][TT];
  auto load = [&](int d, int kb) {
    // chunks past the row's end (and blocks past the last) are read as zeros on both sides
    const bool c0 = kb * 128 + 16 * q < a.in, c1 = kb * 128 + 64 + 16 * q < a.in;
    const bool in = kb < a.nb;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      wf[d][s][0] = __builtin_amdgcn_raw_buffer_load_b128(rw, c0 ? wo[s] + 128u * kb : FB_OOB, 0, 0);
      wf[d][s][1] = __builtin_amdgcn_raw_buffer_load_b128(rw, c1 ? wo[s] + 128u * kb + 64u : FB_OOB, 0, 0);
      ss[d][s] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rws, in ? wso[s] + 4u * kb : FB_OOB, 0, 0));
    }
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const bool row = xo[t] != FB_OOB;
      xf[d][t][0] = __builtin_amdgcn_raw_buffer_load_b128(rx, row && c0 ? xo[t] + 128u * kb : FB_OOB, 0, 0);
      xf[d][t][1] = __builtin_amdgcn_raw_buffer_load_b128(rx, row && c1 ? xo[t] + 128u * kb + 64u : FB_OOB, 0, 0);
      sx[d][t] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rxs, row && in ? xso[t] + 4u * kb : FB_OOB, 0, 0));
    }
  };

  f32x4 acc[TT][NS];
#pragma unroll
  for (int t = 0; t < TT; ++t)
#pragma unroll
    for (int s = 0; s < NS; ++s) acc[t][s] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int d = 0; d < D; ++d) load(d, w + FS_WAVES * d);
  for (int kb = w; kb < a.nb; kb += FS_WAVES * D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (kb + FS_WAVES * d < a.nb) {
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
          for (int s = 0; s < NS; ++s) {
            const f32x4 p = fb_block_product<EXACT>(wf[d][s][0], wf[d][s][1], xf[d][t][0], xf[d][t][1]);
            const float m = sx[d][t] * ss[d][s];
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[t][s][i] = __builtin_fmaf(p[i], m, acc[t][s][i]);
          }
      }
      load(d, kb + FS_WAVES * (D + d));
    }
  }
#pragma unroll
  for (int t = 0; t < TT; ++t)
#pragma unroll
    for (int s = 0; s < NS; ++s) red[w][t * NS + s][lane] = acc[t][s];
  __syncthreads();
  const int t = threadIdx.x >> 6;  // wave t finishes token tile t
  if (t < TT && 16 * t + r < rows) {
    f32x4 sum[NS];
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      sum[s] = red[0][t * NS + s][lane];
#pragma unroll
      for (int v = 1; v < FS_WAVES; ++v) sum[s] += red[v][t * NS + s][lane];
    }
    fb_store<EPI>(a, t0 + 16 * t + r, 16 * strip + 4 * q, sum[0], sum[NS - 1]);
  }
}

template <int EPI>
hipError_t launch_strips(const Fp8b128GemmArgs& a, hipStream_t s) {
  const int64_t strips = a.out / (fb_gated(EPI) ? 32 : 16);
  const int tt = a.T <= 16 ? 1 : a.T <= 32 ? 2 : 4;
  const unsigned grid = (unsigned)(strips * ((a.T + 16 * tt - 1) / (16 * tt)));
  if (tt == 1)
    return launch_timed(fp8b128_strip_kernel<EPI, 1>, dim3(grid), dim3(FS_THREADS), s, a);
  if (tt == 2)
    return launch_timed(fp8b128_strip_kernel<EPI, 2>, dim3(grid), dim3(FS_THREADS), s, a);
  return launch_timed(fp8b128_strip_kernel<EPI, 4>, dim3(grid), dim3(FS_THREADS), s, a);
}

}  // namespace

hipError_t launch_fp8b128_gemm(const Fp8b128GemmArgs& a, int epi, hipStream_t s) {
  switch (epi) {
    case FB_F32: return launch_strips<FB_F32>(a, s);
    case FB_BF16: return launch_strips<FB_BF16>(a, s);
    case FB_GATED: return launch_strips<FB_GATED>(a, s);
    default: return launch_strips<FB_GATED_GRAD>(a, s);
  }
}

}  // namespace tq

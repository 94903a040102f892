// The products over the fp8b128 store (FORMAT F24, F25):
//   y[t][o] = sum over blocks b of 128 inputs of xs[t][b] * ws[o / 128][b] * P_b[t][o],
//   P_b[t][o] = sum over the block's inputs of x code * w code,
// P_b by the matrix cores from zero, then one fp32 multiply-add per block into the sum, since
// a scale belongs to a block. Weights are the A operand and activations the B operand, so a
// lane ends with four consecutive channels of one token.
#include "fp8b128.h"

#include <algorithm>
#include <cstdint>
#include <type_traits>

namespace tq {

namespace {

// ---- one or two tokens, few channels: a channel per wave --------------------------------------
//
// A wave owns one channel (gated: its gate and up rows) and reads the rows 1,024 inputs at a time,
// 16 bytes a lane, D such steps ahead; the products are fp32 multiply-adds of the decoded codes
// (exact products), a lane's 16 are scaled once, and the lanes are added at the end. Bound by
// latency: the waves of all channels read their few kilobytes at once (one token x 5,120 x 1,536
// in 4.6 us, 1.7 TB/s).
constexpr int FR_WAVES = 4;

// Adds v over the 64 lanes (every lane gets the sum; the order is fixed).
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
  return v;
}

__device__ __forceinline__ void fb_f32_of16(u32x4 c, float (&f)[16]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[j], false);
    const f32x2 hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[j], true);
    f[4 * j] = lo.x;
    f[4 * j + 1] = lo.y;
    f[4 * j + 2] = hi.x;
    f[4 * j + 3] = hi.y;
  }
}

template <int EPI, int NT>
__global__ __launch_bounds__(64 * FR_WAVES) void fp8b128_row_kernel(Fp8b128GemmArgs a) {
  constexpr int NS = fb_gated(EPI) ? 2 : 1, D = 4;
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int o = blockIdx.x * FR_WAVES + w, T = (int)a.T;
  const int width = a.out / NS;
  if (o >= width) return;
  const GemmRsrc rx = gemm_rsrc(a.x, (uint32_t)T * (uint32_t)a.in);
  const GemmRsrc rxs = gemm_rsrc(a.xs, (uint32_t)(T * a.nb) * 4u);
  GemmRsrc rw[NS], rws[NS];
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    rw[s] = gemm_rsrc(a.w + (int64_t)(o + s * width) * a.in, (uint32_t)a.in);
    rws[s] = gemm_rsrc(a.ws + (int64_t)((o + s * width) / 128) * a.nb, (uint32_t)a.nb * 4u);
  }
  u32x4 wf[D][NS], xf[D][NT];
  float ss[D][NS], sx[D][NT];
  auto load = [&](int d, int k) {  // past the rows' end: zeros
    const uint32_t at = 1024u * k + 16u * lane;
    const bool in = at < (uint32_t)a.in;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      wf[d][s] = __builtin_amdgcn_raw_buffer_load_b128(rw[s], in ? at : FB_OOB, 0, 0);
      ss[d][s] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rws[s], in ? at / 128 * 4 : FB_OOB, 0, 0));
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {  // tokens past the last: outside the resource
      xf[d][t] = __builtin_amdgcn_raw_buffer_load_b128(rx, in ? t * (uint32_t)a.in + at : FB_OOB, 0, 0);
      sx[d][t] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
          rxs, in ? (uint32_t)(t * a.nb + at / 128) * 4u : FB_OOB, 0, 0));
    }
  };
  float acc[NT][NS];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int s = 0; s < NS; ++s) acc[t][s] = 0.0f;
  const int steps = (a.in + 1023) / 1024;
#pragma unroll
  for (int d = 0; d < D; ++d) load(d, d);
  for (int k = 0; k < steps; k += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (k + d < steps) {
        float wv[NS][16];
#pragma unroll
        for (int s = 0; s < NS; ++s) fb_f32_of16(wf[d][s], wv[s]);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          float xv[16];
          fb_f32_of16(xf[d][t], xv);
#pragma unroll
          for (int s = 0; s < NS; ++s) {
            float p = xv[0] * wv[s][0];
#pragma unroll
            for (int i = 1; i < 16; ++i) p = __builtin_fmaf(xv[i], wv[s][i], p);
            acc[t][s] = __builtin_fmaf(p, sx[d][t] * ss[d][s], acc[t][s]);
          }
        }
      }
      load(d, k + D + d);
    }
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    if (t >= T) break;
    const float g = wave_sum(acc[t][0]), u = wave_sum(acc[t][NS - 1]);
    if (lane != 0) continue;
    uint16_t* y = static_cast<uint16_t*>(a.y);
    if constexpr (EPI == FB_F32) {
      static_cast<float*>(a.y)[(int64_t)t * a.out + o] = g;
    } else if constexpr (EPI == FB_BF16) {
      y[(int64_t)t * a.out + o] = (uint16_t)fb_pack_bf16(g, 0.0f);
    } else if constexpr (EPI == FB_GATED) {
      y[(int64_t)t * width + o] = (uint16_t)fb_gate4((f32x4){g, 0.f, 0.f, 0.f}, (f32x4){u, 0.f, 0.f, 0.f}).x;
    } else {
      u32x2 dg, du;
      fb_gate_grad4((f32x4){g, 0.f, 0.f, 0.f}, (f32x4){u, 0.f, 0.f, 0.f},
                    (u32x2){a.dh[(int64_t)t * width + o], 0u}, &dg, &du);
      y[(int64_t)t * a.out + o] = (uint16_t)dg.x;
      y[(int64_t)t * a.out + width + o] = (uint16_t)du.x;
    }
  }
}

template <int EPI>
hipError_t launch_rows(const Fp8b128GemmArgs& a, hipStream_t s) {
  const unsigned width = a.out / (fb_gated(EPI) ? 2 : 1);
  const dim3 grid((width + FR_WAVES - 1) / FR_WAVES), block(64 * FR_WAVES);
  if (a.T == 1) return launch_timed(fp8b128_row_kernel<EPI, 1>, grid, block, s, a);
  return launch_timed(fp8b128_row_kernel<EPI, 2>, grid, block, s, a);
}

// ---- few tokens: strips of 16 channels, the inputs split over a workgroup's waves ------------
//
// A workgroup owns NS strips of 16 channels (gated: half of them gate strips, half the up strips
// of the same channels) of up to 16 * TT tokens. Its W waves take the blocks of 128 inputs in
// turn, each through LDS of its own (no barrier until the end): a block goes from there to
// registers at once, and the next one's loads are issued between its products. The waves' sums are
// added in wave order, so the result does not depend on timing. One LDS stage and eight waves, two
// on a SIMD, are better than four waves with two or three stages: 213 tokens x 5,120 x 1,536 10.6
// and 11.5 us (fp32 results 11.7 and 14.2). One launch, no workspace. The rows come through LDS
// because a load in operand order has consecutive lanes in different rows, which the memory unit
// takes one by one: strips of 16 channels and tokens loaded that way took 9.9 us at 32 x 5,120 x
// 1,536, against 5.6.
template <int NS, int TT>
struct FbStrip {
  static constexpr int ROWS = 16 * (NS + TT);
  static constexpr int W = 8;
  static constexpr int LOADS = ROWS / 8 + 1;  // per block
  union {
    struct {
      alignas(16) uint8_t rows[ROWS * 128];  // strips, then tokens
      alignas(16) float sx[64];
    } stage[W];
    f32x4 red[W][TT * NS][64];
  };
};

template <int EPI, int NS, int TT, bool EXACT>
__device__ void fb_strip(const Fp8b128GemmArgs& a, FbStrip<NS, TT>& sh) {
  using S = FbStrip<NS, TT>;
  constexpr bool GATED = fb_gated(EPI);
  constexpr int NO = GATED ? NS / 2 : NS;  // strips of results
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int width = GATED ? a.out / 2 : a.out;
  // an XCD (workgroup b belongs to b % 8) has all tokens of consecutive strips, which read the same
  // codes
  const int tiles = (int)((a.T + 16 * TT - 1) / (16 * TT)), all = gridDim.x, x = blockIdx.x & 7;
  const int g = x * (all >> 3) + min(x, all & 7) + (blockIdx.x >> 3);
  const int c0 = g / tiles * (16 * NO);
  const int64_t t0 = (int64_t)(g % tiles) * (16 * TT);
  const int rows = (int)min((int64_t)(16 * TT), a.T - t0);

  const GemmRsrc rw = gemm_rsrc(a.w, (uint32_t)a.out * (uint32_t)a.in);
  const GemmRsrc rx = gemm_rsrc(a.x + t0 * a.in, (uint32_t)rows * (uint32_t)a.in);
  const GemmRsrc rxs = gemm_rsrc(a.xs + t0 * a.nb, (uint32_t)(rows * a.nb) * 4u);
  // an instruction fills 8 rows: lane l writes position l % 8 of row l / 8, chunk
  // (l % 8) ^ (row % 8), as in the tiles
  const int chunk = 16 * ((lane & 7) ^ (lane >> 3));
  uint32_t ro[2 * (NS + TT)];
  const float* ws[NS];
#pragma unroll
  for (int j = 0; j < 2 * (NS + TT); ++j) {
    const int k = 8 * j + (lane >> 3), t = k - 16 * NS;
    if (j < 2 * NS) {
      const int c = c0 + k % (16 * NO);
      ro[j] = c < width ? (uint32_t)(c + k / (16 * NO) * width) * (uint32_t)a.in + chunk : FB_OOB;
    } else {
      ro[j] = t < rows ? (uint32_t)t * (uint32_t)a.in + chunk : FB_OOB;
    }
  }
#pragma unroll
  for (int s = 0; s < NS; ++s)  // a strip past the last channel takes the last one's scale
    ws[s] = a.ws + (int64_t)((min(c0 + 16 * (s % NO), width - 16) + s / NO * width) / 128) * a.nb;
  const uint32_t xso = lane < rows ? (uint32_t)(lane * a.nb) * 4u : FB_OOB;

  // Loads first .. last - 1 of a block's S::LOADS; chunks past the row's end are zeros.
  auto load = [&](int first, int last, int kb) {
    auto& st = sh.stage[w];
    const bool in = 128 * kb + chunk < a.in;
#pragma unroll
    for (int j = first; j < last; ++j)
      if (j < S::LOADS - 1)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(j < 2 * NS ? rw : rx, (LdsPtr)(&st.rows[1024 * j]), 16,
                                                 in ? ro[j] : FB_OOB, 128u * kb, 0, 0);
      else
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rxs, (LdsPtr)(&st.sx[0]), 4, xso, 4u * kb, 0, 0);
  };

  f32x4 acc[TT][NS];
#pragma unroll
  for (int t = 0; t < TT; ++t)
#pragma unroll
    for (int s = 0; s < NS; ++s) acc[t][s] = (f32x4){0.f, 0.f, 0.f, 0.f};
  const int at0 = 128 * r + 16 * (q ^ (r & 7)), at1 = 128 * r + 16 * ((4 + q) ^ (r & 7));
  if (w < a.nb) load(0, S::LOADS, w);
  // A block: into registers, then its products, with the next block's loads between them.
  for (int kb = w; kb < a.nb; kb += S::W) {
    float ss[NS];
#pragma unroll
    for (int s = 0; s < NS; ++s) ss[s] = fb_uniform_load(ws[s] + kb);
    wait_vmcnt<0>();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    const auto& st = sh.stage[w];
    u32x4 codes[NS + TT][2];
    float sx[TT];
#pragma unroll
    for (int s = 0; s < NS + TT; ++s) {
      codes[s][0] = *reinterpret_cast<const u32x4*>(st.rows + 2048 * s + at0);
      codes[s][1] = *reinterpret_cast<const u32x4*>(st.rows + 2048 * s + at1);
    }
#pragma unroll
    for (int t = 0; t < TT; ++t) sx[t] = st.sx[16 * t + r];
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): no read of the stage is outstanding
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    FbOperand<EXACT> wv[NS];
#pragma unroll
    for (int s = 0; s < NS; ++s) wv[s].set(codes[s][0], codes[s][1]);
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      FbOperand<EXACT> xv;
      xv.set(codes[NS + t][0], codes[NS + t][1]);
      if (kb + S::W < a.nb) {
        __builtin_amdgcn_sched_barrier(0);
        load(t * S::LOADS / TT, (t + 1) * S::LOADS / TT, kb + S::W);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const f32x4 p = fb_block_product(wv[s], xv);
        const float m = sx[t] * ss[s];
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[t][s][i] = __builtin_fmaf(p[i], m, acc[t][s][i]);
      }
    }
  }
  __syncthreads();  // no load of this workgroup is writing its LDS, and no wave reads a stage
#pragma unroll
  for (int t = 0; t < TT; ++t)
#pragma unroll
    for (int s = 0; s < NS; ++s) sh.red[w][t * NS + s][lane] = acc[t][s];
  __syncthreads();
  for (int v = w; v < TT * NO; v += S::W) {  // the tiles of results, one after the other
    const int t = v / NO, s = v % NO;
    f32x4 g = sh.red[0][t * NS + s][lane], u = sh.red[0][t * NS + s + NS - NO][lane];
#pragma unroll
    for (int k = 1; k < S::W; ++k) {
      g += sh.red[k][t * NS + s][lane];
      u += sh.red[k][t * NS + s + NS - NO][lane];
    }
    const int o = c0 + 16 * s + 4 * q;
    if (16 * t + r < rows && o < width) fb_store<EPI>(a, t0 + 16 * t + r, o, g, u);
  }
}

template <int EPI, int NS, int TT, bool EXACT>
__global__ __launch_bounds__((64 * FbStrip<NS, TT>::W)) void fp8b128_strip_kernel(Fp8b128GemmArgs a) {
  __shared__ FbStrip<NS, TT> sh;
  fb_strip<EPI, NS, TT, EXACT>(a, sh);
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <int EPI, int NS, int TT>
int64_t strip_groups(const Fp8b128GemmArgs& a) {  // workgroups
  constexpr int NO = fb_gated(EPI) ? NS / 2 : NS;
  return ceil_div(fb_gated(EPI) ? a.out / 2 : a.out, 16 * NO) * ceil_div(a.T, 16 * TT);
}
template <int EPI, int NS, int TT, bool EXACT = EPI == FB_F32>
hipError_t launch_strip(const Fp8b128GemmArgs& a, hipStream_t s) {
  return launch_timed(fp8b128_strip_kernel<EPI, NS, TT, EXACT>, dim3((unsigned)strip_groups<EPI, NS, TT>(a)),
                      dim3(64 * FbStrip<NS, TT>::W), s, a);
}

// ---- many tokens: tiles of both operands in LDS ----------------------------------------------
//
// A workgroup of 2 x WT waves owns 64 * WT tokens and 32 * SW weight rows (gated: the gate rows
// of 16 * SW channels, then their up rows), wave (wc, wt) SW strips of 16 channels (gated: half
// of them gate strips, half the up strips of the same channels, so that both sums of a channel
// end in one lane) and 4 tiles of 16 tokens. Per block of 128 inputs the rows' 128 bytes go
// straight to LDS (16-byte chunk c of row r at position c ^ (r % 8), so that eight lanes reading
// one chunk of eight rows meet eight different banks' worth of LDS), in two or three stages with
// one barrier per block. 8,192 tokens x 5,120 x 7,168 take 266 to 300 us as the clocks go (2.0 to
// 2.26 PFLOP/s), the matrix cores busy 57 % of the cycles at 1.74 to 1.8 GHz: without its loads the
// kernel keeps them busy 65 % at 1.62 GHz, so it is near what power allows; without three quarters
// of its multiply-adds it takes as long. fp32 results take 527 to 552 us.
template <int SW, int WT, int ST>
struct FbTile {
  static constexpr int WAVES = 2 * WT, THREADS = 64 * WAVES, BC = 32 * SW, BT = 64 * WT;
  alignas(16) uint8_t w[ST][BC * 128];
  alignas(16) uint8_t x[ST][BT * 128];
  alignas(16) float sx[ST][BT];
};

// One workgroup per compute unit takes tile after tile: the first block of the next tile is
// loading while a tile's results are stored.
//
// SAME: the wave's strips (gated: its gate strips, and its up strips) lie in one block of 128
// channels, so that a block of inputs has one scale for them.
template <int EPI, int SW, int WT, int ST, bool SAME>
__device__ void fb_tiles(const Fp8b128GemmArgs& a, FbTile<SW, WT, ST>& sh,
                         const FbItems& items) {
  using S = FbTile<SW, WT, ST>;
  constexpr bool GATED = fb_gated(EPI), EXACT = EPI == FB_F32;
  constexpr int NX = S::BT / S::WAVES / 8, NW = S::BC / S::WAVES / 8;
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wc = w & 1, wt = w >> 1;
  const int half = a.out / 2, width = GATED ? half : a.out;
  const GemmRsrc rw = gemm_rsrc(a.w, (uint32_t)a.out * (uint32_t)a.in);
  // an instruction fills 8 rows: lane l writes position l % 8 of row l / 8
  const int chunk = 16 * ((lane & 7) ^ (lane >> 3));
  // the wave's strip s is tile rows strip_row(s) ..
  auto strip_row = [&](int s) {
    if (!GATED) return 16 * (SW * wc + s);
    return (s < SW / 2 ? 0 : S::BC / 2) + 16 * (SW / 2 * wc + s % (SW / 2));
  };

  // the tile: its first token, tokens, first channel (gated: of either half), load offsets
  int64_t t0;
  int rows, c0;
  uint32_t wo[NW], xo[NX], xso;
  // the scales of the wave's strips: one for each, or (SAME) for each half, block by block
  constexpr int NG = !SAME ? SW : GATED ? 2 : 1, PER_GROUP = SW / NG;
  const float* ws[NG];
  auto set_tile = [&](int tile_t, int tile_c, int half_item) {  // the tile, or a half of its tokens
    const int lane = fb_fresh_lane(), chunk = 16 * ((lane & 7) ^ (lane >> 3));
    t0 = (int64_t)tile_t * S::BT + (half_item > 0 ? S::BT / 2 : 0);
    rows = (int)max(min((int64_t)(half_item < 0 ? S::BT : S::BT / 2), a.T - t0), (int64_t)0);
    c0 = tile_c * (GATED ? S::BC / 2 : S::BC);
    // weight row k of the tile: channel and validity
    auto channel = [&](int k) {
      if (!GATED) return c0 + k;
      return k < S::BC / 2 ? c0 + k : half + c0 + k - S::BC / 2;
    };
    auto valid = [&](int k) { return c0 + (GATED && k >= S::BC / 2 ? k - S::BC / 2 : k) < width; };
#pragma unroll
    for (int j = 0; j < NW; ++j) {
      const int k = 8 * (NW * w + j) + (lane >> 3);
      wo[j] = valid(k) ? (uint32_t)channel(k) * (uint32_t)a.in + chunk : FB_OOB;
    }
#pragma unroll
    for (int j = 0; j < NX; ++j) {
      const int k = 8 * (NX * w + j) + (lane >> 3);
      xo[j] = k < rows ? (uint32_t)k * (uint32_t)a.in + chunk : FB_OOB;
    }
    xso = 64 * w + lane < rows ? (uint32_t)((64 * w + lane) * a.nb) * 4u : FB_OOB;
#pragma unroll
    for (int g = 0; g < NG; ++g) {  // a strip past the last channel takes a scale that exists
      const int k = strip_row(g * PER_GROUP);
      ws[g] = a.ws + (int64_t)((valid(k) ? channel(k) : 0) / 128) * a.nb;
    }
  };

  // The loads of one block, in LOADS parts: a wave cannot go on while the memory unit's queue is
  // full, so they are issued a few at a time between the products.
  constexpr int LOADS = NW + NX, PER = (LOADS + SW - 2) / (SW - 1);
  auto load = [&](int n, int st, int kb) {
    const bool in = 128 * kb + chunk < a.in;  // chunks past the row's end are zeros
    if (n < NW) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (LdsPtr)(&sh.w[st][1024 * (NW * w + n)]), 16,
                                               in ? wo[n] : FB_OOB, 128u * kb, 0, 0);
    } else if (n < LOADS) {
      const GemmRsrc rx = gemm_rsrc(a.x + t0 * a.in, (uint32_t)rows * (uint32_t)a.in);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (LdsPtr)(&sh.x[st][1024 * (NX * w + n - NW)]), 16,
                                               in ? xo[n - NW] : FB_OOB, 128u * kb, 0, 0);
    }
    if (n == 0 && w < WT) {
      const GemmRsrc rxs = gemm_rsrc(a.xs + t0 * a.nb, (uint32_t)(rows * a.nb) * 4u);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rxs, (LdsPtr)(&sh.sx[st][64 * w]), 4,
                                               kb < a.nb ? xso : FB_OOB, 4u * kb, 0, 0);
    }
  };
  auto load_blocks = [&](int first, int last) {
#pragma unroll
    for (int kb = first; kb < last; ++kb)
#pragma unroll
      for (int n = 0; n < LOADS; ++n) load(n, kb, kb);
  };

  int tile_t, tile_c, half_item, j = blockIdx.x >> 3;
  const int stream = blockIdx.x & 7;
  if (!items.at(stream, j, &tile_t, &tile_c, &half_item)) return;
  set_tile(tile_t, tile_c, half_item);
  load_blocks(0, ST - 1);
  // One item, whole (NT = 4 token tiles of 16 per wave) or half (NT = 2): its first blocks are
  // loading; afterwards those of the next item are. Returns whether there is one.
  auto item = [&](auto tiles) {
    constexpr int NT = decltype(tiles)::value;
    f32x4 acc[SW][NT], p[NT];
    float m[NT];
    const int at0 = 128 * r + 16 * (q ^ (r & 7)), at1 = 128 * r + 16 * ((4 + q) ^ (r & 7));
    FbOperand<EXACT> av[2], bv[NT];
    float sx[NT];
    auto read_a = [&](int st, int s) {
      const uint8_t* l = sh.w[st] + 128 * strip_row(s);
      av[s & 1].set(*reinterpret_cast<const u32x4*>(l + at0), *reinterpret_cast<const u32x4*>(l + at1));
    };
    auto read_b = [&](int st, int t) {
      const uint8_t* l = sh.x[st] + 128 * (16 * NT * wt + 16 * t);
      bv[t].set(*reinterpret_cast<const u32x4*>(l + at0), *reinterpret_cast<const u32x4*>(l + at1));
    };
    auto read_sx = [&](int st, int t) { sx[t] = sh.sx[st][16 * NT * wt + 16 * t + r]; };
    // Adds the last product of token tile t to the sum of strip s (the strip before the one
    // whose product comes next, so that it has had three products' time to finish).
    auto add = [&](int s, int t) {
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[s][t][i] = __builtin_fmaf(p[t][i], m[t], acc[s][t][i]);
      asm volatile("" : "+v"(acc[s][t]));  // done here, not where the compiler would gather them
    };

    // The results leave through LDS (the last stage: its refill waits for the barrier after), 32
    // (fp32: 16) tokens of the wave at a time: stored straight from registers, by 32 bytes of 16 rows an
    // instruction, the bf16 tile took 30,000 cycles beside the 114,000 of its products at 5,120
    // inputs.
    constexpr int NO = GATED ? SW / 2 : SW, ESIZE = EPI == FB_F32 ? 4 : 2, ROW = 16 * NO * ESIZE;
    constexpr int N = EPI == FB_F32 ? 16 : 32;
    static_assert(N * ROW * S::WAVES <= sizeof(sh.w[0]) + sizeof(sh.x[0]), "results' way out");
    auto store_results = [&](int64_t token, int tokens, int channel0) {
      const int lane = fb_fresh_lane(), r = lane & 15, q = lane >> 4;
      constexpr int IN_W = sizeof(sh.w[0]) / (N * ROW);  // waves whose rows fit the weights' part
      FbRows<ROW, N> out{w < IN_W ? sh.w[ST - 1] + w * (N * ROW) : sh.x[ST - 1] + (w - IN_W) * (N * ROW)};
      const int bytes = min(16 * NO, width - channel0) * ESIZE;
      const int64_t stride = (int64_t)(EPI == FB_GATED ? half : a.out) * ESIZE;
#pragma unroll
      for (int f = 0; f < 16 * NT; f += N) {
        uint8_t* dst = static_cast<uint8_t*>(a.y) + (token + f) * stride + (int64_t)channel0 * ESIZE;
        u32x2 du[NO][N / 16];
#pragma unroll
        for (int s = 0; s < NO; ++s)
#pragma unroll
          for (int v = 0; v < N / 16; ++v) {
            const int t = f / 16 + v, k = 16 * v + r, o = 16 * s + 4 * q;
            const f32x4 g = acc[s][t], u = acc[s + SW - NO][t];
            if constexpr (EPI == FB_F32) {
              out.put(k, 4 * o, g);
            } else if constexpr (EPI == FB_BF16) {
              out.put(k, 2 * o, (u32x2){fb_pack_bf16(g[0], g[1]), fb_pack_bf16(g[2], g[3])});
            } else if constexpr (EPI == FB_GATED) {
              out.put(k, 2 * o, fb_gate4(g, u));
            } else {
              u32x2 dh = (u32x2){0, 0}, dg;
              if (f + k < tokens && channel0 + o < width)
                dh = *reinterpret_cast<const u32x2*>(a.dh + (token + f + k) * half + channel0 + o);
              fb_gate_grad4(g, u, dh, &dg, &du[s][v]);
              out.put(k, 2 * o, dg);
            }
          }
        out.store(dst, stride, tokens - f, bytes, lane);
        if constexpr (EPI == FB_GATED_GRAD) {
#pragma unroll
          for (int s = 0; s < NO; ++s)
#pragma unroll
            for (int v = 0; v < N / 16; ++v) out.put(16 * v + r, 2 * (16 * s + 4 * q), du[s][v]);
          out.store(dst + half * 2, stride, tokens - f, bytes, lane);
        }
      }
    };

#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int s = 0; s < SW; ++s) acc[s][t] = (f32x4){0.f, 0.f, 0.f, 0.f};
      p[t] = (f32x4){0.f, 0.f, 0.f, 0.f};
      m[t] = 0.0f;
    }
#pragma unroll
    for (int n = 0; n < PER; ++n) load(n, ST - 1, ST - 1);
    // block 0 has landed: later blocks' loads (the token scales' not counted: not every wave has
    // one) may be in flight
    wait_vmcnt<(ST - 2) * LOADS + PER>();
    bare_barrier();
    read_a(0, 0);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      read_b(0, t);
      read_sx(0, t);
    }
    float ss[NG];
#pragma unroll
    for (int g = 0; g < NG; ++g) ss[g] = fb_uniform_load(ws[g]);
    // One block. Before its last strip, whose operands are in registers, the next block has
    // landed everywhere and this stage is no longer read: its refill starts, and the next block's
    // operands are read as the last strip's products release the registers.
    int st = 0;
    for (int kb = 0; kb < a.nb; ++kb) {
      const int next = st + 1 == ST ? 0 : st + 1, before = st == 0 ? ST - 1 : st - 1;
      float sn[NG];
#pragma unroll
      for (int s = 0; s < SW; ++s) {
        const bool last = s == SW - 1;
        __builtin_amdgcn_sched_barrier(0);
        if (last) {
          wait_vmcnt<(ST - 2) * LOADS>();
          bare_barrier();
          read_a(next, 0);
#pragma unroll
          for (int g = 0; g < NG; ++g) sn[g] = fb_uniform_load(ws[g] + min(kb + 1, a.nb - 1));
        } else {
          read_a(st, s + 1);
        }
#pragma unroll
        for (int n = 0; n < PER; ++n)
          load(n + (last ? 0 : PER * (s + 1)), last ? st : before, kb + (last ? ST : ST - 1));
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          add((s + SW - 1) % SW, t);
          p[t] = fb_block_product(av[s & 1], bv[t]);
          if (s % PER_GROUP == 0) m[t] = sx[t] * ss[s / PER_GROUP];
          if (last) {
            __builtin_amdgcn_sched_barrier(0);
            read_b(next, t);
            read_sx(next, t);
          }
        }
      }
#pragma unroll
      for (int g = 0; g < NG; ++g) ss[g] = sn[g];
      st = next;
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) add(SW - 1, t);
    // the loads past the last block have landed, and no wave reads a stage any more
    wait_vmcnt<0>();
    bare_barrier();
    const int64_t first_token = t0 + 16 * NT * wt;
    const int tokens = rows - 16 * NT * wt, channel0 = c0 + strip_row(0);
    j += gridDim.x >> 3;
    const bool more = items.at(stream, j, &tile_t, &tile_c, &half_item);
    if (more) {
      set_tile(tile_t, tile_c, half_item);
      load_blocks(0, ST - 1);
    }
    store_results(first_token, tokens, channel0);
    bare_barrier();
    return more;
  };
  while (half_item < 0)  // halves come last, one to a workgroup
    if (!item(std::integral_constant<int, 4>())) {
      wait_vmcnt<0>();  // no load may still be writing this workgroup's LDS when it ends
      return;
    }
  item(std::integral_constant<int, 2>());
  wait_vmcnt<0>();
}

template <int EPI, int SW, int WT, int ST, bool SAME>
__global__ __launch_bounds__(128 * WT) void fp8b128_tile_kernel(Fp8b128GemmArgs a, FbItems items) {
  __shared__ FbTile<SW, WT, ST> sh;
  fb_tiles<EPI, SW, WT, ST, SAME>(a, sh, items);
}

template <int EPI, int SW, int WT, int ST>
FbItems tile_items(const Fp8b128GemmArgs& a) {
  using S = FbTile<SW, WT, ST>;
  return FbItems((int)ceil_div(a.T, S::BT), (int)ceil_div(a.out, S::BC));
}

template <int EPI, int SW, int WT, int ST>
hipError_t launch_tiles(const Fp8b128GemmArgs& a, hipStream_t s) {
  const FbItems n = tile_items<EPI, SW, WT, ST>(a);
  const dim3 grid((unsigned)(8 * std::min(n.items, FB_CUS / 8))), block(FbTile<SW, WT, ST>::THREADS);
  // tiles start at multiples of 64 channels, the up half at channel I = out / 2
  if (!fb_gated(EPI) || a.out % 128 == 0)
    return launch_timed(fp8b128_tile_kernel<EPI, SW, WT, ST, true>, grid, block, s, a, n);
  return launch_timed(fp8b128_tile_kernel<EPI, SW, WT, ST, !fb_gated(EPI)>, grid, block, s, a, n);
}

// One or two tokens: exact products in both kernels. A channel per wave has short waves that all
// read at once, but its time grows with the channels; a strip's waves share a row's inputs and
// its time grows with them. Measured (us, a channel per wave / strips; gated in brackets), one
// token: 5,120 x 1,536 4.7 / 4.9 (4.6 / 5.4), 7,168 x 768 3.9 / 5.7 (4.4 / 6.4), 16,384 x 1,536
// 7.0 / 9.5, 16,384 x 5,120 18.6 / 19.0, 2,048 x 5,120 5.7 / 4.2, 768 x 5,120 5.3 / 3.3, 5,120 x
// 10,240 17.2 / 13.5, 256 x 20,480 14.0 / 4.3; two: 16,384 x 1,536 8.6 / 9.6, 5,120 x 768 4.0 /
// 4.5, 5,120 x 1,536 5.5 / 5.0, 7,168 x 5,120 13.4 / 10.8, 256 x 20,480 19.2 / 4.4. Over 70 sizes
// of 256 to 16,384 inputs and 256 to 20,480 channels the choice took 0.3 % more than the faster on
// average, at most 10 % (gated: 1.2 % and, at 16,384 x 10,240, 28 %).
template <int EPI>
hipError_t launch_few(const Fp8b128GemmArgs& a, hipStream_t s) {
  if (a.in >= 2 * a.T * a.out) return launch_rows<EPI>(a, s);
  return launch_strip<EPI, fb_gated(EPI) ? 2 : 1, 1, true>(a, s);
}

// The kernel with the least time expected, beside the 3.7 us that all have in common (0.01 us; bf16
// results / fp32 results). Of strips, by the rounds of workgroups over the compute units and the
// blocks of 128 inputs of a wave, an eighth of all:
//   (1, 1) 29 / 31 a block and round, (2, 1) 48 / 55, (2, 2) 69 / 89, and 38 for each round after
//   the first; (4, 2) 93 a round and 113 / 147 a block of it, (4, 4) 123 and 161 / 216
// Of tiles, by the rounds of tiles, the last of halves, and all blocks:
//   128 x 128 54 and 75 / 120 a block (for one round: two were never the least); 128 x 256 147 a
//   round and 103 / 145 a block of it, of halves 59 / 104; 256 x 256 83 and 148, 114 (bf16 only)
// The constants are a fit to calls of 3 to 1,024 tokens, 768 to 5,120 inputs and channels; a choice
// by them took 0.5 % more than the fastest on average. Measured, (2, 2) / (4, 4) / 128 x 128 / 128 x
// 256 / 256 x 256: 213 tokens x 768 x 5,120 9.2 / 10.4 / 8.3 / 8.6 / 10.7 us; 768 x 2,576 x 1,440
// 16.4 / 18.7 / 20.6 / 20.3 / 32.6; 1,024 x 5,120 x 5,120 43.9 by 128 x 256 tiles, 49.9 by halves of
// 256 x 256; 8,192 x 5,120 x 7,168 281 in four rounds of 256 x 256, 268 with the last in halves.
template <int EPI>
hipError_t launch_forward(const Fp8b128GemmArgs& a, hipStream_t s) {
  constexpr bool EXACT = EPI == FB_F32;
  if (a.T <= 2) return launch_few<EPI>(a, s);
  typedef hipError_t (*Launch)(const Fp8b128GemmArgs&, hipStream_t);
  int64_t least = INT64_MAX;
  Launch best = nullptr;
  auto offer = [&](int64_t cost, Launch f) {
    if (cost < least) {
      least = cost;
      best = f;
    }
  };
  const int64_t wave_blocks = ceil_div(a.nb, FbStrip<1, 1>::W);
  auto strips = [&](int64_t groups, int block, Launch f) {
    const int64_t rounds = ceil_div(groups, FB_CUS);
    offer(rounds * block * wave_blocks + 38 * (rounds - 1), f);
  };
  if constexpr (!fb_gated(EPI)) strips(strip_groups<EPI, 1, 1>(a), EXACT ? 31 : 29, launch_strip<EPI, 1, 1>);
  strips(strip_groups<EPI, 2, 1>(a), EXACT ? 55 : 48, launch_strip<EPI, 2, 1>);
  strips(strip_groups<EPI, 2, 2>(a), EXACT ? 89 : 69, launch_strip<EPI, 2, 2>);
  offer(ceil_div(strip_groups<EPI, 4, 2>(a), FB_CUS) * (93 + (EXACT ? 147 : 113) * wave_blocks),
        launch_strip<EPI, 4, 2>);
  offer(ceil_div(strip_groups<EPI, 4, 4>(a), FB_CUS) * (123 + (EXACT ? 216 : 161) * wave_blocks),
        launch_strip<EPI, 4, 4>);
  // whole rounds and, where the last one is of halves, that
  auto rounds = [&](const FbItems& n, int64_t round, int64_t whole, int64_t halves) {
    return ceil_div(n.full, FB_CUS / 8) * (round + whole * a.nb) +
           (n.items > n.full ? round + halves * a.nb : 0);
  };
  if (tile_items<EPI, 4, 2, 2>(a).per <= FB_CUS / 8)
    offer(54 + (EXACT ? 120 : 75) * a.nb, launch_tiles<EPI, 4, 2, 2>);
  offer(rounds(tile_items<EPI, 4, 4, 3>(a), 147, EXACT ? 145 : 103, EXACT ? 104 : 59), launch_tiles<EPI, 4, 4, 3>);
  if constexpr (!EXACT)
    offer(rounds(tile_items<EPI, 8, 4, 2>(a), 83, 148, 114), launch_tiles<EPI, 8, 4, 2>);
  return best(a, s);
}

}  // namespace

hipError_t launch_fp8b128_gemm(const Fp8b128GemmArgs& a, int epi, hipStream_t s) {
  switch (epi) {
    case FB_F32: return launch_forward<FB_F32>(a, s);
    case FB_BF16: return launch_forward<FB_BF16>(a, s);
    case FB_GATED: return launch_forward<FB_GATED>(a, s);
    default: return launch_forward<FB_GATED_GRAD>(a, s);
  }
}

}  // namespace tq

// The products over the fp8b128 store (FORMAT F24, F25):
//   y[t][o] = sum over blocks b of 128 inputs of xs[t][b] * ws[o / 128][b] * P_b[t][o],
//   P_b[t][o] = sum over the block's inputs of x code * w code,
// P_b by the matrix cores from zero, then one fp32 multiply-add per block into the sum, since
// a scale belongs to a block. Weights are the A operand and activations the B operand, so a
// lane ends with four consecutive channels of one token.
#include "fp8b128.h"

#include <algorithm>

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
        FbOperand<EXACT> wv[NS];
#pragma unroll
        for (int s = 0; s < NS; ++s) wv[s].set(wf[d][s][0], wf[d][s][1]);
#pragma unroll
        for (int t = 0; t < TT; ++t) {
          FbOperand<EXACT> xv;
          xv.set(xf[d][t][0], xf[d][t][1]);
#pragma unroll
          for (int s = 0; s < NS; ++s) {
            const f32x4 p = fb_block_product(wv[s], xv);
            const float m = sx[d][t] * ss[d][s];
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[t][s][i] = __builtin_fmaf(p[i], m, acc[t][s][i]);
          }
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

// ---- many tokens: tiles of both operands in LDS ----------------------------------------------
//
// A workgroup of 2 x WT waves owns 64 * WT tokens and 32 * SW weight rows (gated: the gate rows
// of 16 * SW channels, then their up rows), wave (wc, wt) SW strips of 16 channels (gated: half
// of them gate strips, half the up strips of the same channels, so that both sums of a channel
// end in one lane) and 4 tiles of 16 tokens. Per block of 128 inputs the rows' 128 bytes go
// straight to LDS (16-byte chunk c of row r at position c ^ (r % 8), so that eight lanes reading
// one chunk of eight rows meet eight different banks' worth of LDS), in two stages with one
// barrier per block.
template <int SW, int WT>
struct FbTile {
  static constexpr int WAVES = 2 * WT, THREADS = 64 * WAVES, BC = 32 * SW, BT = 64 * WT;
  alignas(16) uint8_t w[2][BC * 128];
  alignas(16) uint8_t x[2][BT * 128];
  alignas(16) float sx[2][BT];
};

// One workgroup per compute unit takes tile after tile: the first block of the next tile is
// loading while a tile's results are stored.
//
// SAME: the wave's strips (gated: its gate strips, and its up strips) lie in one block of 128
// channels, so that a block of inputs has one scale for them.
template <int EPI, int SW, int WT, bool SAME>
__device__ void fb_tiles(const Fp8b128GemmArgs& a, FbTile<SW, WT>& sh, int tt, int tc) {
  using S = FbTile<SW, WT>;
  constexpr bool GATED = fb_gated(EPI), EXACT = EPI == FB_F32;
  constexpr int NX = S::BT / S::WAVES / 8, NW = S::BC / S::WAVES / 8;
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wc = w & 1, wt = w >> 1;
  const int half = a.out / 2, width = GATED ? half : a.out;
  const GemmRsrc rw = gemm_rsrc(a.w, (uint32_t)a.out * (uint32_t)a.in);
  const GemmRsrc rws = gemm_rsrc(a.ws, (uint32_t)(((a.out + 127) / 128) * a.nb) * 4u);
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
  uint32_t wo[NW], xo[NX], xso, wso;
  auto set_tile = [&](int tile_t, int tile_c) {
    const int lane = fb_fresh_lane(), chunk = 16 * ((lane & 7) ^ (lane >> 3));
    t0 = (int64_t)tile_t * S::BT;
    rows = (int)min((int64_t)S::BT, a.T - t0);
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
    const int k = strip_row(lane % SW);  // lane s loads strip s's scale
    wso = valid(k) ? (uint32_t)(channel(k) / 128 * a.nb) * 4u : FB_OOB;
  };

  // The loads of one block, in LOADS parts: a wave cannot go on while the memory unit's queue is
  // full, so they are issued a few at a time between the products.
  constexpr int LOADS = 1 + NW + NX, PER = SW == 8 ? 2 : 3;
  float sw_after = 0.0f;  // the wave's weight scales of the block, strip s in lane s
  auto load = [&](int n, int st, int kb) {
    const bool in = 128 * kb + chunk < a.in;  // chunks past the row's end are zeros
    if (n == 0) {
      sw_after = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rws, kb < a.nb ? wso : FB_OOB, 4u * kb, 0));
      const GemmRsrc rxs = gemm_rsrc(a.xs + t0 * a.nb, (uint32_t)(rows * a.nb) * 4u);
      if (w < WT)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rxs, (LdsPtr)(&sh.sx[st][64 * w]), 4,
                                                 kb < a.nb ? xso : FB_OOB, 4u * kb, 0, 0);
    } else if (n <= NW) {
      const int j = n - 1;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (LdsPtr)(&sh.w[st][1024 * (NW * w + j)]), 16,
                                               in ? wo[j] : FB_OOB, 128u * kb, 0, 0);
    } else if (n < LOADS) {
      const int j = n - 1 - NW;
      const GemmRsrc rx = gemm_rsrc(a.x + t0 * a.in, (uint32_t)rows * (uint32_t)a.in);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (LdsPtr)(&sh.x[st][1024 * (NX * w + j)]), 16,
                                               in ? xo[j] : FB_OOB, 128u * kb, 0, 0);
    }
  };

  f32x4 acc[SW][4], p[4];
  float m[4];
  const int at0 = 128 * r + 16 * (q ^ (r & 7)), at1 = 128 * r + 16 * ((4 + q) ^ (r & 7));
  FbOperand<EXACT> av[2], bv[4];
  float sx[4];
  auto read_a = [&](int st, int s) {
    const uint8_t* l = sh.w[st] + 128 * strip_row(s);
    av[s & 1].set(*reinterpret_cast<const u32x4*>(l + at0), *reinterpret_cast<const u32x4*>(l + at1));
  };
  auto read_b = [&](int st, int t) {
    const uint8_t* l = sh.x[st] + 128 * (64 * wt + 16 * t);
    bv[t].set(*reinterpret_cast<const u32x4*>(l + at0), *reinterpret_cast<const u32x4*>(l + at1));
  };
  auto read_sx = [&](int st, int t) { sx[t] = sh.sx[st][64 * wt + 16 * t + r]; };
  // Adds the last product of token tile t to the sum of strip s (the strip before the one
  // whose product comes next, so that it has had three products' time to finish).
  auto add = [&](int s, int t) {
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[s][t][i] = __builtin_fmaf(p[t][i], m[t], acc[s][t][i]);
    asm volatile("" : "+v"(acc[s][t]));  // done here, not where the compiler would gather them
  };

  // The results leave through LDS (the second stage: its refill waits for the barrier after), 32
  // (fp32: 16) tokens of the wave at a time: stored straight from registers, by 32 bytes of 16 rows an
  // instruction, the bf16 tile took 30,000 cycles beside the 114,000 of its products at 5,120
  // inputs.
  constexpr int NO = GATED ? SW / 2 : SW, ESIZE = EPI == FB_F32 ? 4 : 2, ROW = 16 * NO * ESIZE;
  constexpr int N = EPI == FB_F32 ? 16 : 32;
  static_assert(N * ROW * S::WAVES <= sizeof(sh.w[1]) + sizeof(sh.x[1]), "results' way out");
  auto store_results = [&](int64_t token, int tokens, int channel0) {
    const int lane = fb_fresh_lane(), r = lane & 15, q = lane >> 4;
    constexpr int IN_W = sizeof(sh.w[1]) / (N * ROW);  // waves whose rows fit the weights' part
    FbRows<ROW, N> out{w < IN_W ? sh.w[1] + w * (N * ROW) : sh.x[1] + (w - IN_W) * (N * ROW)};
    const int bytes = min(16 * NO, width - channel0) * ESIZE;
    const int64_t stride = (int64_t)(EPI == FB_GATED ? half : a.out) * ESIZE;
#pragma unroll
    for (int f = 0; f < 64; f += N) {
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

  int tile_t, tile_c, j = blockIdx.x >> 3;
  if (!fb_tile_of(tt, tc, j, &tile_t, &tile_c)) return;
  set_tile(tile_t, tile_c);
#pragma unroll
  for (int n = 0; n < LOADS; ++n) load(n, 0, 0);
  for (bool more = true; more;) {
#pragma unroll
    for (int t = 0; t < 4; ++t) {
#pragma unroll
      for (int s = 0; s < SW; ++s) acc[s][t] = (f32x4){0.f, 0.f, 0.f, 0.f};
      p[t] = (f32x4){0.f, 0.f, 0.f, 0.f};
      m[t] = 0.0f;
    }
    float sw = sw_after;
#pragma unroll
    for (int n = 0; n < PER; ++n) load(n, 1, 1);
    wait_vmcnt<PER - 1>();  // part 0 may have no load that writes LDS, and no other is counted on
    bare_barrier();
    read_a(0, 0);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      read_b(0, t);
      read_sx(0, t);
    }
    // One block. Before its last strip, whose operands are in registers, the next block has
    // landed everywhere and this stage is no longer read: its refill starts, and the next block's
    // operands are read as the last strip's products release the registers.
    for (int kb = 0; kb < a.nb; ++kb) {
      const int st = kb & 1;
      float sw_next = 0.0f;
#pragma unroll
      for (int s = 0; s < SW; ++s) {
        const bool last = s == SW - 1;
        __builtin_amdgcn_sched_barrier(0);
        if (last) {
          wait_vmcnt<0>();
          bare_barrier();
          read_a(st ^ 1, 0);
        } else {
          read_a(st, s + 1);
        }
        if (last) sw_next = sw_after;
#pragma unroll
        for (int n = 0; n < PER; ++n)
          load(n + (last ? 0 : PER * (s + 1)), last ? st : st ^ 1, kb + (last ? 2 : 1));
        const float ss = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(sw), s));
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          add((s + SW - 1) % SW, t);
          p[t] = fb_block_product(av[s & 1], bv[t]);
          if (!SAME || s % (GATED ? SW / 2 : SW) == 0) m[t] = sx[t] * ss;
          if (last) {
            __builtin_amdgcn_sched_barrier(0);
            read_b(st ^ 1, t);
            read_sx(st ^ 1, t);
          }
        }
      }
      sw = sw_next;
    }
#pragma unroll
    for (int t = 0; t < 4; ++t) add(SW - 1, t);
    // the loads past the last block have landed, and no wave reads a stage any more
    wait_vmcnt<0>();
    bare_barrier();
    const int64_t first_token = t0 + 64 * wt;
    const int tokens = rows - 64 * wt, channel0 = c0 + strip_row(0);
    j += gridDim.x >> 3;
    more = fb_tile_of(tt, tc, j, &tile_t, &tile_c);
    if (more) {
      set_tile(tile_t, tile_c);
#pragma unroll
      for (int n = 0; n < LOADS; ++n) load(n, 0, 0);
    }
    store_results(first_token, tokens, channel0);
    bare_barrier();
  }
  wait_vmcnt<0>();  // no load may still be writing this workgroup's LDS when it ends
}

template <int EPI, int SW, int WT, bool SAME>
__global__ __launch_bounds__(128 * WT) void fp8b128_tile_kernel(Fp8b128GemmArgs a, int tt, int tc) {
  __shared__ FbTile<SW, WT> sh;
  fb_tiles<EPI, SW, WT, SAME>(a, sh, tt, tc);
}

template <int EPI, int SW, int WT>
hipError_t launch_tiles(const Fp8b128GemmArgs& a, hipStream_t s) {
  using S = FbTile<SW, WT>;
  const int width = fb_gated(EPI) ? a.out / 2 : a.out, bc = fb_gated(EPI) ? S::BC / 2 : S::BC;
  const int tt = (int)((a.T + S::BT - 1) / S::BT), tc = (width + bc - 1) / bc;
  // two workgroups of the smaller tile share a compute unit
  const dim3 grid((unsigned)std::min((tt * tc + 7) & ~7, S::WAVES == 4 ? 2 * FB_CUS : FB_CUS));
  const dim3 block(S::THREADS);
  // tiles start at multiples of 64 channels, the up half at channel I = width
  if (!fb_gated(EPI) || width % 64 == 0)
    return launch_timed(fp8b128_tile_kernel<EPI, SW, WT, true>, grid, block, s, a, tt, tc);
  return launch_timed(fp8b128_tile_kernel<EPI, SW, WT, !fb_gated(EPI)>, grid, block, s, a, tt, tc);
}

template <int EPI>
hipError_t launch_forward(const Fp8b128GemmArgs& a, hipStream_t s) {
  // By the number of 256 x 256 tiles: from half the compute units on they are the fastest
  // (8,192 x 5,120 x 7,168: 359 us, against 439 us with 128 x 128); below it smaller tiles
  // spread the work wider (1,024 x 5,120 x 5,120, 80 tiles: 61 against 80 us; 512 x 5,120 x
  // 1,536: 46 against 79 us), and up to 256 tokens strips wider still (128 x 5,120 x 1,536: 23
  // against 46 us).
  const int64_t big = (a.T + 255) / 256 * ((a.out + 255) / 256);
  if (big >= 128) return launch_tiles<EPI, EPI == FB_F32 ? 4 : 8, 4>(a, s);
  if (a.T > 256) return launch_tiles<EPI, 4, 2>(a, s);
  return launch_strips<EPI>(a, s);
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

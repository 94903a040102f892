// The gradients of a product over the fp8b128 store (FORMAT F26), on the bf16 matrix cores:
//   dx[t][i] = sum over o of dy[t][o] * W[o][i],    W = scale of the block * code
//   dw[o][i] = sum over t of dy[t][o] * X[t][i],    X = scale of the token's block * code
// Both contract over the rows of a row-major operand, so a lane's eight operand values lie in
// eight (bf16: twice four) rows: the LDS transpose reads fetch them. ds_read_b64_tr_b8: of each
// 16 lanes, lanes 2k and 2k + 1 address the two halves of 16 bytes of row k (k = 0..7), and
// lane j gets byte j of the eight rows. ds_read_b64_tr_b16: lanes 4k .. 4k + 3 address the
// quarters of 32 bytes of row k (k = 0..3), and lane j gets half-word j of the four rows.
// Inputs are the A operand, so a lane ends with four consecutive inputs of a token or channel.
#include "fp8b128.h"

#include <algorithm>

namespace tq {

namespace {

typedef int32_t i32x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) i32x2* LdsI32x2;
typedef __attribute__((address_space(3))) s16x4* LdsS16x4;

// The pointers are __restrict__ for the compiler's wait insertion: it makes an LDS read that it
// knows nothing about wait for every load in flight that writes LDS, the ones meant to stay in
// flight across the read included; the kernels' own waits and barriers order the two.
__device__ __forceinline__ u32x2 read_tr8(const uint8_t* __restrict__ p) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr8_b64_v2i32((LdsI32x2)(p)));
}
__device__ __forceinline__ u32x2 read_tr16(const uint8_t* __restrict__ p) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsS16x4)(p)));
}

__device__ __forceinline__ void store4(uint16_t* p, f32x4 v) {
  *reinterpret_cast<u32x2*>(p) = (u32x2){fb_pack_bf16(v[0], v[1]), fb_pack_bf16(v[2], v[3])};
}

// ---- dx, few tokens: 32 inputs of up to 16 * TT tokens per workgroup ------------------------
//
// The eight waves take the blocks of 128 outputs in turn, each with LDS of its own (no barrier
// until the end), one block ahead: the block's 128 x 32 codes straight to LDS, the tokens' dy
// to registers in operand order. A block's sums are scaled by its weight scale; the waves'
// sums are added in wave order.
constexpr int DS_WAVES = 8;
constexpr int DS_THREADS = 64 * DS_WAVES;

template <int TT>
struct DxStripShared {
  alignas(16) uint8_t w[DS_WAVES][2][128 * 32];
  f32x4 red[DS_WAVES][TT * 2][64];
};

template <int TT>
__device__ void dx_strip(const Fp8b128BackwardArgs& a, DxStripShared<TT>& sh) {
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int cols = (a.in + 31) / 32;
  const int i0 = (int)(blockIdx.x % cols) * 32;
  const int64_t t0 = (int64_t)(blockIdx.x / cols) * (16 * TT);
  const int rows = (int)min((int64_t)(16 * TT), a.T - t0);
  const int nob = (a.out + 127) / 128;

  const GemmRsrc rd = gemm_rsrc(a.dy + t0 * a.out, (uint32_t)rows * (uint32_t)a.out * 2u);
  const GemmRsrc rs = gemm_rsrc(a.ws, (uint32_t)(nob * a.nb) * 4u);
  // codes: instruction j fills rows 32 j .. + 31; lane l half l % 2 of row l / 2, which holds
  // the row's half (l % 2) ^ (row / 4 % 2), so that a transpose read's eight rows meet
  // different banks
  const int wrow = lane >> 1, wcol = 16 * ((lane & 1) ^ ((wrow >> 2) & 1));
  const uint32_t wo = i0 + wcol < a.in ? (uint32_t)wrow * (uint32_t)a.in + i0 + wcol : FB_OOB;
  uint32_t dof[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t)
    dof[t] = 16 * t + r < rows ? (uint32_t)(16 * t + r) * (uint32_t)a.out * 2u + 16u * q : FB_OOB;

  // Loads of one block that the waits count: the compiler could move the scale's across a wait,
  // so it is not one of them.
  constexpr int LOADS = 4 + 4 * TT;
  u32x4 d[2][TT][4];
  float sc[2];
  auto load = [&](int k, int ob) {  // blocks past the last are read as zeros
    const int left = min(128, a.out - 128 * ob);
    const GemmRsrc rw = gemm_rsrc(a.w + (int64_t)(left > 0 ? 128 * ob : 0) * a.in,
                                  left > 0 ? (uint32_t)left * (uint32_t)a.in : 0u);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (LdsPtr)(&sh.w[w][k][1024 * j]), 16,
                                               wo == FB_OOB ? FB_OOB : wo + 32u * j * (uint32_t)a.in,
                                               0, 0, 0);
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool in = 128 * ob + 32 * j + 8 * q < a.out && dof[t] != FB_OOB;
        d[k][t][j] = __builtin_amdgcn_raw_buffer_load_b128(rd, in ? dof[t] + 256u * ob + 64u * j : FB_OOB, 0, 0);
      }
    sc[k] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
        rs, ob < nob ? (uint32_t)(ob * a.nb + i0 / 128) * 4u : FB_OOB, 0, 0));
  };
  f32x4 acc[TT][2];
#pragma unroll
  for (int t = 0; t < TT; ++t) acc[t][0] = acc[t][1] = (f32x4){0.f, 0.f, 0.f, 0.f};
  // lane (j = l % 16, q) of a transpose read: row 8 q + j / 2, half j % 2 of 16-byte column c
  auto compute = [&](int k) {
    f32x4 p[TT][2];
#pragma unroll
    for (int t = 0; t < TT; ++t) p[t][0] = p[t][1] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int row = 32 * j + 8 * q + (r >> 1);
        const u32x2 v = read_tr8(&sh.w[w][k][32 * row + 16 * (c ^ ((row >> 2) & 1)) + 8 * (r & 1)]);
        const u32x4 av = fb_bf16_of8(v.x, v.y);
#pragma unroll
        for (int t = 0; t < TT; ++t) p[t][c] = mfma_bf16(av, d[k][t][j], p[t][c]);
      }
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[t][c][i] = __builtin_fmaf(p[t][c][i], sc[k], acc[t][c][i]);
  };
  // one step: the next block's loads, then this block's data (all but those loads have landed)
  auto step = [&](int k, int ob) {
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): no read of the stage is outstanding
    __builtin_amdgcn_sched_barrier(0);
    load(k ^ 1, ob + DS_WAVES);
    __builtin_amdgcn_sched_barrier(0);
    wait_vmcnt<LOADS>();
    __builtin_amdgcn_sched_barrier(0);
    compute(k);
  };
  load(0, w);
  for (int ob = w; ob < nob; ob += 2 * DS_WAVES) {
    step(0, ob);
    if (ob + DS_WAVES < nob) step(1, ob + DS_WAVES);
  }
  wait_vmcnt<0>();  // no load may still be writing this workgroup's LDS when it ends
#pragma unroll
  for (int t = 0; t < TT; ++t)
#pragma unroll
    for (int c = 0; c < 2; ++c) sh.red[w][2 * t + c][lane] = acc[t][c];
  __syncthreads();
  const int v = threadIdx.x >> 6;  // wave v finishes tile v
  if (v < 2 * TT) {
    f32x4 sum = sh.red[0][v][lane];
#pragma unroll
    for (int u = 1; u < DS_WAVES; ++u) sum += sh.red[u][v][lane];
    const int row = 16 * (v >> 1) + r, i = i0 + 16 * (v & 1) + 4 * q;
    if (row < rows && i < a.in) store4(a.dx + (t0 + row) * a.in + i, sum);
  }
}

template <int TT>
__global__ __launch_bounds__(DS_THREADS) void fp8b128_dx_strip_kernel(Fp8b128BackwardArgs a) {
  __shared__ DxStripShared<TT> sh;
  dx_strip<TT>(a, sh);
}

// The 64 x 64 results of each wave of a tile (row 16 t + lane % 16, inputs 16 c + 4 (lane / 16) ..
// + 3 in acc[c][t]) to its rows at dst, of which `rows` exist and `bytes` of each, by whole rows
// through 4096 bytes of LDS of the wave's own.
__device__ __forceinline__ void store_tile(uint8_t* lds, const f32x4 (&acc)[4][4], uint8_t* dst,
                                           int64_t stride, int rows, int bytes) {
  const int lane = fb_fresh_lane(), r = lane & 15, q = lane >> 4;
  FbRows<128, 32> out{lds};
#pragma unroll
  for (int hf = 0; hf < 2; ++hf) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const f32x4 x = acc[c][2 * hf + v];
        out.put(16 * v + r, 2 * (16 * c + 4 * q), (u32x2){fb_pack_bf16(x[0], x[1]), fb_pack_bf16(x[2], x[3])});
      }
    out.store(dst + 32 * hf * stride, stride, rows - 32 * hf, bytes, lane);
  }
}

// ---- dx, many tokens ------------------------------------------------------------------------
//
// A workgroup of eight waves owns 256 inputs of 128 tokens, wave (wi, wt) 64 inputs of 64
// tokens. Steps of 64 outputs: 64 rows of 256 code bytes and 128 rows of 128 bytes of dy go
// straight to a ring of four LDS stages, three steps ahead. The products of two steps (one block
// of 128 outputs) are added from zero and then scaled into the sums.
struct DxShared {
  alignas(16) uint8_t w[4][64 * 256];
  alignas(16) uint8_t d[4][128 * 128];
};

// One workgroup per compute unit takes tile after tile: the first steps of the next tile are
// loading while a tile's results are stored.
struct DxTile {
  int64_t t0;
  int rows, i0, ib;
  uint32_t wo[2], dof[2];
};

__device__ __forceinline__ DxTile dx_tile_at(const Fp8b128BackwardArgs& a, int tile_t, int tile_i, int w) {
  const int lane = fb_fresh_lane();
  DxTile d;
  d.t0 = (int64_t)tile_t * 128;
  d.rows = (int)min((int64_t)128, a.T - d.t0);
  d.i0 = tile_i * 256;
  d.ib = min((d.i0 + 64 * (w & 3)) / 128, a.nb - 1);
  // codes: an instruction fills 4 rows; lane l position l % 16 of row l / 16, which holds the
  // row's 16-byte chunk (l % 16) ^ (row % 16). dy: 8 rows; position l % 8 of row l / 8 holds
  // chunk (l % 8) ^ (row % 8).
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int row = 8 * w + 4 * j + (lane >> 4), col = d.i0 + 16 * ((lane & 15) ^ (row & 15));
    d.wo[j] = col < a.in ? (uint32_t)row * (uint32_t)a.in + col : FB_OOB;
    const int tok = 16 * w + 8 * j + (lane >> 3);
    d.dof[j] = tok < d.rows ? (uint32_t)tok * (uint32_t)a.out * 2u + 16u * ((lane & 7) ^ (lane >> 3)) : FB_OOB;
  }
  return d;
}

__device__ void dx_tiles(const Fp8b128BackwardArgs& a, DxShared& sh, int tt, int ti) {
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wi = w & 3, wt = w >> 2;
  const int nsteps = (a.out + 63) / 64;
  const int dcol = 8 * ((lane & 7) ^ (lane >> 3));  // this lane's first output of a step
  constexpr int LOADS = 4;  // of one step; the scales come through the scalar cache
  DxTile d;
  // A step's loads, in four parts (a wave cannot go on while the memory unit's queue is full, so
  // they are issued between the products); steps past the last are read as zeros.
  auto load = [&](int n, int st, int k) {
    const int left = min(64, a.out - 64 * k);
    if (n < 2) {
      const GemmRsrc rw = gemm_rsrc(a.w + (int64_t)(left > 0 ? 64 * k : 0) * a.in,
                                    left > 0 ? (uint32_t)left * (uint32_t)a.in : 0u);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (LdsPtr)(&sh.w[st][256 * (8 * w + 4 * n)]), 16,
                                               d.wo[n], 0, 0, 0);
    } else {
      const GemmRsrc rd = gemm_rsrc(a.dy + d.t0 * a.out, (uint32_t)d.rows * (uint32_t)a.out * 2u);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rd, (LdsPtr)(&sh.d[st][128 * (16 * w + 8 * (n - 2))]), 16,
                                               dcol < left ? d.dof[n - 2] : FB_OOB, 128u * k, 0, 0);
    }
  };

  f32x4 acc[4][4], p[4][4];
  // operands of 32 outputs (half j of a step)
  u32x2 av[2][4];
  u32x4 bv[2][4];
  auto read = [&](int st, int j) {
#pragma unroll
    for (int t = 0; t < 4; ++t)
      bv[j][t] = *reinterpret_cast<const u32x4*>(
          &sh.d[st][128 * (64 * wt + 16 * t + r) + 16 * ((4 * j + q) ^ (r & 7))]);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int row = 32 * j + 8 * q + (r >> 1);
      av[j][c] = read_tr8(&sh.w[st][256 * row + 16 * ((4 * wi + c) ^ (row & 15)) + 8 * (r & 1)]);
    }
  };
  auto multiply = [&](int j, bool first, int st, int k) {  // with the loads of step k, if k >= 0
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (k >= 0) {
        __builtin_amdgcn_sched_barrier(0);
        load(c, st, k);
      }
      const u32x4 a8 = fb_bf16_of8(av[j][c].x, av[j][c].y);
#pragma unroll
      for (int t = 0; t < 4; ++t)
        p[c][t] = mfma_bf16(a8, bv[j][t], first ? (f32x4){0.f, 0.f, 0.f, 0.f} : p[c][t]);
    }
  };
  // A step's second half is read while its first half is multiplied, and the next step's first
  // half while its second is: between the two, the next step's data have landed everywhere,
  // and this step's stage is no longer read.
  auto step = [&](int st, int k) {
    float s = 0.0f;
    if (st & 1) s = fb_uniform_load(a.ws + (int64_t)(k / 2) * a.nb + d.ib);
    read(st, 1);
    multiply(0, (st & 1) == 0, 0, -1);
    __builtin_amdgcn_sched_barrier(0);
    wait_vmcnt<2 * LOADS>();
    bare_barrier();
    read((st + 1) & 3, 0);
    multiply(1, false, st, k + 4);
    if (st & 1) {  // the block of 128 outputs is complete
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[c][t][i] = __builtin_fmaf(p[c][t][i], s, acc[c][t][i]);
    }
  };
  auto load_steps = [&](int first, int last) {
#pragma unroll
    for (int k = first; k < last; ++k)
#pragma unroll
      for (int n = 0; n < 4; ++n) load(n, k, k);
  };

  int tile_t, tile_i;
  int j = blockIdx.x >> 3;
  if (!fb_tile_of(tt, ti, j, &tile_t, &tile_i)) return;
  d = dx_tile_at(a, tile_t, tile_i, w);
  load_steps(0, 3);
  for (bool more = true; more;) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int t = 0; t < 4; ++t) acc[c][t] = (f32x4){0.f, 0.f, 0.f, 0.f};
    load_steps(3, 4);
    wait_vmcnt<3 * LOADS>();
    bare_barrier();
    read(0, 0);
    // whole blocks (a step past the last adds zeros)
    for (int k = 0; k < nsteps; k += 4) {
      step(0, k);
      step(1, k + 1);
      if (k + 2 < nsteps) {
        step(2, k + 2);
        step(3, k + 3);
      }
    }
    // the loads past the last step have landed, and no wave reads a stage any more
    wait_vmcnt<0>();
    bare_barrier();
    uint8_t* dst = reinterpret_cast<uint8_t*>(a.dx + (d.t0 + 64 * wt) * a.in + d.i0 + 64 * wi);
    const int rows = d.rows - 64 * wt, bytes = (a.in - d.i0 - 64 * wi) * 2;
    j += gridDim.x >> 3;
    more = fb_tile_of(tt, ti, j, &tile_t, &tile_i);
    if (more) {
      d = dx_tile_at(a, tile_t, tile_i, w);
      load_steps(0, 3);
    }
    // through the last stage, which the next tile fills after the barrier
    store_tile(w < 4 ? sh.w[3] + 4096 * w : sh.d[3] + 4096 * (w - 4), acc, dst, (int64_t)a.in * 2, rows, bytes);
    bare_barrier();
  }
  wait_vmcnt<0>();
}

__global__ __launch_bounds__(512) void fp8b128_dx_kernel(Fp8b128BackwardArgs a, int tt, int ti) {
  __shared__ DxShared sh;
  dx_tiles(a, sh, tt, ti);
}

// ---- dw -------------------------------------------------------------------------------------
//
// X as bf16 [T][in] (exact for scales that are powers of two), once per call: every channel
// tile of the product reads it.
__global__ __launch_bounds__(256) void fp8b128_widen_kernel(const uint8_t* __restrict__ x,
                                                            const float* __restrict__ xs, int64_t n16,
                                                            int in, int nb, u32x4* __restrict__ y) {
  const int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x;  // 16 inputs of a row
  if (k >= n16) return;
  const int per = in / 16;
  const int64_t t = k / per;
  const float s = xs[t * nb + (int)(k % per) / 8];
  const u32x4 c = *reinterpret_cast<const u32x4*>(x + 16 * k);
  u32x4 out[2];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const u32x2 v = fb_bf16_of4(c[j]);
    out[j / 2][j % 2 * 2] = fb_pack_bf16(bf16_lo_to_f32(v.x) * s, bf16_hi_to_f32(v.x) * s);
    out[j / 2][j % 2 * 2 + 1] = fb_pack_bf16(bf16_lo_to_f32(v.y) * s, bf16_hi_to_f32(v.y) * s);
  }
  y[2 * k] = out[0];
  y[2 * k + 1] = out[1];
}

// A workgroup of eight waves owns 256 inputs of 128 channels, wave (wi, wo) 64 inputs of 64
// channels; steps of 64 tokens through a ring of three LDS stages, two steps ahead. A row's
// 32-byte chunk c lies at position c ^ swizzle(row): the LDS serves 32 lanes at a time, which
// read one chunk of rows 8 q + 0..3 and 8 (q + 1) + 0..3 (or + 4..7), and those eight rows get
// eight different positions.
__device__ __forceinline__ int dw_swizzle(int row) { return (row & 3) | (row >> 1 & 4); }

struct DwShared {
  alignas(16) uint8_t x[3][64 * 512];
  alignas(16) uint8_t d[3][64 * 256];
};

__device__ void dw_tile(const Fp8b128BackwardArgs& a, DwShared& sh, int tile_o, int tile_i) {
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wi = w & 3, wo = w >> 2;
  const int i0 = tile_i * 256, o0 = tile_o * 128;
  const int nsteps = (int)((a.T + 63) / 64);
  uint32_t xo[4], dof[2];
#pragma unroll
  for (int j = 0; j < 4; ++j) {  // two rows of 512 bytes per instruction
    const int row = 8 * w + 2 * j + (lane >> 5), pos = lane & 31;
    const int i = i0 + 16 * ((pos >> 1) ^ dw_swizzle(row)) + 8 * (pos & 1);
    xo[j] = i < a.in ? ((uint32_t)row * (uint32_t)a.in + i) * 2u : FB_OOB;
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {  // four rows of 256 bytes
    const int row = 8 * w + 4 * j + (lane >> 4), pos = lane & 15;
    const int o = o0 + 16 * ((pos >> 1) ^ dw_swizzle(row)) + 8 * (pos & 1);
    dof[j] = o < a.out ? ((uint32_t)row * (uint32_t)a.out + o) * 2u : FB_OOB;
  }
  constexpr int LOADS = 6;
  // A step's loads, in three parts, as in dx_tile; rows past the last token are read as zeros.
  auto load = [&](int n, int st, int k) {
    const int64_t t = (int64_t)64 * k;
    const int left = (int)min((int64_t)64, a.T - t);
    const int64_t at = left > 0 ? t : 0;
    if (n < 2) {
      const GemmRsrc rx = gemm_rsrc(a.xw + at * a.in, left > 0 ? (uint32_t)left * (uint32_t)a.in * 2u : 0u);
#pragma unroll
      for (int j = 2 * n; j < 2 * n + 2; ++j)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (LdsPtr)(&sh.x[st][512 * (8 * w + 2 * j)]), 16,
                                                 xo[j], 0, 0, 0);
    } else {
      const GemmRsrc rd = gemm_rsrc(a.dy + at * a.out, left > 0 ? (uint32_t)left * (uint32_t)a.out * 2u : 0u);
#pragma unroll
      for (int j = 0; j < 2; ++j)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rd, (LdsPtr)(&sh.d[st][256 * (8 * w + 4 * j)]), 16,
                                                 dof[j], 0, 0, 0);
    }
  };
  f32x4 acc[4][4];
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int t = 0; t < 4; ++t) acc[c][t] = (f32x4){0.f, 0.f, 0.f, 0.f};
  // operands of 32 tokens (half j of a step). Lane (r, q) of half h: row 32 j + 8 q + 4 h + r / 4,
  // quarter r % 4 of a 32-byte chunk
  u32x4 av[2][4], bv[2][4];
  auto read = [&](int st, int j) {
    const int row = 32 * j + 8 * q + (r >> 2), sw = dw_swizzle(row);  // the same for row + 4
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint8_t* p = &sh.d[st][256 * row + 32 * ((4 * wo + c) ^ sw) + 8 * (r & 3)];
      const u32x2 lo = read_tr16(p), hi = read_tr16(p + 4 * 256);
      bv[j][c] = (u32x4){lo.x, lo.y, hi.x, hi.y};
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint8_t* p = &sh.x[st][512 * row + 32 * ((4 * wi + c) ^ sw) + 8 * (r & 3)];
      const u32x2 lo = read_tr16(p), hi = read_tr16(p + 4 * 512);
      av[j][c] = (u32x4){lo.x, lo.y, hi.x, hi.y};
    }
  };
  auto multiply = [&](int j, int st, int k) {  // with the loads of step k, if k >= 0
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (k >= 0) {
        __builtin_amdgcn_sched_barrier(0);
        if (c < 3) load(c, st, k);
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) acc[c][t] = mfma_bf16(av[j][c], bv[j][t], acc[c][t]);
    }
  };
#pragma unroll
  for (int k = 0; k < 3; ++k)
#pragma unroll
    for (int n = 0; n < 3; ++n) load(n, k, k);
  wait_vmcnt<2 * LOADS>();
  bare_barrier();
  read(0, 0);
  auto step = [&](int st, int k) {  // as in dx_tile
    read(st, 1);
    multiply(0, 0, -1);
    __builtin_amdgcn_sched_barrier(0);
    wait_vmcnt<LOADS>();
    bare_barrier();
    read((st + 1) % 3, 0);
    multiply(1, st, k + 3);
  };
  for (int k = 0; k < nsteps; k += 3) {
    step(0, k);
    if (k + 1 < nsteps) step(1, k + 1);
    if (k + 2 < nsteps) step(2, k + 2);
  }
  wait_vmcnt<0>();
  __syncthreads();
  store_tile(sh.x[0] + 4096 * w, acc, reinterpret_cast<uint8_t*>(a.dw + (int64_t)(o0 + 64 * wo) * a.in + i0 + 64 * wi),
             (int64_t)a.in * 2, a.out - o0 - 64 * wo, (a.in - i0 - 64 * wi) * 2);
}

__global__ __launch_bounds__(512) void fp8b128_dw_kernel(Fp8b128BackwardArgs a, int to, int ti) {
  __shared__ DwShared sh;
  int o, i;
  if (fb_tile_of(to, ti, blockIdx.x >> 3, &o, &i)) dw_tile(a, sh, o, i);
}

}  // namespace

hipError_t launch_fp8b128_dx(const Fp8b128BackwardArgs& a, hipStream_t s) {
  // strips spread few tokens wider; tiles move less data once they fill half the GPU
  const int64_t tiles = (a.T + 127) / 128 * ((a.in + 255) / 256);
  if (tiles >= 128) {
    const int tt = (int)((a.T + 127) / 128), ti = (a.in + 255) / 256;
    hipLaunchKernelGGL(fp8b128_dx_kernel, dim3((unsigned)std::min((tt * ti + 7) & ~7, FB_CUS)), dim3(512), 0,
                       s, a, tt, ti);
    return hipGetLastError();
  }
  const int tt = a.T <= 16 ? 1 : 2;
  const unsigned grid = (unsigned)((a.in + 31) / 32 * ((a.T + 16 * tt - 1) / (16 * tt)));
  if (tt == 1)
    hipLaunchKernelGGL(fp8b128_dx_strip_kernel<1>, dim3(grid), dim3(DS_THREADS), 0, s, a);
  else
    hipLaunchKernelGGL(fp8b128_dx_strip_kernel<2>, dim3(grid), dim3(DS_THREADS), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_fp8b128_dw(const Fp8b128BackwardArgs& a, hipStream_t s) {
  const int64_t n16 = a.T * (a.in / 16);
  hipLaunchKernelGGL(fp8b128_widen_kernel, dim3((unsigned)((n16 + 255) / 256)), dim3(256), 0, s, a.x,
                     a.xs, n16, a.in, a.nb, reinterpret_cast<u32x4*>(a.xw));
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  const int to = (a.out + 127) / 128, ti = (a.in + 255) / 256;
  hipLaunchKernelGGL(fp8b128_dw_kernel, dim3((unsigned)((to * ti + 7) & ~7)), dim3(512), 0, s, a, to, ti);
  return hipGetLastError();
}

}  // namespace tq

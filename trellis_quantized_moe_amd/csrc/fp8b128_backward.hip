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
#include <type_traits>

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

// ---- dx, few tokens: strips of inputs, the outputs split over a workgroup's waves ------------
//
// A workgroup owns NS strips of 16 inputs (64 bytes of a row of codes) of up to 16 * TT tokens. Its
// W waves take the blocks of 128 outputs in turn, in two steps of 64, each through LDS of its own
// (no barrier until the end): a step goes from there to registers at once, and the next one's loads
// are issued between its products. A block's products are added from zero and then scaled into the
// sums; the waves' sums are added in wave order. All workgroups together read 11 to 13 TB/s from
// L2, a third of what loads alone reach, as a wave's loads, LDS reads and products follow one
// another: 333 tokens x 768 inputs x 5,120 outputs take 12.6 us. 32 x 5,120 x 4,096 take 10.5 us;
// with neighbouring strips on different XCDs, each reading the lines they share, it was 17.3. The
// kernel that strips share with dw leaves one workgroup to a compute unit; in a kernel of their own
// with 84 to 226 registers and 48 to 128 KiB of LDS, of which two of the smaller fit, they took as
// long (63 calls of 1 to 768 tokens: 0.7 % more on average, within 3 %).
template <int NS, int TT>
struct DxStrip {
  static constexpr int IW = 16 * NS, W = 8;
  static constexpr int LOADS = NS + 2 * TT;  // per step, of 1024 bytes
  union {
    struct {
      alignas(16) uint8_t w[64 * IW];
      alignas(16) uint8_t d[16 * TT * 128];
    } stage[W];
    f32x4 red[W][TT * NS][64];
  };
};

// Workgroup `wg` of `groups`.
template <int NS, int TT>
__device__ void dx_strip(const Fp8b128BackwardArgs& a, DxStrip<NS, TT>& sh, int wg, int groups) {
  using S = DxStrip<NS, TT>;
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // an XCD (workgroup b belongs to b % 8) has all tokens of consecutive strips: they read the same
  // codes, and neighbouring strips the same lines of them
  const int tiles = (int)((a.T + 16 * TT - 1) / (16 * TT)), x = wg & 7;
  const int g = x * (groups >> 3) + min(x, groups & 7) + (wg >> 3);
  const int i0 = g / tiles * S::IW;
  const int64_t t0 = (int64_t)(g % tiles) * (16 * TT);
  const int rows = (int)min((int64_t)(16 * TT), a.T - t0);
  const int nob = (a.out + 127) / 128;
  const GemmRsrc rd = gemm_rsrc(a.dy + t0 * a.out, (uint32_t)rows * (uint32_t)a.out * 2u);
  const float* ws = a.ws + i0 / 128;
  // codes: an instruction fills 64 / NS rows; lane l position l % NS of row l / NS, which holds the
  // row's 16-byte chunk (l % NS) ^ swizzle(row): the LDS serves 32 lanes at a time, which read one
  // chunk of 16 rows, and those get 16 different sixteenths of the 256 bytes that it serves
  auto swizzle = [&](int row) { return row / (16 / NS) & (NS - 1); };
  uint32_t wo[NS], dof[2 * TT];
#pragma unroll
  for (int j = 0; j < NS; ++j) {
    const int row = j * (64 / NS) + lane / NS, col = i0 + 16 * ((lane & (NS - 1)) ^ swizzle(row));
    wo[j] = col < a.in ? (uint32_t)row * (uint32_t)a.in + col : FB_OOB;
  }
  // dy: 8 rows; position l % 8 of row l / 8 holds chunk (l % 8) ^ (row % 8)
  const int dcol = 8 * ((lane & 7) ^ (lane >> 3));  // this lane's first output of a step
#pragma unroll
  for (int j = 0; j < 2 * TT; ++j) {
    const int tok = 8 * j + (lane >> 3);
    dof[j] = tok < rows ? ((uint32_t)tok * (uint32_t)a.out + dcol) * 2u : FB_OOB;
  }
  // Loads first .. last - 1 of a step's S::LOADS, the outputs 64 k ..; past the last they are zeros.
  auto load = [&](int first, int last, int k) {
    auto& st = sh.stage[w];
    const int left = min(64, a.out - 64 * k);
    const GemmRsrc rw = gemm_rsrc(a.w + (int64_t)(left > 0 ? 64 * k : 0) * a.in,
                                  left > 0 ? (uint32_t)left * (uint32_t)a.in : 0u);
#pragma unroll
    for (int j = first; j < last; ++j)
      if (j < NS)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (LdsPtr)(&st.w[1024 * j]), 16, wo[j], 0, 0, 0);
      else
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rd, (LdsPtr)(&st.d[1024 * (j - NS)]), 16,
                                                 dcol < left ? dof[j - NS] : FB_OOB, 128u * k, 0, 0);
  };
  // step n of this wave: half n % 2 of its block n / 2
  auto outputs = [&](int n) { return 2 * (w + S::W * (n >> 1)) + (n & 1); };

  f32x4 acc[TT][NS], p[TT][NS];
#pragma unroll
  for (int t = 0; t < TT; ++t)
#pragma unroll
    for (int c = 0; c < NS; ++c) acc[t][c] = p[t][c] = (f32x4){0.f, 0.f, 0.f, 0.f};
  const int steps = w < nob ? 2 * ((nob - w + S::W - 1) / S::W) : 0;
  if (steps > 0) load(0, S::LOADS, outputs(0));
  // A step: into registers, then its products, with the next step's loads between them.
  auto step = [&](int n, bool second) {
    float s = 0.0f;
    if (second) s = fb_uniform_load(ws + (int64_t)(w + S::W * (n >> 1)) * a.nb);
    wait_vmcnt<0>();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    const auto& st = sh.stage[w];
    u32x4 b[2][TT];
    u32x2 v[2][NS];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int t = 0; t < TT; ++t)
        b[j][t] = *reinterpret_cast<const u32x4*>(&st.d[128 * (16 * t + r) + 16 * ((4 * j + q) ^ (r & 7))]);
#pragma unroll
      for (int c = 0; c < NS; ++c) {
        const int row = 32 * j + 8 * q + (r >> 1);
        v[j][c] = read_tr8(&st.w[S::IW * row + 16 * (c ^ swizzle(row)) + 8 * (r & 1)]);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): no read of the stage is outstanding
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (n + 1 < steps) {
        load(j * S::LOADS / 2, (j + 1) * S::LOADS / 2, outputs(n + 1));
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int c = 0; c < NS; ++c) {
        const u32x4 av = fb_bf16_of8(v[j][c].x, v[j][c].y);
#pragma unroll
        for (int t = 0; t < TT; ++t) p[t][c] = mfma_bf16(av, b[j][t], p[t][c]);
      }
    }
    if (second) {
#pragma unroll
      for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int c = 0; c < NS; ++c) {
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[t][c][i] = __builtin_fmaf(p[t][c][i], s, acc[t][c][i]);
          p[t][c] = (f32x4){0.f, 0.f, 0.f, 0.f};
        }
    }
  };
  for (int n = 0; n < steps; n += 2) {
    step(n, false);
    step(n + 1, true);
  }
  __syncthreads();  // no load of this workgroup is writing its LDS, and no wave reads a stage
#pragma unroll
  for (int t = 0; t < TT; ++t)
#pragma unroll
    for (int c = 0; c < NS; ++c) sh.red[w][NS * t + c][lane] = acc[t][c];
  __syncthreads();
  for (int v = w; v < NS * TT; v += S::W) {  // the tiles of results, one after the other
    f32x4 sum = sh.red[0][v][lane];
#pragma unroll
    for (int u = 1; u < S::W; ++u) sum += sh.red[u][v][lane];
    const int row = 16 * (v / NS) + r, i = i0 + 16 * (v % NS) + 4 * q;
    if (row < rows && i < a.in) store4(a.dx + (t0 + row) * a.in + i, sum);
  }
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <int NS, int TT>
int64_t dx_strip_groups(const Fp8b128BackwardArgs& a) {  // workgroups
  return ceil_div(a.in, 16 * NS) * ceil_div(a.T, 16 * TT);
}

// The 16 NT x 64 results of each wave of a tile (row 16 t + lane % 16, inputs 16 c + 4 (lane / 16)
// .. + 3 in acc[c][t]) to its rows at dst, of which `rows` exist and `bytes` of each, by whole rows
// through 4096 bytes of LDS of the wave's own.
template <int NT>
__device__ __forceinline__ void store_tile(uint8_t* lds, const f32x4 (&acc)[4][NT], uint8_t* dst,
                                           int64_t stride, int rows, int bytes) {
  const int lane = fb_fresh_lane(), r = lane & 15, q = lane >> 4;
  FbRows<128, 32> out{lds};
#pragma unroll
  for (int hf = 0; hf < NT / 2; ++hf) {
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
// A workgroup of eight waves owns 256 inputs of 128 tokens (half an item: of 64), wave (wi, wt) 64
// inputs of 64 (32) tokens. Per block of 128 outputs, 128 rows of 256 code bytes and 128 rows of
// 256 bytes of dy go straight to one of two LDS stages. A wave takes the block strip by strip of 16
// inputs: the strip's codes become bf16 once, its products with the block's dy (in registers for
// all strips) are added from zero, and the strip before it is scaled into its sums meanwhile.
// 8,192 tokens x 5,120 inputs x 1,536 outputs take 119 to 130 us (1.0 to 1.08 PFLOP/s), the matrix
// cores busy 56 % of the cycles at 1.88 GHz; in steps of 64 outputs, with the sums of a whole block
// waiting to be scaled at once, it was 136 us and 48 %.
struct DxShared {
  alignas(16) uint8_t w[2][128 * 256];
  alignas(16) uint8_t d[2][128 * 256];
};

// One workgroup per compute unit takes tile after tile: the first block of the next tile is
// loading while a tile's results are stored.
struct DxTile {
  int64_t t0;
  int rows, i0, ib;
  uint32_t wo[4], dof[4];
};

// The tile, or one half of its tokens.
__device__ __forceinline__ DxTile dx_tile_at(const Fp8b128BackwardArgs& a, int tile_t, int tile_i,
                                             int half, int w) {
  const int lane = fb_fresh_lane();
  DxTile d;
  d.t0 = (int64_t)tile_t * 128 + (half > 0 ? 64 : 0);
  d.rows = (int)max(min((int64_t)(half < 0 ? 128 : 64), a.T - d.t0), (int64_t)0);
  d.i0 = tile_i * 256;
  d.ib = min((d.i0 + 64 * (w & 3)) / 128, a.nb - 1);
  // an instruction fills 4 rows; lane l position l % 16 of row l / 16, which holds the row's
  // 16-byte chunk (l % 16) ^ (row % 16)
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int row = 16 * w + 4 * j + (lane >> 4), chunk = (lane & 15) ^ (row & 15);
    d.wo[j] = d.i0 + 16 * chunk < a.in ? (uint32_t)row * (uint32_t)a.in + d.i0 + 16 * chunk : FB_OOB;
    d.dof[j] = row < d.rows ? (uint32_t)row * (uint32_t)a.out * 2u + 16u * chunk : FB_OOB;
  }
  return d;
}

__device__ void dx_tiles(const Fp8b128BackwardArgs& a, DxShared& sh, const FbItems& items) {
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wi = w & 3, wt = w >> 2;
  const int nob = (a.out + 127) / 128;
  const int dcol = 8 * ((lane & 15) ^ (lane >> 4));  // of part 0; of part n it is dcol ^ 32 n
  constexpr int LOADS = 8, PER = 4;  // of one block; issued at a time
  DxTile d;
  // A block's loads, in parts (a wave cannot go on while the memory unit's queue is full, so
  // they are issued between the products); blocks past the last are read as zeros.
  auto load = [&](int n, int st, int k) {
    const int left = min(128, a.out - 128 * k);
    if (n < 4) {
      const GemmRsrc rw = gemm_rsrc(a.w + (int64_t)(left > 0 ? 128 * k : 0) * a.in,
                                    left > 0 ? (uint32_t)left * (uint32_t)a.in : 0u);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (LdsPtr)(&sh.w[st][256 * (16 * w + 4 * n)]), 16,
                                               d.wo[n], 0, 0, 0);
    } else {
      const GemmRsrc rd = gemm_rsrc(a.dy + d.t0 * a.out, (uint32_t)d.rows * (uint32_t)a.out * 2u);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rd, (LdsPtr)(&sh.d[st][256 * (16 * w + 4 * (n - 4))]), 16,
                                               (dcol ^ (32 * (n - 4))) < left ? d.dof[n - 4] : FB_OOB,
                                               256u * k, 0, 0);
    }
  };

  int tile_t, tile_i, half, j = blockIdx.x >> 3;
  const int stream = blockIdx.x & 7;
  if (!items.at(stream, j, &tile_t, &tile_i, &half)) return;
  d = dx_tile_at(a, tile_t, tile_i, half, w);
#pragma unroll
  for (int n = 0; n < LOADS; ++n) load(n, 0, 0);
  // One item, whole (NT = 4 token tiles of 16 per wave) or half (NT = 2): its first block is
  // loading; afterwards that of the next item is. Returns whether there is one.
  auto item = [&](auto tiles) {
    constexpr int NT = decltype(tiles)::value;
    f32x4 acc[4][NT], p[NT];
    u32x2 av[2][4];   // of a strip: the codes of 32 outputs each
    u32x4 bv[NT][4];  // dy of the block
    auto read_a = [&](int st, int c) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int row = 32 * j + 8 * q + (r >> 1);
        av[c & 1][j] = read_tr8(&sh.w[st][256 * row + 16 * ((4 * wi + c) ^ (row & 15)) + 8 * (r & 1)]);
      }
    };
    auto read_b = [&](int st, int t) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        bv[t][j] = *reinterpret_cast<const u32x4*>(
            &sh.d[st][256 * (16 * NT * wt + 16 * t + r) + 16 * ((4 * j + q) ^ r)]);
    };
    auto add = [&](int c, int t, float s) {
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[c][t][i] = __builtin_fmaf(p[t][i], s, acc[c][t][i]);
      asm volatile("" : "+v"(acc[c][t]));  // done here, not where the compiler would gather them
    };
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[c][t] = (f32x4){0.f, 0.f, 0.f, 0.f};
      p[t] = (f32x4){0.f, 0.f, 0.f, 0.f};
    }
#pragma unroll
    for (int n = 0; n < PER; ++n) load(n, 1, 1);
    wait_vmcnt<PER>();
    bare_barrier();
    read_a(0, 0);
#pragma unroll
    for (int t = 0; t < NT; ++t) read_b(0, t);
    float s = fb_uniform_load(a.ws + d.ib), before = 0.0f;
    // One block. Before its last strip, whose operands are in registers, the next block has
    // landed everywhere and this stage is no longer read: its refill starts, and the next block's
    // operands are read as the last strip's products release the registers.
    int st = 0;
    for (int kb = 0; kb < nob; ++kb) {
      float next_s = 0.0f;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const bool last = c == 3;
        __builtin_amdgcn_sched_barrier(0);
        if (last) {
          wait_vmcnt<0>();
          bare_barrier();
          read_a(st ^ 1, 0);
          next_s = fb_uniform_load(a.ws + (int64_t)min(kb + 1, nob - 1) * a.nb + d.ib);
        } else {
          read_a(st, c + 1);
        }
        if (c == 0)
#pragma unroll
          for (int n = PER; n < LOADS; ++n) load(n, st ^ 1, kb + 1);
        if (last)
#pragma unroll
          for (int n = 0; n < PER; ++n) load(n, st, kb + 2);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const u32x4 a8 = fb_bf16_of8(av[c & 1][j].x, av[c & 1][j].y);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            if (j == 0) add((c + 3) % 4, t, c == 0 ? before : s);
            p[t] = mfma_bf16(a8, bv[t][j], j == 0 ? (f32x4){0.f, 0.f, 0.f, 0.f} : p[t]);
            if (last && j == 3) {
              __builtin_amdgcn_sched_barrier(0);
              read_b(st ^ 1, t);
            }
          }
        }
      }
      before = s;
      s = next_s;
      st ^= 1;
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) add(3, t, before);
    // the loads past the last block have landed, and no wave reads a stage any more
    wait_vmcnt<0>();
    bare_barrier();
    uint8_t* dst = reinterpret_cast<uint8_t*>(a.dx + (d.t0 + 16 * NT * wt) * a.in + d.i0 + 64 * wi);
    const int rows = d.rows - 16 * NT * wt, bytes = (a.in - d.i0 - 64 * wi) * 2;
    j += gridDim.x >> 3;
    const bool more = items.at(stream, j, &tile_t, &tile_i, &half);
    if (more) {
      d = dx_tile_at(a, tile_t, tile_i, half, w);
#pragma unroll
      for (int n = 0; n < LOADS; ++n) load(n, 0, 0);
    }
    // through the second stage, which the next item fills after the barrier
    store_tile(sh.w[1] + 4096 * w, acc, dst, (int64_t)a.in * 2, rows, bytes);
    bare_barrier();
    return more;
  };
  while (half < 0)  // halves come last, one to a workgroup
    if (!item(std::integral_constant<int, 4>())) {
      wait_vmcnt<0>();
      return;
    }
  item(std::integral_constant<int, 2>());
  wait_vmcnt<0>();
}

__global__ __launch_bounds__(512) void fp8b128_dx_kernel(Fp8b128BackwardArgs a, FbItems items) {
  __shared__ DxShared sh;
  dx_tiles(a, sh, items);
}

// ---- dw, many tokens ------------------------------------------------------------------------
//
// X as bf16 [T][in] (exact for scales that are powers of two), once per call: every channel
// tile of the product reads it. Bound by memory: 8,192 x 5,120 take 25 us. Widening in the product
// instead, on the way from registers to LDS, took the product from 112 to 162 us at 1,536 outputs.
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
  fb_widen(c, s, out);
  y[2 * k] = out[0];
  y[2 * k + 1] = out[1];
}

// A workgroup of eight waves owns 256 inputs of 128 channels (half an item: of 64), wave (wi, wo)
// 64 inputs of 64 (32) channels; steps of 64 tokens through a ring of three LDS stages, two steps
// ahead. A row's 32-byte chunk c lies at position c ^ swizzle(row): the LDS serves 32 lanes at a
// time, which read one chunk of rows 8 q + 0..3 and 8 (q + 1) + 0..3 (or + 4..7), and those eight
// rows get eight different positions. 8,192 tokens x 5,120 inputs x 1,536 channels take 112 to 122
// us (1.06 to 1.15 PFLOP/s), the matrix cores busy 61 % of the cycles at 1.75 GHz.
__device__ __forceinline__ int dw_swizzle(int row) { return (row & 3) | (row >> 1 & 4); }

struct DwShared {
  alignas(16) uint8_t x[3][64 * 512];
  alignas(16) uint8_t d[3][64 * 256];
};

// NT tiles of 16 channels per wave: 4, or 2 in half an item, the channels o0 .. o0 + 32 NT - 1.
template <int NT>
__device__ void dw_tile(const Fp8b128BackwardArgs& a, DwShared& sh, int o0, int i0) {
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wi = w & 3, wo = w >> 2;
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
    dof[j] = o < min(a.out, o0 + 32 * NT) ? ((uint32_t)row * (uint32_t)a.out + o) * 2u : FB_OOB;
  }
  constexpr int LOADS = 6;
  // A step's loads, in three parts, issued between the products; rows past the last token are read
  // as zeros.
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
  f32x4 acc[4][NT];
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[c][t] = (f32x4){0.f, 0.f, 0.f, 0.f};
  // operands of 32 tokens (half j of a step). Lane (r, q) of half h: row 32 j + 8 q + 4 h + r / 4,
  // quarter r % 4 of a 32-byte chunk
  u32x4 av[2][4], bv[2][NT];
  auto read = [&](int st, int j) {
    const int row = 32 * j + 8 * q + (r >> 2), sw = dw_swizzle(row);  // the same for row + 4
#pragma unroll
    for (int c = 0; c < NT; ++c) {
      const uint8_t* p = &sh.d[st][256 * row + 32 * ((NT * wo + c) ^ sw) + 8 * (r & 3)];
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
      for (int t = 0; t < NT; ++t) acc[c][t] = mfma_bf16(av[j][c], bv[j][t], acc[c][t]);
    }
  };
#pragma unroll
  for (int k = 0; k < 3; ++k)
#pragma unroll
    for (int n = 0; n < 3; ++n) load(n, k, k);
  wait_vmcnt<2 * LOADS>();
  bare_barrier();
  read(0, 0);
  // A step's second half is read while its first half is multiplied, and the next step's first
  // half while its second is: between the two, the next step's data have landed everywhere, and
  // this step's stage is no longer read.
  auto step = [&](int st, int k) {
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
  store_tile(sh.x[0] + 4096 * w, acc,
             reinterpret_cast<uint8_t*>(a.dw + (int64_t)(o0 + 16 * NT * wo) * a.in + i0 + 64 * wi),
             (int64_t)a.in * 2, a.out - o0 - 16 * NT * wo, (a.in - i0 - 64 * wi) * 2);
}

__global__ __launch_bounds__(512) void fp8b128_dw_kernel(Fp8b128BackwardArgs a, FbItems items) {
  __shared__ DwShared sh;
  int o, i, half;
  if (!items.at(blockIdx.x & 7, blockIdx.x >> 3, &o, &i, &half)) return;
  if (half < 0)
    dw_tile<4>(a, sh, 128 * o, 256 * i);
  else
    dw_tile<2>(a, sh, 128 * o + 64 * half, 256 * i);
}

// ---- dw, few tokens or few tiles ------------------------------------------------------------
//
// A workgroup of four waves owns 128 inputs of 128 channels and one of `splits` ranges of the
// tokens, wave (wi, wo) 64 inputs of 64 channels. X is widened on its way from registers to LDS, so
// that there is no launch before this one; the next step's loads are in flight while a step's
// products are made, and other waves on the compute unit fill the waits. With several ranges the
// sums go to the workspace in fp32, and a second launch adds them in order. 64 tokens x 5,120
// inputs x 1,536 channels take 8.4 us (X widened first: 10.9), bound by the 15.7 MB of results.
struct DwRange {
  alignas(16) uint8_t x[2][64 * 256];
  alignas(16) uint8_t d[2][64 * 256];
};

// The four waves' item `n`: a tile and a range. Items past the last, and steps past a range's last,
// are zeros, so that all waves of a workgroup meet at the same barriers.
__device__ void dw_range(const Fp8b128BackwardArgs& a, DwRange& sh, int n) {
  const int tid = threadIdx.x & 255, lane = tid & 63, r = lane & 15, q = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wi = w & 1, wo = w >> 1;
  const int ti = (a.in + 127) / 128, to = (a.out + 127) / 128;
  const int tile = n % (ti * to), split = n / (ti * to);
  const int i0 = tile % ti * 128, o0 = tile / ti * 128;
  const int nsteps = (int)((a.T + 63) / 64);
  const int per = (nsteps + a.splits - 1) / a.splits, first = split * per;
  const int last = split < a.splits ? min(first + per, nsteps) : 0;
  // this thread's 16-byte pieces of a step: two of the codes (32 bytes of bf16, a chunk of the
  // LDS row), four of dy
  const int xrow = tid >> 3, xcol = i0 + 16 * (tid & 7);
  const int drow = tid >> 4, dcol = o0 + 8 * (tid & 15);
  u32x4 cx[2], cd[4];
  float cs[2];
  auto load = [&](int k) {
    const int64_t t = (int64_t)64 * k;
    const int left = k < last ? (int)min((int64_t)64, a.T - t) : 0;
    const int64_t at = left > 0 ? t : 0;
    const GemmRsrc rx = gemm_rsrc(a.x + at * a.in, (uint32_t)left * (uint32_t)a.in);
    const GemmRsrc rs = gemm_rsrc(a.xs + at * a.nb, (uint32_t)(left * a.nb) * 4u);
    const GemmRsrc rd = gemm_rsrc(a.dy + at * a.out, (uint32_t)left * (uint32_t)a.out * 2u);
#pragma unroll
    for (int j = 0; j < 2; ++j) {  // outside the resource: zeros
      const int row = xrow + 32 * j;
      cx[j] = __builtin_amdgcn_raw_buffer_load_b128(
          rx, xcol < a.in ? (uint32_t)row * (uint32_t)a.in + xcol : FB_OOB, 0, 0);
      cs[j] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
          rs, xcol < a.in ? (uint32_t)(row * a.nb + i0 / 128) * 4u : FB_OOB, 0, 0));
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      cd[j] = __builtin_amdgcn_raw_buffer_load_b128(
          rd, dcol < a.out ? ((uint32_t)(drow + 16 * j) * (uint32_t)a.out + dcol) * 2u : FB_OOB, 0, 0);
  };
  auto store = [&](int st) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int row = xrow + 32 * j;
      u32x4 v[2];
      fb_widen(cx[j], cs[j], v);
      u32x4* p = reinterpret_cast<u32x4*>(&sh.x[st][256 * row + 32 * ((tid & 7) ^ dw_swizzle(row))]);
      p[0] = v[0];
      p[1] = v[1];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row = drow + 16 * j, c = tid & 15;
      *reinterpret_cast<u32x4*>(
          &sh.d[st][256 * row + 32 * ((c >> 1) ^ dw_swizzle(row)) + 16 * (c & 1)]) = cd[j];
    }
  };
  f32x4 acc[4][4];
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int t = 0; t < 4; ++t) acc[c][t] = (f32x4){0.f, 0.f, 0.f, 0.f};
  auto multiply = [&](int st) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {  // 32 tokens, operands as in dw_tile
      const int row = 32 * j + 8 * q + (r >> 2), sw = dw_swizzle(row);
      auto read = [&](const uint8_t* l, int chunk) {
        const uint8_t* p = l + 256 * row + 32 * (chunk ^ sw) + 8 * (r & 3);
        const u32x2 lo = read_tr16(p), hi = read_tr16(p + 4 * 256);
        return (u32x4){lo.x, lo.y, hi.x, hi.y};
      };
      u32x4 bv[4];
#pragma unroll
      for (int t = 0; t < 4; ++t) bv[t] = read(sh.d[st], 4 * wo + t);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const u32x4 av = read(sh.x[st], 4 * wi + c);
#pragma unroll
        for (int t = 0; t < 4; ++t) acc[c][t] = mfma_bf16(av, bv[t], acc[c][t]);
      }
    }
  };
  load(first);
  for (int k = 0; k < per; k += 2) {
#pragma unroll
    for (int st = 0; st < 2; ++st)
      if (k + st < per) {
        store(st);  // the readers of two steps ago have passed the last step's barrier
        load(first + k + st + 1);
        __syncthreads();
        multiply(st);
      }
  }
  __syncthreads();
  const int o = o0 + 64 * wo, i = i0 + 64 * wi;
  if (split >= a.splits) return;
  if (a.splits == 1) {
    store_tile((w < 2 ? sh.x[0] : sh.d[0]) + 4096 * (w & 1), acc,
               reinterpret_cast<uint8_t*>(a.dw + (int64_t)o * a.in + i), (int64_t)a.in * 2, a.out - o, (a.in - i) * 2);
    return;
  }
  float* part = a.part + (int64_t)split * a.out * a.in;
#pragma unroll
  for (int t = 0; t < 4; ++t)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int row = o + 16 * t + r, col = i + 16 * c + 4 * q;
      if (row < a.out && col < a.in) *reinterpret_cast<f32x4*>(part + (int64_t)row * a.in + col) = acc[c][t];
    }
}

__global__ __launch_bounds__(256, 2) void fp8b128_dw_range_kernel(Fp8b128BackwardArgs a) {
  __shared__ DwRange sh;
  dw_range(a, sh, blockIdx.x);
}

// ---- dx of few tokens, with dw -------------------------------------------------------------
//
// The first `dx_groups` workgroups are dx strips, the others (where dw is made of ranges and both
// gradients are wanted) dw ranges: neither fills the compute units for long, and neither needs the
// other. Four waves take an item of dw; a workgroup has two, or one (and four waves that end at
// once) where that still leaves every workgroup a compute unit.
template <int NS, int TT>
union DxDwShared {
  DxStrip<NS, TT> dx;
  DwRange dw[2];
};

template <int NS, int TT>
__device__ void dx_dw(const Fp8b128BackwardArgs& a, DxDwShared<NS, TT>& sh, int dx_groups, int items) {
  const int wg = blockIdx.x;
  if (wg < dx_groups) {
    dx_strip<NS, TT>(a, sh.dx, wg, dx_groups);
  } else {
    const int part = __builtin_amdgcn_readfirstlane(threadIdx.x >> 8);
    if (part < items) dw_range(a, sh.dw[part], items * (wg - dx_groups) + part);
  }
}

template <int NS, int TT>
__global__ __launch_bounds__((64 * DxStrip<NS, TT>::W)) void fp8b128_dx_dw_kernel(Fp8b128BackwardArgs a,
                                                                                 int dx_groups, int items) {
  __shared__ DxDwShared<NS, TT> sh;
  dx_dw<NS, TT>(a, sh, dx_groups, items);
}

// The sums of the ranges, one after the other, as bf16: four results a thread.
__global__ __launch_bounds__(256) void fp8b128_dw_join_kernel(const f32x4* __restrict__ part, int64_t n4,
                                                              int splits, uint16_t* __restrict__ dw) {
  const int64_t k = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (k >= n4) return;
  f32x4 sum = part[k];
#pragma unroll 4
  for (int s = 1; s < splits; ++s) sum += part[s * n4 + k];
  store4(dw + 4 * k, sum);
}

// Ranges of tokens of the dw of few tiles: as many workgroups as two on every compute unit, of one
// step of 64 tokens at least.
int dw_most_splits(int64_t T, int out, int in) {
  const int64_t tiles = ceil_div(out, 128) * ceil_div(in, 128);
  return (int)std::max((int64_t)1, std::min(ceil_div(T, 64), 2 * FB_CUS / tiles));
}

// Expected time of a launch that adds k ranges (0.01 us).
int64_t join_cost(int64_t k, int64_t results) { return 300 + k * (15 + results * 8 / 50000); }

// How dw is computed: X widened first (0), or the number of ranges; whichever has the least time
// expected (0.01 us):
//   widened  500, the widening of 3 bytes an input at 5 TB/s, and for each round of tiles over the
//            compute units 450 + 87 a step of 64 tokens, for a round of halves 200 + 51 a step
//   ranges   400, for each round of two workgroups on every compute unit 230 + 133 a step, of one
//            80 + 90; with several ranges 300 and for each 15 and 8 bytes a result at 5 TB/s
// Measured, widened / one range / the best number of ranges: 64 tokens x 5,120 x 1,536 10.9 / 8.4
// us, x 5,120 x 4,096 20.2 / 15.0; 512 x 5,120 x 4,096 39.1 / 39.2; 2,048 x 5,120 x 1,536 45.8 /
// 50.5; 2,048 x 768 x 768 26.2 / 33.6 / 19.9 (4); 8,192 x 256 x 64 71 / 117 / 13.5 (16), x 768 x
// 768 74.7 / 119 / 31.0 (14), x 768 x 5,120 92.1 / 129 / 109 (2).
struct Plan {
  int kind;      // of dx: a DxKind; of dw: the number of ranges, or 0
  int64_t cost;  // 0.01 us
};
Plan dw_plan(const Fp8b128BackwardArgs& a) {
  const FbItems items((a.out + 127) / 128, (a.in + 255) / 256);
  const int64_t steps = ceil_div(a.T, 64), results = (int64_t)a.out * a.in;
  const int64_t tiles = ceil_div(a.out, 128) * ceil_div(a.in, 128);
  const int most = dw_most_splits(a.T, a.out, a.in);
  int64_t least = 500 + a.T * a.in * 3 / 50000 + ceil_div(items.full, FB_CUS / 8) * (450 + 87 * steps) +
                  (items.items > items.full ? 200 + 51 * steps : 0);
  int best = 0;
  for (int s = 1; s <= most; s += std::max(1, s / 2)) {
    const int64_t n = ceil_div(steps, s), k = ceil_div(steps, n);  // steps of a range, ranges with any
    const int64_t two = 230 + 133 * n, rest = tiles * k % (2 * FB_CUS);
    const int64_t cost = 400 + tiles * k / (2 * FB_CUS) * two +
                         (rest > FB_CUS ? two : rest > 0 ? 80 + 90 * n : 0) +
                         (k > 1 ? join_cost(k, results) : 0);
    if (cost < least) {
      least = cost;
      best = (int)k;
    }
  }
  return {best, least};
}

FbItems dx_items(const Fp8b128BackwardArgs& a) {
  return FbItems((int)ceil_div(a.T, 128), (int)ceil_div(a.in, 256));
}

// The kernel of dx with the least time expected, beside the 2 us that all have in common (0.01 us),
// by the rounds of workgroups over the compute units and the blocks of 128 outputs (strips: of a
// wave, an eighth of all): strips of (4, 1) 96 a round and 159 a block of it, (4, 2) 86 and 205,
// (4, 4) 103 and 314, tiles 260 and 168, of a round of halves 103. The constants are a fit to calls
// of 16 to 1,024 tokens; a choice by them took 0.4 % more than the fastest on average. Measured,
// (4, 1) / (4, 2) / (4, 4) / tiles: 32 tokens x 5,120 inputs x 4,096 outputs 10.5 / 11.7 / 14.3 / 36
// us; 201 x 1,200 x 2,640 9.7 / 9.2 / 11.1 / 23.7; 333 x 5,120 x 1,536 27.0 / 20.2 / 15.8 / 17.5;
// 768 x 2,576 x 1,440 35.4 / 24.7 / 18.9 / 17.9.
enum DxKind { DX_TILES = 0, DX_1 = 1, DX_2 = 2, DX_4 = 4 };
Plan dx_plan(const Fp8b128BackwardArgs& a) {
  const int64_t blocks = ceil_div(a.out, 128), wave_blocks = ceil_div(blocks, DxStrip<4, 1>::W);
  const int64_t s1 = ceil_div(dx_strip_groups<4, 1>(a), FB_CUS) * (96 + 159 * wave_blocks);
  const int64_t s2 = ceil_div(dx_strip_groups<4, 2>(a), FB_CUS) * (86 + 205 * wave_blocks);
  const int64_t s4 = ceil_div(dx_strip_groups<4, 4>(a), FB_CUS) * (103 + 314 * wave_blocks);
  const FbItems items = dx_items(a);
  const int64_t tiles = ceil_div(items.full, FB_CUS / 8) * (260 + 168 * blocks) +
                        (items.items > items.full ? 260 + 103 * blocks : 0);
  const int64_t least = std::min(std::min(s1, s2), std::min(s4, tiles));
  return {least == s1 ? DX_1 : least == s2 ? DX_2 : least == s4 ? DX_4 : DX_TILES, least};
}

int64_t dw_range_items(const Fp8b128BackwardArgs& a) {
  return ceil_div(a.out, 128) * ceil_div(a.in, 128) * a.splits;
}

// Items of dw of a workgroup in a launch with dx_groups of dx.
int items_together(const Fp8b128BackwardArgs& a, int64_t dx_groups) {
  return dx_groups + dw_range_items(a) <= FB_CUS ? 1 : 2;
}

hipError_t launch_dw_join(const Fp8b128BackwardArgs& a, hipStream_t s) {
  const int64_t n4 = (int64_t)a.out * a.in / 4;
  hipLaunchKernelGGL(fp8b128_dw_join_kernel, dim3((unsigned)ceil_div(n4, 256)), dim3(256), 0, s,
                     reinterpret_cast<const f32x4*>(a.part), n4, a.splits, a.dw);
  return hipGetLastError();
}

hipError_t launch_dw(const Fp8b128BackwardArgs& a, hipStream_t s) {
  if (a.splits > 0) {
    hipLaunchKernelGGL(fp8b128_dw_range_kernel, dim3((unsigned)dw_range_items(a)), dim3(256), 0, s, a);
    hipError_t err = hipGetLastError();
    return err == hipSuccess && a.splits > 1 ? launch_dw_join(a, s) : err;
  }
  const int64_t n16 = a.T * (a.in / 16);
  hipLaunchKernelGGL(fp8b128_widen_kernel, dim3((unsigned)((n16 + 255) / 256)), dim3(256), 0, s, a.x,
                     a.xs, n16, a.in, a.nb, reinterpret_cast<u32x4*>(a.xw));
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  const FbItems items((a.out + 127) / 128, (a.in + 255) / 256);
  hipLaunchKernelGGL(fp8b128_dw_kernel, dim3((unsigned)(8 * items.items)), dim3(512), 0, s, a, items);
  return hipGetLastError();
}

// Expected time of dx strips and dw ranges in one launch (0.01 us). A strip's workgroup takes 170
// (TT = 1), 130 or 260 for each block of 128 outputs of a wave, or what it reads at its share of
// 11 TB/s from L2; a workgroup of two ranges 200 + 110 a step of 64 tokens, of one 30 + 70. Where
// all workgroups have a compute unit the longer of the two counts, else their sum over the compute
// units and a last round of the shorter. The constants are a fit to calls of 1 to 512 tokens and 64
// to 5,120 channels; a choice by them, with 250 for the second launch of two apart, took 2.2 % more
// than the fastest on average over 137 such calls, 28 % at most (333 x 4,000 x 800: 22.8 us by (4,
// 2), 17.9 by (4, 4)); with 110 it took 201 x 2,576 x 1,440 apart, 16.9 us, 15.4 by (4, 2), and 48
// x 5,120 x 4,096, 26.1 and 20.9. Measured, apart
// / (4, 1) / (4, 2) / (4, 4): 8 tokens x 768 inputs x 768 outputs 8.4 / 5.7 / 5.4 / 6.5 us, x 5,120
// x 4,096 29.2 / 20.1 / 19.9 / 22.8; 333 x 768 x 5,120 23.6 / 24.2 / 16.4 / 20.7, x 768 x 768 13.5
// / 15.6 / 10.1 / 10.1; 130 x 2,576 x 1,440 15.1 / 15.2 / 15.0 / 10.9; 512 x 5,120 x 1,536 35.2 /
// 59.1 / 45.7 / 39.5.
template <int NS, int TT>
int64_t together_cost(const Fp8b128BackwardArgs& a) {
  using S = DxStrip<NS, TT>;
  const int64_t blocks = ceil_div(a.out, 128), steps = ceil_div(ceil_div(a.T, 64), a.splits);
  const int64_t dx = dx_strip_groups<NS, TT>(a);
  const int items = items_together(a, dx);
  const int64_t dw = ceil_div(dw_range_items(a), items);
  const int64_t read = blocks * (8192 + 4096 * TT) * std::min((int64_t)FB_CUS, dx + dw) / 110000;
  const int64_t strip = std::max(ceil_div(blocks, S::W) * (TT == 1 ? 170 : TT == 2 ? 130 : 260), read);
  const int64_t range = items == 2 ? 200 + 110 * steps : 30 + 70 * steps;
  const int64_t sum = dx + dw <= FB_CUS ? 0 : (dx * strip + dw * range) / FB_CUS + std::min(strip, range);
  return 400 + std::max(sum, std::max(strip, range)) +
         (a.splits > 1 ? join_cost(a.splits, (int64_t)a.out * a.in) : 0);
}

// dx strips, and the ranges of dw if `with_dw`.
template <int NS, int TT>
hipError_t launch_strips(const Fp8b128BackwardArgs& a, bool with_dw, hipStream_t s) {
  const int64_t dx = dx_strip_groups<NS, TT>(a);
  const int items = with_dw ? items_together(a, dx) : 0;
  const int64_t dw = with_dw ? ceil_div(dw_range_items(a), items) : 0;
  hipLaunchKernelGGL((fp8b128_dx_dw_kernel<NS, TT>), dim3((unsigned)(dx + dw)),
                     dim3(64 * DxStrip<NS, TT>::W), 0, s, a, (int)dx, items);
  hipError_t err = hipGetLastError();
  return err == hipSuccess && with_dw && a.splits > 1 ? launch_dw_join(a, s) : err;
}

}  // namespace

size_t fp8b128_dw_part_bytes(int64_t T, int out, int in) {
  const int s = dw_most_splits(T, out, in);
  return s > 1 ? (size_t)s * out * in * 4 : 0;
}

hipError_t launch_fp8b128_backward(const Fp8b128BackwardArgs& args, hipStream_t s) {
  Fp8b128BackwardArgs a = args;
  const Plan dw = dw_plan(a), dx = dx_plan(a);
  a.splits = dw.kind;
  if (!a.dx) return launch_dw(a, s);
  int kind = dx.kind;
  bool with_dw = false;
  if (a.dw && a.splits > 0) {
    int64_t least = dx.cost + dw.cost + 250;
    auto offer = [&](int k, int64_t cost) {
      if (cost < least) {
        least = cost;
        kind = k;
        with_dw = true;
      }
    };
    offer(DX_1, together_cost<4, 1>(a));
    offer(DX_2, together_cost<4, 2>(a));
    offer(DX_4, together_cost<4, 4>(a));
  }
  hipError_t err;
  if (kind == DX_1) {
    err = launch_strips<4, 1>(a, with_dw, s);
  } else if (kind == DX_2) {
    err = launch_strips<4, 2>(a, with_dw, s);
  } else if (kind == DX_4) {
    err = launch_strips<4, 4>(a, with_dw, s);
  } else {
    const FbItems items = dx_items(a);
    hipLaunchKernelGGL(fp8b128_dx_kernel, dim3((unsigned)(8 * std::min(items.items, FB_CUS / 8))), dim3(512),
                       0, s, a, items);
    err = hipGetLastError();
  }
  return err == hipSuccess && a.dw && !with_dw ? launch_dw(a, s) : err;
}

}  // namespace tq

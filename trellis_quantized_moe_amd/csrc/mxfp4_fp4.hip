// The routed product of MXFP4 activations with MXFP4 experts on gfx950's fp4 matrix cores
// (FORMAT F30): both operands are their E2M1 codes with their E8M0 scales as stored, nothing is
// decoded.
//
// A work item is up to 128 (or 256) routed rows of one expert times a group of as many output
// channels over the whole input range, in steps of 128 inputs, on 4 (or 8) waves. The waves share
// out the rows and channels in blocks of 32: a step is two v_mfma_scale_f32_32x32x64_f8f6f4 per
// pair of blocks, lane (n, h) supplying the 32 codes of block 2 s + h of the step (16 bytes) of row
// or channel n to product s, and that block's scale byte.
//   - codes: the item's gathered rows and its channels are loaded into an LDS ring by buffer loads
//     that write LDS, a step's 64 bytes of a row by 4 neighbouring lanes. (Loaded straight into the
//     registers of the lanes that multiply them, neighbouring lanes would read 16 bytes of
//     different rows: the L1 then delivers 16 bytes a clock of its 64, and was busy 86 % of the
//     time.) Chunk c of row r lies at position c ^ (r / 4 % 4) of the row's 64 bytes, so that the
//     16 lanes that the LDS serves together hit all of its banks;
//   - scales: 16 bytes of a row or channel (4 steps) per load, a window of 4 steps ahead. A load's
//     cost is set by the lines it touches: 4 bytes at a time they took as much as the codes.
// The epilogue multiplies by the gate and writes each output once.
#include <type_traits>

#include "gemm_core.h"
#include "mx_unit.h"

namespace tq {

namespace {

typedef int32_t i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int F4_ROW = 64;     // code bytes of a row per step of 128 inputs
constexpr int F4_WINDOW = 4;   // steps whose scales are loaded together (512 inputs)

template <int WAVES>
struct F4Shared {
  static constexpr int kRows = 32 * WAVES;  // of an item, and channels of its group
  static constexpr int kStages = 4;
  // the rows' codes, then the channels'; one scale window of each, two windows
  alignas(16) uint8_t codes[kStages][2 * kRows * F4_ROW];
  alignas(16) uint8_t scales[2][2 * kRows * 16];
  int slot[kRows];
  float gate[kRows];
};

__device__ __forceinline__ i32x8 fp4_operand(u32x4 c) {
  return (i32x8){(int)c.x, (int)c.y, (int)c.z, (int)c.w, 0, 0, 0, 0};
}
// D += A * B over 64 inputs, the scales in byte S of sa and sb
template <int S>
__device__ __forceinline__ f32x16 mfma_fp4(u32x4 a, u32x4 b, f32x16 c, uint32_t sa, uint32_t sb) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fp4_operand(a), fp4_operand(b), c, 4, 4, S,
                                                         (int)sa, S, (int)sb);
}

// WR waves share out the rows (MB blocks of 32 each), WAVES / WR the channels (NB blocks each);
// rows past the item are zeros.
template <int LAYOUT, int WAVES, int WR, int MB, int NB>
__device__ __forceinline__ void f4_item(const Fp4GemmArgs& a, F4Shared<WAVES>& sh, const uint8_t* unit, int first,
                        int nrows, int channels) {
  using U = MxUnit<MX_FP4>;
  using S = F4Shared<WAVES>;
  static_assert(WAVES / WR * NB * 32 == S::kRows && WR * MB * 32 <= S::kRows, "the item's shape");
  static_assert(S::kStages == F4_WINDOW, "a step's stage is its place in the window");
  constexpr int LA = (WR * MB * 2 + WAVES - 1) / WAVES, LB = 2;  // loads of 16 rows per wave and step
  const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, n = lane & 31;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wr = WR == 1 ? 0 : w % WR, wc = w / WR;
  const int nsteps = a.in / 128;  // a multiple of 4

  // Load i of wave w fills rows 16 (w + WAVES i) .. + 15 of a stage: lane l writes position l % 4 of
  // row l / 4 of them. Rows past the item load from beyond the buffers' ends (below 2^31 bytes) and
  // read zeros; channels past the group read its last one (their outputs are not stored).
  const GemmRsrc ra = gemm_rsrc(a.xa, a.xa_bytes), rs = gemm_rsrc(a.xs, a.xs_bytes);
  const GemmRsrc rb = gemm_rsrc(unit, (uint32_t)U::unit_bytes(a.out, a.in));
  uint32_t avo[LA], bvo[LB];
#pragma unroll
  for (int i = 0; i < LA; ++i) {
    const int r = 16 * (w + WAVES * i) + (lane >> 2), c = (lane & 3) ^ ((r >> 2) & 3);
    avo[i] = r < nrows ? (uint32_t)(sh.slot[r] / a.topk) * (uint32_t)(a.in / 2) + 16u * c : 0x80000000u;
  }
  uint32_t pstep = 64;  // a channel's next step, in store order; in the read order, the group's
#pragma unroll
  for (int i = 0; i < LB; ++i) {
    const int r = 16 * (w + WAVES * i) + (lane >> 2), c = (lane & 3) ^ ((r >> 2) & 3);
    const int o = first + (r < channels ? r : channels - 1);
    bvo[i] = LAYOUT ? U::packed_at(a.out, a.in, o, c) : U::stored_at(a.in, o, c);
  }
  uint32_t bstep[LB];
#pragma unroll
  for (int i = 0; i < LB; ++i) {
    const int r = 16 * (w + WAVES * i);
    const int o = first + (r < channels ? r : channels - 1);
    bstep[i] = LAYOUT ? __builtin_amdgcn_readfirstlane(1024u * U::group_strips(a.out, o / 128)) : pstep;
  }
  // load i of this wave: of rows, then of channels
  auto load_codes = [&](int i, int st, int kk, uint32_t past) {
    uint8_t* rows = sh.codes[st] + 16 * F4_ROW * w;
    if (i < LA)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (LdsPtr)(rows + 16 * F4_ROW * WAVES * i), 16, avo[i < LA ? i : 0] | past,
                                               (uint32_t)(F4_ROW * kk), 0, 0);
    else
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (LdsPtr)(rows + S::kRows * F4_ROW + 16 * F4_ROW * WAVES * (i - LA)), 16,
                                               bvo[i < LA ? 0 : i - LA] | past, bstep[i < LA ? 0 : i - LA] * (uint32_t)kk, 0, 0);
  };
  // scales: wave w loads those of rows 64 w .. + 63 of the item's, then of the group's
  const int sr = 64 * (w % (WAVES / 2)) + lane;
  const bool of_rows = w < WAVES / 2;
  const GemmRsrc rscale = of_rows ? rs : rb;
  const uint32_t svo =
      of_rows ? (sr < nrows ? (uint32_t)(sh.slot[sr] / a.topk) * (uint32_t)(a.in / 32) : 0x80000000u)
              : U::scale_at(a.out, a.in, first + (sr < channels ? sr : channels - 1), 0);
  auto load_scales = [&](int slot, int kk, uint32_t past) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rscale, (LdsPtr)(sh.scales[slot] + 64 * 16 * w), 16, svo | past,
                                             (uint32_t)(4 * kk), 0, 0);
  };

  f32x16 acc[MB][NB];
#pragma unroll
  for (int mb = 0; mb < MB; ++mb)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[mb][nb][i] = 0.0f;

  const int row0 = 32 * MB * wr + n, col0 = 32 * NB * wc + n;
  uint32_t at[2];  // chunk 2 s + h of row n (blocks start at multiples of 32 rows)
#pragma unroll
  for (int s = 0; s < 2; ++s) at[s] = 16u * ((2 * s + h) ^ ((n >> 2) & 3));

  uint32_t sa[MB], sb[NB];
  u32x4 wa[MB], wb[NB];  // a window's scales
  u32x4 va[2][MB], vb[2][NB];
  // read i of the codes of product s of the step in stage st: of channels, then of rows
  auto read_codes = [&](int i, int st, int s) {
    if (i < NB)
      vb[s][i < NB ? i : 0] =
          *reinterpret_cast<const u32x4*>(sh.codes[st] + F4_ROW * (S::kRows + col0 + 32 * i) + at[s]);
    else
      va[s][i < NB ? 0 : i - NB] =
          *reinterpret_cast<const u32x4*>(sh.codes[st] + F4_ROW * (row0 + 32 * (i - NB)) + at[s]);
  };
  auto read_scales = [&](int slot) {
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
      wa[mb] = *reinterpret_cast<const u32x4*>(sh.scales[slot] + 16 * (row0 + 32 * mb));
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
      wb[nb] = *reinterpret_cast<const u32x4*>(sh.scales[slot] + 16 * (S::kRows + col0 + 32 * nb));
  };
  load_scales(0, 0, 0);
#pragma unroll
  for (int k = 0; k < S::kStages; ++k)
#pragma unroll
    for (int i = 0; i < LA + LB; ++i) load_codes(i, k, k, 0);
  wait_vmcnt<3 * (LA + LB)>();
  bare_barrier();
  read_scales(0);
#pragma unroll
  for (int i = 0; i < MB + NB; ++i) read_codes(i, 0, 0);
  // A step's reads from LDS run beside products: those of product 1 beside the products 0, those of
  // the next step's product 0 beside the products 1. The barrier between them says that every wave
  // has read all of this step's stage, which the loads of four steps on then fill, and that the
  // next stage has landed. Reads and loads are spread between the products: a wave whose load finds
  // the queue full, because all waves load at once, could not multiply meanwhile. All products stay
  // in the loop: the compiler would sink those behind the last barrier into the epilogue's branches,
  // where lanes that store nothing do not prepare their operands.
#pragma unroll 1
  for (int k0 = 0; k0 < nsteps; k0 += F4_WINDOW) {
    // in the last window nothing is left to load: the same loads, from beyond the buffers' ends
    const uint32_t past = k0 + F4_WINDOW >= nsteps ? 0x80000000u : 0u;
    const int slot = (k0 / F4_WINDOW) & 1;
#pragma unroll
    for (int t = 0; t < F4_WINDOW; ++t) {
      // bytes h and 2 + h of the step's four scales to bytes 0 and 2
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) sa[mb] = wa[mb][t] >> (8 * h);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) sb[nb] = wb[nb][t] >> (8 * h);
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) {
#pragma unroll
        for (int i = (MB + NB) * mb / MB; i < (MB + NB) * (mb + 1) / MB; ++i) read_codes(i, t, 1);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) acc[mb][nb] = mfma_fp4<0>(vb[0][nb], va[0][mb], acc[mb][nb], sb[nb], sa[mb]);
        __builtin_amdgcn_sched_barrier(0);
      }
      // in flight may be the loads of the two stages after the next
      wait_vmcnt<2 * (LA + LB)>();
      bare_barrier();
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) {
        if (mb == 0 && t + 1 == F4_WINDOW) read_scales(slot ^ 1);  // after the last step: of no use
#pragma unroll
        for (int i = (MB + NB) * mb / MB; i < (MB + NB) * (mb + 1) / MB; ++i) read_codes(i, (t + 1) % S::kStages, 0);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) acc[mb][nb] = mfma_fp4<2>(vb[1][nb], va[1][mb], acc[mb][nb], sb[nb], sa[mb]);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = (LA + LB) * mb / MB; i < (LA + LB) * (mb + 1) / MB; ++i) load_codes(i, t, k0 + t + S::kStages, past);
        if (mb == MB - 1 && t == 0) load_scales(slot ^ 1, k0 + F4_WINDOW, past);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  // The epilogue: element 4 j + i of lane (n, h) is channel 8 j + 4 h + i of a block, of the block's
  // row n. Each wave brings its rows together in LDS (its own part of the stages, once no load
  // writes them any more) and writes them in pieces of 128 NB bytes: stored from the lanes as they
  // are, 16 bytes of 32 rows at a time, the results of 8,192 tokens x 8 of 32, 1,536 x 5,120, took 95 us
  // of the 352 that this kernel took then.
  wait_vmcnt<0>();
  bare_barrier();
  constexpr int kLine = 128 * NB + 16;  // the 16 bytes more put a row's pieces on other banks
  static_assert(WAVES * 32 * kLine <= (int)sizeof(sh.codes), "the stages hold the waves' rows");
  uint8_t* part = &sh.codes[0][0] + w * 32 * kLine;
  constexpr int kLanes = 8 * NB, kRowsAt = 64 / kLanes;  // lanes of a row, rows at a time
  const int oc = 32 * NB * wc + 4 * (lane % kLanes);
#pragma unroll
  for (int mb = 0; mb < MB; ++mb) {
    const float gate = sh.gate[row0 + 32 * mb];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<f32x4*>(part + n * kLine + 128 * nb + 32 * j + 16 * h) =
            (f32x4){acc[mb][nb][4 * j] * gate, acc[mb][nb][4 * j + 1] * gate, acc[mb][nb][4 * j + 2] * gate,
                    acc[mb][nb][4 * j + 3] * gate};
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < 32 / kRowsAt; ++i) {
      const int m = kRowsAt * i + lane / kLanes, r = 32 * (MB * wr + mb) + m;
      const f32x4 v = *reinterpret_cast<const f32x4*>(part + m * kLine + 16 * (lane % kLanes));
      if (r < nrows && oc < channels)  // channels is a multiple of 16
        *reinterpret_cast<f32x4*>(a.y + (size_t)sh.slot[r] * a.out + first + oc) = v;
    }
    __builtin_amdgcn_wave_barrier();
  }
}

template <int WAVES, int LAYOUT>
__device__ __forceinline__ void f4_rows(const Fp4GemmArgs& a, F4Shared<WAVES>& sh, const uint8_t* unit, int first,
                        int nrows, int channels) {
  if constexpr (WAVES == 8) {
    if (nrows > 192)
      f4_item<LAYOUT, 8, 2, 4, 2>(a, sh, unit, first, nrows, channels);
    else if (nrows > 128)
      f4_item<LAYOUT, 8, 2, 3, 2>(a, sh, unit, first, nrows, channels);
    else if (nrows > 64)
      f4_item<LAYOUT, 8, 2, 2, 2>(a, sh, unit, first, nrows, channels);
    else
      f4_item<LAYOUT, 8, 1, 2, 1>(a, sh, unit, first, nrows, channels);
  } else {
    if (nrows > 96)
      f4_item<LAYOUT, 4, 2, 2, 2>(a, sh, unit, first, nrows, channels);
    else if (nrows > 64)
      f4_item<LAYOUT, 4, 1, 3, 1>(a, sh, unit, first, nrows, channels);
    else if (nrows > 32)
      f4_item<LAYOUT, 4, 1, 2, 1>(a, sh, unit, first, nrows, channels);
    else
      f4_item<LAYOUT, 4, 1, 1, 1>(a, sh, unit, first, nrows, channels);
  }
}

template <int WAVES>
__global__ __launch_bounds__(64 * WAVES, 2) void fp4_gemm_kernel(Fp4GemmArgs a) {
  __shared__ F4Shared<WAVES> sh;
  constexpr int kRows = F4Shared<WAVES>::kRows;
  int item, grp;
  if (!gemm_unit(a.n_items, a.groups, &item, &grp)) return;
  const int4 itd = reinterpret_cast<const int4*>(a.items)[item];
  const int e = itd.x, nrows = itd.z;
  for (int m = threadIdx.x; m < kRows; m += 64 * WAVES) {
    const int slot = m < nrows ? a.pairs[itd.y + m] : 0;
    sh.slot[m] = slot;
    sh.gate[m] = (m < nrows && a.gates) ? a.gates[slot] : 1.0f;
  }
  __syncthreads();
  const int channels = min(kRows, a.out - grp * kRows);
  const uint8_t* unit = a.units + (size_t)e * MxUnit<MX_FP4>::unit_bytes(a.out, a.in);
  if (a.layout)
    f4_rows<WAVES, 1>(a, sh, unit, grp * kRows, nrows, channels);
  else
    f4_rows<WAVES, 0>(a, sh, unit, grp * kRows, nrows, channels);
}

}  // namespace

// Items of 256 rows and channels read each operand half as often, but one fills a compute unit; they
// are the faster ones where experts have many rows and their items (with half of an expert's last one
// empty) are enough for most of the GPU. The GEMM between events, 256 against 128: 8,192 tokens x 8 of
// 32, 1,536 x 5,120: 314 and 378 us (256 in a trace that alternates between two sets of inputs: 325 to
// 329); 2,048 x 8 of 64, 1,536 x 2,560: 55 and 61; 8,192 x 2 of 64, 512 x 2,560 (192 items): 26 and 28;
// 700 x 6 of 20, 1,424 x 7,168 (156): 45 and 46; 1,024 x 4 of 16, 1,536 x 5,120 (144): 37 and 33; 512 x
// 8 of 8 (120): 35 and 29.
//
// What an item of 256 x 256 x 5,120 spends: 91,000 clocks at 1.9 GHz, of which 67,000 in the loop (the
// products alone need 41,000; the rest waits for loads that take up to 5,000 clocks beside the other
// units' stores), 11,000 until its first stages are there and 12,000 on its stores. 4 waves of 128 x
// 128, which read LDS a third less, take as long (2 % less there, 12 % more in the third case above);
// items of 128 x 256, two on a compute unit, 12 % longer.
int fp4_item_rows(int64_t N, int E, int out) {
  if (out <= 128 || N < 160 * (int64_t)E) return 128;
  const int64_t items = (N / 256 + E / 2) * ((out + 255) / 256);
  return items >= 160 ? 256 : 128;
}

hipError_t launch_fp4_gemm(const Fp4GemmArgs& args, hipStream_t s) {
  Fp4GemmArgs a = args;
  a.groups = (a.out + a.item_rows - 1) / a.item_rows;
  const int blocks = gemm_grid(a.max_items, a.groups);
  if (blocks == 0) return hipSuccess;
  if (a.item_rows == 256) return launch_timed(fp4_gemm_kernel<8>, dim3(blocks), dim3(512), s, a);
  return launch_timed(fp4_gemm_kernel<4>, dim3(blocks), dim3(256), s, a);
}

}  // namespace tq

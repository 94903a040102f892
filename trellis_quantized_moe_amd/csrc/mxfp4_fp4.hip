// The routed product of MXFP4 activations with MXFP4 experts on gfx950's fp4 matrix cores
// (FORMAT F30): both operands are their E2M1 codes with their E8M0 scales as stored, nothing is
// decoded.
//
// A work item is up to 128 routed rows of one expert times one group of 128 NB output channels
// over the whole input range, in steps of 256 inputs, on four waves, wave w owning channels
// 32 NB w .. 32 NB (w + 1) - 1 for all rows. A step is four v_mfma_scale_f32_32x32x64_f8f6f4 per
// 32 rows and 32 channels: lane (n, h) supplies the 32 codes of block 2 s + h of the step (16
// bytes) of row or channel n to product s, and that block's scale byte.
//   - activations: the item's gathered rows are loaded into a 3-stage LDS ring two steps ahead by
//     buffer loads that write LDS, 16-byte chunk c of row r at position c ^ (r % 8), so that the 8
//     lanes the LDS serves together hit 8 chunk columns; with each row's 8 scale bytes;
//   - weights: straight from the unit into registers, each product's codes replaced by those of
//     the next step as soon as they have been used, and the channel's 8 scale bytes of a step too.
// A byte permutation picks the four scale bytes of a lane's blocks, and the products name one of
// them each.
// The epilogue multiplies by the gate and writes each output once.
#include <type_traits>

#include "gemm_core.h"
#include "mx_unit.h"

namespace tq {

namespace {

typedef int32_t i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int F4_THREADS = 256;
constexpr int F4_STAGES = 3;
constexpr int F4_STEP = 256;           // inputs per step
constexpr int F4_ROW = F4_STEP / 2;    // code bytes of one row per step

struct F4Shared {
  alignas(16) uint8_t a[F4_STAGES][GEMM_MT * F4_ROW];
  alignas(16) uint2 s[F4_STAGES][GEMM_MT];  // the row's 8 block scales of the step
  int slot[GEMM_MT];
  float gate[GEMM_MT];
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

// MBK: the blocks of 32 rows that the products run over (rows past the item are zeros).
template <int LAYOUT, int MBK, int NB>
__device__ void f4_item(const Fp4GemmArgs& a, F4Shared& sh, const uint8_t* unit, int grp,
                        int nrows, int channels) {
  using U = MxUnit<MX_FP4>;
  const int tid = threadIdx.x, lane = tid & 63, h = lane >> 5, n = lane & 31;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int nsteps = a.in / F4_STEP;  // even (in is a multiple of 512)

  // instruction j of wave w fills rows 32 w + 8 j .. + 7 of a stage: lane l writes position l % 8
  // of row 32 w + 8 j + l / 8, which holds chunk (l % 8) ^ (row % 8). Rows past the item load from
  // beyond the buffer's end (xa_bytes < 2^31) and read zeros.
  const GemmRsrc ra = gemm_rsrc(a.xa, a.xa_bytes), rs = gemm_rsrc(a.xs, a.xs_bytes);
  uint32_t avo[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int r = 32 * w + 8 * j + (lane >> 3);
    const int c = (lane & 7) ^ (r & 7);
    avo[j] = r < nrows ? (uint32_t)(sh.slot[r] / a.topk) * (uint32_t)(a.in / 2) + 16u * c : 0x80000000u;
  }
  // scales: lane l loads half l % 2 of the 8 bytes of row 32 w + l / 2
  const int srow = 32 * w + (lane >> 1);
  const uint32_t svo = srow < nrows ? (uint32_t)(sh.slot[srow] / a.topk) * (uint32_t)(a.in / 32) + 4u * (lane & 1)
                                    : 0x80000000u;
  // past the last step: the last step's again, into a stage no step reads any more, so every step
  // issues the same loads
  auto load_a = [&](int st, int kk) {
    uint8_t* base = sh.a[st] + 32 * w * F4_ROW;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (LdsPtr)(base + 8 * j * F4_ROW), 16, avo[j],
                                               (uint32_t)(F4_ROW * kk), 0, 0);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (LdsPtr)(&sh.s[st][32 * w]), 4, svo,
                                             (uint32_t)(8 * kk), 0, 0);
  };

  // weights: channels past the group read its last one (their outputs are not stored). Block
  // 2 s + h of step kk is, in store order, 128 kk + 32 s bytes after block h; in the read order it
  // lies in step 2 kk + s / 2 of 128 inputs, 32 (s % 2) bytes further.
  const GemmRsrc rb = gemm_rsrc(unit, (uint32_t)U::unit_bytes(a.out, a.in));
  const int first = grp * 128 * NB;
  uint32_t bvo[NB], bso[NB];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int oc = 32 * (NB * w + nb) + n;
    const int o = first + (oc < channels ? oc : channels - 1);
    bvo[nb] = LAYOUT ? U::packed_at(a.out, a.in, o, h) : U::stored_at(a.in, o, h);
    bso[nb] = U::scale_at(a.out, a.in, o, 0);
  }
  const int oc0 = 32 * NB * w < channels ? 32 * NB * w : channels - 1;
  const uint32_t pstep = 1024u * U::group_strips(a.out, (first + oc0) / 128);
  auto boff = [&](int kk, int s) {
    return LAYOUT ? pstep * (uint32_t)(2 * kk + (s >> 1)) + 32u * (s & 1) : 128u * (uint32_t)kk + 32u * s;
  };
  u32x4 bc[4][NB];
  u32x2 sw[NB];
  auto load_b = [&](int s, int kk) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
      bc[s][nb] = __builtin_amdgcn_raw_buffer_load_b128(rb, bvo[nb], boff(kk, s), 0);
  };
  auto load_s = [&](int kk) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
      sw[nb] = __builtin_amdgcn_raw_buffer_load_b64(rb, bso[nb], 8u * (uint32_t)kk, 0);
  };

  f32x16 acc[MBK][NB];
#pragma unroll
  for (int mb = 0; mb < MBK; ++mb)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[mb][nb][i] = 0.0f;

  const uint32_t sel = h ? 0x07050301u : 0x06040200u;  // bytes 2 s + h of eight
  uint32_t rd[4];  // chunk 2 s + h of row n (row % 8 = n % 8)
#pragma unroll
  for (int s = 0; s < 4; ++s) rd[s] = F4_ROW * n + 16u * ((2 * s + h) ^ (n & 7));

  load_a(0, 0);
  load_s(0);
#pragma unroll
  for (int s = 0; s < 4; ++s) load_b(s, 0);
  load_a(1, 1);

  int stage = 0;
#pragma unroll 1
  for (int kk = 0; kk < nsteps; ++kk) {
    // this wave's loads of stage kk have landed: what may be in flight are those issued since
    // (5 of stage kk + 1, the weights' scales and codes of step kk)
    wait_vmcnt<5 + 5 * NB>();
    bare_barrier();
    load_a(stage >= 1 ? stage - 1 : F4_STAGES - 1, kk + 2 < nsteps ? kk + 2 : nsteps - 1);
    const uint8_t* st = sh.a[stage];
    uint32_t sa[MBK], sb[NB];
#pragma unroll
    for (int mb = 0; mb < MBK; ++mb) {
      const uint2 v = sh.s[stage][32 * mb + n];
      sa[mb] = perm(v.y, v.x, sel);
    }
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) sb[nb] = perm(sw[nb].y, sw[nb].x, sel);
    const int next = kk + 1 < nsteps ? kk + 1 : kk;
    load_s(next);
    auto product = [&](auto S) {
      constexpr int s = decltype(S)::value;
#pragma unroll
      for (int mb = 0; mb < MBK; ++mb) {
        const u32x4 av = *reinterpret_cast<const u32x4*>(st + 32 * F4_ROW * mb + rd[s]);
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) acc[mb][nb] = mfma_fp4<s>(av, bc[s][nb], acc[mb][nb], sa[mb], sb[nb]);
      }
      load_b(s, next);
    };
    product(std::integral_constant<int, 0>{});
    product(std::integral_constant<int, 1>{});
    product(std::integral_constant<int, 2>{});
    product(std::integral_constant<int, 3>{});
    stage = stage + 1 < F4_STAGES ? stage + 1 : 0;
  }
  // no load may still be writing this workgroup's LDS when it ends
  wait_vmcnt<0>();

#pragma unroll
  for (int mb = 0; mb < MBK; ++mb) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int r = 32 * mb + 8 * (i >> 2) + 4 * h + (i & 3);
      if (r < nrows) {
        float* dst = a.y + (size_t)sh.slot[r] * a.out + first;
        const float gate = sh.gate[r];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const int oc = 32 * (NB * w + nb) + n;
          if (oc < channels) dst[oc] = acc[mb][nb][i] * gate;
        }
      }
    }
  }
}

template <int NB>
__global__ __launch_bounds__(F4_THREADS, NB == 2 ? 2 : 3) void fp4_gemm_kernel(Fp4GemmArgs a) {
  __shared__ F4Shared sh;
  int item, grp;
  if (!gemm_unit(a.n_items, a.groups, &item, &grp)) return;
  const int4 itd = reinterpret_cast<const int4*>(a.items)[item];
  const int e = itd.x, nrows = itd.z;
  for (int m = threadIdx.x; m < GEMM_MT; m += F4_THREADS) {
    const int slot = m < nrows ? a.pairs[itd.y + m] : 0;
    sh.slot[m] = slot;
    sh.gate[m] = (m < nrows && a.gates) ? a.gates[slot] : 1.0f;
  }
  __syncthreads();
  const int channels = min(128 * NB, a.out - grp * 128 * NB);
  const uint8_t* unit = a.units + (size_t)e * MxUnit<MX_FP4>::unit_bytes(a.out, a.in);
  auto run = [&](auto MBK) {
    if (a.layout)
      f4_item<1, decltype(MBK)::value, NB>(a, sh, unit, grp, nrows, channels);
    else
      f4_item<0, decltype(MBK)::value, NB>(a, sh, unit, grp, nrows, channels);
  };
  switch ((nrows + 31) >> 5) {
    case 1: run(std::integral_constant<int, 1>{}); break;
    case 2: run(std::integral_constant<int, 2>{}); break;
    case 3: run(std::integral_constant<int, 3>{}); break;
    default: run(std::integral_constant<int, 4>{}); break;
  }
}

}  // namespace

hipError_t launch_fp4_gemm(const Fp4GemmArgs& args, hipStream_t s) {
  Fp4GemmArgs a = args;
  const bool wide = a.out > 128;
  a.groups = (a.out + (wide ? 255 : 127)) / (wide ? 256 : 128);
  const int blocks = gemm_grid(a.max_items, a.groups);
  if (blocks == 0) return hipSuccess;
  if (wide) return launch_timed(fp4_gemm_kernel<2>, dim3(blocks), dim3(F4_THREADS), s, a);
  return launch_timed(fp4_gemm_kernel<1>, dim3(blocks), dim3(F4_THREADS), s, a);
}

}  // namespace tq

// Decode batches of the routed 4-bit product (FORMAT F30) in one launch (gfx950): no plan, no
// routing and no conversion of the activations come before it.
//
// A workgroup has 16 S output channels of one expert. With fewer experts than slots there is a
// workgroup for every expert (and one per 16 slots for the rows of empty and invalid ones), else one
// for every slot, of which those of an expert's first slot work and the others leave at once. Each of
// its waves looks through all route ids for the expert's slots, so every touched weight is read once
// (per 16 rows). The four waves share out the inputs. Per window of 4 steps of 128 inputs a wave
//   - has asked for the window's codes and scales of its channels one window ahead (two windows ahead
//     were 15 % slower for one token): lane (n, q)
//     loads the 16 bytes of block q of a step of channel n, and 16 scale bytes (4 steps) of it;
//   - converts the rows' inputs to MXFP4 (F29): lane p block p % 16 of row p / 16, loaded one
//     conversion ahead, into LDS, from which lane (n, q) reads block q of row n;
//   - multiplies: v_mfma_scale_f32_16x16x128_f8f6f4 per step and 16 channels.
// The waves' sums are added in order, multiplied by the gate and written once.
//
// Bound by the weights' bytes where there are many (64 tokens x 8 of 384 experts, 128 x 5,120: 21.5 us
// for about 98 MB), else by the latency of its dependent loads (one token, 1,536 x 5,120: 8.7 us; 128
// x 5,120: 5.1). 32 channels a workgroup convert the rows half as often, 16 make twice as many
// workgroups, which is faster until there are two for every compute unit (16 and 32 channels, of
// 5,120 inputs: one token x 8 of 128 outputs 5.1 and 5.9 us, of 1,536 outputs 9.0 and 9.5; two tokens
// 15.4 and 14.1; 64 tokens x 8 of 128 outputs over 128 experts 15.2 and 13.0).
#include "gemm_core.h"
#include "mx_unit.h"
#include "mxfp4_quant.h"

namespace tq {

namespace {

typedef int32_t i32x8 __attribute__((ext_vector_type(8)));

constexpr int FD_WAVES = 4;
constexpr int FD_WINDOW = 4;  // steps of 128 inputs whose scales one 16-byte load brings

template <int S>
struct FdShared {
  // per wave: the rows' codes of a window [row][step][block], with their scales [row][step]
  alignas(16) uint8_t codes[FD_WAVES][16 * FD_WINDOW * 64];
  alignas(16) uint8_t scales[FD_WAVES][16 * 16];
  float sums[FD_WAVES][S][16][17];
  int list[FP4_DECODE_SLOTS];
};

__device__ __forceinline__ i32x8 fd_operand(u32x4 c) {
  return (i32x8){(int)c.x, (int)c.y, (int)c.z, (int)c.w, 0, 0, 0, 0};
}

template <int S>
__global__ __launch_bounds__(64 * FD_WAVES) void fp4_decode_kernel(Fp4DecodeArgs a) {
  using U = MxUnit<MX_FP4>;
  __shared__ FdShared<S> sh;
  const int tid = threadIdx.x, lane = tid & 63, q = lane >> 4, n = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int row = blockIdx.x / a.groups;
  const int first = (blockIdx.x % a.groups) * 16 * S;
  const int channels = min(16 * S, a.out - first);
  const bool by_expert = a.E < a.N;
  if (by_expert && row >= a.E) {  // empty and invalid slots of 16
    for (int v = tid; v < 16 * 16 * S; v += 64 * FD_WAVES) {
      const int j = 16 * (row - a.E) + v / (16 * S), o = v % (16 * S);
      if (j >= a.N) break;
      const int id = a.ids[j];
      if (id >= 0 && id < a.E) continue;
      if (o < channels) a.y[(size_t)j * a.out + first + o] = id == -1 ? 0.0f : __builtin_nanf("");
      if (id != -1 && o == 0) set_status(a.status, STATUS_BAD_EXPERT);
    }
    return;
  }
  // 512 ids at a time, the first of them asked for together with this slot's
  const GemmRsrc ri = gemm_rsrc(a.ids, 4u * (uint32_t)a.N);
  uint32_t id[8];
  auto load_ids = [&](int j0) {
#pragma unroll
    for (int u = 0; u < 8; ++u) id[u] = __builtin_amdgcn_raw_buffer_load_b32(ri, 4 * (j0 + 64 * u + lane), 0, 0);
  };
  load_ids(0);
  const int e = by_expert ? row : __builtin_amdgcn_readfirstlane(a.ids[row]);
  if (e < 0 || e >= a.E) {  // an empty or invalid slot
    const float v = e == -1 ? 0.0f : __builtin_nanf("");
    if (tid < channels) a.y[(size_t)row * a.out + first + tid] = v;
    if (e != -1 && tid == 0) set_status(a.status, STATUS_BAD_EXPERT);
    return;
  }
  // the expert's slots; every wave writes the same list
  int cnt = 0, lead = -1;
  for (int j0 = 0; j0 < a.N; j0 += 512) {
    if (j0 > 0) load_ids(j0);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (j0 + 64 * u >= a.N) break;  // uniform
      const int j = j0 + 64 * u + lane;
      const bool hit = j < a.N && (int)id[u] == e;
      const uint64_t m = __ballot(hit);
      if (m && lead < 0) lead = j0 + 64 * u + __builtin_ctzll(m);
      if (hit)
        sh.list[cnt + __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0))] = j;
      cnt += __builtin_popcountll(m);
    }
    if (!by_expert && lead >= 0 && lead != row) return;  // uniform
  }
  if (cnt == 0) return;  // uniform
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
  const uint8_t* unit = a.units + (size_t)e * U::unit_bytes(a.out, a.in);
  const GemmRsrc rb = gemm_rsrc(unit, (uint32_t)U::unit_bytes(a.out, a.in));
  const int s0 = a.in / 128 * w / FD_WAVES, steps = a.in / 128 * (w + 1) / FD_WAVES - s0;  // this wave's
  uint32_t bvo[S], bso[S];
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const int o = first + min(16 * s + n, channels - 1);  // channels past the last read it again
    bvo[s] = a.layout ? U::packed_at(a.out, a.in, o, q) : U::stored_at(a.in, o, q);
    bso[s] = U::scale_at(a.out, a.in, o, 0);
  }
  const uint32_t bstep = a.layout ? 1024u * U::group_strips(a.out, first / 128) : 64u;
  struct Weights {
    u32x4 code[FD_WINDOW][S], scale[S];
  };
  // the window that starts at step k of the wave's; steps past its last read zeros
  auto load_weights = [&](Weights& b, int k) {
#pragma unroll
    for (int t = 0; t < FD_WINDOW; ++t) {
      const uint32_t past = k + t < steps ? 0u : 0x80000000u;
#pragma unroll
      for (int s = 0; s < S; ++s)
        b.code[t][s] = __builtin_amdgcn_raw_buffer_load_b128(rb, bvo[s] | past, bstep * (uint32_t)(s0 + k + t), 0);
    }
    // a wave's first step need not be a multiple of 4: its scales lie at any byte address that is a
    // multiple of 4 (a step's scales)
#pragma unroll
    for (int s = 0; s < S; ++s)
      b.scale[s] = __builtin_amdgcn_raw_buffer_load_b128(rb, bso[s], 4u * (uint32_t)(s0 + k), 0);
  };
  Weights b;
  uint8_t* wcodes = sh.codes[w];
  uint8_t* wscales = sh.scales[w];
  for (int c0 = 0; c0 < cnt; c0 += 16) {
    const int rows = min(16, cnt - c0);
    const int passes = (rows + 3) / 4;  // rows 4 p + lane / 16 are converted in pass p
    auto load_x = [&](u32x4 (&v)[4], int p, int k) {
      const int r = 4 * p + q;
      const int t = r < rows ? sh.list[c0 + r] / a.topk : 0;
      const bool there = r < rows && k + (n >> 2) < steps;  // block n of the window: step n / 4
      const u32x4* src = reinterpret_cast<const u32x4*>(a.x + (size_t)t * a.in + 128 * (size_t)(s0 + k) + 32 * n);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = there ? src[j] : (u32x4){0u, 0u, 0u, 0u};
    };
    f32x4 acc[S];
#pragma unroll
    for (int s = 0; s < S; ++s) acc[s] = (f32x4){0.f, 0.f, 0.f, 0.f};
    u32x4 xv[4];
    load_weights(b, 0);
    load_x(xv, 0, 0);
    for (int k = 0; k < steps; k += FD_WINDOW) {
      for (int p = 0; p < passes; ++p) {
        u32x4 nv[4];
        const bool more = p + 1 < passes;
        load_x(nv, more ? p + 1 : 0, more ? k : k + FD_WINDOW);
        const Fp4Block v = fp4_block(xv);
#pragma unroll
        for (int j = 0; j < 4; ++j) xv[j] = nv[j];
        const int r = 4 * p + q;
        *reinterpret_cast<u32x4*>(wcodes + 256 * r + 16 * n) = v.codes;
        wscales[16 * r + n] = (uint8_t)v.scale;
      }
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
      __builtin_amdgcn_wave_barrier();
      const Weights cur = b;
      if (k + FD_WINDOW < steps) load_weights(b, k + FD_WINDOW);
      const u32x4 sa = *reinterpret_cast<const u32x4*>(wscales + 16 * n);
#pragma unroll
      for (int t = 0; t < FD_WINDOW; ++t) {
        const u32x4 av = *reinterpret_cast<const u32x4*>(wcodes + 256 * n + 64 * t + 16 * q);
#pragma unroll
        for (int s = 0; s < S; ++s)
          acc[s] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              fd_operand(av), fd_operand(cur.code[t][s]), acc[s], 4, 4, 0, (int)(sa[t] >> (8 * q)), 0,
              k + t < steps ? (int)(cur.scale[s][t] >> (8 * q)) : 127);  // past the end: another row's
      }
      __builtin_amdgcn_wave_barrier();
    }
    // element i of lane (q, n) is row 4 q + i, channel n of its 16
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i) sh.sums[w][s][4 * q + i][n] = acc[s][i];
    __syncthreads();
    for (int v = tid; v < rows * 16 * S; v += 64 * FD_WAVES) {
      const int r = v / (16 * S), o = v % (16 * S);
      if (o < channels) {
        const int slot = sh.list[c0 + r];
        float sum = sh.sums[0][o / 16][r][o % 16];
#pragma unroll
        for (int u = 1; u < FD_WAVES; ++u) sum += sh.sums[u][o / 16][r][o % 16];
        a.y[(size_t)slot * a.out + first + o] = a.gates ? sum * a.gates[slot] : sum;
      }
    }
    __syncthreads();
  }
}

}  // namespace

hipError_t launch_fp4_decode(const Fp4DecodeArgs& args, hipStream_t s) {
  Fp4DecodeArgs a = args;
  const int64_t strips = a.out / 16, rows = a.E < a.N ? a.E + (a.N + 15) / 16 : a.N;
  const int S = (strips + 1) / 2 * a.N < 512 ? 1 : 2;
  a.groups = (int)(strips + S - 1) / S;
  const dim3 grid((unsigned)(rows * a.groups)), block(64 * FD_WAVES);
  if (S == 1) return launch_timed(fp4_decode_kernel<1>, grid, block, s, a);
  return launch_timed(fp4_decode_kernel<2>, grid, block, s, a);
}

}  // namespace tq

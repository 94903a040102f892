// The router's choice of experts and its gradient (gfx950; FORMAT F27, F28).
//
// expert_route: one wave per token. Expert e = 64 j + lane is value j of its lane, so a row is
// read by contiguous loads and the lowest index of equal keys is the lowest j, then the lowest
// lane. The wave
//   1. finds the row's largest logit (a row without experts ends here; a NaN, or +inf under
//      softmax, makes it a row of NaN weights);
//   2. makes the keys of the choice: the logits themselves where no bias enters (a score grows
//      with its logit), else score + bias in 64 bits, because keys that differ by less than
//      fp32 shows decide which expert is chosen;
//   3. keeps the best groups: each group's lanes take its one or two best keys, a group's rank
//      is the number of groups before it;
//   4. takes the largest key topk times; lane r keeps the r-th expert;
//   5. weighs: lane r computes its score from its logit in fp32, relative to the largest
//      chosen one where they are renormalised, so that no sum of scores can underflow.
//
// expert_route_backward: one wave per token; lane r holds slot r. Where the weights are
// renormalised, and under sigmoid, only chosen logits have a gradient: the row is zeros in LDS
// into which the lanes write theirs. Softmax without it has one for every logit.
#include <algorithm>

#include "tq_device.h"
#include "tq_internal.h"

namespace tq {

namespace {

constexpr int ROUTE_WAVES = 4;  // rows in flight per workgroup
constexpr float NEG = -__builtin_inff();

template <typename L>
__device__ __forceinline__ float load_logit(const L* p, int64_t i);
template <>
__device__ __forceinline__ float load_logit<float>(const float* p, int64_t i) {
  return p[i];
}
template <>
__device__ __forceinline__ float load_logit<uint16_t>(const uint16_t* p, int64_t i) {
  return __uint_as_float((uint32_t)p[i] << 16);
}
__device__ __forceinline__ void store_grad(float* p, int64_t i, float v) { p[i] = v; }
__device__ __forceinline__ void store_grad(uint16_t* p, int64_t i, float v) {
  p[i] = (uint16_t)f32_to_bf16_rne(v);
}

template <typename K>
__device__ __forceinline__ K wave_max(K v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) {
    const K o = __shfl_xor(v, d, 64);
    v = o > v ? o : v;
  }
  return v;
}
template <typename K>
__device__ __forceinline__ K wave_sum(K v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}

// The score of a logit that is not NaN, and not +inf under softmax.
__device__ __forceinline__ double score64(float x, bool sigmoid, float top, double z) {
  return sigmoid ? 1.0 / (1.0 + exp(-(double)x)) : exp((double)x - (double)top) / z;
}

// The best two of a set of keys, -inf where there are none.
template <typename K>
struct Best2 {
  K a, b;
  __device__ void add(K v) {
    b = v > a ? a : (v > b ? v : b);
    a = v > a ? v : a;
  }
};

// topk times the largest key of the row: lane r gets the r-th choice (its index, or -1).
template <typename K, int PER>
__device__ __forceinline__ int choose(K key[PER], int topk) {
  const int lane = threadIdx.x & 63;
  const K none = (K)NEG;
  int mine = -1;
  K best = none;
  int bj = 0;
  auto refresh = [&]() {
    best = none;
#pragma unroll
    for (int j = 0; j < PER; ++j)
      if (key[j] > best) {
        best = key[j];
        bj = j;
      }
  };
  refresh();
  for (int r = 0; r < topk; ++r) {
    const K top = wave_max(best);
    if (!(top > none)) break;  // uniform
    const int e = best == top ? 64 * bj + lane : 0x7FFFFFFF;
    int first = e;
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) first = min(first, __shfl_xor(first, d, 64));
    if (lane == r) mine = first;
    if (e == first) {
#pragma unroll
      for (int j = 0; j < PER; ++j)
        if (j == bj) key[j] = none;
      refresh();
    }
  }
  return mine;
}

// Closes the experts outside the group_topk best groups. keys: this wave's LDS, E entries
// holding the row's keys of the group scores.
template <typename K, int PER>
__device__ __forceinline__ void keep_groups(const RouterArgs& a, const K* keys, uint64_t& kept) {
  const int lane = threadIdx.x & 63;
  const int size = a.E / a.groups;
  int per = 64;  // lanes per group: the largest power of two with groups * per <= 64
  while (per * a.groups > 64) per >>= 1;
  const int g = lane / per, sub = lane & (per - 1);
  const K none = (K)NEG;
  Best2<K> t{none, none};
  if (g < a.groups)
    for (int i = sub; i < size; i += per) t.add(keys[g * size + i]);
  for (int d = per >> 1; d >= 1; d >>= 1) {
    const K oa = __shfl_xor(t.a, d, 64), ob = __shfl_xor(t.b, d, 64);
    t.add(oa);
    t.add(ob);
  }
  K score = t.a;
  if (a.group_top == 2 && t.b > none) score += t.b;
  int rank = 0;
  for (int h = 0; h < a.groups; ++h) {
    const K o = __shfl(score, h * per, 64);
    rank += o > score || (o == score && h < g);
  }
  const uint64_t m = __ballot(g < a.groups && sub == 0 && rank < a.group_topk);
  // bit g of kept: lane g * per of m
  kept = 0;
  for (int h = 0; h < a.groups; ++h) kept |= ((m >> (h * per)) & 1ull) << h;
}

template <typename L, int PER>
__global__ __launch_bounds__(64 * ROUTE_WAVES) void expert_route_kernel(RouterArgs a) {
  extern __shared__ double group_keys[];  // [waves of the workgroup][E], grouped routers only
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  const bool sigmoid = a.sigmoid;
  const L* logits = static_cast<const L*>(a.logits);
  for (int64_t t = (int64_t)blockIdx.x * waves + w; t < a.T; t += (int64_t)gridDim.x * waves) {
    const L* row = logits + t * a.E;
    float x[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int e = 64 * j + lane;
      x[j] = e < a.E ? load_logit(row, e) : NEG;
    }
    float top = NEG;
    bool nan = false;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      nan |= !(x[j] == x[j]) || (!sigmoid && x[j] == -NEG);
      top = fmaxf(top, x[j]);
    }
    top = wave_max(top);
    const bool by_logit = !a.bias;
    const bool scored = !by_logit || (a.groups > 1 && a.group_top == 2);
    double z = 1.0;
    double key[PER];
    int mine = -1;
    bool bad = __ballot(nan) != 0;
    if (!bad && top > NEG) {
      if (!sigmoid && scored) {
        double s = 0.0;
#pragma unroll
        for (int j = 0; j < PER; ++j) s += exp((double)x[j] - (double)top);
        z = wave_sum(s);
      }
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const int e = 64 * j + lane;
        key[j] = NEG;
        if (x[j] > NEG) {
          key[j] = scored ? score64(x[j], sigmoid, top, z) : (double)x[j];
          if (a.bias) key[j] += (double)a.bias[e];
        }
        nan |= !(key[j] == key[j]);
      }
      bad = __ballot(nan) != 0;
      if (!bad) {
        if (a.groups > 1) {
          double* keys = group_keys + (size_t)w * a.E;
#pragma unroll
          for (int j = 0; j < PER; ++j)
            if (64 * j + lane < a.E) keys[64 * j + lane] = key[j];
          __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
          __builtin_amdgcn_wave_barrier();
          uint64_t kept;
          keep_groups<double, PER>(a, keys, kept);
          const int size = a.E / a.groups;
#pragma unroll
          for (int j = 0; j < PER; ++j) {
            const int g = (64 * j + lane) / size;
            if (by_logit) key[j] = (double)x[j];
            if (g >= a.groups || !((kept >> g) & 1)) key[j] = NEG;
          }
          __builtin_amdgcn_wave_barrier();
        }
        mine = choose<double, PER>(key, a.topk);
      }
    }
    // the weights, slot r in lane r
    float weight = 0.0f;
    const float xs = mine >= 0 ? load_logit(row, mine) : NEG;
    const float most = wave_max(xs);
    if (sigmoid) {
      // e^min(x, 0) / (1 + e^-|x|), the numerator relative to the largest chosen one
      const float ref = a.renorm && most > NEG ? fminf(most, 0.0f) : 0.0f;
      if (mine >= 0) weight = expf(fminf(xs, 0.0f) - ref) / (1.0f + expf(-fabsf(xs)));
    } else if (mine >= 0) {
      weight = expf(xs - (a.renorm ? most : top));
    }
    float sum = 1.0f;
    if (a.renorm) {
      sum = wave_sum(weight);
    } else if (!sigmoid) {
      float s = 0.0f;
#pragma unroll
      for (int j = 0; j < PER; ++j) s += top > NEG ? expf(x[j] - top) : 0.0f;
      sum = wave_sum(s);
    }
    weight = mine >= 0 ? a.scale * (weight / sum) : 0.0f;
    if (lane < a.topk) {
      a.ids[t * a.topk + lane] = bad ? lane : mine;
      a.w[t * a.topk + lane] = bad ? __builtin_nanf("") : weight;
    }
  }
}

template <typename L, int PER>
__global__ __launch_bounds__(64 * ROUTE_WAVES) void expert_route_backward_kernel(RouterArgs a) {
  extern __shared__ float grads[];  // [waves of the workgroup][E]
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  const bool sigmoid = a.sigmoid;
  const L* logits = static_cast<const L*>(a.logits);
  L* dst = static_cast<L*>(a.dlogits);
  float* grad = grads + (size_t)w * a.E;
  for (int64_t t = (int64_t)blockIdx.x * waves + w; t < a.T; t += (int64_t)gridDim.x * waves) {
    const L* row = logits + t * a.E;
    int id = lane < a.topk ? a.chosen[t * a.topk + lane] : -1;
    const bool bad = __ballot(id < -1 || id >= a.E) != 0;
    if (bad) id = -1;
    const float dw = id >= 0 ? a.dw[t * a.topk + lane] : 0.0f;
    const float xs = id >= 0 ? load_logit(row, id) : NEG;
    const float most = wave_max(xs);
    float top = most, z = 1.0f;
    const bool dense = !sigmoid && !a.renorm;
    float x[PER];
    if (dense) {
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const int e = 64 * j + lane;
        x[j] = e < a.E ? load_logit(row, e) : NEG;
        top = fmaxf(top, x[j]);
      }
      top = wave_max(top);
      float s = 0.0f;
#pragma unroll
      for (int j = 0; j < PER; ++j) s += top > NEG ? expf(x[j] - top) : 0.0f;
      z = wave_sum(s);
    }
    // g: the gradient of the slot's score times the score, or (dense) the gradient alone
    float g = 0.0f, c = 0.0f;
    if (sigmoid) {
      const float ref = a.renorm && most > NEG ? fminf(most, 0.0f) : 0.0f;
      const float low = expf(-fabsf(xs));
      const float other = xs >= 0.0f ? low / (1.0f + low) : 1.0f / (1.0f + low);  // 1 - s
      float r = id >= 0 ? expf(fminf(xs, 0.0f) - ref) / (1.0f + low) : 0.0f;
      float mean = 0.0f;
      if (a.renorm) {
        const float sum = wave_sum(r);
        r = id >= 0 ? r / sum : 0.0f;
        mean = wave_sum(r * dw);
      }
      g = id >= 0 ? a.scale * r * (dw - mean) * other : 0.0f;
    } else if (a.renorm) {
      float r = id >= 0 ? expf(xs - most) : 0.0f;
      const float sum = wave_sum(r);
      r = id >= 0 ? r / sum : 0.0f;
      const float mean = wave_sum(r * dw);
      g = id >= 0 ? a.scale * r * (dw - mean) : 0.0f;
    } else {
      g = a.scale * dw;
      c = wave_sum(id >= 0 ? expf(xs - top) / z * g : 0.0f);
    }
    // slots of the same expert add up, in slot order
    float total = 0.0f;
    for (int k = 0; k < a.topk; ++k) {
      const int ik = __shfl(id, k, 64);
      const float gk = __shfl(g, k, 64);
      if (ik == id) total += gk;
    }
    for (int e = lane; e < a.E; e += 64) grad[e] = 0.0f;
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    if (id >= 0) grad[id] = total;
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int e = 64 * j + lane;
      if (e < a.E) {
        float v = grad[e];
        if (dense) v = top > NEG ? expf(x[j] - top) / z * (v - c) : 0.0f;
        store_grad(dst, t * a.E + e, bad ? __builtin_nanf("") : v);
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
}

constexpr int64_t ROUTE_MAX_BLOCKS = 1 << 20;  // the waves walk over further rows

// Rows in flight per workgroup: as many as 64 KB of LDS hold at `bytes` each.
int route_waves(size_t bytes) {
  int waves = ROUTE_WAVES;
  while (waves > 1 && bytes * waves > 65536) waves >>= 1;
  return waves;
}

template <typename L, int PER>
hipError_t start(const RouterArgs& a, bool backward, hipStream_t s) {
  const size_t row = backward ? sizeof(float) * a.E : a.groups > 1 ? sizeof(double) * a.E : 0;
  const int waves = route_waves(row);
  const int64_t blocks = std::min<int64_t>((a.T + waves - 1) / waves, ROUTE_MAX_BLOCKS);
  if (backward)
    hipLaunchKernelGGL((expert_route_backward_kernel<L, PER>), dim3((unsigned)blocks),
                       dim3(64 * waves), row * waves, s, a);
  else
    hipLaunchKernelGGL((expert_route_kernel<L, PER>), dim3((unsigned)blocks), dim3(64 * waves),
                       row * waves, s, a);
  return hipGetLastError();
}

template <typename L>
hipError_t by_size(const RouterArgs& a, bool backward, hipStream_t s) {
  if (a.E <= 64) return start<L, 1>(a, backward, s);
  if (a.E <= 128) return start<L, 2>(a, backward, s);
  if (a.E <= 256) return start<L, 4>(a, backward, s);
  if (a.E <= 384) return start<L, 6>(a, backward, s);
  if (a.E <= 512) return start<L, 8>(a, backward, s);
  if (a.E <= 1024) return start<L, 16>(a, backward, s);
  return start<L, 64>(a, backward, s);
}

}  // namespace

hipError_t launch_expert_route(const RouterArgs& a, bool backward, hipStream_t s) {
  if (a.T == 0) return hipSuccess;
  return a.bf16 ? by_size<uint16_t>(a, backward, s) : by_size<float>(a, backward, s);
}

}  // namespace tq

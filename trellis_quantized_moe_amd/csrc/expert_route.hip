// The router's choice of experts and its gradient (gfx950; FORMAT F27, F28).
//
// expert_route: one wave per token. Expert e = 64 j + lane is value j of its lane, so a row is
// read by contiguous loads and the lowest index of equal keys is the lowest j, then the lowest
// lane. The wave
//   1. looks for a NaN, or +inf under softmax, which makes a row of NaN weights;
//   2. makes the keys of the choice: the logits themselves where no bias enters (a score grows
//      with its logit), else score + bias in fp32, with a bound of their errors;
//   3. keeps the best groups: each group's lanes take its one or two best keys, a group's rank
//      is the number of groups before it;
//   4. takes the largest key topk times, and further ones within the errors of the last of those;
//      lane r keeps the r-th expert;
//   5. checks that fp32 has decided: no further ones, and neighbours in the order either differ by
//      more than their errors or have the same logit and bias. If not (a row in a hundred), each
//      lane computes its expert's key in 64 bits, where the definition lies, and the lanes change
//      places. Where the last group kept is not ahead of the next by more than the errors, or more
//      than 64 experts are candidates, steps 2 to 4 run once more in 64 bits throughout. (All rows
//      in 64 bits took 29 us for 8,192 rows of 384, one wave alone 8.5; now 11.7 under sigmoid and 12.9
//      under softmax, in 8 groups 16 and 17, or up to 26 where some rows run again, which is one chunk
//      in two under sigmoid and most under softmax; rows that all tie 83 to 98.);
//   6. weighs: lane r computes its score from its logit in fp32, relative to the largest
//      chosen one where they are renormalised, so that no sum of scores can underflow.
// One row a wave: a chunk's rows fill the GPU eight times over, and a single row ends soonest.
//
// expert_route_backward: one wave per token; lane r holds slot r. Where the weights are
// renormalised, and under sigmoid, the weights are functions of the chosen logits alone: no other
// is read (reading all of them, to find a NaN among those not chosen, made 8,192 rows of 384 in bf16
// take 8.1 us instead of 6.0), and the row is zeros in LDS into which the lanes write their gradients.
// Softmax without it has one for every logit.
#include <algorithm>
#include <type_traits>

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

// Reductions over the wave in moves that the compiler makes part of the operation: row shifts 1, 2, 4,
// 8, then row broadcasts 15 and 31, after which lane 63 has the result. A lane without a source takes a
// 0, which changes no sum and no maximum of unsigned integers.
template <int CTRL>
__device__ __forceinline__ float add_dpp(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, true));
}
__device__ __forceinline__ float wave_sum(float v) {
  v = add_dpp<0x111>(v);
  v = add_dpp<0x112>(v);
  v = add_dpp<0x114>(v);
  v = add_dpp<0x118>(v);
  v = add_dpp<0x142>(v);
  v = add_dpp<0x143>(v);
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
// fp32 values as integers of the same order (both zeros are one value), and back.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t u) {
  return __uint_as_float(u ^ ((u >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}
template <int CTRL>
__device__ __forceinline__ uint32_t max_dpp(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true));
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = max_dpp<0x111>(v);
  v = max_dpp<0x112>(v);
  v = max_dpp<0x114>(v);
  v = max_dpp<0x118>(v);
  v = max_dpp<0x142>(v);
  v = max_dpp<0x143>(v);
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
// The largest value (no NaN among them).
__device__ __forceinline__ float wave_max(float v) { return unordered(wave_max(ordered(v))); }
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}

// e^x by the hardware's 2^x: off by 2^-22 of it and by 2^-23 |x| of it (the argument's rounding); 0
// where it is below 2^-126.
__device__ __forceinline__ float fast_exp(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504f); }

// How far a score in fp32 is off, in units of 2^-24.
// Sigmoid, 1 / (1 + e): e's relative error of 4 and 2 |x| counts by s (1 - s) <= 1/4 and s (1 - s) |x| <=
// 0.23, the sum's rounding and the reciprocal are 1 and 2 of s: 4.5 in all.
// Softmax, e^d / Z with d = x - top: the exponential 4 of s and 2.5 |d| (its argument rounds twice), of
// which s |d| stays below 0.37; Z's exponentials 4 of it and 2.5 times the mean of |d|, which is at most
// ln 4,096 = 8.4, and its sums 1 each, those of a lane and 6; division and product 1 each: 1 + s (37 +
// the lane's), where s is at most 1 / Z.
template <int PER>
__device__ __forceinline__ float softmax_error(float rz) {
  return 0x1p-24f * (1.0f + rz * (37 + (PER > 8 ? 8 + PER / 8 : PER)));
}
// The sum of a lane's terms, in runs of 8.
template <int PER, typename F>
__device__ __forceinline__ float lane_sum(F term) {
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < PER; i += 8) {
    float run = 0.0f;
#pragma unroll
    for (int j = i; j < i + 8 && j < PER; ++j) run += term(j);
    sum += run;
  }
  return sum;
}
constexpr float SIGMOID_ERROR = 4.5f * 0x1p-24f;
// The sum with a bias rounds by 2^-24 of itself. Two keys are told apart where they differ by more than
// twice all that (with a factor of two to spare).
__device__ __forceinline__ float key_gap(float v, float error) { return 4.0f * error + 0x1p-22f * fabsf(v); }

// The best two of a set of keys, -inf where there are none.
template <typename K>
struct Best2 {
  K a, b;
  __device__ void add(K v) {
    b = v > a ? a : (v > b ? v : b);
    a = v > a ? v : a;
  }
};

// What a lane knows after the choice: the expert that came up in its turn (or -1) and that one's
// key; all lanes: how many came up, and whether more would have to (they do not fit a wave).
struct Choice {
  int e;
  float key;
  int count;
  bool more;
};

// topk times the largest key of the row: lane r gets the r-th. With `near`, further ones as long as
// they are within the errors of the last of those. A turn is a handful of instructions: each lane has
// its best two at hand, and one that gives both away (2 % of rows at 8 of 384) looks through its keys
// again for those behind the last one it gave.
template <int PER>
__device__ __forceinline__ Choice choose(const float (&value)[PER], int topk, bool near, float error) {
  const int lane = threadIdx.x & 63;
  const uint32_t none = ordered(NEG);
  uint32_t key[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) key[j] = ordered(value[j]);
  uint32_t best = none, second = none;
  int bj = 0, sj = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const bool first = key[j] > best, next = key[j] > second;
    sj = first ? bj : next ? j : sj;
    second = first ? best : next ? key[j] : second;
    bj = first ? j : bj;
    best = first ? key[j] : best;
  }
  uint32_t limit = none, mine = none;  // keys up to the limit are not chosen
  int e = -1, count = 0;
  bool more = false;
  uint64_t gave = 0;  // lanes whose second is gone
  for (int r = 0; r < topk || near; ++r) {
    const uint32_t top = wave_max(best);
    if (!(top > limit)) break;  // uniform
    if (r == 64) {
      more = true;
      break;
    }
    count = r + 1;
    if (r == topk - 1 && near) {
      // (an infinite key has no error, and less an infinite gap it would be a NaN, whose sign bit makes
      // it less than no key at all: lanes past the last expert would be chosen)
      const float v = unordered(top);
      limit = ordered(v < -NEG ? v - key_gap(v, error) : v);
    }
    const uint64_t m = __ballot(best == top);
    int winner = __builtin_ctzll(m);
    if (m & (m - 1)) {  // several lanes hold it: the lowest index
      int first = best == top ? 64 * bj + lane : 0x7FFFFFFF;
#pragma unroll
      for (int d = 32; d >= 1; d >>= 1) first = min(first, __shfl_xor(first, d, 64));
      winner = __builtin_amdgcn_readfirstlane(first) & 63;
    }
    const int j = __builtin_amdgcn_readlane(bj, winner);
    const bool turn = lane == r;
    e = turn ? 64 * j + winner : e;
    mine = turn ? top : mine;
    const bool won = lane == winner;
    best = won ? second : best;
    bj = won ? sj : bj;
    if ((gave >> winner) & 1) {  // uniform
      uint32_t b = none;
      int k = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if ((key[i] < top || (key[i] == top && i > j)) && key[i] > b) {
          b = key[i];
          k = i;
        }
      best = won ? b : best;
      bj = won ? k : bj;
    }
    gave |= 1ull << winner;
  }
  return Choice{e, unordered(mine), count, more};
}

// The groups that stay, as bits. keys: this wave's LDS, E entries holding the row's keys of the group
// scores. sure (of fp32 keys): the groups are those of the exact keys. A key plus or minus its error's
// bound orders as the keys do, so the exact best two of a group lie within the bounds of its best two
// here, and no other key counts: an expert out of service costs no certainty.
template <typename K>
__device__ __forceinline__ uint64_t keep_groups(const RouterArgs& a, const K* keys, float error, bool& sure) {
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
  const bool two = a.group_top == 2 && t.b > none;
  const K score = two ? t.a + t.b : t.a;
  int rank = 0;
  for (int h = 0; h < a.groups; ++h) {
    const K o = __shfl(score, h * per, 64);
    rank += o > score || (o == score && h < g);
  }
  const bool leads = g < a.groups && sub == 0;
  const bool stays = leads && rank < a.group_topk;
  if constexpr (std::is_same<K, float>::value) {
    // the least that a group which stays can have, the most that one with experts which goes can have;
    // of an infinite score (two biases beyond half of fp32's range, or no expert) nothing is known
    const float off = key_gap(t.a, error) + (two ? key_gap(t.b, error) : 0.0f);
    const bool known = fabsf(score) < -NEG;
    const bool goes = leads && !stays && t.a > none;
    const float least = -wave_max(stays ? (known ? off - score : -NEG) : NEG);
    const float most = wave_max(goes ? (known ? score + off : -NEG) : NEG);
    sure = __ballot(goes) == 0 || least > most;
  }
  const uint64_t m = __ballot(stays);
  uint64_t kept = 0;  // bit g: lane g * per of m
  for (int h = 0; h < a.groups; ++h) kept |= ((m >> (h * per)) & 1ull) << h;
  return kept;
}

template <typename L, int PER>
__device__ __forceinline__ void load_row(const RouterArgs& a, const L* row, float (&x)[PER]) {
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int e = 64 * j + (threadIdx.x & 63);
    x[j] = e < a.E ? load_logit(row, e) : NEG;
  }
}

// The sum of the softmax in 64 bits. (What hardly any row needs is in loops: its code and registers
// would cost every row.)
template <typename L>
__device__ __forceinline__ double sum64(const RouterArgs& a, const L* row, float top) {
  double s = 0.0;
#pragma unroll 1
  for (int e = threadIdx.x & 63; e < a.E; e += 64) s += exp((double)load_logit(row, e) - (double)top);
  return wave_sum(s);
}

// The key in 64 bits of an expert that is open, given the reciprocal of the sum.
template <bool SIGMOID>
__device__ __forceinline__ double key64(const RouterArgs& a, float x, int e, float top, double rz) {
  const double s = SIGMOID ? 1.0 / (1.0 + exp(-(double)x)) : exp((double)x - (double)top) * rz;
  return a.bias ? s + (double)a.bias[e] : s;
}

// The choice in 64 bits throughout. keys: this wave's LDS, E entries.
template <typename L, bool SIGMOID>
__device__ __forceinline__ int choose64(const RouterArgs& a, const L* row, float top, double* keys) {
  const int lane = threadIdx.x & 63;
  const double rz = SIGMOID ? 1.0 : 1.0 / sum64(a, row, top);
#pragma unroll 1
  for (int e = lane; e < a.E; e += 64) {
    const float x = load_logit(row, e);
    keys[e] = x > NEG ? key64<SIGMOID>(a, x, e, top, rz) : (double)NEG;
  }
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
  if (a.groups > 1) {
    bool sure;
    const uint64_t kept = keep_groups<double>(a, keys, 0.0f, sure);
    const int size = a.E / a.groups;
#pragma unroll 1
    for (int e = lane; e < a.E; e += 64) {
      if (!((kept >> (e / size)) & 1))
        keys[e] = NEG;
      else if (!a.bias && keys[e] > NEG)
        keys[e] = load_logit(row, e);
    }
  }
  double last = -(double)NEG;  // the last key taken, and its expert
  int last_e = -1, mine = -1;
#pragma unroll 1
  for (int r = 0; r < a.topk; ++r) {
    double best = NEG;
    int be = 0x7FFFFFFF;
#pragma unroll 1
    for (int e = lane; e < a.E; e += 64) {
      const double k = keys[e];
      if (k > best && (k < last || (k == last && e > last_e))) {
        best = k;
        be = e;
      }
    }
    // the largest key as an integer of the same order, half by half, then its lowest index
    const uint64_t u = __builtin_bit_cast(uint64_t, best + 0.0);
    const uint64_t o = u ^ ((u >> 63) ? ~0ull : 1ull << 63);
    const uint32_t hi = wave_max((uint32_t)(o >> 32));
    const bool tops = (uint32_t)(o >> 32) == hi;
    const uint32_t lo = wave_max(tops ? (uint32_t)o : 0u);
    const uint64_t top_o = (uint64_t)hi << 32 | lo;
    last = __builtin_bit_cast(double, top_o ^ ((top_o >> 63) ? 1ull << 63 : ~0ull));
    if (!(last > NEG)) break;  // uniform
    last_e = (int)~wave_max(o == top_o ? ~(uint32_t)be : 0u);
    mine = lane == r ? last_e : mine;
  }
  __builtin_amdgcn_wave_barrier();
  return mine;
}

// The candidates of a choice in the order of their keys in 64 bits, equal ones by the lowest index:
// lane r gets the r-th.
template <typename L, bool SIGMOID>
__device__ __forceinline__ int in_order(const RouterArgs& a, const L* row, float top, int e, int count) {
  const int lane = threadIdx.x & 63;
  const double rz = SIGMOID ? 1.0 : 1.0 / sum64(a, row, top);
  const double key = e >= 0 ? key64<SIGMOID>(a, load_logit(row, e), e, top, rz) : (double)NEG;
  int rank = lane < count ? 0 : lane;  // the others keep their places
#pragma unroll 1
  for (int o = 0; o < count; ++o) {
    const double k = __shfl(key, o, 64);
    const int i = __shfl(e, o, 64);
    rank += lane < count && (k > key || (k == key && i < e));
  }
  return __builtin_amdgcn_ds_permute(4 * rank, e);
}

// Steps 2 to 4 in fp32. nan: a key is NaN (the choice is then without meaning). sure: the groups that
// stay are those of the exact keys. error: the scores' bound.
template <int PER, bool SIGMOID, bool SCORED>
__device__ __forceinline__ Choice pick(const RouterArgs& a, const float (&x)[PER], float top, float* keys,
                                       bool near, bool& nan, bool& sure, float& error) {
  const int lane = threadIdx.x & 63;
  float key[PER];
  error = SIGMOID ? SIGMOID_ERROR : 0.0f;
  if constexpr (SCORED) {
    float rz = 1.0f;
    if constexpr (!SIGMOID) {
      rz = 1.0f / wave_sum(lane_sum<PER>([&](int j) { return fast_exp(x[j] - top); }));
      error = softmax_error<PER>(rz);
    }
    float bias[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) bias[j] = 0.0f;
    if (a.bias) {
#pragma unroll
      for (int j = 0; j < PER; ++j)
        if (64 * j + lane < a.E) bias[j] = a.bias[64 * j + lane];
    }
    bool none = false;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const float v = (SIGMOID ? __builtin_amdgcn_rcpf(1.0f + fast_exp(-x[j])) : fast_exp(x[j] - top) * rz) + bias[j];
      key[j] = x[j] > NEG ? v : NEG;
      none |= !(key[j] == key[j]);
    }
    nan = __ballot(none) != 0;
  } else {
#pragma unroll
    for (int j = 0; j < PER; ++j) key[j] = x[j];
    nan = false;
  }
  sure = true;
  if (a.groups > 1 && !nan) {
#pragma unroll
    for (int j = 0; j < PER; ++j)
      if (64 * j + lane < a.E) keys[64 * j + lane] = key[j];
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    const uint64_t kept = keep_groups<float>(a, keys, error, sure);
    if (!SCORED) sure = true;  // logits have no error
    const float inverse = 1.0f / (float)(a.E / a.groups);
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      if (SCORED && !a.bias) key[j] = x[j];
      // the group of e: e and the size are at most 2^12, so that (e + 1/2) / size falls on the right
      // side of every whole number
      const uint32_t g = (uint32_t)(((float)(64 * j + lane) + 0.5f) * inverse);
      if (!((kept >> (g & 63)) & 1) || 64 * j + lane >= a.E) key[j] = NEG;
    }
    __builtin_amdgcn_wave_barrier();
  }
  return choose<PER>(key, a.topk, near, error);
}

// SCORED: scores enter the choice (a bias, or groups by two scores); else it goes by the logits.
template <typename L, int PER, bool SIGMOID, bool SCORED>
__global__ __launch_bounds__(64 * ROUTE_WAVES) void expert_route_kernel(RouterArgs a) {
  extern __shared__ double row_keys[];  // [waves of the workgroup][E], with groups or scores only
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  const L* logits = static_cast<const L*>(a.logits);
  for (int64_t t = (int64_t)blockIdx.x * waves + w; t < a.T; t += (int64_t)gridDim.x * waves) {
    const L* row = logits + t * a.E;
    float x[PER];
    load_row(a, row, x);
    bool odd = false;
#pragma unroll
    for (int j = 0; j < PER; ++j) odd |= !(x[j] == x[j]) || (!SIGMOID && x[j] == -NEG);
    bool bad = __ballot(odd) != 0;
    float top = 0.0f;  // the softmax's largest logit; 0 in a row without experts
    if (!SIGMOID && (SCORED || !a.renorm)) {
      top = x[0];
#pragma unroll
      for (int j = 1; j < PER; ++j) top = fmaxf(top, x[j]);
      top = wave_max(top);
      top = top > NEG ? top : 0.0f;
    }
    int mine = -1;
    if (!bad) {
      double* keys = row_keys + (size_t)w * a.E;
      const bool near = SCORED && a.bias;
      bool sure;
      float error;
      const Choice c =
          pick<PER, SIGMOID, SCORED>(a, x, top, reinterpret_cast<float*>(keys), near, bad, sure, error);
      mine = c.e;
      if constexpr (SCORED) {
        bool again = false;
        if (near) {
          // lane r's key against the next one's
          const float below = __shfl_down(c.key, 1, 64);
          const float xe = mine >= 0 ? load_logit(row, mine) : 0.0f, be = mine >= 0 ? a.bias[mine] : 0.0f;
          const float xn = __shfl_down(xe, 1, 64), bn = __shfl_down(be, 1, 64);
          const bool apart = lane + 1 >= c.count || c.key - below > key_gap(c.key, error) || (xe == xn && be == bn);
          again = c.count > a.topk || __ballot(!apart) != 0;
        }
        if (!bad) {
          if (!sure || c.more)
            mine = choose64<L, SIGMOID>(a, row, top, keys);
          else if (again)
            mine = in_order<L, SIGMOID>(a, row, top, mine, c.count);
        }
        mine = lane < a.topk ? mine : -1;
      }
    }
    // the weights, slot r in lane r
    float weight = 0.0f, sum = 1.0f;
    const float xs = mine >= 0 ? load_logit(row, mine) : NEG;
    if (a.renorm) top = wave_max(xs);
    if constexpr (SIGMOID) {
      // e^min(x, 0) / (1 + e^-|x|), the numerator relative to the largest chosen one
      const float ref = a.renorm && top > NEG ? fminf(top, 0.0f) : 0.0f;
      if (mine >= 0) weight = expf(fminf(xs, 0.0f) - ref) / (1.0f + expf(-fabsf(xs)));
    } else if (mine >= 0) {
      weight = expf(xs - top);
    }
    if (a.renorm) {
      sum = wave_sum(weight);
    } else if constexpr (!SIGMOID) {
      sum = wave_sum(lane_sum<PER>([&](int j) { return fast_exp(x[j] - top); }));
    }
    if (lane < a.topk) {
      weight = mine >= 0 ? a.scale * (weight / sum) : 0.0f;
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
    const bool some = __ballot(id >= 0) != 0;
    const float dw = id >= 0 ? a.dw[t * a.topk + lane] : 0.0f;
    const float xs = id >= 0 ? load_logit(row, id) : NEG;
    const float most = wave_max(xs);
    float top = most, rz = 1.0f;
    const bool dense = !sigmoid && !a.renorm;
    float x[PER];  // logits, then their exponentials
    if (dense) {
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const int e = 64 * j + lane;
        x[j] = e < a.E ? load_logit(row, e) : NEG;
        top = fmaxf(top, x[j]);
      }
      top = wave_max(top);
      top = top > NEG ? top : 0.0f;
      // a NaN, or an infinity's, reaches the sum and so the whole row, also where all others are -inf
#pragma unroll
      for (int j = 0; j < PER; ++j) x[j] = fast_exp(x[j] - top);
      const float sum = wave_sum(lane_sum<PER>([&](int j) { return x[j]; }));
      rz = sum == 0.0f ? 0.0f : 1.0f / sum;  // a row without experts has only scores of 0
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
      c = wave_sum(id >= 0 ? expf(xs - top) * rz * g : 0.0f);
    }
    // slots of the same expert add up, in slot order
    float total = 0.0f;
    for (int k = 0; k < a.topk; ++k) {
      const int ik = __builtin_amdgcn_readlane(id, k);
      const float gk = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(g), k));
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
        if (dense) v = some ? x[j] * rz * (v - c) : 0.0f;
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
  const bool scored = a.bias || (a.groups > 1 && a.group_top == 2);
  const size_t row = backward ? sizeof(float) * a.E : a.groups > 1 || scored ? sizeof(double) * a.E : 0;
  const int waves = route_waves(row);
  const dim3 grid((unsigned)std::min<int64_t>((a.T + waves - 1) / waves, ROUTE_MAX_BLOCKS));
  const dim3 block(64 * waves);
  if (backward)
    hipLaunchKernelGGL((expert_route_backward_kernel<L, PER>), grid, block, row * waves, s, a);
  else if (a.sigmoid && scored)
    hipLaunchKernelGGL((expert_route_kernel<L, PER, true, true>), grid, block, row * waves, s, a);
  else if (a.sigmoid)
    hipLaunchKernelGGL((expert_route_kernel<L, PER, true, false>), grid, block, row * waves, s, a);
  else if (scored)
    hipLaunchKernelGGL((expert_route_kernel<L, PER, false, true>), grid, block, row * waves, s, a);
  else
    hipLaunchKernelGGL((expert_route_kernel<L, PER, false, false>), grid, block, row * waves, s, a);
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

// select.cuh -- expert selection and gate weights from router logits: softmax or sigmoid
// scores, a bias that steers the selection only, expert groups, top-k, renormalised weights.
//
//   s_e = 1 / (1 + exp(-l_e))  or  exp(l_e) / sum_f exp(l_f)          the score
//   c_e = s_e + b_e                                                   what the selection compares
//   group value = sum of the group's best one or two c; the best topk_groups groups stay
//   idx = the k largest c of the groups that stay, descending, ties to the lower index
//   w_j = s_idx[j], divided by their sum when renormalised, times weight_scale
//
// An expert whose logit is -inf or NaN, or whose c is -inf or NaN, is out: it is never selected.
//
// Order.  Without a bias the scores are ordered as the logits are, so the logits themselves are
// compared (exactly).  With a bias, or for sums of two scores, neighbours can be closer than the
// fp32 scores' error; there the fp32 order is taken only where every gap that matters is wider
// than twice a bound on that error (kScoreErr, kSumErr), and a row with a narrower gap is decided
// again from scores in 64 bits: the candidates alone where the groups are sure (order_candidates), else
// all experts (exact_order).
//
// One warp per token, E <= 256: lane l holds the experts l + 32 i.  The logits and choices of a
// token also sit in 2 KB of shared memory, so that a group (any E / n_groups consecutive
// experts) can be read by its own 32 / n_groups lanes.  A lane sorts its
// eight choices once, as integer keys whose low three bits hold the slot; a round of the selection is one
// redux.sync over the lanes' first keys, a ballot and a shift in the lane that won.  Keys that agree but for
// those three bits are told apart by a slower loop over the whole ones.
#pragma once

#include <cuda_bf16.h>

#include <cfloat>

#include "common.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace afd {

struct SelectArgs {
  const void* logits;      // [nsplit][T][ld] partial logits, added in split order
  const float* logit_bias; // [E] added to the logits, or nullptr
  const float* choice_bias;// [E] added to the scores for the selection only, or nullptr
  int32_t* idx;            // [T][k]
  float* w;                // [T][k]
  long long ld;            // elements between tokens
  int nsplit, T, E, k;
  int sigmoid, n_groups, topk_groups, group_best, renormalise;
  float weight_scale;
};

// Bounds on the fp32 scores' error, in steps of 2^-24 and against the largest score of the row.
// sigmoid 1 / (1 + z): expf's 2 ulp (4 steps) times z / (1 + z) <= 1, the addition 1, the division
// 1: 6 steps = 3.6e-7, taken as 4e-7.  softmax: the subtraction |l - max| exp(l - max) <= 0.4, expf 4, the
// sum's own terms 4 and their subtractions' mean under the softmax (|l - max| on average: at most 3.4 for 256
// experts, one at the maximum and the others 4.3 below), its 8 additions in a lane and 5 between
// lanes, the division 1: 26 steps = 1.55e-6, taken as 2e-6.  The sum with the bias rounds by 1 step of |c|, taken as 2.
constexpr float kSigmoidErr = 4e-7f, kSoftmaxErr = 2e-6f;
constexpr float kSumErr = 1.2e-7f;

// Order-preserving map of a float to an unsigned integer; 0 is below every number that can occur.
__device__ __forceinline__ unsigned order_key(float v) {
  const unsigned u = __float_as_uint(v + 0.f);  // -0 -> +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float order_value(unsigned key) {
  return __uint_as_float((key & 0x80000000u) ? (key ^ 0x80000000u) : ~key);
}
__device__ __forceinline__ unsigned long long order_key(double v) {
  const unsigned long long u = static_cast<unsigned long long>(__double_as_longlong(v + 0.0));
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}

__device__ __forceinline__ bool is_out(float c) { return !(c > -INFINITY); }   // -inf or NaN
__device__ __forceinline__ bool is_out(double c) { return !(c > -HUGE_VAL); }

// Which groups stay, as a bit mask: choice [E] in shared memory (out = -inf).  L = 32 / G lanes
// (G = n_groups rounded up to a power of two) read one group and keep its best two, merge by
// shuffles, and count the groups ahead of theirs.  *gap: the distance between the last group
// that stays and the first that does not (+inf where that border separates nothing).
template <typename V>
__device__ __forceinline__ unsigned groups_that_stay(const V* choice, const SelectArgs& a, int lane, V* gap) {
  const V ninf = -static_cast<V>(INFINITY);
  int G = 1;
  while (G < a.n_groups) G <<= 1;
  const int L = 32 / G, g = lane / L, sub = lane % L;
  const int S = a.E / a.n_groups;
  V b1 = ninf, b2 = ninf;
  if (g < a.n_groups) {
    for (int i = sub; i < S; i += L) {
      const V c = choice[g * S + i];
      b2 = c > b1 ? b1 : (c > b2 ? c : b2);
      b1 = c > b1 ? c : b1;
    }
  }
  for (int o = 1; o < L; o <<= 1) {
    const V o1 = __shfl_xor_sync(0xffffffffu, b1, o), o2 = __shfl_xor_sync(0xffffffffu, b2, o);
    const V hi = b1 > o1 ? b1 : o1, lo = b1 > o1 ? o1 : b1;
    const V s2 = b2 > o2 ? b2 : o2;
    b1 = hi;
    b2 = lo > s2 ? lo : s2;
  }
  // a group with one expert left is worth that one; a group with none comes last and never stays
  const V val = (a.group_best == 2 && b2 > ninf) ? b1 + b2 : b1;
  const bool any = b1 > ninf;
  int ahead = 0;
  for (int f = 0; f < a.n_groups; ++f) {
    const V ov = __shfl_sync(0xffffffffu, val, f * L);
    const bool oany = __shfl_sync(0xffffffffu, static_cast<int>(any), f * L) != 0;
    if (oany && (!any || ov > val || (ov == val && f < g))) ++ahead;
  }
  const bool stays = g < a.n_groups && any && ahead < a.topk_groups;
  const bool drops = g < a.n_groups && any && !stays;
  V lo = stays ? val : static_cast<V>(INFINITY), hi = drops ? val : ninf;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const V l = __shfl_xor_sync(0xffffffffu, lo, o), h = __shfl_xor_sync(0xffffffffu, hi, o);
    lo = l < lo ? l : lo;
    hi = h > hi ? h : hi;
  }
  *gap = hi > ninf ? lo - hi : static_cast<V>(INFINITY);
  const unsigned m = __ballot_sync(0xffffffffu, stays && sub == 0);  // bit g * L
  unsigned mask = 0;
  for (int f = 0; f < a.n_groups; ++f) mask |= ((m >> (f * L)) & 1u) << f;
  return mask;
}

// Decides one token in 64 bits; returns lane j's expert for j < k (-1: none left).  logits and
// scratch: the token's shared memory (scratch: E doubles).  Rare: a row with a gap inside the
// fp32 error.
__device__ __noinline__ int exact_order(const float* logits, double* scratch, const SelectArgs& a, int lane) {
  double c[8];
  float top = -INFINITY;
  for (int e = lane; e < a.E; e += 32) top = fmaxf(top, logits[e]);
  top = warp_max(top);
  double sum = 0.0;
  if (!a.sigmoid) {
    for (int e = lane; e < a.E; e += 32)
      if (logits[e] > -INFINITY) sum += exp(static_cast<double>(logits[e]) - top);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int e = lane + 32 * i;
    c[i] = -HUGE_VAL;
    if (e < a.E && logits[e] > -INFINITY) {
      const double l = logits[e];
      const double s = a.sigmoid ? 1.0 / (1.0 + exp(-l)) : exp(l - top) / sum;
      const double v = a.choice_bias ? s + static_cast<double>(a.choice_bias[e]) : s;
      if (!is_out(v)) c[i] = v;
    }
    if (e < a.E) scratch[e] = c[i];
  }
  __syncwarp();
  if (a.topk_groups < a.n_groups) {
    double gap;
    const unsigned mask = groups_that_stay(scratch, a, lane, &gap);
    const int S = a.E / a.n_groups;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = lane + 32 * i;
      if (e < a.E && !(mask >> (e / S) & 1u)) c[i] = -HUGE_VAL;
    }
  }
  if (!a.choice_bias) {  // inside the groups the scores are ordered as the logits are
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (!is_out(c[i])) c[i] = logits[lane + 32 * i];
  }
  unsigned long long key[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) key[i] = is_out(c[i]) ? 0ull : order_key(c[i]);
  int mine = -1;
  for (int j = 0; j < a.k; ++j) {
    unsigned long long m = 0ull;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = key[i] > m ? key[i] : m;
    const unsigned hi = __reduce_max_sync(0xffffffffu, static_cast<unsigned>(m >> 32));
    const unsigned lo = __reduce_max_sync(0xffffffffu, (m >> 32) == hi ? static_cast<unsigned>(m) : 0u);
    const unsigned long long best = (static_cast<unsigned long long>(hi) << 32) | lo;
    if (best == 0ull) break;  // uniform
    unsigned e = 0x7fffffffu;
#pragma unroll
    for (int i = 7; i >= 0; --i)
      if (key[i] == best) e = lane + 32 * i;
    e = __reduce_min_sync(0xffffffffu, e);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (e == static_cast<unsigned>(lane + 32 * i)) key[i] = 0ull;
    if (lane == j) mine = static_cast<int>(e);
  }
  return mine;
}

// The k best in 64 bits of n <= 32 candidates, one a lane (e), which hold them for certain; returns lane
// j's expert for j < k.  order: 32 ints of the warp's shared memory.
__device__ __forceinline__ int order_candidates(const float* logits, int* order, const SelectArgs& a, int lane, int n, int e,
                                                float top) {
  double sum = 1.0;
  if (!a.sigmoid) {
    sum = 0.0;
    for (int i = lane; i < a.E; i += 32)
      if (logits[i] > -INFINITY) sum += exp(static_cast<double>(logits[i]) - top);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  }
  double c = 0.0;
  if (lane < n) {
    const double l = logits[e];
    c = (a.sigmoid ? 1.0 / (1.0 + exp(-l)) : exp(l - top) / sum) + static_cast<double>(a.choice_bias[e]);
  }
  int rank = 0;
  for (int i = 0; i < n; ++i) {
    const double oc = __shfl_sync(0xffffffffu, c, i);
    const int oe = __shfl_sync(0xffffffffu, e, i);
    rank += oc > c || (oc == c && oe < e);
  }
  if (lane < n) order[rank] = e;
  __syncwarp();
  return lane < min(a.k, n) ? order[lane] : -1;
}

// 1 / (1 + exp(-l)); from where exp(-l) nears the end of fp32 on as exp(l), which it is to far more than fp32.
constexpr float kFarDown = -80.f;
__device__ __forceinline__ float sigmoid_of(float l) { return l < kFarDown ? expf(l) : 1.f / (1.f + expf(-l)); }

constexpr int kSelectWarps = 4;  // tokens per CTA

template <typename LT>
__global__ void __launch_bounds__(kSelectWarps * 32)
select_experts_kernel(const SelectArgs a) {
  launch_dependents();
  wait_dependency();
  __shared__ float s_logit[kSelectWarps][256];
  __shared__ double s_choice[kSelectWarps][256];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x * kSelectWarps + warp;
  if (t >= a.T) return;
  float* slog = s_logit[warp];
  float* schoice = reinterpret_cast<float*>(s_choice[warp]);

  float l[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) l[i] = 0.f;
  for (int sp = 0; sp < a.nsplit; ++sp) {
    const LT* row = static_cast<const LT*>(a.logits) + (static_cast<size_t>(sp) * a.T + t) * a.ld;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (lane + 32 * i < a.E) l[i] += static_cast<float>(row[lane + 32 * i]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int e = lane + 32 * i;
    float v = l[i];
    if (e < a.E) {
      if (a.logit_bias) v += a.logit_bias[e];
      v = is_out(v) ? -INFINITY : fminf(v, FLT_MAX);  // NaN and -inf: out; +inf as the largest number
      slog[e] = v;
    } else {
      v = -INFINITY;
    }
    l[i] = v;
  }
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = fmaxf(top, l[i]);
  top = warp_max(top);

  const bool grouped = a.topk_groups < a.n_groups;
  const bool by_logit = a.choice_bias == nullptr;             // selection by the logits themselves
  const bool need_score = !by_logit || (grouped && a.group_best == 2) || (!a.sigmoid && !a.renormalise);
  float s[8], sum = 1.f;
  if (need_score) {
    if (a.sigmoid) {
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = 1.f / (1.f + expf(-l[i]));
    } else {
      float z = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        s[i] = l[i] > -INFINITY ? expf(l[i] - top) : 0.f;
        z += s[i];
      }
      sum = warp_sum(z);
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = s[i] / sum;
    }
  }

  // choices, in fp32, and the bound on their error
  float c[8];
  float err = 0.f;
  if (!by_logit) {
    float bmax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = lane + 32 * i;
      c[i] = -INFINITY;
      if (l[i] > -INFINITY) {
        const float b = a.choice_bias[e];
        const float v = s[i] + b;
        if (!is_out(v)) {
          c[i] = v;
          if (fabsf(b) < INFINITY) bmax = fmaxf(bmax, fabsf(b));
        }
      }
    }
    bmax = warp_max(bmax);
    const float smax = a.sigmoid ? 1.f : 1.f / sum;
    err = (a.sigmoid ? kSigmoidErr : kSoftmaxErr) * smax + kSumErr * (smax + bmax);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = l[i];
  }

  bool sure = true;
  unsigned kept = 0xffffffffu;
  if (grouped) {
    const bool sums = a.group_best == 2;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = lane + 32 * i;
      if (e < a.E) schoice[e] = (by_logit && sums) ? (l[i] > -INFINITY ? s[i] : -INFINITY) : c[i];
    }
    __syncwarp();
    float gap;
    kept = groups_that_stay(schoice, a, lane, &gap);
    if (sums || !by_logit) {
      const float smax = a.sigmoid ? 1.f : 1.f / sum;
      const float one = by_logit ? ((a.sigmoid ? kSigmoidErr : kSoftmaxErr) + kSumErr) * smax : err;
      sure = gap > 6.f * one;  // two sums of two, and their own rounding
    }
    const int S = a.E / a.n_groups;
    const unsigned inv = 65536u / S + 1u;  // e / S for e < 256
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (!(kept >> (((lane + 32 * i) * inv) >> 16) & 1u)) c[i] = -INFINITY;
  }
  const bool groups_sure = sure;

  // the lane's choices, best first: the slot in the low bits, a lower one (a lower index) first
  unsigned key[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) key[i] = is_out(c[i]) ? 0u : (order_key(c[i]) & ~7u) | (7 - i);
  auto sort2 = [&](int x, int y) {
    const unsigned hi = max(key[x], key[y]), lo = min(key[x], key[y]);
    key[x] = hi;
    key[y] = lo;
  };
  sort2(0, 1); sort2(2, 3); sort2(4, 5); sort2(6, 7); sort2(0, 2); sort2(1, 3); sort2(4, 6); sort2(5, 7);
  sort2(1, 2); sort2(5, 6); sort2(0, 4); sort2(1, 5); sort2(2, 6); sort2(3, 7); sort2(2, 4); sort2(3, 5);
  sort2(1, 2); sort2(3, 4); sort2(5, 6);
  int mine = -1, n = 0;
  bool told_apart = true, border = true;  // no two keys agree but for the slot; all candidates are taken
  unsigned before = 0u;
  // bf16 logits: equal but for the slot is equal, and the slot and the lane are the index's order.
  // Else one round more, for the border; with a bias as many as it takes to leave the error behind.
  const bool exact_keys = by_logit && sizeof(LT) == 2 && a.logit_bias == nullptr && a.nsplit == 1;
  const int rounds = by_logit ? a.k + (exact_keys ? 0 : 1) : 33;
  for (int j = 0; j < rounds; ++j) {
    const unsigned best = __reduce_max_sync(0xffffffffu, key[0]);
    if (best == 0u) break;  // uniform: no expert is left
    const int winner = __ffs(__ballot_sync(0xffffffffu, key[0] == best)) - 1;
    if (!by_logit) {
      if (j > 0) {
        const float v = order_value(before & ~7u), u = order_value(best & ~7u);
        const bool apart = v - u > 2.f * err + 0x1p-19f * fmaxf(fabsf(v), fabsf(u));
        if (j >= a.k && apart) break;
        if (j == 32) {
          border = false;
          break;
        }
        sure = sure && apart;
      }
    } else if (!exact_keys && j > 0 && (before ^ best) < 8u) {
      told_apart = false;
    }
    before = best;
    if (lane == winner) {
#pragma unroll
      for (int i = 0; i < 7; ++i) key[i] = key[i + 1];
      key[7] = 0u;
    }
    if (lane == j) mine = winner + 32 * (7 - static_cast<int>(best & 7u));
    n = j + 1;
  }
  if (!told_apart) {  // again, by whole keys
    mine = -1;
#pragma unroll
    for (int i = 0; i < 8; ++i) key[i] = is_out(c[i]) ? 0u : order_key(c[i]);
    for (int j = 0; j < a.k; ++j) {
      unsigned m = 0u;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, key[i]);
      const unsigned best = __reduce_max_sync(0xffffffffu, m);
      if (best == 0u) break;
      unsigned e = 0x7fffffffu;
#pragma unroll
      for (int i = 7; i >= 0; --i)
        if (key[i] == best) e = lane + 32 * i;
      e = __reduce_min_sync(0xffffffffu, e);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (e == static_cast<unsigned>(lane + 32 * i)) key[i] = 0u;
      if (lane == j) mine = static_cast<int>(e);
    }
  }
  __syncwarp();  // slog is complete, schoice free again
  if (!sure || !border) {
    if (groups_sure && border && !by_logit)
      mine = order_candidates(slog, reinterpret_cast<int*>(s_choice[warp]), a, lane, n, mine, top);
    else
      mine = exact_order(slog, s_choice[warp], a, lane);
  }
  if (lane >= a.k) mine = -1;

  // gate weights
  const float lm = mine >= 0 ? slog[mine] : -INFINITY;
  float w = 0.f;
  if (a.renormalise) {
    const float lmax = warp_max(lm);
    // far down a sigmoid is exp(l) to more than fp32, and its ratios are those of exp(l - lmax)
    const bool ratio = !a.sigmoid || lmax < -40.f;
    if (mine >= 0) w = ratio ? expf(lm - lmax) : sigmoid_of(lm);
    const float z = warp_sum(w);
    // one far down beside a best that is not: its own score can be below fp32, its ratio to exp(lmax) is not
    if (!ratio && lm < kFarDown) {
      const float base = fminf(lmax, 0.f);
      w = expf(lm - base) * (expf(base) / z) * a.weight_scale;
    } else if (mine >= 0) {
      w = w / z * a.weight_scale;
    }
  } else if (mine >= 0) {
    w = (a.sigmoid ? sigmoid_of(lm) : expf(lm - top) / sum) * a.weight_scale;
  }
  if (lane < a.k) {
    a.idx[static_cast<size_t>(t) * a.k + lane] = mine;
    a.w[static_cast<size_t>(t) * a.k + lane] = w;
  }
}

template <typename LT>
inline void launch_select_experts(const SelectArgs& a, cudaStream_t s) {
  launch_dependent(select_experts_kernel<LT>, (a.T + kSelectWarps - 1) / kSelectWarps, kSelectWarps * 32, 0, s, a);
}

}  // namespace afd

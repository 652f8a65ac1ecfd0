// Routing of tokens to experts: scores, choice of the experts, weights; and the
// gradient of the weights with respect to the logits.
//
// Mathematics.  A token's logits x_e give scores s = softmax(x) or sigmoid(x).
// Experts are ranked by a key: the score plus the expert's bias, or, without a
// bias, the logit itself (the scores rise with it, and the logits keep apart
// what rounding a score would merge).  With expert groups, a group's score is its
// largest key or the sum of its two largest scores plus biases; only the experts
// of the best topk_groups groups take part.  The topk largest keys are chosen,
// equal keys by the lower number, and w_j = scale * s_j, or scale * s_j / sum s_i
// over the chosen.  Gradient, the choice held fixed, with ds_j = dL/ds_j:
//   plain:        ds_j = scale * g_j
//   renormalised: ds_j = scale * (g_j - sum_i g_i s_i / S) / S,  S = sum of the chosen scores
//   sigmoid:      dx_j = ds_j s_j (1 - s_j) on the chosen, 0 elsewhere
//   softmax:      dx_e = s_e (ds_e [chosen] - sum_j ds_j s_j) for every expert; renormalised,
//                 the sum vanishes and the scores' common denominator cancels, so only the
//                 chosen logits enter.
//
// All statistics are fp32.  Nothing but the logits (and at most one cache line
// of biases per row) is read and the chosen experts are written, so a large call
// is bound by that traffic and by the ranking's vector instructions, a small one
// by its launch.
//
// Layout.  A token belongs to kLanes lanes of one wave (16 up to 256 experts, so
// that a cross-lane maximum takes four DPP steps and serves four tokens at once;
// a whole wave beyond), each lane holding a run of kVals consecutive experts in
// registers: the run makes wide loads, and the lowest lane that holds the
// maximum holds the lowest expert number.
#include "elem_types.h"
#include "moe_internal.h"

namespace dgfp8 {
namespace {

constexpr int kThreads = 256;
constexpr int kNone = INT32_MIN;   // rank of an expert that cannot be chosen

// ---- cross-lane reductions over a token's kLanes lanes; every lane gets the result

template <int CTRL>
__device__ __forceinline__ int dpp(int v) {
  return __builtin_amdgcn_update_dpp(v, v, CTRL, 0xF, 0xF, false);
}
constexpr int kRowRor = 0x120;     // rotate right within a row of 16 lanes

template <int kLanes, class Op>
__device__ __forceinline__ int reduce(int v, Op op) {
  v = op(v, dpp<kRowRor + 8>(v));
  v = op(v, dpp<kRowRor + 4>(v));
  v = op(v, dpp<kRowRor + 2>(v));
  v = op(v, dpp<kRowRor + 1>(v));
  if constexpr (kLanes == 64) {
    v = op(v, __shfl_xor(v, 16, 64));
    v = op(v, __shfl_xor(v, 32, 64));
  }
  return v;
}
template <int kLanes>
__device__ __forceinline__ int max_lanes(int v) {
  return reduce<kLanes>(v, [](int a, int b) { return max(a, b); });
}
template <int kLanes>
__device__ __forceinline__ float sum_lanes(float v) {
  return __int_as_float(reduce<kLanes>(__float_as_int(v), [](int a, int b) {
    return __float_as_int(__int_as_float(a) + __int_as_float(b));
  }));
}
// Bits of a ballot that belong to this lane's token, lowest lane first.
template <int kLanes>
__device__ __forceinline__ uint64_t token_ballot(bool b) {
  const uint64_t m = __builtin_amdgcn_ballot_w64(b);
  if constexpr (kLanes == 64) return m;
  return (m >> (threadIdx.x & 48)) & 0xFFFFu;
}

// fp32 -> int of the same order (NaN excluded); + 0 makes -0 equal to 0.
__device__ __forceinline__ int rank_of(float v) {
  const int b = __float_as_int(v + 0.0f);
  return b ^ ((b >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float value_of(int r) { return __int_as_float(r ^ ((r >> 31) & 0x7FFFFFFF)); }

__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

// A lane's run of logits; experts past the last are -inf.  `wide`: rows start at
// 16-byte boundaries, so whole 16-byte pieces of a run load at once.
template <class T, int kVals>
__device__ __forceinline__ void load_run(const void* logits, int64_t row_off, int e0, int experts, bool wide,
                                         float (&x)[kVals]) {
  typedef typename T::store S;
  const S* src = (const S*)logits + row_off + e0;
  constexpr int kPer = 16 / sizeof(S) < kVals ? 16 / sizeof(S) : kVals;   // values of one wide load
#pragma unroll
  for (int c = 0; c < kVals; c += kPer) {
    if (kPer * sizeof(S) == 16 && wide && e0 + c + kPer <= experts) {
      const u32x4 v = *(const u32x4*)(src + c);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if constexpr (sizeof(S) == 4) {
          x[c + i] = __uint_as_float(v[i]);
        } else {
          x[c + i] = widen(T{}, (uint16_t)(v[i / 2] >> (16 * (i & 1))));
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        x[c + i] = e0 + c + i < experts ? widen(T{}, src[c + i]) : -__builtin_inff();
    }
  }
}

template <int kVals>
__device__ __forceinline__ int largest(const int (&v)[kVals]) {
  int m = v[0];
#pragma unroll
  for (int i = 1; i < kVals; ++i) m = max(m, v[i]);
  return m;
}

// LDS place of expert e's key: one word in 32 is skipped, so that lanes that walk
// groups of 32, 64, ... experts side by side meet different banks.
__device__ __forceinline__ int key_slot(int e) { return e + (e >> 5); }

template <class T, int kLanes, int kVals, bool kGroups>
__global__ void __launch_bounds__(kThreads) route_kernel(RouteParams p) {
  constexpr int kTokens = kThreads / kLanes;   // tokens of a workgroup
  constexpr int kKeys = kLanes * kVals + kLanes * kVals / 32;
  __shared__ float keys[kGroups ? kTokens * kKeys : 1];
  __shared__ float group_score[kGroups ? kTokens * kMaxExpertGroups : 1];
  __shared__ int chosen[kTokens * kMaxTopk];
  const int lane = threadIdx.x % kLanes;
  const int slot = threadIdx.x / kLanes;
  const int64_t token = (int64_t)blockIdx.x * kTokens + slot;
  const bool live = token < p.tokens;
  const int64_t row = (live ? token : p.tokens - 1) * p.ld;   // idle lanes redo the last token and write nothing
  const int e0 = lane * kVals;
  const bool wide = ((uintptr_t)p.logits & 15) == 0 && (p.ld * sizeof(typename T::store)) % 16 == 0;

  float x[kVals];
  load_run<T, kVals>(p.logits, row, e0, p.experts, wide, x);

  // ---- scores, where the ranking or the weights need all of them
  const bool softmax = p.score == DG_ROUTE_SOFTMAX;
  const bool need_scores = p.bias != nullptr || (kGroups && p.group_top2);
  bool nan = false;
  float top = -__builtin_inff();
#pragma unroll
  for (int i = 0; i < kVals; ++i) {
    // no score is defined beside these: the expert is not chosen, the row's weights are NaN
    const bool bad = x[i] != x[i] || (softmax && x[i] == __builtin_inff());
    nan |= bad;
    if (bad) x[i] = -__builtin_inff();
    top = fmaxf(top, x[i]);
  }
  nan = token_ballot<kLanes>(nan) != 0;
  float total = 1.0f;
  if (softmax && (need_scores || !p.renormalize)) {
    top = value_of(max_lanes<kLanes>(rank_of(top)));
    total = 0.0f;
#pragma unroll
    for (int i = 0; i < kVals; ++i) total += x[i] == -__builtin_inff() ? 0.0f : expf(x[i] - top);
    total = sum_lanes<kLanes>(total);
  }

  // ---- keys: rank[i] orders this lane's experts, kNone cannot be chosen
  int rank[kVals];
  float biased[kVals];   // score plus bias
#pragma unroll
  for (int i = 0; i < kVals; ++i) {
    float key = x[i];
    biased[i] = 0.0f;
    if (need_scores) {
      const float s = softmax ? expf(x[i] - top) / total : sigmoid(x[i]);
      biased[i] = p.bias && e0 + i < p.experts ? s + p.bias[e0 + i] : s;
      if (p.bias) key = biased[i];
    }
    if (p.bias) nan |= x[i] > -__builtin_inff() && key != key;
    const bool out = x[i] == -__builtin_inff() || key == -__builtin_inff() || key != key;
    rank[i] = out ? kNone : rank_of(key);
    if (out) biased[i] = -__builtin_inff();
  }
  if (p.bias) nan = token_ballot<kLanes>(nan) != 0;

  // ---- groups: lanes walk the groups' keys in LDS, then rank the groups by counting
  if constexpr (kGroups) {
    float* mine = keys + slot * kKeys;
    float* gscore = group_score + slot * kMaxExpertGroups;
    const int size = p.experts / p.groups;
#pragma unroll
    for (int i = 0; i < kVals; ++i)
      mine[key_slot(e0 + i)] =
          rank[i] == kNone ? -__builtin_inff() : (p.group_top2 ? biased[i] : value_of(rank[i]));
    wave_sync();
    for (int g = lane; g < p.groups; g += kLanes) {
      float a = -__builtin_inff(), b = -__builtin_inff();   // the two largest
      for (int e = g * size; e < (g + 1) * size; ++e) {
        const float v = mine[key_slot(e)];
        b = fmaxf(b, fminf(a, v));
        a = fmaxf(a, v);
      }
      gscore[g] = p.group_top2 && b > -__builtin_inff() ? a + b : a;
    }
    wave_sync();
    uint64_t keep = 0;   // bit g: group g takes part
    for (int g0 = 0; g0 < p.groups; g0 += kLanes) {
      const int g = g0 + lane;
      bool in = false;
      if (g < p.groups) {
        const float v = gscore[g];
        int before = 0;
        for (int h = 0; h < p.groups; ++h) {
          const float o = gscore[h];
          before += (o > v || (o == v && h < g)) ? 1 : 0;
        }
        in = before < p.topk_groups && v > -__builtin_inff();
      }
      keep |= token_ballot<kLanes>(in) << g0;
    }
    int g = e0 / size, in_group = e0 - g * size;
#pragma unroll
    for (int i = 0; i < kVals; ++i) {
      if (g >= p.groups || !((keep >> (g & 63)) & 1)) rank[i] = kNone;
      if (++in_group == size) {
        in_group = 0;
        ++g;
      }
    }
  }

  // ---- the topk largest, one after the other
  int* sel = chosen + slot * kMaxTopk;
  int mine_top = largest(rank);
  for (int j = 0; j < p.topk; ++j) {
    const int best = max_lanes<kLanes>(mine_top);
    const uint64_t holders = token_ballot<kLanes>(mine_top == best);
    const bool winner = lane == __builtin_ctzll(holders);
    int at = 0;
#pragma unroll
    for (int i = kVals - 1; i >= 0; --i) at = rank[i] == best ? i : at;
    if (winner) sel[j] = best == kNone ? -1 : e0 + at;
    at = winner ? at : -1;
#pragma unroll
    for (int i = 0; i < kVals; ++i) rank[i] = i == at ? kNone : rank[i];
    mine_top = largest(rank);
  }
  wave_sync();

  // ---- weights.  Renormalised softmax weights are the softmax over the chosen logits.
  const bool over_chosen = softmax && p.renormalize;
  if (over_chosen) {
    float m = -__builtin_inff();
    for (int j = lane; j < p.topk; j += kLanes)
      if (sel[j] >= 0) m = fmaxf(m, widen(T{}, ((const typename T::store*)p.logits)[row + sel[j]]));
    top = value_of(max_lanes<kLanes>(rank_of(m)));
  }
  float sum = 0.0f;
  float s0 = 0.0f;   // score of slot `lane`; later slots are computed again
  auto score_of = [&](int e) -> float {
    if (e < 0) return 0.0f;
    const float v = widen(T{}, ((const typename T::store*)p.logits)[row + e]);
    if (!softmax) return sigmoid(v);
    const float ex = expf(v - top);
    return over_chosen ? ex : ex / total;
  };
  for (int j = lane; j < p.topk; j += kLanes) {
    const float s = score_of(sel[j]);
    if (j == lane) s0 = s;
    sum += s;
  }
  if (p.renormalize) sum = sum_lanes<kLanes>(sum);
  if (!live) return;
  for (int j = lane; j < p.topk; j += kLanes) {
    const int e = sel[j];
    float w = j == lane ? s0 : score_of(e);
    if (p.renormalize) w = sum == 0.0f ? 0.0f : w / sum;
    w *= p.scale;
    if (nan) w = __builtin_nanf("");
    p.indices[token * p.ldi + j] = e;
    p.weights[token * p.ldw + j] = e < 0 ? 0.0f : w;
  }
}

// Gradient.  The chosen experts' parts are computed by one lane each and placed
// in the token's row in LDS; the lanes then write the row in whole runs.
template <class T, int kLanes, int kVals>
__global__ void __launch_bounds__(kThreads) route_grad_kernel(RouteGradParams p) {
  typedef typename T::store S;
  constexpr int kTokens = kThreads / kLanes;
  constexpr int kRow = kLanes * kVals;
  __shared__ __attribute__((aligned(16))) float part[kTokens * kRow];
  const int lane = threadIdx.x % kLanes;
  const int slot = threadIdx.x / kLanes;
  const int64_t token = (int64_t)blockIdx.x * kTokens + slot;
  const bool live = token < p.tokens;
  const int64_t t = live ? token : p.tokens - 1;
  const int64_t row = t * p.ld;
  const int e0 = lane * kVals;
  const bool softmax = p.score == DG_ROUTE_SOFTMAX;
  const bool dense = softmax && !p.renormalize;   // every expert of the row has a gradient

  float x[kVals];
  float top = -__builtin_inff(), total = 1.0f;
  if (dense) {
    const bool wide = ((uintptr_t)p.logits & 15) == 0 && (p.ld * sizeof(S)) % 16 == 0;
    load_run<T, kVals>(p.logits, row, e0, p.experts, wide, x);
    float m = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < kVals; ++i) m = fmaxf(m, x[i]);
    top = value_of(max_lanes<kLanes>(rank_of(m)));
    total = 0.0f;
#pragma unroll
    for (int i = 0; i < kVals; ++i) {
      x[i] = x[i] == -__builtin_inff() ? 0.0f : expf(x[i] - top);
      total += x[i];
    }
    total = sum_lanes<kLanes>(total);
  }
  float* mine = part + slot * kRow;
#pragma unroll
  for (int i = 0; i < kVals; ++i) mine[e0 + i] = 0.0f;

  auto expert_of = [&](int j) -> int {
    const int e = p.indices[t * p.ldi + j];
    return e >= 0 && e < p.experts ? e : -1;
  };
  auto logit_of = [&](int e) -> float { return widen(T{}, ((const S*)p.logits)[row + e]); };
  if (softmax && p.renormalize) {
    float m = -__builtin_inff();
    for (int j = lane; j < p.topk; j += kLanes) {
      const int e = expert_of(j);
      if (e >= 0) m = fmaxf(m, logit_of(e));
    }
    top = value_of(max_lanes<kLanes>(rank_of(m)));
  }
  auto score_of = [&](int e) -> float {
    const float v = logit_of(e);
    if (!softmax) return sigmoid(v);
    const float ex = expf(v - top);
    return dense ? ex / total : ex;
  };
  float sum = 0.0f, dot = 0.0f;   // of the chosen scores, and of gradient times score
  for (int j = lane; j < p.topk; j += kLanes) {
    const int e = expert_of(j);
    if (e < 0) continue;
    const float s = score_of(e);
    sum += s;
    dot += p.scale * p.dweights[t * p.ldw + j] * s;
  }
  if (p.renormalize || dense) {
    sum = sum_lanes<kLanes>(sum);
    dot = sum_lanes<kLanes>(dot);
  }
  wave_sync();
  for (int j = lane; j < p.topk; j += kLanes) {
    const int e = expert_of(j);
    if (e < 0) continue;
    const float s = score_of(e);
    float ds = p.scale * p.dweights[t * p.ldw + j];
    if (p.renormalize) ds = sum == 0.0f ? 0.0f : (ds - dot / sum) / sum;
    mine[e] = softmax ? ds * s : ds * s * (1.0f - s);
  }
  wave_sync();
  if (!live) return;
  float out[kVals];
#pragma unroll
  for (int i = 0; i < kVals; ++i) {
    out[i] = mine[e0 + i];
    if (dense && total > 0.0f) out[i] -= x[i] / total * dot;
  }
  S* dst = (S*)p.dlogits + t * p.ldd + e0;
  const bool wide_out = ((uintptr_t)p.dlogits & 15) == 0 && (p.ldd * sizeof(S)) % 16 == 0;
  constexpr int kPer = 16 / sizeof(S) < kVals ? 16 / sizeof(S) : kVals;
#pragma unroll
  for (int c = 0; c < kVals; c += kPer) {
    if (kPer * sizeof(S) == 16 && wide_out && e0 + c + kPer <= p.experts) {
      u32x4 v;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(S) == 4) {
          v[i] = __float_as_uint(out[c + i]);
        } else {
          v[i] = (uint32_t)narrow(T{}, out[c + 2 * i]) | ((uint32_t)narrow(T{}, out[c + 2 * i + 1]) << 16);
        }
      }
      *(u32x4*)(dst + c) = v;
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (e0 + c + i < p.experts) dst[c + i] = narrow(T{}, out[c + i]);
    }
  }
}

template <class T, int kLanes, int kVals>
hipError_t route_launch(const RouteParams& p, hipStream_t stream) {
  const int64_t grid = (p.tokens + kThreads / kLanes - 1) / (kThreads / kLanes);
  if (p.groups > 1) {
    hipLaunchKernelGGL((route_kernel<T, kLanes, kVals, true>), dim3((unsigned)grid), dim3(kThreads), 0, stream, p);
  } else {
    hipLaunchKernelGGL((route_kernel<T, kLanes, kVals, false>), dim3((unsigned)grid), dim3(kThreads), 0, stream, p);
  }
  return hipGetLastError();
}

template <class T, int kLanes, int kVals>
hipError_t grad_launch(const RouteGradParams& p, hipStream_t stream) {
  const int64_t grid = (p.tokens + kThreads / kLanes - 1) / (kThreads / kLanes);
  hipLaunchKernelGGL((route_grad_kernel<T, kLanes, kVals>), dim3((unsigned)grid), dim3(kThreads), 0, stream, p);
  return hipGetLastError();
}

// The smallest run that covers the experts.
template <class T>
hipError_t route_sized(const RouteParams& p, hipStream_t s) {
  if (p.experts <= 64) return route_launch<T, 16, 4>(p, s);
  if (p.experts <= 128) return route_launch<T, 16, 8>(p, s);
  if (p.experts <= 256) return route_launch<T, 16, 16>(p, s);
  return route_launch<T, 64, 16>(p, s);
}
template <class T>
hipError_t grad_sized(const RouteGradParams& p, hipStream_t s) {
  if (p.experts <= 64) return grad_launch<T, 16, 4>(p, s);
  if (p.experts <= 128) return grad_launch<T, 16, 8>(p, s);
  if (p.experts <= 256) return grad_launch<T, 16, 16>(p, s);
  return grad_launch<T, 64, 16>(p, s);
}

}  // namespace

hipError_t launch_route(const RouteParams& p, int dtype, hipStream_t s) {
  switch (dtype) {
    case DG_F32: return route_sized<F32>(p, s);
    case DG_BF16: return route_sized<BF16>(p, s);
    case DG_F16: return route_sized<F16>(p, s);
  }
  return hipErrorInvalidValue;
}

hipError_t launch_route_grad(const RouteGradParams& p, int dtype, hipStream_t s) {
  switch (dtype) {
    case DG_F32: return grad_sized<F32>(p, s);
    case DG_BF16: return grad_sized<BF16>(p, s);
    case DG_F16: return grad_sized<F16>(p, s);
  }
  return hipErrorInvalidValue;
}

}  // namespace dgfp8

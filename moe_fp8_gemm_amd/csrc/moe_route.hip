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
// Layout.  A token belongs to kLanes lanes of one wave, each lane holding a run of
// kVals consecutive experts in registers: the run makes wide loads, and lower
// lanes hold lower expert numbers.  16 lanes serve four tokens with each
// instruction; a whole wave takes the sizes that 16 lanes do not hold (over 256
// experts, or over 16 slots).
//
// Choice.  Instead of topk rounds of "find the maximum and take it out", a bound
// that at least topk keys reach is taken from the lanes' maxima; the few keys that
// reach it (about 11 of 256 for the top 8) are packed one to a lane, in
// order of expert number, and each lane counts how many come before its own: its slot.
// Where more than kLanes keys reach the bound it is raised by halving; where that
// does not help (equal keys) the rounds run after all.  Measured on 32768 x 256
// bf16 logits, top 8: 18.1 us with rounds alone, 10.4 us so; with sigmoid
// scores, a bias and 4 of 8 groups 24.6 us; one token 4.0 us.
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
__device__ __forceinline__ int min_lanes(int v) {
  return reduce<kLanes>(v, [](int a, int b) { return min(a, b); });
}
template <int kLanes>
__device__ __forceinline__ float sum_lanes(float v) {
  return __int_as_float(reduce<kLanes>(__float_as_int(v), [](int a, int b) {
    return __float_as_int(__int_as_float(a) + __int_as_float(b));
  }));
}
// Exclusive sum over the lower lanes of the token.
template <int kLanes>
__device__ __forceinline__ int sum_before(int v) {
  int s = v;   // lanes shifted in from outside the row add 0
  s += __builtin_amdgcn_update_dpp(0, s, 0x111, 0xF, 0xF, false);   // row_shr 1
  s += __builtin_amdgcn_update_dpp(0, s, 0x112, 0xF, 0xF, false);   // 2
  s += __builtin_amdgcn_update_dpp(0, s, 0x114, 0xF, 0xF, false);   // 4
  s += __builtin_amdgcn_update_dpp(0, s, 0x118, 0xF, 0xF, false);   // 8
  if constexpr (kLanes == 64) {
    s += __builtin_amdgcn_update_dpp(0, s, 0x142, 0xA, 0xF, false);   // last of rows 0, 2 to rows 1, 3
    s += __builtin_amdgcn_update_dpp(0, s, 0x143, 0xC, 0xF, false);   // last of row 1 to rows 2, 3
  }
  return s - v;
}
// Exchange with the lane whose number differs in one bit (within a row of 16), for
// reductions that join bits 1, 2, 4, 8 in this order.
template <int kBit>
__device__ __forceinline__ int swap_lanes(int v) {
  // the mirrors of 8 and 16 lanes stand for bits 4 and 8 once the lower bits are joined
  return dpp<kBit == 1 ? 0xB1 : kBit == 2 ? 0x4E : kBit == 4 ? 0x141 : 0x140>(v);
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

constexpr int kRankLow = (int)0x807FFFFF;    // rank of -inf: it, and what is below, cannot be chosen
constexpr int kRankHigh = 0x7F800000;        // rank of +inf; above are NaNs

__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

// Scores for the ranking.  Below 0 the argument's one rounding shows as |x| 2^-24 in the
// exponential, which the score keeps or dampens; the weights use expf.
constexpr float kLog2e = 1.44269504088896340736f;
__device__ __forceinline__ float exp_for_rank(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }
__device__ __forceinline__ float sigmoid_for_rank(float x) {
  return __builtin_amdgcn_rcpf(1.0f + exp_for_rank(-x));
}

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

// What a lane holds of the choice: the expert (-1: the slot stays empty), its logit, and
// its slot (topk or more: nothing).
struct Chosen {
  int expert, slot;
  float logit;
};

// The choice in topk rounds; any number of equal keys.
template <int kLanes, int kVals>
__device__ __forceinline__ Chosen choose_by_rounds(int (&rank)[kVals], const float (&x)[kVals], int lane, int e0,
                                                   int topk, int* experts, float* logits) {
  int mine = largest(rank);
  for (int j = 0; j < topk; ++j) {
    const int best = max_lanes<kLanes>(mine);
    const bool winner = lane == __builtin_ctzll(token_ballot<kLanes>(mine == best));
    int at = 0;
    float logit = 0.0f;
#pragma unroll
    for (int i = kVals - 1; i >= 0; --i)
      if (rank[i] == best) {
        at = i;
        logit = x[i];
      }
    if (winner) {
      experts[j] = best <= kRankLow ? -1 : e0 + at;
      logits[j] = logit;
    }
    at = winner ? at : -1;
#pragma unroll
    for (int i = 0; i < kVals; ++i) rank[i] = i == at ? kNone : rank[i];
    mine = largest(rank);
  }
  wave_sync();
  Chosen c{-1, kLanes, 0.0f};
  if (lane < topk) c = {experts[lane], lane, logits[lane]};
  return c;
}

template <int kLanes, int kVals>
__device__ __forceinline__ Chosen choose(int (&rank)[kVals], const float (&x)[kVals], int lane, int e0, int topk,
                                         int* experts, float* logits, int* ranks) {
  // ---- a bound that at least topk keys reach: the topk-th largest of 16 lane
  // maxima, or of a wave's lanes in as many groups as slots the least group maximum
  const int mine = largest(rank);
  int bound;
  if constexpr (kLanes == 16) {
    int above = 0;
    auto count = [&](int other) { above += other > mine ? 1 : 0; };
    count(dpp<kRowRor + 1>(mine)); count(dpp<kRowRor + 2>(mine)); count(dpp<kRowRor + 3>(mine));
    count(dpp<kRowRor + 4>(mine)); count(dpp<kRowRor + 5>(mine)); count(dpp<kRowRor + 6>(mine));
    count(dpp<kRowRor + 7>(mine)); count(dpp<kRowRor + 8>(mine)); count(dpp<kRowRor + 9>(mine));
    count(dpp<kRowRor + 10>(mine)); count(dpp<kRowRor + 11>(mine)); count(dpp<kRowRor + 12>(mine));
    count(dpp<kRowRor + 13>(mine)); count(dpp<kRowRor + 14>(mine)); count(dpp<kRowRor + 15>(mine));
    bound = min_lanes<kLanes>(above < topk ? mine : INT32_MAX);
  } else {
    int g = mine;   // maximum of this lane's group of 64 / 2^n >= topk lanes
    if (topk <= 32) g = max(g, swap_lanes<1>(g));
    if (topk <= 16) g = max(g, swap_lanes<2>(g));
    if (topk <= 8) g = max(g, swap_lanes<4>(g));
    if (topk <= 4) g = max(g, swap_lanes<8>(g));
    bound = min_lanes<kLanes>(g);
  }
  bound = max(bound, kRankLow + 1);

  // ---- the keys that reach it, one to a lane in order of expert number
  auto reach = [&](int b) {
    int n = 0;
#pragma unroll
    for (int i = 0; i < kVals; ++i) n += rank[i] >= b ? 1 : 0;
    return n;
  };
  int n = reach(bound);
  int at = sum_before<kLanes>(n);
  int total = max_lanes<kLanes>(at + n);
  // more than fit: halve the way to the largest key while at least topk reach the middle
  int over = max_lanes<kLanes>(mine);              // fewer than topk keys are above it, or none fits
  for (int pass = 0; pass < 8 && __builtin_amdgcn_ballot_w64(total > kLanes) != 0; ++pass) {
    const int mid = bound + (int)(((uint32_t)over - (uint32_t)bound + 1) >> 1);
    const int nm = reach(mid), am = sum_before<kLanes>(nm), tm = max_lanes<kLanes>(am + nm);
    if (total > kLanes) {
      if (tm >= topk) {
        bound = mid;
        n = nm;
        at = am;
        total = tm;
      } else {
        over = mid - 1;
      }
    }
  }
  if (__builtin_amdgcn_ballot_w64(total > kLanes) != 0)   // any token of the wave
    return choose_by_rounds<kLanes, kVals>(rank, x, lane, e0, topk, experts, logits);
  experts[lane] = -1;
  ranks[lane] = kNone;
  wave_sync();
#pragma unroll
  for (int i = 0; i < kVals; ++i)
    if (rank[i] >= bound) {
      experts[at] = e0 + i;
      ranks[at] = rank[i];
      logits[at] = x[i];
      ++at;
    }
  wave_sync();

  // ---- each lane counts the keys before its own: larger, or equal in a lower lane
  const int key = ranks[lane];
  int before = 0;
  if constexpr (kLanes == 16) {
    auto count = [&](int other, bool lower) { before += other > key || (other == key && lower) ? 1 : 0; };
    // row_ror r hands lane i the key of lane (i + 16 - r) % 16, which is lower where i >= r
    count(dpp<kRowRor + 1>(key), lane >= 1); count(dpp<kRowRor + 2>(key), lane >= 2);
    count(dpp<kRowRor + 3>(key), lane >= 3); count(dpp<kRowRor + 4>(key), lane >= 4);
    count(dpp<kRowRor + 5>(key), lane >= 5); count(dpp<kRowRor + 6>(key), lane >= 6);
    count(dpp<kRowRor + 7>(key), lane >= 7); count(dpp<kRowRor + 8>(key), lane >= 8);
    count(dpp<kRowRor + 9>(key), lane >= 9); count(dpp<kRowRor + 10>(key), lane >= 10);
    count(dpp<kRowRor + 11>(key), lane >= 11); count(dpp<kRowRor + 12>(key), lane >= 12);
    count(dpp<kRowRor + 13>(key), lane >= 13); count(dpp<kRowRor + 14>(key), lane >= 14);
    count(dpp<kRowRor + 15>(key), lane >= 15);
  } else {
    const int keys = __builtin_amdgcn_readfirstlane(total);
    for (int j = 0; j < keys; ++j) {
      const int other = __builtin_amdgcn_readlane(key, j);
      before += other > key || (other == key && j < lane) ? 1 : 0;
    }
  }
  // the lanes without a key stand behind all others, in order: they are the empty slots
  return {experts[lane], lane < total ? before : lane, logits[lane]};
}

template <class T, int kLanes, int kVals, bool kGroups>
__global__ void __launch_bounds__(kThreads) route_kernel(RouteParams p) {
  constexpr int kTokens = kThreads / kLanes;   // tokens of a workgroup
  constexpr int kKeys = kLanes * kVals + kLanes * kVals / 32;
  __shared__ int keys[kGroups ? kTokens * kKeys : 1];
  __shared__ __attribute__((aligned(16))) float group_score[kGroups ? kTokens * kMaxExpertGroups : 1];
  __shared__ int experts[kTokens * kLanes], ranks[kTokens * kLanes];
  __shared__ float logits[kTokens * kLanes];
  const int lane = threadIdx.x % kLanes;
  const int slot = threadIdx.x / kLanes;
  const int64_t token = (int64_t)blockIdx.x * kTokens + slot;
  const bool live = token < p.tokens;
  const int64_t row = (live ? token : p.tokens - 1) * p.ld;   // idle lanes redo the last token and write nothing
  const int e0 = lane * kVals;
  const bool wide = ((uintptr_t)p.logits & 15) == 0 && (p.ld * sizeof(typename T::store)) % 16 == 0;

  float x[kVals];
  load_run<T, kVals>(p.logits, row, e0, p.experts, wide, x);
  float bias[kVals];
  if (p.bias) load_run<F32, kVals>(p.bias, 0, e0, p.experts, ((uintptr_t)p.bias & 15) == 0, bias);

  // ---- logits without a score (NaN; +inf under softmax): taken out, and the
  // token's weights become NaN.  One look at the extremes of the ranks tells
  // whether a wave has any.
  const bool softmax = p.score == DG_ROUTE_SOFTMAX;
  const int limit = softmax ? kRankHigh - 1 : kRankHigh;
  int rank[kVals];
#pragma unroll
  for (int i = 0; i < kVals; ++i) rank[i] = rank_of(x[i]);
  int high = rank[0], low = rank[0];
#pragma unroll
  for (int i = 1; i < kVals; ++i) {
    high = max(high, rank[i]);
    low = min(low, rank[i]);
  }
  bool nan = high > limit || low < kRankLow;
  if (__builtin_amdgcn_ballot_w64(nan) != 0) {
#pragma unroll
    for (int i = 0; i < kVals; ++i)
      if (rank[i] > limit || rank[i] < kRankLow) {
        rank[i] = kRankLow;
        x[i] = -__builtin_inff();
      }
    nan = token_ballot<kLanes>(nan) != 0;
    high = largest(rank);
  }

  // ---- scores, where the ranking or the weights need all of them
  const bool need_scores = p.bias != nullptr || (kGroups && p.group_top2);
  float top = 0.0f, total = 1.0f;
  if (softmax && (need_scores || !p.renormalize)) {
    top = value_of(max_lanes<kLanes>(high));
    total = 0.0f;
#pragma unroll
    for (int i = 0; i < kVals; ++i) total += x[i] == -__builtin_inff() ? 0.0f : exp_for_rank(x[i] - top);
    total = sum_lanes<kLanes>(total);
  }

  // ---- keys: with a bias, or for the groups' sums, scores take the logits' place
  int group_rank[kGroups ? kVals : 1];   // what the groups go by
  if (need_scores) {
    const float inv = 1.0f / total;
#pragma unroll
    for (int i = 0; i < kVals; ++i) {
      float key = softmax ? exp_for_rank(x[i] - top) * inv : sigmoid_for_rank(x[i]);
      if (p.bias) key += bias[i];
      const bool in = x[i] != -__builtin_inff();
      if (p.bias) {
        nan |= in && key != key;
        rank[i] = in && key == key ? rank_of(key) : kRankLow;
      }
      if constexpr (kGroups) group_rank[i] = in && key == key ? rank_of(key) : kRankLow;
    }
    if (p.bias) nan = token_ballot<kLanes>(nan) != 0;
  }

  // ---- groups: their largest and second largest keys, then the groups are ranked
  // by counting
  if constexpr (kGroups) {
    float* gscore = group_score + slot * kMaxExpertGroups;
    const int size = p.experts / p.groups;
    if (!p.group_top2) {
#pragma unroll
      for (int i = 0; i < kVals; ++i) group_rank[i] = rank[i];
    }
    for (int g = lane; g < kMaxExpertGroups; g += kLanes) gscore[g] = -__builtin_inff();
    wave_sync();
    int a = kRankLow, b = kRankLow;   // the two largest, a >= b
    auto take = [&](int v) {
      b = max(min(a, v), b);   // the middle one of the three
      a = max(a, v);
    };
    auto join = [&](int a2, int b2) {
      b = max(min(a, a2), max(b, b2));
      a = max(a, a2);
    };
    auto join_lanes = [&](int lanes) {   // over runs of `lanes` lanes (1, 2, 4, 8 or 16)
      if (lanes >= 2) join(swap_lanes<1>(a), swap_lanes<1>(b));
      if (lanes >= 4) join(swap_lanes<2>(a), swap_lanes<2>(b));
      if (lanes >= 8) join(swap_lanes<4>(a), swap_lanes<4>(b));
      if (lanes >= 16) join(swap_lanes<8>(a), swap_lanes<8>(b));
    };
    auto put = [&](int g) {
      gscore[g] = p.group_top2 && b > kRankLow ? value_of(a) + value_of(b) : value_of(a);
    };
    // a group is a run of whole lanes where its size is kVals times a power of two;
    // other sizes go through LDS, where as many lanes as there are share a group's keys
    const int run = size / kVals;
    const bool whole = size % kVals == 0 && run <= 16 && (run & (run - 1)) == 0;
    if (whole) {
#pragma unroll
      for (int i = 0; i < kVals; ++i) take(group_rank[i]);
      join_lanes(run);
      if (e0 < p.experts && lane % run == 0) put(lane / run);
    } else {
      int* mine = keys + slot * kKeys;
#pragma unroll
      for (int i = 0; i < kVals; ++i) mine[key_slot(e0 + i)] = group_rank[i];
      wave_sync();
      const int share = p.groups * 8 <= kLanes ? 8 : p.groups * 4 <= kLanes ? 4 : p.groups * 2 <= kLanes ? 2 : 1;
      for (int g0 = 0; g0 < p.groups; g0 += kLanes) {   // more than one pass only past kLanes groups
        const int g = g0 + lane / share;
        a = b = kRankLow;
        if (g < p.groups) {
#pragma unroll 4
          for (int e = lane % share; e < size; e += share) take(mine[key_slot(g * size + e)]);
        }
        join_lanes(share);
        if (g < p.groups && lane % share == 0) put(g);
      }
    }
    wave_sync();
    uint64_t keep = 0;   // bit g: group g takes part
    for (int g0 = 0; g0 < p.groups; g0 += kLanes) {
      const int g = g0 + lane;
      const float v = g < p.groups ? gscore[g] : -__builtin_inff();
      int before = 0;
      for (int h = 0; h < p.groups; h += 4) {   // entries past the last group are -inf
        typedef float f32x4 __attribute__((ext_vector_type(4)));
        const f32x4 o = *(const f32x4*)(gscore + h);
#pragma unroll
        for (int i = 0; i < 4; ++i) before += (o[i] > v || (o[i] == v && h + i < g)) ? 1 : 0;
      }
      keep |= token_ballot<kLanes>(before < p.topk_groups && v > -__builtin_inff()) << g0;
    }
    if (whole) {
      const bool in = e0 < p.experts && ((keep >> (lane / run)) & 1) != 0;
#pragma unroll
      for (int i = 0; i < kVals; ++i) rank[i] = in ? rank[i] : kRankLow;
    } else {
      int g = e0 / size, in_group = e0 - g * size;
#pragma unroll
      for (int i = 0; i < kVals; ++i) {
        if (g >= p.groups || !((keep >> (g & 63)) & 1)) rank[i] = kRankLow;
        if (++in_group == size) {
          in_group = 0;
          ++g;
        }
      }
    }
  }

  const Chosen c = choose<kLanes, kVals>(rank, x, lane, e0, p.topk, experts + slot * kLanes, logits + slot * kLanes,
                                         ranks + slot * kLanes);
  const bool filled = c.slot < p.topk && c.expert >= 0;

  // ---- weights.  Renormalised softmax weights are the softmax over the chosen logits.
  float w = 0.0f;
  if (softmax && p.renormalize) {
    const float m = value_of(max_lanes<kLanes>(rank_of(filled ? c.logit : -__builtin_inff())));
    w = filled ? expf(c.logit - m) : 0.0f;
  } else if (filled) {
    w = softmax ? expf(c.logit - top) / total : sigmoid(c.logit);
  }
  if (p.renormalize) {
    const float sum = sum_lanes<kLanes>(w);
    w = sum == 0.0f ? 0.0f : w / sum;
  }
  if (!live || c.slot >= p.topk) return;
  p.indices[token * p.ldi + c.slot] = c.expert;
  p.weights[token * p.ldw + c.slot] = c.expert < 0 ? 0.0f : nan ? __builtin_nanf("") : w * p.scale;
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

// 16 lanes for a token where they hold it, with the smallest run that covers the
// experts; a wave otherwise.  (A wave per token is no faster on few tokens either: 1
// token of 256 experts, top 8: 4.2 us to 4.0; with a bias and 8 groups 8.2 to 7.8.)
template <class T>
hipError_t route_sized(const RouteParams& p, hipStream_t s) {
  if (p.experts > 256) return route_launch<T, 64, 16>(p, s);
  if (p.topk > 16) return route_launch<T, 64, 4>(p, s);
  if (p.experts <= 64) return route_launch<T, 16, 4>(p, s);
  if (p.experts <= 128) return route_launch<T, 16, 8>(p, s);
  return route_launch<T, 16, 16>(p, s);
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

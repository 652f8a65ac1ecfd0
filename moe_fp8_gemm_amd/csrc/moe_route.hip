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
// instruction; a whole wave takes few tokens, where its shorter chain of instructions
// counts, and the sizes that 16 lanes do not hold (over 256 experts, or over 16 slots).
//
// Choice.  Instead of topk rounds of "find the maximum and take it out", a bound
// that at least topk keys reach is taken from 16 maxima; the few keys that
// reach it (about 11 of 256 for the top 8) are packed one to a lane, in
// order of expert number, and each lane counts how many come before its own: its slot.
// Where more than kLanes keys reach the bound it is raised by halving; where that
// does not help (equal keys) the rounds run after all.  Every step is written for all
// values at once and without branches: a lone wave's time is its chain of
// instructions at 7 to 8 cycles each.  Measured on 32768 x 256 bf16 logits, top 8, in a graph
// that goes through eight inputs: 18.1 us with rounds alone, 9.2 us so (16.8 MB; the vector
// instructions bound it; 8.4 us where two inputs take turns); with sigmoid scores, a bias and 4
// of 8 groups of fp32 logits 20 us; one token 2.6 and 3.8 us.
#include "elem_types.h"
#include "moe_internal.h"

namespace dgfp8 {
namespace {

constexpr int kThreads = 256;
constexpr int kNone = INT32_MIN;   // rank of an expert that cannot be chosen

// ---- cross-lane reductions over a token's kLanes lanes; every lane gets the result

template <int CTRL>
__device__ __forceinline__ int dpp(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, true);   // every lane has a source
}
constexpr int kRowRor = 0x120;     // rotate right within a row of 16 lanes
constexpr int kRowLast = 0x15F;    // the value of a row's last lane

// Over the lanes of the same place in a wave's four rows of 16.
template <class Op>
__device__ __forceinline__ int join_rows(int v, Op op) {
  const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);   // even rows' values, odd rows' values
  v = op((int)a[0], (int)a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);   // lower half's, upper half's
  return op((int)b[0], (int)b[1]);
}
template <int kLanes, class Op>
__device__ __forceinline__ int reduce(int v, Op op) {
  v = op(v, dpp<kRowRor + 8>(v));
  v = op(v, dpp<kRowRor + 4>(v));
  v = op(v, dpp<kRowRor + 2>(v));
  v = op(v, dpp<kRowRor + 1>(v));
  if constexpr (kLanes == 64) v = join_rows(v, op);
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

// Values of a lane's run that load at once.
template <class T, int kVals>
constexpr int kPiece = 16 / sizeof(typename T::store) < kVals ? 16 / sizeof(typename T::store) : kVals;   // values
// A lane's kVals logits, -inf past the last expert: piece c of kPer values (8 or 16
// bytes) begins at expert e0 + c * step.  `wide`: rows start at 16-byte boundaries.  Where
// the experts fill whole pieces they load at once.  What lies past the end loads the
// row's first instead, so that no lane goes another way and all loads are in flight
// together.
template <class T, int kVals, int kPer>
__device__ __forceinline__ void load_logits(const void* logits, int64_t row_off, int e0, int step, int experts,
                                            bool wide, float (&x)[kVals]) {
  typedef typename T::store S;
  const S* row = (const S*)logits + row_off;
  if (wide && experts % kPer == 0) {
    typedef uint32_t words __attribute__((ext_vector_type(kPer * sizeof(S) / 4)));
    words v[kVals / kPer];
#pragma unroll
    for (int c = 0; c < kVals / kPer; ++c) v[c] = *(const words*)(row + (e0 + c * step < experts ? e0 + c * step : 0));
#pragma unroll
    for (int i = 0; i < kVals; ++i) {
      const int c = i / kPer, o = i % kPer;
      float f;
      if constexpr (sizeof(S) == 4) {
        f = __uint_as_float(v[c][o]);
      } else {
        f = widen(T{}, (uint16_t)(v[c][o / 2] >> (16 * (o & 1))));
      }
      x[i] = e0 + c * step < experts ? f : -__builtin_inff();
    }
  } else {
#pragma unroll
    for (int i = 0; i < kVals; ++i) {
      const int e = e0 + i / kPer * step + i % kPer;
      const float f = widen(T{}, row[e < experts ? e : 0]);
      x[i] = e < experts ? f : -__builtin_inff();
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

// Words of a token's list of keys: expert numbers, ranks, logits, each with as many places
// for what is not listed.
template <int kLanes>
constexpr int kFound = 2 * kLanes;

// What a lane holds of the choice: the expert (-1: the slot stays empty), its logit, and
// its slot (topk or more: nothing).
struct Chosen {
  int expert, slot;
  float logit;
};

// The choice in topk rounds; any number of equal keys.
template <int kLanes, int kVals>
__device__ __forceinline__ Chosen choose_by_rounds(int (&rank)[kVals], const float (&x)[kVals], int lane, int e0,
                                                   int topk, int* experts, int* logits) {
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
      logits[j] = __float_as_int(logit);
    }
    at = winner ? at : -1;
#pragma unroll
    for (int i = 0; i < kVals; ++i) rank[i] = i == at ? kNone : rank[i];
    mine = largest(rank);
  }
  wave_sync();
  Chosen c{-1, kLanes, 0.0f};
  if (lane < topk) c = {experts[lane], lane, __int_as_float(logits[lane])};
  return c;
}

template <int kLanes, int kVals>
__device__ __forceinline__ Chosen choose(int (&rank)[kVals], const float (&x)[kVals], int lane, int e0, int topk,
                                         int* found) {
  // ---- a bound that at least topk keys reach: the topk-th largest of 16 maxima (of a
  // lane each, or of four lanes of a wave); past 16 slots the least maximum of the wave's
  // lanes, or pairs of them
  const int mine = largest(rank);
  int bound;
  if (kLanes == 16 || topk <= 16) {
    const int m = kLanes == 16 ? mine : join_rows(mine, [](int a, int b) { return max(a, b); });
    int above = 0;
    auto count = [&](int other) { above += other > m ? 1 : 0; };
    count(dpp<kRowRor + 1>(m)); count(dpp<kRowRor + 2>(m)); count(dpp<kRowRor + 3>(m));
    count(dpp<kRowRor + 4>(m)); count(dpp<kRowRor + 5>(m)); count(dpp<kRowRor + 6>(m));
    count(dpp<kRowRor + 7>(m)); count(dpp<kRowRor + 8>(m)); count(dpp<kRowRor + 9>(m));
    count(dpp<kRowRor + 10>(m)); count(dpp<kRowRor + 11>(m)); count(dpp<kRowRor + 12>(m));
    count(dpp<kRowRor + 13>(m)); count(dpp<kRowRor + 14>(m)); count(dpp<kRowRor + 15>(m));
    bound = min_lanes<16>(above < topk ? m : INT32_MAX);   // every row has the same
  } else {
    bound = min_lanes<kLanes>(topk <= 32 ? max(mine, swap_lanes<1>(mine)) : mine);
  }
  bound = max(bound, kRankLow + 1);

  // ---- the keys that reach it, one to a lane in order of expert number
  auto reach = [&](int b) {
    int n = 0;
#pragma unroll
    for (int i = 0; i < kVals; ++i) n += rank[i] >= b ? 1 : 0;
    return n;
  };
  auto sum = [&](int before_and_own) {
    return kLanes == 16 ? dpp<kRowLast>(before_and_own) : __builtin_amdgcn_readlane(before_and_own, 63);
  };
  int n = reach(bound);
  int at = sum_before<kLanes>(n);
  int total = sum(at + n);
  if (__builtin_amdgcn_ballot_w64(total > kLanes) != 0) {
    // more than fit: halve the way to the largest key while at least topk reach the middle
    int over = max_lanes<kLanes>(mine);              // fewer than topk keys are above it, or none fits
    for (int pass = 0; pass < 8 && __builtin_amdgcn_ballot_w64(total > kLanes) != 0; ++pass) {
      const int mid = bound + (int)(((uint32_t)over - (uint32_t)bound + 1) >> 1);
      const int nm = reach(mid), am = sum_before<kLanes>(nm), tm = sum(am + nm);
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
      return choose_by_rounds<kLanes, kVals>(rank, x, lane, e0, topk, found, found + 2 * kFound<kLanes>);
  }
  // every lane writes every value, those below the bound to a place of its own that
  // nobody reads: no branches, which would cost more than the writes
  int* const ranks = found + kFound<kLanes>;
  int* const logits = ranks + kFound<kLanes>;
#pragma unroll
  for (int i = 0; i < kVals; ++i) {
    const bool in = rank[i] >= bound;
    const int to = in ? at : kLanes + lane;
    found[to] = e0 + i;
    ranks[to] = rank[i];
    logits[to] = __float_as_int(x[i]);
    at += in ? 1 : 0;
  }
  wave_sync();

  // ---- each lane counts the keys before its own: larger, or equal in a lower lane
  const bool listed = lane < total;
  const int key = listed ? ranks[lane] : kNone;
  int before = 0;
  const int keys = kLanes == 64 ? __builtin_amdgcn_readfirstlane(total) : 0;
  if (kLanes == 16 || keys <= 16) {   // a row of lanes holds them
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
    for (int j = 0; j < keys; ++j) {
      const int other = __builtin_amdgcn_readlane(key, j);
      before += other > key || (other == key && j < lane) ? 1 : 0;
    }
  }
  // the lanes without a key stand behind all others, in order: they are the empty slots
  return {listed ? found[lane] : -1, listed ? before : lane, __int_as_float(logits[lane])};
}

template <class T, int kLanes, int kVals, bool kGroups>
__global__ void __launch_bounds__(kThreads) route_kernel(RouteParams p) {
  constexpr int kTokens = kThreads / kLanes;   // tokens of a workgroup
  constexpr int kKeys = kLanes * kVals + kLanes * kVals / 32;
  __shared__ int keys[kGroups ? kTokens * kKeys : 1];
  __shared__ __attribute__((aligned(16))) float group_score[kGroups ? kTokens * kMaxExpertGroups : 1];
  __shared__ int found[kTokens * 3 * kFound<kLanes>];
  const int lane = threadIdx.x % kLanes;
  const int slot = threadIdx.x / kLanes;
  const int64_t token = (int64_t)blockIdx.x * kTokens + slot;
  const bool live = token < p.tokens;
  const int64_t row = (live ? token : p.tokens - 1) * p.ld;   // idle lanes redo the last token and write nothing
  const int e0 = lane * kVals;
  const bool wide = ((uintptr_t)p.logits & 15) == 0 && (p.ld * sizeof(typename T::store)) % 16 == 0;

  float x[kVals];
  load_logits<T, kVals, kPiece<T, kVals>>(p.logits, row, e0, kPiece<T, kVals>, p.experts, wide, x);
  float bias[kVals];
  if (p.bias)
    load_logits<F32, kVals, 4>(p.bias, 0, e0, 4, p.experts, ((uintptr_t)p.bias & 15) == 0, bias);

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
    // one decision at a time for all values, so that their chains overlap
    float key[kVals];
    if (softmax) {
      const float inv = 1.0f / total;
#pragma unroll
      for (int i = 0; i < kVals; ++i) key[i] = exp_for_rank(x[i] - top) * inv;
    } else {
#pragma unroll
      for (int i = 0; i < kVals; ++i) key[i] = sigmoid_for_rank(x[i]);
    }
    if (p.bias) {
#pragma unroll
      for (int i = 0; i < kVals; ++i) key[i] += bias[i];
    }
    bool lost = false;   // a NaN key of an expert with a score (from the bias)
    int key_rank[kVals];
#pragma unroll
    for (int i = 0; i < kVals; ++i) {
      const bool in = x[i] != -__builtin_inff(), number = key[i] == key[i];
      lost |= in && !number;
      key_rank[i] = in && number ? rank_of(key[i]) : kRankLow;
    }
    if constexpr (kGroups) {
#pragma unroll
      for (int i = 0; i < kVals; ++i) group_rank[i] = key_rank[i];
    }
    if (p.bias) {
#pragma unroll
      for (int i = 0; i < kVals; ++i) rank[i] = key_rank[i];
      nan |= lost;
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
    // sums are halved: of the same order, and two of the largest numbers stay in fp32's range
    auto put = [&](int g) {
      const float half = 0.5f * value_of(a);
      gscore[g] = !p.group_top2 ? value_of(a) : b > kRankLow ? half + 0.5f * value_of(b) : half;
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

  const Chosen c = choose<kLanes, kVals>(rank, x, lane, e0, p.topk, found + slot * 3 * kFound<kLanes>);
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
  // pieces of 4 experts, kLanes apart: a token's lanes meet whole lines, and the sums'
  // order is that of every type
  constexpr int kPer = 4;
  const int e0 = lane * kPer;
  const bool softmax = p.score == DG_ROUTE_SOFTMAX;
  const bool dense = softmax && !p.renormalize;   // every expert of the row has a gradient

  // every load first: the row's logits, then this lane's slots and their logits
  float x[kVals];
  if (dense) {
    const bool wide = ((uintptr_t)p.logits & 15) == 0 && (p.ld * sizeof(S)) % 16 == 0;
    load_logits<T, kVals, kPer>(p.logits, row, e0, kLanes * kPer, p.experts, wide, x);
  }
  constexpr int kSlots = 64 / kLanes;   // of a lane: slots lane, lane + kLanes, ...
  int chosen[kSlots];                   // -1: none
  float logit[kSlots], g[kSlots];
#pragma unroll
  for (int k = 0; k < kSlots; ++k) {
    chosen[k] = -1;
    logit[k] = g[k] = 0.0f;
    if (k > 0 && k * kLanes >= p.topk) continue;
    const int j = lane + k * kLanes, at = j < p.topk ? j : 0;
    const int e = p.indices[t * p.ldi + at];
    g[k] = p.scale * p.dweights[t * p.ldw + at];
    chosen[k] = j < p.topk && e >= 0 && e < p.experts ? e : -1;
  }
#pragma unroll
  for (int k = 0; k < kSlots; ++k)
    if (k == 0 || k * kLanes < p.topk) logit[k] = widen(T{}, ((const S*)p.logits)[row + (chosen[k] < 0 ? 0 : chosen[k])]);

  float* mine = part + slot * kRow;
#pragma unroll
  for (int i = 0; i < kVals; ++i) mine[e0 + i / kPer * kLanes * kPer + i % kPer] = 0.0f;

  float top = -__builtin_inff(), total = 1.0f;
  if (softmax) {   // over the row, or renormalised over the chosen
    float m = -__builtin_inff();
    if (dense) {
#pragma unroll
      for (int i = 0; i < kVals; ++i) m = fmaxf(m, x[i]);
    } else {
#pragma unroll
      for (int k = 0; k < kSlots; ++k)
        if (chosen[k] >= 0) m = fmaxf(m, logit[k]);
    }
    top = value_of(max_lanes<kLanes>(rank_of(m)));
  }
  if (dense) {
    total = 0.0f;
#pragma unroll
    for (int i = 0; i < kVals; ++i) {
      x[i] = x[i] == -__builtin_inff() ? 0.0f : expf(x[i] - top);
      total += x[i];
    }
    total = sum_lanes<kLanes>(total);
  }
  const float inv = 1.0f / total;
  float sum = 0.0f, dot = 0.0f;   // of the chosen scores, and of gradient times score
  float score[kSlots];
#pragma unroll
  for (int k = 0; k < kSlots; ++k) {
    score[k] = 0.0f;
    if (chosen[k] < 0) continue;
    score[k] = softmax ? expf(logit[k] - top) * inv : sigmoid(logit[k]);
    sum += score[k];
    dot += g[k] * score[k];
  }
  if (p.renormalize || dense) {
    sum = sum_lanes<kLanes>(sum);
    dot = sum_lanes<kLanes>(dot);
  }
  wave_sync();
#pragma unroll
  for (int k = 0; k < kSlots; ++k) {
    if (chosen[k] < 0) continue;
    float dx = g[k] * score[k];
    // shares before gradients: the sum may be subnormal, and its reciprocal out of range
    if (p.renormalize) dx = sum == 0.0f ? 0.0f : (g[k] - dot / sum) * (score[k] / sum);
    mine[chosen[k]] = softmax ? dx : dx * (1.0f - score[k]);
  }
  wave_sync();
  if (!live) return;
  float out[kVals];
#pragma unroll
  for (int i = 0; i < kVals; ++i) out[i] = mine[e0 + i / kPer * kLanes * kPer + i % kPer];
  if (dense && total != 0.0f) {   // 0: no expert has a score; NaN (from the logits): no gradient is known
    const float share = inv * dot;
#pragma unroll
    for (int i = 0; i < kVals; ++i) out[i] -= x[i] * share;
  }
  S* dst = (S*)p.dlogits + t * p.ldd;
  const bool wide_out = ((uintptr_t)p.dlogits & 15) == 0 && (p.ldd * sizeof(S)) % 16 == 0;
#pragma unroll
  for (int c = 0; c < kVals / kPer; ++c) {
    const int e = e0 + c * kLanes * kPer;
    if (wide_out && e + kPer <= p.experts) {
      typedef uint32_t words __attribute__((ext_vector_type(kPer * sizeof(S) / 4)));
      words v;
#pragma unroll
      for (int i = 0; i < (int)(kPer * sizeof(S) / 4); ++i) {
        if constexpr (sizeof(S) == 4) {
          v[i] = __float_as_uint(out[c * kPer + i]);
        } else {
          v[i] = (uint32_t)narrow(T{}, out[c * kPer + 2 * i]) | ((uint32_t)narrow(T{}, out[c * kPer + 2 * i + 1]) << 16);
        }
      }
      *(words*)(dst + e) = v;
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (e + i < p.experts) dst[e + i] = narrow(T{}, out[c * kPer + i]);
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

// 16 lanes for a token where they hold it, with the smallest run that covers the experts,
// when the calls' waves fill the device.  With few tokens each wave's own chain of
// instructions is what takes time, and a whole wave per token has a quarter of them per
// lane (us, a wave to 16 lanes; 256 experts, top 8, sigmoid, bias, 4 of 8 groups: 1 token 4.6 to
// 6.1, 2048 tokens 6.4 to 7.0, 4096 tokens 8.4 to 7.1; bf16 logits alone: 3.3 to 3.7, 4.1 to
// 4.6, 4.9 to 4.7).  Groups that are no whole runs of 16 experts leave few lanes with keys
// and so a low bound; four experts a lane find a better one (160 experts in 8 groups,
// top 6: 1024 tokens 5.8 to 9.5, 8192 tokens 10.5 to 11.3, 16384 tokens 16.8 to 16.0; measured on
// these groups only, and taken to hold for the other sizes above 128 experts).
constexpr int64_t kWaveTokens = 2048, kWaveTokensOddGroups = 8192;
template <class T>
hipError_t route_sized(const RouteParams& p, hipStream_t s) {
  if (p.experts > 256) return route_launch<T, 64, 16>(p, s);
  const bool odd_groups = p.experts > 128 && p.groups > 1 && p.experts / p.groups % 16 != 0;
  if (p.topk > 16 || (p.experts > 64 && p.tokens <= (odd_groups ? kWaveTokensOddGroups : kWaveTokens)))
    return route_launch<T, 64, 4>(p, s);
  if (p.experts <= 64) return route_launch<T, 16, 4>(p, s);
  if (p.experts <= 128) return route_launch<T, 16, 8>(p, s);
  return route_launch<T, 16, 16>(p, s);
}
// As for the forward pass (us, a wave to 16 lanes; 160 fp32 experts, top 6, plain softmax: 1
// token 2.9 to 3.8, 2048 tokens 3.7 to 4.3, 4096 tokens 4.5 to 4.6, 32768 tokens 17.0 to
// 12.4; 256 bf16 experts, renormalised: 2.6 to 3.2, 3.3 to 3.6, 3.8 to 3.8, 12.4 to 7.6).
template <class T>
hipError_t grad_sized(const RouteGradParams& p, hipStream_t s) {
  if (p.experts <= 64) return grad_launch<T, 16, 4>(p, s);
  if (p.experts <= 256 && p.tokens <= kWaveTokens) return grad_launch<T, 64, 4>(p, s);
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

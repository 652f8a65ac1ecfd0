// Weights' gradients, grouped by expert with any number of rows: dW[e] = sum over the rows r
// of expert e of dy[r]^T x[r], x as 16-bit rows or as E4M3 codes with a scale for each 128 columns.
//
// Mathematics.  A product whose contraction runs over rows, the slow dimension of both operands.  dy and x
// enter the bf16 matrix instructions; a code times its scale is rounded to bf16 (not at all where the
// scale is a power of two, as with exponent-only scales: 4 significant bits stay).  That is 2^-8 of a term at most,
// where the code stands for its value within 2^-4; in two halves of 8 bits the product would be all but exact and
// take twice the matrix instructions.  The caller who wants it exact casts with exponent-only scales.  Sums are fp32.
//
// Rows.  A stage is 32 rows of both operands as they lie in memory, brought to LDS by direct loads
// through buffer descriptors that end with the segment's last row: what lies behind reads as
// zero, whatever it holds.  ds_read_b64_tr_b16 (4 rows x 16 columns of 16-bit elements) and _tr_b8 (8 x 16
// codes) turn rows into the matrix instructions' fragments, in which a lane holds 8 rows of one column.  Rows
// are stored with their 16- or 32-byte units permuted by the row's number, so that the rows that half a wave
// reads lie in different banks.
//
// Pipeline.  All other stages of LDS are in flight; a step multiplies the fragments of one stage, held in
// registers, while it reads those of the next into the registers that it has just used (codes are converted on the
// way), and a barrier every step or every other hands the buffers of the stages before to the loads.  Stages follow
// one another across big tiles: while the last stages of one are multiplied and its sums are stored, the
// next one's are on their way.
//
// Bound by matrix instructions, at the clock that the card's power leaves them (1.9 to 2.2 GHz), where groups have
// many rows, and by the operands' and dW's way through memory where they have few.  Measured, with operands that no
// cache holds: 8 experts, 8192 rows, 4096 x 7168: codes 541 us with fp32 sums (889 TFLOP/s, 940 MB of dW) and
// 468 us in bf16 (1027), 16-bit rows 510 and 440 us; 64 experts, 16384 rows, 2048 x 1408: codes 210 and 159 us
// (738 MB of fp32, 369 of bf16), 16-bit rows 221 and 160 us; a dense 8191 x 512 x 2176 in 33 us.  Added to dW, which
// is read after a tile's last product: 8 experts of 1024 rows 763 us (527 without), 64 of 256 437 (196).
// Before dW went out in whole lines 576 and 484, 258 and 172 us (codes): half lines reached memory 1.46 times.  Before
// that, with a prologue for each tile, 600 and 507, 260 and 199 us.
//
// Tried: the 32 x 32 x 16 instruction takes 11% fewer cycles a stage, and the clock falls by 14%; two workgroups of
// 256 x 128 a CU 977 TFLOP/s where one of 256 x 256 does 1062 (4096^3, 16-bit rows 1014 and 1173).
#include "dgfp8_device.h"
#include "layer_internal.h"

namespace dgfp8 {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kStep = 32;   // rows of a stage

template <int kTileN, int kTileK, int kWavesN_, int kWavesK_, bool kFp8_, int kStages_>
struct Config {
  static constexpr int kTn = kTileN, kTk = kTileK, kWavesN = kWavesN_, kWavesK = kWavesK_, kStages = kStages_;
  static constexpr bool kFp8 = kFp8_;
  static constexpr int kWaves = kWavesN * kWavesK, kThreads = kWaves * 64;
  static constexpr int kFragN = kTn / kWavesN / 16, kFragK = kTk / kWavesK / 16;
  // A barrier every other step spares a wave the other half (codes, six stages: 1766 cycles a stage and 1876), but with
  // four stages or fewer it leaves too few loads on their way (16-bit rows: 1597 and 1460).
  static constexpr bool kPairs = kStages > 4;
  // The loads go on to the next tile while this one is finished (64 experts of 256 rows, 2048 x 1408: 199 -> 172 us).
  // Small tiles are all at work at once: a workgroup has one, and the look for the next would cost it 4 to 8%
  // (8191 rows, 512 x 2176: 33 -> 34.5 us).
  static constexpr bool kAcross = kTn >= 256;
  static constexpr int kPitchN = kTn * 2, kPitchK = kTk * (kFp8 ? 1 : 2);   // bytes of an LDS row
  static constexpr int kBytesN = kStep * kPitchN, kBytesK = kStep * kPitchK;
  static constexpr int kBlocks = kTk / 128;
  static constexpr int kScaleBytes = kFp8 ? kBlocks * kStep * 4 : 0;
  static constexpr int kStageBytes = kBytesN + kBytesK + kScaleBytes;
  // direct loads of a wave in a stage: of dy and of x, and the rows of each; the first kBlocks waves load a block's
  // scales too, which the counts that they wait for leave out (they wait a little longer)
  static constexpr int kLoadsN = kBytesN / 1024 / kWaves, kLoadsK = kBytesK / 1024 / kWaves;
  static constexpr int kLoads = kLoadsN + kLoadsK;
  static constexpr int kRowsN = 1024 / kPitchN, kRowsK = 1024 / kPitchK;
  static_assert(kLoadsN * kWaves * 1024 == kBytesN && kLoadsK * kWaves * 1024 == kBytesK, "a wave's share of a stage");
  static_assert(kFragN >= 2 && kTk / kWavesK <= 128, "a wave's columns lie in one block of scales");
  // First row of a wave's load.  The rows of one lane in all its loads have the same order of units
  // (turn16 below), so that its column is the same in each.
  static constexpr __device__ int row_n(int wave, int load) { return load * 16 + wave * kRowsN; }
  static constexpr __device__ int row_k(int wave, int load) { return load * 16 + wave * kRowsK; }
  static_assert(kLoadsN * 16 == kStep, "rows of dy's loads");
  static_assert(kFp8 ? kLoadsK == 1 : kLoadsK * 16 == kStep, "rows of x's loads");
};

// Order of a row's units in LDS.  32-byte units of 16-bit rows: half a wave reads rows 0-3 and 8-11 (or 4-7 and
// 12-15) of a stage, 8 of them.  16-byte units of code rows: it reads 16 rows.
__device__ __forceinline__ int turn16(int row) { return (row & 3) | ((row >> 1) & 4); }
template <int kPitch>
__device__ __forceinline__ int turn8(int row) {
  return kPitch >= 256 ? row & 15 : (row >> 1) & 7;
}

// A buffer descriptor in scalar registers.
struct Rsrc {
  i32x4 w;
};
__device__ __forceinline__ Rsrc rsrc_of(uint64_t base, uint32_t bytes) {
  return {(i32x4){(int)(uint32_t)base, (int)((uint32_t)(base >> 32) & 0xFFFFu), (int)bytes, kRawBufferFlags}};
}
// Direct loads to LDS at M0 + 16 (4) * lane; lanes past the descriptor's end write zeros.  The
// descriptor's words come from scalar instructions, which need no wait state; M0 needs one.
__device__ __forceinline__ void load16_lds(Rsrc r, uint32_t off, uint32_t lds) {
  asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
               :: "v"(off), "s"(r.w), "{m0}"(__builtin_amdgcn_readfirstlane(lds)) : "memory");
}
__device__ __forceinline__ void load4_lds(Rsrc r, uint32_t off, uint32_t lds) {
  asm volatile("s_nop 0\n\tbuffer_load_dword %0, %1, 0 offen lds"
               :: "v"(off), "s"(r.w), "{m0}"(__builtin_amdgcn_readfirstlane(lds)) : "memory");
}

// First row and rows of every group, inside [0, rows], by one wave: up to 16 groups a lane.
__device__ void segments(const WeightGradParams& p, int lane, DG_LAS int32_t* first, DG_LAS int32_t* count) {
  if (!p.counts) {
    if (lane == 0) {
      first[0] = 0;
      count[0] = (int32_t)p.rows;
    }
    return;
  }
  const int per = (p.groups + 63) / 64;
  const int g0 = lane * per, g1 = g0 + per < p.groups ? g0 + per : p.groups;
  const uint32_t align = (uint32_t)p.alignment;   // below 2^31, as every count is
  auto rows_of = [&](int g) -> uint32_t { return p.counts[g] < 0 ? 0u : (uint32_t)p.counts[g]; };
  auto span_of = [&](uint32_t c) -> int64_t {
    return p.max_m > 0 ? p.max_m : (int64_t)((c + align - 1) / align) * align;
  };
  int64_t mine = 0;
  for (int g = g0; g < g1; ++g) mine += span_of(rows_of(g));
  int64_t at = mine;   // rows before this lane's first group
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int64_t v = __shfl_up(at, off, 64);
    if (lane >= off) at += v;
  }
  at -= mine;
  for (int g = g0; g < g1; ++g) {
    const uint32_t c = rows_of(g);
    const int64_t from = at < p.rows ? at : p.rows;
    int64_t n = p.max_m > 0 && c > p.max_m ? p.max_m : c;
    if (n > p.rows - from) n = p.rows - from;
    first[g] = (int32_t)from;
    count[g] = (int32_t)n;
    at += span_of(c);
  }
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// A tile's work: one group, some of its stages, one piece of dW.
struct Unit {
  int g, split;
  int n0, k0;
  int64_t row;         // first row
  int left, stages;    // rows, and the stages that hold them
};

template <class C, bool kF32>
__global__ void __launch_bounds__(C::kThreads)
__attribute__((amdgpu_waves_per_eu(2, 2))) weight_grad_kernel(WeightGradParams p) {
  __shared__ __attribute__((aligned(256))) uint8_t lds[C::kStages * C::kStageBytes];
  __shared__ int32_t group_first[kMaxGroups], group_count[kMaxGroups];
  __shared__ int16_t group_order[kMaxGroups];
  DG_LAS uint8_t* const base = (DG_LAS uint8_t*)lds;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wn = wave / C::kWavesK, wk = wave % C::kWavesK;
  if (wave == 0) segments(p, lane, (DG_LAS int32_t*)group_first, (DG_LAS int32_t*)group_count);
  __syncthreads();
  // groups with the most rows first: what is left for the last round is short
  for (int g = threadIdx.x; g < p.groups; g += C::kThreads) {
    const int32_t c = group_count[g];
    int rank = 0;
    for (int h = 0; h < p.groups; ++h) rank += group_count[h] > c || (group_count[h] == c && h < g);
    group_order[rank] = (int16_t)g;
  }
  __syncthreads();

  const int tiles_n = (int)((p.n + C::kTn - 1) / C::kTn), tiles_k = (int)((p.k + C::kTk - 1) / C::kTk);
  const int tiles = tiles_n * tiles_k;
  const int units = p.groups * p.splits * tiles;
  // Units of a round go to the XCDs in runs, and a run covers 4 rows of tiles side by side, so that the
  // workgroups that share an L2 share the operands' panels.
  auto unit_of = [&](int u) -> Unit {
    Unit w;
    // divisions are vector instructions: their results go back to scalar registers
    const int gs = uniform(u / tiles), t = u - gs * tiles;
    const int turn = uniform(gs / p.splits);
    w.g = uniform(((DG_LAS int16_t*)group_order)[turn]);
    w.split = gs - turn * p.splits;
    const int band = uniform(t / (4 * tiles_k)), in = t - band * 4 * tiles_k;
    const int high = tiles_n - band * 4 < 4 ? tiles_n - band * 4 : 4;
    const int across = uniform(in / high);
    w.n0 = (band * 4 + in - across * high) * C::kTn;
    w.k0 = across * C::kTk;
    const int first = uniform(((DG_LAS int32_t*)group_first)[w.g]);
    // below 2^31; whole stages of that many rows are 2^31 rows, one more than an int holds
    const uint32_t count = (uint32_t)uniform(((DG_LAS int32_t*)group_count)[w.g]);
    const int all = (int)((count + (kStep - 1)) / kStep), share = uniform((all + p.splits - 1) / p.splits);
    const int s0 = w.split * share < all ? w.split * share : all;
    w.stages = share < all - s0 ? share : all - s0;
    w.row = (int64_t)first + (int64_t)s0 * kStep;
    const uint32_t rest = count - (uint32_t)s0 * kStep, whole = (uint32_t)w.stages * kStep;
    w.left = (int)(rest < whole ? rest : whole);
    return w;
  };

  // ---- direct loads: this lane's piece of each
  const uint32_t ldn = (uint32_t)(p.lddy * 2), ldk = (uint32_t)(p.ldx * (C::kFp8 ? 1 : 2));   // bytes
  uint32_t off_n[C::kLoadsN], off_k[C::kLoadsK];
  auto column16 = [&](int row, int slot) {   // byte of the 16 that belong in this slot of the row
    return (uint32_t)((((slot >> 1) ^ turn16(row)) << 1) | (slot & 1)) * 16;
  };
#pragma unroll
  for (int j = 0; j < C::kLoadsN; ++j) {
    constexpr int kSlots = 64 / C::kRowsN;
    const int r = C::row_n(wave, j) + lane / kSlots;
    off_n[j] = (uint32_t)r * ldn + column16(r, lane % kSlots);
  }
#pragma unroll
  for (int j = 0; j < C::kLoadsK; ++j) {
    constexpr int kSlots = 64 / C::kRowsK;
    const int r = C::row_k(wave, j) + lane / kSlots, slot = lane % kSlots;
    off_k[j] = (uint32_t)r * ldk + (C::kFp8 ? (uint32_t)(slot ^ turn8<C::kPitchK>(r)) * 16 : column16(r, slot));
  }
  const uint32_t off_s = C::kFp8 ? (uint32_t)lane * (uint32_t)(p.sf_s0 * 4) : 0;   // lanes 0 .. 31: a block's rows

  const int grid = (int)gridDim.x;   // a multiple of 8
  const int mine = (int)(blockIdx.x & 7) * (grid >> 3) + (int)(blockIdx.x >> 3);
  // unit of a round: forwards and backwards in turn, so that who gets the longest of one gets the shortest
  // of the next (groups come in order of their rows)
  auto unit_in = [&](int round) { return round * grid + (round & 1 ? grid - 1 - mine : mine); };
  if (unit_in(0) >= units) return;

  // where the next stage comes from: the loads walk through the units on their own, ahead of the products
  int load_round = 0, load_left = 0;   // the next unit's round; stages that the present one still has
  uint64_t src_n = 0, src_k = 0, src_s = 0;
  int src_left = 0;
  uint32_t cols_n = 0, cols_k = 0;
  bool block_in = false;
  auto begin = [&](const Unit& w) {
    src_n = (uint64_t)(uintptr_t)p.dy + (uint64_t)w.row * ldn + (uint64_t)w.n0 * 2;
    src_k = (uint64_t)(uintptr_t)p.x + (uint64_t)w.row * ldk + (uint64_t)w.k0 * (C::kFp8 ? 1 : 2);
    cols_n = (uint32_t)(p.n - w.n0) * 2;
    cols_k = (uint32_t)(p.k - w.k0) * (C::kFp8 ? 1 : 2);
    if constexpr (C::kFp8) {
      const int64_t block = w.k0 / 128 + (wave < C::kBlocks ? wave : 0);
      block_in = block * 128 < p.k;
      src_s = (uint64_t)(uintptr_t)p.sf + (uint64_t)(w.row * p.sf_s0 + block * p.sf_s1) * 4;
    }
    src_left = w.left;
  };
  // A stage's loads one by one: what they need first, then each.
  struct Loads {
    Rsrc n, k, s;
    uint32_t at;
  };
  auto next_loads = [&](int buffer) -> Loads {
    // on to the next unit that has rows; behind the last one nothing is left, and the loads write zeros
    if constexpr (C::kAcross) {
      while (__builtin_expect(load_left == 0, 0)) {
        const int u = unit_in(load_round);
        if (u >= units) break;
        ++load_round;
        const Unit w = unit_of(u);
        load_left = w.stages;
        if (load_left > 0) begin(w);
      }
      if (load_left > 0) --load_left;
    }
    const uint32_t rows = src_left > kStep ? kStep : src_left < 0 ? 0 : src_left;
    const uint32_t s0 = C::kFp8 ? (uint32_t)(p.sf_s0 * 4) : 0;
    Loads l;
    l.at = lds_addr(base) + (uint32_t)buffer * C::kStageBytes;
    l.n = rsrc_of(src_n, rows ? (rows - 1) * ldn + cols_n : 0);
    l.k = rsrc_of(src_k, rows ? (rows - 1) * ldk + cols_k : 0);
    if constexpr (C::kFp8) l.s = rsrc_of(src_s, rows && block_in ? (rows - 1) * s0 + 4 : 0);
    src_n += (uint64_t)kStep * ldn;
    src_k += (uint64_t)kStep * ldk;
    src_s += (uint64_t)kStep * s0;
    src_left -= kStep;
    return l;
  };
  auto load_piece = [&](const Loads& l, int i) {
    if (i < C::kLoadsN) {
      load16_lds(l.n, off_n[i < C::kLoadsN ? i : 0], l.at + (uint32_t)C::row_n(wave, i) * C::kPitchN);
    } else if (i < C::kLoadsN + C::kLoadsK) {
      const int j = i - C::kLoadsN;
      load16_lds(l.k, off_k[j < C::kLoadsK ? j : 0], l.at + C::kBytesN + (uint32_t)C::row_k(wave, j) * C::kPitchK);
    } else if (C::kFp8 && wave < C::kBlocks) {
      if (lane < kStep) load4_lds(l.s, off_s, l.at + C::kBytesN + C::kBytesK + (uint32_t)wave * (kStep * 4));
    }
  };
  auto load_stage = [&](int buffer) {
    const Loads l = next_loads(buffer);
#pragma unroll
    for (int i = 0; i <= C::kLoads; ++i) load_piece(l, i);
  };

  // ---- fragments: lane l holds column l % 16 and rows 8 (l / 16) .. + 7
  const int row_n = (lane >> 4) * 8 + ((lane & 15) >> 2);   // and row_n + 4
  // Where a wave's first fragments lie in a stage.  The others' units differ from theirs in the bits of their number,
  // which stand in bits of the address that no sum carries into: xor gives them.
  auto place16 = [&](int unit, int pitch) {
    return (uint32_t)(row_n * pitch + ((unit ^ turn16(row_n)) << 5) + (lane & 3) * 8);
  };
  const uint32_t at_n = place16(wn * C::kFragN, C::kPitchN);
  const int row_c = (lane >> 4) * 8 + ((lane & 15) >> 1);   // of codes
  const uint32_t at_k = C::kBytesN + (C::kFp8 ? (uint32_t)(row_c * C::kPitchK + ((wk * C::kFragK ^ turn8<C::kPitchK>(row_c)) << 4) +
                                                          (lane & 1) * 8)
                                              : place16(wk * C::kFragK, C::kPitchK));
  static_assert(C::kStageBytes % (C::kFragN * 32) == 0 && C::kBytesN % 256 == 0, "units' bits stay clear of sums");
  constexpr int kAhead = C::kPairs ? C::kStages - 4 : C::kStages - 2;   // stages on their way at a barrier
  constexpr int kBegun = C::kPairs ? C::kStages - 1 : C::kStages;       // stages loaded before a tile's first
  constexpr int kStores = kF32 ? C::kFragN * C::kFragK : C::kFragN * C::kFragK / 2;   // of a tile that lies whole in dW
  const uint32_t at_s = C::kBytesN + C::kBytesK + (uint32_t)(wk * C::kFragK / 8 * kStep + (lane >> 4) * 8) * 4;

  f32x4 acc[C::kFragN][C::kFragK];
  struct Pair16 {   // a fragment of 16-bit elements: rows 0 - 3 and 4 - 7 of a lane's 8
    s16x4 lo, hi;
  };
  auto whole = [](const Pair16& f) -> bf16x8 {
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(f.lo, f.hi, 0, 1, 2, 3, 4, 5, 6, 7));
  };
  auto read16 = [&](DG_LAS uint8_t* a, int pitch, Pair16& f, int half) {
    const s16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((DG_LAS s16x4*)(a + half * 4 * pitch));
    if (half == 0) f.lo = v;
    else f.hi = v;
  };
  Pair16 fn[C::kFragN];
  uint32_t an[C::kFragN], ak[C::kFragK];
#pragma unroll
  for (int i = 0; i < C::kFragN; ++i) an[i] = at_n ^ (i << 5);
#pragma unroll
  for (int i = 0; i < C::kFragK; ++i) ak[i] = at_k ^ (i << (C::kFp8 ? 4 : 5));
  struct Right {   // x's fragments of a stage
    u32x4 f[C::kFragK];
  };
  struct Raw {     // and what they are made of
    i32x2 code[C::kFragK];
    Pair16 rows[C::kFragK];
    f32x4 scale[2];
  };
  // x of a stage, one LDS read at a time, and a quarter of a fragment's conversion
  constexpr int kReads = C::kFp8 ? 2 + C::kFragK : 2 * C::kFragK;
  auto read_right = [&](DG_LAS uint8_t* stage, Raw& raw, int i) {
    if constexpr (C::kFp8) {
      if (i < 2) raw.scale[i] = *(DG_LAS f32x4*)(stage + at_s + 16 * i);
      else raw.code[i - 2] = __builtin_amdgcn_ds_read_tr8_b64_v2i32((DG_LAS i32x2*)(stage + ak[i - 2]));
    } else {
      read16(stage + ak[i >> 1], C::kPitchK, raw.rows[i >> 1], i & 1);
    }
  };
  constexpr int kPieces = 4 * C::kFragK;
  auto convert = [&](const Raw& raw, Right& to, int piece) {
    const int j = piece >> 2, q = piece & 3;   // dword q of fragment j: rows 2 q and 2 q + 1
    if constexpr (C::kFp8) {
      const f32x4 s = raw.scale[q >> 1];
      const auto v = q & 1 ? __builtin_amdgcn_cvt_pk_f32_fp8(raw.code[j][q >> 1], true)
                           : __builtin_amdgcn_cvt_pk_f32_fp8(raw.code[j][q >> 1], false);
      to.f[j][q] = q & 1 ? pack_bf16x2(v[0] * s.z, v[1] * s.w) : pack_bf16x2(v[0] * s.x, v[1] * s.y);
    } else if (q == 0) {
      to.f[j] = __builtin_bit_cast(u32x4, whole(raw.rows[j]));
    }
  };

  // One stage: products of the fragments in fn and `now`; those of the next stage (in `buffer`) come into fn and
  // `next`, and loads go to the buffer `spent`; where a big tile ends, both are the next tile's.  A step with a
  // barrier waits until the stages read up to the next barrier have come in every wave, and until all waves have read
  // the buffers that loads go to from then on.  A wave's instructions issue in order, so what the next stage needs
  // stands between the products, a little after each.
  constexpr int kSlots = C::kFragN * C::kFragK;
  constexpr int kConvert = kSlots > 16 ? 12 : 11;   // first slot of a conversion: its codes are read by slot 9
  auto step = [&](bool barrier, const Right& now, Right& next, int spent, int buffer, bool stored) {
    DG_LAS uint8_t* const stage = base + buffer * C::kStageBytes;
    Loads loads;
    Raw raw;
    static_for<0, kSlots>([&](auto slot) {
      constexpr int q = slot, i = q / C::kFragK, j = q % C::kFragK;
      acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, now.f[j]), whole(fn[i]), acc[i][j],
                                                          0, 0, 0);
      if constexpr (q == 1) loads = next_loads(spent);
      if constexpr (q == C::kFragK - 1) {
        if (barrier) {
          // stores of the tile before may be younger than the loads waited for
          if (__builtin_expect(stored, 0)) __builtin_amdgcn_s_waitcnt(WaitVmLgkm0<kAhead * C::kLoads + kStores>::value);
          else __builtin_amdgcn_s_waitcnt(WaitVmLgkm0<kAhead * C::kLoads>::value);
          lds_barrier();
        }
      }
      static_for<0, C::kLoads + 1>([&](auto l) {
        if constexpr (q == C::kFragK + 1 + l * ((kSlots - C::kFragK) / (C::kLoads + 1))) load_piece(loads, l);
      });
      if constexpr (q >= C::kFragK && q < C::kFragK + kReads) read_right(stage, raw, q - C::kFragK);
      static_for<0, C::kFragN - 1>([&](auto f) {
        constexpr int at = (f + 1) * C::kFragK + (f == 0 ? 4 : f == 1 ? 2 : 0);
        if constexpr (q == at || q == at + 1) read16(stage + an[f], C::kPitchN, fn[f], q - at);
      });
      if constexpr (q >= kConvert)
        static_for<(q - kConvert) * kPieces / (kSlots - kConvert), (q + 1 - kConvert) * kPieces / (kSlots - kConvert)>(
            [&](auto piece) { convert(raw, next, piece); });
      __builtin_amdgcn_sched_barrier(0);
    });
    read16(stage + an[C::kFragN - 1], C::kPitchN, fn[C::kFragN - 1], 0);
    read16(stage + an[C::kFragN - 1], C::kPitchN, fn[C::kFragN - 1], 1);
  };

  // Writes a tile; true if that took kStores stores and no loads.  Lanes 8 apart exchange halves of what two neighbouring
  // stores write, so that each writes whole 128-byte lines of 8 rows, not half lines of 16.
  auto halves = [&](uint32_t& a, uint32_t& b) {
    const uint32_t other = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(lane & 8 ? a : b), 0x128 /* row_ror:8 */, 0xF, 0xF, true);
    if (lane & 8) a = other;
    else b = other;
  };
  auto put = [&](const Unit& w) -> bool {
    const bool inside = w.n0 + C::kTn <= p.n && w.k0 + C::kTk <= p.k;
    const int64_t n0 = w.n0 + wn * C::kFragN * 16 + (lane & 7), k0 = w.k0 + wk * C::kFragK * 16;
    const int upper = (lane >> 3) & 1;
    if (kF32 || p.splits > 1) {
      // lane: row n = lane % 16 of fragment i, columns k = 4 (lane / 16) .. of fragment j; then rows lane % 8 and + 8 of
      // fragment j or j + 1
      float* dw = p.splits > 1 ? p.partial + ((int64_t)w.split * p.groups + w.g) * p.n * p.k
                               : (float*)p.dw + w.g * p.dw_gs;
      const int64_t ld = p.splits > 1 ? p.k : p.lddw, k1 = k0 + upper * 16 + (lane >> 4) * 4;
      const bool add = p.accumulate && p.splits == 1;
      auto each = [&](auto&& f) {
#pragma unroll
        for (int i = 0; i < C::kFragN; ++i) {
          float* row = dw + (n0 + i * 16) * ld + k1;
#pragma unroll
          for (int j = 0; j < C::kFragK; j += 2) {
            u32x4 a = __builtin_bit_cast(u32x4, acc[i][j]), b = __builtin_bit_cast(u32x4, acc[i][j + 1]);
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              uint32_t x = a[h], y = b[h];
              halves(x, y);
              a[h] = x;
              b[h] = y;
            }
            // k is a multiple of 8: four columns are in or out together
            const bool in = inside || k1 + j * 16 < p.k;
            if (inside || (in && n0 + i * 16 < p.n)) f((f32x4*)(row + j * 16), __builtin_bit_cast(f32x4, a));
            if (inside || (in && n0 + i * 16 + 8 < p.n)) f((f32x4*)(row + 8 * ld + j * 16), __builtin_bit_cast(f32x4, b));
          }
          __builtin_amdgcn_sched_barrier(0);   // no more than a row's addresses and sums at once
        }
      };
      // dW passes L2 by, which the operands need, where whole lines can; the splits' sums are read again at once
      if (add) each([&](f32x4* dst, f32x4 v) { *dst = *dst + v; });
      else if (p.splits > 1 || !p.past_l2) each([&](f32x4* dst, f32x4 v) { *dst = v; });
      else each([&](f32x4* dst, f32x4 v) { __builtin_nontemporal_store(v, dst); });
      return inside && !add && kF32;
    }
    // Two fragments side by side: lanes 16 apart exchange halves, so that each has eight columns in a row:
    // 16 (lane / 16 % 2) + 8 (lane / 32) ..; then, as above, of the first two fragments or of the last
    uint16_t* dw = (uint16_t*)p.dw + w.g * p.dw_gs;
    const int64_t k1 = k0 + upper * 32 + ((lane >> 4) & 1) * 16 + (lane >> 5) * 8;
    static_assert(C::kFragK == 4, "two stores of two fragments");
    auto each = [&](auto&& f) {
#pragma unroll
      for (int i = 0; i < C::kFragN; ++i) {
        uint16_t* row = dw + (n0 + i * 16) * p.lddw + k1;
        u32x4 v[2];
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t a = pack_bf16x2(acc[i][j][2 * h], acc[i][j][2 * h + 1]);
            const uint32_t b = pack_bf16x2(acc[i][j + 1][2 * h], acc[i][j + 1][2 * h + 1]);
            const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
            v[j >> 1][h] = r[0];
            v[j >> 1][2 + h] = r[1];
          }
        }
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          uint32_t x = v[0][h], y = v[1][h];
          halves(x, y);
          v[0][h] = x;
          v[1][h] = y;
        }
        if (inside || (n0 + i * 16 < p.n && k1 < p.k)) f((u32x4*)row, v[0]);
        if (inside || (n0 + i * 16 + 8 < p.n && k1 < p.k)) f((u32x4*)(row + 8 * p.lddw), v[1]);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    // two loops: the compiler would make one store of two that only differ in their way
    if (p.past_l2) each([&](u32x4* dst, u32x4 v) { __builtin_nontemporal_store(v, dst); });
    else each([&](u32x4* dst, u32x4 v) { *dst = v; });
    return inside;
  };

  Right even, odd;
  int before = 0, buffer = 0;   // of the stage before and of the present one
  bool first = true;            // of a pair, which has the barrier
  auto after = [](int b) { return b + 1 == C::kStages ? 0 : b + 1; };
  // The first loads, and the first stage's fragments.
  auto fill = [&]() {
#pragma unroll 1
    for (int s = 0; s < kBegun; ++s) load_stage(s);
    __builtin_amdgcn_s_waitcnt(WaitVmLgkm0<(kBegun - 1) * C::kLoads>::value);
    lds_barrier();
    Raw raw;
#pragma unroll
    for (int i = 0; i < kReads; ++i) read_right(base, raw, i);
#pragma unroll
    for (int i = 0; i < 2 * C::kFragN; ++i) read16(base + an[i >> 1], C::kPitchN, fn[i >> 1], i & 1);
#pragma unroll
    for (int i = 0; i < kPieces; ++i) convert(raw, even, i);
    before = C::kStages - 1;
    buffer = 0;
    first = true;
  };
  // Steps since a tile's stores.  A barrier waits for loads that were issued kStages - 3 (pairs) or kStages - 1
  // steps earlier: until that many steps later they are older than the stores.
  constexpr int kGrace = C::kPairs ? C::kStages - 3 : C::kStages - 1;
  int since = kGrace;
  auto next_step = [&](const Right& now, Right& next) {
    const int to = after(buffer);
    step(!C::kPairs || first, now, next, C::kPairs ? before : buffer, to, ++since <= kGrace);
    before = buffer;
    buffer = to;
    first = !first;
  };
  Unit w = unit_of(unit_in(0));
  if constexpr (C::kAcross) fill();
  for (int round = 0;;) {
    if constexpr (!C::kAcross) {
      begin(w);
      fill();
    }
#pragma unroll
    for (int i = 0; i < C::kFragN; ++i)
#pragma unroll
      for (int j = 0; j < C::kFragK; ++j) acc[i][j] = (f32x4){0.f, 0.f, 0.f, 0.f};
    // one way out of the loop: with two the compiler gives each its own registers for the sums
    for (int s = 0; s < w.stages; s += 2) {
      next_step(even, odd);
      if (s + 1 < w.stages) next_step(odd, even);
      else even = odd;
    }
    const bool counted = put(w);
    since = C::kAcross && counted ? 0 : kGrace;
    const int u = unit_in(++round);
    if (u >= units) break;   // only the last round is not whole
    w = unit_of(u);
    if constexpr (!C::kAcross) {
      // nothing may be on its way to LDS, nor be read there, when the next tile's loads begin
      __builtin_amdgcn_s_waitcnt(WaitVmLgkm0<0>::value);
      lds_barrier();
    }
  }
  // no load may be on its way to LDS when the workgroup ends
  __builtin_amdgcn_s_waitcnt(WaitVmLgkm0<0>::value);
}

// dW from the partial sums of the splits, in their order; four columns a thread.
template <bool kF32>
__global__ void __launch_bounds__(256) weight_grad_sum_kernel(WeightGradParams p) {
  const int64_t per = p.n * (p.k / 4), all = per * p.groups;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= all) return;
  const int64_t g = i / per, in = i - g * per, n = in / (p.k / 4), k = (in - n * (p.k / 4)) * 4;
  f32x4 v = *(const f32x4*)(p.partial + i * 4);
  for (int s = 1; s < p.splits; ++s) v += *(const f32x4*)(p.partial + (s * all + i) * 4);
  if constexpr (kF32) {
    f32x4* dst = (f32x4*)((float*)p.dw + g * p.dw_gs + n * p.lddw + k);
    if (p.accumulate) v += *dst;
    *dst = v;
  } else {
    *(u32x2*)((uint16_t*)p.dw + g * p.dw_gs + n * p.lddw + k) = (u32x2){pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w)};
  }
}

int64_t tiles(int64_t n, int64_t k, int64_t tn, int64_t tk) { return ((n + tn - 1) / tn) * ((k + tk - 1) / tk); }

// 256 x 256 tiles, which read less for each product, from 129 of them on; 128 x 128 tiles, two workgroups a CU, below:
// where n and k are multiples of 256 as many small tiles as run at once.  8192 rows, bf16, fp32 sums: 2048 x 4096 (128
// big tiles) 137 us in small tiles and 179 in big ones, 4096 x 2816 (176) 254 and 183, 4096 x 4096 269 and 223.
// Where n or k are not, small tiles could run at once beyond that (up to 512 of them), and win or lose: 8192 rows, 2064 x
// 3840 (135 big, 510 small) 150 and 178 us; 170 groups of 256 rows, 128 x 384 19 and 29; 256 groups, 128 x 128, of 128
// rows 15.6 and 18.8, of 1024 rows 51.8 and 45.5; 512 groups of 64 rows, 64 x 128 37.6 and 30.5.
bool big_tiles(int64_t n, int64_t k, int groups) { return tiles(n, k, 256, 256) * groups > 128; }

template <class C>
void launch_of(const WeightGradParams& p, bool f32, int per_cu, hipStream_t stream) {
  const int64_t units = (int64_t)p.groups * p.splits * tiles(p.n, p.k, C::kTn, C::kTk);
  const int64_t most = (int64_t)dg_get_num_cus() * per_cu, want = units < most ? units : most;
  const dim3 grid((unsigned)((want + 7) / 8 * 8)), block(C::kThreads);
  if (f32) hipLaunchKernelGGL((weight_grad_kernel<C, true>), grid, block, 0, stream, p);
  else hipLaunchKernelGGL((weight_grad_kernel<C, false>), grid, block, 0, stream, p);
}

hipError_t launch(const WeightGradParams& p, bool x_fp8, bool f32, hipStream_t stream) {
  if (big_tiles(p.n, p.k, p.groups)) {
    if (x_fp8) launch_of<Config<256, 256, 2, 4, true, 6>>(p, f32, 1, stream);
    else launch_of<Config<256, 256, 2, 4, false, 4>>(p, f32, 1, stream);
  } else {
    if (x_fp8) launch_of<Config<128, 128, 2, 2, true, 5>>(p, f32, 2, stream);
    else launch_of<Config<128, 128, 2, 2, false, 4>>(p, f32, 2, stream);
  }
  return hipGetLastError();
}

}  // namespace

// Workgroups that share the rows of a small tile: as many as run at once (512), each with eight stages or more of
// a group of average size, so that the sums they hand over stay the smaller part.  32768 rows, 512 x 2048, bf16: 75 us
// with 8 (64 tiles), 8191 rows, 512 x 2112: 28 us and 6 for the sum of the 7 parts.
int weight_grad_splits(int64_t rows, int64_t n, int64_t k, int groups) {
  if (big_tiles(n, k, groups)) return 1;
  const int64_t units = tiles(n, k, 128, 128) * groups;
  const int64_t steps = (rows / groups + kStep - 1) / kStep;
  int64_t s = 512 / units;
  if (s > steps / 8) s = steps / 8;
  return (int)(s < 1 ? 1 : s > 64 ? 64 : s);
}

// dW's rows begin at multiples of 64 bytes: what a workgroup writes of them are whole lines, or halves at its edges.
// Elsewhere the pieces of a line have to meet in L2.  16-bit rows, 64 experts of 10 rows, 1152 x k, past L2 and
// through it: k 1152 78 and 80 us (fp32), 41 and 44 (bf16), 1160 168 and 96, 87 and 54; of 256 rows on average
// 1152 110 and 142, 84 and 101, 1160 168 and 143, 94 and 104; 8 of 1024, 4096 x 7176: 639 and 554, 498 and 479.
static bool whole_lines(const WeightGradParams& p, int64_t elem) {
  return (uintptr_t)p.dw % 64 == 0 && p.lddw * elem % 64 == 0 && (p.groups == 1 || p.dw_gs * elem % 64 == 0);
}

hipError_t launch_weight_grad(const WeightGradParams& given, bool x_fp8, int out_dtype, hipStream_t stream) {
  const bool f32 = out_dtype == DG_F32;
  WeightGradParams p = given;
  p.past_l2 = whole_lines(p, f32 ? 4 : 2);
  const hipError_t err = launch(p, x_fp8, f32, stream);
  if (err != hipSuccess || p.splits <= 1) return err;
  const int64_t all = (int64_t)p.groups * p.n * (p.k / 4);
  const dim3 grid((unsigned)((all + 255) / 256));
  if (f32) hipLaunchKernelGGL((weight_grad_sum_kernel<true>), grid, dim3(256), 0, stream, p);
  else hipLaunchKernelGGL((weight_grad_sum_kernel<false>), grid, dim3(256), 0, stream, p);
  return hipGetLastError();
}

}  // namespace dgfp8

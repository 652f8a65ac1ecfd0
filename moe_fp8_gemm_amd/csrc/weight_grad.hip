// Weights' gradients, grouped by expert with any number of rows: dW[e] = sum over the rows r
// of expert e of dy[r]^T x[r], x as 16-bit rows or as E4M3 codes with a scale for each 128 columns.
//
// Mathematics.  A product whose contraction runs over rows, the slow dimension of both operands.  dy and x
// enter the bf16 matrix instructions; a code times its scale is rounded to bf16 (not at all where the
// scale is a power of two, as with exponent-only scales: 4 significant bits stay).  Sums are
// fp32.
//
// Rows.  A stage is 32 rows of both operands as they lie in memory, brought to LDS by direct loads
// through buffer descriptors that end with the segment's last row: what lies behind reads as
// zero, whatever it holds.  ds_read_b64_tr_b16 (4 rows x 16 columns of 16-bit elements) and _tr_b8 (8 x 16
// codes) turn rows into the matrix instructions' fragments, in which a lane holds 8 rows of one column.  Rows
// are stored with their 16- or 32-byte units permuted by the row's number, so that the rows that half a wave
// reads lie in different banks.
//
// Pipeline.  All stages of LDS are in flight; a step multiplies the fragments of one stage, held in
// registers, while it reads those of the next into the registers that it has just used (codes are converted on the
// way), and a barrier after the step's first products hands the buffer of the stage before to the loads.
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
  static constexpr int kPitchN = kTn * 2, kPitchK = kTk * (kFp8 ? 1 : 2);   // bytes of an LDS row
  static constexpr int kBytesN = kStep * kPitchN, kBytesK = kStep * kPitchK;
  static constexpr int kBlocks = kTk / 128;
  static constexpr int kScaleBytes = kFp8 ? kBlocks * kStep * 4 : 0;
  static constexpr int kStageBytes = kBytesN + kBytesK + kScaleBytes;
  // direct loads of a wave in a stage: two of dy, and of x two, or one of codes and one of scales
  static constexpr int kLoads = 4;
  static_assert(kBytesN == kWaves * 2048 && kBytesK == kWaves * (kFp8 ? 1024 : 2048), "a wave's share of a stage");
  static_assert(kFragN >= 2 && kTk / kWavesK <= 128, "a wave's columns lie in one block of scales");
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
  __shared__ __attribute__((aligned(128))) uint8_t lds[C::kStages * C::kStageBytes];
  __shared__ int32_t group_first[kMaxGroups], group_count[kMaxGroups];
  DG_LAS uint8_t* const base = (DG_LAS uint8_t*)lds;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wn = wave / C::kWavesK, wk = wave % C::kWavesK;
  if (wave == 0) segments(p, lane, (DG_LAS int32_t*)group_first, (DG_LAS int32_t*)group_count);
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
    w.g = uniform(gs / p.splits);
    w.split = gs - w.g * p.splits;
    const int band = uniform(t / (4 * tiles_k)), in = t - band * 4 * tiles_k;
    const int high = tiles_n - band * 4 < 4 ? tiles_n - band * 4 : 4;
    const int across = uniform(in / high);
    w.n0 = (band * 4 + in - across * high) * C::kTn;
    w.k0 = across * C::kTk;
    const int first = uniform(((DG_LAS int32_t*)group_first)[w.g]);
    const int count = uniform(((DG_LAS int32_t*)group_count)[w.g]);
    const int all = (count + kStep - 1) / kStep, share = uniform((all + p.splits - 1) / p.splits);
    const int s0 = w.split * share < all ? w.split * share : all;
    w.stages = share < all - s0 ? share : all - s0;
    w.row = (int64_t)first + (int64_t)s0 * kStep;
    w.left = count - s0 * kStep < w.stages * kStep ? count - s0 * kStep : w.stages * kStep;
    return w;
  };

  // ---- direct loads: this lane's piece of each
  constexpr int kRowsN = 1024 / C::kPitchN, kRowsK = 1024 / C::kPitchK;   // rows of a wave's load
  const uint32_t ldn = (uint32_t)(p.lddy * 2), ldk = (uint32_t)(p.ldx * (C::kFp8 ? 1 : 2));   // bytes
  uint32_t off_n[2], off_k[2];
  {
    const int r = wave * kRowsN + lane / (64 / kRowsN), slot = lane % (64 / kRowsN);
    const uint32_t col = (uint32_t)(((((slot >> 1) ^ turn16(r)) << 1) | (slot & 1)) * 16);
    off_n[0] = (uint32_t)r * ldn + col;
    off_n[1] = off_n[0] + 16 * ldn;
  }
  {
    const int r = wave * kRowsK + lane / (64 / kRowsK), slot = lane % (64 / kRowsK);
    if constexpr (C::kFp8) {
      off_k[0] = (uint32_t)r * ldk + (uint32_t)(slot ^ turn8<C::kPitchK>(r)) * 16;
      off_k[1] = 0;
    } else {
      off_k[0] = (uint32_t)r * ldk + (uint32_t)(((((slot >> 1) ^ turn16(r)) << 1) | (slot & 1)) * 16);
      off_k[1] = off_k[0] + 16 * ldk;
    }
  }
  // scales: 8 rows of one block by 8 lanes of each wave
  constexpr int kScaleRows = kStep * C::kBlocks / C::kWaves;
  static_assert(!C::kFp8 || kScaleRows == 8, "8 scales a wave");
  const int scale_row = wave * kScaleRows % kStep, scale_block = wave * kScaleRows / kStep;
  const uint32_t off_s = C::kFp8 ? (uint32_t)(scale_row + lane) * (uint32_t)(p.sf_s0 * 4) : 0;

  // where the next stage comes from
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
      const int64_t block = w.k0 / 128 + scale_block;
      block_in = block * 128 < p.k;
      src_s = (uint64_t)(uintptr_t)p.sf + (uint64_t)(w.row * p.sf_s0 + block * p.sf_s1) * 4;
    }
    src_left = w.left;
  };
  auto load_stage = [&](int buffer) {
    const uint32_t at = lds_addr(base) + (uint32_t)buffer * C::kStageBytes;
    const uint32_t rows = src_left > kStep ? kStep : src_left < 0 ? 0 : src_left;
    const Rsrc rn = rsrc_of(src_n, rows ? (rows - 1) * ldn + cols_n : 0);
    const Rsrc rk = rsrc_of(src_k, rows ? (rows - 1) * ldk + cols_k : 0);
    const uint32_t at_n = at + (uint32_t)(wave * kRowsN) * C::kPitchN;
    load16_lds(rn, off_n[0], at_n);
    load16_lds(rn, off_n[1], at_n + 16 * C::kPitchN);
    const uint32_t at_k = at + C::kBytesN + (uint32_t)(wave * kRowsK) * C::kPitchK;
    load16_lds(rk, off_k[0], at_k);
    if constexpr (C::kFp8) {
      const uint32_t s0 = (uint32_t)(p.sf_s0 * 4);
      const Rsrc rs = rsrc_of(src_s, rows && block_in ? (rows - 1) * s0 + 4 : 0);
      const uint32_t at_s = at + C::kBytesN + C::kBytesK + (uint32_t)(scale_block * kStep + scale_row) * 4;
      if (lane < kScaleRows) load4_lds(rs, off_s, at_s);
      src_s += (uint64_t)kStep * s0;
    } else {
      load16_lds(rk, off_k[1], at_k + 16 * C::kPitchK);
    }
    src_n += (uint64_t)kStep * ldn;
    src_k += (uint64_t)kStep * ldk;
    src_left -= kStep;
  };

  // ---- fragments: lane l holds column l % 16 and rows 8 (l / 16) .. + 7
  const int row_n = (lane >> 4) * 8 + ((lane & 15) >> 2);   // and row_n + 4
  uint32_t at_n[C::kFragN], at_k[C::kFragK];
#pragma unroll
  for (int i = 0; i < C::kFragN; ++i)
    at_n[i] = (uint32_t)row_n * C::kPitchN + (uint32_t)(((wn * C::kFragN + i) ^ turn16(row_n)) * 32 + (lane & 3) * 8);
#pragma unroll
  for (int j = 0; j < C::kFragK; ++j) {
    if constexpr (C::kFp8) {
      const int r = (lane >> 4) * 8 + ((lane & 15) >> 1);
      at_k[j] = (uint32_t)(C::kBytesN + r * C::kPitchK + ((wk * C::kFragK + j) ^ turn8<C::kPitchK>(r)) * 16 + (lane & 1) * 8);
    } else {
      at_k[j] = (uint32_t)(C::kBytesN + row_n * C::kPitchK + ((wk * C::kFragK + j) ^ turn16(row_n)) * 32 + (lane & 3) * 8);
    }
  }
  const uint32_t at_s = C::kBytesN + C::kBytesK + (uint32_t)(wk * C::kFragK / 8 * kStep + (lane >> 4) * 8) * 4;

  auto frag16 = [&](DG_LAS uint8_t* a, int pitch) -> bf16x8 {
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((DG_LAS s16x4*)a);
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((DG_LAS s16x4*)(a + 4 * pitch));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  };

  f32x4 acc[C::kFragN][C::kFragK];
  bf16x8 fn[C::kFragN];
  struct Right {   // x's fragments of a stage
    bf16x8 f[C::kFragK];
  };
  struct Raw {     // and what they are made of
    i32x2 code[C::kFp8 ? C::kFragK : 1];
    f32x4 scale[2];
  };
  auto read_right = [&](DG_LAS uint8_t* stage, Raw& raw, Right& to) {
    if constexpr (C::kFp8) {
#pragma unroll
      for (int j = 0; j < C::kFragK; ++j)
        raw.code[j] = __builtin_amdgcn_ds_read_tr8_b64_v2i32((DG_LAS i32x2*)(stage + at_k[j]));
      raw.scale[0] = *(DG_LAS f32x4*)(stage + at_s);
      raw.scale[1] = *(DG_LAS f32x4*)(stage + at_s + 16);
    } else {
#pragma unroll
      for (int j = 0; j < C::kFragK; ++j) to.f[j] = frag16(stage + at_k[j], C::kPitchK);
    }
  };
  auto convert = [&](const Raw& raw, Right& to, int j) {
    if constexpr (C::kFp8) {
      uint32_t w[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const auto a = __builtin_amdgcn_cvt_pk_f32_fp8(raw.code[j][h], false);
        const auto b = __builtin_amdgcn_cvt_pk_f32_fp8(raw.code[j][h], true);
        w[2 * h] = pack_bf16x2(a[0] * raw.scale[h].x, a[1] * raw.scale[h].y);
        w[2 * h + 1] = pack_bf16x2(b[0] * raw.scale[h].z, b[1] * raw.scale[h].w);
      }
      to.f[j] = __builtin_bit_cast(bf16x8, (u32x4){w[0], w[1], w[2], w[3]});
    }
  };

  auto products = [&](int i, const Right& r) {
#pragma unroll
    for (int j = 0; j < C::kFragK; ++j)
      acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(r.f[j], fn[i], acc[i][j], 0, 0, 0);
  };
  // One stage: products of the fragments in fn and `now`; those of the next stage (in `buffer`)
  // come into fn and `next`.  `spent` is the buffer of this stage, which goes to the loads.
  auto step = [&](const Right& now, Right& next, int spent, int buffer) {
    DG_LAS uint8_t* const stage = base + buffer * C::kStageBytes;
    products(0, now);
    __builtin_amdgcn_sched_barrier(0);
    // the next stage's loads are done in every wave, and so are the reads of the spent one
    __builtin_amdgcn_s_waitcnt(WaitVmLgkm0<(C::kStages - 2) * C::kLoads>::value);
    lds_barrier();
    load_stage(spent);
    Raw raw;
    read_right(stage, raw, next);
    fn[0] = frag16(stage + at_n[0], C::kPitchN);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 1; i < C::kFragN; ++i) {
      products(i, now);
      fn[i] = frag16(stage + at_n[i], C::kPitchN);
      // conversions follow the reads at some distance
#pragma unroll
      for (int j = 0; j < C::kFragK; ++j)
        if (1 + j * (C::kFragN - 1) / C::kFragK == i)
          convert(raw, next, j);
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  auto put = [&](const Unit& w) {
    // lane: row n = lane % 16 of fragment i, columns k = 4 (lane / 16) .. of fragment j
    const int64_t n0 = w.n0 + wn * C::kFragN * 16 + (lane & 15), k0 = w.k0 + wk * C::kFragK * 16 + (lane >> 4) * 4;
    const bool whole = w.n0 + C::kTn <= p.n && w.k0 + C::kTk <= p.k;
    auto each = [&](auto&& f) {
#pragma unroll
      for (int i = 0; i < C::kFragN; ++i) {
#pragma unroll
        for (int j = 0; j < C::kFragK; ++j)
          // k is a multiple of 8: four columns are in or out together
          if (whole || (n0 + i * 16 < p.n && k0 + j * 16 < p.k)) f(acc[i][j], n0 + i * 16, k0 + j * 16);
        __builtin_amdgcn_sched_barrier(0);   // no more than a row's addresses and sums at once
      }
    };
    if (p.splits > 1) {
      float* part = p.partial + ((int64_t)w.split * p.groups + w.g) * p.n * p.k;
      each([&](f32x4 v, int64_t n, int64_t k) { *(f32x4*)(part + n * p.k + k) = v; });
    } else if constexpr (kF32) {
      float* dw = (float*)p.dw + w.g * p.dw_gs;
      if (p.accumulate)
        each([&](f32x4 v, int64_t n, int64_t k) {
          f32x4* dst = (f32x4*)(dw + n * p.lddw + k);
          *dst = *dst + v;
        });
      else
        each([&](f32x4 v, int64_t n, int64_t k) { *(f32x4*)(dw + n * p.lddw + k) = v; });
    } else {
      uint16_t* dw = (uint16_t*)p.dw + w.g * p.dw_gs;
      each([&](f32x4 v, int64_t n, int64_t k) {
        *(u32x2*)(dw + n * p.lddw + k) = (u32x2){pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w)};
      });
    }
  };

  const int grid = (int)gridDim.x;   // a multiple of 8
  int u = (int)(blockIdx.x & 7) * (grid >> 3) + (int)(blockIdx.x >> 3);
  if (u >= units) return;
  Unit w = unit_of(u);
  begin(w);
  for (int s = 0; s < C::kStages; ++s) load_stage(s);
  while (true) {
#pragma unroll
    for (int i = 0; i < C::kFragN; ++i)
#pragma unroll
      for (int j = 0; j < C::kFragK; ++j) acc[i][j] = (f32x4){0.f, 0.f, 0.f, 0.f};
    if (w.stages > 0) {
      Right even, odd;
      __builtin_amdgcn_s_waitcnt(WaitVmLgkm0<(C::kStages - 1) * C::kLoads>::value);
      lds_barrier();
      {
        Raw raw;
        read_right(base, raw, even);
#pragma unroll
        for (int i = 0; i < C::kFragN; ++i) fn[i] = frag16(base + at_n[i], C::kPitchN);
#pragma unroll
        for (int j = 0; j < C::kFragK; ++j) convert(raw, even, j);
      }
      int buffer = 0;
      auto after = [](int b) { return b + 1 == C::kStages ? 0 : b + 1; };
      for (int s = 0;;) {
        int to = after(buffer);
        step(even, odd, buffer, to);
        buffer = to;
        if (++s == w.stages) break;
        to = after(buffer);
        step(odd, even, buffer, to);
        buffer = to;
        if (++s == w.stages) break;
      }
    }
    // nothing may be on its way to LDS, nor be read there, when the next tile's loads begin
    __builtin_amdgcn_s_waitcnt(WaitVmLgkm0<0>::value);
    lds_barrier();
    const Unit last = w;
    u += grid;
    const bool more = u < units;
    if (more) {
      w = unit_of(u);
      begin(w);
      for (int s = 0; s < C::kStages; ++s) load_stage(s);
    }
    put(last);
    if (!more) break;
  }
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

// 256 x 256 tiles need 256 of them to fill the device.
bool big_tiles(int64_t n, int64_t k, int groups) { return tiles(n, k, 256, 256) * groups >= 200; }

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

int weight_grad_splits(int64_t rows, int64_t n, int64_t k, int groups) {
  if (big_tiles(n, k, groups)) return 1;
  const int64_t units = tiles(n, k, 128, 128) * groups;
  const int64_t steps = (rows / groups + kStep - 1) / kStep;   // of a group of average size
  int64_t s = units > 0 ? 512 / units : 1;
  if (s > steps / 8) s = steps / 8;
  return (int)(s < 1 ? 1 : s > 64 ? 64 : s);
}

hipError_t launch_weight_grad(const WeightGradParams& p, bool x_fp8, int out_dtype, hipStream_t stream) {
  const bool f32 = out_dtype == DG_F32;
  const hipError_t err = launch(p, x_fp8, f32, stream);
  if (err != hipSuccess || p.splits <= 1) return err;
  const int64_t all = (int64_t)p.groups * p.n * (p.k / 4);
  const dim3 grid((unsigned)((all + 255) / 256));
  if (f32) hipLaunchKernelGGL((weight_grad_sum_kernel<true>), grid, dim3(256), 0, stream, p);
  else hipLaunchKernelGGL((weight_grad_sum_kernel<false>), grid, dim3(256), 0, stream, p);
  return hipGetLastError();
}

}  // namespace dgfp8

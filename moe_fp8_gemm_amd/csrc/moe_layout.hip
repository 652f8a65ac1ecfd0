// Layout of the chosen experts' rows.
//
// Mathematics.  Slot s = t * topk + j holds expert e(s) (or none).  With
// count_e = #{s : e(s) = e}, slot s gets the row
//   start_e + #{s' < s : e(s') = e(s)},
// where start_e is the sum of the earlier experts' counts, each rounded up to a
// multiple of 128 (contiguous layout), or e * max_m (masked layout).  The sort is
// stable, so the layout is a function of the indices alone: no result depends on
// the order in which workgroups or atomics run.
//
// Little is read and written (12 bytes a slot, 8 a row), so the time is launches
// and dependent steps.  Up to 3072 slots one launch does it all: every workgroup
// counts all slots by itself, the first writes the slots' rows, and all share the
// rows that hold nothing.  Beyond, a first launch counts each workgroup's slots
// per expert, and in the second each workgroup adds up the counts before its
// own; past kSumBlocks workgroups, where that grows with their square, a launch between the
// two replaces the counts by their sums.  Inside a workgroup each wave ranks its consecutive slots 64 at a time
// with ballots over the bits of the expert number.
// Measured, 256 experts, top 8: 1 token 4.2 us, 64 tokens 4.8, 256 tokens 6.9 (two launches: 9.1), 320
// tokens 8.1 (8.4), 512 tokens 8.6 (one launch: 9.9), 4096 tokens 8.6, 32768 tokens 17, 1 M
// tokens 124.
#include "elem_types.h"
#include "moe_internal.h"

namespace dgfp8 {
namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
static_assert(kThreads >= kMaxExperts, "one thread for each expert");

// Expert of slot s, -1 for none.
__device__ __forceinline__ int expert_at(const LayoutParams& p, int64_t s) {
  if (s >= p.slots) return -1;
  int64_t at = s;
  if (p.ldi != p.topk) {   // slots are below 2^30: 32-bit division
    const uint32_t t = (uint32_t)s / (uint32_t)p.topk;
    at = t * p.ldi + ((uint32_t)s - t * p.topk);
  }
  const int e = p.indices[at];
  return e >= 0 && e < p.experts ? e : -1;
}

template <int kSteps>
__global__ void __launch_bounds__(kThreads) layout_count_kernel(LayoutParams p) {
  __shared__ int count[kMaxExperts];
  count[threadIdx.x] = 0;
  __syncthreads();
  const int64_t s0 = (int64_t)blockIdx.x * (kSteps * kThreads);
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int e = expert_at(p, s0 + i * kThreads + threadIdx.x);
    if (e >= 0) atomicAdd(&count[e], 1);   // whole numbers: any order gives the same count
  }
  __syncthreads();
  if ((int)threadIdx.x < p.experts) p.hist[(int64_t)blockIdx.x * p.experts + threadIdx.x] = count[threadIdx.x];
}

// Each workgroup's counts become the sums over the workgroups before it, and the row behind the last
// the sums over all.  A workgroup takes 64 experts; each of its waves adds up a run of rows, then
// walks it again from the sum of the earlier runs.
__global__ void __launch_bounds__(kThreads) layout_sum_kernel(LayoutParams p) {
  __shared__ int run_sum[kWaves][64];
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const int e = blockIdx.x * 64 + lane;
  const int per = (p.blocks + kWaves - 1) / kWaves;
  const int b0 = wave * per, b1 = min(b0 + per, p.blocks);
  int sum = 0;
  if (e < p.experts) {
#pragma unroll 8
    for (int b = b0; b < b1; ++b) sum += p.hist[(int64_t)b * p.experts + e];
  }
  run_sum[wave][lane] = sum;
  __syncthreads();
  if (e >= p.experts) return;
  int before = 0;
  for (int w = 0; w < wave; ++w) before += run_sum[w][lane];
  if (wave == kWaves - 1) p.hist[(int64_t)p.blocks * p.experts + e] = before + sum;
  constexpr int kBatch = 8;   // counts in flight
  for (int b = b0; b < b1; b += kBatch) {
    int c[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) c[i] = b + i < b1 ? p.hist[(int64_t)(b + i) * p.experts + e] : 0;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (b + i < b1) p.hist[(int64_t)(b + i) * p.experts + e] = before;
      before += c[i];
    }
  }
}

// kCounted: layout_count_kernel has filled p.hist, and each workgroup places its
// own slots; otherwise every workgroup counts all slots and the first places them.
// kSteps: runs of 64 slots of a wave.
template <bool kCounted, int kExperts, int kSteps>
__global__ void __launch_bounds__(kThreads) layout_place_kernel(LayoutParams p) {
  __shared__ int wave_count[kWaves][kExperts];   // slots of an expert in each wave; then the slots before the wave's
  __shared__ int wave_sum[kWaves];
  __shared__ int start[kExperts];                // first row of an expert
  __shared__ int held[kExperts];                 // its rows that hold a slot
  __shared__ int end_row;
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const int e_mine = threadIdx.x;                // the expert this thread adds up
  for (int i = threadIdx.x; i < kWaves * kExperts; i += kThreads) (&wave_count[0][0])[i] = 0;
  __syncthreads();

  // ---- rank each slot among its wave's slots of the same expert
  const int64_t s0 = (kCounted ? (int64_t)blockIdx.x * (kSteps * kThreads) : 0) + wave * (kSteps * 64);
  const int bits = 32 - __builtin_clz(p.experts);   // experts <= 2^bits - 1
  int expert[kSteps], rank[kSteps];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) expert[i] = expert_at(p, s0 + i * 64 + lane);
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int e = expert[i];
    uint64_t same = __builtin_amdgcn_ballot_w64(e >= 0);
    if (same == 0) {   // a whole run past the end
      rank[i] = 0;
      continue;
    }
    for (int b = 0; b < bits; ++b) {
      const bool set = (e >> b) & 1;
      const uint64_t m = __builtin_amdgcn_ballot_w64(set);
      same &= set ? m : ~m;
    }
    const int before = __builtin_popcountll(same & ((1ull << lane) - 1));
    const int seen = e >= 0 ? wave_count[wave][e] : 0;
    rank[i] = seen + before;
    wave_sync();   // every read of a count comes before its update
    if (e >= 0 && before == 0) wave_count[wave][e] = seen + __builtin_popcountll(same);
    wave_sync();
  }
  __syncthreads();

  // ---- counts, and the rows the experts start at
  int mine = 0, earlier = 0;   // of expert e_mine: all slots, slots of earlier workgroups
  if (e_mine < p.experts) {
    if constexpr (kCounted) {
      if (p.blocks > kSumBlocks) {
        mine = p.hist[(int64_t)p.blocks * p.experts + e_mine];
        earlier = p.hist[(int64_t)blockIdx.x * p.experts + e_mine];
      } else {
#pragma unroll 8
        for (int b = 0; b < p.blocks; ++b) {
          const int c = p.hist[(int64_t)b * p.experts + e_mine];
          mine += c;
          earlier += b < (int)blockIdx.x ? c : 0;
        }
      }
    } else {
#pragma unroll
      for (int w = 0; w < kWaves; ++w) mine += wave_count[w][e_mine];
    }
  }
  const int padded = (mine + kExpertAlignment - 1) / kExpertAlignment * kExpertAlignment;
  int incl = padded;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int v = __shfl_up(incl, off, 64);
    if (lane >= off) incl += v;
  }
  if (lane == 63) wave_sum[wave] = incl;
  __syncthreads();
  int first = incl - padded;
  for (int w = 0; w < wave; ++w) first += wave_sum[w];
  if (threadIdx.x == kThreads - 1) end_row = first + padded;
  const bool masked = p.max_m > 0;
  if (e_mine < p.experts) {
    const int64_t limit = masked ? p.max_m : p.rows;   // of rows of this expert / of all rows
    if (masked) first = e_mine * (int)p.max_m;
    start[e_mine] = first;
    held[e_mine] = masked ? (int)(mine < limit ? mine : limit) : mine;
    if (blockIdx.x == 0) p.counts[e_mine] = held[e_mine];
    int run = earlier;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const int c = wave_count[w][e_mine];
      wave_count[w][e_mine] = run;
      run += c;
    }
  }
  __syncthreads();

  // ---- the slots' rows
  if (kCounted || blockIdx.x == 0) {
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int64_t s = s0 + i * 64 + lane;
      if (s >= p.slots) continue;
      const int e = expert[i];
      int row = -1;
      if (e >= 0) {
        const int64_t in_expert = wave_count[wave][e] + rank[i], at = start[e] + in_expert;
        if (masked ? in_expert < p.max_m : at < p.rows) row = (int)at;   // else no room: the slot is dropped
      }
      p.slot_row[s] = row;
      if (row >= 0) {
        p.row_slot[row] = (int)s;
        if (!masked) p.m_indices[row] = e;
      }
    }
  }

  // ---- the rows that hold nothing: between the experts, then behind the last
  auto clear = [&](int64_t r) {
    p.row_slot[r] = -1;
    if (!masked) p.m_indices[r] = -1;
  };
  for (int e = blockIdx.x * kWaves + wave; e < p.experts; e += gridDim.x * kWaves) {
    const int h = held[e];
    const int64_t r0 = (int64_t)start[e] + h;
    int64_t r1 = masked ? (int64_t)(e + 1) * p.max_m
                        : (int64_t)start[e] + (h + kExpertAlignment - 1) / kExpertAlignment * kExpertAlignment;
    if (r1 > p.rows) r1 = p.rows;
    for (int64_t r = r0 + lane; r < r1; r += 64) clear(r);
  }
  if (!masked)
    for (int64_t r = (int64_t)end_row + blockIdx.x * kThreads + threadIdx.x; r < p.rows;
         r += (int64_t)gridDim.x * kThreads)
      clear(r);
}

template <bool kCounted, int kSteps>
void place(const LayoutParams& p, int grid, hipStream_t stream) {
  if (p.experts <= 256) {
    hipLaunchKernelGGL((layout_place_kernel<kCounted, 256, kSteps>), dim3(grid), dim3(kThreads), 0, stream, p);
  } else {
    hipLaunchKernelGGL((layout_place_kernel<kCounted, kMaxExperts, kSteps>), dim3(grid), dim3(kThreads), 0, stream, p);
  }
}

template <int kSteps>
hipError_t count_and_place(const LayoutParams& p, hipStream_t stream) {
  hipLaunchKernelGGL((layout_count_kernel<kSteps>), dim3(p.blocks), dim3(kThreads), 0, stream, p);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  if (p.blocks > kSumBlocks) {
    hipLaunchKernelGGL(layout_sum_kernel, dim3((p.experts + 63) / 64), dim3(kThreads), 0, stream, p);
    if ((err = hipGetLastError()) != hipSuccess) return err;
  }
  place<true, kSteps>(p, p.blocks, stream);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_layout(const LayoutParams& p, hipStream_t stream) {
  static_assert(kOneLaunchSlots == 3 * kThreads, "steps of the one launch");
  if (p.slots <= kOneLaunchSlots) {
    // one workgroup for each 4096 rows and each 32 experts, which they share the clearing of
    int64_t grid = (p.rows + 4095) / 4096;
    if (grid < (p.experts + 31) / 32) grid = (p.experts + 31) / 32;
    if (grid > 64) grid = 64;
    if (p.slots <= kThreads) {
      place<false, 1>(p, (int)grid, stream);
    } else if (p.slots <= 2 * kThreads) {
      place<false, 2>(p, (int)grid, stream);
    } else {
      place<false, 3>(p, (int)grid, stream);
    }
    return hipGetLastError();
  }
  return layout_block_slots(p.slots) == kThreads ? count_and_place<1>(p, stream) : count_and_place<4>(p, stream);
}

}  // namespace dgfp8

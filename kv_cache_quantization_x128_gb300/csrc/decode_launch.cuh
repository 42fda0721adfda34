// What the launches of decode attention share: the scan of the sequences' tiles.
#pragma once
#include "decode_tile.cuh"
#include "kvarn_launch.h"
#include "kvarn_pdl.cuh"

namespace kvarn {
namespace {

// ------------------------------------------------------------------ scan
// Exclusive prefix of full tiles per sequence: each thread a contiguous chunk of
// sequences, then a warp-shuffle scan and a scan of the 32 warp totals.
__global__ void __launch_bounds__(1024) decode_scan_kernel(DecodeArgs a) {
  griddep_launch_dependents();          // the split kernel waits for this grid itself
  __shared__ int64_t warp_sums[32];
  const int t = threadIdx.x, lane = t & 31, w = t >> 5;
  const int per = (a.n_seqs + 1023) / 1024;
  const int s0 = min(t * per, a.n_seqs), s1 = min(s0 + per, a.n_seqs);
  int64_t sum = 0;
  bool clipped = false;
  for (int s = s0; s < s1; ++s) {
    sum += full_tiles(a, s);
    clipped |= max(a.seq_lens[s], 0) / kB > a.max_blocks;
  }
  if (clipped) raise_flag(a.flags, KVARN_FLAG_BAD_LENGTH);
  int64_t incl = sum;                   // inclusive scan inside the warp
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) warp_sums[w] = incl;
  __syncthreads();
  if (w == 0) {                         // inclusive scan of the warp totals
    int64_t v = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    warp_sums[lane] = v;
  }
  __syncthreads();
  int64_t run = incl - sum + (w > 0 ? warp_sums[w - 1] : 0);
  for (int s = s0; s < s1; ++s) {
    a.prefix[s] = run;
    run += full_tiles(a, s);
  }
  if (t == 1023) a.prefix[a.n_seqs] = warp_sums[31];
  // no unit has a first or last split warp yet (the split kernel marks them)
  const int64_t n_cover = 2 * static_cast<int64_t>(a.n_seqs) * a.hkv;
  for (int64_t i = t; i < n_cover; i += 1024) a.cover[i] = -1;
}

// The merge kernel's wait for the split kernel (its ranges, marks and records).
struct SplitWait {
  static constexpr bool kReady = false;
  __device__ void operator()() const { griddep_wait(); }
};

}  // namespace
}  // namespace kvarn

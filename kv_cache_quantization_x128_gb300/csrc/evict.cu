// Eviction of packed tiles by accumulated attention weight (kvarn_evict_tiles). Per sequence
// and kv-head, of n packed tiles b stay: the first keep_first, the last keep_last, and of
// those between the ones of most weight. A record moves whole, bit for bit.
//
// Attention does not see the order of the tiles between, so nothing is shifted together:
// the tiles that stay at slots [b - last, n) fill the evicted slots below, and the last ones
// slide down in order. A random choice of b of n tiles then moves about b (n - b) / n records a
// kv-head instead of nearly b, and a sequence one tile above its budget keep_last + 1.
//
// evict_select_kernel - a block per (sequence, kv-head), about eight tiles a thread. The
//   smallest weight that stays is found bit by bit from the top (a count over the block for
//   each bit, until one leaves exactly as many tiles as may stay); ranks by ballots give
//   the slots. No atomics: the same slots at every call.
// evict_move_kernel - the copies, bound by memory. An evicted slot below b starts a path: it takes
//   the record of slot kept[.], whose place, where it is below b itself, takes the next. Paths
//   share no slot, so blocks take paths independently, and a thread copies the same bytes of each
//   record of its path: it has read them before it writes there, and no barrier is needed.
#include "kvarn_common.cuh"
#include "kvarn_launch.h"
#include "kvarn_pdl.cuh"

namespace kvarn {
namespace {

struct EvictArgs {
  const float* weights;         // [n_seqs][hkv][max_blocks]
  float* weights_out;           // the same, or weights itself
  const int32_t* seq_lens;
  int32_t* seq_lens_out;
  const int32_t* block_tables;  // [n_seqs][max_blocks]
  const int32_t* budgets;       // [n_seqs]
  int32_t* kept;                // [n_seqs][hkv][max_blocks]
  uint8_t* cache;
  unsigned* flags;
  int64_t num_blocks;
  int n_seqs, hkv, max_blocks;
  int first, last;
  int key_slots;                // keys held in shared memory
  int per_unit;                 // blocks of the move kernel a (sequence, kv-head)
  int record_bytes;
};

constexpr int kEvictMaxThreads = 1024;
constexpr int kKeySlots = 10240;      // 40 KB; weights of further tiles are read again for every bit
constexpr int kMoveThreads = 128;

// Whole numbers in the order of the weights: -0 as 0, NaN below everything.
__device__ __forceinline__ uint32_t weight_key(float w) {
  const uint32_t u = __float_as_uint(w + 0.f);
  return w != w ? 0u : (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// Sum over the block; `sums` holds a number a warp, and is free again after the next barrier.
__device__ __forceinline__ int block_sum(int x, int* sums) {
  x = __reduce_add_sync(0xffffffffu, x);
  if (blockDim.x == 32) return x;
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = x;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  return __reduce_add_sync(0xffffffffu, lane < static_cast<int>(blockDim.x >> 5) ? sums[lane] : 0);
}

// The thread's rank among those with `p`, counted from `base`, which moves on by their number.
__device__ __forceinline__ int block_rank(bool p, int& base, int* sums) {
  const uint32_t votes = __ballot_sync(0xffffffffu, p);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int rank = base + __popc(votes & ((1u << lane) - 1u));
  if (warps == 1) {
    base += __popc(votes);
    return rank;
  }
  __syncthreads();
  if (lane == 0) sums[warp] = __popc(votes);
  __syncthreads();
  const int v = lane < warps ? sums[lane] : 0;
  rank += __reduce_add_sync(0xffffffffu, lane < warp ? v : 0);
  base += __reduce_add_sync(0xffffffffu, v);
  return rank;
}

__global__ void __launch_bounds__(kEvictMaxThreads) evict_select_kernel(const EvictArgs a) {
  griddep_launch_dependents();          // the move kernel waits for this grid itself
  extern __shared__ uint32_t keys[];
  __shared__ int sums[2][32];
  const int h = blockIdx.x, s = blockIdx.y, tid = threadIdx.x, threads = blockDim.x;
  const int64_t u = static_cast<int64_t>(s) * a.hkv + h;
  const float* w = a.weights + u * a.max_blocks;
  float* wo = a.weights_out + u * a.max_blocks;
  int32_t* kept = a.kept + u * a.max_blocks;
  const int length = a.seq_lens[s], tiles = max(length, 0) / kB, n = min(tiles, a.max_blocks);
  const int budget = a.budgets[s];
  int b = budget < 0 ? n : min(n, budget);
  bool sound = tiles <= a.max_blocks;
  if (!sound && tid == 0) raise_flag(a.flags, KVARN_FLAG_BAD_LENGTH);
  if (b < n && sound) {                 // every block that could be read or written
    bool ok = true;
    for (int t = tid; t < n; t += threads) {
      const int64_t blk = a.block_tables[static_cast<int64_t>(s) * a.max_blocks + t];
      ok &= blk >= 0 && blk < a.num_blocks;
    }
    sound = __syncthreads_and(ok);
    if (!sound && tid == 0) raise_flag(a.flags, KVARN_FLAG_BAD_BLOCK);
  }
  if (!sound) {                         // the sequence stays as it is
    for (int t = tid; t < a.max_blocks; t += threads) {
      kept[t] = t < n ? t : -1;
      const float x = w[t];
      wo[t] = x;
    }
    if (h == 0 && tid == 0) a.seq_lens_out[s] = length;
    return;
  }

  const int first = min(a.first, b), last = min(a.last, b - first);
  const int lo = first, hi = n - last, quota = b - first - last, edge = b - last;
  // the smallest key that stays is above `cut`, or is `cut` for the first `ties` tiles that have it
  uint32_t cut = 0;
  int ties = 0;
  const bool choose = quota > 0 && quota < hi - lo;
  if (choose) {
    const int held = min(hi, lo + a.key_slots);
    for (int i = lo + tid; i < held; i += threads) keys[i - lo] = weight_key(w[i]);   // (each thread reads its own)
    auto count_from = [&](uint32_t least, int* sm) {
      int c = 0;
      for (int i = lo + tid; i < hi; i += threads) c += (i < held ? keys[i - lo] : weight_key(w[i])) >= least;
      return block_sum(c, sm);
    };
    bool exact = false;
    for (int bit = 31; bit >= 0 && !exact; --bit) {
      const uint32_t least = cut | 1u << bit;
      const int c = count_from(least, sums[bit & 1]);
      if (c >= quota) cut = least;
      exact = c == quota;
    }
    if (exact) {
      --cut;                            // cut > 0: a bit was just set
    } else {
      __syncthreads();
      // (no key has all bits set, so cut + 1 does not wrap: that would be a NaN's)
      ties = quota - count_from(cut + 1u, sums[0]);
    }
  }
  int eq = 0, gone = 0, late = 0;       // ties, evicted tiles and moved tiles so far
  for (int i0 = lo; i0 < hi; i0 += threads) {
    const int i = i0 + tid;
    const bool live = i < hi;
    bool stays = live && (!choose ? quota > 0 : false);
    if (choose) {
      const uint32_t k = live ? (i - lo < a.key_slots ? keys[i - lo] : weight_key(w[i])) : 0u;
      const bool tie = live && ties > 0 && k == cut;
      if (ties > 0) {
        const int r = block_rank(tie, eq, sums[0]);
        stays = live && (k > cut || (tie && r < ties));
      } else {
        stays = live && k > cut;
      }
    }
    const int g = block_rank(live && !stays, gone, sums[0]);
    const bool moves = stays && i >= edge;
    const int m = block_rank(moves, late, sums[1]);
    if (live && !stays) kept[b + g] = i;
    if (stays && !moves) kept[i] = i;
    __syncthreads();                    // the evicted slots so far are listed; the m-th is the moved tile's place
    if (moves) kept[kept[b + m]] = i;
  }
  for (int i = tid; i < first; i += threads) kept[i] = i;
  for (int i = tid; i < last; i += threads) kept[edge + i] = hi + i;
  for (int i = n + tid; i < a.max_blocks; i += threads) kept[i] = -1;
  __syncthreads();
  // Weights follow their tiles, the partial tile's the last of them (kept[i] >= i: where weights_out
  // is weights, what a round reads no earlier round has written).
  for (int i0 = 0; i0 < a.max_blocks; i0 += threads) {
    const int i = i0 + tid;
    const bool take = i < b || (i == b && n < a.max_blocks);
    float x = 0.f;
    if (i < a.max_blocks && take) x = w[i < b ? kept[i] : n];
    __syncthreads();
    if (i < a.max_blocks) wo[i] = x;
  }
  if (h == 0 && tid == 0) a.seq_lens_out[s] = length - (n - b) * kB;
}

template <int kPieces>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictArgs a) {
  griddep_wait();                       // the slots and the lengths
  const int64_t u = blockIdx.x / a.per_unit;
  const int part = blockIdx.x - static_cast<int>(u) * a.per_unit;
  const int s = static_cast<int>(u / a.hkv), h = static_cast<int>(u - static_cast<int64_t>(s) * a.hkv);
  const int length = a.seq_lens[s], n = min(max(length, 0) / kB, a.max_blocks);
  const int dropped = (length - a.seq_lens_out[s]) / kB, b = n - dropped;
  const int32_t* kept = a.kept + u * a.max_blocks;
  const int32_t* table = a.block_tables + static_cast<int64_t>(s) * a.max_blocks;
  const int pieces = a.record_bytes / 16;
  for (int i = part; i < dropped; i += a.per_unit) {
    int slot = kept[b + i];
    if (slot >= b) return;              // (ascending: no evicted slot below b is left)
    uint4* dst = reinterpret_cast<uint4*>(a.cache + (static_cast<int64_t>(table[slot]) * a.hkv + h) * a.record_bytes);
    do {
      slot = kept[slot];
      uint4* src = reinterpret_cast<uint4*>(a.cache + (static_cast<int64_t>(table[slot]) * a.hkv + h) * a.record_bytes);
      uint4 v[kPieces];
#pragma unroll
      for (int p = 0; p < kPieces; ++p)
        if (p * kMoveThreads + threadIdx.x < pieces) v[p] = __ldcg(src + p * kMoveThreads + threadIdx.x);
#pragma unroll
      for (int p = 0; p < kPieces; ++p)
        if (p * kMoveThreads + threadIdx.x < pieces) __stcg(dst + p * kMoveThreads + threadIdx.x, v[p]);
      dst = src;
    } while (slot < b);
  }
}

template <int kPieces>
cudaError_t launch_move(const EvictArgs& a, int64_t grid, cudaStream_t stream) {
  return launch_after(evict_move_kernel<kPieces>, dim3(static_cast<unsigned>(grid)), dim3(kMoveThreads), 0, stream, a);
}

}  // namespace

cudaError_t launch_evict(const float* weights, float* weights_out, const int32_t* seq_lens, int32_t* seq_lens_out,
                         const int32_t* block_tables, const int32_t* budgets, int n_seqs, int hkv, int max_blocks,
                         int64_t num_blocks, int keep_first, int keep_last, int32_t* kept, uint8_t* cache,
                         int record_bytes, unsigned* flags, cudaStream_t stream) {
  EvictArgs a{};
  a.weights = weights;
  a.weights_out = weights_out;
  a.seq_lens = seq_lens;
  a.seq_lens_out = seq_lens_out;
  a.block_tables = block_tables;
  a.budgets = budgets;
  a.kept = kept;
  a.cache = cache;
  a.flags = flags;
  a.num_blocks = num_blocks;
  a.n_seqs = n_seqs;
  a.hkv = hkv;
  a.max_blocks = max_blocks;
  a.first = keep_first;
  a.last = keep_last;
  a.record_bytes = record_bytes;
  a.key_slots = max_blocks < kKeySlots ? max_blocks : kKeySlots;
  int threads = (max_blocks / 8 + 31) / 32 * 32;
  threads = threads < 32 ? 32 : threads > kEvictMaxThreads ? kEvictMaxThreads : threads;
  evict_select_kernel<<<dim3(hkv, n_seqs), threads, a.key_slots * sizeof(uint32_t), stream>>>(a);
  const cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess) return err;
  // as many blocks a unit as fill the GPU, at most one for each of a unit's paths (no more than half its tiles)
  const int64_t units = static_cast<int64_t>(n_seqs) * hkv, fill = 16 * static_cast<int64_t>(decode_num_ctas());
  int64_t per = (fill + units - 1) / units;
  if (per > max_blocks / 2) per = max_blocks / 2;
  a.per_unit = static_cast<int>(per < 1 ? 1 : per);
  const int64_t grid = units * a.per_unit;
  const int pieces = (record_bytes / 16 + kMoveThreads - 1) / kMoveThreads;   // 5, 7 or 9
  return pieces <= 5 ? launch_move<5>(a, grid, stream)
         : pieces <= 7 ? launch_move<7>(a, grid, stream) : launch_move<9>(a, grid, stream);
}

}  // namespace kvarn

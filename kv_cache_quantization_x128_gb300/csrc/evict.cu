// Eviction of packed tiles by accumulated attention weight (kvarn_evict_tiles). Per sequence
// and kv-head, of n packed tiles b stay: the first keep_first, the last keep_last, and of
// those between the ones of most weight. A record moves whole, bit for bit.
//
// Attention does not see the order of the tiles between, so nothing is shifted together:
// the tiles that stay at slots [b - last, n) fill the evicted slots below, and the last ones
// slide down in order. A random choice of b of n tiles then moves about b (n - b) / n records a
// kv-head instead of nearly b, and a sequence one tile above its budget keep_last + 1.
//
// evict_select_kernel - a block per (sequence, kv-head), about two tiles a thread. The
//   smallest weight that stays is found two bits at a time from the top, by one warp without a barrier for up to 512
//   tiles to choose from (search_warp), else by the block with a barrier a count (search_block); ranks by ballots,
//   two barriers each, give the slots. No atomics: the same slots at every call. Bound by latency: a thread's first
//   weights and table entries are loaded with the length and the budget, then come the search, the
//   ranks and the lists (128 tiles 5.6 us, 1024 tiles 8.2, 2048 blocks of up to 256 at once 8.8).
// evict_move_kernel - the copies, at the rate of a plain copy (16 x 16384 tokens to half, k4v2: 20 us of 127 MB).
//   An evicted slot below b starts a path: it takes the record of slot kept[.], whose place, where it is
//   below b itself, takes the next. Paths share no slot, so blocks take paths independently, and a thread
//   copies the same bytes of each record of its path: it has read them before it writes there, and
//   no barrier is needed.
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
  int key_slots;                // keys held in shared memory (of the first tiles to choose from), and behind them
  int list_slots;               // max_blocks where the slots' list is held there too, 0 where `kept` is the list
  int per_unit;                 // blocks of the move kernel a (sequence, kv-head)
  int record_bytes;
};

constexpr int kEvictMaxThreads = 1024;
// 40 KB. Keys are held by their place among the tiles to choose from, lo .. hi - 1, which may lie anywhere
// in the row (a long keep_first); weights behind the held ones are read again for every two bits.
constexpr int kKeySlots = 10240;
constexpr int kListSlots = 5120;      // the most blocks of a row whose list is held beside the keys
// Up to so many tiles to choose from are one warp's: every warp of a block with tiles of its own and barriers between
// the counts took 2048 blocks of 256 tiles 22 us, bound by instructions, where the warp took 11 (8.8 since the first
// loads go out together).
constexpr int kWarpTiles = 512;
static_assert(kWarpTiles <= kKeySlots, "its keys, of places 0 .. kWarpTiles - 1, are held");
constexpr int kMoveThreads = 128;

// Whole numbers in the order of the weights: -0 as 0, NaN below everything.
__device__ __forceinline__ uint32_t weight_key(float w) {
  const uint32_t u = __float_as_uint(w + 0.f);
  return w != w ? 0u : (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// Of the keys at places 0 .. count - 1, the smallest that stays where `quota` (0 < quota < count) stay: it is above `cut`, or is `cut` for
// the first `ties` places that have it. One warp, with KPL keys a lane in registers (count <= 32 KPL, all held).
//   Few tiles to evict (a sequence at its budget has one): the smallest key, then the next one, ...
//   until enough are counted.
//   Else two bits at a time from the top: three counts each, until one leaves exactly the quota.
template <int KPL>
__device__ __forceinline__ void search_warp(const uint32_t* keys, int count, int quota, uint32_t& cut, int& ties) {
  constexpr uint32_t kAll = 0xffffffffu;           // above every key: what is behind the last
  uint32_t k[KPL];
#pragma unroll
  for (int j = 0; j < KPL; ++j) {
    const int i = static_cast<int>(threadIdx.x & 31) + 32 * j;
    k[j] = i < count ? keys[i] : kAll;
  }
  const int evict = count - quota;
  if (evict <= 4) {
    bool any = false;
    int below = 0;                                 // keys up to `cut`
    do {
      uint32_t least = kAll;
#pragma unroll
      for (int j = 0; j < KPL; ++j)
        if (!any || k[j] > cut) least = min(least, k[j]);
      cut = __reduce_min_sync(kAll, least);
      any = true;
      int c = 0;
#pragma unroll
      for (int j = 0; j < KPL; ++j) c += k[j] <= cut;
      below = __reduce_add_sync(kAll, c);
    } while (below < evict);
    ties = below - evict;
    return;
  }
  const int want = quota + KPL * 32 - count;       // (what is behind the last is counted too)
  cut = 0;
  ties = 0;
#pragma unroll 1
  for (int bit = 30; bit >= 0; bit -= 2) {
    const uint32_t k0 = cut | 1u << bit, k1 = cut | 2u << bit, k2 = cut | 3u << bit;
    int c0 = 0, c1 = 0, c2 = 0;
#pragma unroll
    for (int j = 0; j < KPL; ++j) {
      c0 += k[j] >= k0;
      c1 += k[j] >= k1;
      c2 += k[j] >= k2;
    }
    c0 = __reduce_add_sync(kAll, c0);
    c1 = __reduce_add_sync(kAll, c1);
    c2 = __reduce_add_sync(kAll, c2);
    const int c = c2 >= want ? c2 : c1 >= want ? c1 : c0;
    cut = c2 >= want ? k2 : c1 >= want ? k1 : c0 >= want ? k0 : cut;
    if (c == want) {
      --cut;                                       // (a bit was just set)
      return;
    }
  }
  int c = 0;
#pragma unroll
  for (int j = 0; j < KPL; ++j) c += k[j] > cut;
  ties = want - __reduce_add_sync(kAll, c);
}

// The same for any number of tiles, by the whole block; keys from place `slots` on come from the weights w.
__device__ __forceinline__ void search_block(const uint32_t* keys, int slots, const float* w, int count, int quota, uint32_t& cut,
                                             int& ties) {
  __shared__ int sums[2][3][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  // a thread's first two keys stay in registers (0 where there is none: below every threshold)
  const int i0 = static_cast<int>(threadIdx.x), i1 = i0 + static_cast<int>(blockDim.x);
  const uint32_t key0 = i0 < min(count, slots) ? keys[i0] : i0 < count ? weight_key(w[i0]) : 0u;
  const uint32_t key1 = i1 < min(count, slots) ? keys[i1] : i1 < count ? weight_key(w[i1]) : 0u;
  auto tally = [&](int (&c)[3], uint32_t k0, uint32_t k1, uint32_t k2, int (*sm)[32]) {
    c[0] = (key0 >= k0) + (key1 >= k0);
    c[1] = (key0 >= k1) + (key1 >= k1);
    c[2] = (key0 >= k2) + (key1 >= k2);
    for (int i = i1 + static_cast<int>(blockDim.x); i < count; i += static_cast<int>(blockDim.x)) {
      const uint32_t k = i < slots ? keys[i] : weight_key(w[i]);
      c[0] += k >= k0;
      c[1] += k >= k1;
      c[2] += k >= k2;
    }
#pragma unroll
    for (int j = 0; j < 3; ++j) c[j] = __reduce_add_sync(0xffffffffu, c[j]);
    if (lane == 0)
#pragma unroll
      for (int j = 0; j < 3; ++j) sm[j][warp] = c[j];
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 3; ++j) c[j] = __reduce_add_sync(0xffffffffu, lane < warps ? sm[j][lane] : 0);
  };
  cut = 0;
  ties = 0;
  int c[3];
#pragma unroll 1
  for (int bit = 30; bit >= 0; bit -= 2) {         // (sums alternate: a barrier lies between their uses)
    const uint32_t k0 = cut | 1u << bit, k1 = cut | 2u << bit, k2 = cut | 3u << bit;
    tally(c, k0, k1, k2, sums[bit >> 1 & 1]);
    const int most = c[2] >= quota ? c[2] : c[1] >= quota ? c[1] : c[0];
    cut = c[2] >= quota ? k2 : c[1] >= quota ? k1 : c[0] >= quota ? k0 : cut;
    if (most == quota) {
      --cut;
      return;
    }
  }
  // (no key has all bits set, so cut + 1 does not wrap: that would be a NaN's)
  tally(c, cut + 1u, cut + 1u, cut + 1u, sums[1]);
  ties = quota - c[0];
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
  __shared__ int ranks[3][32];
  __shared__ uint32_t found[2];
  const int h = blockIdx.x, s = blockIdx.y, tid = threadIdx.x, threads = blockDim.x;
  const int64_t u = static_cast<int64_t>(s) * a.hkv + h;
  const float* w = a.weights + u * a.max_blocks;
  float* wo = a.weights_out + u * a.max_blocks;
  int32_t* kept = a.kept + u * a.max_blocks;
  int32_t* list = a.list_slots > 0 ? reinterpret_cast<int32_t*>(keys + a.key_slots) : kept;
  const int32_t* table = a.block_tables + static_cast<int64_t>(s) * a.max_blocks;
  // a thread's first two tiles, in flight with the length
  float w2[2] = {0.f, 0.f};
  int32_t blk2[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 2; ++j)
    if (tid + j * threads < a.max_blocks) {
      w2[j] = w[tid + j * threads];
      blk2[j] = table[tid + j * threads];
    }
  const int length = a.seq_lens[s], budget = a.budgets[s];
  const int tiles = max(length, 0) / kB, n = min(tiles, a.max_blocks), b = budget < 0 ? n : min(n, budget);
  const int first = min(a.first, b), last = min(a.last, b - first);
  const int lo = first, hi = n - last, quota = b - first - last, edge = b - last;
  const unsigned held = static_cast<unsigned>(min(hi - lo, a.key_slots));    // keys in shared memory: of tiles lo ..
  bool sound = tiles <= a.max_blocks;
  if (!sound && tid == 0) raise_flag(a.flags, KVARN_FLAG_BAD_LENGTH);
  if (b < n && sound) {                 // every block that could be read or written, and the keys
    bool ok = true;
    auto look = [&](int t, int64_t blk, float x) {
      ok &= blk >= 0 && blk < a.num_blocks;
      if (static_cast<unsigned>(t - lo) < held) keys[t - lo] = weight_key(x);
    };
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (tid + j * threads < n) look(tid + j * threads, blk2[j], w2[j]);
    for (int t = tid + 2 * threads; t < n; t += threads) look(t, table[t], w[t]);
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

  uint32_t cut = 0;
  int ties = 0;
  const bool choose = quota > 0 && quota < hi - lo;
  if (choose && hi - lo <= kWarpTiles) {
    if (tid < 32) {
      if (hi - lo <= 64) search_warp<2>(keys, hi - lo, quota, cut, ties);
      else if (hi - lo <= 128) search_warp<4>(keys, hi - lo, quota, cut, ties);
      else if (hi - lo <= 256) search_warp<8>(keys, hi - lo, quota, cut, ties);
      else search_warp<16>(keys, hi - lo, quota, cut, ties);
      if (tid == 0) {
        found[0] = cut;
        found[1] = static_cast<uint32_t>(ties);
      }
    }
    __syncthreads();
    cut = found[0];
    ties = static_cast<int>(found[1]);
  } else if (choose) {
    search_block(keys, a.key_slots, w + lo, hi - lo, quota, cut, ties);
  }
  int eq = 0, gone = 0, late = 0;       // ties, evicted tiles and moved tiles so far
  for (int i0 = lo; i0 < hi; i0 += threads) {
    const int i = i0 + tid;
    const bool live = i < hi;
    bool stays = live && !choose && quota > 0;
    if (choose) {
      const uint32_t k = !live ? 0u : i - lo < a.key_slots ? keys[i - lo] : weight_key(w[i]);
      stays = live && k > cut;
      if (ties > 0) {
        const bool tie = live && k == cut;
        const int r = block_rank(tie, eq, ranks[0]);
        stays |= tie && r < ties;
      }
    }
    const bool moves = stays && i >= edge;
    const int g = block_rank(live && !stays, gone, ranks[1]);
    const int m = block_rank(moves, late, ranks[2]);
    if (live && !stays) list[b + g] = i;
    if (stays && !moves) list[i] = i;
    __syncthreads();                    // the evicted slots so far are listed; the m-th is the moved tile's place
    if (moves) list[list[b + m]] = i;
  }
  for (int i = tid; i < first; i += threads) list[i] = i;
  for (int i = tid; i < last; i += threads) list[edge + i] = hi + i;
  for (int i = n + tid; i < a.max_blocks; i += threads) list[i] = -1;
  __syncthreads();
  // Weights follow their tiles, the partial tile's the last of them (list[i] >= i: where weights_out
  // is weights, what a round reads no earlier round has written).
  for (int i0 = 0; i0 < a.max_blocks; i0 += threads) {
    const int i = i0 + tid;
    float x = 0.f;
    if (i < a.max_blocks) {
      const int from = list[i];
      if (i < b || (i == b && n < a.max_blocks)) x = w[i < b ? from : n];
      if (a.list_slots > 0) kept[i] = from;
    }
    __syncthreads();
    if (i < a.max_blocks) wo[i] = x;
  }
  if (h == 0 && tid == 0) a.seq_lens_out[s] = length - (n - b) * kB;
}

template <int kPieces>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictArgs a) {
  const int64_t u = blockIdx.x / a.per_unit;
  const int part = blockIdx.x - static_cast<int>(u) * a.per_unit;
  const int s = static_cast<int>(u / a.hkv), h = static_cast<int>(u - static_cast<int64_t>(s) * a.hkv);
  const int32_t* kept = a.kept + u * a.max_blocks;
  const int32_t* table = a.block_tables + static_cast<int64_t>(s) * a.max_blocks;
  const int length = a.seq_lens[s], budget = a.budgets[s], n = min(max(length, 0) / kB, a.max_blocks);
  const int b = budget < 0 ? n : min(n, budget), dropped = n - b;
  griddep_wait();                       // the slots and the lengths
  if (dropped <= part || a.seq_lens_out[s] == length) return;       // (as it was: nothing to evict, or not sound)
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
  a.list_slots = max_blocks <= kListSlots ? max_blocks : 0;
  // about two tiles a thread (eight: 16 x 16384 tokens, 128 tiles, 15.5 us of choosing)
  int threads = max_blocks / 2 / 32 * 32;
  threads = threads < 32 ? 32 : threads > kEvictMaxThreads ? kEvictMaxThreads : threads;
  evict_select_kernel<<<dim3(hkv, n_seqs), threads, (a.key_slots + a.list_slots) * sizeof(uint32_t), stream>>>(a);
  const cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess) return err;
  // About three times the blocks that the GPU holds, at most one for each of a unit's paths (no more than half its
  // tiles): paths of a unit are few or many (4 x 131072 to a quarter: 8 blocks an SM 50.6 us, 16 47.9, 32 47.6).
  const int64_t units = static_cast<int64_t>(n_seqs) * hkv, fill = 32 * static_cast<int64_t>(decode_num_ctas());
  int64_t per = (fill + units - 1) / units;
  if (per > max_blocks / 2) per = max_blocks / 2;
  a.per_unit = static_cast<int>(per < 1 ? 1 : per);
  const int64_t grid = units * a.per_unit;
  const int pieces = (record_bytes / 16 + kMoveThreads - 1) / kMoveThreads;   // 5, 7 or 9
  return pieces <= 5 ? launch_move<5>(a, grid, stream)
         : pieces <= 7 ? launch_move<7>(a, grid, stream) : launch_move<9>(a, grid, stream);
}

}  // namespace kvarn

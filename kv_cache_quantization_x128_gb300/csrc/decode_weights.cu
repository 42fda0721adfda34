// Decode attention that also adds up each packed tile's attention weight (what eviction by
// accumulated weight goes by) and gives the log-sum-exp: with x_gj the scores of q-head g,
//   out_g = sum_j p_gj v_j,  p_gj = exp(x_gj - lse_g),  lse_g = ln sum_j exp(x_gj)
//   w_t <- decay w_t + sum over the group's heads g and the tile's tokens j of p_gj
// in one pass over the records. The weights need lse, which is known when the pass is over,
// so the pass leaves (m, l) of each tile and q-head: the running maximum behind the tile and the
// tile's sum of 2^(score - m), 64 bytes beside the record's 10 to 18 KB; the merge, which has
// the unit's maximum and sum, turns them into weights, a thread a tile.
// The tile is the unit of weight because it is that of the record: its per-channel scales
// bind 128 tokens, which cannot leave one record for another without being quantized again.
//
// Two launches (three for few units with many records), each a programmatic dependent of the one before:
//   weigh_split_kernel - persistent, a CTA an SM. The packed tiles of all units (a unit is a sequence and
//     kv-head) lie in one row, and each warp takes an equal part of it (a block finds its
//     warps' parts with a scan over the lengths of its own). A warp copies its next tile into its stage while
//     other warps of its scheduler compute, with the tile after that on its way into L2, and writes
//     a partial record (output, maximum, sum) for each unit that it leaves;
//   weigh_merge_kernel - a block a unit: attends the workspace tokens, joins the records,
//     un-rotates, normalises, and writes the weights (for few units a block a q-head, and
//     weigh_tiles_kernel writes the weights).
//
// Bound by arithmetic: a tile and kv-head is 256 m16n8k16 products (2048 cycles of a scheduler's tensor pipe; the
// legacy products are what small N needs, decode_tc.cuh has the tcgen05 form), 890 instructions of the ALU
// pipe, two cycles each, and about 850 cycles of the fp32 pipe, which hardly overlap: measured 4110
// cycles, ncu 50, 43 and 22 % of them. 64 x 16384 tokens, 64 heads over 8, k4v2: 236 us, 4.0 TB/s of records
// (60 % of the copy rate; the plain decode 239), with groups of four 178 us, 79 %. Batches of short sequences: 256 x 1000
// tokens 103 us, of which the merge has 40 %: a chain of dependent loads a block, which hardly starts beside
// the split, whose CTAs hold nearly all shared memory (alone, ncu: split 64 us, merge 45).
#include "decode_tile.cuh"
#include "kvarn_common.cuh"
#include "kvarn_launch.h"
#include "kvarn_pdl.cuh"
#include "weigh_tile.cuh"

namespace kvarn {
namespace {

struct WeighArgs : DecodeArgs {
  const uint16_t* ws;
  float2* stats;        // [n_seqs][hkv][max_blocks][8]: (m, l) of a tile and q-head
  float* weights;       // [n_seqs][hkv][max_blocks], updated
  float* lse;           // [n_seqs][hkv * group] or NULL
  float4* ends;         // [n_seqs][hkv][8]: HeadEnd of each q-head (few units)
  float decay;
};

// Warps with a record stage and q_r each: 12 (10 for k4v4's 18 KB records), at 168 registers.
template <int KB, int VB, bool kLean>
struct WeighCfg {
  using L = RecordLayout<KB, VB, kLean>;
  static constexpr int kWarps = SplitCfg<KB, VB, kLean>::kWarps;
  static constexpr int kQOff = kWarps * L::kBytes;                  // q_r: [warp][group][lane] float4
  static constexpr int kBarOff = kQOff + kWarps * 4096;
  static constexpr int kSmem = kBarOff + kWarps * 8;
};

// ------------------------------------------------------------------ parts
__device__ __forceinline__ int seq_len(const WeighArgs& a, int s) { return max(a.seq_lens[s], 0); }
__device__ __forceinline__ int tiles_of(const WeighArgs& a, int len) { return min(len / kB, a.max_blocks); }

struct Tile {
  int s, h, it, tiles;  // tile `it` of the `tiles` of unit (s, h)
};

// The first tile of the next unit that has any (s = n_seqs: none).
__device__ __forceinline__ void next_unit(const WeighArgs& a, Tile& c) {
  c.it = 0;
  if (++c.h < a.hkv) return;
  c.h = 0;
  do {
    if (++c.s >= a.n_seqs) return;
    c.tiles = tiles_of(a, seq_len(a, c.s));
  } while (c.tiles == 0);
}

// A warp's part of the row of tiles.
struct Part {
  Tile first;
  int64_t count;
  int id;               // of the warp among those with parts; -1: no part
};

// The row in equal parts, one at least a tile; consecutive parts go to different SMs, so that few of them spread
// out. The block scans the sequences' lengths, then each warp looks its own up. (64-bit divisions
// are few: twelve for every warp had cost the largest batches 16 us.)
template <int kWarps>
__device__ __forceinline__ Part find_part(const WeighArgs& a) {
  constexpr int kThreads = kWarps * 32;
  __shared__ int64_t before[kThreads];              // tiles before a thread's sequences, of one kv-head
  __shared__ int64_t sums[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.n_seqs + kThreads - 1) / kThreads;
  const int s0 = min(tid * per, a.n_seqs), s1 = min(s0 + per, a.n_seqs);
  int64_t own = 0;
  bool cut = false;
#pragma unroll 4
  for (int s = s0; s < s1; ++s) {
    const int len = seq_len(a, s);
    own += tiles_of(a, len);
    cut |= len / kB > a.max_blocks;
  }
  if (cut && blockIdx.x == 0) raise_flag(a.flags, KVARN_FLAG_BAD_LENGTH);
  int64_t upto = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += v;
  }
  if (lane == 31) sums[warp] = upto;
  __syncthreads();
  int64_t total = 0, mine = upto - own;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) mine += sums[w];
    total += sums[w];
  }
  before[tid] = mine;
  __syncthreads();
  total *= a.hkv;
  Part p;
  p.id = warp * gridDim.x + blockIdx.x;
  const unsigned n = static_cast<unsigned>(min(static_cast<int64_t>(gridDim.x) * kWarps, total));
  if (static_cast<unsigned>(p.id) >= n) {
    p.id = -1;
    return p;
  }
  const int64_t whole = total / n;
  const unsigned rest = static_cast<unsigned>(total - whole * n);    // below n <= 2^14
  const int64_t begin = whole * p.id + rest * p.id / n;
  p.count = whole * (p.id + 1) + rest * (p.id + 1) / n - begin;
  // the last thread whose sequences begin at or before the part
  int lo = 0;
#pragma unroll
  for (int step = 256; step > 0; step >>= 1)
    if (lo + step < kThreads && before[lo + step] * a.hkv <= begin) lo += step;
  int64_t off = begin - before[lo] * a.hkv;
  Tile c;
  for (c.s = min(lo * per, a.n_seqs - 1);; ++c.s) { // (a sequence at or behind c.s holds it)
    c.tiles = tiles_of(a, seq_len(a, c.s));
    const int64_t here = static_cast<int64_t>(c.tiles) * a.hkv;
    if (off < here || c.s + 1 >= a.n_seqs) break;
    off -= here;
  }
  c.h = off >> 32 ? static_cast<int>(off / c.tiles) : static_cast<int>(static_cast<unsigned>(off) / static_cast<unsigned>(c.tiles));
  c.it = static_cast<int>(off - static_cast<int64_t>(c.h) * c.tiles);
  p.first = c;
  return p;
}

// Lane 0: the record of a tile; NULL (flag raised) where its block is not there.
template <int kRecBytes>
__device__ __forceinline__ const uint8_t* record_of(const WeighArgs& a, const Tile& c) {
  const int64_t blk = a.block_tables[static_cast<int64_t>(c.s) * a.max_blocks + c.it];
  if (blk < 0 || blk >= a.num_blocks) {
    raise_flag(a.flags, KVARN_FLAG_BAD_BLOCK);
    return nullptr;
  }
  return a.cache + (blk * a.hkv + c.h) * static_cast<int64_t>(kRecBytes);
}

// Lane 0: its copy into the stage (NULL: the barrier's phase completes without one).
template <int kRecBytes>
__device__ __forceinline__ void issue_record(uint8_t* stage, const uint8_t* src, uint64_t* bar) {
  if (src == nullptr) {
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
    return;
  }
  mbar_arrive_expect_tx(bar, kRecBytes);
  bulk_g2s(stage, src, kRecBytes, bar);
}

// ------------------------------------------------------------------ split
template <int KB, int VB, bool kLean, bool kNarrow>
__global__ void __launch_bounds__(WeighCfg<KB, VB, kLean>::kWarps * 32, 1) weigh_split_kernel(const __grid_constant__ WeighArgs a) {
  using Cfg = WeighCfg<KB, VB, kLean>;
  constexpr int kRecBytes = RecordLayout<KB, VB, kLean>::kBytes;
  extern __shared__ __align__(1024) uint8_t smem[];
  griddep_launch_dependents();          // the merge kernel waits for this grid itself
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + Cfg::kBarOff) + warp;
  if (lane == 0) {
    mbar_init(bar, 1);
    fence_mbar_init();
  }
  const Part part = find_part<Cfg::kWarps>(a);
  const int id = part.id;
  if (id < 0) return;                   // warps are independent: no block-wide barrier below
  float4* qsm = reinterpret_cast<float4*>(smem + Cfg::kQOff) + warp * 256 + lane;
  uint8_t* stage = smem + warp * kRecBytes;
  Tile cur = part.first, next = cur;    // the tile in the stage, and the one on its way into L2
  int64_t left = part.count;            // tiles from `cur` on
  const uint8_t *src = nullptr, *ahead = nullptr;   // lane 0: their records
  auto look_ahead = [&] {               // `next` moves on, and into L2
    if (++next.it >= next.tiles) next_unit(a, next);
    if (lane == 0) {
      ahead = record_of<kRecBytes>(a, next);
      if (ahead != nullptr)
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(ahead), "r"(kRecBytes) : "memory");
    }
  };
  if (lane == 0) {
    src = record_of<kRecBytes>(a, cur);
    issue_record<kRecBytes>(stage, src, bar);
  }
  if (left > 1) look_ahead();

  UnitState<kNarrow> state;
  state.reset();
  int first = -1;                       // the warp's first tile of the unit
  for (uint32_t phase = 0;; phase ^= 1u) {
    const int64_t u = static_cast<int64_t>(cur.s) * a.hkv + cur.h;
    if (first < 0) {
      first = cur.it;
      float qv[8][4];
      load_q(a, cur.s, cur.h, state.head(g), c, qv);
      store_q<KB>(qsm, qv);
    }
    float2* stat = a.stats + (u * a.max_blocks + cur.it) * 8;
    // (a copy that never arrives raises its flag and ends the warp)
    if (!__all_sync(0xffffffffu, mbar_wait(bar, phase, a.flags))) return;
    if (__shfl_sync(0xffffffffu, src != nullptr, 0)) {
      state.template attend<KB, VB, kLean>(stage, qsm, g, c, stat);
    } else if (c == 0) {
      stat[g] = make_float2(-INFINITY, 0.f);
    }
    __syncwarp();
    const bool more = --left > 0, same = ++cur.it < cur.tiles;
    if (lane == 0 && more) issue_record<kRecBytes>(stage, ahead, bar);
    if (!more || !same) {               // the warp's last tile of the unit
      state.write(a.part + (id + u) * kRecFloats, kPartStride, a.group, g, c);
      if (lane == 0) {                  // the unit's first and last warp
        if (first == 0) a.cover[2 * u] = id;
        if (!same) a.cover[2 * u + 1] = id;
      }
      if (!more) return;
      first = -1;
      state.reset();
      cur = next;
    }
    src = ahead;
    if (left > 1) look_ahead();
  }
}

// ------------------------------------------------------------------ merge
// The workspace tokens of a unit (exact, unrotated rows of its partial last tile), 16 a warp: per
// warp and q-head the maximum, sum and output (a row padded against bank conflicts).
constexpr int kWsRow = kD + 4;
template <int kHeads>
struct WeighWs {
  float o[8][kHeads][kWsRow];
  float m[8][kHeads], l[8][kHeads];
};

// Warp w's tokens 16 w .. of the n_ws, all q-heads of the group at once. The products' K index is permuted alike in
// both operands, so that the loads are 16 bytes and neighbouring lanes' adjacent: for
// q k, k-steps 2 j and 2 j + 1 of thread (g, c) carry channels 32 j + 8 c + 0..7 of token 16 w + 8 nt + g; for p v, n-tile i's column g is channel 64 half + 8 g + i. Rows 0-7 of q are
// the heads, 8-15 zero; p enters as hi and lo rows, scaled to 2^15, so that weights down to 2^-28 keep their bits.
// kHeads 1: head `only` alone is kept.
template <int kHeads>
__device__ __forceinline__ void weigh_ws(const WeighArgs& a, int64_t u, int n_ws, int w, int only, WeighWs<kHeads>& sm) {
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3, t0 = 16 * w;
  if (t0 >= n_ws) return;
  const uint16_t* wk = a.ws + u * (2 * kB * kD) + t0 * kD;
  const uint16_t* wv = wk + kB * kD;
  asm volatile("prefetch.global.L2 [%0];" ::"l"(wv + lane * 64));    // the 16 rows of V, 128 bytes a lane
  float d[2][4];
  {
    const uint4* qr = reinterpret_cast<const uint4*>(a.q + (u * a.group + min(g, a.group - 1)) * kD + 8 * c);
    const uint4* kr = reinterpret_cast<const uint4*>(wk + g * kD + 8 * c);
    uint4 qv[4], k0[4], k1[4];                     // (rows past n_ws, still inside the unit's, are read and masked out)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      k0[j] = kr[4 * j];
      k1[j] = kr[8 * kD / 8 + 4 * j];
      qv[j] = g < a.group ? qr[4 * j] : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t a0[4] = {qv[j].x, 0u, qv[j].y, 0u}, a1[4] = {qv[j].z, 0u, qv[j].w, 0u};
      if (j == 0) {
        mma16816_first(d[0], a0, k0[j].x, k0[j].y);
        mma16816_first(d[1], a0, k1[j].x, k1[j].y);
      } else {
        mma16816(d[0], a0, k0[j].x, k0[j].y);
        mma16816(d[1], a0, k1[j].x, k1[j].y);
      }
      mma16816(d[0], a1, k0[j].z, k0[j].w);
      mma16816(d[1], a1, k1[j].z, k1[j].w);
    }
  }
  constexpr float kScale = kLog2e * kInvSqrt128, kUp = 32768.f;
  // tokens t0 + 8 nt + 2 c + {0, 1} of head g. The maximum starts finite, below every finite score (|q.k| < 2^40), so that
  // scores of minus infinity (keys beyond fp16's end), even of all the rows, are weights of 0.
  float p[2][2], mx = -1e30f, sum = 0.f;
#pragma unroll
  for (int nt = 0; nt < 2; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      p[nt][e] = t0 + 8 * nt + 2 * c + e < n_ws ? d[nt][e] * kScale : -INFINITY;
      mx = fmaxf(mx, p[nt][e]);
    }
  mx = quad_max(mx);
#pragma unroll
  for (int nt = 0; nt < 2; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      p[nt][e] = exp2f(p[nt][e] - mx);
      sum += p[nt][e];
    }
  sum = quad_sum(sum);
  uint32_t pa[4];
  split2p(make_float2(p[0][0] * kUp, p[0][1] * kUp), pa[0], pa[1]);
  split2p(make_float2(p[1][0] * kUp, p[1][1] * kUp), pa[2], pa[3]);
  const int tk[4] = {2 * c, 2 * c + 1, 2 * c + 8, 2 * c + 9};
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint4 vr[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)                    // (rows behind the last token may hold anything: not multiplied)
      vr[i] = t0 + tk[i] < n_ws ? *reinterpret_cast<const uint4*>(wv + tk[i] * kD + 64 * half + 8 * g)
                                : make_uint4(0u, 0u, 0u, 0u);
    float o[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t sel = (i & 1) ? 0x7632u : 0x5410u;   // high or low halves of two words
      mma16816_first(o[i], pa, __byte_perm((&vr[0].x)[i >> 1], (&vr[1].x)[i >> 1], sel),
                     __byte_perm((&vr[2].x)[i >> 1], (&vr[3].x)[i >> 1], sel));
    }
    // columns 2 c and 2 c + 1 of n-tile i: channels 64 half + 16 c + i and + 8 + i; rows g and g + 8 add up to head g
    if (kHeads == 1 && g != only) continue;
    float4* dst = reinterpret_cast<float4*>(&sm.o[w][kHeads == 1 ? 0 : g][64 * half + 16 * c]);
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int i = 0; i < 8; i += 4)
        dst[2 * e + i / 4] = make_float4((o[i][e] + o[i][e + 2]) / kUp, (o[i + 1][e] + o[i + 1][e + 2]) / kUp,
                                         (o[i + 2][e] + o[i + 2][e + 2]) / kUp, (o[i + 3][e] + o[i + 3][e + 2]) / kUp);
  }
  if (c == 0 && (kHeads > 1 || g == only)) {
    sm.m[w][kHeads == 1 ? 0 : g] = mx;
    sm.l[w][kHeads == 1 ? 0 : g] = sum;
  }
}

// What the weights of a unit's tiles need of q-head g: its maximum, 1 / sum, and the weight of the workspace tokens.
struct HeadEnd {
  float top, inv, tail, pad;
};

// The weight of the tile whose (m, l) are at `stat`, summed in the order of the heads: the same number at every call.
__device__ __forceinline__ float tile_weight(const WeighArgs& a, const float2* stat, const HeadEnd* heads) {
  float w = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float4 v = reinterpret_cast<const float4*>(stat)[j];
    // (a sum of 0: not attended, or too little to count; its maximum is not looked at)
    if (2 * j < a.group && v.y != 0.f) w = fmaf(v.y * exp2f(v.x - heads[2 * j].top), heads[2 * j].inv, w);
    if (2 * j + 1 < a.group && v.w != 0.f) w = fmaf(v.w * exp2f(v.z - heads[2 * j + 1].top), heads[2 * j + 1].inv, w);
  }
  return w;
}
__device__ __forceinline__ void add_weight(const WeighArgs& a, float* at, float w) {
  *at = a.decay == 0.f ? w : fmaf(a.decay, *at, w);
}

// Tiles first, first + stride, ... of the unit, and (first == 0) its partial one, whose weight from the step is
// 0 without a workspace (the old one fades all the same).
__device__ __forceinline__ void weigh_unit(const WeighArgs& a, int64_t u, int len, const HeadEnd* heads, int first, int stride) {
  const int tiles = tiles_of(a, len), last = len / kB;
  float* row = a.weights + u * a.max_blocks;
  for (int t = first; t < tiles; t += stride) add_weight(a, row + t, tile_weight(a, a.stats + (u * a.max_blocks + t) * 8, heads));
  if (first == 0 && len % kB > 0 && last < a.max_blocks) {
    float w = 0.f;
    for (int g = 0; g < a.group; ++g) w += heads[g].tail;
    add_weight(a, row + last, w);
  }
}

// kHeads 8: a block a unit, kShares warps a q-head with every kShares-th record each, then the unit's weights. kHeads 1
// (few units with very many records): a block a q-head; the weights are weigh_tiles_kernel's. Warps 0-7 attend the workspace tokens, which are the call's
// inputs, before the wait for the split kernel.
template <int kHeads, int kShares>
__global__ void __launch_bounds__(32 * kHeads * kShares, kHeads * kShares > 8 ? 1 : 4)
    weigh_merge_kernel(const __grid_constant__ WeighArgs a, uint16_t* __restrict__ out) {
  static_assert(kHeads * kShares >= 8 && (kHeads == 8 || kHeads == 1), "8 warps for the workspace tokens");
  constexpr int kBatch = 4;             // records in flight (8 spill: 1 x 1000 tokens 13.1 us, 12.1 so)
  __shared__ WeighWs<kHeads> ws;
  __shared__ float shares[kShares > 1 ? kShares - 1 : 1][kHeads][kPartStride];
  __shared__ HeadEnd heads[8];
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, s = blockIdx.y;
  const int gg = kHeads == 8 ? warp & 7 : static_cast<int>(blockIdx.x) % a.group, share = warp / kHeads;
  const int wg = kHeads == 8 ? gg : 0;  // the head's row in shared memory
  const int64_t u = static_cast<int64_t>(s) * a.hkv + (kHeads == 8 ? blockIdx.x : blockIdx.x / a.group);
  const int len = seq_len(a, s), tiles = tiles_of(a, len);
  const int n_ws = ws_tokens(a, a.ws, s, threadIdx.x == 0), n_wsw = (n_ws + 15) >> 4;
  if (warp < 8) weigh_ws<kHeads>(a, u, n_ws, warp, gg, ws);
  griddep_wait();
  float M = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};   // channels 4 lane .. 4 lane + 3, rotated
  if (gg < a.group && tiles > 0) {
    const int2 cv = *reinterpret_cast<const int2*>(a.cover + 2 * u);
    // (marks that a warp which gave up did not write may hold anything: nothing outside the records is read)
    const bool sound = cv.x >= 0 && cv.y >= cv.x && cv.y < a.n_ctas * a.warps;
    const int w1 = sound ? cv.y : -1;
    for (int w0 = sound ? cv.x + share : 0; w0 <= w1; w0 += kBatch * kShares) {
      float4 v[kBatch];
      float2 ml[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const float* p = a.part + (min(w0 + j * kShares, w1) + u) * kRecFloats + gg * kPartStride;
        ml[j] = *reinterpret_cast<const float2*>(p + 128);
        v[j] = *reinterpret_cast<const float4*>(p + 4 * lane);
        if (w0 + j * kShares > w1) ml[j] = make_float2(-INFINITY, 0.f);
      }
      float mb = M;
#pragma unroll
      for (int j = 0; j < kBatch; ++j) mb = fmaxf(mb, ml[j].x);
      if (mb > M) {
        const float sc = exp2f(M - mb);           // 0 while M is -inf (nothing summed yet)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[k] *= sc;
        l *= sc;
        M = mb;
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {          // (a sum of 0: nothing was attended)
        const bool use = ml[j].y != 0.f;
        const float f = use ? exp2f(ml[j].x - M) : 0.f;
        acc[0] = fmaf(use ? v[j].x : 0.f, f, acc[0]);
        acc[1] = fmaf(use ? v[j].y : 0.f, f, acc[1]);
        acc[2] = fmaf(use ? v[j].z : 0.f, f, acc[2]);
        acc[3] = fmaf(use ? v[j].w : 0.f, f, acc[3]);
        l = fmaf(use ? ml[j].y : 0.f, f, l);
      }
    }
  }
  if (kShares > 1 && share > 0) {
    *reinterpret_cast<float4*>(&shares[share - 1][wg][4 * lane]) = make_float4(acc[0], acc[1], acc[2], acc[3]);
    if (lane == 0) *reinterpret_cast<float2*>(&shares[share - 1][wg][128]) = make_float2(M, l);
  }
  __syncthreads();
  if (share == 0 && gg < a.group) {
    float Mt = M;
    if (kShares > 1)
      for (int p = 0; p < kShares - 1; ++p) Mt = fmaxf(Mt, shares[p][wg][128]);
    for (int w = 0; w < n_wsw; ++w) Mt = fmaxf(Mt, ws.m[w][wg]);
    const float sc = l == 0.f ? 0.f : exp2f(M - Mt);
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[k] *= sc;
    l *= sc;
    if (kShares > 1)
      for (int p = 0; p < kShares - 1; ++p) {
        if (shares[p][wg][129] == 0.f) continue;
        const float f = exp2f(shares[p][wg][128] - Mt);
        const float4 v = *reinterpret_cast<const float4*>(&shares[p][wg][4 * lane]);
        acc[0] = fmaf(v.x, f, acc[0]);
        acc[1] = fmaf(v.y, f, acc[1]);
        acc[2] = fmaf(v.z, f, acc[2]);
        acc[3] = fmaf(v.w, f, acc[3]);
        l = fmaf(shares[p][wg][129], f, l);
      }
    // un-rotate: H over the 128 channels
    const float a0 = acc[0] + acc[1], a1 = acc[0] - acc[1], a2 = acc[2] + acc[3], a3 = acc[2] - acc[3];
    acc[0] = a0 + a2;
    acc[1] = a1 + a3;
    acc[2] = a0 - a2;
    acc[3] = a1 - a3;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const bool upper = (lane & o) != 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float other = __shfl_xor_sync(0xffffffffu, acc[k], o);
        acc[k] = upper ? other - acc[k] : acc[k] + other;
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[k] *= kInvSqrt128;
    float tail = 0.f;
    for (int w = 0; w < n_wsw; ++w) {
      const float f = exp2f(ws.m[w][wg] - Mt);
      const float4 v = *reinterpret_cast<const float4*>(&ws.o[w][wg][4 * lane]);
      acc[0] = fmaf(v.x, f, acc[0]);
      acc[1] = fmaf(v.y, f, acc[1]);
      acc[2] = fmaf(v.z, f, acc[2]);
      acc[3] = fmaf(v.w, f, acc[3]);
      tail = fmaf(ws.l[w][wg], f, tail);
    }
    l += tail;
    const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;       // (a sum that is not a number stays one)
    uint16_t r[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) r[k] = f2h_bits(acc[k] * inv);
    *reinterpret_cast<uint2*>(out + (u * a.group + gg) * kD + 4 * lane) =
        make_uint2(r[0] | static_cast<uint32_t>(r[1]) << 16, r[2] | static_cast<uint32_t>(r[3]) << 16);
    if (lane == 0) {
      const HeadEnd e{Mt, inv, tail == 0.f ? 0.f : tail * inv, 0.f};   // (as a tile's: a sum of 0 is none)
      if (kHeads == 8) heads[gg] = e;
      else reinterpret_cast<HeadEnd*>(a.ends)[u * 8 + gg] = e;
      if (a.lse != nullptr) a.lse[u * a.group + gg] = (Mt + log2f(l)) * 0.693147180559945309f;
    }
  }
  if (kHeads == 8) {
    // (the length is read again, not held: that spills, and 256 x 1000 tokens take 105 us instead of 103.3)
    const int again = seq_len(a, s);
    __syncthreads();
    weigh_unit(a, u, again, heads, threadIdx.x, blockDim.x);
  }
}

// The weights of few units, gridDim.z blocks each.
__global__ void __launch_bounds__(256) weigh_tiles_kernel(const __grid_constant__ WeighArgs a) {
  __shared__ HeadEnd heads[8];
  const int s = blockIdx.y, len = seq_len(a, s);
  const int64_t u = static_cast<int64_t>(s) * a.hkv + blockIdx.x;
  griddep_wait();
  if (threadIdx.x < a.group) heads[threadIdx.x] = reinterpret_cast<const HeadEnd*>(a.ends)[u * 8 + threadIdx.x];
  __syncthreads();
  weigh_unit(a, u, len, heads, blockIdx.z * 256 + threadIdx.x, gridDim.z * 256);
}

template <int KB, int VB, bool kLean, bool kNarrow>
cudaError_t launch_split(const WeighArgs& a, cudaStream_t stream) {
  using C = WeighCfg<KB, VB, kLean>;
  static std::atomic<unsigned long long> smem_set{0};
  const cudaError_t err = set_smem_once(weigh_split_kernel<KB, VB, kLean, kNarrow>, C::kSmem, smem_set);
  if (err != cudaSuccess) return err;
  weigh_split_kernel<KB, VB, kLean, kNarrow><<<a.n_ctas, C::kWarps * 32, C::kSmem, stream>>>(a);
  return cudaGetLastError();
}

template <int KB, int VB, bool kLean>
cudaError_t launch_weigh(WeighArgs& a, cudaStream_t stream) {
  a.warps = WeighCfg<KB, VB, kLean>::kWarps;
  return a.group <= 4 ? launch_split<KB, VB, kLean, true>(a, stream) : launch_split<KB, VB, kLean, false>(a, stream);
}

// Scratch: the partial records and marks (within the decode's), HeadEnds, (m, l) of the tiles.
size_t ends_offset(int n_seqs, int hkv, int max_blocks) {
  return (decode_part_bytes(n_seqs, hkv, max_blocks) + 255) & ~size_t(255);
}

}  // namespace

size_t decode_weights_scratch_bytes(int n_seqs, int hkv, int max_blocks) {
  return ends_offset(n_seqs, hkv, max_blocks) +
         static_cast<size_t>(n_seqs) * hkv * (sizeof(HeadEnd) + static_cast<size_t>(max_blocks) * sizeof(float2)) * 8;
}

cudaError_t launch_decode_weights(const uint16_t* q, const uint8_t* cache, const uint16_t* ws, const int32_t* block_tables,
                                  const int32_t* seq_lens, int n_seqs, int hkv, int group, int max_blocks,
                                  int64_t num_blocks, int k_bits, int v_bits, bool lean, float decay, float* weights,
                                  uint16_t* out, float* lse, void* scratch, unsigned* flags, cudaStream_t stream) {
  uint8_t* at = static_cast<uint8_t*>(scratch);
  WeighArgs a{};
  a.q = q;
  a.cache = cache;
  a.block_tables = block_tables;
  a.seq_lens = seq_lens;
  a.flags = flags;
  a.num_blocks = num_blocks;
  a.n_seqs = n_seqs;
  a.hkv = hkv;
  a.group = group;
  a.max_blocks = max_blocks;
  a.n_ctas = decode_num_ctas();
  a.part = reinterpret_cast<float*>(at);
  a.cover = cover_ptr(a.part, n_seqs, hkv, a.n_ctas);
  a.ws = ws;
  a.ends = reinterpret_cast<float4*>(at + ends_offset(n_seqs, hkv, max_blocks));
  a.stats = reinterpret_cast<float2*>(a.ends + static_cast<size_t>(n_seqs) * hkv * 8);
  a.weights = weights;
  a.lse = lse;
  a.decay = decay;
  cudaError_t err = k_bits == 2   ? launch_weigh<2, 2, false>(a, stream)
                    : v_bits == 4 ? launch_weigh<4, 4, false>(a, stream)
                    : lean        ? launch_weigh<4, 2, true>(a, stream)
                                  : launch_weigh<4, 2, false>(a, stream);
  if (err != cudaSuccess) return err;
  // By the partial records of a unit, on average (as many as parts, or tiles). 64 heads over 8, k4v2:
  // from 8 records on 4 warps a q-head (16 x 1000 tokens: 15.6 us, 20.1 with one), from 96 on a block a q-head
  // (1 x 131072: 46 us against 64; 3 x 16389, 76 records: 30 against 28).
  const int64_t units = static_cast<int64_t>(n_seqs) * hkv, parts = static_cast<int64_t>(a.n_ctas) * a.warps;
  const int64_t records = parts / units < max_blocks ? parts / units : max_blocks;
  if (records < 8) return launch_after(weigh_merge_kernel<8, 1>, dim3(hkv, n_seqs), dim3(256), 0, stream, a, out);
  if (records < 96) return launch_after(weigh_merge_kernel<8, 4>, dim3(hkv, n_seqs), dim3(1024), 0, stream, a, out);
  err = launch_after(weigh_merge_kernel<1, 32>, dim3(hkv * group, n_seqs), dim3(1024), 0, stream, a, out);
  if (err != cudaSuccess) return err;
  int64_t z = (max_blocks + 255) / 256;
  if (z > 64) z = 64;
  return launch_after(weigh_tiles_kernel, dim3(hkv, n_seqs, static_cast<unsigned>(z)), dim3(256), 0, stream, a);
}

}  // namespace kvarn

// Attention of drafted tokens over the packed cache, the workspace and the drafted
// tokens themselves (KVarN README, "How KVarN works": the scales are re-applied on read,
// the orthonormal rotation keeps attention scores, the output is un-rotated).
//
// The rows of a (sequence, kv-head) are its drafted tokens times the group's q-heads
// (row = token * group + head), cut into units of up to R = 32 or 64 rows. A unit's items are
// its packed tiles and then its fresh tiles (up to 128 tokens each: the workspace tokens
// followed by the drafted ones). The flattened items are cut into one contiguous range
// per team (stream-K), so a few long sequences fill the GPU and ragged batches balance.
//   tree_scan_kernel   prefix of items per sequence, first tile inside the window
//   tree_split_kernel  one persistent CTA per SM with two or three teams of 8 warps; a team
//                      leaving a unit writes a partial record
//   tree_merge_kernel  a warp per output row joins the records
//
// Per item and team, all products with M = 128 on the 5th-generation tensor core, tokens
// (then channels) as TMEM lanes and rows as columns, A in TMEM, B in shared memory:
//   keys    thread (lane = token, half = channels 64 half ..) turns codes into fp16 in TMEM
//   fold    q' = q_r r^K s^K 2^e as fp16 hi + lo rows, beta = sum_i q_r,i r_i z_i
//   QK^T    S[token][row] = codes . q' + 1 beta  (8 K steps, hi and lo, and one of beta)
//           x = c^K_t S in the log2 domain, cap, bias, masks
//   values  thread (lane = channel) turns codes into fp16 in TMEM (under QK^T)
//   PV      O[channel][row] = (codes + u^) . p' + 1 (u - u^) . p',
//           p' = p c^V s^V 2^e as fp16 hi + lo, u = z^V / s^V of the token
//           acc += r^V_channel O
// The hi + lo pairs carry q' and p' to ~22 bits: rounded once to fp16, scores of keys with
// outlier channels are off by some 1e-3 and so are the outputs. The powers of two leave the pairs fp16's range, down to its
// subnormal steps (the products keep them): q' to 2^-37 of the unit's largest, so that a row of q loses bits only
// beside one whose scores are above some 10^7; p' to 2^-30 of the running max's, of which 131072 tokens together are 1e-4.
// Sums are fp32, in the tensor core's accumulators within a tile; exponentials, the cap's and the rows' divisions are
// the approximate instructions (about 2^-22).
// The running max is lazy: a tile rescales only when a score exceeds it by more than
// kTau, so that most tiles need no reduction over tokens (lanes); p stays <= 2^kTau.
// Before fresh tiles, or before a record is written, the accumulator of the packed part is
// rotated back by one more product, with the +-1 Hadamard matrix as A.
//
// Measured (fp16 out, k4v2, 64 q-heads over 8 kv-heads): 64 sequences of 16384 tokens with 8
// drafted 873 us, 1.1 TB/s of records and 315 TFLOP/s of 275 GFLOP (the pairs double what the
// tensor core does). No unit is at its limit: 8.4 K warp instructions a tile of 64 rows at 2.0 a
// cycle and SM of 4, shared memory 47 % and the tensor pipe 32 % busy, DRAM 14 %; 16 warps an SM, whose phases wait
// for one another. Left out in turn, the fold is worth 22 % of the time, p's writing 5 %, the softmax 8 %, the
// conversions of codes 3 and 2 %, the accumulation 3 %. Spilled registers (128 / 192 bytes of stores / loads for 64
// rows, 264 to 344 / 364 to 480 for 32 rows) are 1 % of the instructions. Slower were one warp of 17
// that issues all products (registers capped at 96: 1603 us), the fold one tile ahead
// (982), and the next keys' conversion under PV (922).
#include <cuda_runtime.h>

#include <algorithm>

#include "decode_tc.cuh"
#include "kvarn_codes.cuh"
#include "kvarn_launch.h"
#include "tree_unit.cuh"

namespace kvarn {
namespace {

constexpr int kTreeTeamThreads = 256;
constexpr int kTreeIssuer = 7;         // the warp of a team that issues its UMMAs
constexpr int kTreeStages = 2;
constexpr int kTreeMaxCtas = 160;      // sizes the scratch
constexpr int kTreeMaxTeams = 3;
// Units of 32 rows: three teams, 80 registers a thread, accumulators in registers (4 sequences of
// 131072 tokens, 4 drafted: 316 us; two teams of 128 registers 321). Units of 64 rows: two teams,
// 128 registers, accumulators in TMEM (32 more of them a thread would not fit).
__host__ __device__ constexpr int tree_teams(int r) { return r == 32 ? 3 : 2; }
// TMEM columns of a team: the key and value operands, S and O (O is written once S has been
// read), and for 64 rows the accumulator.
constexpr uint32_t kTrAK = 0, kTrAV = 64, kTrS = 128, kTrAcc = 192;
__host__ __device__ constexpr uint32_t tree_cols(int r) { return r == 32 ? 160 : 256; }
constexpr float kTau = 8.0f;
constexpr float kFloatMax = 3.402823466e+38f;
constexpr float kNoMax = -1.0e30f;     // running max of a record whose row saw no key

struct TreeArgs {
  const uint16_t *q, *k_new, *v_new;
  const uint64_t* mask;
  const int32_t *positions, *cu, *seq_lens, *block_tables;
  const uint8_t* cache;
  const uint16_t* ws;
  const float* slopes;
  uint16_t* out;
  unsigned* flags;
  int64_t* prefix;       // [n_seqs + 1] items of the sequences before
  int32_t* first;        // [n_seqs] first packed tile that a window leaves
  float* part;           // partial records
  int64_t num_blocks, n_tokens;
  int n_seqs, max_tree, hkv, group, max_blocks, window;
  int n_teams, max_units;   // teams; units of a (sequence, kv-head) at most
  int group_inv;            // ceil(2^16 / group)
  float scale;              // of q.k, times log2(e)
  float none;               // -0: a product that a sum follows is fma(x, y, -0), which the compiler cannot contract with it
  float cap, cap_two;       // cap times log2(e) (0: none), and 2 log2(e) over that
};

// Row count and layout of a record: acc [R][128], then (max, sum) [R].
__host__ __device__ constexpr int tree_rec_floats(int r) { return r * 130; }

__device__ __forceinline__ void tree_dep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void tree_dep_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Sizes of sequence s.
struct TreeSeq {
  int nt;       // drafted tokens that are computed (0: none, nothing to do)
  int full;     // packed tiles [first, full)
  int ws;       // workspace tokens
  int units;    // of a kv-head
  int fresh;    // fresh tiles
};
template <int R>
__device__ __forceinline__ TreeSeq tree_seq(const TreeArgs& a, int s, bool report) {
  TreeSeq q{};
  const int64_t c0 = a.cu[s];
  const int64_t n = a.cu[s + 1] - c0;
  const int len = max(a.seq_lens[s], 0);
  unsigned bad = 0;
  q.nt = static_cast<int>(max(min(n, static_cast<int64_t>(a.max_tree)), static_cast<int64_t>(0)));
  if (n > a.max_tree) bad = KVARN_FLAG_BAD_LENGTH;
  if (q.nt > 0 && (c0 < 0 || c0 + q.nt > a.n_tokens)) {
    q.nt = 0;
    bad = KVARN_FLAG_BAD_LENGTH;
  }
  q.full = min(len / kB, a.max_blocks);
  q.ws = len % kB;
  if (q.nt > 0 && (len / kB > a.max_blocks || (q.ws > 0 && a.ws == nullptr))) bad = KVARN_FLAG_BAD_LENGTH;
  if (a.ws == nullptr) q.ws = 0;
  q.units = (q.nt * a.group + R - 1) / R;
  q.fresh = (q.ws + q.nt + kB - 1) / kB;
  if (report && bad) raise_flag(a.flags, bad);
  return q;
}

// ------------------------------------------------------------------ scan
template <int R>
__global__ void __launch_bounds__(1024) tree_scan_kernel(const TreeArgs a) {
  tree_dep_launch();
  __shared__ int64_t warp_sums[32];
  const int t = threadIdx.x, lane = t & 31, w = t >> 5;
  const int per = (a.n_seqs + 1023) / 1024;
  const int s0 = min(t * per, a.n_seqs), s1 = min(s0 + per, a.n_seqs);
  int64_t sum = 0;
  for (int s = s0; s < s1; ++s) {
    const TreeSeq q = tree_seq<R>(a, s, true);
    int first = 0;
    if (a.window > 0 && q.nt > 0) {   // tiles that no drafted token's window reaches are left out
      int64_t pmin = INT32_MAX;
      for (int i = 0; i < q.nt; ++i) pmin = min(pmin, static_cast<int64_t>(a.positions[a.cu[s] + i]));
      const int64_t lo = max(pmin - a.window + 1, static_cast<int64_t>(0)) / kB;
      first = static_cast<int>(min(lo, static_cast<int64_t>(q.full)));
    }
    a.first[s] = first;
    const int64_t items = static_cast<int64_t>(a.hkv) * q.units * (q.full - first + q.fresh);
    a.prefix[s] = items;              // turned into the prefix below
    sum += items;
  }
  int64_t incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) warp_sums[w] = incl;
  __syncthreads();
  if (w == 0) {
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
    const int64_t n = a.prefix[s];
    a.prefix[s] = run;
    run += n;
  }
  if (t == 1023) a.prefix[a.n_seqs] = warp_sums[31];
}

// ------------------------------------------------------------------ cursor over items
// Kept in shared memory: thread 0 of the team moves it, everyone reads what it needs.
struct TreeCursor {
  int s, h, u;           // sequence, kv-head, unit of it
  int ti;                // item of the unit
  int packed, items;     // packed tiles, all items of the unit
  int units, nt, ws;     // units of a kv-head, drafted and workspace tokens
  int first;             // first packed tile
  int64_t c0;            // first drafted token's row of q
};
template <int R>
__device__ __forceinline__ void tree_enter(const TreeArgs& a, TreeCursor& c) {
  const TreeSeq q = tree_seq<R>(a, c.s, false);
  c.first = a.first[c.s];
  c.c0 = a.cu[c.s];
  c.packed = q.full - c.first;
  c.items = c.packed + q.fresh;
  c.units = q.units;
  c.nt = q.nt;
  c.ws = q.ws;
}
template <int R>
__device__ __forceinline__ void tree_locate(const TreeArgs& a, int64_t g, TreeCursor& c) {
  int lo = 0, hi = a.n_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.prefix[mid] <= g) lo = mid; else hi = mid - 1;
  }
  c.s = lo;
  tree_enter<R>(a, c);
  const int64_t off = g - a.prefix[lo];
  const int64_t un = off / c.items;
  c.ti = static_cast<int>(off - un * c.items);
  c.h = static_cast<int>(un / c.units);
  c.u = static_cast<int>(un - static_cast<int64_t>(c.h) * c.units);
}
// To the next unit's first item.
template <int R>
__device__ __forceinline__ void tree_next_unit(const TreeArgs& a, TreeCursor& c) {
  c.ti = 0;
  if (++c.u < c.units) return;
  c.u = 0;
  if (++c.h < a.hkv) return;
  c.h = 0;
  do {
    ++c.s;
    if (c.s >= a.n_seqs) return;
  } while (a.prefix[c.s + 1] == a.prefix[c.s]);
  tree_enter<R>(a, c);
}

// ------------------------------------------------------------------ shared memory of a team
template <int KB, int VB, bool kLean, int R>
struct TreeSm {
  using L = RecordLayout<KB, VB, kLean>;
  static constexpr int kTeams = tree_teams(R);
  static constexpr int kB0 = 0;                                  // B operand, hi rows (R = 32: and lo rows)
  static constexpr int kExt = R == 64 ? 32768 : 16384;           // B of beta: [16][64 rows]
  static constexpr int kQ = kExt + 2048;                         // q_r scaled, [R][128] f32
  static constexpr int kRec = kQ + R * 512;
  static constexpr int kRecPitch = (L::kBytes + 15) / 16 * 16;
  static constexpr int kU = kRec + kTreeStages * kRecPitch;      // A of gamma: [128 tokens][8 x u]
  static constexpr int kOne = kU + 2048;                         // A of beta: [16][8]
  static constexpr int kAdd = kOne + 256;                        // [128] fp16: what the values' operand adds
  static constexpr int kX = kAdd + 256;
  // small arrays at kX, [R] each: negated maxima, sums, positions, slopes; mask words
  static constexpr int kMax = 0, kGam = 4 * R, kPos = 8 * R, kSlope = 12 * R, kMask = 16 * R;
  static constexpr int kPart = 24 * R;                           // [8 warps][R / 2] f32
  static constexpr int kSmall = kPart + 16 * R;                  // 16 floats
  static constexpr int kBars = kSmall + 64;
  static constexpr int kCur = kBars + 48, kAhead = kCur + 48;    // cursors: the team's, the copies'
  static constexpr int kAheadN = kAhead + 48, kValid = kAheadN + 8;   // items left to the copies; valid tiles in the stages
  static constexpr int kXBytes = kValid + 8;
  static constexpr int kTeam = (kX + kXBytes + 1023) / 1024 * 1024;
  static constexpr int kSlot = kTeams * kTeam;
  static constexpr int kBytes = kSlot + 16;
  static_assert(kBytes <= 232448, "tree shared memory");
  static_assert(sizeof(TreeCursor) <= 48, "cursor");
};
constexpr int kTbRec = 0, kTbQkDone = 2, kTbPvDone = 3, kTbFin = 4;

// Sum (or maximum) over the warp's 32 lanes of 16 values: lane l returns that of value l % 16.
template <bool kMaxOp>
__device__ __forceinline__ float tree_reduce(float (&g)[16], int lane) {
#pragma unroll
  for (int o = 8; o >= 1; o >>= 1) {
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float send = up ? g[i] : g[i + o], keep = up ? g[i + o] : g[i];
      const float got = __shfl_xor_sync(0xffffffffu, send, o);
      g[i] = kMaxOp ? fmaxf(keep, got) : keep + got;
    }
  }
  const float got = __shfl_xor_sync(0xffffffffu, g[0], 16);
  return kMaxOp ? fmaxf(g[0], got) : g[0] + got;
}

// x to cap tanh(f x / cap) (f x and cap times log2(e); two_inv = 2 log2(e) / cap): cap (1 - 2 / (1 + e^(2 z))), off by
// some 2^-22 cap. Caps above kCapNear, where that is more than 2e-5 of a score, have tanh to a few 2^-22 of its own size, so that
// a cap far above the scores leaves them as they are: below |z| = 0.55 by z's continued fraction (Lambert)
// z / (1 + z^2 / (3 + z^2 / (5 + z^2 / (7 + z^2 / 9)))), whose error there is below 2^-32. With that for every cap, 37 ragged sequences
// in a window of 4096 took 579 us, against 505.
constexpr float kCapNear = 64.f;
__device__ __forceinline__ void tree_cap(float (&x)[16], float f, float cap, float two_inv) {
  const float fe = fminf(f * two_inv, kFloatMax);  // (a cap near 0: not an infinity, which a score of 0 would turn into NaN)
  if (cap <= kCapNear * kLog2e) {
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = fmaf(-2.f * cap, __fdividef(1.f, 1.f + ex2(x[i] * fe)), cap);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float z = x[i] * f * (two_inv * (0.5f / kLog2e)), z2 = z * z, e = 1.f + ex2(z * (2.f * kLog2e));
      const bool small = z2 < 0.3025f;
      const float r = __fdividef(1.f, small ? fmaf(fmaf(z2, 15.f, 420.f), z2, 945.f) : e);
      x[i] = cap * (small ? z * fmaf(z2 + 105.f, z2, 945.f) * r : fmaf(-2.f, r, 1.f));
    }
  }
}

// Byte offset of (row, K index) in a 64-row fp16 B operand, K = channels: 128-byte
// swizzled K-major, halves of 64 channels 8192 bytes apart.
__device__ __forceinline__ uint32_t tree_qo(int r, int ch) {
  return static_cast<uint32_t>((ch >> 6) * 8192 + (r >> 3) * 1024 + (r & 7) * 128 +
                               ((((ch & 63) >> 3) ^ (r & 7)) << 4));
}
// Byte offset of (8 rows from 8 c, token) in a 64-row fp16 B operand, K = tokens: 128-byte
// swizzled with the rows contiguous (N-major), a token's 64 rows in 128 bytes.
__device__ __forceinline__ uint32_t tree_po(int c, int tok) {
  return static_cast<uint32_t>(tok * 128 + ((c ^ (tok & 7)) << 4));
}

// ------------------------------------------------------------------ operands
// Thread t of the warp: 16 consecutive columns of TMEM lane (base lane + t) from r.
__device__ __forceinline__ void tree_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tree_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tree_add16(uint32_t (&r)[16], const uint16_t* add) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4 v = reinterpret_cast<const uint4*>(add)[i];
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __half2 x = __hadd2(*reinterpret_cast<const __half2*>(&r[4 * i + e]), *reinterpret_cast<const __half2*>(&w[e]));
      r[4 * i + e] = *reinterpret_cast<const uint32_t*>(&x);
    }
  }
}
// Keys of token `tok`, and values of channel t plus their token's `add` (by K element; sums
// exact in fp16), to 32 TMEM columns.
template <int KB>
__device__ __forceinline__ void tree_keys(const uint8_t* codes, int tok, int half, uint32_t taddr) {
  key_codes<KB>(codes, tok, half, [&](int i, uint32_t (&r)[16]) { tree_st16(taddr + 16 * i, r); });
}
template <int VB>
__device__ __forceinline__ void tree_values(const uint8_t* codes, int t, int half, const uint16_t* add, uint32_t taddr) {
  value_codes<VB>(codes, t, half, [&](int i, uint32_t (&r)[16]) {
    tree_add16(r, add + 64 * half + 32 * i);
    tree_st16(taddr + 16 * i, r);
  });
}

// An operand with its M (or N) elements contiguous, not swizzled, whose groups of 8 are all the
// same 16 bytes a K element (stride 0): the operand's 128 rows are 8 that repeat.
__device__ __forceinline__ uint64_t tree_desc_same(uint32_t saddr) {
  uint64_t d = static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>(128u >> 4) << 16;    // leading byte offset: the next 8 K elements
  d |= static_cast<uint64_t>(1) << 46;            // (stride byte offset 0; no swizzle)
  return d;
}

// A team's work. Thread tt of 256: lane t = tt & 127 (token or channel), half = tt >> 7.
template <int KB, int VB, bool kLean, int R, bool kMod>
struct TreeTeam {
  using L = RecordLayout<KB, VB, kLean>;
  using S = TreeSm<KB, VB, kLean, R>;
  static constexpr int CT = R / 2;               // rows (columns of the products) of a thread
  static constexpr float kKF = KB == 4 ? 8.f : 2.f, kVF = VB == 4 ? 8.f : 2.f;   // codes were converted to code / kKF
  // beta is carried over this constant of its other operand. In units of S it is sum q_r r z / kKF over 128
  // channels with |q_r| < 2^13 and |r z| < 2^7 (fold's scaling), so the operand stays below 128 2^13 2^7 / (kKF kBetaOne) =
  // 2^15 for either width (fp16 ends at 65504); keys that are flat after the rotation, and a query along them, come near.
  static constexpr float kBetaOne = 4096.f / kKF;
  // What fp16 leaves of it goes in 2^11 larger (below 2^14), over a constant as much smaller: a row of q far below the
  // unit's largest, whose power of two it shares, keeps its bits (10^7 below: scores off by 1e-2 of themselves otherwise).
  static constexpr float kBetaLo = 2048.f;
  // A token's value is s (code + u), u = z / s. Most of u goes into the operand: code + u^, u^ the
  // multiple of a power of two nearest to u that fp16 holds exactly with every code (2^-6 below
  // |u| = 16, twice that below 48, ..). The rest u - u^ goes in as one more product, whose A has the same value in every
  // channel's row. A token whose zero is more than kWide steps from 0 (a constant group, whose
  // step has its least value) has neither; its part p c z is summed over the lanes.
  static constexpr float kWide = 1000.f;
  const TreeArgs& a;
  uint8_t* sm;
  uint32_t tm, trow;                             // TMEM address of the team, of the thread's warp
  int tt, t, half, lane, warp, bar_id;
  float acc[R == 32 ? CT : 1], lsum[CT];
  float qinv;                                    // 2^-e of the stored q_r
  uint32_t qph, pph;
  uint32_t issued, used;                         // packed tiles: copies started (thread 0), taken
  bool ok;                                       // no wait of the thread has run out; the team's only where a barrier agreed on it
  bool row_set;                                  // thread tt < R: row tt has seen a key
  bool pending;                                  // some row of the unit has not (the team agrees)

  __device__ TreeTeam(const TreeArgs& a_, uint8_t* sm_, uint32_t tm_, int team)
      : a(a_), sm(sm_), tm(tm_), bar_id(1 + 2 * team), qinv(1.f), qph(0), pph(0), issued(0), used(0), ok(true), row_set(false), pending(true) {
    tt = static_cast<int>(threadIdx.x) - team * kTreeTeamThreads;
    t = tt & 127;
    half = tt >> 7;
    lane = tt & 31;
    warp = __shfl_sync(0xffffffffu, tt >> 5, 0);   // known to be the same for the warp
    trow = tm + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
  }
  __device__ float* mrow() const { return reinterpret_cast<float*>(sm + S::kX + S::kMax); }
  __device__ float* gam() const { return reinterpret_cast<float*>(sm + S::kX + S::kGam); }
  __device__ float* part() const { return reinterpret_cast<float*>(sm + S::kX + S::kPart); }
  __device__ float* small() const { return reinterpret_cast<float*>(sm + S::kX + S::kSmall); }
  __device__ float* slope() const { return reinterpret_cast<float*>(sm + S::kX + S::kSlope); }
  __device__ int32_t* pos() const { return reinterpret_cast<int32_t*>(sm + S::kX + S::kPos); }
  __device__ uint64_t* mask() const { return reinterpret_cast<uint64_t*>(sm + S::kX + S::kMask); }
  __device__ uint64_t* bars() const { return reinterpret_cast<uint64_t*>(sm + S::kX + S::kBars); }
  __device__ TreeCursor& cur() const { return *reinterpret_cast<TreeCursor*>(sm + S::kX + S::kCur); }
  __device__ TreeCursor& ahead() const { return *reinterpret_cast<TreeCursor*>(sm + S::kX + S::kAhead); }
  __device__ int64_t& ahead_n() const { return *reinterpret_cast<int64_t*>(sm + S::kX + S::kAheadN); }
  __device__ volatile uint32_t* valid_of() const { return reinterpret_cast<volatile uint32_t*>(sm + S::kX + S::kValid); }
  __device__ void bar() { named_bar(bar_id, kTreeTeamThreads); }
  // Drafted token of a row (row / group, exact for the 512 rows there can be) and the row of q.
  __device__ int token_of(int row) const { return (row * a.group_inv) >> 16; }
  __device__ const uint16_t* q_row(int64_t c0, int h, int row, int p) const {
    return a.q + ((c0 + p) * a.hkv * a.group + h * a.group + (row - p * a.group)) * kD;
  }
  static __device__ uint32_t tree_qo_lo(int r, int k) { return R == 64 ? 16384 + tree_qo(r, k) : tree_qo(r + 32, k); }

  // The thread's operand writes are done; once everyone's are, the issuer starts the product.
  // QK^T: the whole team meets (what it wrote for the values is visible then).
  __device__ void product_qk(bool fresh) {
    tc_operands_written();
    bar();
    if (warp != kTreeIssuer) return;
    if (elect_one()) {
      tc_fence_after();
      // bit 15: A, bit 16: B with M or N contiguous
      constexpr uint32_t kId = idesc_f16_f32(128, R), kIdSame = kId | (1u << 15) | (1u << 16);
      const uint64_t d = smem_desc_sw128(smem_u32(sm + S::kB0));
#pragma unroll
      for (int s = 0; s < 8; ++s)
        tc_umma_ts(tm + kTrS, tm + kTrAK + 8 * s, d + (((s >> 2) * 8192 + (s & 3) * 32) >> 4), kId, s > 0);
      if (!fresh) {                              // (fresh: q is exact in fp16)
#pragma unroll
        for (int s = 0; s < 8; ++s)
          tc_umma_ts(tm + kTrS, tm + kTrAK + 8 * s,
                     d + (((R == 64 ? 16384 : 4096) + (s >> 2) * 8192 + (s & 3) * 32) >> 4), kId, 1);
        umma_f16(tm + kTrS, tree_desc_same(smem_u32(sm + S::kOne)), smem_desc_sw128(smem_u32(sm + S::kExt)), kIdSame, 1);
      }
      umma_commit(&bars()[kTbQkDone]);
    }
    __syncwarp();
  }
  // PV: only the issuer waits.
  __device__ void product_pv(bool gamma) {
    tc_operands_written();
    if (warp != kTreeIssuer) {
      asm volatile("bar.arrive %0, %1;" ::"r"(bar_id + 1), "r"(kTreeTeamThreads) : "memory");
      return;
    }
    named_bar(bar_id + 1, kTreeTeamThreads);
    if (elect_one()) {
      tc_fence_after();
      constexpr uint32_t kId = idesc_f16_f32(128, R) | (1u << 16), kIdSame = kId | (1u << 15);
      const uint64_t d = smem_desc_sw128(smem_u32(sm + S::kB0));
#pragma unroll
      for (int p = 0; p < 2; ++p)                // lo rows: the next operand, or 64 bytes along a token's rows
#pragma unroll
        for (int s = 0; s < 8; ++s)
          tc_umma_ts(tm + kTrS, tm + kTrAV + 8 * s, d + ((p * (R == 64 ? 16384 : 64) + s * 2048) >> 4), kId, p + s > 0);
      if (gamma) {
        const uint64_t u = tree_desc_same(smem_u32(sm + S::kU));
#pragma unroll
        for (int s = 0; s < 8; ++s) umma_f16(tm + kTrS, u + ((s * 256) >> 4), d + ((s * 2048) >> 4), kIdSame, 1);
      }
      umma_commit(&bars()[kTbPvDone]);
    }
    __syncwarp();
  }
  // 16 of the thread's rows of S or O, and of the accumulator.
  __device__ void read16(int ch, float (&v)[16]) { tc_ld16(trow + kTrS + CT * half + 16 * ch, v); }
  __device__ void get_acc(int ch, float (&v)[16]) {
    if constexpr (R == 32) {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = acc[i];
    } else {
      tc_ld16(trow + kTrAcc + CT * half + 16 * ch, v);
    }
  }
  __device__ void put_acc(int ch, const float (&v)[16]) {
    if constexpr (R == 32) {
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[i] = v[i];
    } else {
      tree_st16(trow + kTrAcc + CT * half + 16 * ch, reinterpret_cast<const uint32_t(&)[16]>(v));
      asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
    }
  }

  // The constant operand of beta (kBetaOne for the high part, kBetaOne / kBetaLo for the low one, at K elements 0
  // and 1) and the zeros of its other one.
  __device__ void init() {
    constexpr uint32_t kHi2 = KB == 4 ? 0x60006000u : 0x68006800u, kLo2 = KB == 4 ? 0x34003400u : 0x3C003C00u;   // fp16 pairs
    static_assert(kBetaOne == (KB == 4 ? 512.f : 2048.f) && kBetaLo == 2048.f, "the constants as fp16");
    for (int i = tt; i < 16; i += kTreeTeamThreads)
      reinterpret_cast<uint4*>(sm + S::kOne)[i] =
          i == 0 ? make_uint4(kHi2, kHi2, kHi2, kHi2) : i == 1 ? make_uint4(kLo2, kLo2, kLo2, kLo2) : make_uint4(0, 0, 0, 0);
    for (int i = tt; i < 128; i += kTreeTeamThreads) reinterpret_cast<uint4*>(sm + S::kExt)[i] = make_uint4(0, 0, 0, 0);
  }

  static __device__ int q_slot(int g) { return 16 * ((g >> 1) & 1) + (g >> 2) + 8 * (g & 1); }

  // Rows of the unit at the cursor: row tables, q_r scaled by a power of two in shared memory.
  __device__ void enter() {
    const TreeCursor& c = cur();
    const int64_t c0 = c.c0;
    const int row0 = c.u * R, nt = c.nt, h = c.h;
    if (tt < R) {
      const int row = row0 + tt, p = token_of(row);
      const bool live = p < nt;
      mrow()[tt] = 0.f;
      uint64_t w = 0;
      if (live) w = a.mask != nullptr ? a.mask[c0 + p] : ~0ull >> (63 - p);
      mask()[tt] = w;
      if (kMod) {
        pos()[tt] = live && a.positions != nullptr ? a.positions[c0 + p] : 0;
        slope()[tt] = live && a.slopes != nullptr ? a.slopes[h * a.group + (row - p * a.group)] * kLog2e : 0.f;
      }
    }
    const int jj = tt & 15, r0 = tt >> 4;
    float m = 0.f;
    float* qs = reinterpret_cast<float*>(sm + S::kQ);
    auto load = [&](int k) {
      const int row = row0 + r0 + 16 * k, p = token_of(row);
      return p < nt ? *reinterpret_cast<const uint4*>(q_row(c0, h, row, p) + 8 * jj) : make_uint4(0, 0, 0, 0);
    };
    uint4 next = load(0);
#pragma unroll 1
    for (int k = 0; k < R / 16; ++k) {             // (not unrolled: run once, its time is that of fetching the code)
      float x[8];
      const uint32_t ws[4] = {next.x, next.y, next.z, next.w};
      if (k + 1 < R / 16) next = load(k + 1);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = h2pair(reinterpret_cast<const uint16_t*>(&ws[e]));
        x[2 * e] = f.x;
        x[2 * e + 1] = f.y;
      }
#pragma unroll
      for (int bit = 1; bit < 8; bit <<= 1)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if ((i & bit) == 0) {
            const float u = x[i], v = x[i | bit];
            x[i] = u + v;
            x[i | bit] = u - v;
          }
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) {
        const float sg = (jj & o) != 0 ? -1.f : 1.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = fmaf(x[i], sg, __shfl_xor_sync(0xffffffffu, x[i], o));
      }
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[i]));
      m = fmaxf(m, top <= kFloatMax ? top : 0.f);   // (a row with an infinity spoils itself only)
      // channels 4 G .. at 16-byte slot 16 e + j of the row (fold's thread j reads slots j, 16 + j)
      float4* dst = reinterpret_cast<float4*>(qs + (r0 + 16 * k) * kD);
      dst[q_slot(2 * jj)] = make_float4(x[0], x[1], x[2], x[3]);
      dst[q_slot(2 * jj + 1)] = make_float4(x[4], x[5], x[6], x[7]);
    }
    m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
    if (lane == 0) part()[warp] = m;
    bar();
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, part()[i]);
    const float2 sc = tc_pow2_scale(m, 12);        // the largest |q_r| into [2^12, 2^13)
    qinv = sc.y;
#pragma unroll
    for (int k = 0; k < R / 16; ++k) {             // the thread's own elements
      float4* p = reinterpret_cast<float4*>(qs + (r0 + 16 * k) * kD);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int i = q_slot(2 * jj + e);
        const float4 v = p[i];
        p[i] = make_float4(v.x * sc.x, v.y * sc.x, v.z * sc.x, v.w * sc.x);
      }
    }
#pragma unroll
    for (int i = 0; i < CT; ++i) lsum[i] = 0.f;
    const float zero[16] = {};
#pragma unroll
    for (int ch = 0; ch < CT / 16; ++ch) put_acc(ch, zero);
    row_set = false;
    pending = true;
    bar();                                          // part is used again
  }

  // q' rows and beta of a packed tile; returns 2^-k of the tile's scaling of r s. Thread j of a
  // row's 16 takes channels ch .. ch + 3 and ch + 8 .. ch + 11, ch = 16 (j >> 1) + 4 (j & 1).
  __device__ float fold(const uint8_t* rec) {
    const uint16_t* km = reinterpret_cast<const uint16_t*>(rec + L::kKMetaOff);
    const int jj = tt & 15, r0 = tt >> 4, ch = 16 * (jj & 7) + 4 * (jj >> 3);
    float2 rs[4], rz[4];
    float m = 0.f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint2 sv = *reinterpret_cast<const uint2*>(km + L::kKs + ch + 8 * e);
      const uint2 zv = *reinterpret_cast<const uint2*>(km + L::kKz + ch + 8 * e);
      uint2 rv = make_uint2(kH_One, kH_One);
      if (!kLean) rv = *reinterpret_cast<const uint2*>(km + L::kKr + ch + 8 * e);
      rs[2 * e] = mul_h2(rv.x, sv.x);
      rs[2 * e + 1] = mul_h2(rv.y, sv.y);
      rz[2 * e] = mul_h2(rv.x, zv.x);
      rz[2 * e + 1] = mul_h2(rv.y, zv.y);
      m = fmax3f(m, rs[2 * e].x, rs[2 * e].y);
      m = fmax3f(m, rs[2 * e + 1].x, rs[2 * e + 1].y);
      m = fmax3f(m, fabsf(rz[2 * e].x) * (1.f / 64.f), fabsf(rz[2 * e].y) * (1.f / 64.f));
      m = fmax3f(m, fabsf(rz[2 * e + 1].x) * (1.f / 64.f), fabsf(rz[2 * e + 1].y) * (1.f / 64.f));
    }
    // the scales are positive: their maximum over the tile's channels as integers
    m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
    const float2 sc = tc_pow2_scale(m, 0);          // the largest r s into [1, 2)
    const float2 sc2 = make_float2(sc.x, sc.x);
    const float zf = sc.x * (1.f / (kKF * kBetaOne));        // beta in the units of S, over kBetaOne
    const float2 zf2 = make_float2(zf, zf);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      rs[e] = __fmul2_rn(rs[e], sc2);
      rz[e] = __fmul2_rn(rz[e], zf2);
    }
    const float* qs = reinterpret_cast<const float*>(sm + S::kQ);
    float b[R / 16];
#pragma unroll
    for (int k = 0; k < R / 16; ++k) {
      const int r = r0 + 16 * k;
      const float4* p = reinterpret_cast<const float4*>(qs + r * kD);
      const float4 u = p[jj], v = p[16 + jj];
      const float2 x[4] = {make_float2(u.x, u.y), make_float2(u.z, u.w), make_float2(v.x, v.y), make_float2(v.z, v.w)};
      uint32_t hi[4], lo[4];
      float2 b2 = make_float2(0.f, 0.f);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        split2p(__fmul2_rn(x[e], rs[e]), hi[e], lo[e]);
        b2 = __ffma2_rn(x[e], rz[e], b2);
      }
      b[k] = b2.x + b2.y;
      const int kk = 64 * (jj >> 3) + 8 * (jj & 7);
      *reinterpret_cast<uint4*>(sm + S::kB0 + tree_qo(r, kk)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      *reinterpret_cast<uint4*>(sm + S::kB0 + tree_qo_lo(r, kk)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
    // over the row's 16 threads: thread j ends up with row r0 + 16 (j & 3)'s sum (or (j & 1)'s)
    constexpr int kRows = R / 16;
#pragma unroll
    for (int o = kRows / 2; o >= 1; o >>= 1) {
      const bool up = (jj & o) != 0;
#pragma unroll
      for (int i = 0; i < o; ++i) {
        const float send = up ? b[i] : b[i + o], keep = up ? b[i + o] : b[i];
        b[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
      }
    }
#pragma unroll
    for (int o = kRows; o < 16; o <<= 1) b[0] += __shfl_xor_sync(0xffffffffu, b[0], o);
    if (jj < kRows) {
      const int r = r0 + 16 * jj;
      const __half h = __float2half_rn(b[0]);
      uint8_t* ext = sm + S::kExt + (r & 7) * 2;
      *reinterpret_cast<__half*>(ext + ((r >> 3) << 4)) = h;                                     // K element 0
      *reinterpret_cast<__half*>(ext + 128 + (((r >> 3) ^ 1) << 4)) = __float2half_rn((b[0] - __half2float(h)) * kBetaLo);   // 1
    }
    return sc.y;
  }

  // Operands of fresh tokens [f0, f0 + 128) of the cursor's sequence: keys and values as
  // they are, q as it is (hi rows).
  __device__ const uint16_t* fresh_row(int f, bool value) const {
    const TreeCursor& c = cur();
    if (f < c.ws) return a.ws + ((static_cast<int64_t>(c.s) * a.hkv + c.h) * 2 + (value ? 1 : 0)) * (kB * kD) + f * kD;
    return (value ? a.v_new : a.k_new) + ((c.c0 + (f - c.ws)) * a.hkv + c.h) * kD;
  }
  __device__ void fresh_keys(int f0) {
    const TreeCursor& c = cur();
    const int f = f0 + t, n = c.ws + c.nt, jj = tt & 15, r0 = tt >> 4;
    const int64_t c0 = c.c0;
    uint4 w[R / 16];
    const uint4* src = reinterpret_cast<const uint4*>(fresh_row(min(f, n - 1), false) + 64 * half);
#pragma unroll
    for (int i = 0; i < R / 16; ++i) {
      const int row = c.u * R + r0 + 16 * i, p = token_of(row);
      w[i] = make_uint4(0, 0, 0, 0);
      if (p < c.nt) w[i] = *reinterpret_cast<const uint4*>(q_row(c0, c.h, row, p) + 8 * jj);
    }
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      uint4 k[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) k[i] = src[4 * p + i];
      uint32_t r[16];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        r[4 * i] = f < n ? k[i].x : 0;
        r[4 * i + 1] = f < n ? k[i].y : 0;
        r[4 * i + 2] = f < n ? k[i].z : 0;
        r[4 * i + 3] = f < n ? k[i].w : 0;
      }
      tree_st16(trow + kTrAK + 32 * half + 16 * p, r);
    }
#pragma unroll
    for (int i = 0; i < R / 16; ++i) *reinterpret_cast<uint4*>(sm + S::kB0 + tree_qo(r0 + 16 * i, 8 * jj)) = w[i];
  }
  // A value that is not finite is left out of the product, where it would reach the rows that do
  // not attend its token (0 x infinity), and reported in small()[12].
  static __device__ bool finite(uint32_t h) { return (h & 0x7C00u) != 0x7C00u; }
  // Channel t of value f of a tile's (the workspace's rows from w on, then the drafted tokens').
  struct FreshValues {
    const uint16_t *w, *v;
    int64_t step;
    int nw, n;         // workspace tokens, all tokens from f0 on
    __device__ uint32_t at(int f) const { return *(f < nw ? w + f * kD : v + f * step); }
  };
  __device__ FreshValues fresh_source(int f0) const {
    const TreeCursor& c = cur();
    FreshValues x;
    x.nw = c.ws - f0;
    x.n = x.nw + c.nt;
    x.w = a.ws + ((static_cast<int64_t>(c.s) * a.hkv + c.h) * 2 + 1) * (kB * kD) + f0 * kD + t;
    x.step = static_cast<int64_t>(a.hkv) * kD;
    x.v = a.v_new + (c.c0 * a.hkv + c.h) * kD + t - x.nw * x.step;
    return x;
  }
  __device__ void fresh_values(int f0) {
    const FreshValues src = fresh_source(f0);
    bool all = true;
#pragma unroll 1
    for (int part = 0; part < 4; ++part) {
      const int p0 = 64 * half + 16 * part;
      uint32_t x[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = src.at(min(p0 + i, src.n - 1));   // loads of rows that are there, none waits for another
      uint32_t r[8];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const bool live = p0 + i < src.n, ok_i = finite(x[i]);
        all = all && (ok_i || !live);
        x[i] = live && ok_i ? x[i] : 0u;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) r[i] = x[2 * i] | (x[2 * i + 1] << 16);
      tree_st8(trow + kTrAV + 32 * half + 8 * part, r);
    }
    if (!all) small()[12] = 1.f;
  }
  // What rows attend, token by token (bit i: the thread's i-th row), and the values left out
  // above added to the rows that attend them.
  __device__ uint32_t* attended() const { return reinterpret_cast<uint32_t*>(sm + S::kU) + half * kB; }
  __device__ void add_infinite(int f0) {
    const FreshValues src = fresh_source(f0);
#pragma unroll 1
    for (int f = 0; f < min(src.n, kB); ++f) {
      const uint32_t x = src.at(f), bits = attended()[f];
      if (__all_sync(0xffffffffu, finite(x))) continue;
      const float add = finite(x) ? 0.f : h2f_bits(static_cast<uint16_t>(x));
#pragma unroll
      for (int ch = 0; ch < CT / 16; ++ch) {
        float y[16];
        get_acc(ch, y);
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] += (bits >> (16 * ch + i)) & 1u ? add : 0.f;
        put_acc(ch, y);
      }
    }
  }

  // Wait for a product; every thread of the team agrees on the outcome at the next barrier.
  __device__ void wait_qk() {
    ok = mbar_wait(&bars()[kTbQkDone], qph, a.flags) && ok;
    qph ^= 1u;
    tc_fence_after();
  }
  __device__ void wait_pv() {
    ok = mbar_wait(&bars()[kTbPvDone], pph, a.flags) && ok;
    pph ^= 1u;
    tc_fence_after();
  }

  struct Keys {        // what the thread's token (lane) is in the current item
    float f;           // factor of S
    int pk;            // position
    uint32_t seen;     // fresh tiles: bit i, whether the thread's i-th row attends it
    bool fresh;
  };
  // Scores of 16 rows relative to their running max: x = f S (then cap and bias) - max; masked keys -inf. f S is rounded
  // before the maximum is taken off, as it was for that: the largest is 0, however large it is. kWhole: f S without it.
  template <bool kWhole = false>
  __device__ void scores(int ch, const Keys& k, float (&x)[16]) {
    read16(ch, x);
    const float2 f2 = make_float2(k.f, k.f);
    if (kMod && a.cap > 0.f) {
      tree_cap(x, k.f, a.cap, a.cap_two);
    } else if (kMod) {
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] *= k.f;
    }
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const int col = CT * half + 16 * ch + i;
      const float4 m = kWhole ? make_float4(0.f, 0.f, 0.f, 0.f) : *reinterpret_cast<const float4*>(mrow() + col);
      if (!kMod) {
        const float2 none = make_float2(a.none, a.none);
        const float2 u = __fadd2_rn(__ffma2_rn(make_float2(x[i], x[i + 1]), f2, none), make_float2(m.x, m.y));
        const float2 v = __fadd2_rn(__ffma2_rn(make_float2(x[i + 2], x[i + 3]), f2, none), make_float2(m.z, m.w));
        x[i] = u.x; x[i + 1] = u.y; x[i + 2] = v.x; x[i + 3] = v.y;
      } else {
        const float mm[4] = {m.x, m.y, m.z, m.w};
        const int4 pq = *reinterpret_cast<const int4*>(pos() + col);
        const float4 sl = *reinterpret_cast<const float4*>(slope() + col);
        const int pp[4] = {pq.x, pq.y, pq.z, pq.w};
        const float ss[4] = {sl.x, sl.y, sl.z, sl.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int64_t gap = static_cast<int64_t>(pp[e]) - k.pk;
          float y = fmaf(-ss[e], static_cast<float>(gap), x[i + e]);
          if (a.window > 0 && gap >= a.window) y = -INFINITY;
          x[i + e] = y + mm[e];
        }
      }
      if (k.fresh) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (!((k.seen >> (16 * ch + i + e)) & 1u)) x[i + e] = -INFINITY;
      }
    }
  }

  // Some score exceeds its row's running max by more than kTau, or a row has not seen a key
  // yet: exact maxima of the tile, and everything moved to them.
  __device__ void rescale(const Keys& k, bool valid) {
#pragma unroll
    for (int ch = 0; ch < CT / 16; ++ch) {
      float x[16];
      scores<true>(ch, k, x);
      float m = tree_reduce<true>(x, lane);
      if (lane < 16) part()[warp * CT + 16 * ch + lane] = valid ? m : -INFINITY;
    }
    bar();
    if (tt < R) {                                   // row tt: its half's four warps
      const float* p = part() + 4 * (tt / CT) * CT + tt % CT;
      const float tile = fmax3f(fmaxf(p[0], p[CT]), p[2 * CT], p[3 * CT]), old = -mrow()[tt];
      float top = tile;                            // a row's first max may be any
      if (row_set || tile == -INFINITY) top = fmaxf(tile, old);
      else row_set = true;
      gam()[tt] = top - old;
      mrow()[tt] = -top;
      const bool miss = __any_sync(0xffffffffu, !row_set);
      if (lane == 0) small()[8 + warp] = miss ? 1.f : 0.f;
    }
    bar();
    pending = small()[8] != 0.f || (R == 64 && small()[9] != 0.f);
#pragma unroll
    for (int i = 0; i < CT; i += 4) {
      const float4 d = *reinterpret_cast<const float4*>(gam() + CT * half + i);
      // (a row's first max: nothing to scale yet)
      lsum[i] *= ex2(fminf(-d.x, 0.f));
      lsum[i + 1] *= ex2(fminf(-d.y, 0.f));
      lsum[i + 2] *= ex2(fminf(-d.z, 0.f));
      lsum[i + 3] *= ex2(fminf(-d.w, 0.f));
    }
#pragma unroll
    for (int ch = 0; ch < CT / 16; ++ch) {
      float v[16];
      get_acc(ch, v);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] *= ex2(fminf(-gam()[CT * half + 16 * ch + i], 0.f));
      put_acc(ch, v);
    }
  }

  // 16 rows' values of the thread's token into the B operand as hi and lo.
  __device__ void store_p(int ch, const float2 (&pp)[8]) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) split2p(pp[4 * c + e], hi[e], lo[e]);
      const int cc = CT / 8 * half + 2 * ch + c;
      uint8_t* b = sm + S::kB0;
      *reinterpret_cast<uint4*>(b + tree_po(cc, t)) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      *reinterpret_cast<uint4*>(R == 64 ? b + 16384 + tree_po(cc, t) : b + tree_po(cc + 4, t)) =
          make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
  }

  // Second half of a sum over tokens: part (written per warp) -> gam()[row]. Ends with a barrier.
  __device__ void join_rows() {
    bar();
    if (tt < R) {
      const float* p = part() + 4 * (tt / CT) * CT + tt % CT;
      gam()[tt] = (p[0] + p[CT]) + (p[2 * CT] + p[3 * CT]);
    }
    bar();
  }
  __device__ void sum_lsum() {
#pragma unroll
    for (int ch = 0; ch < CT / 16; ++ch) {
      float v[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = lsum[16 * ch + i];
      const float m = tree_reduce<false>(v, lane);
      if (lane < 16) part()[warp * CT + 16 * ch + lane] = m;
    }
    join_rows();
  }

  // acc (rotated channels) -> H acc / sqrt(128), by one more product with A = H. Rows are
  // divided by their sums on the way and scaled by a power of two, for the fp16 pairs.
  __device__ bool unrotate() {
    sum_lsum();
    {
      // row t of H: bit b of the column flips the sign where t has it; two columns a register
      uint32_t h[32];
      h[0] = 0x3C003C00u ^ ((t & 1) ? 0x80000000u : 0u) ^ ((half && (t & 64)) ? 0x80008000u : 0u);
#pragma unroll
      for (int b = 0; b < 5; ++b)
#pragma unroll
        for (int i = 0; i < (1 << b); ++i) h[i | (1 << b)] = h[i] ^ ((t >> (b + 1)) & 1 ? 0x80008000u : 0u);
      tc_st32(trow + kTrAV + 32 * half, h);
    }
    float top = 0.f;
#pragma unroll
    for (int ch = 0; ch < CT / 16; ++ch) {
      float v[16];
      get_acc(ch, v);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float l = gam()[CT * half + 16 * ch + i];
        v[i] = l > 0.f ? __fdividef(v[i], l) : 0.f;
        top = fmaxf(top, fabsf(v[i]));
      }
      put_acc(ch, v);
    }
    top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
    if (lane == 0) small()[warp] = top;
    bar();
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, small()[i]);
    const float2 sc = tc_pow2_scale(top, 13);
    const float2 sc2 = make_float2(sc.x, sc.x);
#pragma unroll
    for (int ch = 0; ch < CT / 16; ++ch) {
      float v[16];
      get_acc(ch, v);
      float2 pp[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) pp[i] = __fmul2_rn(make_float2(v[2 * i], v[2 * i + 1]), sc2);
      store_p(ch, pp);
    }
    product_pv(false);
    wait_pv();
#pragma unroll
    for (int ch = 0; ch < CT / 16; ++ch) {
      float v[16];
      read16(ch, v);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] *= gam()[CT * half + 16 * ch + i] * (kInvSqrt128 * sc.y);
      put_acc(ch, v);
    }
    tc_fence_before();
    return named_bar_and(bar_id, kTreeTeamThreads, ok);
  }

  __device__ void flush(int64_t rec_idx) {
    sum_lsum();
    float* out = a.part + rec_idx * tree_rec_floats(R);
#pragma unroll
    for (int ch = 0; ch < CT / 16; ++ch) {
      float v[16];
      get_acc(ch, v);
#pragma unroll
      for (int i = 0; i < 16; ++i) out[(CT * half + 16 * ch + i) * kD + t] = v[i];
    }
    if (tt < R) *reinterpret_cast<float2*>(out + R * kD + 2 * tt) = make_float2(row_set ? -mrow()[tt] : kNoMax, gam()[tt]);
    bar();
  }

  // Thread 0: starts copies until `limit` packed tiles have been issued (of `issued` so far);
  // a tile in a block that does not exist is flagged and marked.
  __device__ uint32_t refill(uint32_t issued, uint32_t limit) {
    TreeCursor& c = ahead();
    int64_t left = ahead_n();
    while (issued < limit && left > 0) {
      if (c.ti >= c.packed) {                    // on to the next unit
        left -= c.items - c.ti;
        if (left > 0) tree_next_unit<R>(a, c);
        continue;
      }
      const uint32_t stg = issued % kTreeStages;
      uint64_t* rec_bar = &bars()[kTbRec + stg];
      const int64_t blk = a.block_tables[static_cast<int64_t>(c.s) * a.max_blocks + c.first + c.ti];
      if (blk < 0 || blk >= a.num_blocks) {
        raise_flag(a.flags, KVARN_FLAG_BAD_BLOCK);
        valid_of()[stg] = 0;
        tc_arrive(rec_bar);
      } else {
        valid_of()[stg] = 1;
        mbar_arrive_expect_tx(rec_bar, L::kBytes);
        bulk_g2s(sm + S::kRec + stg * S::kRecPitch, a.cache + (blk * a.hkv + c.h) * static_cast<int64_t>(L::kBytes), L::kBytes,
                 rec_bar);
      }
      ++c.ti;
      ++issued;
      --left;
    }
    ahead_n() = left;
    return issued;
  }

  // One item: packed tile `ti` in stage used % kTreeStages, or the fresh tile at f0. False where the
  // team agreed that a wait has run out; the wait for the last product counts at the next agreement.
  __device__ bool item(bool fresh, int ti, int f0) {
    bool valid = true, wide = false;
    float cs = 1.f, cw = 0.f, rv = 1.f, cmax = 1.f;
    Keys key{0.f, 0, 0u, fresh};
    if (!fresh) {
      const uint32_t stg = used % kTreeStages;
      const uint8_t* rec = sm + S::kRec + stg * S::kRecPitch;
      const uint16_t* km = reinterpret_cast<const uint16_t*>(rec + L::kKMetaOff);
      const uint16_t* vm = reinterpret_cast<const uint16_t*>(rec + L::kVMetaOff);
      ok = mbar_wait(&bars()[kTbRec + stg], (used / kTreeStages) & 1u, a.flags) && ok;
      valid = valid_of()[stg] != 0;
      const bool go = __all_sync(0xffffffffu, ok) && valid;
      const int tok = code_token(t);
      if (go) {
        tree_keys<KB>(rec + L::kKCodeOff, tok, half, trow + kTrAK + 32 * half);
        const float kinv = fold(rec);
        // S is in units of code / kKF, q 2^e, r s 2^k, and q_r lacks its 1 / sqrt(128)
        key.f = h2f_bits(km[L::kKc + tok]) * (a.scale * kInvSqrt128 * kKF * kinv * qinv);
        const float cv = kLean ? 1.f : h2f_bits(vm[L::kVc + tok]);
        const float sv = h2f_bits(vm[L::kVs + tok]);
        const float zv = h2f_bits(vm[L::kVz + tok]);
        const float u0 = __fdividef(zv, sv);
        const bool near = fabsf(u0) <= kWide;
        const float u = near ? u0 : 0.f;
        // 2^(e - 10) where 2^e <= |u| + 16 < 2^(e + 1): |code + u^| < 2^(e + 1) has 11 bits above it
        const int e = __float_as_int(fabsf(u) + 16.f) & 0x7f800000;
        const float step = __int_as_float(e - (10 << 23)), inv = __int_as_float((264 << 23) - e);
        const float uh = rintf(u * inv) * step;
        cs = cv * sv;
        cw = near ? 0.f : cv * zv;
        rv = h2f_bits(vm[L::kVr + t]);
        if (half == 0) {
          const __half2 u2 = __float2half2_rn(near ? (u - uh) * (1.f / kVF) : 0.f);
          const uint32_t uu = *reinterpret_cast<const uint32_t*>(&u2);
          reinterpret_cast<uint4*>(sm + S::kU)[t] = make_uint4(uu, uu, uu, uu);
          reinterpret_cast<__half*>(sm + S::kAdd)[t] = __float2half_rn(uh * (1.f / kVF));
          // the warp's largest c s; negative where a token's zero is far off
          const float cm = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(cs)));
          const bool far = __any_sync(0xffffffffu, !near);
          if (lane == 0) small()[warp] = far ? -cm : cm;
        }
      }
      key.pk = (cur().first + ti) * kB + tok;
      product_qk(false);
      if (go) tree_values<VB>(rec + L::kVCodeOff, t, half, reinterpret_cast<const uint16_t*>(sm + S::kAdd), trow + kTrAV + 32 * half);
      const float4 c4 = *reinterpret_cast<const float4*>(small());
      cmax = fmaxf(fmaxf(fabsf(c4.x), fabsf(c4.y)), fmaxf(fabsf(c4.z), fabsf(c4.w)));
      wide = valid && fminf(fminf(c4.x, c4.y), fminf(c4.z, c4.w)) < 0.f;
    } else {
      if (tt == 0) small()[12] = 0.f;            // (read last behind the barriers of the tile before)
      fresh_keys(f0);
      product_qk(true);
      fresh_values(f0);
      const TreeCursor& c = cur();
      const int ft = f0 + t;
      const int ci = ft - c.ws;                  // index among the drafted tokens (negative: a workspace token)
      key.f = a.scale;
      if (ci < 0) {
        // behind all of the sequence's tiles, also those that a short block table leaves out
        if (kMod) key.pk = a.seq_lens[c.s] / kB * kB + ft;
        key.seen = ~0u;
      } else if (ci < c.nt) {
#pragma unroll
        for (int i = 0; i < CT; ++i) key.seen |= static_cast<uint32_t>((mask()[CT * half + i] >> ci) & 1u) << i;
        if (kMod && a.positions != nullptr) key.pk = a.positions[c.c0 + ci];
      }
    }

    wait_qk();
    float x[CT];
    float top = -INFINITY;
#pragma unroll
    for (int ch = 0; ch < CT / 16; ++ch) {
      scores(ch, key, *reinterpret_cast<float(*)[16]>(&x[16 * ch]));
#pragma unroll
      for (int i = 0; i < 16; i += 2) top = fmax3f(top, x[16 * ch + i], x[16 * ch + i + 1]);
    }
    // p' <= 2^kTau max(c s) 2^e < 2^14
    const float2 psc = tc_pow2_scale(cmax, 13 - static_cast<int>(kTau));
    if (tc_bar_or(bar_id, kTreeTeamThreads, (valid && top > kTau) || pending || !ok)) {
      ok = named_bar_and(bar_id, kTreeTeamThreads, ok);
      if (!ok) return false;
      rescale(key, valid);
#pragma unroll
      for (int ch = 0; ch < CT / 16; ++ch) scores(ch, key, *reinterpret_cast<float(*)[16]>(&x[16 * ch]));
    }
    if (valid) {
      const float csq = cs * psc.x;
      const float2 cs2 = make_float2(csq, csq);
#pragma unroll
      for (int ch = 0; ch < CT / 16; ++ch) {
        float2 pp[8];
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          const int j = 16 * ch + i;
          const float2 p = make_float2(ex2(x[j]), ex2(x[j + 1]));
          const float2 l = __fadd2_rn(make_float2(lsum[j], lsum[j + 1]), p);
          lsum[j] = l.x;
          lsum[j + 1] = l.y;
          pp[i / 2] = __fmul2_rn(p, cs2);
        }
        store_p(ch, pp);
      }
    }
    if (wide) {                            // the far tokens' part of gamma, summed over the lanes
#pragma unroll
      for (int ch = 0; ch < CT / 16; ++ch) {
        float g[16];
        scores(ch, key, g);
#pragma unroll
        for (int i = 0; i < 16; ++i) g[i] = cw != 0.f ? ex2(g[i]) * cw : 0.f;
        const float m = tree_reduce<false>(g, lane);
        if (lane < 16) part()[warp * CT + 16 * ch + lane] = m;
      }
    }
    const bool infinite = fresh && small()[12] != 0.f;
    if (infinite) {
      uint32_t bits = 0;
#pragma unroll
      for (int i = 0; i < CT; ++i) bits |= (x[i] != -INFINITY ? 1u : 0u) << i;
      attended()[t] = bits;
    }
    product_pv(!fresh);
    // while PV runs; the record was read before the barriers above
    if (tt == 0 && !fresh) issued = refill(issued, used + 1 + kTreeStages);
    if (wide) join_rows();
    wait_pv();
    if (valid) {
      const float of = rv * ((fresh ? 1.f : kVF) * psc.y);
      const float2 of2 = make_float2(of, of);
#pragma unroll
      for (int ch = 0; ch < CT / 16; ++ch) {
        float o[16], y[16];
        read16(ch, o);
        get_acc(ch, y);
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          const float2 v = __ffma2_rn(of2, make_float2(o[i], o[i + 1]), make_float2(y[i], y[i + 1]));
          y[i] = v.x;
          y[i + 1] = v.y;
        }
        if (wide) {
#pragma unroll
          for (int i = 0; i < 16; ++i) y[i] = fmaf(rv, gam()[CT * half + 16 * ch + i], y[i]);
        }
        put_acc(ch, y);
      }
    }
    if (infinite) {
      bar();
      add_infinite(f0);
      bar();
    }
    tc_fence_before();
    return true;
  }

  // The steps of tree_unit.
  __device__ bool packed_item(int ti) {
    const bool go = item(false, ti, 0);
    ++used;
    return go;
  }
  __device__ bool fresh_item(int ti) { return item(true, 0, (ti - cur().packed) * kB); }
  __device__ bool agreed() { return ok = named_bar_and(bar_id, kTreeTeamThreads, ok); }

  // Items [gb, ge).
  __device__ void run(int64_t gb, int64_t ge, int64_t team) {
    if (gb >= ge) return;
    if (tt == 0) {
      TreeCursor c;
      tree_locate<R>(a, gb, c);
      cur() = c;
      ahead() = c;
      ahead_n() = ge - gb;
      issued = refill(0, kTreeStages);
    }
    bar();
    for (int64_t left = ge - gb; left > 0;) {  // a unit
      const TreeCursor& c = cur();
      const int ti = c.ti;
      const int end = static_cast<int>(min(static_cast<int64_t>(c.items), ti + left));
      left -= end - ti;
      const int last = min(c.packed, end);
      enter();
      if (!tree_unit(*this, ti, last, end)) break;
      flush(team + (static_cast<int64_t>(c.s) * a.hkv + c.h) * a.max_units + c.u);
      if (tt == 0 && left > 0) tree_next_unit<R>(a, cur());
      bar();
    }
    if (tt == 0)                               // after a timeout: copies still in flight
      for (; used < issued; ++used) mbar_wait(&bars()[kTbRec + used % kTreeStages], (used / kTreeStages) & 1u, a.flags);
  }

  // Every product complete before TMEM is released.
  __device__ void finish() {
    if (warp == kTreeIssuer) {
      if (elect_one()) {
        umma_commit(&bars()[kTbFin]);
        mbar_wait(&bars()[kTbFin], 0, a.flags);
      }
      __syncwarp();
    }
  }
};

template <int KB, int VB, bool kLean, int R, bool kMod>
__global__ void __launch_bounds__(tree_teams(R) * kTreeTeamThreads, 1) tree_split_kernel(const __grid_constant__ TreeArgs a) {
  using S = TreeSm<KB, VB, kLean, R>;
  extern __shared__ __align__(1024) uint8_t smem[];
  tree_dep_launch();
  uint32_t* slot = reinterpret_cast<uint32_t*>(smem + S::kSlot);
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) >> 5, 0);
  if (threadIdx.x == 0) {
    for (int j = 0; j < S::kTeams; ++j) {
      uint64_t* bars = reinterpret_cast<uint64_t*>(smem + j * S::kTeam + S::kX + S::kBars);
      for (int i = 0; i <= kTbFin; ++i) mbar_init(&bars[i], 1);
    }
    fence_mbar_init();
  }
  if (warp == 0) tmem_alloc(slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *slot, 0);
  tree_dep_wait();                               // the scan's prefix
  const int j = warp >> 3;
  const int64_t team = static_cast<int64_t>(blockIdx.x) * S::kTeams + j;
  const int64_t total = a.prefix[a.n_seqs];
  TreeTeam<KB, VB, kLean, R, kMod> tm(a, smem + j * S::kTeam, tmem + j * tree_cols(R), j);
  tm.init();                                     // (made visible with the first operands)
  tm.run(team * total / a.n_teams, (team + 1) * total / a.n_teams, team);
  tm.finish();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ merge
// A warp per output row (token p, q-head m) of sequence blockIdx.y: joins the records of the teams
// that had items of the row's unit, 32 at a time (their maxima and sums one a lane, then the
// rows, lane l channels 4l .. 4l + 3, their loads independent of each other).
template <int R>
__global__ void __launch_bounds__(256) tree_merge_kernel(const TreeArgs a) {
  const int s = blockIdx.y, lane = threadIdx.x & 31, hq = a.hkv * a.group;
  const int id = blockIdx.x * 8 + (threadIdx.x >> 5), p = id / hq, m = id - p * hq;
  const TreeSeq q = tree_seq<R>(a, s, false);
  tree_dep_wait();
  if (p >= q.nt) return;
  const int64_t total = a.prefix[a.n_seqs], n = a.n_teams;
  const int64_t items = q.full - a.first[s] + q.fresh;
  const int h = m / a.group, row = p * a.group + (m - h * a.group), u = row / R, r = row - u * R;
  const int64_t g0 = a.prefix[s] + (static_cast<int64_t>(h) * q.units + u) * items;
  const int64_t unit = (static_cast<int64_t>(s) * a.hkv + h) * a.max_units + u;
  // team k owns items [k total / n, (k + 1) total / n): item g belongs to ((g + 1) n - 1) / total. Where
  // there are fewer items than teams every item has a team of its own.
  const bool sparse = total < n;
  const int64_t k0 = ((g0 + 1) * n - 1) / total;
  const int count = static_cast<int>(sparse ? items : ((g0 + items) * n - 1) / total - k0 + 1);
  float top = kNoMax, sum = 0.f;
  float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = 0; i0 < count; i0 += 32) {
    const int left = min(count - i0, 32);
    int64_t rec = 0;
    float2 ml = make_float2(kNoMax, 0.f);
    if (lane < left) {
      const int64_t k = sparse ? ((g0 + i0 + lane + 1) * n - 1) / total : k0 + i0 + lane;
      rec = (k + unit) * tree_rec_floats(R);
      ml = *reinterpret_cast<const float2*>(a.part + rec + R * kD + 2 * r);
    }
    float mx = ml.x;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float mn = fmaxf(top, mx), c0 = ex2(top - mn), w = ex2(ml.x - mn);
    top = mn;
    float l = ml.y * w;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    sum = sum * c0 + l;
    y.x *= c0;
    y.y *= c0;
    y.z *= c0;
    y.w *= c0;
#pragma unroll 4
    for (int j = 0; j < left; ++j) {
      const float wj = __shfl_sync(0xffffffffu, w, j);
      const float4 v = *reinterpret_cast<const float4*>(a.part + __shfl_sync(0xffffffffu, rec, j) + r * kD + 4 * lane);
      y.x = fmaf(v.x, wj, y.x);
      y.y = fmaf(v.y, wj, y.y);
      y.z = fmaf(v.z, wj, y.z);
      y.w = fmaf(v.w, wj, y.w);
    }
  }
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  const __half2 o0 = __floats2half2_rn(y.x * inv, y.y * inv), o1 = __floats2half2_rn(y.z * inv, y.w * inv);
  *reinterpret_cast<uint2*>(a.out + ((static_cast<int64_t>(a.cu[s]) + p) * hq + m) * kD + 4 * lane) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&o0), *reinterpret_cast<const uint32_t*>(&o1));
}

template <typename... KArgs, typename... Args>
cudaError_t tree_launch(void (*kernel)(KArgs...), dim3 grid, int block, size_t smem, bool after, cudaStream_t stream,
                        const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = after ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int KB, int VB, bool kLean, int R, bool kMod>
cudaError_t launch_tree_cfg(const TreeArgs& a, cudaStream_t stream) {
  using S = TreeSm<KB, VB, kLean, R>;
  static std::atomic<unsigned long long> smem_set{0};
  cudaError_t err = set_smem_once(tree_split_kernel<KB, VB, kLean, R, kMod>, S::kBytes, smem_set);
  if (err == cudaSuccess) err = tree_launch(tree_scan_kernel<R>, dim3(1), 1024, 0, false, stream, a);
  if (err == cudaSuccess)
    err = tree_launch(tree_split_kernel<KB, VB, kLean, R, kMod>, dim3(a.n_teams / S::kTeams), S::kTeams * kTreeTeamThreads, S::kBytes,
                      true, stream, a);
  if (err == cudaSuccess) err = tree_launch(tree_merge_kernel<R>, dim3((a.max_tree * a.hkv * a.group + 7) / 8, a.n_seqs), 256, 0,
                      true, stream, a);
  return err;
}

template <int KB, int VB, bool kLean>
cudaError_t launch_tree_preset(const TreeArgs& a, int rows, bool mod, cudaStream_t stream) {
  if (rows == 64)
    return mod ? launch_tree_cfg<KB, VB, kLean, 64, true>(a, stream) : launch_tree_cfg<KB, VB, kLean, 64, false>(a, stream);
  return mod ? launch_tree_cfg<KB, VB, kLean, 32, true>(a, stream) : launch_tree_cfg<KB, VB, kLean, 32, false>(a, stream);
}

// Rows of a unit: 32 where the longest tree has no more (a tile of 4 drafted tokens of 8 heads costs
// 0.76 of the 64-row one: 195 against 255 us for 16 sequences of 16384 tokens), 64 otherwise (a tile
// is unpacked once for them, against twice).
int tree_rows(int group, int max_tree) { return group * max_tree <= 32 ? 32 : 64; }

size_t tree_head_bytes(int n_seqs) {   // prefix, first
  return (static_cast<size_t>(n_seqs + 1) * 8 + static_cast<size_t>(n_seqs) * 4 + 255) / 256 * 256;
}

}  // namespace

size_t tree_scratch_bytes(int n_seqs, int hkv, int group, int max_tree) {
  const int r = tree_rows(group, max_tree);
  const size_t units = static_cast<size_t>(n_seqs) * hkv * ((group * max_tree + r - 1) / r);
  return tree_head_bytes(n_seqs) + (units + kTreeMaxTeams * kTreeMaxCtas) * tree_rec_floats(r) * sizeof(float);
}

cudaError_t launch_tree(const uint16_t* q, const uint16_t* k_new, const uint16_t* v_new, const uint64_t* tree_mask,
                        const int32_t* positions, const int32_t* cu_tokens, const int32_t* seq_lens, int n_seqs,
                        int64_t n_tokens, int max_tree, const int32_t* block_tables, const uint8_t* cache,
                        const uint16_t* ws, int hkv, int group, int max_blocks, int64_t num_blocks, int k_bits,
                        int v_bits, bool lean, const kvarn_score& score, uint16_t* out, void* scratch, unsigned* flags,
                        cudaStream_t stream) {
  TreeArgs a{};
  a.q = q; a.k_new = k_new; a.v_new = v_new;
  a.mask = tree_mask;
  a.positions = positions; a.cu = cu_tokens; a.seq_lens = seq_lens; a.block_tables = block_tables;
  a.cache = cache; a.ws = ws;
  a.slopes = score.slopes;
  a.out = out;
  a.flags = flags;
  a.prefix = static_cast<int64_t*>(scratch);
  a.first = reinterpret_cast<int32_t*>(a.prefix + n_seqs + 1);
  a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(scratch) + tree_head_bytes(n_seqs));
  a.num_blocks = num_blocks; a.n_tokens = n_tokens;
  a.n_seqs = n_seqs; a.max_tree = max_tree; a.hkv = hkv; a.group = group; a.max_blocks = max_blocks;
  a.window = score.window;
  a.scale = score.scale * kLog2e;
  a.none = -0.f;
  if (score.softcap > 0.f) {                     // (2^125 for every larger one, which leaves scores as they are too)
    a.cap = std::min(score.softcap * kLog2e, 4.2535296e+37f);
    a.cap_two = 2.f * kLog2e / a.cap;
  }
  a.group_inv = (65536 + group - 1) / group;
  const int rows = tree_rows(group, max_tree);
  a.max_units = (group * max_tree + rows - 1) / rows;
  int dev = 0, sms = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err == cudaSuccess) err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (err != cudaSuccess) return err;
  a.n_teams = tree_teams(rows) * std::max(1, std::min(sms, kTreeMaxCtas));
  const bool mod = score.softcap > 0.f || score.window > 0 || score.slopes != nullptr;
  if (k_bits == 4 && v_bits == 2)
    return lean ? launch_tree_preset<4, 2, true>(a, rows, mod, stream) : launch_tree_preset<4, 2, false>(a, rows, mod, stream);
  if (k_bits == 4 && v_bits == 4 && !lean) return launch_tree_preset<4, 4, false>(a, rows, mod, stream);
  if (k_bits == 2 && v_bits == 2 && !lean) return launch_tree_preset<2, 2, false>(a, rows, mod, stream);
  return cudaErrorInvalidValue;
}

}  // namespace kvarn

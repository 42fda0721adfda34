// Cached tokens back as plain K and V rows (KVarN README, "How KVarN works", read
// backwards): a packed tile's row is X[t] = H (r c_t (code s + z)), a token of the
// partial last tile is copied from the workspace; fp32 arithmetic, one rounding to the
// output's type.
//
// A work item is one tensor (K or V) of one tile of one (sequence, kv-head). With w_i the
// scale that belongs to a channel (keys r_i s_i, values r_i) a packed tile is
//   X[t][ch] = a_t sum_i (H_ch,i w_i) code_i,t + b_t sum_i H_ch,i y_i      (y: keys r z, values r)
// whose second sum is one transform of 128 numbers and whose first is a product:
//   fp16, bf16   read_tc_kernel: D[channel][token] on the 5th-generation tensor core. A = the signed
//                w_i as fp16 hi + lo (22 bits; rounded once to fp16 they alone would cost as
//                much as the output's rounding) in TMEM, lane = channel, one XOR a word from
//                a table of w; B = the codes, exact in fp16, in shared memory.
//   fp32         read_kernel: thread t decodes token t's 128 channels and rotates them in
//                registers (seven butterfly stages). The tensor core adds with fewer bits than fp32 has.
// Memory bound: 7 KB read, 32 KB written an item (fp16, k4v2).
// 16 sequences of 16384 tokens, 8 kv-heads, fp16 out: 330 us, 4.0 TB/s of 1.31 GB (58 % of a plain
// copy's rate, five bytes of six written; the registers' transform took 443). Without the front's work
// 266, without the products 3 less: operands and rows contend for shared memory. Two teams at the front
// took 333, two at the back 358 (72 registers a thread); rows stored by threads instead of by boxes 372. (24 to 36 bytes of
// spill stores at 96 registers.) fp32 out: 604 us of 2.38 GB, 58 %; k4v4 548 us, 66 % (60 bytes of spills but for k4v4).
//
// Items are found on the device: a warp walks the sequences 32 at a time (one a lane, their
// tile counts scanned by shuffles) and takes every n-th item, so a ragged batch costs no
// empty blocks and the host needs no lengths.
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

#include "decode_tc.cuh"
#include "kvarn_codes.cuh"
#include "kvarn_launch.h"
#include "kvarn_unpack.cuh"

namespace kvarn {
namespace {

constexpr int kReadThreads = 128;
constexpr int kReadPitch = 272;   // bytes of a staged 256-byte row: 8 rows' 16-byte pieces hit 32 banks

struct ReadArgs {
  CUtensorMap map[2];             // fp16, bf16: k and v as [n_tokens][hkv * 128]
  const uint8_t* cache;
  const uint16_t* ws;
  const int32_t *block_tables, *seq_lens, *first, *cu;
  void *k, *v;
  unsigned* flags;
  int64_t num_blocks, n_tokens;   // n_tokens: rows of k and v
  int n_seqs, hkv, max_blocks;
};

// The range of sequence s: tokens [beg, end) that exist, at output row row0 + (token - beg).
struct ReadRange {
  int beg, end, full;     // full: its packed tiles
  int64_t row0;
};
__device__ __forceinline__ ReadRange read_range(const ReadArgs& a, int s, bool report) {
  ReadRange r;
  const int64_t c0 = a.cu[s], c1 = a.cu[s + 1];
  const int64_t f = a.first != nullptr ? a.first[s] : 0;
  const int64_t len = max(a.seq_lens[s], 0);
  int64_t lo = max(f, static_cast<int64_t>(0)), hi = min(f + (c1 - c0), len);
  if (c0 < 0) hi = lo;                                    // offsets that are none
  hi = min(hi, f + (a.n_tokens - c0));                    // rows behind the output's end
  if (report && c1 > c0 && (c0 < 0 || lo != f || hi != f + (c1 - c0))) raise_flag(a.flags, KVARN_FLAG_BAD_LENGTH);
  r.beg = static_cast<int>(lo);
  r.end = static_cast<int>(max(hi, lo));
  r.full = static_cast<int>(len / kB);
  r.row0 = c0 + (lo - f);
  return r;
}

template <class T>
__device__ __forceinline__ uint32_t pack2(float2 v);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float2 v) {
  const __half2 h = __floats2half2_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float2 v) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

struct ReadItem {
  int sq, h, ti, g;       // sequence, kv-head, tile, 0 keys / 1 values
  int lo, hi;             // rows [lo, hi) of the tile are read
  int full;               // packed tiles of the sequence
  int64_t row0;           // output row of the tile's row 0
};
// Items first, first + stride, .. of all; the warp calls and answers together.
struct ReadCursor {
  int64_t item, base, total, incl, mine;   // base: items of the sequences before the current 32
  ReadRange rg;
  int s0;
  __device__ explicit ReadCursor(int64_t first) : item(first), base(0), total(0), incl(0), mine(0), rg{0, 0, 0, 0}, s0(-32) {}
  __device__ bool next(const ReadArgs& a, int64_t stride, bool report, ReadItem& it) {
    const int lane = threadIdx.x & 31;
    while (item - base >= total) {
      base += total;
      s0 += 32;
      if (s0 >= a.n_seqs) {
        s0 -= 32;
        base -= total;
        return false;
      }
      const int s = s0 + lane;
      int tiles = 0;
      rg = ReadRange{0, 0, 0, 0};
      if (s < a.n_seqs) {
        rg = read_range(a, s, report);
        if (rg.end > rg.beg) tiles = (rg.end - 1) / kB - rg.beg / kB + 1;
      }
      incl = mine = static_cast<int64_t>(tiles) * a.hkv * 2;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
      }
      total = __shfl_sync(0xffffffffu, incl, 31);
    }
    const int64_t off = item - base;
    item += stride;
    const int src = __popc(__ballot_sync(0xffffffffu, incl <= off));       // the sequence's lane
    it.sq = s0 + src;
    const int beg = __shfl_sync(0xffffffffu, rg.beg, src), end = __shfl_sync(0xffffffffu, rg.end, src);
    const int64_t in = off - __shfl_sync(0xffffffffu, incl - mine, src);
    it.g = static_cast<int>(in & 1);
    const int64_t th = in >> 1;
    const int64_t tile = (th >> 31) == 0 ? static_cast<int>(th) / a.hkv : th / a.hkv;
    it.h = static_cast<int>(th - tile * a.hkv);
    it.ti = beg / kB + static_cast<int>(tile);
    it.full = __shfl_sync(0xffffffffu, rg.full, src);
    it.lo = max(beg - it.ti * kB, 0);
    it.hi = min(end - it.ti * kB, kB);
    it.row0 = __shfl_sync(0xffffffffu, rg.row0, src) + (static_cast<int64_t>(it.ti) * kB - beg);
    return true;
  }
};
// The entry of the block table of an item's tile (-1 where the table has none, or none is needed).
__device__ __forceinline__ int read_block(const ReadArgs& a, const ReadItem& it) {
  return it.ti < min(it.full, a.max_blocks) ? a.block_tables[static_cast<int64_t>(it.sq) * a.max_blocks + it.ti] : -1;
}
// What an item's rows come from: the packed tile's record, or the workspace (the partial last
// tile). Neither: flagged, nothing is written.
__device__ __forceinline__ bool read_source(const ReadArgs& a, const ReadItem& it, int blk, bool report,
                                            int64_t record_bytes, const uint8_t*& rec, const uint16_t*& ws) {
  rec = nullptr;
  ws = nullptr;
  unsigned bad = 0;
  if (it.ti >= it.full) {
    if (a.ws == nullptr) bad = KVARN_FLAG_BAD_LENGTH;
    else ws = a.ws + ((static_cast<int64_t>(it.sq) * a.hkv + it.h) * 2 + it.g) * (kB * kD);
  } else if (it.ti >= a.max_blocks) {
    bad = KVARN_FLAG_BAD_LENGTH;
  } else if (blk < 0 || blk >= a.num_blocks) {
    bad = KVARN_FLAG_BAD_BLOCK;
  } else {
    rec = a.cache + (static_cast<int64_t>(blk) * a.hkv + it.h) * record_bytes;
  }
  if (bad && report) raise_flag(a.flags, bad);
  return bad == 0;
}
template <class T>
__device__ __forceinline__ T* read_out(const ReadArgs& a, int g, int64_t row, int h) {
  return static_cast<T*>(g ? a.v : a.k) + (row * a.hkv + h) * kD;
}
// Rows [lo, hi) of the workspace's tile, by `n` threads.
template <class T>
__device__ __forceinline__ void read_workspace(const uint16_t* w, T* out, int64_t stride, int lo, int hi, int t, int n) {
  for (int r = lo + (t >> 4); r < hi; r += n / 16) {
    const uint4 u = *reinterpret_cast<const uint4*>(w + r * kD + 8 * (t & 15));
    T* dst = out + r * stride + 8 * (t & 15);
    if constexpr (std::is_same<T, __half>::value) {
      *reinterpret_cast<uint4*>(dst) = u;
    } else {
      const uint32_t uu[4] = {u.x, u.y, u.z, u.w};
      float2 f[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = __half22float2(*reinterpret_cast<const __half2*>(&uu[i]));
      if constexpr (sizeof(T) == 4) {
        reinterpret_cast<float4*>(dst)[0] = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
        reinterpret_cast<float4*>(dst)[1] = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
      } else {
        *reinterpret_cast<uint4*>(dst) = make_uint4(pack2<T>(f[0]), pack2<T>(f[1]), pack2<T>(f[2]), pack2<T>(f[3]));
      }
    }
  }
}

// ------------------------------------------------------------------ fp32
template <int KB, int VB, bool kLean>
__global__ void __launch_bounds__(kReadThreads, 3) read_kernel(const ReadArgs a) {
  using L = RecordLayout<KB, VB, kLean>;
  constexpr int kCodes = L::kKCodeBytes > L::kVCodeBytes ? L::kKCodeBytes : L::kVCodeBytes;
  // codes and metadata of one tensor, then the staged rows (128 of 256 bytes at kReadPitch)
  __shared__ __align__(16) uint8_t sm_codes[kCodes];
  __shared__ __align__(16) uint8_t sm_meta[L::kMetaBytes];
  __shared__ __align__(16) float2 sm_ab[128];
  extern __shared__ __align__(16) uint8_t sm_rows[];
  const int t = threadIdx.x;
  const int64_t stride = static_cast<int64_t>(a.hkv) * kD;

  ReadCursor cursor(blockIdx.x);
  ReadItem it;
  while (cursor.next(a, gridDim.x, blockIdx.x == 0 && t < 32, it)) {
    const uint8_t* rec;
    const uint16_t* w;
    if (!read_source(a, it, read_block(a, it), t == 0, L::kBytes, rec, w)) continue;
    float* out = read_out<float>(a, it.g, it.row0, it.h);
    if (w != nullptr) {
      read_workspace<float>(w, out, stride, it.lo, it.hi, t, kReadThreads);
      continue;
    }
    const int g = it.g;
    const uint8_t* codes = rec + (g ? L::kVCodeOff : L::kKCodeOff);
    const uint8_t* meta = rec + (g ? L::kVMetaOff : L::kKMetaOff);
    __syncthreads();                          // the previous item's shared memory is read
    const int nc = (g ? L::kVCodeBytes : L::kKCodeBytes) / 16;
#pragma unroll 4
    for (int i = t; i < nc; i += kReadThreads)
      reinterpret_cast<uint4*>(sm_codes)[i] = reinterpret_cast<const uint4*>(codes)[i];
    if (t < L::kMetaBytes / 16) reinterpret_cast<uint4*>(sm_meta)[t] = reinterpret_cast<const uint4*>(meta)[t];
    __syncthreads();
    const uint16_t* m = reinterpret_cast<const uint16_t*>(sm_meta);
    float scale = kInvSqrt128;                // H is orthonormal; for keys the token's c_t too
    float av = 0.f, bv = 0.f;
    if (g == 0) {
      const float r = kLean ? 1.f : h2f_bits(m[L::kKr + t]);
      const float s16 = r * h2f_bits(m[L::kKs + t]) * static_cast<float>(1 << KB);
      sm_ab[t] = make_float2(s16, fmaf(r, h2f_bits(m[L::kKz + t]), -s16));
      scale *= h2f_bits(m[L::kKc + t]);
    } else {
      const float c = kLean ? 1.f : h2f_bits(m[L::kVc + t]);
      av = c * h2f_bits(m[L::kVs + t]) * static_cast<float>(1 << VB);
      bv = fmaf(c, h2f_bits(m[L::kVz + t]), -av);
      reinterpret_cast<float*>(sm_ab)[t] = h2f_bits(m[L::kVr + t]);
    }
    __syncthreads();
    float2 x[64];
    if (g == 0)
      read_keys<KB>(sm_codes, sm_ab, t, x);
    else
      read_values<VB>(sm_codes, reinterpret_cast<const float*>(sm_ab), av, bv, t, x);
    fwht128(x);
    const float2 s2 = make_float2(scale, scale);
    // rows through shared memory, 64 channels at a time, so that 16 lanes store 256 bytes together
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      if (part > 0) __syncthreads();
      uint8_t* mine_row = sm_rows + t * kReadPitch;
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        const float2 p = __fmul2_rn(x[32 * part + 2 * c], s2), q = __fmul2_rn(x[32 * part + 2 * c + 1], s2);
        *reinterpret_cast<float4*>(mine_row + 16 * c) = make_float4(p.x, p.y, q.x, q.y);
      }
      __syncthreads();
#pragma unroll 4
      for (int r = t >> 4; r < kB; r += kReadThreads / 16)
        if (r >= it.lo && r < it.hi)
          *reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(out + r * stride) + 256 * part + 16 * (t & 15)) =
              *reinterpret_cast<const uint4*>(sm_rows + r * kReadPitch + 16 * (t & 15));
    }
  }
}

// ------------------------------------------------------------------ fp16, bf16
// One block an SM. Warps 0-7 (the front) turn an item's record into its product's operands, warps 8-15
// (the back) turn the product into rows, one warp fetches records, one issues products; operands,
// product and rows are double buffered, so that each works on an item of its own. Handed on by
// mbarriers, each of two (an item's by its number's parity):
//   filled  the record is there                    fetch  -> front
//   ready   the operands are, the record is free   front  -> issue, fetch
//   done    the product is                         issue  -> back
//   free    and has been read, the tables too      back   -> front
constexpr int kRtTeam = 256, kRtThreads = 2 * kRtTeam + 64;
constexpr uint32_t kRtHi = 0, kRtLo = 64, kRtA = 128, kRtD = 256, kRtCols = 512;   // TMEM: two A, two D of 128 columns
constexpr int kRtFilled = 0, kRtReady = 2, kRtDone = 4, kRtFree = 6;
struct ReadDesc {
  void* out;              // output row of the tile's row 0, and its place in the output's map
  int x, y;
  const uint16_t* ws;     // workspace rows, or NULL
  int lo, hi, g, live;
};
template <int KB, int VB, bool kLean>
struct ReadSm {
  using L = RecordLayout<KB, VB, kLean>;
  static constexpr int kCodes = L::kKCodeBytes > L::kVCodeBytes ? L::kKCodeBytes : L::kVCodeBytes;
  static constexpr int kB0 = 0, kBPitch = 32768;
  static constexpr int kRows = 2 * kBPitch, kRowsPitch = 32768;   // staged output rows, as the map's boxes
  static constexpr int kStage = kCodes + L::kMetaBytes;
  static constexpr int kRec = kRows + 2 * kRowsPitch;    // two stages of codes and metadata
  static constexpr int kW = kRec + 2 * kStage;           // [8 warps] 64 fp16 hi, 64 fp16 lo of w
  static constexpr int kA = kW + 8 * 256, kBt = kA + 512, kBeta = kBt + 512;   // [128] f32 each, twice
  static constexpr int kTab = 1536;
  static constexpr int kDesc = kA + 2 * kTab;            // two for the front, two for issue and back
  static constexpr int kBars = kDesc + 4 * static_cast<int>(sizeof(ReadDesc));
  static constexpr int kSlot = kBars + 64, kBytes = kSlot + 8;
  static_assert(kBytes <= 232448, "read shared memory");
};

// 16 lanes x 32 columns: thread T has lanes T / 4 and T / 4 + 8, columns 8 j + 2 (T % 4) and the next,
// in registers 4 j .. 4 j + 3 (the layout of a matrix product's accumulator).
__device__ __forceinline__ void read_ld16x32(uint32_t taddr, float (&v)[16]) {
  uint32_t(&r)[16] = reinterpret_cast<uint32_t(&)[16]>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ uint32_t read_xor3(uint32_t a, uint32_t b, uint32_t c) {   // one instruction
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0x96;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
// Four 8 x 8 matrices of 16-bit elements, each written transposed.
__device__ __forceinline__ void read_stmatrix(void* p, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(smem_u32(p)), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}

template <class T, int KB, int VB, bool kLean>
struct ReadTeam {
  using L = RecordLayout<KB, VB, kLean>;
  using S = ReadSm<KB, VB, kLean>;
  const ReadArgs& a;
  uint8_t* sm;
  uint32_t tm, trow;
  int tt, t, half, lane, warp;             // thread tt of front or back: TMEM lane t, half of the columns

  __device__ ReadTeam(const ReadArgs& a_, uint8_t* sm_, uint32_t tm_) : a(a_), sm(sm_), tm(tm_) {
    tt = threadIdx.x & (kRtTeam - 1);
    t = tt & 127;
    half = tt >> 7;
    lane = tt & 31;
    warp = __shfl_sync(0xffffffffu, tt >> 5, 0);
    trow = tm + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
  }
  __device__ uint64_t* bar(int kind, uint32_t k) const { return reinterpret_cast<uint64_t*>(sm + S::kBars) + kind + (k & 1); }
  // Item k's turn at a barrier (warp-uniform).
  __device__ bool wait(int kind, uint32_t k) const {
    return __all_sync(0xffffffffu, mbar_wait(bar(kind, k), (k >> 1) & 1u, a.flags));
  }
  __device__ void arrive(int kind, uint32_t k) const {   // one of the team's 8 warps
    __syncwarp();
    if (lane == 0) tc_arrive(bar(kind, k));
  }
  __device__ ReadDesc& desc(int k) const { return reinterpret_cast<ReadDesc*>(sm + S::kDesc)[k]; }
  __device__ float* table(int off, int stg) const { return reinterpret_cast<float*>(sm + off + stg * S::kTab); }

  // The fetching warp: the block's items into the two stages in turn, as they become free; the last is
  // none. The cursor is an item ahead, so that the block table's entry is there.
  __device__ void fetch() {
    const bool report = blockIdx.x == 0;
    ReadCursor c(blockIdx.x);
    ReadItem ahead{};
    int blk = -1;
    bool more = c.next(a, gridDim.x, report, ahead), live = true;
    if (more) blk = read_block(a, ahead);
    for (uint32_t k = 0; live; ++k) {
      const uint8_t* rec = nullptr;
      const uint16_t* ws = nullptr;
      ReadItem it = ahead;
      live = false;
      while (!live && more) {
        it = ahead;
        const int b = blk;
        more = c.next(a, gridDim.x, report, ahead);
        if (more) blk = read_block(a, ahead);
        live = read_source(a, it, b, lane == 0, L::kBytes, rec, ws);
      }
      if (k >= 2 && !wait(kRtReady, k - 2)) {
        wait(kRtFilled, k - 1);                 // (timed out: the copy still in flight)
        return;
      }
      if (lane == 0) {
        ReadDesc& d = desc(k & 1);
        d.live = live;
        if (live) {
          d.out = read_out<T>(a, it.g, it.row0, it.h);
          d.x = it.h * kD;
          d.y = static_cast<int>(it.row0);
          d.ws = ws;
          d.lo = it.lo;
          d.hi = it.hi;
          d.g = it.g;
        }
        uint64_t* filled = bar(kRtFilled, k);
        if (live && rec != nullptr) {
          uint8_t* dst = sm + S::kRec + (k & 1) * S::kStage;
          const uint32_t codes = it.g ? L::kVCodeBytes : L::kKCodeBytes;
          mbar_arrive_expect_tx(filled, codes + L::kMetaBytes);
          bulk_g2s(dst, rec + (it.g ? L::kVCodeOff : L::kKCodeOff), codes, filled);
          bulk_g2s(dst + S::kCodes, rec + (it.g ? L::kVMetaOff : L::kKMetaOff), L::kMetaBytes, filled);
        } else {
          tc_arrive(filled);
        }
      }
      __syncwarp();
    }
  }

  // The lane's channels 4 lane .. 4 lane + 3: w, and y of the transform.
  __device__ void channels(const uint16_t* m, int g, float (&w)[4], float (&y)[4]) const {
    const uint2 one = make_uint2(kH_One, kH_One);
    const uint2 rv = g ? *reinterpret_cast<const uint2*>(m + L::kVr + 4 * lane)
                       : kLean ? one : *reinterpret_cast<const uint2*>(m + (kLean ? 0 : L::kKr) + 4 * lane);
    const uint2 sv = g ? one : *reinterpret_cast<const uint2*>(m + L::kKs + 4 * lane);
    const uint2 zv = g ? one : *reinterpret_cast<const uint2*>(m + L::kKz + 4 * lane);
    const float2 w0 = mul_h2(rv.x, sv.x), w1 = mul_h2(rv.y, sv.y), y0 = mul_h2(rv.x, zv.x), y1 = mul_h2(rv.y, zv.y);
    w[0] = w0.x; w[1] = w0.y; w[2] = w1.x; w[3] = w1.y;
    y[0] = y0.x; y[1] = y0.y; y[2] = y1.x; y[3] = y1.y;
  }

  // What the packed tile in stage `stg` needs before its product: B, the warp's table of w, and the
  // epilogue's tables.
  __device__ void prepare(int stg, int g) {
    const uint8_t* codes = sm + S::kRec + stg * S::kStage;
    const uint16_t* m = reinterpret_cast<const uint16_t*>(codes + S::kCodes);
    uint8_t* brow = sm + S::kB0 + stg * S::kBPitch + half * 16384 + t * 128;
    auto put = [&](int i, uint32_t (&r)[16]) {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        *reinterpret_cast<uint4*>(brow + (((4 * i + c) ^ (t & 7)) << 4)) =
            make_uint4(r[4 * c], r[4 * c + 1], r[4 * c + 2], r[4 * c + 3]);
    };
    if (g == 0)
      key_codes<KB>(codes, t, half, put);    // row = token, K = channels in code_token's order
    else
      value_codes<VB>(codes, t, half, put);  // K = channel, its row the tokens in that order
    // w as fp16 hi + lo in the order of K, the warp's half
    float w[4], y[4];
    channels(m, g, w, y);
    float top = fmaxf(fmaxf(fabsf(w[0]), fabsf(w[1])), fmaxf(fabsf(w[2]), fabsf(w[3])));
    top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
    const float2 sc = tc_pow2_scale(top, 13);
    uint32_t hi[2], lo[2];
    split2p(make_float2(w[0] * sc.x, w[1] * sc.x), hi[0], lo[0]);
    split2p(make_float2(w[2] * sc.x, w[3] * sc.x), hi[1], lo[1]);
    uint8_t* wt = sm + S::kW + warp * 256;
    if ((g ? lane >> 4 : lane & 1) == half) {
      const int k = g ? 4 * (lane & 15) : ((lane >> 1) & 1) * 4 + (lane >> 2) * 8;   // in the half
      *reinterpret_cast<uint2*>(wt + 2 * k) = make_uint2(hi[0], hi[1]);
      *reinterpret_cast<uint2*>(wt + 128 + 2 * k) = make_uint2(lo[0], lo[1]);
    }
    if (warp == 0) transform(stg, y);
    if (warp >= 4) columns(m, g, t, sc.y, stg);
    __syncwarp();
  }
  // A of the product: A[channel t][k] = w_k with the sign of H: the parity of channel & k, in
  // K's order of bits.
  __device__ void signs(int stg, int g) {
    const uint8_t* wt = sm + S::kW + warp * 256;
    const int p = g ? t : (t & 3) | ((t >> 3) & 1) << 2 | ((t >> 4) & 7) << 3 | ((t >> 2) & 1) << 6;
    const uint32_t s0 = ((p & 1) ? 0x80000000u : 0u) ^ ((half && (p & 64)) ? 0x80008000u : 0u);
    const uint32_t b1 = (p & 2) ? 0x80008000u : 0u, b2 = (p & 4) ? 0x80008000u : 0u;
    const uint32_t low[4] = {s0, s0 ^ b1, s0 ^ b2, s0 ^ b1 ^ b2};
    uint32_t f[8] = {};
#pragma unroll
    for (int b = 0; b < 3; ++b)
#pragma unroll
      for (int i = 0; i < (1 << b); ++i) f[i | (1 << b)] = f[i] ^ ((p >> (3 + b)) & 1 ? 0x80008000u : 0u);
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      uint32_t r[32];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const uint4 v = reinterpret_cast<const uint4*>(wt + 128 * part)[q];
        r[4 * q] = read_xor3(v.x, low[0], f[q]);
        r[4 * q + 1] = read_xor3(v.y, low[1], f[q]);
        r[4 * q + 2] = read_xor3(v.z, low[2], f[q]);
        r[4 * q + 3] = read_xor3(v.w, low[3], f[q]);
      }
      tc_st32(trow + stg * kRtA + (part ? kRtLo : kRtHi) + 32 * half, r);
    }
  }
  __device__ void product(int stg, int g) {
    tc_fence_after();
    const uint64_t b = smem_desc_sw128(smem_u32(sm + S::kB0 + stg * S::kBPitch));
    const uint32_t at = tm + stg * kRtA + kRtHi, d = tm + kRtD + stg * 128;
    if (g == 0) {
      constexpr uint32_t kId = idesc_f16_f32(128, 128);
#pragma unroll
      for (int s = 0; s < 16; ++s)
        tc_umma_ts(d, at + 8 * s, b + ((((s >> 2) & 1) * 16384 + (s & 3) * 32) >> 4), kId, s > 0);
    } else {
      constexpr uint32_t kId = idesc_f16_f32(128, 64) | (1u << 16);   // B with N contiguous
#pragma unroll
      for (int s = 0; s < 16; ++s)
#pragma unroll
        for (int n = 0; n < 2; ++n)
          tc_umma_ts(d + 64 * n, at + 8 * s, b + ((n * 16384 + (s & 7) * 2048) >> 4), kId, s > 0);
    }
    umma_commit(bar(kRtDone, stg));
  }
  // sum_i H_ch,i y_i for the 128 channels, lane l holding y of 4 l .. 4 l + 3.
  __device__ void transform(int stg, float (&y)[4]) {
    const float u0 = y[0] + y[1], u1 = y[0] - y[1], u2 = y[2] + y[3], u3 = y[2] - y[3];
    y[0] = u0 + u2; y[1] = u1 + u3; y[2] = u0 - u2; y[3] = u1 - u3;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float sg = (lane & o) ? -1.f : 1.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = fmaf(y[i], sg, __shfl_xor_sync(0xffffffffu, y[i], o));
    }
    reinterpret_cast<float4*>(table(S::kBeta, stg))[lane] = make_float4(y[0], y[1], y[2], y[3]);
  }
  // a and b of D's column n (its token).
  __device__ void columns(const uint16_t* m, int g, int n, float inv, int stg) {
    float av, bv;
    if (g == 0) {
      bv = h2f_bits(m[L::kKc + n]) * kInvSqrt128;
      av = bv * ((KB == 4 ? 8.f : 2.f) * inv);
    } else {
      const int tok = code_token(n);
      const float c = (kLean ? 1.f : h2f_bits(m[(kLean ? 0 : L::kVc) + tok])) * kInvSqrt128;
      bv = c * h2f_bits(m[L::kVz + tok]);
      av = c * h2f_bits(m[L::kVs + tok]) * ((VB == 4 ? 8.f : 2.f) * inv);
    }
    table(S::kA, stg)[n] = av;
    table(S::kBt, stg)[n] = bv;
  }
  // D to the item's rows, staged by token as two boxes of 64 channels (128-byte swizzled; the tokens
  // of 8 columns of values differ in 4 of their low bits only, which puts two lanes on a bank).
  __device__ void stage_rows(int stg, int g) {
    const int q = warp & 3, r0 = 32 * q + (lane >> 2), mt = lane >> 3, l7 = lane & 7;
    const int tok0 = g ? (l7 & 3) | half << 2 | (l7 >> 2) << 3 | (mt >> 1) << 4 : l7 | (mt >> 1) << 3 | half << 6;
    uint8_t* const rows = sm + S::kRows + stg * S::kRowsPitch + (q >> 1) * 16384 + tok0 * 128;
    const int sw = tok0 & 7, chunk = 4 * (q & 1) + (mt & 1), cj = g ? 4096 : 2048;   // bytes between columns 16 apart
    float be[2][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) be[i >> 1][i & 1] = table(S::kBeta, stg)[r0 + 8 * i];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int n0 = 64 * half + 32 * c;
      float2 av[4], bv[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        av[j] = *reinterpret_cast<const float2*>(table(S::kA, stg) + n0 + 8 * j + 2 * (lane & 3));
        bv[j] = *reinterpret_cast<const float2*>(table(S::kBt, stg) + n0 + 8 * j + 2 * (lane & 3));
      }
#pragma unroll
      for (int sub = 0; sub < 2; ++sub) {
        float x[16];
        read_ld16x32(trow + (static_cast<uint32_t>(16 * sub) << 16) + kRtD + stg * 128 + n0, x);
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
          uint32_t r[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {          // (columns 8 (j + e / 2) .., rows 8 (e % 2) ..)
            const int jj = j + (e >> 1), k = 4 * jj + 2 * (e & 1);
            const float b = be[sub][e & 1];
            r[e] = pack2<T>(__ffma2_rn(make_float2(x[k], x[k + 1]), av[jj], __fmul2_rn(bv[jj], make_float2(b, b))));
          }
          read_stmatrix(rows + (2 * c + (j >> 1)) * cj + (((chunk + 2 * sub) ^ sw) << 4), r);
        }
      }
    }
  }

  // Rows [lo, hi) of a tile that is not read as a whole, 16 lanes a row.
  __device__ void store_rows(int stg, const ReadDesc& d) {
    const int l = tt & 15, row = a.hkv * (kD * static_cast<int>(sizeof(T)));          // bytes
    const uint8_t* src = sm + S::kRows + stg * S::kRowsPitch + (l >> 3) * 16384;
    uint8_t* out = static_cast<uint8_t*>(d.out) + 16 * l;
    for (int r = d.lo + (tt >> 4); r < d.hi; r += kRtTeam / 16)
      *reinterpret_cast<uint4*>(out + static_cast<int64_t>(r) * row) =
          *reinterpret_cast<const uint4*>(src + r * 128 + (((l & 7) ^ (r & 7)) << 4));
  }

  __device__ void front() {
    for (uint32_t k = 0;; ++k) {
      const int stg = k & 1;
      if (!wait(kRtFilled, k)) return;
      const ReadDesc d = desc(stg);
      if (k >= 2 && !wait(kRtFree, k - 2)) return;
      if (d.live && d.ws == nullptr) {
        prepare(stg, d.g);
        signs(stg, d.g);
      }
      if (tt == 0) desc(2 + stg) = d;
      tc_operands_written();
      arrive(kRtReady, k);
      if (!d.live) return;
    }
  }
  __device__ void issue() {
    for (uint32_t k = 0;; ++k) {
      const int stg = k & 1;
      if (!wait(kRtReady, k)) break;
      const ReadDesc d = desc(2 + stg);
      const bool packed = d.live && d.ws == nullptr;
      if (packed && elect_one()) product(stg, d.g);
      __syncwarp();
      if (lane == 0) {                          // with the product's own arrival, two
        tc_arrive(bar(kRtDone, k));
        if (!packed) tc_arrive(bar(kRtDone, k));
      }
      if (!d.live) break;
    }
  }
  __device__ void back() {
    for (uint32_t k = 0;; ++k) {
      const int stg = k & 1;
      bool ok = wait(kRtDone, k);
      tc_fence_after();
      ReadDesc d{};
      if (ok) d = desc(2 + stg);
      const bool packed = d.live && d.ws == nullptr;
      if (packed) stage_rows(stg, d.g);
      tc_fence_before();
      arrive(kRtFree, k);
      fence_proxy_async_smem();
      if (tt == 0) bulk_wait_read_all();        // the rows of the item before have left
      ok = named_bar_and(1, kRtTeam, ok);
      if (!ok || !d.live) return;
      if (packed && d.lo == 0 && d.hi == kB) {
        if (tt == 0) {
          const uint8_t* src = sm + S::kRows + stg * S::kRowsPitch;
          tma_store_2d(&a.map[d.g], d.x, d.y, src);
          tma_store_2d(&a.map[d.g], d.x + 64, d.y, src + 16384);
          bulk_commit();
        }
      } else if (packed) {
        store_rows(stg, d);
      } else {
        read_workspace<T>(d.ws, static_cast<T*>(d.out), static_cast<int64_t>(a.hkv) * kD, d.lo, d.hi, tt, kRtTeam);
      }
    }
  }
};

template <class T, int KB, int VB, bool kLean>
__global__ void __launch_bounds__(kRtThreads, 1) read_tc_kernel(const __grid_constant__ ReadArgs a) {
  using S = ReadSm<KB, VB, kLean>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint32_t* slot = reinterpret_cast<uint32_t*>(smem + S::kSlot);
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) >> 5, 0);
  if (threadIdx.x == 0) {
    for (int i = 0; i < 8; ++i)
      mbar_init(reinterpret_cast<uint64_t*>(smem + S::kBars) + i, i < kRtReady ? 1 : i >= kRtDone && i < kRtFree ? 2 : 8);
    fence_mbar_init();
  }
  if (warp == 0) tmem_alloc(slot, kRtCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *slot, 0);
  ReadTeam<T, KB, VB, kLean> team(a, smem, tmem);
  if (warp < 8)
    team.front();
  else if (warp < 16)
    team.back();
  else if (warp == 16)
    team.fetch();
  else
    team.issue();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, kRtCols);
}

template <class T, int KB, int VB, bool kLean>
cudaError_t launch_read_cfg(ReadArgs& a, int sms, cudaStream_t stream) {
  constexpr bool kTc = sizeof(T) == 2;
  constexpr int kSmem = kTc ? ReadSm<KB, VB, kLean>::kBytes : kB * kReadPitch;
  static std::atomic<unsigned long long> smem_set{0};
  // no more blocks than items could exist
  const int64_t most = (a.n_tokens / kB + 2 * static_cast<int64_t>(a.n_seqs)) * a.hkv * 2;
  cudaError_t err;
  if constexpr (kTc) {
    err = set_smem_once(read_tc_kernel<T, KB, VB, kLean>, kSmem, smem_set);
    for (int g = 0; g < 2 && err == cudaSuccess; ++g)
      err = tile_map(&a.map[g], g ? a.v : a.k, static_cast<uint64_t>(a.hkv) * kD,
                     static_cast<uint64_t>(std::max<int64_t>(a.n_tokens, kB)));   // (used for whole tiles only)
    if (err != cudaSuccess) return err;
    const int64_t grid = std::min(static_cast<int64_t>(sms), most);
    read_tc_kernel<T, KB, VB, kLean><<<static_cast<unsigned>(grid), kRtThreads, kSmem, stream>>>(a);
  } else {
    err = set_smem_once(read_kernel<KB, VB, kLean>, kSmem, smem_set);
    if (err != cudaSuccess) return err;
    const int64_t grid = std::min(3 * static_cast<int64_t>(sms), most);   // three blocks an SM (their registers' limit)
    read_kernel<KB, VB, kLean><<<static_cast<unsigned>(grid), kReadThreads, kSmem, stream>>>(a);
  }
  return cudaGetLastError();
}

template <class T>
cudaError_t launch_read_type(ReadArgs& a, int k_bits, int v_bits, bool lean, int sms, cudaStream_t stream) {
  if (k_bits == 4 && v_bits == 2)
    return lean ? launch_read_cfg<T, 4, 2, true>(a, sms, stream) : launch_read_cfg<T, 4, 2, false>(a, sms, stream);
  if (k_bits == 4 && v_bits == 4 && !lean) return launch_read_cfg<T, 4, 4, false>(a, sms, stream);
  if (k_bits == 2 && v_bits == 2 && !lean) return launch_read_cfg<T, 2, 2, false>(a, sms, stream);
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_read(const uint8_t* cache, const uint16_t* ws, const int32_t* block_tables, const int32_t* seq_lens,
                        const int32_t* first, const int32_t* cu_tokens, int n_seqs, int64_t n_tokens, int hkv,
                        int max_blocks, int64_t num_blocks, int k_bits, int v_bits, bool lean, int dtype, void* k,
                        void* v, unsigned* flags, cudaStream_t stream) {
  ReadArgs a{};
  a.cache = cache; a.ws = ws;
  a.block_tables = block_tables; a.seq_lens = seq_lens; a.first = first; a.cu = cu_tokens;
  a.k = k; a.v = v;
  a.flags = flags;
  a.num_blocks = num_blocks; a.n_tokens = n_tokens;
  a.n_seqs = n_seqs; a.hkv = hkv; a.max_blocks = max_blocks;
  int dev = 0, sms = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err == cudaSuccess) err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (err != cudaSuccess) return err;
  return dtype == KVARN_F16    ? launch_read_type<__half>(a, k_bits, v_bits, lean, sms, stream)
         : dtype == KVARN_BF16 ? launch_read_type<__nv_bfloat16>(a, k_bits, v_bits, lean, sms, stream)
                               : launch_read_type<float>(a, k_bits, v_bits, lean, sms, stream);
}

}  // namespace kvarn

// Cached tokens back as plain K and V rows (KVarN README, "How KVarN works", read
// backwards): a packed tile's row is X[t] = H (r c_t (code s + z)), a token of the
// partial last tile is copied from the workspace; fp32 arithmetic, one rounding to the
// output's type.
//
// A work item is one tensor (K or V) of one tile of one (sequence, kv-head), 128
// threads. Packed tiles: thread t decodes token t's 128 channels into registers and
// rotates them there (seven butterfly stages between registers, no shuffles); 1/sqrt(128)
// and the token's scale are applied at the end. The rows then go through shared memory
// so that 16 lanes store a row's 256 bytes together. Memory bound: 7 KB read, 32 KB
// written an item (fp16).
//
// Items are found on the device: every block walks the sequences 32 at a time (one a
// lane, their tile counts scanned by shuffles) and takes items blockIdx.x + k gridDim.x,
// so a ragged batch costs no empty blocks and the host needs no lengths.
#include <cuda_bf16.h>

#include <type_traits>

#include "kvarn_common.cuh"
#include "kvarn_launch.h"
#include "kvarn_unpack.cuh"

namespace kvarn {
namespace {

constexpr int kReadThreads = 128;
constexpr int kReadPitch = 272;   // bytes of a staged 256-byte row: 8 rows' 16-byte pieces hit 32 banks

struct ReadArgs {
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
  int beg, end;
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

template <class T, int KB, int VB, bool kLean>
__global__ void __launch_bounds__(kReadThreads, 3) read_kernel(const ReadArgs a) {
  using L = RecordLayout<KB, VB, kLean>;
  constexpr int kElem = static_cast<int>(sizeof(T));
  constexpr int kCodes = L::kKCodeBytes > L::kVCodeBytes ? L::kKCodeBytes : L::kVCodeBytes;
  // codes and metadata of one tensor, then the staged rows (128 of 256 bytes at kReadPitch)
  __shared__ __align__(16) uint8_t sm_codes[kCodes];
  __shared__ __align__(16) uint8_t sm_meta[L::kMetaBytes];
  __shared__ __align__(16) float2 sm_ab[128];
  extern __shared__ __align__(16) uint8_t sm_rows[];
  const int t = threadIdx.x, lane = t & 31;
  const int per_tile = a.hkv * 2;

  int64_t base = 0;                     // items of the sequences before this round's 32
  int64_t item = blockIdx.x;
  for (int s0 = 0; s0 < a.n_seqs; s0 += 32) {
    const int s = s0 + lane;
    int tiles = 0;
    ReadRange rg{0, 0, 0};
    if (s < a.n_seqs) {
      rg = read_range(a, s, blockIdx.x == 0 && t < 32);
      if (rg.end > rg.beg) tiles = (rg.end - 1) / kB - rg.beg / kB + 1;
    }
    int64_t incl = static_cast<int64_t>(tiles) * per_tile;
    const int64_t mine = incl;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    const int64_t total = __shfl_sync(0xffffffffu, incl, 31);
    for (; item - base < total; item += gridDim.x) {
      const int64_t off = item - base;
      const int src = __popc(__ballot_sync(0xffffffffu, incl <= off));       // the sequence's lane
      const int sq = s0 + src;
      const int beg = __shfl_sync(0xffffffffu, rg.beg, src), end = __shfl_sync(0xffffffffu, rg.end, src);
      const int64_t row0 = __shfl_sync(0xffffffffu, rg.row0, src);
      const int64_t in = off - (__shfl_sync(0xffffffffu, incl, src) - __shfl_sync(0xffffffffu, mine, src));
      const int g = static_cast<int>(in & 1);
      const int64_t th = in >> 1;
      const int h = static_cast<int>(th % a.hkv), ti = beg / kB + static_cast<int>(th / a.hkv);
      const int lo = max(beg - ti * kB, 0), hi = min(end - ti * kB, kB);      // rows of the tile
      T* out = static_cast<T*>(g ? a.v : a.k) + ((row0 + (static_cast<int64_t>(ti) * kB - beg)) * a.hkv + h) * kD;
      const int64_t stride = static_cast<int64_t>(a.hkv) * kD;
      if (ti >= a.seq_lens[sq] / kB) {          // the partial tile: workspace rows
        if (a.ws == nullptr) {
          if (t == 0) raise_flag(a.flags, KVARN_FLAG_BAD_LENGTH);
          continue;
        }
        const uint16_t* w = a.ws + ((static_cast<int64_t>(sq) * a.hkv + h) * 2 + g) * (kB * kD);
        for (int r = lo + (t >> 4); r < hi; r += kReadThreads / 16) {
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
              *reinterpret_cast<uint4*>(dst) =
                  make_uint4(pack2<T>(f[0]), pack2<T>(f[1]), pack2<T>(f[2]), pack2<T>(f[3]));
            }
          }
        }
        continue;
      }
      if (ti >= a.max_blocks) {
        if (t == 0) raise_flag(a.flags, KVARN_FLAG_BAD_LENGTH);
        continue;
      }
      const int64_t blk = a.block_tables[static_cast<int64_t>(sq) * a.max_blocks + ti];
      if (blk < 0 || blk >= a.num_blocks) {
        if (t == 0) raise_flag(a.flags, KVARN_FLAG_BAD_BLOCK);
        continue;
      }
      const uint8_t* rec = a.cache + (blk * a.hkv + h) * static_cast<int64_t>(L::kBytes);
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
      // rows through shared memory, 256 bytes (all 128 channels of a 2-byte type, 64 of fp32) at a time
#pragma unroll
      for (int part = 0; part < kElem / 2; ++part) {
        if (part > 0) __syncthreads();
        uint8_t* mine_row = sm_rows + t * kReadPitch;
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          uint4 u;
          if constexpr (sizeof(T) == 4) {
            const float2 p = __fmul2_rn(x[32 * part + 2 * c], s2), q = __fmul2_rn(x[32 * part + 2 * c + 1], s2);
            u = make_uint4(__float_as_uint(p.x), __float_as_uint(p.y), __float_as_uint(q.x), __float_as_uint(q.y));
          } else {
            u = make_uint4(pack2<T>(__fmul2_rn(x[4 * c], s2)), pack2<T>(__fmul2_rn(x[4 * c + 1], s2)),
                           pack2<T>(__fmul2_rn(x[4 * c + 2], s2)), pack2<T>(__fmul2_rn(x[4 * c + 3], s2)));
          }
          *reinterpret_cast<uint4*>(mine_row + 16 * c) = u;
        }
        __syncthreads();
#pragma unroll 4
        for (int r = t >> 4; r < kB; r += kReadThreads / 16)
          if (r >= lo && r < hi)
            *reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(out + r * stride) + 256 * part + 16 * (t & 15)) =
                *reinterpret_cast<const uint4*>(sm_rows + r * kReadPitch + 16 * (t & 15));
      }
    }
    base += total;
  }
}

template <class T, int KB, int VB, bool kLean>
cudaError_t launch_read_cfg(const ReadArgs& a, int sms, cudaStream_t stream) {
  constexpr int kSmem = kB * kReadPitch;
  static std::atomic<unsigned long long> smem_set{0};
  cudaError_t err = set_smem_once(read_kernel<T, KB, VB, kLean>, kSmem, smem_set);
  if (err != cudaSuccess) return err;
  // three blocks an SM (their registers' limit); no more blocks than items could exist
  int64_t grid = 3 * static_cast<int64_t>(sms);
  const int64_t most = (a.n_tokens / kB + 2 * static_cast<int64_t>(a.n_seqs)) * a.hkv * 2;
  if (grid > most) grid = most;
  read_kernel<T, KB, VB, kLean><<<static_cast<unsigned>(grid), kReadThreads, kSmem, stream>>>(a);
  return cudaGetLastError();
}

template <class T>
cudaError_t launch_read_type(const ReadArgs& a, int k_bits, int v_bits, bool lean, int sms, cudaStream_t stream) {
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

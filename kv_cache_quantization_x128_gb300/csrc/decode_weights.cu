// Decode attention that also adds up each packed tile's attention weight (what eviction by
// accumulated weight goes by) and gives the log-sum-exp: with x_gj the scores of q-head g,
//   out_g = sum_j p_gj v_j,  p_gj = exp(x_gj - lse_g),  lse_g = ln sum_j exp(x_gj)
//   w_t <- decay w_t + sum over the group's heads g and the tile's tokens j of p_gj
// in one pass over the records. The weights need lse, which is known when the pass is over,
// so the split phase leaves (m, l) of each tile and q-head: the running maximum behind the tile and the
// tile's sum of 2^(score - m), 64 bytes beside the record's 10 to 18 KB; the merge, which has
// the unit's maximum and sum, turns them into weights, a thread a tile.
// The tile is the unit of weight because it is that of the record: its per-channel scales
// bind 128 tokens, which cannot leave one record for another without being quantized again.
//
// Launches and shapes are those of kvarn_decode_attention (decode.cu: scan, split, merge; the
// device code is shared, decode_tile.cuh). q' and p' are scaled by powers of two, per head
// and tile, before they become fp16 pairs, so keys and values of any scales keep 22 bits.
#include "decode_launch.cuh"
#include "decode_tile.cuh"
#include "kvarn_common.cuh"
#include "kvarn_launch.h"

namespace kvarn {
namespace {

template <int KB, int VB, bool kLean, class Cfg>
__global__ void __launch_bounds__(Cfg::kWarps * 32, 1) weigh_split_kernel(WeighArgs a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  griddep_launch_dependents();          // the merge kernel waits for this grid itself
  griddep_wait();                       // the scan's prefix
  split_body<KB, VB, kLean, Cfg, WeighArgs>(a, smem, blockIdx.x);
}

template <int kMinBlocks, int kParts>
__global__ void __launch_bounds__(256 * kParts, kMinBlocks) weigh_merge_kernel(WeighArgs a, const uint16_t* __restrict__ ws,
                                                                              uint16_t* __restrict__ out) {
  __shared__ WsPart sm;
  __shared__ RecShares<kParts> rs;
  __shared__ WeighPart wp;
  merge_body<8, kParts, SplitWait, WeighArgs>(a, ws, out, blockIdx.x, blockIdx.y, sm, &rs, a.ranges, SplitWait(), &wp);
}

template <int KB, int VB, bool kLean, class C>
cudaError_t launch_weigh_cfg(WeighArgs& a, cudaStream_t stream) {
  static std::atomic<unsigned long long> smem_set{0};
  cudaError_t err = set_smem_once(weigh_split_kernel<KB, VB, kLean, C>, C::kSmem, smem_set);
  if (err != cudaSuccess) return err;
  return launch_after(weigh_split_kernel<KB, VB, kLean, C>, dim3(a.n_ctas), dim3(C::kWarps * 32), C::kSmem, stream, a);
}

template <int KB, int VB, bool kLean>
cudaError_t launch_weigh(WeighArgs& a, bool few_units, cudaStream_t stream) {
  a.warps = few_units ? SplitCfg2<KB, VB, kLean>::kWarps : SplitCfg<KB, VB, kLean>::kWarps;
  decode_scan_kernel<<<1, 1024, 0, stream>>>(a);
  const cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess || a.max_blocks == 0) return err;
  return few_units ? launch_weigh_cfg<KB, VB, kLean, SplitCfg2<KB, VB, kLean>>(a, stream)
                   : launch_weigh_cfg<KB, VB, kLean, SplitCfg<KB, VB, kLean>>(a, stream);
}

size_t stats_offset(int n_seqs, int hkv, int max_blocks) {
  return (decode_part_bytes(n_seqs, hkv, max_blocks) + 255) & ~size_t(255);
}

}  // namespace

size_t decode_weights_scratch_bytes(int n_seqs, int hkv, int max_blocks) {
  return stats_offset(n_seqs, hkv, max_blocks) + static_cast<size_t>(n_seqs) * hkv * max_blocks * 8 * sizeof(float2);
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
  a.prefix = reinterpret_cast<int64_t*>(at);
  a.ranges = reinterpret_cast<int64_t*>(at + prefix_bytes(n_seqs));
  a.part = reinterpret_cast<float*>(at + prefix_bytes(n_seqs) + kRangeBytes);
  a.flags = flags;
  a.num_blocks = num_blocks;
  a.n_seqs = n_seqs;
  a.hkv = hkv;
  a.group = group;
  a.max_blocks = max_blocks;
  a.n_ctas = decode_num_ctas();
  a.cover = cover_ptr(a.part, n_seqs, hkv, a.n_ctas);
  a.stats = reinterpret_cast<float2*>(at + stats_offset(n_seqs, hkv, max_blocks));
  a.weights = weights;
  a.lse = lse;
  a.decay = decay;
  // (the shapes are chosen as in launch_decode)
  const int64_t units = static_cast<int64_t>(n_seqs) * hkv;
  const bool few = units <= a.n_ctas;
  const cudaError_t err = k_bits == 2   ? launch_weigh<2, 2, false>(a, few, stream)
                          : v_bits == 4 ? launch_weigh<4, 4, false>(a, few, stream)
                          : lean        ? launch_weigh<4, 2, true>(a, few, stream)
                                        : launch_weigh<4, 2, false>(a, few, stream);
  if (err != cudaSuccess) return err;
  const bool long_units = static_cast<int64_t>(a.n_ctas) * a.warps >= 8 * units && max_blocks >= 8;
  return long_units ? launch_after(weigh_merge_kernel<1, 4>, dim3(hkv, n_seqs), dim3(1024), 0, stream, a, ws, out)
                    : launch_after(weigh_merge_kernel<4, 1>, dim3(hkv, n_seqs), dim3(256), 0, stream, a, ws, out);
}

}  // namespace kvarn

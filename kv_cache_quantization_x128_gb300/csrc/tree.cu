// Attention of drafted tokens over the packed cache, the workspace and the drafted
// tokens themselves: one block per (new token, kv-head, sequence), 128 threads, fp32.
#include "kvarn_common.cuh"
#include "kvarn_launch.h"
#include "kvarn_unpack.cuh"

namespace kvarn {
namespace {

struct TreeArgs {
  const uint16_t *q, *k_new, *v_new;
  const uint64_t* mask;
  const int32_t *positions, *cu, *seq_lens, *block_tables;
  const uint8_t* cache;
  const uint16_t* ws;
  const float* slopes;
  uint16_t* out;
  unsigned* flags;
  int64_t num_blocks, n_tokens;
  int n_seqs, max_tree, hkv, group, max_blocks, window;
  float scale, softcap;
};

struct TreeSmem {
  float q[8][128], qr[8][128], p[8][128], red[8][4];
  float2 ab[128];
  float rv[128];
  float rows[128][129];
};

// Score of (query at pq, key at pk).
__device__ __forceinline__ float tree_score(const TreeArgs& a, float x, float slope, int pq, int pk) {
  x *= a.scale;
  if (a.softcap > 0.f) x = a.softcap * tanhf(x / a.softcap);
  if (a.slopes != nullptr) x -= slope * static_cast<float>(pq - pk);
  if (a.window > 0 && static_cast<int64_t>(pq) - pk >= a.window) x = -INFINITY;
  return x;
}

// One block of up to 128 keys: thread t's key row dots are sc[g] (-inf: none); V rows in
// sm.rows. Updates the running max, sum and the thread's channel of acc.
__device__ __forceinline__ void tree_step(TreeSmem& sm, int t, float (&sc)[8], float (&m)[8], float (&l)[8],
                                          float (&acc)[8], float (&other)[8]) {
  const int w = t >> 5;
#pragma unroll
  for (int g = 0; g < 8; ++g) {
    float v = sc[g];
    for (int o = 16; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    if ((t & 31) == 0) sm.red[g][w] = v;
  }
  __syncthreads();
#pragma unroll
  for (int g = 0; g < 8; ++g) {
    const float mt = fmaxf(fmaxf(sm.red[g][0], sm.red[g][1]), fmaxf(sm.red[g][2], sm.red[g][3]));
    const float mn = fmaxf(m[g], mt);
    const float corr = mn == -INFINITY ? 1.f : expf(m[g] - mn);
    const float p = mn == -INFINITY ? 0.f : expf(sc[g] - mn);
    m[g] = mn;
    l[g] = l[g] * corr + p;
    acc[g] *= corr;
    other[g] *= corr;
    sm.p[g][t] = p;
  }
  __syncthreads();
  for (int j = 0; j < 128; ++j) {
    const float v = sm.rows[j][t];
#pragma unroll
    for (int g = 0; g < 8; ++g) acc[g] = fmaf(sm.p[g][j], v, acc[g]);
  }
  __syncthreads();
}

template <int KB, int VB, bool kLean>
__global__ void __launch_bounds__(128) tree_kernel(const TreeArgs a) {
  using L = RecordLayout<KB, VB, kLean>;
  extern __shared__ __align__(16) uint8_t raw[];
  TreeSmem& sm = *reinterpret_cast<TreeSmem*>(raw);
  const int t = threadIdx.x, h = blockIdx.y, s = blockIdx.z, p = blockIdx.x;
  const int c0 = a.cu[s];
  const int n = a.cu[s + 1] - c0;
  if (n > a.max_tree && p == 0 && h == 0 && t == 0) raise_flag(a.flags, KVARN_FLAG_BAD_LENGTH);
  const int nt = min(n, a.max_tree);
  if (p >= nt) return;
  if (c0 < 0 || static_cast<int64_t>(c0) + nt > a.n_tokens) {
    if (t == 0) raise_flag(a.flags, KVARN_FLAG_BAD_LENGTH);
    return;
  }
  const int64_t tok = c0 + p;
  const int len = max(a.seq_lens[s], 0), full = min(len / kB, a.max_blocks);
  if (len / kB > a.max_blocks && t == 0) raise_flag(a.flags, KVARN_FLAG_BAD_LENGTH);
  const int pq = a.positions != nullptr ? a.positions[tok] : 0;
  const int hq = a.hkv * a.group;
  float slope[8], m[8], l[8], acc[8], accr[8];
#pragma unroll
  for (int g = 0; g < 8; ++g) {
    const bool live = g < a.group;
    slope[g] = a.slopes != nullptr && live ? a.slopes[h * a.group + g] : 0.f;
    sm.q[g][t] = live ? h2f_bits(a.q[(tok * hq + h * a.group + g) * kD + t]) : 0.f;
    m[g] = -INFINITY;
    l[g] = acc[g] = accr[g] = 0.f;
  }
  __syncthreads();
#pragma unroll
  for (int g = 0; g < 8; ++g) {
    float x = 0.f;
    for (int i = 0; i < 128; ++i) x += (__popc(i & t) & 1) ? -sm.q[g][i] : sm.q[g][i];
    sm.qr[g][t] = x * kInvSqrt128;
  }
  __syncthreads();
  float sc[8];
  for (int ti = 0; ti < full; ++ti) {
    const int64_t blk = a.block_tables[static_cast<int64_t>(s) * a.max_blocks + ti];
    if (blk < 0 || blk >= a.num_blocks) {
      if (t == 0) raise_flag(a.flags, KVARN_FLAG_BAD_BLOCK);
      continue;
    }
    const uint8_t* rec = a.cache + (blk * a.hkv + h) * static_cast<int64_t>(L::kBytes);
    const uint16_t* km = reinterpret_cast<const uint16_t*>(rec + L::kKMetaOff);
    const uint16_t* vm = reinterpret_cast<const uint16_t*>(rec + L::kVMetaOff);
    const float r = kLean ? 1.f : h2f_bits(km[L::kKr + t]);
    const float s16 = r * h2f_bits(km[L::kKs + t]) * static_cast<float>(1 << KB);
    sm.ab[t] = make_float2(s16, fmaf(r, h2f_bits(km[L::kKz + t]), -s16));
    sm.rv[t] = h2f_bits(vm[L::kVr + t]);
    __syncthreads();
    float2 x[64];
    read_keys<KB>(rec + L::kKCodeOff, sm.ab, t, x);
    const float ck = h2f_bits(km[L::kKc + t]);
#pragma unroll
    for (int g = 0; g < 8; ++g) {
      float d = 0.f;
#pragma unroll
      for (int i = 0; i < 64; ++i) d += x[i].x * sm.qr[g][2 * i] + x[i].y * sm.qr[g][2 * i + 1];
      sc[g] = tree_score(a, d * ck, slope[g], pq, ti * kB + t);
    }
    const float c = kLean ? 1.f : h2f_bits(vm[L::kVc + t]);
    const float av = c * h2f_bits(vm[L::kVs + t]) * static_cast<float>(1 << VB);
    read_values<VB>(rec + L::kVCodeOff, sm.rv, av, fmaf(c, h2f_bits(vm[L::kVz + t]), -av), t, x);
#pragma unroll
    for (int i = 0; i < 64; ++i) {
      sm.rows[t][2 * i] = x[i].x;
      sm.rows[t][2 * i + 1] = x[i].y;
    }
    tree_step(sm, t, sc, m, l, accr, acc);
  }
  // workspace, then new tokens
  const uint64_t word = a.mask != nullptr ? a.mask[tok] : ~0ull >> (63 - p);
  for (int part = 0; part < 2; ++part) {
    const int cnt = part == 0 ? len % kB : nt;
    if (cnt == 0) continue;
    if (part == 0 && a.ws == nullptr) {
      if (t == 0) raise_flag(a.flags, KVARN_FLAG_BAD_LENGTH);
      continue;
    }
    const uint16_t* kr = part == 0 ? a.ws + (static_cast<int64_t>(s) * a.hkv + h) * 2 * kB * kD
                                   : a.k_new + (static_cast<int64_t>(c0) * a.hkv + h) * kD;
    const uint16_t* vr = part == 0 ? kr + kB * kD : a.v_new + (static_cast<int64_t>(c0) * a.hkv + h) * kD;
    const int64_t stride = part == 0 ? kD : static_cast<int64_t>(a.hkv) * kD;
    const bool live = t < cnt && (part == 0 || ((word >> (t & 63)) & 1));
    const int pk = part == 0 ? len / kB * kB + t : (a.positions != nullptr && t < cnt ? a.positions[c0 + t] : 0);
#pragma unroll
    for (int g = 0; g < 8; ++g) {
      float d = 0.f;
      if (t < cnt)
        for (int i = 0; i < 128; ++i) d += h2f_bits(kr[t * stride + i]) * sm.q[g][i];
      sc[g] = live ? tree_score(a, d, slope[g], pq, pk) : -INFINITY;
    }
    for (int j = 0; j < 128; ++j) sm.rows[j][t] = j < cnt ? h2f_bits(vr[j * stride + t]) : 0.f;
    tree_step(sm, t, sc, m, l, acc, accr);
  }
  // rotate the packed part back, join, normalise
  __syncthreads();
#pragma unroll
  for (int g = 0; g < 8; ++g) {
    sm.q[g][t] = accr[g];
    sm.p[g][t] = l[g];
  }
  __syncthreads();
#pragma unroll
  for (int g = 0; g < 8; ++g) {
    if (g >= a.group) continue;
    float x = 0.f, sum = 0.f;
    for (int i = 0; i < 128; ++i) {
      x += (__popc(i & t) & 1) ? -sm.q[g][i] : sm.q[g][i];
      sum += sm.p[g][i];
    }
    const float y = sum > 0.f ? (x * kInvSqrt128 + acc[g]) / sum : 0.f;
    a.out[(tok * hq + h * a.group + g) * kD + t] = f2h_bits(y);
  }
}

template <int KB, int VB, bool kLean>
cudaError_t launch_tree_cfg(const TreeArgs& a, cudaStream_t stream) {
  static std::atomic<unsigned long long> smem_set{0};
  cudaError_t err = set_smem_once(tree_kernel<KB, VB, kLean>, sizeof(TreeSmem), smem_set);
  if (err != cudaSuccess) return err;
  tree_kernel<KB, VB, kLean><<<dim3(a.max_tree, a.hkv, a.n_seqs), 128, sizeof(TreeSmem), stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

size_t tree_scratch_bytes(int n_seqs, int hkv, int group, int max_tree) {
  (void)n_seqs; (void)hkv; (void)group; (void)max_tree;
  return 256;
}

cudaError_t launch_tree(const uint16_t* q, const uint16_t* k_new, const uint16_t* v_new, const uint64_t* tree_mask,
                        const int32_t* positions, const int32_t* cu_tokens, const int32_t* seq_lens, int n_seqs,
                        int64_t n_tokens, int max_tree, const int32_t* block_tables, const uint8_t* cache,
                        const uint16_t* ws, int hkv, int group, int max_blocks, int64_t num_blocks, int k_bits,
                        int v_bits, bool lean, const kvarn_score& score, uint16_t* out, void* scratch, unsigned* flags,
                        cudaStream_t stream) {
  (void)scratch;
  TreeArgs a{};
  a.q = q; a.k_new = k_new; a.v_new = v_new;
  a.mask = tree_mask;
  a.positions = positions; a.cu = cu_tokens; a.seq_lens = seq_lens; a.block_tables = block_tables;
  a.cache = cache; a.ws = ws;
  a.slopes = score.slopes;
  a.out = out;
  a.flags = flags;
  a.num_blocks = num_blocks; a.n_tokens = n_tokens;
  a.n_seqs = n_seqs; a.max_tree = max_tree; a.hkv = hkv; a.group = group; a.max_blocks = max_blocks;
  a.window = score.window;
  a.scale = score.scale; a.softcap = score.softcap;
  if (k_bits == 4 && v_bits == 2)
    return lean ? launch_tree_cfg<4, 2, true>(a, stream) : launch_tree_cfg<4, 2, false>(a, stream);
  if (k_bits == 4 && v_bits == 4 && !lean) return launch_tree_cfg<4, 4, false>(a, stream);
  if (k_bits == 2 && v_bits == 2 && !lean) return launch_tree_cfg<2, 2, false>(a, stream);
  return cudaErrorInvalidValue;
}

}  // namespace kvarn

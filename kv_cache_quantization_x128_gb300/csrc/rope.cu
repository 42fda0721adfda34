// Per-head RMS norm of queries and keys and their position rotation in one pass, from
// the rows of a model's projection (fp16, bf16 or fp32, any row stride) to the
// contiguous fp16 rows that the append and attention calls take:
//   x' = x / sqrt(mean(x^2) + eps) * w                 (each head of q and k; optional)
//   (a, b) -> (a cos t - b sin t, b cos t + a sin t),  t = position * inv_freq[i]
// for the pairs of the first rotary_dim channels; v is converted and copied. Everything
// is fp32 and rounded once, on the store.
//
// The angle is exact to the definition at every position: inv_freq / (2 pi) is held as
// a 64-bit fixed-point fraction of a turn F, and position * F modulo 2^64 (one integer
// multiplication) is the fraction of a turn left, so no precision goes into whole turns
// (an fp32 product loses 0.004 rad at position 10^5). F is computed once per block, the
// sines and cosines once per token for all its heads, in shared memory.
//
// Memory bound: a row is read and written once, 16 lanes a row of 128 channels with 16-byte
// accesses, several rows of a thread in flight.
#include <cuda_bf16.h>

#include "kvarn_common.cuh"
#include "kvarn_launch.h"

namespace kvarn {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeRows = kRopeThreads / 16;   // rows of a block at a time
constexpr int kRopeBatch = 4;                  // rows of a thread in flight

struct RopeArgs {
  const void *q, *k, *v, *qw, *kw;
  const float* inv_freq;      // [rotary / 2] or NULL
  const int32_t* positions;   // [n]
  uint16_t *qo, *ko, *vo;
  int64_t qs, ks, vs;         // row strides, elements
  int64_t n;
  int hq, hkv, heads;         // heads: q, k and (unless v is NULL) v heads of a token
  int rotary;
  float eps;
  int tokens, split;          // tokens of a work item; blocks that share a token's heads
};

template <class T>
struct Vec8;   // eight channels of a row
template <>
struct Vec8<__half> {
  uint4 w;
  __device__ void load(const __half* p) { w = *reinterpret_cast<const uint4*>(p); }
  __device__ void get(float (&x)[8]) const {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
};
template <>
struct Vec8<__nv_bfloat16> {
  uint4 w;
  __device__ void load(const __nv_bfloat16* p) { w = *reinterpret_cast<const uint4*>(p); }
  __device__ void get(float (&x)[8]) const {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
  }
};
template <>
struct Vec8<float> {
  float4 a, b;
  __device__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ void get(float (&x)[8]) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
};

// Row of token t, head hh (q heads, then k heads, then v heads), channels 8l..8l+7.
template <class T>
__device__ __forceinline__ const T* rope_src(const RopeArgs& a, int64_t t, int hh, int l) {
  if (hh < a.hq) return static_cast<const T*>(a.q) + t * a.qs + hh * kD + 8 * l;
  if (hh < a.hq + a.hkv) return static_cast<const T*>(a.k) + t * a.ks + (hh - a.hq) * kD + 8 * l;
  return static_cast<const T*>(a.v) + t * a.vs + (hh - a.hq - a.hkv) * kD + 8 * l;
}
__device__ __forceinline__ uint16_t* rope_dst(const RopeArgs& a, int64_t t, int hh, int l) {
  if (hh < a.hq) return a.qo + (t * a.hq + hh) * kD + 8 * l;
  if (hh < a.hq + a.hkv) return a.ko + (t * a.hkv + (hh - a.hq)) * kD + 8 * l;
  return a.vo + (t * a.hkv + (hh - a.hq - a.hkv)) * kD + 8 * l;
}

// Work items are groups of a.tokens tokens; a.split blocks share an item's heads.
template <class T, bool kInter>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs a) {
  __shared__ unsigned long long turn[64];        // inv_freq / (2 pi), 2^64 to a turn
  __shared__ __align__(16) float2 cs[2][4][64];  // (cos, sin) of an item's tokens, double buffered
  const int tid = threadIdx.x, l = tid & 15, row = tid >> 4;
  const int half = a.rotary / 2;
  const bool rotate = a.inv_freq != nullptr;
  if (rotate) {
    if (tid < half) {
      double f = static_cast<double>(a.inv_freq[tid]) * 0.15915494309189535;   // 1 / (2 pi)
      f -= floor(f);
      turn[tid] = f < 1.0 ? static_cast<unsigned long long>(f * 18446744073709551616.0) : 0ull;
    }
    __syncthreads();
  }
  float wq[8], wk[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) wq[i] = wk[i] = 1.f;
  if (a.qw != nullptr) {
    Vec8<T> w;
    w.load(static_cast<const T*>(a.qw) + 8 * l);
    w.get(wq);
  }
  if (a.kw != nullptr) {
    Vec8<T> w;
    w.load(static_cast<const T*>(a.kw) + 8 * l);
    w.get(wk);
  }
  const bool in_rot = rotate && 8 * l < a.rotary;
  const int xl = a.rotary >> 4;                                // lanes between the two halves of a pair
  const bool second = !kInter && in_rot && (l & xl) != 0;
  const int f0 = kInter ? 4 * l : (8 * l) & (half - 1);        // first frequency of this thread's channels

  const int64_t items = (a.n + a.tokens - 1) / a.tokens;
  const int part = blockIdx.x % a.split;
  int buf = 0;
  for (int64_t it = blockIdx.x / a.split; it < items; it += gridDim.x / a.split, buf ^= 1) {
    const int64_t t0 = it * a.tokens;
    const int nt = static_cast<int>(min(static_cast<int64_t>(a.tokens), a.n - t0));
    if (rotate) {
      const int j = tid >> 6, f = tid & 63;
      if (j < nt && f < half) {
        const unsigned long long p =
            static_cast<unsigned long long>(static_cast<long long>(a.positions[t0 + j])) * turn[f];
        float s, c;
        sincospif(static_cast<float>(static_cast<int>(p >> 32)) * 4.656612873077393e-10f, &s, &c);   // 2^-31: half turns
        cs[buf][j][f] = make_float2(c, s);
      }
      __syncthreads();   // the other buffer was read before the previous item's barrier
    }
    for (int j = 0; j < nt; ++j) {
      float co[8], si[8];
      if (in_rot) {
        const float4* p = reinterpret_cast<const float4*>(&cs[buf][j][f0]);
#pragma unroll
        for (int i = 0; i < (kInter ? 2 : 4); ++i) {
          const float4 x = p[i];
          co[2 * i] = x.x; si[2 * i] = x.y; co[2 * i + 1] = x.z; si[2 * i + 1] = x.w;
        }
      }
      // the bound is the same for the whole warp: its two rows shuffle together
      for (int hb = part * kRopeRows; hb < a.heads; hb += kRopeBatch * kRopeRows * a.split) {
        const int h0 = hb + row;
        Vec8<T> in[kRopeBatch];
#pragma unroll
        for (int b = 0; b < kRopeBatch; ++b) {
          const int hh = h0 + b * kRopeRows * a.split;
          if (hh < a.heads) in[b].load(rope_src<T>(a, t0 + j, hh, l));
        }
#pragma unroll
        for (int b = 0; b < kRopeBatch; ++b) {
          const int hh = h0 + b * kRopeRows * a.split;
          const bool live = hh < a.heads;      // the same for a row's 16 lanes
          float x[8];
          if (live) {
            in[b].get(x);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = 0.f;
          }
          const bool is_q = hh < a.hq, is_v = hh >= a.hq + a.hkv;
          if (a.qw != nullptr || a.kw != nullptr) {   // grid-uniform: the shuffles are warp-wide
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (!is_v && (is_q ? a.qw : a.kw) != nullptr) {
              const float inv = rsqrtf(fmaf(ss, 1.f / kD, a.eps));
#pragma unroll
              for (int i = 0; i < 8; ++i) x[i] = x[i] * inv * (is_q ? wq[i] : wk[i]);
            }
          }
          if (rotate) {
            if (kInter) {
              if (in_rot && !is_v) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const float u = x[2 * i], w = x[2 * i + 1];
                  x[2 * i] = u * co[i] - w * si[i];
                  x[2 * i + 1] = w * co[i] + u * si[i];
                }
              }
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float o = __shfl_xor_sync(0xffffffffu, x[i], xl);
                if (in_rot && !is_v) x[i] = second ? x[i] * co[i] + o * si[i] : x[i] * co[i] - o * si[i];
              }
            }
          }
          if (live) {
            uint32_t u[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const __half2 hp = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
              u[i] = *reinterpret_cast<const uint32_t*>(&hp);
            }
            *reinterpret_cast<uint4*>(rope_dst(a, t0 + j, hh, l)) = make_uint4(u[0], u[1], u[2], u[3]);
          }
        }
      }
    }
  }
}

template <class T>
cudaError_t launch_rope_type(const RopeArgs& a, bool interleaved, int64_t grid, cudaStream_t stream) {
  if (interleaved)
    rope_kernel<T, true><<<static_cast<unsigned>(grid), kRopeThreads, 0, stream>>>(a);
  else
    rope_kernel<T, false><<<static_cast<unsigned>(grid), kRopeThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const void* q, const void* k, const void* v, const kvarn_rope* r, const void* qw,
                        const void* kw, const float* inv_freq, const int32_t* positions, int64_t n, int hq, int hkv,
                        uint16_t* qo, uint16_t* ko, uint16_t* vo, cudaStream_t stream) {
  RopeArgs a{};
  a.q = q; a.k = k; a.v = v; a.qw = qw; a.kw = kw;
  a.inv_freq = inv_freq;
  a.positions = positions;
  a.qo = qo; a.ko = ko; a.vo = vo;
  a.qs = r->q_stride; a.ks = r->k_stride; a.vs = r->v_stride;
  a.n = n;
  a.hq = hq; a.hkv = hkv;
  a.heads = hq + hkv + (v != nullptr ? hkv : 0);
  a.rotary = r->rotary_dim;
  a.eps = r->norm_eps;
  int dev = 0, sms = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err == cudaSuccess) err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (err != cudaSuccess) return err;
  // Few tokens: an item is one token, whose heads several blocks share, so that a call of
  // one token keeps more than one SM's loads in flight. Many: four tokens an item (their
  // 256 angles are one a thread), all heads in one block, blocks over items in turn.
  const int64_t passes = (a.heads + kRopeRows - 1) / kRopeRows;
  int64_t grid;
  if (n < 4 * 2 * static_cast<int64_t>(sms)) {
    a.tokens = 1;
    const int64_t split = (2 * static_cast<int64_t>(sms) + n - 1) / n;
    a.split = static_cast<int>(split < passes ? split : passes);
    grid = n * a.split;
  } else {
    a.tokens = 4;
    a.split = 1;
    const int64_t items = (n + 3) / 4;
    grid = 8 * static_cast<int64_t>(sms);
    if (grid > items) grid = items;
  }
  return r->dtype == KVARN_F16    ? launch_rope_type<__half>(a, r->interleaved != 0, grid, stream)
         : r->dtype == KVARN_BF16 ? launch_rope_type<__nv_bfloat16>(a, r->interleaved != 0, grid, stream)
                                  : launch_rope_type<float>(a, r->interleaved != 0, grid, stream);
}

}  // namespace kvarn

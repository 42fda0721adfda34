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
// sines and cosines once per item (a warp's part of a token's heads).
//
// Memory bound: a row is read and written once. Eight lanes take a row, a lane sixteen of its
// channels as two 16-byte accesses, chosen so that both members of a pair are its own and
// a rotation needs no exchange; the norm's sum takes three shuffles for the four rows of a warp.
// 65536 tokens of 64 q-heads over 8 kv-heads, fp16, normed: 456 us, 5.9 TB/s of 2.68 GB (87 % of a
// plain copy's rate); two blocks an SM at 128 registers, three at 80 spill (599 us). fp32 rows: 715 us of 4.03 GB, 83 %,
// with 104 to 128 bytes of spill stores (the 16-bit types have none).
#include <cuda_bf16.h>

#include "kvarn_common.cuh"
#include "kvarn_launch.h"

namespace kvarn {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeWarps = kRopeThreads / 32;

struct RopeArgs {
  const void *q, *k, *v, *qw, *kw;
  const float* inv_freq;      // [rotary / 2] or NULL
  const int32_t* positions;   // [n]
  uint16_t *qo, *ko, *vo;
  int64_t qs, ks, vs;         // row strides, elements
  int64_t n;
  int hq, hkv;
  int rotary;
  float eps;
  int passes[3];              // passes of four rows over the q, k and v heads of a token
  int split;                  // items (of passes) of a token
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

__device__ __forceinline__ void rope_store(uint16_t* dst, const float (&x)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 hp = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t*>(&hp);
  }
  *reinterpret_cast<uint4*>(dst) = make_uint4(u[0], u[1], u[2], u[3]);
}

// Passes [p0, p1) over a token's rows of q or k (head 4 pass + lane / 8): normed with w where it is
// not NULL and, where `turn`, rotated by c (cos, sin of the thread's eight pairs). Channels
// of the thread: 8 from ch0, 8 from ch1; rot0, rot1: whether they are rotated.
template <class T, bool kInter>
__device__ __forceinline__ void rope_rows(const T* src, uint16_t* dst, int heads, int p0, int p1, const float* w, float eps,
                                          bool turn, const float2* c, int ch0, int ch1, bool rot0, bool rot1) {
  constexpr int kBatch = 2;   // passes in flight: 456 us for 65536 tokens of 64 + 8 + 8 rows; 1 548, 4 478 (spills)
  const int row = (threadIdx.x & 31) >> 3;
  // a pair is (xa, xb): channels i of the two groups, or two neighbours of one
  float ca[8], sa[8], cb[8], sb[8];                // w cos, w sin of a pair's members
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const bool rot = i < 4 || !kInter ? rot0 : rot1;
    const float2 t = turn && rot ? c[i] : make_float2(1.f, 0.f);
    float wa = 1.f, wb = 1.f;
    if (w != nullptr) {
      wa = kInter ? w[(i < 4 ? ch0 : ch1) + 2 * (i & 3)] : w[ch0 + i];
      wb = kInter ? w[(i < 4 ? ch0 : ch1) + 2 * (i & 3) + 1] : w[ch1 + i];
    }
    ca[i] = wa * t.x;
    sa[i] = wa * t.y;
    cb[i] = wb * t.x;
    sb[i] = wb * t.y;
  }
  for (int p = p0; p < p1; p += kBatch) {
    Vec8<T> in[kBatch][2];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int h = 4 * (p + b) + row;
      if (p + b < p1 && h < heads) {
        in[b][0].load(src + h * kD + ch0);
        in[b][1].load(src + h * kD + ch1);
      }
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      if (p + b >= p1) break;                      // the same for the warp
      const int h = 4 * (p + b) + row;
      const bool live = h < heads;
      float x[2][8];
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        if (live) {
          in[b][g].get(x[g]);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) x[g][i] = 0.f;
        }
      }
      if (w != nullptr) {
        float2 ss = make_float2(0.f, 0.f);
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            const float2 v = make_float2(x[g][i], x[g][i + 1]);
            ss = __ffma2_rn(v, v, ss);
          }
        float sum = ss.x + ss.y;
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float inv = rsqrtf(fmaf(sum, 1.f / kD, eps));
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
          for (int i = 0; i < 8; ++i) x[g][i] *= inv;
      }
      float y[2][8];
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        float2 ua, ub;                             // members of pairs i, i + 1
        if (kInter) {
          const float* v = x[i >> 2] + 2 * (i & 3);
          ua = make_float2(v[0], v[2]);
          ub = make_float2(v[1], v[3]);
        } else {
          ua = make_float2(x[0][i], x[0][i + 1]);
          ub = make_float2(x[1][i], x[1][i + 1]);
        }
        // (channels that are not rotated take nothing from a neighbour, not even an infinity)
        const bool rot = turn && (i < 4 || !kInter ? rot0 : rot1);
        float2 va = __fmul2_rn(ua, make_float2(ca[i], ca[i + 1])), vb = __fmul2_rn(ub, make_float2(cb[i], cb[i + 1]));
        if (rot) {
          va = __ffma2_rn(ub, make_float2(-sb[i], -sb[i + 1]), va);
          vb = __ffma2_rn(ua, make_float2(sa[i], sa[i + 1]), vb);
        }
        if (kInter) {
          float* v = y[i >> 2] + 2 * (i & 3);
          v[0] = va.x; v[1] = vb.x; v[2] = va.y; v[3] = vb.y;
        } else {
          y[0][i] = va.x; y[0][i + 1] = va.y;
          y[1][i] = vb.x; y[1][i + 1] = vb.y;
        }
      }
      if (live) {
        rope_store(dst + h * kD + ch0, y[0]);
        rope_store(dst + h * kD + ch1, y[1]);
      }
    }
  }
}
// The same passes over a token's rows of v: converted, nothing else.
template <class T>
__device__ __forceinline__ void rope_copy(const T* src, uint16_t* dst, int heads, int p0, int p1, int ch0, int ch1) {
  const int row = (threadIdx.x & 31) >> 3;
#pragma unroll 2
  for (int p = p0; p < p1; ++p) {
    const int h = 4 * p + row;
    if (h >= heads) continue;
    Vec8<T> in[2];
    in[0].load(src + h * kD + ch0);
    in[1].load(src + h * kD + ch1);
    float x[8];
    in[0].get(x);
    rope_store(dst + h * kD + ch0, x);
    in[1].get(x);
    rope_store(dst + h * kD + ch1, x);
  }
}

template <class T, bool kInter>
__global__ void __launch_bounds__(kRopeThreads, 2) rope_kernel(const RopeArgs a) {
  __shared__ unsigned long long turn[64];                      // inv_freq / (2 pi), 2^64 to a turn
  __shared__ float off[64];                                    // 0; NaN where inv_freq is not finite: so are its angles, at any position
  __shared__ __align__(16) float2 cs[kRopeWarps][64];          // (cos, sin) of a warp's token
  __shared__ float ws[2][kD];                                  // norm weights of q and k
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, l = lane & 7;
  const int half = a.rotary / 2;
  const bool rotate = a.inv_freq != nullptr;
  if (rotate && tid < half) {
    double f = static_cast<double>(a.inv_freq[tid]) * 0.15915494309189535;   // 1 / (2 pi)
    off[tid] = static_cast<float>(f - f);
    f -= floor(f);
    turn[tid] = f < 1.0 ? static_cast<unsigned long long>(f * 18446744073709551616.0) : 0ull;
  }
  {
    const T* w = static_cast<const T*>(tid < kD ? a.qw : a.kw);
    if (w != nullptr) ws[tid >> 7][tid & (kD - 1)] = static_cast<float>(w[tid & (kD - 1)]);
  }
  __syncthreads();
  // The thread's channels. Pairs half a rotation apart: lanes below half / 8 take 8 channels and
  // their partners, the others the rest of the row. Neighbouring pairs: any 8 will do.
  const int pairs = rotate ? half >> 3 : 8;
  const bool mine = !kInter && rotate && l < pairs;
  const int ch0 = kInter || !rotate ? 8 * l : mine ? 8 * l : a.rotary + 16 * (l - pairs);
  const int ch1 = kInter || !rotate ? 64 + 8 * l : mine ? 8 * l + half : ch0 + 8;
  const bool rot0 = kInter ? rotate && ch0 < a.rotary : mine, rot1 = kInter ? rotate && ch1 < a.rotary : mine;

  const int passes = a.passes[0] + a.passes[1] + a.passes[2];
  const int64_t items = a.n * a.split;
  for (int64_t it = static_cast<int64_t>(blockIdx.x) * kRopeWarps + warp; it < items; it += static_cast<int64_t>(gridDim.x) * kRopeWarps) {
    int64_t t = it;
    int p0 = 0, p1 = passes;
    if (a.split > 1) {
      t = it / a.split;
      const int part = static_cast<int>(it - t * a.split);
      p0 = part * passes / a.split;
      p1 = (part + 1) * passes / a.split;
    }
    float2 c[8];
    if (rotate) {
      const long long pos = a.positions[t];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int f = lane + 32 * e;
        if (f < half) {
          const unsigned long long p = static_cast<unsigned long long>(pos) * turn[f];
          float sn, cn;
          sincospif(static_cast<float>(static_cast<int>(p >> 32)) * 4.656612873077393e-10f, &sn, &cn);   // 2^-31: half turns
          cs[warp][f] = make_float2(cn + off[f], sn + off[f]);
        }
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int f = kInter ? ((i < 4 ? ch0 : ch1) >> 1) + (i & 3) : ch0 + i;
        c[i] = (i < 4 || !kInter ? rot0 : rot1) ? cs[warp][f] : make_float2(1.f, 0.f);
      }
      __syncwarp();                                // read before the next token's are written
    }
    const int k0 = a.passes[0], v0 = k0 + a.passes[1];
    if (p0 < k0)
      rope_rows<T, kInter>(static_cast<const T*>(a.q) + t * a.qs, a.qo + t * a.hq * kD, a.hq, p0, min(p1, k0),
                           a.qw != nullptr ? ws[0] : nullptr, a.eps, rotate, c, ch0, ch1, rot0, rot1);
    if (p1 > k0 && p0 < v0)
      rope_rows<T, kInter>(static_cast<const T*>(a.k) + t * a.ks, a.ko + t * a.hkv * kD, a.hkv, max(p0 - k0, 0),
                           min(p1, v0) - k0, a.kw != nullptr ? ws[1] : nullptr, a.eps, rotate, c, ch0, ch1, rot0, rot1);
    if (p1 > v0)
      rope_copy<T>(static_cast<const T*>(a.v) + t * a.vs, a.vo + t * a.hkv * kD, a.hkv, max(p0 - v0, 0), p1 - v0, ch0, ch1);
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
  a.rotary = r->rotary_dim;
  a.eps = r->norm_eps;
  int dev = 0, sms = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err == cudaSuccess) err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (err != cudaSuccess) return err;
  a.passes[0] = (hq + 3) / 4;
  a.passes[1] = (hkv + 3) / 4;
  a.passes[2] = v != nullptr ? a.passes[1] : 0;
  // An item is a token and a warp's. Few tokens: their passes are split over several warps, so
  // that a call of one token keeps more than one SM's loads in flight.
  const int64_t warps = 2 * static_cast<int64_t>(sms) * kRopeWarps, passes = a.passes[0] + a.passes[1] + a.passes[2];
  const int64_t split = (warps + n - 1) / n;
  a.split = static_cast<int>(split < passes ? split : passes);
  int64_t grid = (n * a.split + kRopeWarps - 1) / kRopeWarps;
  if (grid > 2 * static_cast<int64_t>(sms)) grid = 2 * static_cast<int64_t>(sms);
  return r->dtype == KVARN_F16    ? launch_rope_type<__half>(a, r->interleaved != 0, grid, stream)
         : r->dtype == KVARN_BF16 ? launch_rope_type<__nv_bfloat16>(a, r->interleaved != 0, grid, stream)
                                  : launch_rope_type<float>(a, r->interleaved != 0, grid, stream);
}

}  // namespace kvarn

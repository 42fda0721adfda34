// Packed codes to fp32 rows in registers: thread t of a tile's 128 decodes token t's 128
// channels (rotated domain), and the 128-point transform between them.
#pragma once
#include <stdint.h>

#include "kvarn_common.cuh"

namespace kvarn {

__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 sub2(float2 a, float2 b) { return __ffma2_rn(b, make_float2(-1.f, -1.f), a); }

// 128-point Walsh-Hadamard transform of x[i >> 1].{x, y} = element i.
__device__ __forceinline__ void fwht128(float2 (&x)[64]) {
#pragma unroll
  for (int i = 0; i < 64; ++i) x[i] = make_float2(x[i].x + x[i].y, x[i].x - x[i].y);
#pragma unroll
  for (int bit = 1; bit < 64; bit <<= 1)
#pragma unroll
    for (int i = 0; i < 64; ++i)
      if ((i & bit) == 0) {
        const float2 u = x[i], w = x[i | bit];
        x[i] = add2(u, w);
        x[i | bit] = sub2(u, w);
      }
}

// A code of kBits bits at bit `at` of w as 1 + code / 2^kBits (the code in the top
// mantissa bits of 1.0f), at most one shift and one logic operation.
template <int kBits>
__device__ __forceinline__ float code_float(uint32_t w, int at) {
  constexpr uint32_t kMask = ((1u << kBits) - 1) << (23 - kBits);
  const int sh = 23 - kBits - at;
  const uint32_t m = sh >= 0 ? w << sh : w >> -sh;
  return __uint_as_float((m & kMask) | 0x3F800000u);
}
// The same for a bit position that a thread knows at run time only: one rotation and one
// logic operation; `turn` is code_turn(at).
template <int kBits>
__device__ __forceinline__ int code_turn(int at) {
  return (at + 32 - (23 - kBits)) & 31;
}
template <int kBits>
__device__ __forceinline__ float code_float_at(uint32_t w, int turn) {
  constexpr uint32_t kMask = ((1u << kBits) - 1) << (23 - kBits);
  return __uint_as_float((__funnelshift_r(w, w, turn) & kMask) | 0x3F800000u);
}

// Token t's K row, before rotation and without c_t: r (code s + z) = f a + b of the
// channel, f = 1 + code / 2^bits (ab: [channel] (a, b)).
template <int KB>
__device__ __forceinline__ void read_keys(const uint8_t* codes, const float2* ab, int t, float2 (&x)[64]) {
  const float4* ab4 = reinterpret_cast<const float4*>(ab);   // channels 2j, 2j + 1
  if (KB == 4) {
    const uint4* row = reinterpret_cast<const uint4*>(codes + t * 64);
    uint32_t w[4][4];
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const uint4 u = row[g];
      w[g][0] = u.x; w[g][1] = u.y; w[g][2] = u.z; w[g][3] = u.w;
    }
#pragma unroll
    for (int j = 0; j < 64; ++j) {
      const int i = 2 * j;
      const uint32_t word = w[(i >> 1) & 3][i >> 5];
      const int p = 4 * ((i >> 3) & 1) + ((i >> 4) & 1);   // bit 0 of the channel adds 2
      const float4 c = ab4[j];
      x[j] = __ffma2_rn(make_float2(code_float<4>(word, 4 * p), code_float<4>(word, 4 * p + 8)),
                        make_float2(c.x, c.z), make_float2(c.y, c.w));
    }
  } else {
    const uint4* row = reinterpret_cast<const uint4*>(codes + t * 32);
    const uint4 u0 = row[0], u1 = row[1];
    const uint32_t w[4][2] = {{u0.x, u0.y}, {u0.z, u0.w}, {u1.x, u1.y}, {u1.z, u1.w}};
#pragma unroll
    for (int j = 0; j < 64; ++j) {
      const int i = 2 * j;
      const uint32_t word = w[(i >> 1) & 3][i >> 6];
      const int p = 4 * ((i >> 4) & 3) + ((i >> 3) & 1);
      const float4 c = ab4[j];
      x[j] = __ffma2_rn(make_float2(code_float<2>(word, 2 * p), code_float<2>(word, 2 * p + 4)),
                        make_float2(c.x, c.z), make_float2(c.y, c.w));
    }
  }
}

// Token t's V row before rotation: r_i (code s_t + z_t) c_t = (f a + b) r_i (r: [channel];
// a, b of the token).
template <int VB>
__device__ __forceinline__ void read_values(const uint8_t* codes, const float* r, float av, float bv, int t,
                                            float2 (&x)[64]) {
  const float2 a2 = make_float2(av, av), b2 = make_float2(bv, bv);
  const float2* r2 = reinterpret_cast<const float2*>(r);
  if (VB == 4) {
    const uint8_t* col = codes + ((t >> 1) & 3) * 16 + (t >> 5) * 4;
    const int turn = code_turn<4>(4 * (4 * ((t >> 3) & 1) + 2 * (t & 1) + ((t >> 4) & 1)));
#pragma unroll
    for (int j = 0; j < 64; ++j) {
      float f[2];
#pragma unroll
      for (int e = 0; e < 2; ++e)
        f[e] = code_float_at<4>(*reinterpret_cast<const uint32_t*>(col + (2 * j + e) * 64), turn);
      x[j] = __fmul2_rn(__ffma2_rn(make_float2(f[0], f[1]), a2, b2), r2[j]);
    }
  } else {
    // channel i: panel i >> 4, cell (i & 7) * 4 + group, 8 bytes for bit 3 of i clear then set
    const uint8_t* col = codes + ((t >> 1) & 3) * 16;
    const bool up = t >= 64;
    const int turn = code_turn<2>(2 * (4 * ((t >> 4) & 3) + 2 * (t & 1) + ((t >> 3) & 1)));
#pragma unroll
    for (int pn = 0; pn < 8; ++pn)
#pragma unroll
      for (int i7 = 0; i7 < 8; i7 += 2) {
        float f[2][2];   // [bit 3][bit 0] of the channel
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint4 u = *reinterpret_cast<const uint4*>(col + pn * 512 + (i7 + e) * 64);
          f[0][e] = code_float_at<2>(up ? u.y : u.x, turn);
          f[1][e] = code_float_at<2>(up ? u.w : u.z, turn);
        }
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const int j = (16 * pn + 8 * b + i7) >> 1;
          x[j] = __fmul2_rn(__ffma2_rn(make_float2(f[b][0], f[b][1]), a2, b2), r2[j]);
        }
      }
  }
}

}  // namespace kvarn

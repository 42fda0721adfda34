// Device code of the decode attention that weighs its tiles (decode_weights.cu): one packed
// tile into a warp's running softmax state of a
// (sequence, kv-head): thread (g, c) = (lane / 4, lane % 4) holds q-head g's running maximum and sum
// (log2 domain) and its outputs of channels 8 n + 2 c + {0, 1}, n = 0..15.
#pragma once
#include <stdint.h>

#include "kvarn_common.cuh"
#include "kvarn_frag.cuh"

namespace kvarn {
namespace {

// Powers of two (up, down = 1 / up) that bring `top` >= 0 into [2^14, 2^15). Exponents stay
// clear of subnormal and infinite factors (top below 2^-112, above 2^102 or not finite).
__device__ __forceinline__ void range_scale(float top, float& up, float& down) {
  const uint32_t e = min(max(__float_as_uint(top) >> 23, 15u), 229u);
  up = __uint_as_float((268u - e) << 23);
  down = __uint_as_float((e - 14u) << 23);
}

__device__ __forceinline__ float abs_max(float m, float2 x) { return fmaxf(fmaxf(m, fabsf(x.x)), fabsf(x.y)); }

// The products of the fp16 pairs a0 b0 and a1 b1 in fp32 (exact), crossed: lo = the low halves' products, hi = the high ones'.
__device__ __forceinline__ void mul_cross(uint32_t a0, uint32_t b0, uint32_t a1, uint32_t b1, float2& lo, float2& hi) {
  asm("{\n .reg .f16 x0, x1, y0, y1, u0, u1, v0, v1;\n"
      " mov.b32 {x0, x1}, %4;\n mov.b32 {y0, y1}, %5;\n mov.b32 {u0, u1}, %6;\n mov.b32 {v0, v1}, %7;\n"
      " fma.rn.f32.f16 %0, x0, y0, 0f00000000;\n fma.rn.f32.f16 %1, u0, v0, 0f00000000;\n"
      " fma.rn.f32.f16 %2, x1, y1, 0f00000000;\n fma.rn.f32.f16 %3, u1, v1, 0f00000000;\n}"
      : "=f"(lo.x), "=f"(lo.y), "=f"(hi.x), "=f"(hi.y)
      : "r"(a0), "r"(b0), "r"(a1), "r"(b1));
}

// d = A B (fp16 in, fp32 out); mma16816 (kvarn_frag.cuh) adds to d.
__device__ __forceinline__ void mma16816_first(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// Codes as operands without a conversion: the bits of two 4-bit codes, masked out of a 32-bit
// word's halves, are the fp16 subnormals code 2^-24, or 16 code 2^-24 from the place above. The
// places' factors are taken out of the other operand, 2^24 out of the result. A word takes 5
// instructions of the ALU pipe instead of 7 with the fp6 conversions of the plain decode; that pipe, the fp32 pipe and the
// tensor core's share an issue path here: together they are busy 100 % of the time.
//
// The tensor core adds products in a window of 24 bits below the largest, which it takes by the
// operands' exponent fields: leading zeros of subnormals cost bits (measured: outputs off by 2.5e-3
// with the other operand split as fp16 rounds it). So the other operand, scaled to 2^15 at most,
// is split on a grid: its hi part is a multiple of 2^4, whose products with codes are multiples
// of 2^-20 below 2^2 in all, sums included, which the window holds exactly; the lo part, up to 2^3, has
// 2^-11 of the window's unit. Together: 2^-24 of a row's largest element.
//
// 4-bit codes only: a word of 2-bit codes saves 2 instructions of 11, less than the grid costs (64 x 16384
// tokens, k4v2: 236 us so, 241 with both masked, 245 with both converted; k2v2 129 either way).
template <int BITS>
struct Masked { static constexpr bool value = BITS == 4; };

// Operand group q = 0..7 of a thread: the rows 16 q + 2 c + {0, 1} (word a) and {8, 9} (word b), channels for keys, tokens
// for values. Converted codes take them in pairs of neighbours, masked ones crossed, (0, 8) and
// (1, 9), which share a mask (groups of even and odd q take turns in a word). The products of the fp16
// words xa ya and xb yb, in the group's pairs:
template <int BITS>
__device__ __forceinline__ void group_mul(uint32_t xa, uint32_t ya, uint32_t xb, uint32_t yb, float2 (&r)[2]) {
  if (Masked<BITS>::value) {
    mul_cross(xa, ya, xb, yb, r[0], r[1]);
  } else {
    r[0] = mul_h2(xa, ya);
    r[1] = mul_h2(xb, yb);
  }
}

// The other operand: E[q] = the group's two pairs, to the hi (rows 0-7) and lo (8-15) parts of both; f takes
// all factors back.
template <int BITS>
__device__ __forceinline__ void make_operand(const float2 (&E)[8][2], float top, float& f, uint32_t (&A)[8][4]) {
  float up, down;
  range_scale(top, up, down);
  f = down * (Masked<BITS>::value ? 16777216.f : BITS == 4 ? 8.f : 2.f);   // (conversions give code / 8 and code / 2)
#pragma unroll
  for (int q = 0; q < 8; ++q)
#pragma unroll
    for (int odd = 0; odd < 2; ++odd) {
      if (!Masked<BITS>::value) {
        split2p(__fmul2_rn(E[q][odd], make_float2(up, up)), A[q][2 * odd], A[q][2 * odd + 1]);
        continue;
      }
      // x up 2^-k, on a grid of 2^(4 - k): adding 1.5 2^(27 - k) rounds to it (odd groups' codes stand 4 bits up)
      const float factor = q & 1 ? 0.0625f : 1.f;
      const float2 s = make_float2(up * factor, up * factor), grid = make_float2(201326592.f * factor, 201326592.f * factor);
      const float2 t = __ffma2_rn(E[q][odd], s, grid);
      const float2 n = __ffma2_rn(t, make_float2(-1.f, -1.f), grid);    // - hi
      const float2 r = __ffma2_rn(E[q][odd], s, n);
      const __half2 hi = __floats2half2_rn(-n.x, -n.y), lo = __floats2half2_rn(r.x, r.y);
      A[q][2 * odd] = *reinterpret_cast<const uint32_t*>(&hi);
      A[q][2 * odd + 1] = *reinterpret_cast<const uint32_t*>(&lo);
    }
}

// The products of one word of codes: word m of four 4-bit ones (two steps), of two 2-bit ones (four).
template <int BITS>
__device__ __forceinline__ void mma_word(float* d, const uint32_t (&A)[8][4], int m, uint32_t w) {
  constexpr int kSteps = 8 / BITS;
  uint32_t b[kSteps][2];
  if constexpr (BITS == 4) {
    const uint32_t h = w >> 8;
    b[0][0] = w & 0x000F000Fu; b[0][1] = h & 0x000F000Fu; b[1][0] = w & 0x00F000F0u; b[1][1] = h & 0x00F000F0u;
  } else {
    uint32_t x[4], y[4];
    cvt2(w & 0x33333333u, x);
    cvt2((w >> 2) & 0x33333333u, y);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      b[i][0] = x[i];
      b[i][1] = y[i];
    }
  }
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    if (m == 0 && i == 0) mma16816_first(d, A[0], b[0][0], b[0][1]);
    else mma16816(d, A[kSteps * m + i], b[i][0], b[i][1]);
  }
}

// The running maximum moves only when a score is 2^8 above it (weights are then up to 2^8, which
// the sums and the scaled operands carry), each head by itself.
__device__ __forceinline__ void raise_max(float tmax, float& m_run, float& l_run, float (&acc)[16][2]) {
  const bool up = tmax > m_run + 8.f;
  if (!__any_sync(0xffffffffu, up)) return;
  const float m_new = up ? tmax : m_run, corr = up ? ex2(m_run - m_new) : 1.f;
  m_run = m_new;
  l_run *= corr;
  const float2 corr2 = make_float2(corr, corr);
#pragma unroll
  for (int n = 0; n < 16; ++n) {
    const float2 v = __fmul2_rn(make_float2(acc[n][0], acc[n][1]), corr2);
    acc[n][0] = v.x;
    acc[n][1] = v.y;
  }
}

// q_r as load_q gives it (channels 16 ks + 2 c + {0, 1, 8, 9}) to the operand groups' order.
template <int KB>
__device__ __forceinline__ void store_q(float4* qsm, const float (&qv)[8][4]) {
#pragma unroll
  for (int q = 0; q < 8; ++q)
    qsm[32 * q] = Masked<KB>::value ? make_float4(qv[q][0], qv[q][2], qv[q][1], qv[q][3])
                                    : make_float4(qv[q][0], qv[q][1], qv[q][2], qv[q][3]);
}

// q' = q_r r s of a head's operand groups, the largest of them, and beta's terms.
template <int KB, class L, bool kLean>
__device__ __forceinline__ void fold_keys(const uint16_t* km, const float4* qsm, int c, float2 (&E)[8][2], float& top, float2& sum2) {
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const int ca = 16 * q + 2 * c, cb = ca + 8;
    const uint32_t ra = kLean ? kH_One : h2raw(km + L::kKr + ca), rb = kLean ? kH_One : h2raw(km + L::kKr + cb);
    float2 rs[2], rz[2];
    group_mul<KB>(ra, h2raw(km + L::kKs + ca), rb, h2raw(km + L::kKs + cb), rs);
    group_mul<KB>(ra, h2raw(km + L::kKz + ca), rb, h2raw(km + L::kKz + cb), rz);
    const float4 qq = qsm[32 * q];
    const float2 q2[2] = {make_float2(qq.x, qq.y), make_float2(qq.z, qq.w)};
#pragma unroll
    for (int odd = 0; odd < 2; ++odd) {
      E[q][odd] = __fmul2_rn(q2[odd], rs[odd]);
      top = abs_max(top, E[q][odd]);
      sum2 = __ffma2_rn(q2[odd], rz[odd], sum2);
    }
  }
}

// One packed tile, rotated domain, in two halves: as
// attend_tile (decode_tile.cuh), but q' and p' on grids (make_operand). The scores, log2 domain, of
// head g and tokens 8 nt + 2 c + {0, 1}; qsm[32 q]: q_r of the thread's operand group q (store_q).
template <int KB, int VB, bool kLean>
__device__ __forceinline__ void weigh_keys(const uint8_t* rec, const float4* qsm, int g, int c, float2 (&sc)[16]) {
  using L = RecordLayout<KB, VB, kLean>;
  const uint16_t* km = reinterpret_cast<const uint16_t*>(rec + L::kKMetaOff);

  float2 E[8][2];
  uint32_t A[8][4];
  float2 sum2 = make_float2(0.f, 0.f);
  float top = 0.f, f;
  fold_keys<KB, L, kLean>(km, qsm, c, E, top, sum2);
  make_operand<KB>(E, quad_max(top), f, A);
  const float beta = quad_sum(sum2.x + sum2.y);
  const float2 beta_2 = make_float2(beta, beta), kf2 = make_float2(f, f);

  // four n-tiles at a time (independent chains)
#pragma unroll
  for (int ntg = 0; ntg < 4; ++ntg) {
    float d[4][4];
    constexpr int kWords = KB;                     // words of a thread and token row: 4 or 2
    uint32_t kw[4][kWords];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint8_t* row = rec + L::kKCodeOff + (8 * (4 * ntg + j) + g) * (16 * KB) + c * (4 * KB);
      if constexpr (KB == 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(row);
        kw[j][0] = v.x; kw[j][1] = v.y; kw[j][2] = v.z; kw[j][3] = v.w;
      } else {
        const uint2 v = *reinterpret_cast<const uint2*>(row);
        kw[j][0] = v.x; kw[j][1] = v.y;
      }
    }
#pragma unroll
    for (int m = 0; m < kWords; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j) mma_word<KB>(d[j], A, m, kw[j][m]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int nt = 4 * ntg + j;
      const float2 ck = h2pair(km + L::kKc + 8 * nt + 2 * c);
      sc[nt] = __fmul2_rn(ck, __ffma2_rn(__fadd2_rn(make_float2(d[j][0], d[j][1]), make_float2(d[j][2], d[j][3])),
                                         kf2, beta_2));
    }
  }

}

// The second half: the running maximum and sum, and the values. stat[g] receives the tile's
// (running maximum, sum of 2^(score - maximum)).
template <int KB, int VB, bool kLean>
__device__ __forceinline__ void weigh_values(const uint8_t* rec, float2 (&sc)[16], int g, int c, float& m_run, float& l_run,
                                             float (&acc)[16][2], float2* stat) {
  using L = RecordLayout<KB, VB, kLean>;
  const uint16_t* vm = reinterpret_cast<const uint16_t*>(rec + L::kVMetaOff);
  float2 E[8][2];
  uint32_t A[8][4];
  float tmax = -INFINITY;
#pragma unroll
  for (int nt = 0; nt < 16; ++nt) tmax = fmax3f(tmax, sc[nt].x, sc[nt].y);
  raise_max(quad_max(tmax), m_run, l_run, acc);
  const float2 mneg = make_float2(-m_run, -m_run);
#pragma unroll
  for (int nt = 0; nt < 16; ++nt) sc[nt] = __fadd2_rn(sc[nt], mneg);
  // p in the values' pairs, their sum; p' and gamma
  float2 lsum2 = make_float2(0.f, 0.f), sum2 = make_float2(0.f, 0.f);
  float top = 0.f, f;
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const float2 pa = make_float2(ex2(sc[2 * q].x), ex2(sc[2 * q].y)), pb = make_float2(ex2(sc[2 * q + 1].x), ex2(sc[2 * q + 1].y));
    const float2 p[2] = {Masked<VB>::value ? make_float2(pa.x, pb.x) : pa, Masked<VB>::value ? make_float2(pa.y, pb.y) : pb};
    const int ta = 16 * q + 2 * c, tb = ta + 8;
    const uint32_t va = kLean ? kH_One : h2raw(vm + L::kVc + ta), vb = kLean ? kH_One : h2raw(vm + L::kVc + tb);
    float2 cs[2], cz[2];
    group_mul<VB>(va, h2raw(vm + L::kVs + ta), vb, h2raw(vm + L::kVs + tb), cs);
    group_mul<VB>(va, h2raw(vm + L::kVz + ta), vb, h2raw(vm + L::kVz + tb), cz);
#pragma unroll
    for (int odd = 0; odd < 2; ++odd) {
      lsum2 = __fadd2_rn(lsum2, p[odd]);
      E[q][odd] = __fmul2_rn(p[odd], cs[odd]);
      top = abs_max(top, E[q][odd]);
      sum2 = __ffma2_rn(p[odd], cz[odd], sum2);
    }
  }
  const float lt = quad_sum(lsum2.x + lsum2.y);
  l_run += lt;
  if (c == 0) stat[g] = make_float2(m_run, lt);
  make_operand<VB>(E, quad_max(top), f, A);
  const float gamma = quad_sum(sum2.x + sum2.y);
  const float2 gamma_2 = make_float2(gamma, gamma), vf2 = make_float2(f, f);

#pragma unroll
  for (int npg = 0; npg < 4; ++npg) {
    float d[4][4];
    constexpr int kWords = VB;
    uint32_t vw[4][kWords];                        // of channels 8 (4 npg + j) + g
    if constexpr (VB == 4) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint4 v = *reinterpret_cast<const uint4*>(rec + L::kVCodeOff + (8 * (4 * npg + j) + g) * 64 + c * 16);
        vw[j][0] = v.x; vw[j][1] = v.y; vw[j][2] = v.z; vw[j][3] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {                // a cell serves channel g of a 16-channel panel and its partner g + 8
        const uint4 v = *reinterpret_cast<const uint4*>(rec + L::kVCodeOff + (2 * npg + i) * 512 + (g * 4 + c) * 16);
        vw[2 * i][0] = v.x; vw[2 * i][1] = v.y; vw[2 * i + 1][0] = v.z; vw[2 * i + 1][1] = v.w;
      }
    }
#pragma unroll
    for (int m = 0; m < kWords; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j) mma_word<VB>(d[j], A, m, vw[j][m]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = 4 * npg + j;
      const float2 rv = h2pair(vm + L::kVr + 8 * n + 2 * c);
      const float2 v = __ffma2_rn(
          rv, __ffma2_rn(__fadd2_rn(make_float2(d[j][0], d[j][1]), make_float2(d[j][2], d[j][3])), vf2, gamma_2),
          make_float2(acc[n][0], acc[n][1]));
      acc[n][0] = v.x;
      acc[n][1] = v.y;
    }
  }
}

// ------------------------------------------------------------------ groups of up to four q-heads
// With four heads, hi and lo parts fill the eight columns of the other operand of the m16n8k16 products:
// codes are A (16 tokens, then 16 channels, a product), columns 0-3 the heads' hi, 4-7 their lo
// parts; half the products of the wide form above. Thread (g, c) folds head g % 4 (as its hi part
// for g < 4, its lo part else), and holds, of heads 2 (c % 2) + {0, 1}: the scores of tokens 16 b + g + 8 (c / 2);
// maximum and sum; and acc[2 n + e] = the part of channel 16 n + 8 e + g that came through hi columns
// (c < 2) or lo columns, added up when the record is written.
// 64 x 16384 tokens, 32 heads over 8: k4v2 175 us (the wide form 234), k4v4 224 (274), k2v2 174 (231).
// Nothing is at its limit: 1793 instructions a tile and kv-head with 2-bit keys, 1796 with 4-bit ones, of which 949 and
// 920 are the ALU pipe's (ncu 61 and 59 % of it; tensor pipe 33, fp32 19 and 20, issue 58), on three warps a scheduler. The
// fold is a part of them that is done twice: lanes g and g + 4 fold the same head, and each keeps one of its parts.

// x of head g % 4, the same in a quad, for the thread's two heads.
__device__ __forceinline__ float2 two_heads(float x, int c) {
  return make_float2(__shfl_sync(0xffffffffu, x, 8 * (c & 1)), __shfl_sync(0xffffffffu, x, 8 * (c & 1) + 4));
}
// Over the lanes that hold tokens of the thread's heads.
__device__ __forceinline__ float2 token_max(float2 x) {
#pragma unroll
  for (int o = 2; o < 32; o <<= 1)
    x = make_float2(fmaxf(x.x, __shfl_xor_sync(0xffffffffu, x.x, o)), fmaxf(x.y, __shfl_xor_sync(0xffffffffu, x.y, o)));
  return x;
}
__device__ __forceinline__ float2 token_sum(float2 x) {
#pragma unroll
  for (int o = 2; o < 32; o <<= 1)
    x = __fadd2_rn(x, make_float2(__shfl_xor_sync(0xffffffffu, x.x, o), __shfl_xor_sync(0xffffffffu, x.y, o)));
  return x;
}
// Product of two fp16 numbers in fp32 (exact).
__device__ __forceinline__ float mul_h(uint16_t a, uint16_t b) {
  float r;
  asm("fma.rn.f32.f16 %0, %1, %2, 0f00000000;" : "=f"(r) : "h"(a), "h"(b));
  return r;
}

// A operands of one word of each of two rows of codes (r: row g, s: row g + 8), and their products.
template <int BITS, bool kMasked>
__device__ __forceinline__ void mma_rows(float* d, const uint32_t (&B)[8][2], int m, uint32_t r, uint32_t s) {
  constexpr int kSteps = 8 / BITS;
  uint32_t a[kSteps][4];
  const uint32_t w[2] = {r, s};
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    if constexpr (kMasked) {
      static_assert(BITS == 4, "see Masked");
      const uint32_t h = w[e] >> 8;
      a[0][e] = w[e] & 0x000F000Fu; a[0][e + 2] = h & 0x000F000Fu; a[1][e] = w[e] & 0x00F000F0u; a[1][e + 2] = h & 0x00F000F0u;
    } else if constexpr (BITS == 4) {
      cvt4(w[e] & 0x0F0F0F0Fu, a[0][e], a[0][e + 2]);
      cvt4((w[e] >> 4) & 0x0F0F0F0Fu, a[1][e], a[1][e + 2]);
    } else {
      uint32_t x[4], y[4];
      cvt2(w[e] & 0x33333333u, x);
      cvt2((w[e] >> 2) & 0x33333333u, y);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i][e] = x[i];
        a[i][e + 2] = y[i];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    if (m == 0 && i == 0) mma16816_first(d, a[0], B[0][0], B[0][1]);
    else mma16816(d, a[i], B[kSteps * m + i][0], B[kSteps * m + i][1]);
  }
}

// The first half: sc[b] = the scores of the thread's two heads and token 16 b + g + 8 (c / 2).
template <int KB, int VB, bool kLean>
__device__ __forceinline__ void narrow_keys(const uint8_t* rec, const float4* qsm, int g, int c, float2 (&sc)[8]) {
  using L = RecordLayout<KB, VB, kLean>;
  const uint16_t* km = reinterpret_cast<const uint16_t*>(rec + L::kKMetaOff);
  uint32_t B[8][2];
  float2 f2, beta2;
  {
    float2 E[8][2], sum2 = make_float2(0.f, 0.f);
    uint32_t A[8][4];
    float top = 0.f, f;
    fold_keys<KB, L, kLean>(km, qsm, c, E, top, sum2);
    make_operand<KB>(E, quad_max(top), f, A);
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      B[q][0] = g < 4 ? A[q][0] : A[q][1];
      B[q][1] = g < 4 ? A[q][2] : A[q][3];
    }
    f2 = two_heads(f, c);
    beta2 = two_heads(quad_sum(sum2.x + sum2.y), c);
  }
  const bool hi = c < 2;
#pragma unroll
  for (int half = 0; half < 2; ++half) {           // four blocks of 16 tokens at a time (independent chains)
    float d[4][4];
    uint32_t kw[4][2][KB];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint8_t* row = rec + L::kKCodeOff + (16 * (4 * half + i) + 8 * e + g) * (16 * KB) + c * (4 * KB);
        if constexpr (KB == 4) {
          const uint4 v = *reinterpret_cast<const uint4*>(row);
          kw[i][e][0] = v.x; kw[i][e][1] = v.y; kw[i][e][2] = v.z; kw[i][e][3] = v.w;
        } else {
          const uint2 v = *reinterpret_cast<const uint2*>(row);
          kw[i][e][0] = v.x; kw[i][e][1] = v.y;
        }
      }
#pragma unroll
    for (int m = 0; m < KB; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) mma_rows<KB, Masked<KB>::value>(d[i], B, m, kw[i][0][m], kw[i][1][m]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int b = 4 * half + i;
      // hi parts stand in lanes c < 2, lo parts two lanes on; each keeps one of the two tokens
      const float2 keep = hi ? make_float2(d[i][0], d[i][1]) : make_float2(d[i][2], d[i][3]);
      const float2 give = hi ? make_float2(d[i][2], d[i][3]) : make_float2(d[i][0], d[i][1]);
      const float2 got = make_float2(__shfl_xor_sync(0xffffffffu, give.x, 2), __shfl_xor_sync(0xffffffffu, give.y, 2));
      const float ck = h2f_bits(km[L::kKc + 16 * b + g + 8 * (c >> 1)]);
      sc[b] = __fmul2_rn(make_float2(ck, ck), __ffma2_rn(__fadd2_rn(keep, got), f2, beta2));
    }
  }
}

// The second half, as weigh_values; m and l of the thread's two heads, stat as there.
template <int KB, int VB, bool kLean>
__device__ __forceinline__ void narrow_values(const uint8_t* rec, float2 (&sc)[8], int g, int c, float2& m_run, float2& l_run,
                                              float (&acc)[16][2], float2* stat) {
  using L = RecordLayout<KB, VB, kLean>;
  const uint16_t* vm = reinterpret_cast<const uint16_t*>(rec + L::kVMetaOff);
  float2 top = sc[0];
#pragma unroll
  for (int b = 1; b < 8; ++b) top = make_float2(fmaxf(top.x, sc[b].x), fmaxf(top.y, sc[b].y));
  top = token_max(top);
  const bool ux = top.x > m_run.x + 8.f, uy = top.y > m_run.y + 8.f;     // (raise_max's rule)
  if (__any_sync(0xffffffffu, ux || uy)) {
    const float2 m_new = make_float2(ux ? top.x : m_run.x, uy ? top.y : m_run.y);
    const float2 corr = make_float2(ux ? ex2(m_run.x - m_new.x) : 1.f, uy ? ex2(m_run.y - m_new.y) : 1.f);
    m_run = m_new;
    l_run = __fmul2_rn(l_run, corr);
#pragma unroll
    for (int n = 0; n < 16; ++n) {
      const float2 v = __fmul2_rn(make_float2(acc[n][0], acc[n][1]), corr);
      acc[n][0] = v.x;
      acc[n][1] = v.y;
    }
  }
  float2 lt = make_float2(0.f, 0.f), sum2 = lt;
  top = lt;
#pragma unroll
  for (int b = 0; b < 8; ++b) {
    const int t = 16 * b + g + 8 * (c >> 1);
    const float2 p = make_float2(ex2(sc[b].x - m_run.x), ex2(sc[b].y - m_run.y));
    const uint16_t vc = kLean ? 0x3C00 : vm[L::kVc + t];
    const float cs = mul_h(vc, vm[L::kVs + t]), cz = mul_h(vc, vm[L::kVz + t]);
    lt = __fadd2_rn(lt, p);
    sum2 = __ffma2_rn(p, make_float2(cz, cz), sum2);
    sc[b] = __fmul2_rn(p, make_float2(cs, cs));
    top = make_float2(fmaxf(top.x, fabsf(sc[b].x)), fmaxf(top.y, fabsf(sc[b].y)));
  }
  lt = token_sum(lt);
  l_run = __fadd2_rn(l_run, lt);
  if (g == 0 && c < 2) *reinterpret_cast<float4*>(stat + 2 * c) = make_float4(m_run.x, lt.x, m_run.y, lt.y);
  top = token_max(top);
  float2 up, f2;
  range_scale(top.x, up.x, f2.x);
  range_scale(top.y, up.y, f2.y);
  constexpr float kf = VB == 4 ? 8.f : 2.f;        // (conversions give code / 8 and code / 2)
  f2 = __fmul2_rn(f2, make_float2(kf, kf));
  const bool hi = c < 2;
  const float2 gamma = token_sum(sum2), g2 = hi ? gamma : make_float2(0.f, 0.f);   // (once: with the hi parts)
  // p' of both heads as one fp16 pair a token; rows of 8 tokens (hi parts in lanes c < 2, lo parts two lanes on), transposed
  uint32_t B[8][2];
#pragma unroll
  for (int b = 0; b < 8; ++b) {
    uint32_t h, l;
    split2p(__fmul2_rn(sc[b], up), h, l);
    const uint32_t got = __shfl_xor_sync(0xffffffffu, hi ? l : h, 2);
    const uint32_t r0 = hi ? h : got, r1 = hi ? got : l;       // tokens 16 b + g and 16 b + 8 + g
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(B[b][0]) : "r"(r0));
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(B[b][1]) : "r"(r1));
  }
#pragma unroll
  for (int half = 0; half < 2; ++half) {           // four blocks of 16 channels at a time
    float d[4][4];
    uint32_t vw[4][2][VB];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = 4 * half + i;
      if constexpr (VB == 4) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint4 v = *reinterpret_cast<const uint4*>(rec + L::kVCodeOff + (16 * n + 8 * e + g) * 64 + c * 16);
          vw[i][e][0] = v.x; vw[i][e][1] = v.y; vw[i][e][2] = v.z; vw[i][e][3] = v.w;
        }
      } else {                                     // a cell serves channel g of a 16-channel panel and its partner g + 8
        const uint4 v = *reinterpret_cast<const uint4*>(rec + L::kVCodeOff + n * 512 + (g * 4 + c) * 16);
        vw[i][0][0] = v.x; vw[i][0][1] = v.y; vw[i][1][0] = v.z; vw[i][1][1] = v.w;
      }
    }
#pragma unroll
    for (int m = 0; m < VB; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) mma_rows<VB, false>(d[i], B, m, vw[i][0][m], vw[i][1][m]);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int n = 2 * (4 * half + i) + e;
        const float r = h2f_bits(vm[L::kVr + 8 * n + g]);
        const float2 v = __ffma2_rn(make_float2(r, r), __ffma2_rn(make_float2(d[i][2 * e], d[i][2 * e + 1]), f2, g2),
                                    make_float2(acc[n][0], acc[n][1]));
        acc[n][0] = v.x;
        acc[n][1] = v.y;
      }
  }
}

// ------------------------------------------------------------------ a warp's state of a unit
// kNarrow: groups of up to four q-heads.
template <bool kNarrow>
struct UnitState;

template <>
struct UnitState<false> {
  float acc[16][2], m, l;
  __device__ __forceinline__ void reset() {
    m = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int n = 0; n < 16; ++n) acc[n][0] = acc[n][1] = 0.f;
  }
  __device__ static __forceinline__ int head(int g) { return g; }          // that the thread folds
  template <int KB, int VB, bool kLean>
  __device__ __forceinline__ void attend(const uint8_t* rec, const float4* qsm, int g, int c, float2* stat) {
    float2 sc[16];
    weigh_keys<KB, VB, kLean>(rec, qsm, g, c, sc);
    weigh_values<KB, VB, kLean>(rec, sc, g, c, m, l, acc, stat);
  }
  // rec: [head][stride]: 128 channels, maximum, sum
  __device__ __forceinline__ void write(float* rec, int stride, int group, int g, int c) {
    if (g >= group) return;
    float* row = rec + g * stride;
#pragma unroll
    for (int n = 0; n < 16; ++n) *reinterpret_cast<float2*>(row + 8 * n + 2 * c) = make_float2(acc[n][0], acc[n][1]);
    if (c == 0) *reinterpret_cast<float2*>(row + 128) = make_float2(m, l);
  }
};

template <>
struct UnitState<true> {
  float acc[16][2];
  float2 m, l;
  __device__ __forceinline__ void reset() {
    m = make_float2(-INFINITY, -INFINITY);
    l = make_float2(0.f, 0.f);
#pragma unroll
    for (int n = 0; n < 16; ++n) acc[n][0] = acc[n][1] = 0.f;
  }
  __device__ static __forceinline__ int head(int g) { return g & 3; }
  template <int KB, int VB, bool kLean>
  __device__ __forceinline__ void attend(const uint8_t* rec, const float4* qsm, int g, int c, float2* stat) {
    float2 sc[8];
    narrow_keys<KB, VB, kLean>(rec, qsm, g, c, sc);
    narrow_values<KB, VB, kLean>(rec, sc, g, c, m, l, acc, stat);
  }
  __device__ __forceinline__ void write(float* rec, int stride, int group, int g, int c) {
#pragma unroll
    for (int n = 0; n < 16; ++n)
#pragma unroll
      for (int k = 0; k < 2; ++k) acc[n][k] += __shfl_xor_sync(0xffffffffu, acc[n][k], 2);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int h = 2 * c + k;
      if (c >= 2 || h >= group) continue;
#pragma unroll
      for (int n = 0; n < 16; ++n) rec[h * stride + 8 * n + g] = acc[n][k];
      if (g == 0) *reinterpret_cast<float2*>(rec + h * stride + 128) = k ? make_float2(m.y, l.y) : make_float2(m.x, l.x);
    }
  }
};

}  // namespace
}  // namespace kvarn

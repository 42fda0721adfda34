// Packed codes of a record as fp16 rows for the tensor core, and the lane that issues its products.
#pragma once
#include <stdint.h>

#include "kvarn_common.cuh"
#include "kvarn_frag.cuh"

namespace kvarn {

// A record's 16-byte parts (keys: of a token; 4-bit values: of a channel; 2-bit values: the
// cells of a channel) hold the elements 16 j + 8 a + 2 c + e in part c. Half h of a team takes
// parts 2h and 2h + 1, so the K index of such an operand is not the element's own but
//   64 (c >> 1) + 8 j + 4 a + 2 (c & 1) + e,
// and the other operand is laid out to match: q' by its writer, p' by the token that a lane
// stands for (code_token is the inverse for tokens).
__device__ __forceinline__ int code_token(int t) {
  return (t & 3) | ((t >> 6) & 1) << 2 | ((t >> 2) & 1) << 3 | ((t >> 3) & 7) << 4;
}
// Row `row` of 64 bytes of 4-bit codes: its parts 2 half, 2 half + 1 as fp16 code / 8, K elements
// 64 half + 32 i .. 64 half + 32 i + 31 to put(i, words). Lanes read their two parts in an order
// of their own, which leaves 2-way bank conflicts of 4-way ones.
template <class Put>
__device__ __forceinline__ void codes4(const uint8_t* codes, int row, int half, Put put) {
  const uint4* p = reinterpret_cast<const uint4*>(codes + row * 64) + 2 * half;
  const bool swap = (row >> 1) & 1;
  const uint4 x = p[swap ? 1 : 0], y = p[swap ? 0 : 1];
  const uint32_t w[2][4] = {{swap ? y.x : x.x, swap ? y.y : x.y, swap ? y.z : x.z, swap ? y.w : x.w},
                            {swap ? x.x : y.x, swap ? x.y : y.y, swap ? x.z : y.z, swap ? x.w : y.w}};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t r[16];
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const uint32_t u = w[c][2 * i + m];
        cvt4(u & 0x0F0F0F0Fu, r[8 * m + c], r[8 * m + 2 + c]);
        cvt4((u >> 4) & 0x0F0F0F0Fu, r[8 * m + 4 + c], r[8 * m + 6 + c]);
      }
    put(i, r);
  }
}
// 2-bit codes [part][word] as fp16 code / 2, the same way.
template <class Put>
__device__ __forceinline__ void codes2(const uint32_t (&w)[2][2], Put put) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t r[16];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      uint32_t v0[4], v1[4];
      cvt2(w[c][i] & 0x33333333u, v0);
      cvt2((w[c][i] >> 2) & 0x33333333u, v1);
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        r[4 * b + c] = v0[b];
        r[4 * b + 2 + c] = v1[b];
      }
    }
    put(i, r);
  }
}
// Key codes of token `tok` over its channels.
template <int KB, class Put>
__device__ __forceinline__ void key_codes(const uint8_t* codes, int tok, int half, Put put) {
  if constexpr (KB == 4) {
    codes4(codes, tok, half, put);
  } else {
    const uint4 v = reinterpret_cast<const uint4*>(codes + tok * 32)[half];
    const uint32_t w[2][2] = {{v.x, v.y}, {v.z, v.w}};
    codes2(w, put);
  }
}
// Value codes of channel t over its tokens.
template <int VB, class Put>
__device__ __forceinline__ void value_codes(const uint8_t* codes, int t, int half, Put put) {
  if constexpr (VB == 4) {
    codes4(codes, t, half, put);
  } else {
    const uint2* p = reinterpret_cast<const uint2*>(codes + (t >> 4) * 512 + (t & 7) * 64 + ((t >> 3) & 1) * 8 + half * 32);
    const bool swap = (t >> 1) & 1;
    const uint2 x = p[swap ? 2 : 0], y = p[swap ? 0 : 2];
    const uint32_t w[2][2] = {{swap ? y.x : x.x, swap ? y.y : x.y}, {swap ? x.x : y.x, swap ? x.y : y.y}};
    codes2(w, put);
  }
}

// One lane of the (converged) warp. Chosen this way, rather than by its number, the compiler
// keeps the operands of the UMMAs it issues in uniform registers: 16 of them (N = 64) take
// 600 cycles from the first to the completion of the last, 1020 otherwise.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}
}  // namespace kvarn

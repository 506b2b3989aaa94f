// Activation checkpoints: 8-bit integers in blocks of 32 along a row with one power of two each
// (MXINT8 of the OCP microscaling formats: scale byte s, value = code 2^(s - 127) / 64).
//
// s is the smallest that brings the block's largest magnitude to at most 127 steps, so a value
// is off by at most half a step, 2^-8 to 2^-7 of the block's largest.  A power of two rather than
// largest / 127: the codes are then the same in any precision that holds the inputs, and a
// decoded value has 7 bits, which BF16 holds exactly, so the backward's matrix products take the
// checkpoint itself and not a second rounding of it.  s = 255 marks a block that held an
// infinity or NaN; it decodes to NaN.  The largest finite FP32 and BF16 values (above 127.5 2^121) are
// stored as 127 2^121.
#pragma once
#include "common.hpp"
#include "reduce.hpp"

namespace moe {

// Scale byte from the largest of the block's magnitude bits (an integer maximum, which keeps a NaN).
__device__ __forceinline__ int int8_scale_byte(uint32_t amax) {
  if (amax >= 0x7f800000u) return 255;
  const int b = (int)(amax >> 23);
  const uint32_t m = amax & 0x7fffffu;
  // 127 / 64 = 1 + 0x7e0000 / 2^23; below 2^-126 the step is 2^-133 (s = 0) up to 127 of those
  if (b == 0) return m > 0x7f0000u ? 1 : 0;
  const int s = b + (m > 0x7e0000u ? 1 : 0);
  return s > 254 ? 254 : s;
}

// the step 2^(s - 133) (NaN for s = 255)
__device__ __forceinline__ float int8_step(int s) {
  return s == 255 ? __builtin_nanf("") : ldexpf(1.0f, s - 133);
}

__device__ __forceinline__ uint32_t abs_bits8(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t u = __float_as_uint(v[i]) & 0x7fffffffu;
    m = u > m ? u : m;
  }
  return m;
}
// largest over the four lanes of a quad
__device__ __forceinline__ uint32_t quad_max_u(uint32_t v) {
  v = max(v, (uint32_t)dpp_i<kDppXor1>((int)v));
  return max(v, (uint32_t)dpp_i<kDppXor2>((int)v));
}

// 8 values of a block with scale byte s -> 8 codes, to nearest, ties to even
__device__ __forceinline__ uint2 int8_codes8(const float (&v)[8], int s) {
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float q = rintf(ldexpf(v[i], 133 - s));
    q = s == 255 ? 0.0f : fminf(fmaxf(q, -127.0f), 127.0f);
    w[i >> 2] |= ((uint32_t)(int)q & 0xffu) << (8 * (i & 3));
  }
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void int8_values8(const uint2& q, float step, float* v) {
  const uint32_t w[2] = {q.x, q.y};
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = (float)((int)(w[i >> 2] << (24 - 8 * (i & 3))) >> 24) * step;
}

}  // namespace moe

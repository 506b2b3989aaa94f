// Values to E4M3 codes with one FP32 scale a block of 128 (along a row, or 128 x 128 tiles):
//   scale = m / 448, code = E4M3(448 v / m) to nearest even, m the block's largest magnitude
// One pass bound by memory: 2 (4) bytes read and 1 written a value (8192 x 7168 BF16 along rows: 38 us, 4.7 TB/s, a large
// copy's 4.9; the transposed form turns codes, not values, through LDS).
//
// The quotient is formed as the formula says, not as v times a rounded 448 / m: products of that
// kind land on either side of a tie by chance, and with BF16 values exact ties are common.
#include <hip/hip_runtime.h>

#include "../../include/moe.h"
#include "fp8.hpp"
#include "host.hpp"
#include "reduce.hpp"

namespace moe {
namespace fp8 {

namespace {

constexpr int kThreads = 256;

// What a block's values are multiplied and divided by.  m and v are brought next to 1 by a power of two
// first (exact for every value that does not round to code 0), so nothing overflows.
struct Divisor {
  float m, r;      // m 2^-e in [1, 2) and about 1 / m
  int e;
  float scale;     // 1 for a block of zeros, NaN for one with an infinity or NaN
  bool live;       // codes are not all 0
};
__device__ __forceinline__ Divisor divisor(uint32_t amax) {
  Divisor d;
  const float m = __uint_as_float(amax);
  d.live = amax != 0 && amax < 0x7f800000u;
  int e;
  d.m = 2.0f * frexpf(d.live ? m : 1.0f, &e);
  d.e = e - 1;
  d.r = __builtin_amdgcn_rcpf(d.m);
  d.scale = amax == 0 ? 1.0f : (d.live ? m / 448.0f : __builtin_nanf(""));
  return d;
}
// 448 v / m, the quotient's remainder folded back in once (r is off by 1 ulp; exact quotients, the
// ties among them, come out exact)
__device__ __forceinline__ float quotient(float v, const Divisor& d) {
  const float x = 448.0f * ldexpf(v, -d.e);
  const float q = x * d.r;
  return d.live ? fmaf(fmaf(-q, d.m, x), d.r, q) : 0.0f;
}
__device__ __forceinline__ uint2 codes8(const float (&v)[8], const Divisor& d) {
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = quotient(v[i], d);
  return make_uint2(pack_e4m3x4(q[0], q[1], q[2], q[3]), pack_e4m3x4(q[4], q[5], q[6], q[7]));
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }
// maximum over a row of 16 lanes
__device__ __forceinline__ uint32_t row16_max_u(uint32_t v) {
  v = max(v, (uint32_t)dpp_i<kDppXor1>((int)v));
  v = max(v, (uint32_t)dpp_i<kDppXor2>((int)v));
  v = max(v, (uint32_t)dpp_i<kDppHalfMirror>((int)v));
  return max(v, (uint32_t)dpp_i<kDppMirror>((int)v));
}

// 8 columns from col on of a row (row < R), zeros past the last
template <bool F32, bool WHOLE>
__device__ __forceinline__ void load8(const QuantArgs& a, int64_t row, int64_t col, float (&v)[8]) {
  const uint8_t* p = a.x + (row * a.ld + col) * (F32 ? 4 : 2);
  if constexpr (WHOLE) {
    if (row < a.R && col < a.C) {
      if constexpr (F32) {
        const f32x4_t x0 = reinterpret_cast<const f32x4_t*>(p)[0], x1 = reinterpret_cast<const f32x4_t*>(p)[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) { v[i] = x0[i]; v[4 + i] = x1[i]; }
      } else {
        unpack_bf16x8(*reinterpret_cast<const uint4*>(p), v);
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = 0.0f;
      if (row < a.R && col + i < a.C)
        v[i] = F32 ? reinterpret_cast<const float*>(p)[i] : bf2f(reinterpret_cast<const uint16_t*>(p)[i]);
    }
  }
}

// Blocks of 128 along a row.  16 lanes hold a block, a wave 512 neighbouring columns; a workgroup
// takes kRows rows a wave.  scales[block][row].
constexpr int kRows = 4;
template <bool F32, bool WHOLE>
__global__ __launch_bounds__(kThreads) void k_fp8_rows(QuantArgs a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t spans = (uint32_t)((a.C + 511) / 512);
  const uint32_t span = blockIdx.x % spans;
  const int64_t row0 = (int64_t)(blockIdx.x / spans) * (4 * kRows) + wave;
  const int64_t col = (int64_t)span * 512 + 8 * lane;
  float v[kRows][8];
#pragma unroll
  for (int u = 0; u < kRows; ++u) load8<F32, WHOLE>(a, row0 + 4 * u, col, v[u]);
#pragma unroll
  for (int u = 0; u < kRows; ++u) {
    const int64_t row = row0 + 4 * u;
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, abs_bits(v[u][i]));
    const Divisor d = divisor(row16_max_u(m));
    if (row >= a.R) continue;
    if (col < a.ldq) *reinterpret_cast<uint2*>(a.codes + row * a.ldq + col) = codes8(v[u], d);
    if ((lane & 15) == 0 && col < a.C) a.scales[(col >> 7) * a.lds + row] = d.scale;
  }
}

// A tile of 128 x 128 a workgroup: thread (g, c) has rows 8 g .. 8 g + 7 of columns 8 c .. 8 c + 7.
//  TILES: one scale a tile, scales[row tile][column tile] (transposed: the other way round);
//  else (TRANSPOSE only): blocks of 128 along a column, scales[row tile][column].
template <bool F32, bool WHOLE, bool TILES, bool TRANSPOSE>
__global__ __launch_bounds__(kThreads) void k_fp8_tile(QuantArgs a) {
  static_assert(TILES || TRANSPOSE, "blocks along a row have a kernel of their own");
  constexpr int kPitch = 128 + 16;       // bytes of a column of codes in LDS, its 16-byte pieces p at p ^ (column / 16)
  __shared__ __align__(16) uint8_t turned[TRANSPOSE ? 128 * kPitch : 16];
  __shared__ uint32_t part[16][TILES ? 1 : 128];
  const int c = threadIdx.x & 15, g = threadIdx.x >> 4;
  const uint32_t ct = (uint32_t)((a.C + 127) / 128);
  const int64_t tr = blockIdx.x / ct, tc = blockIdx.x % ct;
  const int64_t row0 = tr * 128 + 8 * g, col = tc * 128 + 8 * c;
  float v[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) load8<F32, WHOLE>(a, row0 + i, col, v[i]);
  Divisor d[TILES ? 1 : 8];
  if constexpr (TILES) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) m = max(m, abs_bits(v[i][j]));
    m = row16_max_u(m);
    if (c == 0) part[g][0] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 16; ++i) m = max(m, part[i][0]);
    d[0] = divisor(m);
    if (threadIdx.x == 0) a.scales[TRANSPOSE ? tc * a.lds + tr : tr * a.lds + tc] = d[0].scale;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, abs_bits(v[i][j]));
      part[g][8 * c + j] = m;
    }
    __syncthreads();
    if (threadIdx.x < 128) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) m = max(m, part[i][threadIdx.x]);
      part[0][threadIdx.x] = m;
      if (tc * 128 + threadIdx.x < a.C) a.scales[tr * a.lds + tc * 128 + threadIdx.x] = divisor(m).scale;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) d[j] = divisor(part[0][8 * c + j]);
  }
  if constexpr (!TRANSPOSE) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (row0 + i < a.R && col < a.ldq)
        *reinterpret_cast<uint2*>(a.codes + (row0 + i) * a.ldq + col) = codes8(v[i], d[0]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float t[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = v[i][j];
      *reinterpret_cast<uint2*>(turned + (8 * c + j) * kPitch + (((g >> 1) ^ (c >> 1)) << 4) + 8 * (g & 1)) =
          codes8(t, d[TILES ? 0 : j]);
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int piece = u * kThreads + threadIdx.x, j = piece >> 3, k = 16 * (piece & 7);
      if (tc * 128 + j < a.C && tr * 128 + k < a.ldq)
        *reinterpret_cast<uint4*>(a.codes + (tc * 128 + j) * a.ldq + tr * 128 + k) =
            *reinterpret_cast<const uint4*>(turned + j * kPitch + (((piece & 7) ^ (j >> 4)) << 4));
    }
  }
}

int64_t workgroups(int64_t R, int64_t C, bool tile) {
  return tile ? ((R + 127) / 128) * ((C + 127) / 128) : ((R + 4 * kRows - 1) / (4 * kRows)) * ((C + 511) / 512);
}

template <bool F32, bool WHOLE>
void launch_as(hipStream_t st, const QuantArgs& a, bool tiles, bool transpose) {
  const dim3 block(kThreads), grid((unsigned)workgroups(a.R, a.C, tiles || transpose));
  if (!tiles && !transpose) hipLaunchKernelGGL((k_fp8_rows<F32, WHOLE>), grid, block, 0, st, a);
  else if (!tiles) hipLaunchKernelGGL((k_fp8_tile<F32, WHOLE, false, true>), grid, block, 0, st, a);
  else if (transpose) hipLaunchKernelGGL((k_fp8_tile<F32, WHOLE, true, true>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((k_fp8_tile<F32, WHOLE, true, false>), grid, block, 0, st, a);
}

}  // namespace

void launch_quantize(hipStream_t st, const QuantArgs& a, bool fp32, bool tiles, bool transpose) {
  const bool whole = a.C % 8 == 0 && (a.ld * (fp32 ? 4 : 2)) % 16 == 0 && aligned16(a.x);
  if (fp32) {
    if (whole) launch_as<true, true>(st, a, tiles, transpose);
    else launch_as<true, false>(st, a, tiles, transpose);
  } else {
    if (whole) launch_as<false, true>(st, a, tiles, transpose);
    else launch_as<false, false>(st, a, tiles, transpose);
  }
}

}  // namespace fp8
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_block_quantize(const moe_block_quantize_problem* p, const moe_rows* x, void* codes,
                                       float* scales, void* stream) {
  if (!p) return MOE_ERR_NULL;
  if (p->rows < 0 || p->rows > (1ll << 31) || p->cols < 1 || p->cols > (1 << 24)) return MOE_ERR_SHAPE;
  if (p->kind != MOE_FP8_ROWS && p->kind != MOE_FP8_TILES) return MOE_ERR_UNSUPPORTED;
  if (p->dtype != MOE_BF16 && p->dtype != MOE_FP32) return MOE_ERR_DTYPE;
  if (p->flags & ~MOE_FP8_TRANSPOSE) return MOE_ERR_UNSUPPORTED;
  const bool tiles = p->kind == MOE_FP8_TILES, turn = (p->flags & MOE_FP8_TRANSPOSE) != 0;
  if (fp8::workgroups(p->rows, p->cols, tiles || turn) >= (1ll << 32) / fp8::kThreads) return MOE_ERR_SHAPE;
  if (p->rows == 0) return MOE_OK;
  if (!x || !x->base || !codes || !scales) return MOE_ERR_NULL;
  if (x->ld < p->cols || !elem_aligned(x->base, p->dtype) || !aligned16(codes) || !aligned4(scales)) return MOE_ERR_LAYOUT;
  const int64_t R = p->rows, C = p->cols, up16 = ((turn ? R : C) + 15) / 16 * 16;
  const int64_t lds = tiles ? ((turn ? R : C) + 127) / 128 : (turn ? C : R);
  const fp8::QuantArgs a{static_cast<const uint8_t*>(x->base), x->ld, R, C, static_cast<uint8_t*>(codes), up16, scales, lds};
  hipStream_t st = static_cast<hipStream_t>(stream);
  return launch("block_quantize", st, [&] { fp8::launch_quantize(st, a, p->dtype == MOE_FP32, tiles, turn); });
}

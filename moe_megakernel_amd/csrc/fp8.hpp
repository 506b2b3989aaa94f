// 8-bit matrix products with a scale for each block of 128: arguments and launchers.
#pragma once
#include "common.hpp"

namespace moe {
namespace fp8 {

constexpr int kMaxGroups = 256;            // MOE_FP8_MAX_GROUPS

struct QuantArgs {
  const uint8_t* x;       // [R][C] BF16 or FP32, rows ld elements apart
  int64_t ld;
  int64_t R, C;
  uint8_t* codes;         // [R][Cp], or transposed [C][Rp]; padded to multiples of 16
  int64_t ldq;
  float* scales;          // see moe_block_quantize
  int64_t lds;            // floats between rows of the scales
};
void launch_quantize(hipStream_t st, const QuantArgs& a, bool fp32, bool tiles, bool transpose);

struct MatmulArgs {
  const uint8_t* a;       // [M][K] codes, rows lda bytes apart
  const float* sa;        // [K / 128][M]
  const uint8_t* b;       // [G][N][K] codes
  const float* sb;        // tiles: [G][N / 128][K / 128]; rows: [K / 128][N]
  uint8_t* out;           // [M][N]
  const int32_t* offsets; // [G + 1], or null: one group of M rows
  int64_t lda, ldb, stride_b, ldo;
  int M, N, K, G;
  int out_fp32, accumulate, rows_b;
};
void launch_matmul(hipStream_t st, const MatmulArgs& a);
constexpr int kFewRows = 64;               // in all groups together
void launch_few(hipStream_t st, const MatmulArgs& a);

}  // namespace fp8
}  // namespace moe

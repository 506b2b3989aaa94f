// 8-bit products with a scale for each block of 128 for a few rows in all (serving): one read of the
// weights of the groups that have rows (stream.hpp).  A workgroup takes 16 columns of the result of one
// group; its waves share the contraction, a stage is a block of 128.  The weights' bytes bound it, so BF16 results take the
// BF16 instruction too, whose sums are FP32 ones (fp8_wide.hpp): 19 x 7168 over 2048 8.3 us, with the 8-bit instruction 8.0;
// 64 x 4096 over 7168 16.3, 15.2; 64 rows in 32 groups, 2048 over 4096 66.8, 64.8.
#include <hip/hip_runtime.h>

#include "fp8.hpp"
#include "fp8_wide.hpp"
#include "stream.hpp"

namespace moe {
namespace fp8 {

using namespace gemm;

namespace {

constexpr int kWaves = 8;

// Rows m0 .. m0 + rows - 1 (rows <= 16 NF) of group g, columns n0 .. n0 + 15.
template <bool ROWS_B, bool F32, bool ADD, int NF, int D>
__device__ __forceinline__ void few(const MatmulArgs& p, uint8_t* lds, int g, int m0, int rows, int n0) {
  constexpr int W = kWaves, EX = 2;
  using G = stream::Ring<1, NF, EX, D>;
  const int lane = threadIdx.x & 63, r16 = lane & 15, q4 = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kb = (p.K + 127) / 128, s0 = wave * kb / W, s1 = (wave + 1) * kb / W;
  const int cols = min(16, p.N - n0);
  const uint8_t* b = p.b + (int64_t)g * p.stride_b + (int64_t)n0 * p.ldb;
  const uint8_t* a = p.a + (int64_t)m0 * p.lda;
  auto w = [&](int r) { return r < cols ? b + (int64_t)r * p.ldb : nullptr; };
  auto x = [&](int c) { return c < rows ? a + (int64_t)c * p.lda : nullptr; };
  const float* sb = ROWS_B ? p.sb + n0 : p.sb + ((int64_t)g * ((p.N + 127) / 128) + n0 / 128) * kb;
  // a stage's scales: of the tokens, then of the weights' rows or (word 0) their tile
  auto ex = [&](int e, int s) __attribute__((always_inline)) {
    const void* z = reinterpret_cast<const uint8_t*>(g_zero_page) + 4 * lane;
    if (e == 0) return lane < rows ? (const void*)(p.sa + (int64_t)s * p.M + m0 + lane) : z;
    if (ROWS_B) return lane < cols ? (const void*)(sb + (int64_t)s * p.N + lane) : z;
    return lane == 0 ? (const void*)(sb + s) : z;
  };
  f32x4_t acc[NF] = {};
  stream::run<1, NF, EX, D>(lds + wave * G::kBytes, s0, s1 - s0, p.K, w, x, ex,
                            [&](const uint8_t* wt, const uint8_t* xt, const float* sc) {
    auto frag = [&](const uint8_t* t) __attribute__((always_inline)) {
      const u32x4_t u0 = *reinterpret_cast<const u32x4_t*>(stream::chunk(t, r16, q4));
      const u32x4_t u1 = *reinterpret_cast<const u32x4_t*>(stream::chunk(t, r16, q4 + 4));
      return i32x8_t{(int)u0[0], (int)u0[1], (int)u0[2], (int)u0[3], (int)u1[0], (int)u1[1], (int)u1[2], (int)u1[3]};
    };
    const Wide wf = widen(frag(wt));
    const f32x4_t sw = ROWS_B ? *reinterpret_cast<const f32x4_t*>(sc + 64 + 4 * q4)
                              : f32x4_t{sc[64], sc[64], sc[64], sc[64]};
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      const f32x4_t d = wide_product(wf, widen(frag(xt + f * stream::kTile)));
      const float s = sc[16 * f + r16];
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[f][e] += s * sw[e] * d[e];
    }
  });
  // the waves' sums, [token][16], over the rings
  float* red = reinterpret_cast<float*>(lds);
  __syncthreads();
#pragma unroll
  for (int f = 0; f < NF; ++f)
    *reinterpret_cast<f32x4_t*>(red + ((wave * NF + f) * 16 + r16) * 16 + 4 * q4) = acc[f];
  __syncthreads();
  for (int o = threadIdx.x; o < rows * 16; o += 64 * W) {
    const int t = o >> 4, n = o & 15;
    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < W; ++k) v += red[(k * NF * 16 + t) * 16 + n];
    if (n >= cols) continue;
    const int64_t at = (int64_t)(m0 + t) * p.ldo + n0 + n;
    if constexpr (F32) {
      float* to = reinterpret_cast<float*>(p.out) + at;
      *to = ADD ? *to + v : v;
    } else {
      uint16_t* to = reinterpret_cast<uint16_t*>(p.out) + at;
      const uint32_t z = f2bf(v);
      *to = (uint16_t)(ADD ? f2bf(bf2f(*to) + bf2f(z)) : z);
    }
  }
}

template <bool ROWS_B, bool F32, bool ADD>
__global__ __launch_bounds__(64 * kWaves) void k_fp8_few(MatmulArgs p) {
  constexpr int ring1 = kWaves * stream::Ring<1, 1, 2, 3>::kBytes, ring2 = kWaves * stream::Ring<1, 2, 2, 2>::kBytes;
  __shared__ __align__(16) uint8_t lds[ring1 > ring2 ? ring1 : ring2];
  const int g = blockIdx.y, n0 = blockIdx.x * 16;
  int m0 = 0, rows = p.M;
  if (p.offsets) {
    m0 = min(max(p.offsets[g], 0), p.M);
    rows = min(max(p.offsets[g + 1], 0), p.M) - m0;
  }
  for (int done = 0; done < rows; done += 32) {   // more than 32 rows: the weights again, from the caches
    if (done) __syncthreads();
    const int n = min(32, rows - done);
    if (n <= 16) few<ROWS_B, F32, ADD, 1, 3>(p, lds, g, m0 + done, n, n0);
    else few<ROWS_B, F32, ADD, 2, 2>(p, lds, g, m0 + done, n, n0);
  }
}

template <bool ROWS_B, bool F32>
void launch_as(hipStream_t st, const MatmulArgs& a) {
  const dim3 grid((unsigned)((a.N + 15) / 16), (unsigned)(a.offsets ? a.G : 1)), block(64 * kWaves);
  if (a.accumulate) hipLaunchKernelGGL((k_fp8_few<ROWS_B, F32, true>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((k_fp8_few<ROWS_B, F32, false>), grid, block, 0, st, a);
}

}  // namespace

void launch_few(hipStream_t st, const MatmulArgs& a) {
  if (a.rows_b) {
    if (a.out_fp32) launch_as<true, true>(st, a);
    else launch_as<true, false>(st, a);
  } else {
    if (a.out_fp32) launch_as<false, true>(st, a);
    else launch_as<false, false>(st, a);
  }
}

}  // namespace fp8
}  // namespace moe

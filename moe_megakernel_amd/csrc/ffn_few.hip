// The gated feed-forward block for a few tokens (serving): two kernels built around one read of the
// weights (stream.hpp).
//
//   k_few_up    h = act(a) b, a and b kept in BF16 where asked for: a fragment of 16 rows is 8 gate and
//               8 up rows in turn, so a pair ends in neighbouring results of a lane
//   k_few_down  out = h down^T
// h goes between them in two BF16 parts, its rounding and what that left, 16 of its 24 bits, so that nothing but the output is
// rounded to BF16: one part would be off by as much as the output's own rounding (0.235% of the output's size against 64
// bits, 0.166% with two).  Rows of the second part lie T rows after the first's.  What that costs is the second read of h: whole
// forwards, one part and two, 1 token, H 4096, I 1024 10.5 and 10.5 us; 13, H 4096, I 12288 57.7 and 63.1; 37, H 7168,
// I 2048 28.7 and 31.9; 64, H 4096, I 4096 32.1 and 36.5; 64, H 4096, I 12288 86.9 and 91.5.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "ffn.hpp"
#include "ffn_act.hpp"
#include "stream.hpp"

namespace moe {
namespace ffn {

using namespace gemm;

namespace {

// acc[g][f] += 16 rows of weight tile g times 16 tokens of the P tiles from P f, one stage (64 elements)
template <int R, int NF, int P = 1>
__device__ __forceinline__ void stage(const uint8_t* w, const uint8_t* x, f32x4_t (&acc)[R][NF]) {
  const int lane = threadIdx.x & 63, row = lane & 15, q = lane >> 4;
#pragma unroll
  for (int ks = 0; ks < 2; ++ks) {
    bf16x8_t b[NF * P];
#pragma unroll
    for (int f = 0; f < NF * P; ++f)
      b[f] = *reinterpret_cast<const bf16x8_t*>(stream::chunk(x + f * stream::kTile, row, 4 * ks + q));
#pragma unroll
    for (int g = 0; g < R; ++g) {
      const bf16x8_t a = *reinterpret_cast<const bf16x8_t*>(stream::chunk(w + g * stream::kTile, row, 4 * ks + q));
#pragma unroll
      for (int f = 0; f < NF * P; ++f)
        acc[g][f / P] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b[f], acc[g][f / P], 0, 0, 0);
    }
  }
}

// Sums of the waves: each leaves its own, [token][16 R] floats, over its ring; then f(token, row, v) of two
// neighbouring rows.  FOLD: columns 8 to 15 are the second parts of columns 0 to 7.
template <int R, int NF, int W, bool FOLD, class F>
__device__ __forceinline__ void join(const f32x4_t (&acc)[R][NF], uint8_t* lds, int T, const F& f) {
  constexpr int ROWS = 16 * R;
  float* red = reinterpret_cast<float*>(lds);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  __syncthreads();
#pragma unroll
  for (int g = 0; g < R; ++g)
#pragma unroll
    for (int u = 0; u < NF; ++u)
      *reinterpret_cast<f32x4_t*>(red + ((wave * NF + u) * 16 + (lane & 15)) * ROWS + 16 * g + 4 * (lane >> 4)) = acc[g][u];
  __syncthreads();
  for (int o = threadIdx.x; o < T * (ROWS / 2); o += 64 * W) {
    const int t = o / (ROWS / 2), row = 2 * (o % (ROWS / 2));
    float2 v = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < W; ++k) {
      const float2 z = *reinterpret_cast<const float2*>(red + (k * NF * 16 + t) * ROWS + row);
      v.x += z.x;
      v.y += z.y;
      if constexpr (FOLD) {
        const float2 z2 = *reinterpret_cast<const float2*>(red + (k * NF * 16 + t + 8) * ROWS + row);
        v.x += z2.x;
        v.y += z2.y;
      }
    }
    f(t, row, v);
  }
}

template <int R, int NF, int W, int D, int P = 1>
constexpr int lds_bytes() {
  constexpr int ring = W * stream::Ring<R, NF * P, 0, D>::kBytes, sums = W * NF * 16 * 16 * R * 4;
  return ring > sums ? ring : sums;
}

template <int ACT, int R, int NF, int W, int D>
__global__ __launch_bounds__(64 * W) void k_few_up(UpArgs p) {
  __shared__ __align__(16) uint8_t lds[lds_bytes<R, NF, W, D>()];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), i0 = blockIdx.x * 8 * R;
  const int S = p.H / 64, s0 = wave * S / W, s1 = (wave + 1) * S / W;
  f32x4_t acc[R][NF] = {};
  auto w = [&](int r) {
    const int64_t i = min(i0 + (r >> 1), p.I - 1);
    return reinterpret_cast<const uint8_t*>(r & 1 ? p.up.p + i * p.up.ld : p.gate.p + i * p.gate.ld);
  };
  auto x = [&](int c) { return c < p.T ? reinterpret_cast<const uint8_t*>(p.x.p + (int64_t)c * p.x.ld) : nullptr; };
  stream::run<R, NF, 0, D>(lds + wave * stream::Ring<R, NF, 0, D>::kBytes, s0, s1 - s0, 2 * (int64_t)p.H, w, x,
                           [](int, int) { return (const void*)nullptr; },
                           [&](const uint8_t* wt, const uint8_t* xt, const float*) { stage<R, NF>(wt, xt, acc); });
  join<R, NF, W, false>(acc, lds, p.T, [&](int t, int row, float2 v) {
    const int i = i0 + row / 2;
    if (i >= p.I) return;
    const float h = act<ACT>(v.x) * v.y, upper = bf2f(f2bf(h));
    p.h.p[(int64_t)t * p.h.ld + i] = (uint16_t)f2bf(h);
    p.h.p[(int64_t)(p.T + t) * p.h.ld + i] = (uint16_t)(fabsf(upper) < __builtin_inff() ? f2bf(h - upper) : 0);   // (not of inf, NaN)
    if (p.saved == kBf16) {
      uint16_t* ab = reinterpret_cast<uint16_t*>(p.kept.ab) + (int64_t)t * 2 * p.I + i;
      ab[0] = (uint16_t)f2bf(v.x);
      ab[p.I] = (uint16_t)f2bf(v.y);
    }
  });
}

// A contraction split over grid rows leaves its sums for k_ffn_rows_sum, as over many tokens.
// P = 1: up to 8 tokens, both parts of h in one tile (the parts' sums meet at the end); P = 2: a tile each
template <int R, int NF, int W, int D, int P>
__global__ __launch_bounds__(64 * W) void k_few_down(RowsArgs p) {
  static_assert(P == 2 || NF == 1, "8 tokens a tile");
  __shared__ __align__(16) uint8_t lds[lds_bytes<R, NF, W, D, P>()];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n0 = blockIdx.x * 16 * R;
  const int parts = p.plan.split.n, part = blockIdx.y, S = p.K / 64;
  const int s0 = (part * W + wave) * S / (parts * W), s1 = (part * W + wave + 1) * S / (parts * W);
  f32x4_t acc[R][NF] = {};
  auto w = [&](int r) { return reinterpret_cast<const uint8_t*>(p.b0.p + (int64_t)min(n0 + r, p.N - 1) * p.b0.ld); };
  auto x = [&](int c) {
    const int t = P == 1 ? c & 7 : (c >> 5) * 16 + (c & 15), part = P == 1 ? c >> 3 : (c >> 4) & 1;
    return t < p.T ? reinterpret_cast<const uint8_t*>(p.a.p + (int64_t)(part * p.T + t) * p.a.ld) : nullptr;
  };
  using G = stream::Ring<R, NF * P, 0, D>;
  stream::run<R, NF * P, 0, D>(lds + wave * G::kBytes, s0, s1 - s0, 2 * (int64_t)p.K, w, x,
                               [](int, int) { return (const void*)nullptr; },
                               [&](const uint8_t* wt, const uint8_t* xt, const float*) { stage<R, NF, P>(wt, xt, acc); });
  join<R, NF, W, P == 1>(acc, lds, p.T, [&](int t, int row, float2 v) {
    const int n = n0 + row;                // N is a multiple of 64
    if (n >= p.N) return;
    if (parts > 1) *reinterpret_cast<float2*>(p.plan.split.sums + ((int64_t)part * p.T + t) * p.N + n) = v;
    else *reinterpret_cast<uint32_t*>(p.c.p + (int64_t)t * p.c.ld + n) = pack_bf2(v.x, v.y);
  });
}

template <int R, int NF, int W, int D>
void up_as(hipStream_t st, const UpArgs& a) {
  const dim3 grid((unsigned)((a.I + 8 * R - 1) / (8 * R))), block(64 * W);
  if (a.act == kSilu) hipLaunchKernelGGL((k_few_up<kSilu, R, NF, W, D>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((k_few_up<kGelu, R, NF, W, D>), grid, block, 0, st, a);
}
template <int R, int NF, int W, int D, int P>
void down_as(hipStream_t st, const RowsArgs& a) {
  const dim3 grid((unsigned)((a.N + 16 * R - 1) / (16 * R)), (unsigned)a.plan.split.n), block(64 * W);
  hipLaunchKernelGGL((k_few_down<R, NF, W, D, P>), grid, block, 0, st, a);
}

// The first kernel: f(fragments a workgroup, token tiles, waves, stages in flight).  Two fragments share the tokens' copies, which
// pays where one would leave more workgroups than CUs anyway (T > 32: 48 tokens, H 4096, I 12288 45 us against 67; but 37 of
// I 2048, 256 workgroups, 16 against 15.4) or, with two token tiles, many more (24 tokens, H 4096, I 12288 39 us
// against 47).  Four waves and two stages in flight leave room for two workgroups a CU; one token tile is so small that eight
// waves do (13 tokens, H 4096, I 12288, with both kernels so and h in one part: 57 us, 64 with four stages).
template <class F>
void by_tokens(int T, int64_t frags, const F& f) {
  using std::integral_constant;
  constexpr integral_constant<int, 1> c1{};
  constexpr integral_constant<int, 2> c2{};
  constexpr integral_constant<int, 3> c3{};
  constexpr integral_constant<int, 4> c4{};
  constexpr integral_constant<int, 8> c8{};
  if (T <= 16) f(c1, c1, c8, c2);
  else if (T <= 32) frags > 512 ? f(c2, c2, c4, c2) : f(c1, c2, c4, c3);
  else if (T <= 48) frags > 256 ? f(c2, c3, c4, c2) : f(c1, c3, c8, c2);
  else frags > 256 ? f(c2, c4, c4, c2) : f(c1, c4, c4, c2);
}

}  // namespace

void launch_up_few(hipStream_t st, const UpArgs& a) {
  by_tokens(a.T, a.I / 8, [&](auto r, auto nf, auto w, auto d) {
    up_as<decltype(r)::value, decltype(nf)::value, decltype(w)::value, decltype(d)::value>(st, a);
  });
}
// The second kernel's tokens come twice (both parts of h) and with every weight tile, from L2, so two fragments share them as
// soon as that leaves a workgroup for most CUs (whole forwards: 32 tokens, H 7168, I 2048 27.4 us against 31.5, 16 of H 5120,
// I 4096 32.2 against 35.3, 64 of H 6144, I 1024 28.4 against 33.0); up to 8 tokens are too few to share (1 of H 7168, I 2048 19.8
// against 19.4).  With fewer weight tiles and a long contraction, parts of that fill the CUs: 24 tokens, H 4096, I 12288
// 67 us, 73 with one fragment a workgroup and no parts; 64 of H 4096, I 4096 36.7, 39.8; 34 of H 2112, I 9024 42.4, 57.5; 60
// of H 1024, I 2816 19.1, 24.1; 64 of H 1024, I 2048 16.7, 18.9; but 20 of that 12.4, 12.1, 21 of H 1216, I 1664 12.8, 12.2,
// and 13 of H 4096, I 12288 62.3, 62.8.  Three stages in flight where there is room (13 of H 4096, I 12288 62.8, 64.3 with two).
int few_parts(int T, int N, int K) {
  const int frags = N / 16;
  return T > 16 && frags <= 256 && K >= 2048 ? std::min(512 / frags, std::min(K / 256, 16)) : 1;
}
void launch_down_few(hipStream_t st, const RowsArgs& a) {
  const int T = a.T;
  const bool two = a.N / 16 > 256 || a.plan.split.n > 1;
  if (T <= 8) down_as<1, 1, 4, 3, 1>(st, a);
  else if (T <= 16) two ? down_as<2, 1, 4, 2, 2>(st, a) : down_as<1, 1, 4, 3, 2>(st, a);
  else if (T <= 32) two ? down_as<2, 2, 4, 2, 2>(st, a) : down_as<1, 2, 4, 3, 2>(st, a);
  else if (T <= 48) two ? down_as<2, 3, 4, 2, 2>(st, a) : down_as<1, 3, 4, 2, 2>(st, a);
  else two ? down_as<2, 4, 4, 2, 2>(st, a) : down_as<1, 4, 4, 2, 2>(st, a);
}

}  // namespace ffn
}  // namespace moe

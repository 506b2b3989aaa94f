// The gated feed-forward block for a few tokens (serving): two kernels built around one read of the
// weights (stream.hpp).
//
//   k_few_up    h = act(a) b, a and b kept in BF16 where asked for: a fragment of 16 rows is 8 gate and
//               8 up rows in turn, so a pair ends in neighbouring results of a lane
//   k_few_down  out = h down^T
// h is rounded to BF16 between them, as over many tokens.  (34 tokens, H 2112, I 9024, a and b kept: 32 us, 44 in the
// tiles of many tokens; 21, H 1216, I 1664: 11 and 18.)
#include <hip/hip_runtime.h>

#include "ffn.hpp"
#include "ffn_act.hpp"
#include "stream.hpp"

namespace moe {
namespace ffn {

using namespace gemm;

namespace {

// acc[g][f] += 16 rows of weight tile g times 16 tokens of tile f, one stage (64 elements)
template <int R, int NF>
__device__ __forceinline__ void stage(const uint8_t* w, const uint8_t* x, f32x4_t (&acc)[R][NF]) {
  const int lane = threadIdx.x & 63, row = lane & 15, q = lane >> 4;
#pragma unroll
  for (int ks = 0; ks < 2; ++ks) {
    bf16x8_t b[NF];
#pragma unroll
    for (int f = 0; f < NF; ++f)
      b[f] = *reinterpret_cast<const bf16x8_t*>(stream::chunk(x + f * stream::kTile, row, 4 * ks + q));
#pragma unroll
    for (int g = 0; g < R; ++g) {
      const bf16x8_t a = *reinterpret_cast<const bf16x8_t*>(stream::chunk(w + g * stream::kTile, row, 4 * ks + q));
#pragma unroll
      for (int f = 0; f < NF; ++f) acc[g][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b[f], acc[g][f], 0, 0, 0);
    }
  }
}

// Sums of the waves: each leaves its own, [token][16 R] floats, over its ring; then f(token, row, v) of two
// neighbouring rows.
template <int R, int NF, int W, class F>
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
    }
    f(t, row, v);
  }
}

template <int R, int NF, int W, int D>
constexpr int lds_bytes() {
  constexpr int ring = W * stream::Ring<R, NF, 0, D>::kBytes, sums = W * NF * 16 * 16 * R * 4;
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
  join<R, NF, W>(acc, lds, p.T, [&](int t, int row, float2 v) {
    const int i = i0 + row / 2;
    if (i >= p.I) return;
    p.h.p[(int64_t)t * p.h.ld + i] = (uint16_t)f2bf(act<ACT>(v.x) * v.y);
    if (p.saved == kBf16) {
      uint16_t* ab = reinterpret_cast<uint16_t*>(p.kept.ab) + (int64_t)t * 2 * p.I + i;
      ab[0] = (uint16_t)f2bf(v.x);
      ab[p.I] = (uint16_t)f2bf(v.y);
    }
  });
}

template <int R, int NF, int W, int D>
__global__ __launch_bounds__(64 * W) void k_few_down(RowsArgs p) {
  __shared__ __align__(16) uint8_t lds[lds_bytes<R, NF, W, D>()];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n0 = blockIdx.x * 16 * R;
  const int S = p.K / 64, s0 = wave * S / W, s1 = (wave + 1) * S / W;
  f32x4_t acc[R][NF] = {};
  auto w = [&](int r) { return reinterpret_cast<const uint8_t*>(p.b0.p + (int64_t)min(n0 + r, p.N - 1) * p.b0.ld); };
  auto x = [&](int c) { return c < p.T ? reinterpret_cast<const uint8_t*>(p.a.p + (int64_t)c * p.a.ld) : nullptr; };
  stream::run<R, NF, 0, D>(lds + wave * stream::Ring<R, NF, 0, D>::kBytes, s0, s1 - s0, 2 * (int64_t)p.K, w, x,
                           [](int, int) { return (const void*)nullptr; },
                           [&](const uint8_t* wt, const uint8_t* xt, const float*) { stage<R, NF>(wt, xt, acc); });
  join<R, NF, W>(acc, lds, p.T, [&](int t, int row, float2 v) {
    const int n = n0 + row;                // N is a multiple of 64
    if (n < p.N) *reinterpret_cast<uint32_t*>(p.c.p + (int64_t)t * p.c.ld + n) = pack_bf2(v.x, v.y);
  });
}

template <int R, int NF, int W, int D>
void up_as(hipStream_t st, const UpArgs& a) {
  const dim3 grid((unsigned)((a.I + 8 * R - 1) / (8 * R))), block(64 * W);
  if (a.act == kSilu) hipLaunchKernelGGL((k_few_up<kSilu, R, NF, W, D>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((k_few_up<kGelu, R, NF, W, D>), grid, block, 0, st, a);
}
template <int R, int NF, int W, int D>
void down_as(hipStream_t st, const RowsArgs& a) {
  const dim3 grid((unsigned)((a.N + 16 * R - 1) / (16 * R))), block(64 * W);
  hipLaunchKernelGGL((k_few_down<R, NF, W, D>), grid, block, 0, st, a);
}

// f(fragments a workgroup, token tiles, waves, stages in flight).  Two fragments share the tokens' copies, which pays where
// one would leave more workgroups than CUs anyway (T > 32: first kernel of 48 tokens, H 4096, I 12288 45 us against 67, second
// one of 37, H 7168, I 2048 10 against 12.5; but its first one, 256 workgroups, 16 against 15.4) or, with two token
// tiles, many more (first kernel of 24 tokens, H 4096, I 12288 39 us against 47).  Four waves and two stages in flight leave
// room for two workgroups a CU; one token tile is so small that eight waves do (13 tokens, H 4096, I 12288: 57 us,
// 64 with four stages).
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
void launch_down_few(hipStream_t st, const RowsArgs& a) {
  by_tokens(a.T, a.N / 16, [&](auto r, auto nf, auto w, auto d) {
    down_as<decltype(r)::value, decltype(nf)::value, decltype(w)::value, decltype(d)::value>(st, a);
  });
}

}  // namespace ffn
}  // namespace moe

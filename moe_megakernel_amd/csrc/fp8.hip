// 8-bit matrix products with a scale for each block of 128, for rows in groups:
//   out[m][n] = sum over blocks b of 128 k:  sa[b][m] sb[..n..][b]  sum_{k in b} A[m][k] B[g(m)][n][k]
//
// One v_mfma_f32_16x16x128 covers a block of k.  Weights are its 16-row operand and tokens its 16
// columns, so a lane's four results belong to one token: with a scale a 128 x 128 weight tile a
// lane multiplies its four results by one number, 16 cycles of vector work next to the 32 of the
// product, which the other accumulators' products cover.  The sums over a block start from zero, are scaled
// and added in FP32.
#include <hip/hip_runtime.h>

#include "../../include/moe.h"
#include "fp8.hpp"
#include "fp8_wide.hpp"
#include "gemm.hpp"
#include "host.hpp"

namespace moe {
namespace fp8 {

using gemm::dma16;
using gemm::dma4;
using gemm::g_zero_page;
using gemm::lds_off;
using gemm::swz_kc;
using gemm::u32x4_t;
using gemm::wait_vm;

namespace {

constexpr int kKB = 128;                   // k of a stage, and of a scale

// Tile of TN weight rows and TM tokens; NSW stages of weights in LDS, two of tokens.
template <int TN_, int TM_, int NWN_, int NWM_, int MINB_, int NSW_>
struct Shape {
  static constexpr int TN = TN_, TM = TM_, NWN = NWN_, NWM = NWM_, MINB = MINB_, NSW = NSW_;
  static constexpr int NW = NWN * NWM, NTH = 64 * NW;
  static constexpr int NB = TN / NWN / 16, MB = TM / NWM / 16;   // 16 x 16 blocks of a wave
  static constexpr int W_BYTES = TN * kKB, A_BYTES = TM * kKB;
  static constexpr int W_DMA = W_BYTES / 1024 / NW, A_DMA = A_BYTES / 1024 / NW;   // copies a wave and stage
  static_assert(W_BYTES % (1024 * NW) == 0 && A_BYTES % (1024 * NW) == 0, "copies a wave");
  static_assert(TN % 64 == 0 && TM % 64 == 0 && (NSW == 2 || NSW == 3), "scale copies, ring");
  static_assert(NB * 16 <= 128 && 128 % (NB * 16) == 0 && NB >= 4 && NB % 2 == 0 && NB * MB % 2 == 0, "one weight scale a wave");
  // copies of 64 scales: the tokens', then the weights' rows' or those of the tile's 128-row parts; the same
  // number a wave, so that its copies can be counted
  template <bool ROWS_B>
  static constexpr int scale_copies() { return (TM / 64 + (ROWS_B ? TN / 64 : 1) + NW - 1) / NW * NW; }
  template <bool ROWS_B>
  static constexpr int lds() { return NSW * (W_BYTES + 256 * scale_copies<ROWS_B>()) + 2 * A_BYTES; }
};

struct Tile {
  int g, m0, rows, n0;
  bool ok;
};

// Tile of a block.  Groups' tile counts come from the offsets, one thread a group; entries outside
// [0, M] are taken as the nearest end, so every row index stays inside.
template <class S>
__device__ __forceinline__ Tile find_tile(const MatmulArgs& p, int* prefix) {
  const int nt = (p.N + S::TN - 1) / S::TN;
  Tile t{0, 0, 0, 0, false};
  int mt = (p.M + S::TM - 1) / S::TM, begin = 0, count = p.M, lo = 0;
  const int x = blockIdx.x & 7, j = blockIdx.x >> 3;
  if (p.offsets) {
    if (threadIdx.x < 64) {                // an inclusive scan by one wave, 64 groups at a time
      const int lane = threadIdx.x;
      int carry = 0;
      for (int g0 = 0; g0 < p.G; g0 += 64) {
        int n = 0;
        if (g0 + lane < p.G) {
          const int o0 = min(max(p.offsets[g0 + lane], 0), p.M), o1 = min(max(p.offsets[g0 + lane + 1], 0), p.M);
          n = max(o1 - o0, 0);
          n = (n + S::TM - 1) / S::TM;
        }
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
          const int v = __shfl_up(n, o);
          n += lane >= o ? v : 0;
        }
        if (g0 + lane < p.G) prefix[g0 + lane + 1] = carry + n;
        carry += __shfl(n, 63);
      }
      if (lane == 0) prefix[0] = 0;
    }
    __syncthreads();
    mt = prefix[p.G];
  }
  const int64_t total = (int64_t)mt * nt;
  const int64_t t0 = total * x / 8, t1 = total * (x + 1) / 8;
  if (j >= t1 - t0) return t;
  const int64_t L = t0 + j;
  int first = 0, tiles = mt;
  if (p.offsets) {
    const int at = (int)(L / nt);
    int hi = p.G - 1;
    while (lo < hi) {                      // the last group that starts at or before the tile
      const int mid = (lo + hi + 1) >> 1;
      if (prefix[mid] <= at) lo = mid;
      else hi = mid - 1;
    }
    first = prefix[lo];
    tiles = prefix[lo + 1] - first;
    begin = min(max(p.offsets[lo], 0), p.M);
    count = min(max(p.offsets[lo + 1], 0), p.M) - begin;
  }
  // bands of m tiles, m fastest, as in the layer's products
  const int64_t in = L - (int64_t)first * nt;
  const int band = (int)(in / (gemm::kBandM * nt));
  const int r = (int)(in - (int64_t)band * gemm::kBandM * nt), h = min(gemm::kBandM, tiles - band * gemm::kBandM);
  const int m = (band * gemm::kBandM + r % h) * S::TM;
  t.g = lo;
  t.m0 = begin + m;
  t.rows = min(S::TM, count - m);
  t.n0 = r / h * S::TN;
  t.ok = true;
  return t;
}

template <class S, bool ROWS_B, bool F32, bool ADD>
__global__ __launch_bounds__(S::NTH, S::MINB) void k_fp8_matmul(MatmulArgs p) {
  __shared__ __align__(16) uint8_t lds[S::template lds<ROWS_B>()];
  const Tile t = find_tile<S>(p, reinterpret_cast<int*>(lds));
  if (!t.ok) return;
  __syncthreads();                         // the groups' table is read before the stages take its place
  const int lane = threadIdx.x & 63, r16 = lane & 15, q4 = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), wn = w % S::NWN, wm = w / S::NWN;
  const int cols = min(S::TN, p.N - t.n0), rows = t.rows;
  const uint32_t lds0 = lds_off(lds);
  const uint8_t* zp = reinterpret_cast<const uint8_t*>(g_zero_page) + 16 * lane;
  const int nk = (p.K + kKB - 1) / kKB;

  // LDS: the weights' stages [NSW][TN][128], the tokens' [2][TM][128] (16-byte chunks swizzled by row), the
  // scales' [NSW].  Rows past the last repeat it, their results go nowhere; chunks past the last k are zeros.
  constexpr int SC = S::template scale_copies<ROWS_B>(), SC_DMA = SC / S::NW;
  constexpr int A0 = S::NSW * S::W_BYTES, SC0 = A0 + 2 * S::A_BYTES;
  const uint8_t *pw[S::W_DMA], *pa[S::A_DMA];
#pragma unroll
  for (int i = 0; i < S::W_DMA; ++i) {
    const int off = (w * S::W_DMA + i) * 1024 + 16 * lane, r = off / kKB, c = ((off % kKB) >> 4) ^ swz_kc<128>(r);
    pw[i] = p.b + (int64_t)t.g * p.stride_b + (int64_t)(t.n0 + min(r, cols - 1)) * p.ldb + 16 * c;
  }
#pragma unroll
  for (int i = 0; i < S::A_DMA; ++i) {
    const int off = (w * S::A_DMA + i) * 1024 + 16 * lane, r = off / kKB, c = ((off % kKB) >> 4) ^ swz_kc<128>(r);
    pa[i] = p.a + (int64_t)(t.m0 + min(r, rows - 1)) * p.lda + 16 * c;
  }
  // copies of a stage; `copy` holds rows 8 copy .. 8 copy + 7, and swz_kc has period 16
  auto copies = [&](int kt, const uint8_t** q, int n, int first, uint32_t to) __attribute__((always_inline)) {
    if (kt * kKB + kKB <= p.K) {
      for (int i = 0; i < n; ++i) {
        dma16(q[i], to + (first + i) * 1024);
        q[i] += kKB;
      }
    } else {
      for (int i = 0; i < n; ++i) {
        const int k = kt * kKB + 16 * ((lane & 7) ^ swz_kc<128>(8 * (first + i) + (lane >> 3)));
        dma16(k < p.K ? q[i] : zp, to + (first + i) * 1024);
      }
    }
  };
  const int sb_rows = (p.N + 127) / 128;
  const float* sb0 = ROWS_B ? p.sb + t.n0
                            : p.sb + ((int64_t)t.g * sb_rows + min(t.n0 / 128 + min(lane, S::TN / 128 - 1), sb_rows - 1)) * nk;
  auto issue_w = [&](int kt, int slot) __attribute__((always_inline)) {
    copies(kt, pw, S::W_DMA, w * S::W_DMA, lds0 + slot * S::W_BYTES);
#pragma unroll
    for (int u = 0; u < SC_DMA; ++u) {
      const int i = u * S::NW + w;
      const float* src;
      if (i < S::TM / 64) src = p.sa + (int64_t)kt * p.M + t.m0 + min(64 * i + lane, rows - 1);
      else if (ROWS_B) src = sb0 + (int64_t)kt * p.N + min(64 * (i - S::TM / 64) + lane, cols - 1);
      else src = sb0 + kt;
      dma4(src, lds0 + SC0 + (slot * SC + i) * 256);
    }
  };
  auto issue_a = [&](int kt) __attribute__((always_inline)) {
    copies(kt, pa, S::A_DMA, w * S::A_DMA, lds0 + A0 + (kt & 1) * S::A_BYTES);
  };

  f32x4_t acc[S::NB][S::MB];
#pragma unroll
  for (int i = 0; i < S::NB; ++i)
#pragma unroll
    for (int j = 0; j < S::MB; ++j) acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  // A lane's 32 codes of row r16 of a 16-row block: chunks q4 and q4 + 4 (which 32 is free, as long as
  // both operands agree).  The swizzle is the same for every block, so the blocks lie at constant distances.
  const int f0 = r16 * kKB + ((q4 ^ swz_kc<128>(r16)) << 4), f1 = f0 ^ 64;
  auto frag = [&](const uint8_t* block) __attribute__((always_inline)) {
    const u32x4_t u0 = *reinterpret_cast<const u32x4_t*>(block + f0), u1 = *reinterpret_cast<const u32x4_t*>(block + f1);
    return i32x8_t{(int)u0[0], (int)u0[1], (int)u0[2], (int)u0[3], (int)u1[0], (int)u1[1], (int)u1[2], (int)u1[3]};
  };
  struct Tokens {                          // a stage's token fragments and scales
    i32x8_t x[S::MB];
    float s[S::MB];
  };
  struct Weights {                         // 16 weight rows and their scales
    i32x8_t w;
    f32x4_t s;
  };
  const uint8_t *lw = lds + wn * S::NB * 16 * kKB, *la = lds + A0 + wm * S::MB * 16 * kKB;
  const float* ls = reinterpret_cast<const float*>(lds + SC0);
  auto load_tokens = [&](int kt, int slot, int j, Tokens& o) __attribute__((always_inline)) {
    const float* sc = ls + slot * SC * 64;
    o.x[j] = frag(la + (kt & 1) * S::A_BYTES + j * 16 * kKB);
    o.s[j] = sc[(wm * S::MB + j) * 16 + r16];
    if constexpr (!ROWS_B) o.s[j] *= sc[S::TM + wn * S::NB * 16 / 128];
  };
  auto load_weights = [&](int slot, int i, Weights& o) __attribute__((always_inline)) {
    o.w = frag(lw + slot * S::W_BYTES + i * 16 * kKB);
    if constexpr (ROWS_B)
      o.s = *reinterpret_cast<const f32x4_t*>(ls + slot * SC * 64 + S::TM + (wn * S::NB + i) * 16 + 4 * q4);
  };

  // Barrier B(kt) opens stage kt: its copies have landed.  The weights' fragment of block i + 1 is read while
  // block i multiplies, and the last block of a stage multiplies behind the barrier that opens the next, each
  // token fragment replaced by the next stage's as soon as it has been used.  So the weights' slot of stage
  // kt - 1 is free at B(kt), and the tokens' of stage kt once every wave has started it: a second barrier behind
  // the first block, which gives their copies two stages of lead with two slots.  A product's result is scaled
  // and added two products later, when it is there.
  constexpr int FLY = S::A_DMA + (S::NSW == 3 ? S::W_DMA + SC_DMA : 0);   // copies younger than stage kt + 1's at B(kt + 1)
  issue_w(0, 0);
  issue_a(0);
  if (nk > 1) {
    if constexpr (S::NSW == 3) issue_w(1, 1);
    issue_a(1);
    wait_vm<FLY>();
  } else {
    wait_vm<0>();
  }
  __syncthreads();
  Tokens tk;
  Weights wt[2];
#pragma unroll
  for (int j = 0; j < S::MB; ++j) load_tokens(0, 0, j, tk);
  load_weights(0, 0, wt[0]);
  constexpr int LAST = S::NB * S::MB;
  struct Pending {
    f32x4_t d, s;
  };
  Pending pend[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) pend[u].d = pend[u].s = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  auto settle = [&](f32x4_t& a, const Pending& q) __attribute__((always_inline)) {
#pragma unroll
    for (int e = 0; e < 4; ++e) a[e] += q.s[ROWS_B ? e : 0] * q.d[e];
  };
  int slot = 0;                            // the stage's weights
  auto run_stage = [&](int kt, auto more) __attribute__((always_inline)) {
    constexpr bool MORE = decltype(more)::value;
    const int next = slot + 1 == S::NSW ? 0 : slot + 1, last = slot == 0 ? S::NSW - 1 : slot - 1;
    if (MORE && kt + S::NSW - 1 < nk) issue_w(kt + S::NSW - 1, last);
#pragma unroll
    for (int i = 0; i < S::NB; ++i) {
      // products stay on their side of the barriers (they touch no memory, so the compiler would move all of
      // them behind the last one, and every copy would be waited for where it is issued)
      __builtin_amdgcn_sched_barrier(0);
      if (i == 1 && MORE) {
        __syncthreads();
        if (kt + 2 < nk) issue_a(kt + 2);
      }
      if (i + 1 < S::NB) {
        load_weights(slot, i + 1, wt[(i + 1) & 1]);
      } else if constexpr (MORE) {
        if (kt + 2 < nk) wait_vm<FLY>();
        else wait_vm<0>();
        __syncthreads();
        __builtin_amdgcn_sched_barrier(0);
        load_weights(next, 0, wt[0]);
      }
#pragma unroll
      for (int j = 0; j < S::MB; ++j) {
        const int k = i * S::MB + j;
        Pending q;
        if constexpr (F32) q.d = wide_product(widen(wt[i & 1].w), widen(tk.x[j]));
        else q.d = code_product(wt[i & 1].w, tk.x[j]);
        if constexpr (ROWS_B) q.s = wt[i & 1].s * tk.s[j];
        else q.s[0] = tk.s[j];
        const int o = (k + LAST - 2) % LAST;
        settle(acc[o / S::MB][o % S::MB], pend[k & 1]);
        pend[k & 1] = q;
        if (MORE && i + 1 == S::NB) load_tokens(kt + 1, next, j, tk);
      }
    }
    slot = next;
  };
  for (int kt = 0; kt + 1 < nk; ++kt) run_stage(kt, std::true_type{});
  run_stage(nk - 1, std::false_type{});
#pragma unroll
  for (int u = 0; u < 2; ++u) settle(acc[(LAST - 2 + u) / S::MB][(LAST - 2 + u) % S::MB], pend[(LAST - 2 + u) & 1]);

  // lane: token r16 of a block, columns 4 q4 .. 4 q4 + 3
  const bool vec = p.ldo % 4 == 0 && (reinterpret_cast<uintptr_t>(p.out) & (F32 ? 15u : 7u)) == 0;
#pragma unroll
  for (int j = 0; j < S::MB; ++j) {
    const int m = (wm * S::MB + j) * 16 + r16;
    if (m >= rows) continue;
#pragma unroll
    for (int i = 0; i < S::NB; ++i) {
      const int n = (wn * S::NB + i) * 16 + 4 * q4;
      if (n >= cols) continue;
      uint8_t* to = p.out + ((int64_t)(t.m0 + m) * p.ldo + t.n0 + n) * (F32 ? 4 : 2);
      const f32x4_t v = acc[i][j];
      if (vec && n + 4 <= cols) {
        if constexpr (F32) {
          f32x4_t* o = reinterpret_cast<f32x4_t*>(to);
          *o = ADD ? *o + v : v;
        } else {
          uint2* o = reinterpret_cast<uint2*>(to);
          uint2 z = make_uint2(pack_bf2(v[0], v[1]), pack_bf2(v[2], v[3]));
          if constexpr (ADD) {
            const uint2 y = *o;
            z = make_uint2(pack_bf2(lo_bf(y.x) + lo_bf(z.x), hi_bf(y.x) + hi_bf(z.x)),
                           pack_bf2(lo_bf(y.y) + lo_bf(z.y), hi_bf(y.y) + hi_bf(z.y)));
          }
          *o = z;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (n + e >= cols) break;
          if constexpr (F32) {
            float* o = reinterpret_cast<float*>(to) + e;
            *o = ADD ? *o + v[e] : v[e];
          } else {
            uint16_t* o = reinterpret_cast<uint16_t*>(to) + e;
            const uint32_t z = f2bf(v[e]);
            *o = (uint16_t)(ADD ? f2bf(bf2f(*o) + bf2f(z)) : z);
          }
        }
      }
    }
  }
}

using Large = Shape<256, 192, 2, 2, 1, 3>;
using Wide32 = Shape<128, 128, 2, 2, 1, 3>;

template <class S>
int64_t tiles(const MatmulArgs& a) {
  const int64_t m = (a.M + S::TM - 1) / S::TM + (a.offsets ? a.G : 0);
  return m * ((a.N + S::TN - 1) / S::TN);
}

template <class S, bool ROWS_B, bool F32>
void launch_as(hipStream_t st, const MatmulArgs& a) {
  const dim3 grid((unsigned)((tiles<S>(a) + 7) / 8 * 8 + 8)), block(S::NTH);
  if (a.accumulate) hipLaunchKernelGGL((k_fp8_matmul<S, ROWS_B, F32, true>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((k_fp8_matmul<S, ROWS_B, F32, false>), grid, block, 0, st, a);
}
template <class S, bool F32>
void launch_shape(hipStream_t st, const MatmulArgs& a) {
  if (a.rows_b) launch_as<S, true, F32>(st, a);
  else launch_as<S, false, F32>(st, a);
}

moe_status check(const moe_block_matmul_problem* p) {
  if (!p) return MOE_ERR_NULL;
  const int64_t M = p->rows, N = p->cols, K = p->depth;
  if (M < 0 || M > (1 << 24) || N < 1 || N > (1 << 20) || K < 16 || K > (1 << 24) || K % 16) return MOE_ERR_SHAPE;
  if (p->groups < 1 || p->groups > kMaxGroups) return MOE_ERR_SHAPE;
  if ((M / 64 + 1 + p->groups) * (N / 128 + 1) > (1 << 22)) return MOE_ERR_SHAPE;   // a launch holds 2^32 threads
  if (p->scales != MOE_FP8_ROWS && p->scales != MOE_FP8_TILES) return MOE_ERR_UNSUPPORTED;
  if (p->scales == MOE_FP8_ROWS && p->groups != 1) return MOE_ERR_UNSUPPORTED;
  if (p->out_dtype != MOE_BF16 && p->out_dtype != MOE_FP32) return MOE_ERR_DTYPE;
  if (p->flags & ~MOE_FP8_ACCUMULATE) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace

void launch_matmul(hipStream_t st, const MatmulArgs& a) {
  if (a.M <= kFewRows) launch_few(st, a);
  else if (a.out_fp32) launch_shape<Wide32, true>(st, a);
  else launch_shape<Large, false>(st, a);
}

}  // namespace fp8
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_block_matmul(const moe_block_matmul_problem* p, const moe_rows* a, const float* a_scales,
                                     const moe_mat* b, const float* b_scales, const int32_t* offsets,
                                     const moe_rows* out, void* stream) {
  MOE_TRY(fp8::check(p));
  if (p->rows == 0) return MOE_OK;
  if (!a || !a->base || !a_scales || !b || !b->base || !b_scales || !out || !out->base) return MOE_ERR_NULL;
  if (p->groups > 1 && !offsets) return MOE_ERR_NULL;
  if (b->table) return MOE_ERR_LAYOUT;
  if (a->ld < p->depth || a->ld % 16 || !aligned16(a->base)) return MOE_ERR_LAYOUT;
  if (b->ld < p->depth || b->ld % 16 || !aligned16(b->base)) return MOE_ERR_LAYOUT;
  if (p->groups > 1 && (b->expert_stride < 0 || b->expert_stride % 16)) return MOE_ERR_LAYOUT;
  if (out->ld < p->cols || !elem_aligned(out->base, p->out_dtype)) return MOE_ERR_LAYOUT;
  if (!aligned4(a_scales) || !aligned4(b_scales) || !aligned4(offsets)) return MOE_ERR_LAYOUT;
  fp8::MatmulArgs m{};
  m.a = static_cast<const uint8_t*>(a->base);
  m.sa = a_scales;
  m.b = static_cast<const uint8_t*>(b->base);
  m.sb = b_scales;
  m.out = static_cast<uint8_t*>(out->base);
  m.offsets = offsets;
  m.lda = a->ld; m.ldb = b->ld; m.stride_b = b->expert_stride; m.ldo = out->ld;
  m.M = (int)p->rows; m.N = (int)p->cols; m.K = (int)p->depth; m.G = p->groups;
  m.out_fp32 = p->out_dtype == MOE_FP32;
  m.accumulate = (p->flags & MOE_FP8_ACCUMULATE) != 0;
  m.rows_b = p->scales == MOE_FP8_ROWS;
  hipStream_t st = static_cast<hipStream_t>(stream);
  return launch("block_matmul", st, [&] { fp8::launch_matmul(st, m); });
}

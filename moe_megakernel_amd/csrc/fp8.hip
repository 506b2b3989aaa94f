// 8-bit matrix products with a scale for each block of 128, for rows in groups:
//   out[m][n] = sum over blocks b of 128 k:  sa[b][m] sb[..n..][b]  sum_{k in b} A[m][k] B[g(m)][n][k]
//
// One v_mfma_f32_16x16x128 covers a block of k.  Weights are its 16-row operand and tokens its 16
// columns, so a lane's four results belong to one token: with a scale a 128 x 128 weight tile a
// lane multiplies its four results by one number, 16 cycles of vector work next to the 32 of the
// product, which the other accumulators' products cover.  The sums over a block start from zero, are scaled
// and added in FP32.
//
// 8192 x 4096 x 7168: 242 us among other work, 215 back to back (2240 TFLOP/s; registers alone multiply and scale at 3970).
// The matrix units are busy 44 % of the time, the vector units as long; one wave a SIMD issues both, and the
// LDS reads, the copies' addresses and the stage's ends come on top.
#include <hip/hip_runtime.h>

#include "../../include/moe.h"
#include "fp8.hpp"
#include "fp8_wide.hpp"
#include "gemm.hpp"
#include "host.hpp"

namespace moe {
namespace fp8 {

static_assert(kFewRows == MOE_FP8_FEW_ROWS, "as the header says");

using gemm::dma16;
using gemm::dma16s;
using gemm::dma4;
using gemm::g_zero_page;
using gemm::lds_off;
using gemm::swz_kc;
using gemm::u32x4_t;
using gemm::wait_vm;

namespace {

constexpr int kKB = 128;                   // k of a stage, and of a scale
constexpr int kStages = 3;                 // in LDS

// Tile of TN weight rows and TM tokens.
template <int TN_, int TM_, int NWN_, int NWM_, int MINB_>
struct Shape {
  static constexpr int TN = TN_, TM = TM_, NWN = NWN_, NWM = NWM_, MINB = MINB_;
  static constexpr int NW = NWN * NWM, NTH = 64 * NW;
  static constexpr int NB = TN / NWN / 16, MB = TM / NWM / 16;   // 16 x 16 blocks of a wave
  static constexpr int W_BYTES = TN * kKB, A_BYTES = TM * kKB;
  static constexpr int W_DMA = W_BYTES / 1024 / NW, A_DMA = A_BYTES / 1024 / NW;   // copies a wave and stage
  static_assert(W_BYTES % (1024 * NW) == 0 && A_BYTES % (1024 * NW) == 0, "copies a wave");
  static_assert(TN % 64 == 0 && TM % 64 == 0, "scale copies");
  static_assert(NB * 16 <= 128 && 128 % (NB * 16) == 0, "one weight scale a wave");
  static_assert(NB % 4 == 0, "fragment buffers");
  // copies of 64 scales: the tokens', then the weights' rows' or those of the tile's 128-row parts; the same
  // number a wave, so that its copies can be counted
  template <bool ROWS_B>
  static constexpr int scale_copies() { return (TM / 64 + (ROWS_B ? TN / 64 : 1) + NW - 1) / NW * NW; }
  template <bool ROWS_B>
  static constexpr int lds() { return kStages * (W_BYTES + A_BYTES + 256 * scale_copies<ROWS_B>()); }
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

// The steady loop has no branch, and products stay on their side of the barriers: they touch no memory, so the compiler
// would move them to where their results are used, behind the last barrier.  Code that runs once a tile is kept
// short: a workgroup fetches it anew, at about 60 ns for each 64 bytes.
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
  const int nk = (p.K + kKB - 1) / kKB;

  // LDS: the weights' stages [3][TN][128], the tokens' [3][TM][128] (16-byte chunks swizzled by row), the
  // scales' [3].  Rows past the last repeat it, their results go nowhere; chunks past the last k are zeros.
  constexpr int SC = S::template scale_copies<ROWS_B>(), SC_DMA = SC / S::NW;
  constexpr int A0 = kStages * S::W_BYTES, SC0 = A0 + kStages * S::A_BYTES;
  // The lane's offset of each copy from the stage's first byte (host checks keep them below 2^32).
  const uint8_t* gw = p.b + (int64_t)t.g * p.stride_b + (int64_t)t.n0 * p.ldb;
  const uint8_t* ga = p.a + (int64_t)t.m0 * p.lda;
  uint32_t ow[S::W_DMA], oa[S::A_DMA];
#pragma unroll
  for (int i = 0; i < S::W_DMA; ++i) {
    const int off = (w * S::W_DMA + i) * 1024 + 16 * lane, r = off / kKB, c = ((off % kKB) >> 4) ^ swz_kc<128>(r);
    ow[i] = (uint32_t)(min(r, cols - 1) * p.ldb) + 16 * c;
  }
#pragma unroll
  for (int i = 0; i < S::A_DMA; ++i) {
    const int off = (w * S::A_DMA + i) * 1024 + 16 * lane, r = off / kKB, c = ((off % kKB) >> 4) ^ swz_kc<128>(r);
    oa[i] = (uint32_t)(min(r, rows - 1) * p.lda) + 16 * c;
  }
  // scales, 64 a copy: the tokens', then the weights' rows' or those of the tile's 128-row parts
  const float* ps[SC_DMA];
  int64_t step[SC_DMA];                    // floats from a stage's to the next one's
#pragma unroll
  for (int u = 0; u < SC_DMA; ++u) {
    const int i = u * S::NW + w;
    const int nb = (p.N + 127) / 128;
    const bool tok = i < S::TM / 64;
    const int64_t tiles = ((int64_t)t.g * nb + min(t.n0 / 128 + min(lane, S::TN / 128 - 1), nb - 1)) * nk;
    ps[u] = tok ? p.sa + t.m0 + min(64 * i + lane, rows - 1)
                : p.sb + (ROWS_B ? t.n0 + min(64 * (i - S::TM / 64) + lane, cols - 1) : tiles);
    step[u] = tok ? p.M : (ROWS_B ? p.N : 1);
  }
  int put = 0;                             // ring slot of the next stage
  auto after = [](int slot) __attribute__((always_inline)) { return slot + 1 == kStages ? 0 : slot + 1; };
  auto copy_scales = [&](int u) __attribute__((always_inline)) {
    dma4(ps[u], lds0 + SC0 + (put * SC + u * S::NW + w) * 256);
    ps[u] += step[u];
  };
  auto to_w = [&](int i) __attribute__((always_inline)) { return lds0 + put * S::W_BYTES + (w * S::W_DMA + i) * 1024; };
  auto to_a = [&](int i) __attribute__((always_inline)) { return lds0 + A0 + put * S::A_BYTES + (w * S::A_DMA + i) * 1024; };
  constexpr int COPIES = S::W_DMA + S::A_DMA + SC_DMA;       // a wave and stage
  auto copy = [&](int i) __attribute__((always_inline)) {
    if (i < S::W_DMA) dma16s(gw, ow[i], to_w(i));
    else if (i < S::W_DMA + S::A_DMA) dma16s(ga, oa[i - S::W_DMA], to_a(i - S::W_DMA));
    else copy_scales(i - S::W_DMA - S::A_DMA);
  };
  auto advance = [&]() __attribute__((always_inline)) {
    gw += kKB;
    ga += kKB;
    put = after(put);
  };
  // Any stage: of the last, chunks past K come from the zero page.  (Copy c holds rows 8 c .. 8 c + 7, and
  // swz_kc has period 16.)
  auto chunk = [&](int kt, const uint8_t* q, int c) __attribute__((always_inline)) {
    return kt * kKB + 16 * ((lane & 7) ^ swz_kc<128>(8 * c + (lane >> 3))) < p.K
               ? q : reinterpret_cast<const uint8_t*>(g_zero_page) + 16 * lane;
  };
  auto issue = [&](int kt) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < S::W_DMA; ++i) dma16(chunk(kt, gw + ow[i], w * S::W_DMA + i), to_w(i));
#pragma unroll
    for (int i = 0; i < S::A_DMA; ++i) dma16(chunk(kt, ga + oa[i], w * S::A_DMA + i), to_a(i));
#pragma unroll
    for (int u = 0; u < SC_DMA; ++u) copy_scales(u);
    advance();
  };

  f32x4_t acc[S::NB][S::MB];
  {
    float z = 0.0f;                        // not known to be zero: see the dense products
    asm volatile("" : "+v"(z));
#pragma unroll
    for (int i = 0; i < S::NB; ++i)
#pragma unroll
      for (int j = 0; j < S::MB; ++j) acc[i][j] = f32x4_t{z, z, z, z};
  }

  // A lane's 32 codes of row r16 of a 16-row block: chunks q4 and q4 + 4 (which 32 is free, as long as
  // both operands agree).  The swizzle is the same for every block, so the blocks lie at constant distances.
  const int f0 = r16 * kKB + ((q4 ^ swz_kc<128>(r16)) << 4), f1 = f0 ^ 64;
  auto frag = [&](const uint8_t* block) __attribute__((always_inline)) {
    const u32x4_t u0 = *reinterpret_cast<const u32x4_t*>(block + f0), u1 = *reinterpret_cast<const u32x4_t*>(block + f1);
    return i32x8_t{(int)u0[0], (int)u0[1], (int)u0[2], (int)u0[3], (int)u1[0], (int)u1[1], (int)u1[2], (int)u1[3]};
  };
  i32x8_t x[S::MB], wf[4];                 // token fragments of a stage, weight fragments of a block and the next two
  float s[S::MB], st[S::MB], swt;          // the tokens' scales (times the weight tile's), the next stage's as read
  f32x4_t sw[4];                           // ROWS_B: the weight rows' scales
  const uint8_t *lw = lds + wn * S::NB * 16 * kKB, *la = lds + A0 + wm * S::MB * 16 * kKB;
  const float* ls = reinterpret_cast<const float*>(lds + SC0);
  auto load_tokens = [&](int slot, int j) __attribute__((always_inline)) {
    const float* sc = ls + slot * SC * 64;
    x[j] = frag(la + slot * S::A_BYTES + j * 16 * kKB);
    st[j] = sc[(wm * S::MB + j) * 16 + r16];
    if (!ROWS_B && j == 0) swt = sc[S::TM + wn * S::NB * 16 / 128];
  };
  auto load_weights = [&](int slot, int i) __attribute__((always_inline)) {
    wf[i % 4] = frag(lw + slot * S::W_BYTES + i * 16 * kKB);
    if constexpr (ROWS_B)
      sw[i % 4] = *reinterpret_cast<const f32x4_t*>(ls + slot * SC * 64 + S::TM + (wn * S::NB + i) * 16 + 4 * q4);
  };

  // Stage kt multiplies NB blocks of 16 weight rows, each with the MB token fragments; the last two blocks in turn, a token
  // fragment at a time, which is replaced by the next stage's as soon as both have used it (in the last block
  // alone, those reads would crowd the LDS: 3 % of the whole).  A block's weights are read two blocks ahead.  So the
  // barrier that opens stage kt + 1 (its copies have landed) stands two blocks before the end of stage kt, whose
  // slot has then been read for good; the copies of stage kt + 2 take the slot of stage kt - 1, freed a barrier ago.  A
  // product's result is scaled and added two products later, when it is there.
  constexpr int LAST = S::NB * S::MB, OPEN = (S::NB - 2) * S::MB;   // products a stage, those before the barrier
  auto copies_before = [](int product) constexpr { return product * COPIES / LAST; };
  constexpr int FLY = copies_before(OPEN);                 // copies of stage kt + 2 at the barrier
  f32x4_t pd[2], pq[2];                    // results on their way and their scales
#pragma unroll
  for (int u = 0; u < 2; ++u) pd[u] = pq[u] = acc[0][0];
  auto settle = [&](f32x4_t& a, int u) __attribute__((always_inline)) {
    if constexpr (ROWS_B) a = __builtin_elementwise_fma(pq[u], pd[u], a);
    else a = __builtin_elementwise_fma(f32x4_t{pq[u][0], pq[u][0], pq[u][0], pq[u][0]}, pd[u], a);
  };
  auto block_of = [](int k) constexpr { return k < OPEN ? k / S::MB : S::NB - 2 + (k - OPEN) % 2; };
  auto token_of = [](int k) constexpr { return k < OPEN ? k % S::MB : (k - OPEN) / 2; };
  // product k of a stage and what is read behind it
  auto product = [&](int k, int slot, int next) __attribute__((always_inline)) {
    const int i = block_of(k), j = token_of(k), o = (k + LAST - 2) % LAST;
    if (i == 0) s[j] = ROWS_B ? st[j] : st[j] * swt;   // not where they are read: that would wait for them
    f32x4_t d;
    if constexpr (F32) d = wide_product(widen(wf[i % 4]), widen(x[j]));
    else d = code_product(wf[i % 4], x[j]);
    settle(acc[block_of(o)][token_of(o)], k & 1);
    pd[k & 1] = d;
    if constexpr (ROWS_B) pq[k & 1] = sw[i % 4] * s[j];
    else pq[k & 1][0] = s[j];
    if (k < OPEN && j == 0) load_weights(slot, i + 2);
    if (k == OPEN) load_weights(next, 0);
    if (k == OPEN + S::MB) load_weights(next, 1);
    if (k >= OPEN && (k - OPEN) % 2) load_tokens(next, j);
  };
  static_assert(LAST % 2 == 0, "results on their way");
  int slot = 0;                            // the stage's
  auto steady = [&]() __attribute__((always_inline)) {
    const int next = after(slot);
#pragma unroll
    for (int k = 0; k < LAST; ++k) {
      if (k == OPEN) {
        wait_vm<FLY>();
        __syncthreads();
      }
      __builtin_amdgcn_sched_barrier(0);
      product(k, slot, next);
#pragma unroll
      for (int c = copies_before(k); c < copies_before(k + 1); ++c) copy(c);
    }
    __builtin_amdgcn_sched_barrier(0);
    advance();
    slot = next;
  };
  auto any = [&](int kt) __attribute__((always_inline)) {   // the last stages; behind the last one nothing is used that is read
    const int next = after(slot);
    if (kt + 2 < nk) issue(kt + 2);
#pragma unroll
    for (int k = 0; k < LAST; ++k) {
      if (k == OPEN) {
        if (kt + 2 < nk) wait_vm<COPIES>();
        else wait_vm<0>();
        __syncthreads();
      }
      product(k, slot, next);
    }
    slot = next;
  };

  issue(0);
  if (nk > 1) {
    issue(1);
    wait_vm<COPIES>();
  } else {
    wait_vm<0>();
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < S::MB; ++j) load_tokens(0, j);
  load_weights(0, 0);
  load_weights(0, 1);
  int kt = 0;
  if (kt + 3 < nk) {
    do steady();                           // its copies are whole stages
    while (++kt + 3 < nk);
    asm volatile("; steady done" ::: "memory");   // a block of its own, for what the register allocator moves on the way out
  }
#pragma unroll 1
  for (; kt < nk; ++kt) any(kt);
#pragma unroll
  for (int u = 0; u < 2; ++u) settle(acc[block_of(LAST - 2 + u)][token_of(LAST - 2 + u)], (LAST - 2 + u) & 1);

  // Results through LDS, a wave row's tokens at a time, so that a lane has 8 neighbouring columns.  Row r holds
  // 16-byte chunk c at c ^ (r % 16): the 16 rows a wave writes at once fall in disjoint banks.
  constexpr int WT = S::TM / S::NWM, PPR = S::TN / 8;
  static_assert(WT * S::TN * 4 <= S::template lds<ROWS_B>(), "epilogue round");
  float* ct = reinterpret_cast<float*>(lds);
  const int es = F32 ? 4 : 2;
  const bool vec = (p.ldo * es) % 16 == 0 && (reinterpret_cast<uintptr_t>(p.out) & 15u) == 0;
#pragma unroll 1
  for (int k = 0; k < S::NWM; ++k) {
    __syncthreads();
    if (wm == k) {
#pragma unroll
      for (int i = 0; i < S::NB; ++i)
#pragma unroll
        for (int j = 0; j < S::MB; ++j) {
          const int r = j * 16 + r16, c = (wn * S::NB + i) * 4 + q4;
          *reinterpret_cast<f32x4_t*>(ct + r * S::TN + ((c ^ r16) << 2)) = acc[i][j];
        }
    }
    __syncthreads();
    if (!vec) {                            // rows that no 16 bytes fit: a column a lane, eight rows at once
      constexpr int RPP = S::NTH / S::TN;  // rows a pass of the workgroup
      static_assert(S::NTH % S::TN == 0 && WT % (8 * RPP) == 0, "rows at once");
      const int n = threadIdx.x % S::TN, r0 = threadIdx.x / S::TN;
      if (n >= cols) continue;
#pragma unroll 1
      for (int e = 0; e < WT; e += 8 * RPP) {
        if (k * WT + e >= rows) break;
        float v[8], old[8];
        uint8_t* to[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int r = e + r0 + u * RPP, m = k * WT + r;
          v[u] = ct[r * S::TN + (((n / 4) ^ (r & 15)) << 2) + n % 4];
          to[u] = p.out + ((int64_t)(t.m0 + m) * p.ldo + t.n0 + n) * es;
          if constexpr (ADD)
            if (m < rows) old[u] = F32 ? *reinterpret_cast<const float*>(to[u]) : bf2f(*reinterpret_cast<const uint16_t*>(to[u]));
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          if (k * WT + e + r0 + u * RPP >= rows) continue;
          if constexpr (F32) *reinterpret_cast<float*>(to[u]) = ADD ? old[u] + v[u] : v[u];
          else *reinterpret_cast<uint16_t*>(to[u]) = (uint16_t)f2bf(ADD ? old[u] + bf2f(f2bf(v[u])) : v[u]);
        }
      }
      continue;
    }
#pragma unroll 1
    for (int o = threadIdx.x; o < WT * PPR; o += S::NTH) {
      const int r = o / PPR, n = 8 * (o % PPR), m = k * WT + r;
      if (m >= rows || n >= cols) continue;
      float v[8];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const f32x4_t q = *reinterpret_cast<const f32x4_t*>(ct + r * S::TN + (((n / 4 + h) ^ (r & 15)) << 2));
#pragma unroll
        for (int e = 0; e < 4; ++e) v[4 * h + e] = q[e];
      }
      uint8_t* to = p.out + ((int64_t)(t.m0 + m) * p.ldo + t.n0 + n) * es;
      if (n + 8 <= cols) {
        if constexpr (F32) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            f32x4_t* q = reinterpret_cast<f32x4_t*>(to) + h;
            const f32x4_t z{v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]};
            *q = ADD ? *q + z : z;
          }
        } else {
          if constexpr (ADD) {
            float old[8];
            unpack_bf16x8(*reinterpret_cast<const uint4*>(to), old);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = old[e] + bf2f(f2bf(v[e]));
          }
          *reinterpret_cast<uint4*>(to) = make_uint4(pack_bf2(v[0], v[1]), pack_bf2(v[2], v[3]), pack_bf2(v[4], v[5]),
                                                     pack_bf2(v[6], v[7]));
        }
      } else {                             // the last columns
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (n + e >= cols) break;
          if constexpr (F32) {
            float* q = reinterpret_cast<float*>(to) + e;
            *q = ADD ? *q + v[e] : v[e];
          } else {
            uint16_t* q = reinterpret_cast<uint16_t*>(to) + e;
            const uint32_t z = f2bf(v[e]);
            *q = (uint16_t)(ADD ? f2bf(bf2f(*q) + bf2f(z)) : z);
          }
        }
      }
    }
  }
}

// Large is the fastest where there are tiles for every CU (8192 x 4096 x 7168: 242 us; 256 x 192 is 7 % faster where one round
// of it covers what takes Large two, and up to 7 % slower elsewhere; 256 x 256 does not fit the registers).  FP32 results go in
// Medium tiles: 473 us, which 128 x 128 take too, and 88 against 94 for 8245 x 7334 over 224.
using Large = Shape<256, 128, 2, 2, 1>;
using Medium = Shape<128, 64, 2, 2, 2>;

template <class S>
int64_t tiles(const MatmulArgs& a) {
  const int64_t m = (a.M + S::TM - 1) / S::TM + (a.offsets ? a.G : 0);
  return m * ((a.N + S::TN - 1) / S::TN);
}

// Whether Medium tiles are the faster ones, from the rounds each needs: a Large round of w tiles (up to 256, one a CU) takes
// 0.78 + 0.12 w / 256 us a stage of k and 7 us; 512 Medium ones (two a CU) 0.58 and 6, up to 256 of them 0.42 and 6.  Measured,
// Large and Medium, in us at N 4096, K 7168: M 128 51.4 and 29.6, 1024 55.6 and 38.7, 1500 58.4 and 65.5, 4096 115 and 149; at
// N 2048, K 4096: M 2000 33.8 and 24.9, 3000 35.8 and 41.1; at N 1024, K 1024: M 4096 14.5 and 10.4, 16384 28.9 and 32.4.  Groups
// are taken to end in the middle of a tile.
bool medium(const MatmulArgs& a) {
  const int stages = (a.K + kKB - 1) / kKB;
  auto count = [&](int tm, int tn) {
    const int64_t m = a.offsets ? a.M / tm + (a.G + 1) / 2 : (a.M + tm - 1) / tm;
    return m * ((a.N + tn - 1) / tn);
  };
  auto large_us = [&](int64_t w) { return w ? (0.78f + 0.12f * w / 256) * stages + 7.0f : 0.0f; };
  auto medium_us = [&](int64_t w) { return w ? (w > 256 ? 0.58f : 0.42f) * stages + 6.0f : 0.0f; };
  const int64_t l = count(Large::TM, Large::TN), m = count(Medium::TM, Medium::TN);
  return m / 512 * medium_us(512) + medium_us(m % 512) < l / 256 * large_us(256) + large_us(l % 256);
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
  if (M < 0 || M > (1 << 24) || N < 1 || N > (1 << 20) || K < 16 || K > (1 << 22) || K % 16) return MOE_ERR_SHAPE;
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
  else if (a.out_fp32) launch_shape<Medium, true>(st, a);
  else if (medium(a)) launch_shape<Medium, false>(st, a);
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
  if (a->ld < p->depth || a->ld % 16 || a->ld > MOE_FP8_MAX_LD || !aligned16(a->base)) return MOE_ERR_LAYOUT;
  if (b->ld < p->depth || b->ld % 16 || b->ld > MOE_FP8_MAX_LD || !aligned16(b->base)) return MOE_ERR_LAYOUT;
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

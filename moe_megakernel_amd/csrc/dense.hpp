// Dense BF16 matrix products on gfx950 matrix cores: the core of the feed-forward block.
//
// A tile is TM x TN of the result, each wave a block of MI x NJ 16x16 accumulators.  Operands
// come through LDS by the load unit's own copies, NS stages of 32 K elements in a ring (rows of 64 bytes, or K
// rows of the tile's width read with the transposing reads; 16-byte chunks swizzled so that neither copies nor
// reads collide on banks).  A stage's fragments are read while the one before multiplies, so one wave a SIMD with a
// 128 x 128 block is enough.  That block is what the LDS rate asks for: per stage and
// 256 x 256 tile, the four waves read 64 KB, which leaves them most of the time to multiply.
//
// The instruction is the 16 x 16 x 32 one.  On random values the card is held by its power, and registers alone
// multiply at 1885 TFLOP/s with it, at 1617 with 32 x 32 x 16 (one wave a SIMD; on zeros 2327 and 2117).
#pragma once
#include "gemm.hpp"

namespace moe {
namespace dense {

using namespace gemm;

// A wave's 16 x 16 blocks.  B is the instruction's first operand, so lane (r = lane % 16, q = lane / 16) of block
// (i, j) holds row 16 i + r of the wave's rows and its columns 16 j + 4 q .. + 3.
template <class TL>
struct Blocks {
  static constexpr int MI = TL::WMR / 16, NJ = TL::WNC / 16;
};
template <class TL>
using Sums = f32x4_t[Blocks<TL>::MI][Blocks<TL>::NJ];

// K-contiguous stages, rows of 64 bytes.  A 16-byte read of 64 lanes takes four clocks of 256 bytes, and a clock serves
// lanes 0-3, 12-15, 20-23 and 24-27 (or 4-7, 8-11, 16-19 and 28-31; the same 32 on): of 16 rows' chunk 0 and 1 some
// each, which this puts in different places (290 B/ns a CU with (r >> 2) & 3, 570 without collisions).
__device__ __forceinline__ int swz_rows(int r) { return ((r >> 1) & 2) ^ ((r >> 3) & 1 ? 3 : 0); }

// Row-contiguous stages: a transposing read takes 32 bytes of 4 k rows for each of two groups 8 rows apart at once,
// which this moves to eight different places of 256 bytes.
__device__ __forceinline__ int swz_rc(int k) { return ((k & 3) << 2) | ((k >> 2) & 2); }

// An operand of tile_product: `p` its element (tile row 0, K = 0), rows `ld` bytes apart (64 rows, and a KC
// tile's rows, span less than 2^32 bytes), `rows` > 0 tile rows exist (RC: a multiple of 8).
//  KC: consecutive K, rows of the tile `ld` apart; RC: consecutive tile rows, K `ld` apart;
//  KC2: as KC, 32 rows of one matrix and 32 of a second one (p2, ld2) in turn; rows counts both.
struct Operand {
  const uint16_t* p;
  int64_t ld;
  int rows;
  const uint16_t* p2 = nullptr;
  int64_t ld2 = 0;
};
constexpr int KC2 = 2;

// acc += A[TM x K] B[TN x K]^T.  Tile rows past the last repeat it (their results are not used).  With a KC operand
// K is a multiple of the stage; with two RC ones the last stage's k past K are zeros.
template <class TL, int AM, int BM>
__device__ __forceinline__ void tile_product(Sums<TL>& acc, int kdim, const Operand& A, const Operand& B, uint8_t* lds) {
  constexpr int KB = TL::KB, KST = KB / 2, NS = TL::NS;
  constexpr int MI = Blocks<TL>::MI, NJ = Blocks<TL>::NJ;
  constexpr int RBA = TL::TM * 2, RBB = TL::TN * 2;       // bytes of a row-contiguous stage row
  constexpr int LPS = TL::A_DMA + TL::B_DMA;              // copies a stage and wave
  static_assert(KST == 32 && TL::NSB == NS && TL::PF == 0 && NS >= 3, "a stage is one K step");
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = w / TL::NWN, wn = w % TL::NWN;
  const uint32_t lds0 = lds_off(lds);
  const int nk = (kdim + KST - 1) / KST;
  if (nk == 0) return;

  // the lane's offset of each copy from the stage's first byte, and (RC) its k within the stage
  uint32_t oa[TL::A_DMA], ob[TL::B_DMA];
  auto rc_k = [&](int copy, int rb) { return (copy * 1024 + 16 * lane) / rb; };
  auto setup = [&](auto mode, int dma, int rb, const Operand& X, uint32_t* o) __attribute__((always_inline)) {
    for (int i = 0; i < dma; ++i) {
      const int off = (w * dma + i) * 1024 + 16 * lane;
      if constexpr (decltype(mode)::value == KC) {
        const int r = off / KB, c = ((off % KB) >> 4) ^ swz_rows(r);
        o[i] = (uint32_t)(min(r, X.rows - 1) * X.ld) + 16 * c;
      } else if constexpr (decltype(mode)::value == KC2) {
        const int r = off / KB, c = ((off % KB) >> 4) ^ swz_rows(r);
        o[i] = (uint32_t)(min((r >> 6) * 32 + (r & 31), X.rows / 2 - 1) * ((r >> 5) & 1 ? X.ld2 : X.ld)) + 16 * c;
      } else {
        const int k = off / rb, c = ((off % rb) >> 4) ^ swz_rc(k);
        o[i] = (uint32_t)(k * X.ld) + 16 * min(c, X.rows / 8 - 1);
      }
    }
  };
  using MA = std::integral_constant<int, AM>;
  using MB = std::integral_constant<int, BM>;
  setup(MA{}, TL::A_DMA, RBA, A, oa);
  setup(MB{}, TL::B_DMA, RBB, B, ob);
  const uint8_t *ga = reinterpret_cast<const uint8_t*>(A.p), *gb = reinterpret_cast<const uint8_t*>(B.p);   // the next stage's
  const uint8_t* gb2 = reinterpret_cast<const uint8_t*>(B.p2);
  const int64_t sa = AM == RC ? KST * A.ld : KB, sb = BM == RC ? KST * B.ld : KB;
  static_assert(AM != KC2, "the second operand may come from two matrices");
  int put = 0;                                              // its slot in the ring
  // copy i of the stage, A's first
  auto copy = [&](int i) __attribute__((always_inline)) {
    if (i < TL::A_DMA) {
      dma16s(ga, oa[i], lds0 + put * TL::A_BYTES + (w * TL::A_DMA + i) * 1024);
    } else {
      constexpr int kCopies = 32 * KB / 1024;   // of 32 rows
      const int c = w * TL::B_DMA + i - TL::A_DMA;
      dma16s(BM == KC2 && ((c / kCopies) & 1) ? gb2 : gb, ob[i - TL::A_DMA],
             lds0 + NS * TL::A_BYTES + put * TL::B_BYTES + c * 1024);
    }
  };
  auto advance = [&]() __attribute__((always_inline)) {
    ga += sa;
    gb += sb;
    if constexpr (BM == KC2) gb2 += sb;
    put = put + 1 == NS ? 0 : put + 1;
  };
  const int left = kdim - (nk - 1) * KST;                   // k of the last stage
  auto issue = [&](int kt) __attribute__((always_inline)) {
    if (AM == RC && BM == RC && kt == nk - 1) {             // rows past K repeat the last one
#pragma unroll
      for (int i = 0; i < TL::A_DMA; ++i) oa[i] -= (uint32_t)(max(rc_k(w * TL::A_DMA + i, RBA) - left + 1, 0) * A.ld);
#pragma unroll
      for (int i = 0; i < TL::B_DMA; ++i) ob[i] -= (uint32_t)(max(rc_k(w * TL::B_DMA + i, RBB) - left + 1, 0) * B.ld);
    }
#pragma unroll
    for (int i = 0; i < LPS; ++i) copy(i);
    advance();
  };

  const int r16 = lane & 15, q4 = lane >> 4;
  // A's fragments are replaced one by one as the stage uses them, B's are used to its end
  bf16x8_t fa[MI], fb[2][NJ];
  // One 16-row fragment from a stage's operand tile, tile rows from r0: the lane's 8 elements from 8 q4 of row r16.
  auto frag = [&](auto mode, const uint8_t* tile, int rb, int r0) __attribute__((always_inline)) {
    if constexpr (decltype(mode)::value != RC) {
      const int r = r0 + r16;
      return *reinterpret_cast<const bf16x8_t*>(tile + r * KB + ((q4 ^ swz_rows(r16)) << 4));
    } else {
      i16x4_t h[2];
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const int k = 8 * q4 + 4 * hh + (r16 >> 2);
        const int byte = 2 * (r0 + 4 * (r16 & 3));
        h[hh] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (lds_i16x4*)((lds_u8*)tile + k * rb + ((((byte >> 4) ^ swz_rc(k)) << 4) | (byte & 15))));
      }
      return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7));
    }
  };
  auto load_a = [&](int slot, int i) __attribute__((always_inline)) {
    fa[i] = frag(MA{}, lds + slot * TL::A_BYTES, RBA, wm * TL::WMR + i * 16);
  };
  auto load_b = [&](int slot, int j, int to) __attribute__((always_inline)) {
    fb[to][j] = frag(MB{}, lds + NS * TL::A_BYTES + slot * TL::B_BYTES, RBB, wn * TL::WNC + j * 16);
  };
  auto mma = [&](int i, int with) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[with][j], fa[i], acc[i][j], 0, 0, 0);
  };

  // Stage kt multiplies from registers.  Its first act is the barrier that opens stage kt + 1 (whose copies have
  // landed by then, those of up to NS - 2 stages after it may fly) and with it frees slot kt % NS, whose
  // fragments every wave has: stage kt + NS goes there, and the next fragments are read, both spread over
  // the products, since the load unit takes 16 clocks a copy and a wave that waits for it multiplies nothing.
  // The steady loop has no branch: products touch no memory, so the compiler would move them past branches
  // and barriers to where their results are used.
  auto steady = [&](int next, int now) __attribute__((always_inline)) {
    wait_vm<(NS - 2) * LPS>();
    __syncthreads();
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int c = i * LPS / MI; c < (i + 1) * LPS / MI; ++c) copy(c);
      // B's first, which the next stage's first products need
#pragma unroll
      for (int j = 2 * i; j < min(2 * i + 2, NJ); ++j) load_b(next, j, now ^ 1);
      mma(i, now);
      load_a(next, i);
    }
    __builtin_amdgcn_sched_barrier(0);
    advance();
  };
  static_assert(NJ <= 2 * MI, "two of B's fragments with each of A's");
  // the last NS + 2 stages; behind the last one nothing waits and what is read is not used
  auto any = [&](int kt, int next) __attribute__((always_inline)) {
    const int later = min(NS - 2, nk - 2 - kt);
    static_assert(NS <= 5 && 3 * LPS < 64, "counted waits");
    if (later == 3) wait_vm<3 * LPS>();
    else if (later == 2) wait_vm<2 * LPS>();
    else if (later == 1) wait_vm<LPS>();
    else wait_vm<0>();
    __syncthreads();
    if (kt + NS < nk) issue(kt + NS);
#pragma unroll
    for (int j = 0; j < NJ; ++j) load_b(next, j, 1);
    if (AM == RC && BM == RC && kt == nk - 1 && left < KST) {   // and count as zeros
      u32x4_t keep;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int k = 8 * q4 + 2 * e;
        keep[e] = (k < left ? 0xffffu : 0u) | (k + 1 < left ? 0xffff0000u : 0u);
      }
#pragma unroll
      for (int i = 0; i < MI; ++i) fa[i] = __builtin_bit_cast(bf16x8_t, __builtin_bit_cast(u32x4_t, fa[i]) & keep);
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        fb[0][j] = __builtin_bit_cast(bf16x8_t, __builtin_bit_cast(u32x4_t, fb[0][j]) & keep);
    }
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      mma(i, 0);
      load_a(next, i);
    }
  };

#pragma unroll 1
  for (int kt = 0; kt < min(NS, nk); ++kt) issue(kt);
  if (nk >= NS) wait_vm<(NS - 1) * LPS>();
  else wait_vm<0>();
  __syncthreads();
#pragma unroll
  for (int j = 0; j < NJ; ++j) load_b(0, j, 0);
#pragma unroll
  for (int i = 0; i < MI; ++i) load_a(0, i);
  auto after = [](int s) { return s + 1 == NS ? 0 : s + 1; };
  int kt = 0, s = after(0);
  for (; kt + NS + 2 < nk; kt += 2) {      // both stages issued here are whole
    steady(s, 0);
    s = after(s);
    steady(s, 1);
    s = after(s);
  }
  for (; kt < nk; ++kt) {
    any(kt, s);
#pragma unroll
    for (int j = 0; j < NJ; ++j) fb[0][j] = fb[1][j];
    s = after(s);
  }
}

// Code that runs once a tile is kept short (here and below by loops that are not unrolled, and by zeros from the
// matrix unit, 64 instructions instead of 256): a workgroup fetches it anew, at about 60 ns for each 64
// bytes.  (Zeros that the compiler knows as such have the register allocator move accumulators about in the loop.)
template <class TL>
__device__ __forceinline__ void zero(Sums<TL>& acc) {
  u32x4_t z{0u, 0u, 0u, 0u};
  asm volatile("" : "+v"(z));
  const bf16x8_t f = __builtin_bit_cast(bf16x8_t, z);
#pragma unroll
  for (int i = 0; i < Blocks<TL>::MI; ++i)
#pragma unroll
    for (int j = 0; j < Blocks<TL>::NJ; ++j)
      acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f, f, f32x4_t{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0);
}

// Tile of a block: the blocks that one XCD receives (blockIdx % 8) walk a contiguous eighth of the
// tiles, in bands of kBandM m-tiles, m fastest: an XCD's 32 CUs then share about 8 row panels and
// 4 column panels in its L2.
struct TileAt {
  int m, n, part;
  bool ok;
};
// With a split contraction the parts are walked one after the other.
__device__ __forceinline__ TileAt tile_at(int mt, int nt, int split = 1) {
  const int total = mt * nt * split, x = blockIdx.x & 7, j = blockIdx.x >> 3;
  const int t0 = (int)((int64_t)total * x / 8), t1 = (int)((int64_t)total * (x + 1) / 8);
  TileAt t{0, 0, 0, j < t1 - t0};
  if (!t.ok) return t;
  t.part = (t0 + j) / (mt * nt);
  const int L = t0 + j - t.part * mt * nt;
  const int band = L / (kBandM * nt), r = L - band * kBandM * nt, h = min(kBandM, mt - band * kBandM);
  t.n = r / h;
  t.m = band * kBandM + r % h;
  return t;
}
inline unsigned tile_grid(int64_t tiles) { return (unsigned)((tiles + 7) / 8 * 8 + 8); }

// A contraction split over `n` workgroups a tile: their sums, [n][rows][cols] of the whole result, which a second kernel
// adds up.  (The last workgroup of a tile to do that itself, as the layer's kernels for a few tokens have it, keeps the
// registers of these tiles from fitting.)
struct Split {
  float* sums;
  int n;
};
// First stage of a part.
__device__ __forceinline__ int part_begin(int stages, int part, int n) { return (int)((int64_t)stages * part / n); }

// The tile's sums to their part's, from `to` (row 0, column 0 of the tile), rows ld apart.  PAIR: gate and up columns
// alternate in 32s; the up ones' sums lie `up` on.
template <class TL, bool PAIR>
__device__ __forceinline__ void leave(const Sums<TL>& acc, float* to, int64_t ld, int rows, int cols, int up) {
  const int lane = threadIdx.x & 63, r0 = wave_m<TL>() * TL::WMR + (lane & 15), c0 = wave_n<TL>() * TL::WNC + 4 * (lane >> 4);
#pragma unroll
  for (int i = 0; i < Blocks<TL>::MI; ++i) {
    if (r0 + 16 * i >= rows) continue;
    float* line = to + (int64_t)(r0 + 16 * i) * ld;
#pragma unroll
    for (int j = 0; j < Blocks<TL>::NJ; ++j) {
      const int c = c0 + 16 * j, col = PAIR ? (c >> 6) * 32 + (c & 31) : c;
      if (col < cols) *reinterpret_cast<f32x4_t*>(line + col + (PAIR && ((c >> 5) & 1) ? up : 0)) = acc[i][j];
    }
  }
}

// Hands the accumulators out through LDS, a wave row at a time, so that a lane has 8
// neighbouring columns: f(row, col, v, q) for row < rows, col < cols.  PAIR: gate and up columns
// alternate in 32s, f(row, col, g, u, q) with col < cols of the tile's TN / 2 pairs.  q = pre(row, col) is what the
// lane needs from memory besides, asked for kAhead pieces before.  LDS row r holds 16-byte chunk c at
// c ^ (r % 16), so that the 16 rows a wave writes at once fall in disjoint banks.
struct Nothing {};
template <class TL, bool PAIR, class PRE, class F>
__device__ __forceinline__ void each_piece(const Sums<TL>& acc, uint8_t* lds, int rows, int cols, const PRE& pre, const F& f) {
  constexpr int PPR = PAIR ? TL::TN / 16 : TL::TN / 8, PPT = TL::WMR * PPR / TL::NTH;
  constexpr int kAhead = PPT % 8 == 0 ? 4 : PPT % 6 == 0 ? 3 : PPT / 2, RPP = TL::NTH / PPR;   // rows a pass of the workgroup
  static_assert(TL::WMR * TL::TN * 4 <= TL::LDS && TL::NTH % PPR == 0 && PPT % (2 * kAhead) == 0, "epilogue round");
  float* ct = reinterpret_cast<float*>(lds);
  const int t = threadIdx.x, lane = t & 63, wm = wave_m<TL>(), wn = wave_n<TL>();
  const int row0 = t / PPR, col = 8 * (t % PPR), c0 = PAIR ? (col >> 5) * 64 + (col & 31) : col;
  using Q = decltype(pre(0, 0));
  // piece p of the thread: row row0 + p RPP
  auto ask = [&](int p, Q (&q)[kAhead]) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int row = row0 + (p + u) * RPP;
      if (row < rows && col < cols) q[u] = pre(row, col);
    }
  };
  auto give = [&](int p, int first, const Q (&q)[kAhead]) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int row = row0 + (p + u) * RPP, r = row - first;
      if (row >= rows || col >= cols) continue;
      const float* line = ct + r * TL::TN;
      auto get8 = [&](int c, float* v) __attribute__((always_inline)) {
        const f32x4_t x0 = *reinterpret_cast<const f32x4_t*>(line + (((c >> 2) ^ (r & 15)) << 2));
        const f32x4_t x1 = *reinterpret_cast<const f32x4_t*>(line + ((((c >> 2) + 1) ^ (r & 15)) << 2));
#pragma unroll
        for (int k = 0; k < 4; ++k) { v[k] = x0[k]; v[4 + k] = x1[k]; }
      };
      float v[8];
      get8(c0, v);
      if constexpr (PAIR) {
        float w[8];
        get8(c0 + 32, w);
        f(row, col, v, w, q[u]);
      } else {
        f(row, col, v, q[u]);
      }
    }
  };
  Q qa[kAhead] = {}, qb[kAhead] = {};
  ask(0, qa);
  int p = 0;
#pragma unroll 1
  for (int k = 0; k < TL::NWM; ++k) {
    __syncthreads();                       // the stages, or the round before, have been read
    if (wm == k) {
#pragma unroll
      for (int i = 0; i < Blocks<TL>::MI; ++i)
#pragma unroll
        for (int j = 0; j < Blocks<TL>::NJ; ++j) {
          const int r = i * 16 + (lane & 15), c = (wn * TL::WNC + j * 16) / 4 + (lane >> 4);
          *reinterpret_cast<f32x4_t*>(ct + r * TL::TN + ((c ^ (r & 15)) << 2)) = acc[i][j];
        }
    }
    __syncthreads();
#pragma unroll 1
    for (int e = 0; e < PPT; e += 2 * kAhead, p += 2 * kAhead) {
      ask(p + kAhead, qb);
      give(p, k * TL::WMR, qa);
      ask(p + 2 * kAhead, qa);
      give(p + kAhead, k * TL::WMR, qb);
    }
  }
}

}  // namespace dense
}  // namespace moe

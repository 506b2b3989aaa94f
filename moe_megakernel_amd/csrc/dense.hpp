// Dense BF16 matrix products on gfx950 matrix cores: the core of the feed-forward block.
//
// A tile is TM x TN of the result, each wave a block of MI x NJ 32x32 accumulators.  Operands
// come through LDS by the load unit's own copies (gemm.hpp: stage layout, swizzles, transposing
// reads), NS stages in a ring.  What differs from the grouped products there is the order of
// a stage: the fragments of K step ks + 1 are read while step ks multiplies, and the
// last step of a stage multiplies behind the barrier that opens the next one, whose first
// fragments and copies then start under it.  So neither the barrier nor the first LDS reads of a stage
// leave the matrix unit idle, and one wave a SIMD with a 128 x 128 block is enough.  That block is
// what the LDS rate asks for: per stage of 64 K elements and 256 x 256 tile, the four waves
// read 128 KB and the copies write 64 KB, 1536 cycles at 128 bytes a clock, against 2048 cycles
// of multiplying (eight waves of 128 x 64 read 192 KB, 2048 cycles).
#pragma once
#include "gemm.hpp"

namespace moe {
namespace dense {

using namespace gemm;

// LDS copy with a uniform base and a 32-bit offset a lane: no vector instruction moves the address on.
__device__ __forceinline__ void dma16s(const uint8_t* base, uint32_t off, uint32_t m0v) {
  const uint32_t m = __builtin_amdgcn_readfirstlane(m0v);
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" : : "v"(off), "s"(base), "s"(m)
               : "memory", "m0");
}

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
__device__ __forceinline__ void tile_product(Acc<TL>& acc, int kdim, const Operand& A, const Operand& B, uint8_t* lds) {
  constexpr int KB = TL::KB, KST = KB / 2, NKS = KST / 16, NS = TL::NS;
  constexpr int RBA = TL::TM * 2, RBB = TL::TN * 2;       // bytes of a row-contiguous stage row
  constexpr int LPS = TL::A_DMA + TL::B_DMA;              // copies a stage and wave
  static_assert(NKS % 2 == 0 && TL::NSB == NS && TL::PF == 0, "stage shape");
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
        const int r = off / KB, c = ((off % KB) >> 4) ^ swz_kc<KB>(r);
        o[i] = (uint32_t)(min(r, X.rows - 1) * X.ld) + 16 * c;
      } else if constexpr (decltype(mode)::value == KC2) {
        const int r = off / KB, c = ((off % KB) >> 4) ^ swz_kc<KB>(r);
        o[i] = (uint32_t)(min((r >> 6) * 32 + (r & 31), X.rows / 2 - 1) * ((r >> 5) & 1 ? X.ld2 : X.ld)) + 16 * c;
      } else {
        const int k = off / rb, c = ((off % rb) >> 4) ^ swz_rc16(k);
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
  auto issue = [&]() __attribute__((always_inline)) {
    const uint32_t la = lds0 + put * TL::A_BYTES, lb = lds0 + NS * TL::A_BYTES + put * TL::B_BYTES;
#pragma unroll
    for (int i = 0; i < TL::A_DMA; ++i) dma16s(ga, oa[i], la + (w * TL::A_DMA + i) * 1024);
#pragma unroll
    for (int i = 0; i < TL::B_DMA; ++i) {
      constexpr int kCopies = 32 * KB / 1024;   // of 32 rows
      const bool second = BM == KC2 && (((w * TL::B_DMA + i) / kCopies) & 1);
      dma16s(second ? gb2 : gb, ob[i], lb + (w * TL::B_DMA + i) * 1024);
    }
    ga += sa;
    gb += sb;
    if constexpr (BM == KC2) gb2 += sb;
    put = put + 1 == NS ? 0 : put + 1;
  };
  // the last stage, which may end early
  auto issue_last = [&]() __attribute__((always_inline)) {
    const int left = kdim - (nk - 1) * KST;
    if (AM != RC || BM != RC || left == KST) {
      issue();
      return;
    }
    const uint32_t la = lds0 + put * TL::A_BYTES, lb = lds0 + NS * TL::A_BYTES + put * TL::B_BYTES;
    const uint8_t* zp = reinterpret_cast<const uint8_t*>(g_zero_page) + 16 * lane;
    for (int i = 0; i < TL::A_DMA; ++i) dma16(rc_k(w * TL::A_DMA + i, RBA) < left ? ga + oa[i] : zp, la + (w * TL::A_DMA + i) * 1024);
    for (int i = 0; i < TL::B_DMA; ++i) dma16(rc_k(w * TL::B_DMA + i, RBB) < left ? gb + ob[i] : zp, lb + (w * TL::B_DMA + i) * 1024);
  };

  const int g = lane >> 5, grp = lane >> 4, j16 = lane & 15;
  struct Frags {
    bf16x8_t a[TL::MI], b[TL::NJ];
  };
  // one 32-row fragment of K step ks from a stage's operand tile, tile rows from r0
  auto frag = [&](auto mode, const uint8_t* tile, int rb, int r0, int ks) __attribute__((always_inline)) {
    if constexpr (decltype(mode)::value != RC) {
      const int r = r0 + (lane & 31);
      return *reinterpret_cast<const bf16x8_t*>(tile + r * KB + (((2 * ks + g) ^ swz_kc<KB>(r)) << 4));
    } else {
      const int m0 = r0 + 16 * (grp & 1);
      i16x4_t h[2];
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        const int k = 16 * ks + 8 * (grp >> 1) + 4 * hh + (j16 >> 2);
        const int byte = 2 * (m0 + 4 * (j16 & 3));
        h[hh] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (lds_i16x4*)((lds_u8*)tile + k * rb + ((((byte >> 4) ^ swz_rc16(k)) << 4) | (byte & 15))));
      }
      return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(h[0], h[1], 0, 1, 2, 3, 4, 5, 6, 7));
    }
  };
  auto load = [&](int slot, int ks, Frags& f) __attribute__((always_inline)) {
    const uint8_t* At = lds + slot * TL::A_BYTES;
    const uint8_t* Bt = lds + NS * TL::A_BYTES + slot * TL::B_BYTES;
#pragma unroll
    for (int j = 0; j < TL::NJ; ++j) f.b[j] = frag(MB{}, Bt, RBB, wn * TL::WNC + j * 32, ks);
#pragma unroll
    for (int i = 0; i < TL::MI; ++i) f.a[i] = frag(MA{}, At, RBA, wm * TL::WMR + i * 32, ks);
  };
  auto mma = [&](const Frags& f) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < TL::MI; ++i)
#pragma unroll
      for (int j = 0; j < TL::NJ; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.a[i], f.b[j], acc[i][j], 0, 0, 0);
  };

  for (int s = 0; s < min(NS - 1, nk - 1); ++s) issue();
  if (nk < NS) {
    issue_last();
    wait_vm<0>();
  } else {
    wait_vm<(NS - 2) * LPS>();
  }
  __syncthreads();
  Frags f[2];
  int slot = 0;
  load(0, 0, f[0]);
  // A stage: its first fragments are on their way.  Its copies go to the slot of the stage before, which every
  // wave has read by the barrier that opened this one; that of the next stage waits for its copies, those of
  // FLY stages after it may fly.  The steady loop has no branch: products touch no memory, so the compiler would
  // move them past branches and barriers to where their results are used.
  auto stage = [&](auto what, auto fly) __attribute__((always_inline)) {
    const int next = slot + 1 == NS ? 0 : slot + 1;
    if constexpr (decltype(what)::value == 0) issue();
    if constexpr (decltype(what)::value == 1) issue_last();
#pragma unroll
    for (int ks = 0; ks < NKS; ++ks) {
      __builtin_amdgcn_sched_barrier(0);
      if (ks + 1 < NKS) {
        load(slot, ks + 1, f[(ks + 1) & 1]);
      } else if constexpr (decltype(what)::value != 3) {
        wait_vm<decltype(fly)::value * LPS>();
        __syncthreads();
        __builtin_amdgcn_sched_barrier(0);
        load(next, 0, f[0]);
      }
      mma(f[ks & 1]);
    }
    slot = next;
  };
  using std::integral_constant;
  for (int kt = 0; kt < nk - NS; ++kt) stage(integral_constant<int, 0>{}, integral_constant<int, NS - 2>{});
  if (nk >= NS) stage(integral_constant<int, 1>{}, integral_constant<int, NS - 2>{});
  for (int kt = max(nk - NS + 1, 0); kt < nk - 1; ++kt) stage(integral_constant<int, 2>{}, integral_constant<int, 0>{});
  stage(integral_constant<int, 3>{}, integral_constant<int, 0>{});
}

// Tile of a block: the blocks that one XCD receives (blockIdx % 8) walk a contiguous eighth of the
// tiles, in bands of kBandM m-tiles, m fastest: an XCD's 32 CUs then share about 8 row panels and
// 4 column panels in its L2.
struct TileAt {
  int m, n;
  bool ok;
};
__device__ __forceinline__ TileAt tile_at(int mt, int nt) {
  const int total = mt * nt, x = blockIdx.x & 7, j = blockIdx.x >> 3;
  const int t0 = (int)((int64_t)total * x / 8), t1 = (int)((int64_t)total * (x + 1) / 8);
  TileAt t{0, 0, j < t1 - t0};
  if (!t.ok) return t;
  const int L = t0 + j, band = L / (kBandM * nt), r = L - band * kBandM * nt, h = min(kBandM, mt - band * kBandM);
  t.n = r / h;
  t.m = band * kBandM + r % h;
  return t;
}
inline unsigned tile_grid(int64_t tiles) { return (unsigned)((tiles + 7) / 8 * 8 + 8); }

// Hands the accumulators out through LDS, a wave row at a time, so that a lane has 8
// neighbouring columns: f(row, col, v) for row < rows, col < cols.  PAIR: gate and up columns
// alternate in 32s, f(row, col, g, u) with col < cols of the tile's TN / 2 pairs.  LDS row r
// holds 16-byte chunk c at c ^ 8 ((r >> 2) & 1), so that the two row groups a wave writes at once
// fall in disjoint banks.
template <class TL, bool PAIR, class F>
__device__ __forceinline__ void each_piece(const Acc<TL>& acc, uint8_t* lds, int rows, int cols, const F& f) {
  constexpr int PPR = PAIR ? TL::TN / 16 : TL::TN / 8, PPT = TL::WMR * PPR / TL::NTH;
  static_assert(TL::WMR * TL::TN * 4 <= TL::LDS && (TL::WMR * PPR) % TL::NTH == 0, "epilogue round");
  float* ct = reinterpret_cast<float*>(lds);
  const int t = threadIdx.x, lane = t & 63, wm = wave_m<TL>(), wn = wave_n<TL>();
  auto sw = [](int r) { return ((r >> 2) & 1) << 3; };
  auto get8 = [&](int r, int c0, float* v) __attribute__((always_inline)) {
    const float* p = ct + r * TL::TN;
    const f32x4_t x0 = *reinterpret_cast<const f32x4_t*>(p + (((c0 >> 2) ^ sw(r)) << 2));
    const f32x4_t x1 = *reinterpret_cast<const f32x4_t*>(p + ((((c0 >> 2) + 1) ^ sw(r)) << 2));
#pragma unroll
    for (int k = 0; k < 4; ++k) { v[k] = x0[k]; v[4 + k] = x1[k]; }
  };
#pragma unroll
  for (int q = 0; q < TL::NWM; ++q) {
    if (q * TL::WMR >= rows) break;
    __syncthreads();
    if (wm == q) {
#pragma unroll
      for (int i = 0; i < TL::MI; ++i)
#pragma unroll
        for (int j = 0; j < TL::NJ; ++j)
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const int row = i * 32 + (r >> 2) * 8 + (lane >> 5) * 4 + (r & 3), col = acc_col<TL>(wn, j, lane);
            ct[row * TL::TN + (((col >> 2) ^ sw(row)) << 2) + (col & 3)] = acc[i][j][r];
          }
    }
    __syncthreads();
#pragma unroll 2
    for (int u = 0; u < PPT; ++u) {
      const int pi = u * TL::NTH + t, row = pi / PPR, col = 8 * (pi % PPR), trow = q * TL::WMR + row;
      if (trow >= rows || col >= cols) continue;
      if constexpr (PAIR) {
        const int c0 = (col >> 5) * 64 + (col & 31);
        float g[8], v[8];
        get8(row, c0, g);
        get8(row, c0 + 32, v);
        f(trow, col, g, v);
      } else {
        float v[8];
        get8(row, col, v);
        f(trow, col, v);
      }
    }
  }
}

}  // namespace dense
}  // namespace moe

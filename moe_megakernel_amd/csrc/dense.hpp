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

// acc += A[TM x K] B[TN x K]^T.
//  KC operand: f(r) -> bytes of tile row r at K = 0, called for r < rows (the others are zero);
//              K is then a multiple of the stage.
//  RC operand: f(k) -> bytes of element (k, tile row 0), called for k < kdim; tile rows at or past
//              rows (a multiple of 8) are zero.
template <class TL, int AM, int BM, class FA, class FB>
__device__ __forceinline__ void tile_product(Acc<TL>& acc, int kdim, const FA& fa, int arows, const FB& fb, int brows,
                                             uint8_t* lds) {
  constexpr int KB = TL::KB, KST = KB / 2, NKS = KST / 16, NS = TL::NS;
  constexpr int RBA = TL::TM * 2, RBB = TL::TN * 2;       // bytes of a row-contiguous stage row
  constexpr int LPS = TL::A_DMA + TL::B_DMA;              // copies a stage and wave
  static_assert(NKS % 2 == 0 && TL::NSB == NS && TL::PF == 0, "stage shape");
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = w / TL::NWN, wn = w % TL::NWN;
  const uint32_t lds0 = lds_off(lds);
  const uint8_t* zp = reinterpret_cast<const uint8_t*>(g_zero_page) + 16 * lane;
  const int nk = (kdim + KST - 1) / KST;
  if (nk == 0) return;

  // the lane's source of each copy: KC: a pointer that moves KB a stage (or stays, on zeros); RC:
  // the row within the stage and the byte inside it
  const uint8_t *pa[TL::A_DMA], *pb[TL::B_DMA];
  int ka[TL::A_DMA], kb[TL::B_DMA], ca[TL::A_DMA], cb[TL::B_DMA];
  auto setup = [&](auto mode, int dma, int rb, const auto& f, int rows, const uint8_t** p, int* kr, int* cr)
                   __attribute__((always_inline)) {
    for (int i = 0; i < dma; ++i) {
      const int off = (w * dma + i) * 1024 + 16 * lane;
      if constexpr (decltype(mode)::value == KC) {
        const int r = off / KB, c = ((off % KB) >> 4) ^ swz_kc<KB>(r);
        p[i] = r < rows ? reinterpret_cast<const uint8_t*>(f(r)) + 16 * c : zp;
        kr[i] = r < rows ? KB : 0;
        cr[i] = 0;
      } else {
        const int k = off / rb, c = ((off % rb) >> 4) ^ swz_rc16(k);
        p[i] = nullptr;
        kr[i] = 8 * c < rows ? k : (1 << 30);
        cr[i] = 16 * c;
      }
    }
  };
  setup(std::integral_constant<int, AM>{}, TL::A_DMA, RBA, fa, arows, pa, ka, ca);
  setup(std::integral_constant<int, BM>{}, TL::B_DMA, RBB, fb, brows, pb, kb, cb);

  auto issue = [&](int kt) __attribute__((always_inline)) {
    const uint32_t sa = lds0 + (kt % NS) * TL::A_BYTES;
    const uint32_t sb = lds0 + NS * TL::A_BYTES + (kt % NS) * TL::B_BYTES;
#pragma unroll
    for (int i = 0; i < TL::A_DMA; ++i) {
      const uint32_t m0v = sa + (w * TL::A_DMA + i) * 1024;
      if constexpr (AM == KC) {
        dma16(pa[i], m0v);
        pa[i] += ka[i];
      } else {
        const int k = kt * KST + ka[i];
        dma16(k < kdim ? reinterpret_cast<const uint8_t*>(fa(k)) + ca[i] : zp, m0v);
      }
    }
#pragma unroll
    for (int i = 0; i < TL::B_DMA; ++i) {
      const uint32_t m0v = sb + (w * TL::B_DMA + i) * 1024;
      if constexpr (BM == KC) {
        dma16(pb[i], m0v);
        pb[i] += kb[i];
      } else {
        const int k = kt * KST + kb[i];
        dma16(k < kdim ? reinterpret_cast<const uint8_t*>(fb(k)) + cb[i] : zp, m0v);
      }
    }
  };

  const int g = lane >> 5, grp = lane >> 4, j16 = lane & 15;
  struct Frags {
    bf16x8_t a[TL::MI], b[TL::NJ];
  };
  // one 32-row fragment of K step ks from a stage's operand tile, tile rows from r0
  auto frag = [&](auto mode, const uint8_t* tile, int rb, int r0, int ks) __attribute__((always_inline)) {
    if constexpr (decltype(mode)::value == KC) {
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
  auto load = [&](int kt, int ks, Frags& f) __attribute__((always_inline)) {
    const uint8_t* At = lds + (kt % NS) * TL::A_BYTES;
    const uint8_t* Bt = lds + NS * TL::A_BYTES + (kt % NS) * TL::B_BYTES;
#pragma unroll
    for (int j = 0; j < TL::NJ; ++j) f.b[j] = frag(std::integral_constant<int, BM>{}, Bt, RBB, wn * TL::WNC + j * 32, ks);
#pragma unroll
    for (int i = 0; i < TL::MI; ++i) f.a[i] = frag(std::integral_constant<int, AM>{}, At, RBA, wm * TL::WMR + i * 32, ks);
  };
  auto mma = [&](const Frags& f) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < TL::MI; ++i)
#pragma unroll
      for (int j = 0; j < TL::NJ; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.a[i], f.b[j], acc[i][j], 0, 0, 0);
  };
  // waits until stage kt of the wave's copies is in LDS (those of `later` stages may fly)
  auto landed = [&](int later) __attribute__((always_inline)) {
    if (NS >= 4 && later >= 2) wait_vm<NS >= 4 ? 2 * LPS : 0>();
    else if (NS >= 3 && later >= 1) wait_vm<NS >= 3 ? LPS : 0>();
    else wait_vm<0>();
  };

  for (int s = 0; s < NS - 1; ++s)
    if (s < nk) issue(s);
  landed(min(NS - 2, nk - 1));
  __syncthreads();
  Frags f[2];
  load(0, 0, f[0]);
  // Stage kt: its first fragments are on their way.  Its copies' ring slot for stage kt + NS - 1 is
  // that of stage kt - 1, which every wave has read by the barrier that opened stage kt.
  for (int kt = 0; kt < nk - 1; ++kt) {
    if (kt + NS - 1 < nk) issue(kt + NS - 1);
#pragma unroll
    for (int ks = 0; ks < NKS; ++ks) {
      if (ks + 1 < NKS) {
        load(kt, ks + 1, f[(ks + 1) & 1]);
      } else {
        landed(min(NS - 2, nk - 2 - kt));
        __syncthreads();
        load(kt + 1, 0, f[0]);
      }
      mma(f[ks & 1]);
    }
  }
#pragma unroll
  for (int ks = 0; ks < NKS; ++ks) {
    if (ks + 1 < NKS) load(nk - 1, ks + 1, f[(ks + 1) & 1]);
    mma(f[ks & 1]);
  }
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

// Products of a few rows (tokens) with a long matrix, bound by one read of the matrix.
//
// Weights are the 16-row operand of a 16 x 16 matrix instruction, tokens its 16 columns.  A wave runs a
// stretch of the contraction by itself: its rows come in stages of 128 bytes a row by the load
// unit's copies into a ring of its own in LDS, D stages in flight, with no register and no
// barrier between; the waves of a workgroup meet once, to add up their sums.
//
// A copy moves 8 rows of 128 bytes (whole cache lines); 16-byte chunks are swizzled by row, so that the
// fragments' reads (16 rows, one chunk) touch all banks.
#pragma once
#include "gemm.hpp"

namespace moe {
namespace stream {

using namespace gemm;

constexpr int kRowBytes = 128;             // of a stage
constexpr int kTile = 16 * kRowBytes;      // 16 rows

// R weight tiles and NF token tiles of 16 rows, and EX copies of 64 words, a stage.
template <int R, int NF, int EX, int D>
struct Ring {
  static constexpr int kStage = (R + NF) * kTile + EX * 256;
  static constexpr int kBytes = D * kStage;
  static constexpr int kCopies = 2 * (R + NF) + EX;
};

__device__ __forceinline__ const uint8_t* chunk(const uint8_t* tile, int row, int c) {
  return tile + row * kRowBytes + ((c ^ swz_kc<kRowBytes>(row)) << 4);
}

// Runs stages s0 .. s0 + n - 1.  w(r) for r < 16 R, x(c) for c < 16 NF: bytes of a row at the start of the
// contraction, or null for a row of zeros; `bytes` of a row exist (a multiple of 16).  ex(e, s): the lane's
// word of extra copy e of stage s.  mul(weights, tokens, extra): the stage, in LDS.
template <int R, int NF, int EX, int D, class FW, class FX, class FE, class MUL>
__device__ __forceinline__ void run(uint8_t* ring, int s0, int n, int64_t bytes, const FW& w, const FX& x, const FE& ex,
                                    const MUL& mul) {
  using G = Ring<R, NF, EX, D>;
  const int lane = threadIdx.x & 63;
  const uint32_t base = lds_off(ring);
  const uint8_t* zp = reinterpret_cast<const uint8_t*>(g_zero_page) + 16 * lane;
  constexpr int N = 2 * (R + NF);
  const uint8_t* p[N];
  int64_t left[N];                         // bytes from the chunk to the row's end; <= 0: zeros
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int row = 8 * i + (lane >> 3), c = (lane & 7) ^ swz_kc<kRowBytes>(row & 15);
    const uint8_t* q = i < 2 * R ? w(row) : x(row - 16 * R);
    p[i] = q + (int64_t)s0 * kRowBytes + 16 * c;
    left[i] = q ? bytes - ((int64_t)s0 * kRowBytes + 16 * c) : 0;
  }
  auto issue = [&](int s, int slot) __attribute__((always_inline)) {
    const uint32_t at = base + slot * G::kStage;
    const int64_t gone = (int64_t)(s - s0) * kRowBytes;
#pragma unroll
    for (int i = 0; i < N; ++i) dma16(left[i] > gone ? p[i] + gone : zp, at + i * 1024);
#pragma unroll
    for (int e = 0; e < EX; ++e) dma4(ex(e, s), at + (R + NF) * kTile + 256 * e);
  };
#pragma unroll
  for (int d = 0; d < D; ++d)
    if (d < n) issue(s0 + d, d);
  int slot = 0;
  for (int s = 0; s < n; ++s) {
    const int later = min(D - 1, n - 1 - s);   // stages that may still fly
    static_assert(D >= 2 && D <= 4 && (D - 1) * G::kCopies < 64, "vmcnt range");
    if (D >= 4 && later == 3) wait_vm<D >= 4 ? 3 * G::kCopies : 0>();
    else if (D >= 3 && later == 2) wait_vm<D >= 3 ? 2 * G::kCopies : 0>();
    else if (later == 1) wait_vm<G::kCopies>();
    else wait_vm<0>();
    asm volatile("" ::: "memory");
    const uint8_t* st = ring + slot * G::kStage;
    mul(st, st + R * kTile, reinterpret_cast<const float*>(st + (R + NF) * kTile));
    if (s + D < n) {
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the slot has been read
      issue(s0 + s + D, slot);
    }
    slot = slot + 1 == D ? 0 : slot + 1;
  }
}

}  // namespace stream
}  // namespace moe

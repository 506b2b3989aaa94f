// The gated feed-forward block: kernels over tiles of many tokens.
//
//   k_ffn_up     h = act(a) b, a = x gate^T, b = x up^T     both products in one tile, a and b kept
//   k_ffn_rows   out = h down^T; grad_x = da gate + db up
//   k_ffn_dh     dh = dy down; da = dh b act'(a), db = dh act(a), h again
//   k_ffn_wgrad  grad_down (+)= dy^T h; grad_gate, grad_up (+)= da^T x, db^T x
//
// Sums are FP32 (the matrix unit's accumulators).  Rounded to BF16, each once: h (the second
// product's operand; the output's own rounding is as large), a and b where they are kept so, da and
// db (operands again), and the outputs.
#include <hip/hip_runtime.h>

#include "dense.hpp"
#include "ffn.hpp"
#include "ffn_act.hpp"
#include "mxint8.hpp"

namespace moe {
namespace ffn {

using namespace dense;

namespace {

using Large = Tile<256, 256, 2, 2, 4, 1, 0, 64>;
using Medium = Tile<128, 128, 2, 2, 4, 2, 0, 64>;

constexpr auto no_more = [](int, int) { return Nothing{}; };   // an epilogue without operands from memory

__device__ __forceinline__ uint4 pack8(const float* v) {
  return make_uint4(pack_bf2(v[0], v[1]), pack_bf2(v[2], v[3]), pack_bf2(v[4], v[5]), pack_bf2(v[6], v[7]));
}

template <class TL, int ACT, int SAVED>
__global__ __launch_bounds__(TL::NTH, TL::MINB) void k_ffn_up(UpArgs p) {
  static_assert(TL::WNC % 64 == 0, "gate / up pairs in a wave");
  __shared__ __align__(16) uint8_t lds[TL::LDS];
  constexpr int TI = TL::TN / 2;            // columns of h a tile
  const TileAt at = tile_at((p.T + TL::TM - 1) / TL::TM, (p.I + TI - 1) / TI);
  if (!at.ok) return;
  const int m0 = at.m * TL::TM, i0 = at.n * TI, rows = min(TL::TM, p.T - m0), cols = min(TI, p.I - i0);
  Sums<TL> acc;
  zero<TL>(acc);
  // 32 gate rows, 32 up rows in turn: a lane's accumulators of blocks 2j and 2j + 1 are a and b of the
  // same elements; cols is a multiple of 64, so the rows that exist come first
  const Operand x{p.x.p + (int64_t)m0 * p.x.ld, 2 * p.x.ld, rows};
  const Operand w{p.gate.p + (int64_t)i0 * p.gate.ld, 2 * p.gate.ld, 2 * cols,
                  p.up.p + (int64_t)i0 * p.up.ld, 2 * p.up.ld};
  tile_product<TL, KC, KC2>(acc, p.H, x, w, lds);
  each_piece<TL, true>(acc, lds, rows, cols, no_more, [&](int row, int col, const float* a, const float* b, Nothing) {
    const int64_t R = m0 + row;
    const int i = i0 + col;
    float h[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) h[k] = act<ACT>(a[k]) * b[k];
    *reinterpret_cast<uint4*>(p.h.p + R * p.h.ld + i) = pack8(h);
    if constexpr (SAVED == kBf16) {
      uint16_t* ab = reinterpret_cast<uint16_t*>(p.kept.ab) + R * 2 * p.I + i;
      *reinterpret_cast<uint4*>(ab) = pack8(a);
      *reinterpret_cast<uint4*>(ab + p.I) = pack8(b);
    }
    if constexpr (SAVED == kInt8) {   // the four lanes of a quad hold a block of 32
      const float(&av)[8] = *reinterpret_cast<const float(*)[8]>(a);
      const float(&bv)[8] = *reinterpret_cast<const float(*)[8]>(b);
      const int sa = int8_scale_byte(quad_max_u(abs_bits8(av))), sb = int8_scale_byte(quad_max_u(abs_bits8(bv)));
      uint8_t* ab = p.kept.ab + R * 2 * p.I + i;
      *reinterpret_cast<uint2*>(ab) = int8_codes8(av, sa);
      *reinterpret_cast<uint2*>(ab + p.I) = int8_codes8(bv, sb);
      if ((i & 31) == 0) {
        uint8_t* sc = p.kept.scales + R * (p.I / 16) + i / 32;
        sc[0] = (uint8_t)sa;
        sc[p.I / 32] = (uint8_t)sb;
      }
    }
  });
}

// BM = KC: b0 rows are the result's columns (ksplit = K); RC: b0 rows run along K, those of its second half in
// b1 (K = 2 ksplit)
template <class TL, int BM>
__global__ __launch_bounds__(TL::NTH, TL::MINB) void k_ffn_rows(RowsArgs p) {
  __shared__ __align__(16) uint8_t lds[TL::LDS];
  const TileAt at = tile_at((p.T + TL::TM - 1) / TL::TM, (p.N + TL::TN - 1) / TL::TN);
  if (!at.ok) return;
  const int m0 = at.m * TL::TM, n0 = at.n * TL::TN, rows = min(TL::TM, p.T - m0), cols = min(TL::TN, p.N - n0);
  Sums<TL> acc;
  zero<TL>(acc);
  Operand a{p.a.p + (int64_t)m0 * p.a.ld, 2 * p.a.ld, rows};
  Operand b{BM == KC ? p.b0.p + (int64_t)n0 * p.b0.ld : p.b0.p + n0, 2 * p.b0.ld, cols};
  for (int k = 0; k < p.K; k += p.ksplit) {
    if (k > 0) {
      __syncthreads();                       // the first part's stages have been read
      a.p += k;
      b.p = p.b1.p + n0;
      b.ld = 2 * p.b1.ld;
    }
    tile_product<TL, KC, BM>(acc, p.ksplit, a, b, lds);
  }
  each_piece<TL, false>(acc, lds, rows, cols, no_more, [&](int row, int col, const float* v, Nothing) {
    *reinterpret_cast<uint4*>(p.c.p + (int64_t)(m0 + row) * p.c.ld + n0 + col) = pack8(v);
  });
}

template <class TL, int ACT, int SAVED>
__global__ __launch_bounds__(TL::NTH, TL::MINB) void k_ffn_dh(DhArgs p) {
  __shared__ __align__(16) uint8_t lds[TL::LDS];
  const TileAt at = tile_at((p.T + TL::TM - 1) / TL::TM, (p.I + TL::TN - 1) / TL::TN);
  if (!at.ok) return;
  const int m0 = at.m * TL::TM, n0 = at.n * TL::TN, rows = min(TL::TM, p.T - m0), cols = min(TL::TN, p.I - n0);
  Sums<TL> acc;
  zero<TL>(acc);
  tile_product<TL, KC, RC>(acc, p.H, {p.dy.p + (int64_t)m0 * p.dy.ld, 2 * p.dy.ld, rows},
                           {p.down.p + n0, 2 * p.down.ld, cols}, lds);
  // a and b of a piece: 8 BF16 values each, or 8 codes and a scale byte
  struct Saved8 {
    uint4 a, b;
    int sa, sb;
  };
  auto pre = [&](int row, int col) {
    const int64_t R = m0 + row;
    const int i = n0 + col;
    Saved8 q{};
    if constexpr (SAVED == kBf16) {
      const uint16_t* ab = reinterpret_cast<const uint16_t*>(p.kept.ab) + R * 2 * p.I + i;
      q.a = *reinterpret_cast<const uint4*>(ab);
      q.b = *reinterpret_cast<const uint4*>(ab + p.I);
    } else {
      const uint8_t *ab = p.kept.ab + R * 2 * p.I + i, *sc = p.kept.scales + R * (p.I / 16) + i / 32;
      const uint2 a = *reinterpret_cast<const uint2*>(ab), b = *reinterpret_cast<const uint2*>(ab + p.I);
      q.a.x = a.x, q.a.y = a.y, q.b.x = b.x, q.b.y = b.y;
      q.sa = sc[0], q.sb = sc[p.I / 32];
    }
    return q;
  };
  each_piece<TL, false>(acc, lds, rows, cols, pre, [&](int row, int col, const float* dh, const Saved8& q) {
    const int64_t R = m0 + row;
    const int i = n0 + col;
    float a[8], b[8], da[8], db[8], h[8];
    if constexpr (SAVED == kBf16) {
      unpack_bf16x8(q.a, a);
      unpack_bf16x8(q.b, b);
    } else {
      int8_values8(make_uint2(q.a.x, q.a.y), int8_step(q.sa), a);
      int8_values8(make_uint2(q.b.x, q.b.y), int8_step(q.sb), b);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float f, d;
      act_grad<ACT>(a[k], f, d);
      da[k] = dh[k] * b[k] * d;
      db[k] = dh[k] * f;
      h[k] = f * b[k];
    }
    uint16_t* dab = p.dab + R * 2 * p.I + i;
    *reinterpret_cast<uint4*>(dab) = pack8(da);
    *reinterpret_cast<uint4*>(dab + p.I) = pack8(db);
    *reinterpret_cast<uint4*>(p.h + R * p.I + i) = pack8(h);
  });
}

// FP32 or BF16 gradients; an accumulated BF16 gradient takes the rounded contribution, as a BF16
// main_grad does.
template <class TL, bool F32, bool OVER>
__global__ __launch_bounds__(TL::NTH, TL::MINB) void k_ffn_wgrad(WgradArgs p) {
  __shared__ __align__(16) uint8_t lds[TL::LDS];
  const TileAt at = tile_at((p.M + TL::TM - 1) / TL::TM, (p.N + TL::TN - 1) / TL::TN);
  if (!at.ok) return;
  const int m0 = at.m * TL::TM, n0 = at.n * TL::TN, rows = min(TL::TM, p.M - m0), cols = min(TL::TN, p.N - n0);
  Sums<TL> acc;
  zero<TL>(acc);
  tile_product<TL, RC, RC>(acc, p.T, {p.a.p + m0, 2 * p.a.ld, rows}, {p.b.p + n0, 2 * p.b.ld, cols}, lds);
  auto place = [&](int row, int col) {
    const int m = m0 + row;
    const int64_t at = m < p.msplit ? (int64_t)m * p.ldc0 : (int64_t)(m - p.msplit) * p.ldc1;
    return static_cast<uint8_t*>(m < p.msplit ? p.c0 : p.c1) + (at + n0 + col) * (F32 ? 4 : 2);
  };
  struct Old {
    uint4 v[OVER ? 1 : (F32 ? 2 : 1)];
  };
  auto pre = [&](int row, int col) {
    Old q{};
    if constexpr (!OVER) {
      const uint4* from = reinterpret_cast<const uint4*>(place(row, col));
      q.v[0] = from[0];
      if constexpr (F32) q.v[1] = from[1];
    }
    return q;
  };
  each_piece<TL, false>(acc, lds, rows, cols, pre, [&](int row, int col, const float* v, const Old& q) {
    uint8_t* c = place(row, col);
    if constexpr (F32) {
      f32x4_t* to = reinterpret_cast<f32x4_t*>(c);
      f32x4_t r[2] = {f32x4_t{v[0], v[1], v[2], v[3]}, f32x4_t{v[4], v[5], v[6], v[7]}};
#pragma unroll
      for (int u = 0; u < 2; ++u) to[u] = OVER ? r[u] : __builtin_bit_cast(f32x4_t, q.v[OVER ? 0 : u]) + r[u];
    } else {
      uint4 r = pack8(v);
      if constexpr (!OVER) {
        float old[8], add[8];
        unpack_bf16x8(q.v[0], old);
        unpack_bf16x8(r, add);
#pragma unroll
        for (int k = 0; k < 8; ++k) old[k] += add[k];
        r = pack8(old);
      }
      *reinterpret_cast<uint4*>(c) = r;
    }
  });
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <class TL, class A>
dim3 grid_of(const A& a, int64_t m, int64_t n, int tn) {
  return dim3(tile_grid(ceil_div(m, TL::TM) * ceil_div(n, tn)));
}

template <class TL, int ACT>
void up_as(hipStream_t st, const UpArgs& a) {
  const dim3 grid = grid_of<TL>(a, a.T, a.I, TL::TN / 2), block(TL::NTH);
  if (a.saved == kNone) hipLaunchKernelGGL((k_ffn_up<TL, ACT, kNone>), grid, block, 0, st, a);
  else if (a.saved == kBf16) hipLaunchKernelGGL((k_ffn_up<TL, ACT, kBf16>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((k_ffn_up<TL, ACT, kInt8>), grid, block, 0, st, a);
}
template <class TL, int ACT>
void dh_as(hipStream_t st, const DhArgs& a) {
  const dim3 grid = grid_of<TL>(a, a.T, a.I, TL::TN), block(TL::NTH);
  if (a.saved == kBf16) hipLaunchKernelGGL((k_ffn_dh<TL, ACT, kBf16>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((k_ffn_dh<TL, ACT, kInt8>), grid, block, 0, st, a);
}
template <class TL, bool F32>
void wgrad_as(hipStream_t st, const WgradArgs& a) {
  const dim3 grid = grid_of<TL>(a, a.M, a.N, TL::TN), block(TL::NTH);
  if (a.overwrite) hipLaunchKernelGGL((k_ffn_wgrad<TL, F32, true>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((k_ffn_wgrad<TL, F32, false>), grid, block, 0, st, a);
}

}  // namespace

// Large or Medium tiles for an m x n result over k, whichever is expected to end first.  A round of 256 Large
// tiles (one a CU) takes 0.60 us a stage of 32 k and 14 us for its start and end; one of 512 Medium tiles (two
// a CU, half the work) 0.57 and 10, of up to 256 of them (one a CU) 0.21 and 8.  Measured, Large against
// Medium: 777 x 24576 over 4096 200 us and 263, 777 x 4096 over 12288 231 and 131, 4096 x 4096 over 4096 118 and
// 173, 2048 x 2048 over 8192 161 and 75, 256 x 4096 over 4096 81 and 33.
bool large(int64_t m, int64_t n, int64_t k) {
  const double stages = (double)ceil_div(k, 32);
  const int64_t l = ceil_div(m, Large::TM) * ceil_div(n, Large::TN), s = ceil_div(m, Medium::TM) * ceil_div(n, Medium::TN);
  const int64_t rest = s % 512;
  const double tl = (double)ceil_div(l, 256) * (0.60 * stages + 14.0);
  const double ts = (double)(s / 512 + (rest > 256)) * (0.57 * stages + 10.0) +
                    (rest > 0 && rest <= 256 ? 0.21 * stages + 8.0 : 0.0);
  return tl <= ts;
}

void launch_up(hipStream_t st, const UpArgs& a) {
  const bool l = large(a.T, 2 * a.I, a.H);
  if (a.act == kSilu) l ? up_as<Large, kSilu>(st, a) : up_as<Medium, kSilu>(st, a);
  else l ? up_as<Large, kGelu>(st, a) : up_as<Medium, kGelu>(st, a);
}
template <int BM>
void rows_as(hipStream_t st, const RowsArgs& a) {
  if (large(a.T, a.N, a.K))
    hipLaunchKernelGGL((k_ffn_rows<Large, BM>), grid_of<Large>(a, a.T, a.N, Large::TN), dim3(Large::NTH), 0, st, a);
  else
    hipLaunchKernelGGL((k_ffn_rows<Medium, BM>), grid_of<Medium>(a, a.T, a.N, Medium::TN), dim3(Medium::NTH), 0, st, a);
}
void launch_down(hipStream_t st, const RowsArgs& a) { rows_as<KC>(st, a); }
void launch_dx(hipStream_t st, const RowsArgs& a) { rows_as<RC>(st, a); }
void launch_dh(hipStream_t st, const DhArgs& a) {
  const bool l = large(a.T, a.I, a.H);
  if (a.act == kSilu) l ? dh_as<Large, kSilu>(st, a) : dh_as<Medium, kSilu>(st, a);
  else l ? dh_as<Large, kGelu>(st, a) : dh_as<Medium, kGelu>(st, a);
}
void launch_wgrad(hipStream_t st, const WgradArgs& a) {
  const bool l = large(a.M, a.N, a.T);
  if (a.fp32) l ? wgrad_as<Large, true>(st, a) : wgrad_as<Medium, true>(st, a);
  else l ? wgrad_as<Large, false>(st, a) : wgrad_as<Medium, false>(st, a);
}

}  // namespace ffn
}  // namespace moe

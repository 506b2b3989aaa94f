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

// Bound by the matrix units and their power: at 4096 tokens, H 4096, I 12288 grad_x runs at 1340 to 1370 TFLOP/s with
// the matrix units busy 69 % of the time at 1.75 GHz, the weight gradients at 1230, and dh at 930, since its end reads a and b and
// writes da, db and h, 10 bytes an element (500 MB, 100 us at a copy's rate), which a tile with a CU to itself hides
// behind nothing.  256 x 128 with two a CU is slower there (480 us against 445) and 10 % faster only where the contraction is
// short (up of 4690 tokens, H 1024, I 5504: 122 us against 135).
using Large = Tile<256, 256, 2, 2, 4, 1, 0, 64>;
using Mid = Tile<192, 256, 2, 2, 4, 1, 0, 64>;
using Medium = Tile<128, 128, 2, 2, 4, 2, 0, 64>;

// The k of a part, whole stages but for the last one's end.
struct Part {
  int lo, hi;
};
__device__ __forceinline__ Part part_of(int k, const TileAt& at, const Split& s) {
  const int stages = (k + 31) / 32;
  return {32 * part_begin(stages, at.part, s.n), min(k, 32 * part_begin(stages, at.part + 1, s.n))};
}

constexpr auto no_more = [](int, int) { return Nothing{}; };   // an epilogue without operands from memory

__device__ __forceinline__ uint4 pack8(const float* v) {
  return make_uint4(pack_bf2(v[0], v[1]), pack_bf2(v[2], v[3]), pack_bf2(v[4], v[5]), pack_bf2(v[6], v[7]));
}

// ---- what is done with eight neighbouring sums
template <int ACT, int SAVED>
__device__ __forceinline__ void up_end(const UpArgs& p, int row, int i, const float* a, const float* b) {
  float h[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) h[k] = act<ACT>(a[k]) * b[k];
  *reinterpret_cast<uint4*>(p.h.p + row * p.h.ld + i) = pack8(h);
  if constexpr (SAVED == kBf16) {
    uint16_t* ab = reinterpret_cast<uint16_t*>(p.kept.ab) + (int64_t)row * 2 * p.I + i;
    *reinterpret_cast<uint4*>(ab) = pack8(a);
    *reinterpret_cast<uint4*>(ab + p.I) = pack8(b);
  }
  if constexpr (SAVED == kInt8) {   // the four lanes of a quad hold a block of 32
    const float(&av)[8] = *reinterpret_cast<const float(*)[8]>(a);
    const float(&bv)[8] = *reinterpret_cast<const float(*)[8]>(b);
    const int sa = int8_scale_byte(quad_max_u(abs_bits8(av))), sb = int8_scale_byte(quad_max_u(abs_bits8(bv)));
    uint8_t* ab = p.kept.ab + (int64_t)row * 2 * p.I + i;
    *reinterpret_cast<uint2*>(ab) = int8_codes8(av, sa);
    *reinterpret_cast<uint2*>(ab + p.I) = int8_codes8(bv, sb);
    if ((i & 31) == 0) {
      uint8_t* sc = p.kept.scales + (int64_t)row * (p.I / 16) + i / 32;
      sc[0] = (uint8_t)sa;
      sc[p.I / 32] = (uint8_t)sb;
    }
  }
}

__device__ __forceinline__ void rows_end(const RowsArgs& p, int row, int col, const float* v) {
  *reinterpret_cast<uint4*>(p.c.p + row * p.c.ld + col) = pack8(v);
}

// a and b of a piece: 8 BF16 values each, or 8 codes and a scale byte
struct Saved8 {
  uint4 a, b;
  int sa, sb;
};
template <int SAVED>
__device__ __forceinline__ Saved8 dh_pre(const DhArgs& p, int row, int i) {
  Saved8 q{};
  if constexpr (SAVED == kBf16) {
    const uint16_t* ab = reinterpret_cast<const uint16_t*>(p.kept.ab) + (int64_t)row * 2 * p.I + i;
    q.a = *reinterpret_cast<const uint4*>(ab);
    q.b = *reinterpret_cast<const uint4*>(ab + p.I);
  } else {
    const uint8_t *ab = p.kept.ab + (int64_t)row * 2 * p.I + i, *sc = p.kept.scales + (int64_t)row * (p.I / 16) + i / 32;
    const uint2 a = *reinterpret_cast<const uint2*>(ab), b = *reinterpret_cast<const uint2*>(ab + p.I);
    q.a.x = a.x, q.a.y = a.y, q.b.x = b.x, q.b.y = b.y;
    q.sa = sc[0], q.sb = sc[p.I / 32];
  }
  return q;
}
template <int ACT, int SAVED>
__device__ __forceinline__ void dh_end(const DhArgs& p, int row, int i, const float* dh, const Saved8& q) {
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
    da[k] = dh[k] * (b[k] * d);              // d may be 0 where dh b overflows
    db[k] = dh[k] * f;
    h[k] = f * b[k];
  }
  uint16_t* dab = p.dab + (int64_t)row * 2 * p.I + i;
  *reinterpret_cast<uint4*>(dab) = pack8(da);
  *reinterpret_cast<uint4*>(dab + p.I) = pack8(db);
  *reinterpret_cast<uint4*>(p.h + (int64_t)row * p.I + i) = pack8(h);
}

// FP32 or BF16 gradients; an accumulated BF16 gradient takes the rounded contribution, as a BF16
// main_grad does.
template <bool F32, bool OVER>
struct Old {
  uint4 v[!OVER && F32 ? 2 : 1];
};
template <bool F32>
__device__ __forceinline__ uint8_t* grad_at(const WgradArgs& p, int m, int n) {
  const int64_t at = m < p.msplit ? m * p.ldc0 : (m - p.msplit) * p.ldc1;
  return static_cast<uint8_t*>(m < p.msplit ? p.c0 : p.c1) + (at + n) * (F32 ? 4 : 2);
}
template <bool F32, bool OVER>
__device__ __forceinline__ Old<F32, OVER> wgrad_pre(const WgradArgs& p, int m, int n) {
  Old<F32, OVER> q{};
  if constexpr (!OVER) {
    const uint4* from = reinterpret_cast<const uint4*>(grad_at<F32>(p, m, n));
    q.v[0] = from[0];
    if constexpr (F32) q.v[1] = from[1];
  }
  return q;
}
template <bool F32, bool OVER>
__device__ __forceinline__ void wgrad_end(const WgradArgs& p, int m, int n, const float* v, const Old<F32, OVER>& q) {
  uint8_t* c = grad_at<F32>(p, m, n);
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
}

// ---- the products
template <class TL, int ACT, int SAVED>
__global__ __launch_bounds__(TL::NTH, TL::MINB) void k_ffn_up(UpArgs p) {
  static_assert(TL::WNC % 64 == 0, "gate / up pairs in a wave");
  __shared__ __align__(16) uint8_t lds[TL::LDS];
  constexpr int TI = TL::TN / 2;            // columns of h a tile
  const TileAt at = tile_at((p.T + TL::TM - 1) / TL::TM, (p.I + TI - 1) / TI, p.plan.split.n);
  if (!at.ok) return;
  const int m0 = at.m * TL::TM, i0 = at.n * TI, rows = min(TL::TM, p.T - m0), cols = min(TI, p.I - i0);
  Sums<TL> acc;
  zero<TL>(acc);
  // 32 gate rows, 32 up rows in turn: a lane's accumulators of blocks 2j and 2j + 1 are a and b of the
  // same elements; cols is a multiple of 64, so the rows that exist come first
  const Part k = part_of(p.H, at, p.plan.split);
  const Operand x{p.x.p + (int64_t)m0 * p.x.ld + k.lo, 2 * p.x.ld, rows};
  const Operand w{p.gate.p + (int64_t)i0 * p.gate.ld + k.lo, 2 * p.gate.ld, 2 * cols,
                  p.up.p + (int64_t)i0 * p.up.ld + k.lo, 2 * p.up.ld};
  tile_product<TL, KC, KC2>(acc, k.hi - k.lo, x, w, lds);
  if (p.plan.split.n > 1) {
    const int64_t ld = 2 * (int64_t)p.I;
    leave<TL, true>(acc, p.plan.split.sums + ((int64_t)at.part * p.T + m0) * ld + i0, ld, rows, cols, p.I);
    return;
  }
  each_piece<TL, true>(acc, lds, rows, cols, no_more, [&](int row, int col, const float* a, const float* b, Nothing) {
    up_end<ACT, SAVED>(p, m0 + row, i0 + col, a, b);
  });
}

// BM = KC: b0 rows are the result's columns (ksplit = K); RC: b0 rows run along K, those of its second half in
// b1 (K = 2 ksplit)
template <class TL, int BM>
__global__ __launch_bounds__(TL::NTH, TL::MINB) void k_ffn_rows(RowsArgs p) {
  __shared__ __align__(16) uint8_t lds[TL::LDS];
  const TileAt at = tile_at((p.T + TL::TM - 1) / TL::TM, (p.N + TL::TN - 1) / TL::TN, p.plan.split.n);
  if (!at.ok) return;
  const int m0 = at.m * TL::TM, n0 = at.n * TL::TN, rows = min(TL::TM, p.T - m0), cols = min(TL::TN, p.N - n0);
  Sums<TL> acc;
  zero<TL>(acc);
  const Part part = part_of(p.K, at, p.plan.split);
  for (int k = part.lo; k < part.hi;) {
    const bool first = k < p.ksplit;
    const int end = first ? min(part.hi, p.ksplit) : part.hi, in = first ? k : k - p.ksplit;   // in b0 or b1
    const Mat& b = first ? p.b0 : p.b1;
    if (k > part.lo) __syncthreads();        // the first half's stages have been read
    tile_product<TL, KC, BM>(acc, end - k, {p.a.p + (int64_t)m0 * p.a.ld + k, 2 * p.a.ld, rows},
                             {BM == KC ? b.p + (int64_t)n0 * b.ld + in : b.p + (int64_t)in * b.ld + n0, 2 * b.ld, cols}, lds);
    k = end;
  }
  if (p.plan.split.n > 1) {
    leave<TL, false>(acc, p.plan.split.sums + ((int64_t)at.part * p.T + m0) * p.N + n0, p.N, rows, cols, 0);
    return;
  }
  each_piece<TL, false>(acc, lds, rows, cols, no_more,
                        [&](int row, int col, const float* v, Nothing) { rows_end(p, m0 + row, n0 + col, v); });
}

template <class TL, int ACT, int SAVED>
__global__ __launch_bounds__(TL::NTH, TL::MINB) void k_ffn_dh(DhArgs p) {
  __shared__ __align__(16) uint8_t lds[TL::LDS];
  const TileAt at = tile_at((p.T + TL::TM - 1) / TL::TM, (p.I + TL::TN - 1) / TL::TN, p.plan.split.n);
  if (!at.ok) return;
  const int m0 = at.m * TL::TM, n0 = at.n * TL::TN, rows = min(TL::TM, p.T - m0), cols = min(TL::TN, p.I - n0);
  Sums<TL> acc;
  zero<TL>(acc);
  const Part k = part_of(p.H, at, p.plan.split);
  tile_product<TL, KC, RC>(acc, k.hi - k.lo, {p.dy.p + (int64_t)m0 * p.dy.ld + k.lo, 2 * p.dy.ld, rows},
                           {p.down.p + k.lo * p.down.ld + n0, 2 * p.down.ld, cols}, lds);
  if (p.plan.split.n > 1) {
    leave<TL, false>(acc, p.plan.split.sums + ((int64_t)at.part * p.T + m0) * p.I + n0, p.I, rows, cols, 0);
    return;
  }
  each_piece<TL, false>(acc, lds, rows, cols, [&](int row, int col) { return dh_pre<SAVED>(p, m0 + row, n0 + col); },
                        [&](int row, int col, const float* dh, const Saved8& q) {
                          dh_end<ACT, SAVED>(p, m0 + row, n0 + col, dh, q);
                        });
}

template <class TL, bool F32, bool OVER>
__global__ __launch_bounds__(TL::NTH, TL::MINB) void k_ffn_wgrad(WgradArgs p) {
  __shared__ __align__(16) uint8_t lds[TL::LDS];
  const TileAt at = tile_at((p.M + TL::TM - 1) / TL::TM, (p.N + TL::TN - 1) / TL::TN, p.plan.split.n);
  if (!at.ok) return;
  const int m0 = at.m * TL::TM, n0 = at.n * TL::TN, rows = min(TL::TM, p.M - m0), cols = min(TL::TN, p.N - n0);
  Sums<TL> acc;
  zero<TL>(acc);
  const Part k = part_of(p.T, at, p.plan.split);
  tile_product<TL, RC, RC>(acc, k.hi - k.lo, {p.a.p + k.lo * p.a.ld + m0, 2 * p.a.ld, rows},
                           {p.b.p + k.lo * p.b.ld + n0, 2 * p.b.ld, cols}, lds);
  if (p.plan.split.n > 1) {
    leave<TL, false>(acc, p.plan.split.sums + ((int64_t)at.part * p.M + m0) * p.N + n0, p.N, rows, cols, 0);
    return;
  }
  each_piece<TL, false>(acc, lds, rows, cols, [&](int row, int col) { return wgrad_pre<F32, OVER>(p, m0 + row, n0 + col); },
                        [&](int row, int col, const float* v, const Old<F32, OVER>& q) {
                          wgrad_end<F32, OVER>(p, m0 + row, n0 + col, v, q);
                        });
}

// ---- sums of split contractions, added up in their order: a thread has 8 neighbouring columns
constexpr int kSumThreads = 256;

// The thread's row and column of a result of `cols` columns (a multiple of 64, so a quad of lanes stays in a row).
struct Piece {
  int row, col;
};
__device__ __forceinline__ Piece piece_at(int cols) {
  const int64_t o = (int64_t)blockIdx.x * kSumThreads + threadIdx.x;
  const int row = (int)(o / (cols / 8));
  return {row, 8 * (int)(o - (int64_t)row * (cols / 8))};
}
// Adds the parts' 8 sums from `at` of a result of `all` elements.
__device__ __forceinline__ void add_parts(const Split& s, int64_t all, int64_t at, float* v) {
  f32x4_t x{0.0f, 0.0f, 0.0f, 0.0f}, y = x;
#pragma unroll 4
  for (int k = 0; k < s.n; ++k) {
    const f32x4_t* p = reinterpret_cast<const f32x4_t*>(s.sums + k * all + at);
    x += p[0];
    y += p[1];
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = x[e], v[4 + e] = y[e];
}

template <int ACT, int SAVED>
__global__ __launch_bounds__(kSumThreads) void k_ffn_up_sum(UpArgs p) {
  const Piece o = piece_at(p.I);
  if (o.row >= p.T) return;
  const int64_t ld = 2 * (int64_t)p.I, at = o.row * ld + o.col;
  float a[8], b[8];
  add_parts(p.plan.split, p.T * ld, at, a);
  add_parts(p.plan.split, p.T * ld, at + p.I, b);
  up_end<ACT, SAVED>(p, o.row, o.col, a, b);
}
__global__ __launch_bounds__(kSumThreads) void k_ffn_rows_sum(RowsArgs p) {
  const Piece o = piece_at(p.N);
  if (o.row >= p.T) return;
  float v[8];
  add_parts(p.plan.split, (int64_t)p.T * p.N, (int64_t)o.row * p.N + o.col, v);
  rows_end(p, o.row, o.col, v);
}
template <int ACT, int SAVED>
__global__ __launch_bounds__(kSumThreads) void k_ffn_dh_sum(DhArgs p) {
  const Piece o = piece_at(p.I);
  if (o.row >= p.T) return;
  const Saved8 q = dh_pre<SAVED>(p, o.row, o.col);
  float v[8];
  add_parts(p.plan.split, (int64_t)p.T * p.I, (int64_t)o.row * p.I + o.col, v);
  dh_end<ACT, SAVED>(p, o.row, o.col, v, q);
}
template <bool F32, bool OVER>
__global__ __launch_bounds__(kSumThreads) void k_ffn_wgrad_sum(WgradArgs p) {
  const Piece o = piece_at(p.N);
  if (o.row >= p.M) return;
  const Old<F32, OVER> q = wgrad_pre<F32, OVER>(p, o.row, o.col);
  float v[8];
  add_parts(p.plan.split, (int64_t)p.M * p.N, (int64_t)o.row * p.N + o.col, v);
  wgrad_end<F32, OVER>(p, o.row, o.col, v, q);
}

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <class TL, class A>
dim3 grid_of(const A& a, int64_t m, int64_t n) {
  return dim3(tile_grid(ceil_div(m, TL::TM) * ceil_div(n, TL::TN) * a.plan.split.n));
}

template <class TL, int ACT>
void up_as(hipStream_t st, const UpArgs& a) {
  const dim3 grid = grid_of<TL>(a, a.T, 2 * (int64_t)a.I), block(TL::NTH);
  if (a.saved == kNone) hipLaunchKernelGGL((k_ffn_up<TL, ACT, kNone>), grid, block, 0, st, a);
  else if (a.saved == kBf16) hipLaunchKernelGGL((k_ffn_up<TL, ACT, kBf16>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((k_ffn_up<TL, ACT, kInt8>), grid, block, 0, st, a);
}
template <class TL, int ACT>
void dh_as(hipStream_t st, const DhArgs& a) {
  const dim3 grid = grid_of<TL>(a, a.T, a.I), block(TL::NTH);
  if (a.saved == kBf16) hipLaunchKernelGGL((k_ffn_dh<TL, ACT, kBf16>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((k_ffn_dh<TL, ACT, kInt8>), grid, block, 0, st, a);
}
template <class TL, int BM>
void rows_as(hipStream_t st, const RowsArgs& a) {
  hipLaunchKernelGGL((k_ffn_rows<TL, BM>), grid_of<TL>(a, a.T, a.N), dim3(TL::NTH), 0, st, a);
}
template <class TL, bool F32>
void wgrad_as(hipStream_t st, const WgradArgs& a) {
  const dim3 grid = grid_of<TL>(a, a.M, a.N), block(TL::NTH);
  if (a.overwrite) hipLaunchKernelGGL((k_ffn_wgrad<TL, F32, true>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((k_ffn_wgrad<TL, F32, false>), grid, block, 0, st, a);
}

// f with the plan's tile
template <class F>
void by_shape(int shape, const F& f) {
  if (shape == kLarge) f(Large{});
  else if (shape == kMid) f(Mid{});
  else f(Medium{});
}

}  // namespace

void launch_up(hipStream_t st, const UpArgs& a) {
  by_shape(a.plan.shape, [&](auto t) {
    if (a.act == kSilu) up_as<decltype(t), kSilu>(st, a);
    else up_as<decltype(t), kGelu>(st, a);
  });
}
void launch_down(hipStream_t st, const RowsArgs& a) {
  by_shape(a.plan.shape, [&](auto t) { rows_as<decltype(t), KC>(st, a); });
}
void launch_dx(hipStream_t st, const RowsArgs& a) {
  by_shape(a.plan.shape, [&](auto t) { rows_as<decltype(t), RC>(st, a); });
}
void launch_dh(hipStream_t st, const DhArgs& a) {
  by_shape(a.plan.shape, [&](auto t) {
    if (a.act == kSilu) dh_as<decltype(t), kSilu>(st, a);
    else dh_as<decltype(t), kGelu>(st, a);
  });
}
void launch_wgrad(hipStream_t st, const WgradArgs& a) {
  auto as = [&](auto t) {
    if (a.fp32) wgrad_as<decltype(t), true>(st, a);
    else wgrad_as<decltype(t), false>(st, a);
  };
  if (a.plan.shape == kLarge) as(Large{});
  else as(Medium{});
}

// f with each of the constants
template <class F>
void by_act(int act, const F& f) {
  if (act == kSilu) f(std::integral_constant<int, kSilu>{});
  else f(std::integral_constant<int, kGelu>{});
}
static dim3 sum_grid(int64_t rows, int64_t cols) { return dim3((unsigned)ceil_div(rows * (cols / 8), kSumThreads)); }

void launch_up_sum(hipStream_t st, const UpArgs& a) {
  const dim3 grid = sum_grid(a.T, a.I), block(kSumThreads);
  by_act(a.act, [&](auto act) {
    constexpr int A = decltype(act)::value;
    if (a.saved == kNone) hipLaunchKernelGGL((k_ffn_up_sum<A, kNone>), grid, block, 0, st, a);
    else if (a.saved == kBf16) hipLaunchKernelGGL((k_ffn_up_sum<A, kBf16>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((k_ffn_up_sum<A, kInt8>), grid, block, 0, st, a);
  });
}
void launch_rows_sum(hipStream_t st, const RowsArgs& a) {
  hipLaunchKernelGGL(k_ffn_rows_sum, sum_grid(a.T, a.N), dim3(kSumThreads), 0, st, a);
}
void launch_dh_sum(hipStream_t st, const DhArgs& a) {
  const dim3 grid = sum_grid(a.T, a.I), block(kSumThreads);
  by_act(a.act, [&](auto act) {
    constexpr int A = decltype(act)::value;
    if (a.saved == kBf16) hipLaunchKernelGGL((k_ffn_dh_sum<A, kBf16>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((k_ffn_dh_sum<A, kInt8>), grid, block, 0, st, a);
  });
}
void launch_wgrad_sum(hipStream_t st, const WgradArgs& a) {
  const dim3 grid = sum_grid(a.M, a.N), block(kSumThreads);
  if (a.fp32) {
    if (a.overwrite) hipLaunchKernelGGL((k_ffn_wgrad_sum<true, true>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((k_ffn_wgrad_sum<true, false>), grid, block, 0, st, a);
  } else {
    if (a.overwrite) hipLaunchKernelGGL((k_ffn_wgrad_sum<false, true>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((k_ffn_wgrad_sum<false, false>), grid, block, 0, st, a);
  }
}

}  // namespace ffn
}  // namespace moe

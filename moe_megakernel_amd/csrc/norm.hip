// Layer norm and RMS norm of rows, forward and backward (C ABI: moe_norm_forward,
// moe_norm_backward).
//
// Each row is held in the registers of `tpr` threads (16, 32 or a multiple of 64, EPT = 8 or 16
// elements a thread), so x is read once and every statistic is taken from registers:
//   m = sum x / N;  d = x - m;  delta = sum d / N;  var = sum d^2 / N - delta^2
// mean = m + delta.  The second pass over the registers removes what rounding m cost: with
// m already close, delta is tiny and var has no cancellation.  Except in rows whose spread is no
// more than that rounding (one value far from zero): there the difference of the two squares
// would be rounding alone, and below -eps at times, so var = sum (d - delta)^2 / N by a third pass.
//
// Backward, with xh = (x - mean) rstd and g = dy w:
//   dx = rstd (g - sum(g) / N - xh sum(g xh) / N)    (RMS norm: without the sum(g) term)
//   dw = sum over rows of dy xh,   db = sum over rows of dy
// A workgroup walks rows and keeps its columns' dw and db in registers; the row groups
// of a workgroup are joined in LDS, workgroups write one partial row each, and a second
// kernel adds the partials in a fixed order.
//
// Bound by memory from some thousand rows on: RMS norm with a residual, 8192 x 7168 BF16, 89 us
// (5.3 TB/s; a large copy runs at 5.0); layer norm's backward, 4096 x 4096 BF16, 25 us and 3.6 for
// the second kernel (20 at the copy's rate; the partial rows add a sixth to the bytes).  FP32
// rows that are no whole pieces, backward of 1023 x 2055: 15 us (7), single elements, a fifth of the
// threads without one and a third of the row places empty in the second trip.  Below that by the
// launch: one row of 4096 takes 3 us on the GPU.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "../../include/moe.h"
#include "common.hpp"
#include "host.hpp"
#include "reduce.hpp"

using namespace moe;

namespace {

constexpr int kNormThreads = 1024;    // largest workgroup
constexpr int kNormGroups = 256;      // workgroups of the backward (partial rows): one per CU
constexpr int kFinalCols = 32, kFinalLanes = 16;   // columns and row lanes of the second kernel's workgroups

struct Rows {
  uint8_t* base;
  int64_t ld;      // elements
};

struct NormArgs {
  Rows x, res, sum, y;      // forward
  Rows dy, gsum, dx;        // backward (x: what was normalised)
  const void *w, *b;
  float* stats;
  float* part;              // backward: [groups][nsum][cols], null if there is one group or no sum
  uint8_t *gw, *gb;         // backward: weight's and bias's gradient (null: not wanted)
  int g16, overwrite;       // BF16 gradients; not accumulated
  int64_t rows;
  int N;                    // cols
  int tpr;                  // threads per row
  int rms, wbf16, w16, b16;  // w16, b16: 16-byte aligned weight, bias
  float eps;
};

// Columns of a thread: VEC (whole pieces, rows 4-byte aligned, as all of FP32 are) pieces of 16
// bytes, 8 BF16 or 4 FP32 elements, at pieces j, j + tpr, ..: neighbouring lanes read neighbouring
// pieces (with 8 FP32 elements a lane, 32 bytes apart, 4453 x 3584 took 73 us in the backward).
// Global memory takes 16 bytes at any multiple of 4: 8192 x 4096 BF16 at a stride of 4098 takes 32
// us in the forward and 50 in the backward, 30 and 48 at 4096, 52 and 56 by elements.  Otherwise
// single elements j + i tpr; pieces with a shorter last one gained nothing over those for FP32
// (4096 x 2047: 20 us and 32, against 16 and 28).
template <bool BF16>
constexpr int piece() { return BF16 ? 8 : 4; }
template <bool VEC, bool BF16>
__device__ __forceinline__ int col_of(int j, int i, int tpr) {
  constexpr int P = piece<BF16>();
  return VEC ? P * (j + i / P * tpr) + i % P : j + i * tpr;
}

// 16 bytes at a multiple of 4
typedef uint32_t piece_t __attribute__((ext_vector_type(4), aligned(4)));
__device__ __forceinline__ uint4 ld_piece(const void* p) {
  const piece_t v = *static_cast<const piece_t*>(p);
  return make_uint4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void st_piece(void* p, uint4 v) { *static_cast<piece_t*>(p) = piece_t{v.x, v.y, v.z, v.w}; }

// A thread's EPT elements of a row as loaded.
template <int EPT, bool VEC, bool BF16>
struct Raw;
template <int EPT, bool BF16>
struct Raw<EPT, true, BF16> { uint4 q[EPT / piece<BF16>()]; };
template <int EPT>
struct Raw<EPT, false, true> { uint16_t q[EPT]; };
template <int EPT>
struct Raw<EPT, false, false> { float q[EPT]; };

template <int EPT, bool VEC, bool BF16>
__device__ __forceinline__ Raw<EPT, VEC, BF16> ld_row(const Rows& m, int64_t r, int j, int tpr, int N) {
  Raw<EPT, VEC, BF16> v;
  const uint8_t* p = m.base + r * m.ld * (BF16 ? 2 : 4);
  if constexpr (VEC) {
#pragma unroll
    for (int u = 0; u < EPT / piece<BF16>(); ++u) {
      const int c = piece<BF16>() * (j + u * tpr);
      v.q[u] = c < N ? ld_piece(p + c * (BF16 ? 2 : 4)) : make_uint4(0, 0, 0, 0);
    }
  } else {
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
      const int c = j + i * tpr;
      if constexpr (BF16) v.q[i] = c < N ? reinterpret_cast<const uint16_t*>(p)[c] : (uint16_t)0;
      else v.q[i] = c < N ? reinterpret_cast<const float*>(p)[c] : 0.0f;
    }
  }
  return v;
}

template <int EPT, bool VEC, bool BF16>
__device__ __forceinline__ void unpack(const Raw<EPT, VEC, BF16>& v, float (&f)[EPT]) {
  if constexpr (VEC && BF16) {
#pragma unroll
    for (int u = 0; u < EPT / 8; ++u) unpack_bf16x8(v.q[u], f + 8 * u);
  } else if constexpr (VEC) {
#pragma unroll
    for (int u = 0; u < EPT / 4; ++u) {
      f[4 * u] = __uint_as_float(v.q[u].x);
      f[4 * u + 1] = __uint_as_float(v.q[u].y);
      f[4 * u + 2] = __uint_as_float(v.q[u].z);
      f[4 * u + 3] = __uint_as_float(v.q[u].w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
      if constexpr (BF16) f[i] = bf2f(v.q[i]);
      else f[i] = v.q[i];
    }
  }
}

template <int EPT, bool VEC, bool BF16>
__device__ __forceinline__ void st_row(const Rows& m, int64_t r, int j, int tpr, int N, const float (&f)[EPT]) {
  uint8_t* p = m.base + r * m.ld * (BF16 ? 2 : 4);
  if constexpr (VEC) {
#pragma unroll
    for (int u = 0; u < EPT / piece<BF16>(); ++u) {
      const int c = piece<BF16>() * (j + u * tpr);
      if (c >= N) continue;
      const float* s = f + piece<BF16>() * u;
      if constexpr (BF16) {
        st_piece(p + 2 * c, make_uint4(pack_bf2(s[0], s[1]), pack_bf2(s[2], s[3]), pack_bf2(s[4], s[5]),
                                       pack_bf2(s[6], s[7])));
      } else {
        st_piece(p + 4 * c, make_uint4(__float_as_uint(s[0]), __float_as_uint(s[1]), __float_as_uint(s[2]),
                                       __float_as_uint(s[3])));
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
      const int c = j + i * tpr;
      if (c >= N) continue;
      if constexpr (BF16) reinterpret_cast<uint16_t*>(p)[c] = (uint16_t)f2bf(f[i]);
      else reinterpret_cast<float*>(p)[c] = f[i];
    }
  }
}

// weight or bias of a thread's columns (0 past the end), PBF: stored as BF16; aligned:
// 16-byte aligned, so whole pieces can be read
template <int EPT, bool VEC, bool BF16, bool PBF>
__device__ __forceinline__ void ld_param_as(const void* w, int aligned, int j, int tpr, int N, float (&f)[EPT]) {
  constexpr int P = piece<BF16>();
  if (VEC && aligned) {
#pragma unroll
    for (int u = 0; u < EPT / P; ++u) {
      const int c = P * (j + u * tpr);
      float* o = f + P * u;
#pragma unroll
      for (int i = 0; i < P; ++i) o[i] = 0.0f;
      if (c >= N) continue;
      if constexpr (PBF && P == 8) {
        unpack_bf16x8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(w) + c), o);
      } else if constexpr (PBF) {
        const uint2 q = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(w) + c);
        o[0] = lo_bf(q.x); o[1] = hi_bf(q.x); o[2] = lo_bf(q.y); o[3] = hi_bf(q.y);
      } else {
#pragma unroll
        for (int h = 0; h < P; h += 4) {
          const float4 q = *reinterpret_cast<const float4*>(static_cast<const float*>(w) + c + h);
          o[h] = q.x; o[h + 1] = q.y; o[h + 2] = q.z; o[h + 3] = q.w;
        }
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < EPT; ++i) {
    const int c = col_of<VEC, BF16>(j, i, tpr);
    if constexpr (PBF) f[i] = bf2f(c < N ? static_cast<const uint16_t*>(w)[c] : (uint16_t)0);
    else f[i] = c < N ? static_cast<const float*>(w)[c] : 0.0f;
  }
}
template <int EPT, bool VEC, bool BF16>
__device__ __forceinline__ void ld_param(const void* w, int pbf, int aligned, int j, int tpr, int N,
                                         float (&f)[EPT]) {
  if (pbf) ld_param_as<EPT, VEC, BF16, true>(w, aligned, j, tpr, N, f);
  else ld_param_as<EPT, VEC, BF16, false>(w, aligned, j, tpr, N, f);
}

// Sums over the `tpr` threads of a row group; every thread of it gets them.  Up to 64 they are
// lanes of one wave; else up to 16 waves, for which `red` holds one place per wave of the
// workgroup and call parity, so one barrier a call is enough (a place is rewritten two calls
// later, behind the next call's barrier).
__device__ __forceinline__ float group_sum(float a, int tpr, float2* red, int parity) {
  a = row16_sum(a);
  if (tpr == 16) return a;
  a = add_row_pairs(a);
  if (tpr == 32) return a;
  a = add_halves(a);
  if (tpr == 64) return a;
  const int w = threadIdx.x >> 6, nw = tpr >> 6;
  float2* slot = red + parity * (kNormThreads / 64);
  if ((threadIdx.x & 63) == 0) slot[w].x = a;
  __syncthreads();
  const int l = threadIdx.x & 15;          // every 16 lanes add the group's sums up alike
  return row16_sum(l < nw ? slot[w - w % nw + l].x : 0.0f);
}
__device__ __forceinline__ void group_sum2(float& a, float& b, int tpr, float2* red, int parity) {
  a = row16_sum(a);
  b = row16_sum(b);
  if (tpr == 16) return;
  a = add_row_pairs(a);
  b = add_row_pairs(b);
  if (tpr == 32) return;
  a = add_halves(a);
  b = add_halves(b);
  if (tpr == 64) return;
  const int w = threadIdx.x >> 6, nw = tpr >> 6;
  float2* slot = red + parity * (kNormThreads / 64);
  if ((threadIdx.x & 63) == 0) slot[w] = make_float2(a, b);
  __syncthreads();
  const int l = threadIdx.x & 15;          // every 16 lanes add the group's sums up alike
  float2 v = make_float2(0.0f, 0.0f);
  if (l < nw) v = slot[w - w % nw + l];
  a = row16_sum(v.x);
  b = row16_sum(v.y);
}

// Forward: blockDim.x = row groups * tpr, the groups walk rows with a common trip count
// (the barriers are the workgroup's).
template <int EPT, bool VEC, bool BF16>
__global__ __launch_bounds__(kNormThreads) void k_norm_fwd(NormArgs a) {
  __shared__ float2 red[2 * (kNormThreads / 64)];
  const int tpr = a.tpr, N = a.N;
  const int j = threadIdx.x % tpr;
  const int rg = threadIdx.x / tpr, ng = blockDim.x / tpr;
  const int64_t stride = (int64_t)gridDim.x * ng;
  // the next row's loads are under way while a row is reduced and written
  Raw<EPT, VEC, BF16> nx{}, nr{};
  auto fetch = [&](int64_t r) __attribute__((always_inline)) {
    if (r < a.rows) {
      nx = ld_row<EPT, VEC, BF16>(a.x, r, j, tpr, N);
      if (a.res.base) nr = ld_row<EPT, VEC, BF16>(a.res, r, j, tpr, N);
    }
  };
  fetch((int64_t)blockIdx.x * ng + rg);
  float w[EPT], b[EPT];
  ld_param<EPT, VEC, BF16>(a.w, a.wbf16, a.w16, j, tpr, N, w);
#pragma unroll
  for (int i = 0; i < EPT; ++i) b[i] = 0.0f;
  if (a.b) ld_param<EPT, VEC, BF16>(a.b, a.wbf16, a.b16, j, tpr, N, b);
  const float inv_n = 1.0f / (float)N;
  int parity = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * ng; r0 < a.rows; r0 += stride) {
    const int64_t r = r0 + rg;
    const bool on = r < a.rows;
    float v[EPT], q[EPT];
    unpack(nx, v);
    if (a.res.base) {
      unpack(nr, q);
#pragma unroll
      for (int i = 0; i < EPT; ++i) {
        v[i] += q[i];
        if constexpr (BF16) v[i] = bf2f(f2bf(v[i]));
      }
      if (on) st_row<EPT, VEC, BF16>(a.sum, r, j, tpr, N, v);
    }
    fetch(r + stride);
    float mean = 0.0f, s = 0.0f, s2 = 0.0f;
    if (!a.rms) {
#pragma unroll
      for (int i = 0; i < EPT; ++i) s += v[i];
      mean = group_sum(s, tpr, red, parity) / (float)N;
      parity ^= 1;
    }
    float off = mean, delta, var;
    float square = 0.0f;             // what var still holds of delta
#pragma clang loop unroll(disable)
    for (bool again = false;; again = true) {
      s = s2 = 0.0f;
#pragma unroll
      for (int i = 0; i < EPT; ++i) {
        v[i] = col_of<VEC, BF16>(j, i, tpr) < N ? v[i] - off : 0.0f;
        s += v[i];
        s2 += v[i] * v[i];
      }
      group_sum2(s, s2, tpr, red, parity);
      parity ^= 1;
      delta = a.rms ? 0.0f : s * inv_n;
      var = s2 / (float)N;
      if (a.rms || again) break;
      // Unless delta is an eighth of the spread, the difference of the squares is as exact as the
      // sum (a 64th more).  Going round again for every row instead: 51.3 us against 48.9 at
      // 8192 x 7168 BF16, 33.3 against 29.9 at 2048 x 12304.
      auto lost = [&](float t, float t2) __attribute__((always_inline)) { return 64.0f * t * t > t2 * (float)N; };
      bool round;
      if (tpr <= 64 || ng == 1) {
        round = lost(s, s2);       // the row's threads have the same bits
      } else {                     // two rows of 128 threads: the barrier is the workgroup's, so they go together
        const float2* p = red + (parity ^ 1) * (kNormThreads / 64);
        round = lost(p[0].x + p[1].x, p[0].y + p[1].y) || lost(p[2].x + p[3].x, p[2].y + p[3].y);
      }
      const bool mine = lost(s, s2);
      square = mine ? 0.0f : delta * delta;
      if (!round) break;
      off = mine ? s / (float)N : 0.0f;      // only the other row's: the same sums again
      mean += off;
    }
    var -= square;
    const float rstd = 1.0f / sqrtf(var + a.eps);
    if (on) {
      if (a.stats && j == 0) reinterpret_cast<float2*>(a.stats)[r] = make_float2(mean + delta, rstd);
#pragma unroll
      for (int i = 0; i < EPT; ++i) v[i] = (v[i] - delta) * rstd * w[i] + b[i];
      st_row<EPT, VEC, BF16>(a.y, r, j, tpr, N, v);
    }
  }
}

// grad[c] (+)= v
__device__ __forceinline__ void add_grad(uint8_t* grad, int bf16, int overwrite, int c, float v) {
  if (bf16) {
    uint16_t* o = reinterpret_cast<uint16_t*>(grad) + c;
    float r = bf2f(f2bf(v));
    if (!overwrite) r = bf2f(*o) + r;
    *o = (uint16_t)f2bf(r);
  } else {
    float* o = reinterpret_cast<float*>(grad) + c;
    *o = overwrite ? v : *o + v;
  }
}

template <int EPT, bool VEC, bool BF16>
__global__ __launch_bounds__(kNormThreads) void k_norm_bwd(NormArgs a) {
  // EPT 8: the row groups' sums, [ng][tpr * 8], one gradient after the other.  EPT 16 (one row
  // group): both gradients' running sums, [32][tpr], which would not fit the registers.
  extern __shared__ float join[];
  constexpr bool kLdsSums = EPT == 16;
  __shared__ float2 red[2 * (kNormThreads / 64)];
  const int tpr = a.tpr, N = a.N;
  const int j = threadIdx.x % tpr;
  const int rg = threadIdx.x / tpr, ng = blockDim.x / tpr;
  const int64_t stride = (int64_t)gridDim.x * ng;
  // The next row's loads are under way while a row is reduced and written (25 us against 35 at
  // 4096 x 4096 BF16); 16 elements a thread leave no registers for that.
  constexpr bool kAhead = EPT == 8;
  Raw<EPT, VEC, BF16> nx{}, ndy{}, ngs{};
  float2 nst = make_float2(0.0f, 0.0f);
  auto fetch = [&](int64_t r) __attribute__((always_inline)) {
    if (r < a.rows) {
      nst = reinterpret_cast<const float2*>(a.stats)[r];
      nx = ld_row<EPT, VEC, BF16>(a.x, r, j, tpr, N);
      ndy = ld_row<EPT, VEC, BF16>(a.dy, r, j, tpr, N);
      if (a.gsum.base) ngs = ld_row<EPT, VEC, BF16>(a.gsum, r, j, tpr, N);
    } else {   // past the last row: nothing for the column sums
      ndy = Raw<EPT, VEC, BF16>{};
    }
  };
  if (kAhead) fetch((int64_t)blockIdx.x * ng + rg);
  float w[EPT];
  ld_param<EPT, VEC, BF16>(a.w, a.wbf16, a.w16, j, tpr, N, w);
  float dw[kLdsSums ? 1 : EPT], db[kLdsSums ? 1 : EPT];
  if constexpr (kLdsSums) {
#pragma unroll
    for (int i = 0; i < 2 * EPT; ++i) join[i * tpr + j] = 0.0f;
  } else {
#pragma unroll
    for (int i = 0; i < EPT; ++i) dw[i] = db[i] = 0.0f;
  }
  const float inv_n = 1.0f / (float)N;
  int parity = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * ng; r0 < a.rows; r0 += stride) {
    const int64_t r = r0 + rg;
    const bool on = r < a.rows;
    if (!kAhead) fetch(r);
    float xh[EPT], g[EPT];
    unpack(nx, xh);
    unpack(ndy, g);
    const Raw<EPT, VEC, BF16> gs = ngs;
    const float mean = nst.x, rstd = nst.y;
    if (kAhead) fetch(r + stride);
#pragma unroll
    for (int i = 0; i < EPT; ++i) xh[i] = on && col_of<VEC, BF16>(j, i, tpr) < N ? (xh[i] - mean) * rstd : 0.0f;
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
      if constexpr (kLdsSums) {
        join[i * tpr + j] += g[i] * xh[i];
        join[(EPT + i) * tpr + j] += g[i];
      } else {
        dw[i] += g[i] * xh[i];
        db[i] += g[i];
      }
      g[i] *= w[i];
      s1 += g[i];
      s2 += g[i] * xh[i];
    }
    group_sum2(s1, s2, tpr, red, parity);
    parity ^= 1;
    if (on) {
      const float m1 = a.rms ? 0.0f : s1 * inv_n, m2 = s2 * inv_n;
#pragma unroll
      for (int i = 0; i < EPT; ++i) g[i] = rstd * (g[i] - m1 - xh[i] * m2);
      if (a.gsum.base) {
        unpack(gs, xh);
#pragma unroll
        for (int i = 0; i < EPT; ++i) g[i] += xh[i];
      }
      st_row<EPT, VEC, BF16>(a.dx, r, j, tpr, N, g);
    }
  }
  if (!a.gw && !a.gb) return;
  // join the row groups in order; then a partial row of this workgroup, or, if it is the
  // only one, the gradients
  float* out = a.part ? a.part + (int64_t)blockIdx.x * ((a.gw ? N : 0) + (a.gb ? N : 0)) : nullptr;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    uint8_t* grad = which ? a.gb : a.gw;
    if (!grad) continue;
    auto put = [&](int i, int jj, float v) __attribute__((always_inline)) {
      const int c = col_of<VEC, BF16>(jj, i, tpr);
      if (c >= N) return;
      if (out) out[(which && a.gw ? N : 0) + c] = v;
      else add_grad(grad, a.g16, a.overwrite, c, v);
    };
    if constexpr (kLdsSums) {
#pragma unroll
      for (int i = 0; i < EPT; ++i) put(i, j, join[(which * EPT + i) * tpr + j]);
    } else if (ng == 1) {
#pragma unroll
      for (int i = 0; i < EPT; ++i) put(i, j, which ? db[i] : dw[i]);
    } else {
      const int row = tpr * EPT;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < EPT; ++i) join[rg * row + i * tpr + j] = which ? db[i] : dw[i];
      __syncthreads();
      for (int k = threadIdx.x; k < row; k += blockDim.x) {
        float v = 0.0f;
#pragma unroll 4
        for (int q = 0; q < ng; ++q) v += join[q * row + k];
        put(k / tpr, k % tpr, v);
      }
    }
  }
}

// grad[c] (+)= sum over the partial rows: kFinalCols columns a workgroup, kFinalLanes lanes
// of rows per column, eight rows of a lane in flight, joined in order.
__global__ __launch_bounds__(kFinalCols * kFinalLanes) void k_norm_bwd_final(const float* __restrict__ part,
                                                                            int groups, int width, int N,
                                                                            uint8_t* g0, uint8_t* g1, int bf16,
                                                                            int overwrite) {
  __shared__ float red[kFinalLanes][kFinalCols];
  const int cl = threadIdx.x % kFinalCols, q = threadIdx.x / kFinalCols;
  const int c = blockIdx.x * kFinalCols + cl;
  float v = 0.0f;
  if (c < width) {
    for (int p = q; p < groups; p += 8 * kFinalLanes) {
      float t[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int pu = p + u * kFinalLanes;
        t[u] = pu < groups ? part[(int64_t)pu * width + c] : 0.0f;
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) v += t[u];
    }
  }
  red[q][cl] = v;
  __syncthreads();
  if (q != 0 || c >= width) return;
  v = red[0][cl];
#pragma unroll
  for (int i = 1; i < kFinalLanes; ++i) v += red[i][cl];
  add_grad(c < N ? g0 : g1, bf16, overwrite, c < N ? c : c - N, v);
}

// ---------------------------------------------------------------- host side
moe_status check_norm(const moe_norm_problem* p) {
  if (!p) return MOE_ERR_NULL;
  if (p->rows < 0 || p->rows > ((int64_t)1 << 30)) return MOE_ERR_SHAPE;
  if (p->cols < 1 || p->cols > MOE_NORM_MAX_COLS) return MOE_ERR_SHAPE;
  if (p->kind != MOE_NORM_LAYER && p->kind != MOE_NORM_RMS) return MOE_ERR_UNSUPPORTED;
  for (int32_t d : {p->dtype, p->param_dtype, p->grad_dtype})
    if (d != MOE_BF16 && d != MOE_FP32) return MOE_ERR_DTYPE;
  if (p->flags & ~MOE_NORM_OVERWRITE_GRADS) return MOE_ERR_UNSUPPORTED;
  if (!(p->eps >= 0.0f && p->eps < 3.0e38f)) return MOE_ERR_UNSUPPORTED;   // NaN, < 0, infinite
  return MOE_OK;
}

moe_status check_rows(const moe_norm_problem* p, const moe_rows* m) {
  if (!m || (p->rows > 0 && !m->base)) return MOE_ERR_NULL;
  if (m->ld < p->cols || m->ld > ((int64_t)1 << 40) || !elem_aligned(m->base, p->dtype)) return MOE_ERR_LAYOUT;
  return MOE_OK;
}

// every row 4-byte aligned (m: an optional matrix may be null)
bool rows4(const moe_norm_problem* p, const moe_rows* m) {
  return !m || p->dtype == MOE_FP32 || (aligned4(m->base) && m->ld % 2 == 0);
}

bool whole_pieces(const moe_norm_problem* p) {
  return p->cols % (p->dtype == MOE_BF16 ? piece<true>() : piece<false>()) == 0;
}

Rows rows_of(const moe_rows* m) { return m ? Rows{static_cast<uint8_t*>(m->base), m->ld} : Rows{nullptr, 0}; }

// Short rows share a wave: a wave of its own for each would leave most lanes without elements
// (RMS norm of 131072 rows of 128 BF16: 18 us against 46 in the forward, 23 against 45 in the
// backward).
int threads_per_row(int64_t cols, int ept) {
  for (int tpr : {16, 32})
    if (cols <= tpr * ept) return tpr;
  return 64 * (int)((cols + 64 * ept - 1) / (64 * ept));
}

// Elements per thread.  The forward in 16-byte pieces takes 16 (fewer waves meet at the
// barriers: 89 us against 112 at 8192 x 7168 BF16); single elements at 16 a thread would
// spill, as would the backward's accumulators, so those take 8 wherever 1024 threads then hold a row.
// Above 8192 columns all variants but the forward in pieces and the BF16 backward in pieces do
// spill; 2048 rows take, forward and backward: 12304 BF16 31 and 59 us, FP32 39 and 140; by elements,
// 12301 BF16 53 and 195, FP32 50 and 214 (8192 BF16: 17 and 31).
int fwd_ept(int64_t cols, bool vec) { return !vec && cols <= 8 * kNormThreads ? 8 : 16; }
int bwd_ept(int64_t cols) { return cols <= 8 * kNormThreads ? 8 : 16; }

NormArgs norm_args(const moe_norm_problem* p, int ept) {
  NormArgs a{};
  a.rows = p->rows;
  a.N = (int)p->cols;
  a.tpr = threads_per_row(p->cols, ept);
  a.rms = p->kind == MOE_NORM_RMS;
  a.wbf16 = p->param_dtype == MOE_BF16;
  a.eps = p->eps;
  return a;
}

// FWD: the forward has no variant of 8 elements a thread in 16-byte pieces (fwd_ept).
template <bool FWD, class F>
void with_variant(int ept, bool vec, bool bf16, F&& f) {
  using E8 = std::integral_constant<int, 8>;
  using E16 = std::integral_constant<int, 16>;
  auto types = [&](auto e, auto v) {
    if (bf16) f(e, v, std::true_type{});
    else f(e, v, std::false_type{});
  };
  if (!vec && ept == 8) types(E8{}, std::false_type{});
  else if (!vec) types(E16{}, std::false_type{});
  else if (FWD || ept == 16) types(E16{}, std::true_type{});
  else if constexpr (!FWD) types(E8{}, std::true_type{});
}

// The backward's launch: row groups a workgroup, workgroups, LDS bytes.  Up to twice the rows
// that one workgroup holds stay in one, which writes the gradients itself (no second kernel);
// otherwise first a workgroup for each of the kNormGroups, then row groups up to 1024 threads.
struct BwdShape {
  int ept, ng, groups;
  size_t lds;
};
BwdShape bwd_shape(const moe_norm_problem* p) {
  BwdShape b;
  b.ept = bwd_ept(p->cols);
  const int tpr = threads_per_row(p->cols, b.ept);
  const int64_t fit = kNormThreads / tpr, rows = p->rows > 0 ? p->rows : 1;
  if (rows <= 2 * fit) {
    b.ng = (int)(rows < fit ? rows : fit);
    b.groups = 1;
  } else {
    const int64_t want = (rows + kNormGroups - 1) / kNormGroups;
    b.ng = (int)(want < fit ? want : fit);
    const int64_t need = (rows + b.ng - 1) / b.ng;
    b.groups = (int)(need < kNormGroups ? need : kNormGroups);
  }
  b.lds = sizeof(float) * tpr * (b.ept == 16 ? 32 : (b.ng > 1 ? 8 * b.ng : 0));
  return b;
}

}  // namespace

extern "C" {

moe_status moe_norm_forward(const moe_norm_problem* p, const moe_rows* x, const moe_rows* residual,
                            const void* weight, const void* bias, const moe_rows* sum, const moe_rows* y,
                            float* stats, void* stream) {
  MOE_TRY(check_norm(p));
  MOE_TRY(check_rows(p, x));
  MOE_TRY(check_rows(p, y));
  if ((residual != nullptr) != (sum != nullptr)) return residual ? MOE_ERR_NULL : MOE_ERR_LAYOUT;
  if (residual) {
    MOE_TRY(check_rows(p, residual));
    MOE_TRY(check_rows(p, sum));
    if (p->rows > 0 && sum->base == y->base) return MOE_ERR_LAYOUT;   // one would overwrite the other
  }
  if (!weight) return MOE_ERR_NULL;
  if (!elem_aligned(weight, p->param_dtype) || !elem_aligned(bias, p->param_dtype)) return MOE_ERR_LAYOUT;
  if (reinterpret_cast<uintptr_t>(stats) & 7u) return MOE_ERR_LAYOUT;
  if (p->rows == 0) return MOE_OK;
  const bool vec = whole_pieces(p) && rows4(p, x) && rows4(p, residual) && rows4(p, sum) && rows4(p, y);
  const int ept = fwd_ept(p->cols, vec);
  NormArgs a = norm_args(p, ept);
  a.x = rows_of(x); a.res = rows_of(residual); a.sum = rows_of(sum); a.y = rows_of(y);
  a.w = weight; a.b = bias;
  a.w16 = aligned16(weight); a.b16 = aligned16(bias);
  a.stats = stats;
  // about 256 threads a workgroup, and enough workgroups for 2048 threads per CU
  int ng = 256 / a.tpr;
  if (ng < 1) ng = 1;
  if (ng > p->rows) ng = (int)p->rows;
  const int64_t need = (p->rows + ng - 1) / ng, most = 256 * 2048 / (ng * a.tpr);
  const dim3 grid((unsigned)(need < most ? need : most)), block(ng * a.tpr);
  hipStream_t st = static_cast<hipStream_t>(stream);
  return launch("norm_fwd", st, [&] {
    with_variant<true>(ept, vec, p->dtype == MOE_BF16, [&](auto e, auto v, auto bf) {
      hipLaunchKernelGGL((k_norm_fwd<e(), v(), bf()>), grid, block, 0, st, a);
    });
  });
}

size_t moe_norm_workspace_bytes(const moe_norm_problem* p) {
  if (check_norm(p) != MOE_OK) return 0;
  // Not the launch's own number of partial rows, which falls where a workgroup takes another row
  // group (256 rows of 4096 in 256 workgroups, 257 in 129): a workspace sized for some rows has to serve
  // every smaller batch.
  const int64_t groups = bwd_shape(p).groups == 1 ? 1 : (p->rows < kNormGroups ? p->rows : kNormGroups);
  return align_up((size_t)groups * 2 * p->cols * sizeof(float) + 1);
}

moe_status moe_norm_backward(const moe_norm_problem* p, const moe_rows* grad_y, const moe_rows* x,
                             const void* weight, const float* stats, const moe_rows* grad_sum,
                             const moe_rows* grad_x, void* grad_weight, void* grad_bias, void* workspace,
                             size_t workspace_bytes, void* stream) {
  MOE_TRY(check_norm(p));
  MOE_TRY(check_rows(p, grad_y));
  MOE_TRY(check_rows(p, x));
  MOE_TRY(check_rows(p, grad_x));
  if (grad_sum) MOE_TRY(check_rows(p, grad_sum));
  if (!weight || (p->rows > 0 && !stats)) return MOE_ERR_NULL;
  if (!elem_aligned(weight, p->param_dtype) || (reinterpret_cast<uintptr_t>(stats) & 7u)) return MOE_ERR_LAYOUT;
  if (!elem_aligned(grad_weight, p->grad_dtype) || !elem_aligned(grad_bias, p->grad_dtype)) return MOE_ERR_LAYOUT;
  const bool sums = grad_weight || grad_bias;
  if (sums) {
    if (!workspace || workspace_bytes < moe_norm_workspace_bytes(p)) return MOE_ERR_WORKSPACE;
    if (!aligned16(workspace)) return MOE_ERR_LAYOUT;
  }
  const BwdShape b = bwd_shape(p);
  NormArgs a = norm_args(p, b.ept);
  a.dy = rows_of(grad_y); a.x = rows_of(x); a.gsum = rows_of(grad_sum); a.dx = rows_of(grad_x);
  a.w = weight;
  a.w16 = aligned16(weight);
  a.stats = const_cast<float*>(stats);
  a.part = sums && b.groups > 1 ? static_cast<float*>(workspace) : nullptr;
  a.gw = static_cast<uint8_t*>(grad_weight);
  a.gb = static_cast<uint8_t*>(grad_bias);
  a.g16 = p->grad_dtype == MOE_BF16;
  a.overwrite = (p->flags & MOE_NORM_OVERWRITE_GRADS) != 0;
  const bool vec = whole_pieces(p) && rows4(p, grad_y) && rows4(p, x) && rows4(p, grad_sum) && rows4(p, grad_x);
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (p->rows > 0) {
    MOE_TRY(launch("norm_bwd", st, [&] {
      with_variant<false>(b.ept, vec, p->dtype == MOE_BF16, [&](auto e, auto v, auto bf) {
        hipLaunchKernelGGL((k_norm_bwd<e(), v(), bf()>), dim3(b.groups), dim3(b.ng * a.tpr), b.lds, st, a);
      });
    }));
    if (!a.part) return MOE_OK;
  }
  if (!sums) return MOE_OK;
  // with no rows: an overwriting call leaves zeros
  const int width = a.N * ((a.gw ? 1 : 0) + (a.gb ? 1 : 0)), groups = p->rows > 0 ? b.groups : 0;
  return launch("norm_bwd_final", st, [&] {
    hipLaunchKernelGGL(k_norm_bwd_final, dim3((width + kFinalCols - 1) / kFinalCols), dim3(kFinalCols * kFinalLanes), 0,
                       st, (const float*)workspace, groups, width, a.N, a.gw ? a.gw : a.gb, a.gb, a.g16, a.overwrite);
  });
}

}  // extern "C"

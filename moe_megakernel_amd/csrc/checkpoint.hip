// Activation checkpoints in 8 bits (mxint8.hpp has the format): rows of values to codes and scale
// bytes, and back.  Both are one pass bound by memory: BF16 2 + 33/32 bytes a value, FP32 4 + 33/32 (8192 x 7168 BF16 put
// away and fetched: 72 us, 4.9 TB/s, a large copy's rate).
//
// A thread takes 8 neighbouring columns, the four threads of a quad a block.  Rows whose starts
// and length are multiples of 8 elements (16 bytes of BF16) move in whole pieces, others by
// elements.
#include <hip/hip_runtime.h>

#include "../../include/moe.h"
#include "checkpoint.hpp"
#include "host.hpp"
#include "mxint8.hpp"

namespace moe {
namespace checkpoint {

namespace {

constexpr int kThreads = 256;
constexpr int kPieces = 4;       // pieces of 8 columns a thread takes, kThreads apart

template <bool F32, bool STORE, bool WHOLE>
__global__ __launch_bounds__(kThreads) void k_checkpoint(Args a) {
  const uint32_t blocks = (uint32_t)((a.cols + 31) / 32), per_row = 4 * blocks;
  const int64_t total = a.rows * per_row;
  constexpr int ES = F32 ? 4 : 2;
  // the workgroup's first piece, then 32-bit steps from there
  const int64_t first = (int64_t)blockIdx.x * kPieces * kThreads, row0 = first / per_row;
  const uint32_t c0 = (uint32_t)(first - row0 * per_row);
  int64_t row[kPieces];
  uint32_t c8[kPieces];
  bool in[kPieces];
  float v[kPieces][8];
  uint2 q[kPieces];
  int s[kPieces];
  // every piece's loads go out before the first is used
#pragma unroll
  for (int u = 0; u < kPieces; ++u) {
    const uint32_t off = c0 + u * kThreads + threadIdx.x, r = off / per_row;
    in[u] = first + u * kThreads + threadIdx.x < total;
    row[u] = row0 + r;
    c8[u] = in[u] ? off - r * per_row : per_row;   // past the end: no columns
    const int64_t col = 8 * (int64_t)c8[u];
    if constexpr (STORE) {
      const uint8_t* p = a.x + (row[u] * a.ld + col) * ES;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[u][i] = 0.0f;
      if constexpr (WHOLE) {
        if (col < a.cols) {
          if constexpr (F32) {
            const f32x4_t x0 = reinterpret_cast<const f32x4_t*>(p)[0], x1 = reinterpret_cast<const f32x4_t*>(p)[1];
#pragma unroll
            for (int i = 0; i < 4; ++i) { v[u][i] = x0[i]; v[u][4 + i] = x1[i]; }
          } else {
            unpack_bf16x8(*reinterpret_cast<const uint4*>(p), v[u]);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (col + i < a.cols)
            v[u][i] = F32 ? reinterpret_cast<const float*>(p)[i] : bf2f(reinterpret_cast<const uint16_t*>(p)[i]);
      }
    } else {
      q[u] = make_uint2(0, 0);
      s[u] = 0;
      if (col < a.cols) {
        const uint8_t* p = a.codes + row[u] * a.cols + col;
        s[u] = a.scales[row[u] * blocks + (c8[u] >> 2)];
        if constexpr (WHOLE) {
          q[u] = *reinterpret_cast<const uint2*>(p);
        } else {
          uint32_t w[2] = {0, 0};
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (col + i < a.cols) w[i >> 2] |= (uint32_t)p[i] << (8 * (i & 3));
          q[u] = make_uint2(w[0], w[1]);
        }
      }
    }
  }
#pragma unroll
  for (int u = 0; u < kPieces; ++u) {
    const int64_t col = 8 * (int64_t)c8[u];
    if constexpr (STORE) {
      const int sb = int8_scale_byte(quad_max_u(abs_bits8(v[u])));
      if (!in[u] || col >= a.cols) continue;
      const uint2 codes = int8_codes8(v[u], sb);
      uint8_t* p = a.codes + row[u] * a.cols + col;
      if constexpr (WHOLE) {
        *reinterpret_cast<uint2*>(p) = codes;
      } else {
        const uint32_t w[2] = {codes.x, codes.y};
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (col + i < a.cols) p[i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
      }
      if ((c8[u] & 3) == 0) a.scales[row[u] * blocks + (c8[u] >> 2)] = (uint8_t)sb;
    } else {
      if (col >= a.cols) continue;
      float o[8];
      int8_values8(q[u], int8_step(s[u]), o);
      uint8_t* p = a.x + (row[u] * a.ld + col) * ES;
      if constexpr (WHOLE) {
        if constexpr (F32) {
          reinterpret_cast<f32x4_t*>(p)[0] = f32x4_t{o[0], o[1], o[2], o[3]};
          reinterpret_cast<f32x4_t*>(p)[1] = f32x4_t{o[4], o[5], o[6], o[7]};
        } else {
          *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf2(o[0], o[1]), pack_bf2(o[2], o[3]), pack_bf2(o[4], o[5]),
                                                    pack_bf2(o[6], o[7]));
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (col + i < a.cols) {
            if constexpr (F32) reinterpret_cast<float*>(p)[i] = o[i];
            else reinterpret_cast<uint16_t*>(p)[i] = (uint16_t)f2bf(o[i]);
          }
      }
    }
  }
}

int64_t groups(int64_t rows, int64_t cols) {
  const int64_t pieces = rows * 4 * ((cols + 31) / 32), each = (int64_t)kThreads * kPieces;
  return (pieces + each - 1) / each;
}

template <bool STORE>
void launch(hipStream_t st, const Args& a, bool fp32) {
  const int es = fp32 ? 4 : 2;
  const bool whole = a.cols % 8 == 0 && (a.ld * es) % 16 == 0 && aligned16(a.x) &&
                     (reinterpret_cast<uintptr_t>(a.codes) & 7u) == 0;
  const dim3 grid((unsigned)groups(a.rows, a.cols)), block(kThreads);
  if (fp32) {
    if (whole) hipLaunchKernelGGL((k_checkpoint<true, STORE, true>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((k_checkpoint<true, STORE, false>), grid, block, 0, st, a);
  } else {
    if (whole) hipLaunchKernelGGL((k_checkpoint<false, STORE, true>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((k_checkpoint<false, STORE, false>), grid, block, 0, st, a);
  }
}

moe_status check(const moe_checkpoint_problem* p, const moe_rows* x, const void* codes, const void* scales) {
  if (!p) return MOE_ERR_NULL;
  if (p->rows < 0 || p->cols < 1 || p->rows > (1ll << 31) || p->cols > MOE_CHECKPOINT_MAX_COLS) return MOE_ERR_SHAPE;
  if (!fits(p->rows, p->cols)) return MOE_ERR_SHAPE;
  if (p->dtype != MOE_BF16 && p->dtype != MOE_FP32) return MOE_ERR_DTYPE;
  if (p->rows == 0) return MOE_OK;
  if (!x || !x->base || !codes || !scales) return MOE_ERR_NULL;
  if (x->ld < p->cols || !elem_aligned(x->base, p->dtype)) return MOE_ERR_LAYOUT;
  return MOE_OK;
}

}  // namespace

bool fits(int64_t rows, int64_t cols) { return groups(rows, cols) < (1ll << 32) / kThreads; }
void launch_store(hipStream_t st, const Args& a, bool fp32) { launch<true>(st, a, fp32); }
void launch_load(hipStream_t st, const Args& a, bool fp32) { launch<false>(st, a, fp32); }

}  // namespace checkpoint
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_checkpoint_store(const moe_checkpoint_problem* p, const moe_rows* x, void* codes, void* scales,
                                void* stream) {
  MOE_TRY(checkpoint::check(p, x, codes, scales));
  if (p->rows == 0) return MOE_OK;
  const checkpoint::Args a{static_cast<uint8_t*>(x->base), x->ld, p->rows, p->cols, static_cast<uint8_t*>(codes),
                           static_cast<uint8_t*>(scales)};
  hipStream_t st = static_cast<hipStream_t>(stream);
  return launch("checkpoint_store", st, [&] { checkpoint::launch_store(st, a, p->dtype == MOE_FP32); });
}

moe_status moe_checkpoint_load(const moe_checkpoint_problem* p, const void* codes, const void* scales,
                               const moe_rows* x, void* stream) {
  MOE_TRY(checkpoint::check(p, x, codes, scales));
  if (p->rows == 0) return MOE_OK;
  const checkpoint::Args a{static_cast<uint8_t*>(x->base), x->ld, p->rows, p->cols,
                           static_cast<uint8_t*>(const_cast<void*>(codes)),
                           static_cast<uint8_t*>(const_cast<void*>(scales))};
  hipStream_t st = static_cast<hipStream_t>(stream);
  return launch("checkpoint_load", st, [&] { checkpoint::launch_load(st, a, p->dtype == MOE_FP32); });
}

}  // extern "C"

// The layer's forward for a few tokens, in two kernels.
//
//   k_decode_fc1:  h_r = silu(min(a, L)) clamp(b, -L, L), a = Wg_e x_t, b = Wu_e x_t,  r = (t, k)
//   k_decode_fc2:  out_t = s_t Wd_s h_ts + sum_k w_tk Wd_e h_tk
//
// With few tokens the time is the time to read the chosen experts' weights once; the
// matrix instructions are far from their limit even with most token columns empty.  So
// weights go from memory straight to registers as the 16-row operand of
// v_mfma_f32_16x16x32_bf16, tokens are its 16 columns, and nothing but partial sums passes
// through LDS.  A lane holds 16 consecutive elements of its row per 64 of the contraction
// (32 bytes of BF16, 16 of E4M3): any assignment of elements to lanes is right as long as
// both operands use the same one, and this one makes every load 16 bytes wide in both
// formats and keeps a lane inside one block of 32 scaled elements.
//
// MXFP8 weights are decoded to BF16 in registers, which is exact (E4M3 has 3 fraction
// bits and the scale is a power of two); the tokens stay BF16.  h is rounded to BF16, as
// moe_forward stores it.  Accumulators, the SwiGLU and the combine are FP32, and the output is
// rounded once.  Every sum has a fixed order.
#include <hip/hip_runtime.h>

#include "decode.hpp"

namespace moe {
namespace decode {

namespace {

constexpr int kStep = 128;          // elements of the contraction per step (the ABI's multiple)
constexpr int kFc1Waves = 4, kFc2Waves = 8;

// One step of 16 weight rows: lane (r = lane & 15, q = lane >> 4) has elements
// 64 s + 16 q .. + 15 of row r, s = 0, 1.
template <bool MX>
struct WStep;
template <>
struct WStep<false> {
  uint4 v[4];
  __device__ __forceinline__ void load(const uint8_t* p, const uint8_t*) {
    v[0] = *reinterpret_cast<const uint4*>(p);
    v[1] = *reinterpret_cast<const uint4*>(p + 16);
    v[2] = *reinterpret_cast<const uint4*>(p + 128);
    v[3] = *reinterpret_cast<const uint4*>(p + 144);
  }
  // the 8 elements 64 s + 16 q + 8 u ..
  __device__ __forceinline__ bf16x8_t frag(int s, int u, int) const {
    return __builtin_bit_cast(bf16x8_t, v[2 * s + u]);
  }
  static constexpr int kBytes = 2 * kStep, kLane = 32;   // bytes per row and step; per q
};
template <>
struct WStep<true> {
  uint4 v[2];
  uint32_t sc;   // E8M0 of the row's four blocks of 32
  __device__ __forceinline__ void load(const uint8_t* p, const uint8_t* s) {
    v[0] = *reinterpret_cast<const uint4*>(p);
    v[1] = *reinterpret_cast<const uint4*>(p + 64);
    sc = *reinterpret_cast<const uint32_t*>(s);
  }
  __device__ __forceinline__ bf16x8_t frag(int s, int u, int q) const {
    const float scale = __uint_as_float(((sc >> (16 * s + 8 * (q >> 1))) & 0xffu) << 23);
    const uint32_t lo = u ? v[s].z : v[s].x, hi = u ? v[s].w : v[s].y;
    typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
    const u32x4_t r = {
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false)),
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true)),
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false)),
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true))};
    return __builtin_bit_cast(bf16x8_t, r);
  }
  static constexpr int kBytes = kStep, kLane = 16;
};

// acc[f] += W (16 rows) X_f^T (16 columns) over n steps.  w, ws: the lane's row at its first
// element (scales: the row's first block); x[f]: the lane's column at its first element.
// D steps are in flight; the steady loop has no conditions.
template <bool MX, int NF, int D>
__device__ __forceinline__ void dot_steps(const uint8_t* w, const uint8_t* ws, const uint8_t* const (&x)[NF], int n,
                                          f32x4_t (&acc)[NF]) {
  const int q = (threadIdx.x & 63) >> 4;
  WStep<MX> wr[D];
  WStep<false> xr[D][NF];
  auto load = [&](int d, int i) __attribute__((always_inline)) {
    wr[d].load(w + (int64_t)i * WStep<MX>::kBytes, ws + i * 4);
#pragma unroll
    for (int f = 0; f < NF; ++f) xr[d][f].load(x[f] + i * WStep<false>::kBytes, nullptr);
  };
  auto mul = [&](int d) __attribute__((always_inline)) {
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const bf16x8_t a = wr[d].frag(s, u, q);
#pragma unroll
        for (int f = 0; f < NF; ++f)
          acc[f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, xr[d][f].frag(s, u, q), acc[f], 0, 0, 0);
      }
  };
#pragma unroll
  for (int d = 0; d < D; ++d)
    if (d < n) load(d, d);
  int i = 0;
  for (; i + 2 * D <= n; i += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      mul(d);
      load(d, i + D + d);
    }
  }
#pragma unroll
  for (int d = 0; d < D; ++d)
    if (i + d < n) {
      mul(d);
      if (i + D + d < n) load(d, i + D + d);
    }
#pragma unroll
  for (int d = 0; d < D; ++d)
    if (i + D + d < n) mul(d);
}

// Steps in flight by the number of 16-token column groups: about 100 registers each.
template <int NF>
constexpr int depth() { return NF == 1 ? 2 : 1; }

__device__ __forceinline__ float swiglu(float a, float b, float L) {
  if (L > 0.0f) {   // comparisons that keep a NaN
    a = a > L ? L : a;
    b = b > L ? L : (b < -L ? -L : b);
  }
  return a * sigmoidf_(a) * b;
}

// ---------------------------------------------------------------- FC1 + SwiGLU
// A workgroup computes 8 intermediate columns of one expert for all its tokens: the 16
// operand rows are 8 gate and 8 up rows in turn, and its 4 waves split the contraction.
// Grid: [plan] [shared expert's tiles] [min(E, T K) experts' tiles] [gate scores, 4 tokens each].
struct Fc1Shared {
  uint32_t mask[8];
  int16_t id[kMaxRoutes];          // expert of each route, -1: none
  int16_t list[kMaxTokens];        // the group's routes
  int count, invalid;
};

// Marks the experts in use; every thread returns behind a barrier.
__device__ __forceinline__ void read_table(const Args& a, Fc1Shared& s) {
  const int tid = threadIdx.x, n = a.T * a.K;
  if (tid < 8) s.mask[tid] = 0;
  if (tid == 0) s.invalid = 0;
  for (int i = tid; i < n; i += 64 * kFc1Waves) {
    const int e = a.top[i];
    s.id[i] = (int16_t)(e >= 0 && e < a.E ? e : (e == -1 ? -1 : -2));
  }
  __syncthreads();
  int keep[(kMaxRoutes + 64 * kFc1Waves - 1) / (64 * kFc1Waves)];
#pragma unroll
  for (int u = 0; u < kMaxRoutes / (64 * kFc1Waves); ++u) {
    const int i = tid + u * 64 * kFc1Waves;
    int e = i < n ? s.id[i] : -1;
    for (int j = i - i % a.K; j < i && i < n; ++j)   // an expert listed again in its row is dropped
      if (e >= 0 && s.id[j] == e) e = -2;
    keep[u] = e;
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kMaxRoutes / (64 * kFc1Waves); ++u) {
    const int i = tid + u * 64 * kFc1Waves;
    if (i < n) {
      if (keep[u] == -2) s.invalid = 1;
      s.id[i] = (int16_t)(keep[u] < 0 ? -1 : keep[u]);
      if (keep[u] >= 0) atomicOr(&s.mask[keep[u] >> 5], 1u << (keep[u] & 31));
    }
  }
  __syncthreads();
}

// Expert of group g (ascending), or -1 past the last.
__device__ __forceinline__ int group_expert(const Fc1Shared& s, int g) {
  for (int w = 0; w < 8; ++w) {
    uint32_t m = s.mask[w];
    const int c = __popc(m);
    if (g < c) {
      for (; g > 0; --g) m &= m - 1;
      return 32 * w + __ffs(m) - 1;
    }
    g -= c;
  }
  return -1;
}

// The routes of expert e in order (wave 0; visible behind the next barrier).
__device__ __forceinline__ void list_routes(const Args& a, Fc1Shared& s, int e) {
  if (threadIdx.x >= 64) return;
  const int lane = threadIdx.x, n = a.T * a.K;
  int pos = 0;
  for (int i0 = 0; i0 < n; i0 += 64) {
    const int i = i0 + lane;
    const bool hit = i < n && s.id[i] == e;
    const uint64_t m = __ballot(hit);
    if (hit) s.list[pos + __popcll(m & ((1ull << lane) - 1))] = (int16_t)i;
    pos += __popcll(m);
  }
  if (lane == 0) s.count = pos;
}

// The first workgroup leaves the plan for the second kernel: one wave a group lists its
// routes by ballot, at the sum of the counts of the groups before it.
__device__ __forceinline__ void write_plan(const Args& a, Fc1Shared& s, int* cnt /* LDS [kMaxExperts + 1] */) {
  const int tid = threadIdx.x, n = a.T * a.K, lane = tid & 63;
  if (tid == 0) a.plan->status = s.invalid ? 9 /* MOE_ERR_ROUTE_INVALID */ : 0;
  for (int e = tid; e <= kMaxExperts; e += 64 * kFc1Waves) cnt[e] = 0;
  __syncthreads();
  for (int i = tid; i < n; i += 64 * kFc1Waves)
    if (s.id[i] >= 0) atomicAdd(&cnt[s.id[i]], 1);
  __syncthreads();
  int groups = 0;
  for (int w = 0; w < 8; ++w) groups += __popc(s.mask[w]);
  for (int g = tid >> 6; g <= groups; g += kFc1Waves) {
    const int e = group_expert(s, g);       // -1 for the end mark
    int before = 0;
    for (int f = lane; f < (e < 0 ? kMaxExperts : e); f += 64) before += cnt[f];
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) before += __shfl_xor(before, o);
    if (lane == 0) {
      a.plan->first[g] = before;
      if (e >= 0) a.plan->expert[g] = e;
      else a.plan->groups = groups;
    }
    if (e < 0) break;
    for (int i0 = 0; i0 < n; i0 += 64) {
      const bool hit = i0 + lane < n && s.id[i0 + lane] == e;
      const uint64_t m = __ballot(hit);
      if (hit) a.plan->route[before + __popcll(m & ((1ull << lane) - 1))] = i0 + lane;
      before += __popcll(m);
    }
  }
}

template <bool MX, int NF>
__device__ __forceinline__ void fc1_tile(const Args& a, const Fc1Shared& s, float* red, int e, int i0, int count) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, q = lane >> 4;
  const int row = i0 + (r >> 1);
  const uint8_t *w, *ws = nullptr;
  if (e < 0) {
    w = (r & 1 ? a.sup : a.sgate).row(0, row);
  } else {
    const MxRef& m = r & 1 ? a.up : a.gate;
    w = m.data.row(e, row);
    if constexpr (MX) ws = m.scale.row(e, row);
  }
  const int steps = a.H / kStep;
  const int s0 = wave * steps / kFc1Waves, s1 = (wave + 1) * steps / kFc1Waves;
  w += (int64_t)s0 * WStep<MX>::kBytes + q * WStep<MX>::kLane;
  ws += s0 * 4;
  const uint8_t* x[NF];
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    const int c = 16 * f + r < count ? 16 * f + r : 0;     // columns past the last repeat the first
    const int t = e < 0 ? c : s.list[c] / a.K;
    x[f] = reinterpret_cast<const uint8_t*>(a.x + (int64_t)t * a.H) + (int64_t)s0 * WStep<false>::kBytes +
           q * WStep<false>::kLane;
  }
  f32x4_t acc[NF];
#pragma unroll
  for (int f = 0; f < NF; ++f) acc[f] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  dot_steps<MX, NF, depth<NF>()>(w, ws, x, s1 - s0, acc);
  // [wave][column][row]: a lane has rows 4 q .. 4 q + 3 of column r
#pragma unroll
  for (int f = 0; f < NF; ++f)
    *reinterpret_cast<f32x4_t*>(red + ((wave * NF + f) * 16 + r) * 16 + 4 * q) = acc[f];
  __syncthreads();
  for (int o = threadIdx.x; o < 8 * count; o += 64 * kFc1Waves) {
    const int c = o >> 3, p = o & 7;
    float g = 0.0f, u = 0.0f;
#pragma unroll
    for (int v = 0; v < kFc1Waves; ++v) {
      const float2 z = *reinterpret_cast<const float2*>(red + (v * NF * 16 + c) * 16 + 2 * p);
      g += z.x;
      u += z.y;
    }
    const int64_t hrow = e < 0 ? (int64_t)a.T * a.K + c : s.list[c];
    a.h[hrow * a.I + i0 + p] = (uint16_t)f2bf(swiglu(g, u, a.limit));
  }
}

template <bool MX>
__device__ __forceinline__ void fc1_group(const Args& a, const Fc1Shared& s, float* red, int e, int i0, int count) {
  if (count <= 16) fc1_tile<MX, 1>(a, s, red, e, i0, count);
  else if (count <= 32) fc1_tile<MX, 2>(a, s, red, e, i0, count);
  else fc1_tile<MX, 4>(a, s, red, e, i0, count);
}

template <bool MX>
__global__ __launch_bounds__(64 * kFc1Waves, 4) void k_decode_fc1(Args a) {
  __shared__ Fc1Shared s;
  __shared__ __align__(16) float red[kFc1Waves * 4 * 256];
  const int tiles = a.I / 8;
  const int shared_blocks = a.shared ? tiles : 0;
  const int routed_blocks = min(a.E, a.T * a.K) * tiles;
  if (blockIdx.x == 0) {
    read_table(a, s);
    write_plan(a, s, reinterpret_cast<int*>(red));
    return;
  }
  int b = blockIdx.x - 1;
  if (b >= shared_blocks + routed_blocks) {   // shared output gate: one wave a token
    const int t = (b - shared_blocks - routed_blocks) * kFc1Waves + (threadIdx.x >> 6), lane = threadIdx.x & 63;
    if (t >= a.T) return;
    float v = 0.0f;
    for (int c = lane; c < a.H / 8; c += 64) {
      float p[8], g[8];
      unpack_bf16x8(reinterpret_cast<const uint4*>(a.x + (int64_t)t * a.H)[c], p);
      unpack_bf16x8(reinterpret_cast<const uint4*>(a.gw)[c], g);
#pragma unroll
      for (int i = 0; i < 8; ++i) v += p[i] * g[i];
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
    if (lane == 0) a.gate_s[t] = 1.0f / (1.0f + expf(-v));
    return;
  }
  if (b < shared_blocks) {
    fc1_group<false>(a, s, red, -1, b * 8, a.T);
    return;
  }
  b -= shared_blocks;
  read_table(a, s);
  const int e = group_expert(s, b / tiles);
  if (e < 0) return;
  list_routes(a, s, e);
  __syncthreads();
  fc1_group<MX>(a, s, red, e, b % tiles * 8, s.count);
}

// ---------------------------------------------------------------- FC2 + combine
// A workgroup owns 16 output columns of every token.  Its 8 waves split the steps of all
// experts in use evenly; each adds w_tk times what it has of an expert's product to an
// accumulator [token][16] of its own in LDS, and the waves' accumulators are joined in
// order at the end.
struct Fc2Shared {
  int32_t expert[kMaxExperts + 1], first[kMaxExperts + 2];
  int16_t route[kMaxRoutes], token[kMaxRoutes];
  float weight[kMaxRoutes], gate[kMaxTokens];
};

template <bool MX, int NF>
__device__ __forceinline__ void fc2_part(const Args& a, const Fc2Shared& s, float* acc_lds, int n0, int e, int first,
                                         int count, int s0, int n) {
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const uint8_t *w, *ws = nullptr;
  if (e < 0) {
    w = a.sdown.row(0, n0 + r);
  } else {
    w = a.down.data.row(e, n0 + r);
    if constexpr (MX) ws = a.down.scale.row(e, n0 + r);
  }
  w += (int64_t)s0 * WStep<MX>::kBytes + q * WStep<MX>::kLane;
  ws += s0 * 4;
  const uint8_t* x[NF];
  int tok[NF];
  float wt[NF];
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    const int c = 16 * f + r;
    const bool on = c < count;
    const int cc = on ? c : 0;
    tok[f] = !on ? -1 : (e < 0 ? cc : s.token[first + cc]);
    wt[f] = e < 0 ? s.gate[cc] : s.weight[first + cc];
    const int64_t hrow = e < 0 ? (int64_t)a.T * a.K + cc : s.route[first + cc];
    x[f] = reinterpret_cast<const uint8_t*>(a.h + hrow * a.I) + (int64_t)s0 * WStep<false>::kBytes +
           q * WStep<false>::kLane;
  }
  f32x4_t acc[NF];
#pragma unroll
  for (int f = 0; f < NF; ++f) acc[f] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  dot_steps<MX, NF, depth<NF>()>(w, ws, x, n, acc);
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    if (tok[f] < 0) continue;
    f32x4_t* o = reinterpret_cast<f32x4_t*>(acc_lds + tok[f] * 16 + 4 * q);   // the wave's own
    f32x4_t v = *o;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += wt[f] * acc[f][i];
    *o = v;
  }
}

template <bool MX>
__device__ __forceinline__ void fc2_group(const Args& a, const Fc2Shared& s, float* acc_lds, int n0, int e, int first,
                                          int count, int s0, int n) {
  if (count <= 16) fc2_part<MX, 1>(a, s, acc_lds, n0, e, first, count, s0, n);
  else if (count <= 32) fc2_part<MX, 2>(a, s, acc_lds, n0, e, first, count, s0, n);
  else fc2_part<MX, 4>(a, s, acc_lds, n0, e, first, count, s0, n);
}

template <bool MX>
__global__ __launch_bounds__(64 * kFc2Waves, 2) void k_decode_fc2(Args a) {
  extern __shared__ __align__(16) float acc_all[];   // [kFc2Waves][T][16]
  __shared__ Fc2Shared s;
  const int tid = threadIdx.x, wave = tid >> 6;
  const int routed = a.plan->groups;
  for (int g = tid; g < routed; g += 64 * kFc2Waves) s.expert[g] = a.plan->expert[g];
  for (int g = tid; g <= routed; g += 64 * kFc2Waves) s.first[g] = a.plan->first[g];
  const int routes = a.plan->first[routed];
  for (int i = tid; i < routes; i += 64 * kFc2Waves) {
    const int rt = a.plan->route[i];
    s.route[i] = (int16_t)rt;
    s.token[i] = (int16_t)(rt / a.K);
    s.weight[i] = a.rw[rt];
  }
  if (tid < a.T) s.gate[tid] = a.gw ? a.gate_s[tid] : 1.0f;
  for (int i = tid; i < kFc2Waves * a.T * 16; i += 64 * kFc2Waves) acc_all[i] = 0.0f;
  __syncthreads();

  float* mine = acc_all + wave * a.T * 16;
  const int n0 = blockIdx.x * 16, steps = a.I / kStep;
  const int groups = routed + (a.shared ? 1 : 0);
  const int64_t total = (int64_t)groups * steps;
  int64_t p = wave * total / kFc2Waves;
  const int64_t end = (wave + 1) * total / kFc2Waves;
  while (p < end) {
    const int g = (int)(p / steps), s0 = (int)(p % steps);
    const int n = (int)min((int64_t)(steps - s0), end - p);
    if (a.shared && g == 0) {
      fc2_group<false>(a, s, mine, n0, -1, 0, a.T, s0, n);
    } else {
      const int u = g - (a.shared ? 1 : 0);
      fc2_group<MX>(a, s, mine, n0, s.expert[u], s.first[u], s.first[u + 1] - s.first[u], s0, n);
    }
    p += n;
  }
  __syncthreads();
  for (int o = tid; o < a.T * 16; o += 64 * kFc2Waves) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kFc2Waves; ++w) v += acc_all[w * a.T * 16 + o];
    a.out[(int64_t)(o >> 4) * a.H + n0 + (o & 15)] = (uint16_t)f2bf(v);
  }
}

}  // namespace

template <bool MX>
void launch_fc1(hipStream_t st, const Args& a) {
  const int tiles = a.I / 8, used = a.E < a.T * a.K ? a.E : a.T * a.K;
  const int gate = a.gw ? (a.T + kFc1Waves - 1) / kFc1Waves : 0;
  hipLaunchKernelGGL((k_decode_fc1<MX>), dim3((unsigned)(1 + (used + (a.shared ? 1 : 0)) * tiles + gate)),
                     dim3(64 * kFc1Waves), 0, st, a);
}
template <bool MX>
void launch_fc2(hipStream_t st, const Args& a) {
  hipLaunchKernelGGL((k_decode_fc2<MX>), dim3(a.H / 16), dim3(64 * kFc2Waves),
                     (size_t)kFc2Waves * a.T * 16 * sizeof(float), st, a);
}
template void launch_fc1<false>(hipStream_t, const Args&);
template void launch_fc1<true>(hipStream_t, const Args&);
template void launch_fc2<false>(hipStream_t, const Args&);
template void launch_fc2<true>(hipStream_t, const Args&);

}  // namespace decode
}  // namespace moe

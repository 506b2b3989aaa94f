// The layer's forward for a few tokens, in two kernels.
//
//   k_decode_fc1:  h_r = silu(min(a, L)) clamp(b, -L, L), a = Wg_e x_t, b = Wu_e x_t,  r = (t, k)
//   k_decode_fc2:  out_t = s_t Wd_s h_ts + sum_k w_tk Wd_e h_tk
//
// With few tokens the time is the time to read the chosen experts' weights once; the matrix
// instructions are far from their limit even with most token columns empty.  So weights are
// the 16-row operand of v_mfma_f32_16x16x32_bf16, tokens its 16 columns, each wave runs its own
// stretch of the contraction with its own loads in flight, and waves meet only to add up
// partial sums.
//
// What it reaches (read floor: the weights in use at 6.35 TB/s, what a plain read kernel gets):
//   1 token, 96 BF16 experts top-4, H 4096, I 1024, shared expert    28 us, floor 20
//   7 tokens, the same with E4M3 experts                             70 us, floor 55
//   19 tokens, BF16, no shared expert                               215 us, floor 196
//   64 tokens, 64 E4M3 experts top-6, H 7168, I 2048                570 us, floor 471
// Bound by the weight stream, in the last case with the reads of h; at one token by the two kernels'
// start and end (about 4 us each: table, first loads, last sums).
//
// MXFP8 weights are decoded to BF16 in registers, which is exact (E4M3 has 3 fraction
// bits and the scale is a power of two) wherever the product is a normal BF16 number; the tokens
// stay BF16.  h is held in two BF16 parts, 16 of its 24 bits, so that nothing but the output is
// rounded to BF16: its error against 64 bits is 0.166% of its size, a plain FP32 form's too, and
// 0.235% with h in one part.  That costs at most 2.5% up to 16 tokens (empty columns of a fragment
// hold the second part) and 5% with BF16 weights up to 32 tokens an expert, but with many tokens and
// E4M3 the doubled reads of h show: 570 us against 528 in the last case above, 171 against 139 where
// experts get 33 of 64 tokens.  Accumulators, the SwiGLU and the combine are FP32.  Every sum has a
// fixed order.
#include <hip/hip_runtime.h>

#include "decode.hpp"
#include "reduce.hpp"

namespace moe {
namespace decode {

namespace {

constexpr int kStep = 128;          // elements of the contraction per step (the ABI's multiple)
constexpr int kFc1Waves = 4;

// Loads through global (not flat) addresses: the pointers may come out of a table in
// memory, which hides their address space, and a flat load is waited for with every other
// load in flight.
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
__device__ __forceinline__ uint4 ld16(const uint8_t* p) {
  const u32x4_t v = *(const __attribute__((address_space(1))) u32x4_t*)(uintptr_t)p;
  return make_uint4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ uint32_t ld4(const uint8_t* p) {
  return *(const __attribute__((address_space(1))) uint32_t*)(uintptr_t)p;
}

// One step is 128 elements of the contraction, four products of 32.  Lane (r, q) of a
// product (r = lane & 15, q = lane >> 4) holds 8 elements of row r (weights) or column r
// (tokens); which 8 is free as long as both operands agree:
//   BF16 weights:  product j takes elements 32 j + 8 q .. + 7
//   E4M3 weights:  products 2 s and 2 s + 1 take elements 64 s + 16 q .. + 7 and + 8 .. + 15, so
//                  that a lane's 16 bytes serve two products and lie in one block of 32
// Loading straight into that layout would give neighbouring lanes different rows, and the
// address unit then handles one lane a clock: 64 clocks a load instead of 16 (measured on
// E4M3 experts, 64 tokens, H 7168: 327 us against 244 us).  So a load takes 64 consecutive bytes
// of 16 rows, four lanes a row, and each wave turns it round through 1 KB of LDS of its
// own.  LDS operations of a wave run in order, so one such slot serves every load in turn and
// needs no barrier.

// Slot position (16-byte cells) of chunk c of row `row`: rows two apart land in different
// banks, for the writes (2 rows, 4 chunks by 8 lanes) and the reads (8 rows, one chunk) alike.
__device__ __forceinline__ int cell(int row, int c) { return 4 * row + (c ^ ((row >> 1) & 3)); }

// The wave's turn-round slots: one for weights, two for tokens (E4M3 products take their
// 8 elements from every other chunk of two loads).
struct Turn {
  uint4* w;
  uint4* x;
  uint32_t* scale;         // [R][16][kScaleRow] (MXFP8)
  int put;                 // cell this lane's loads go to
  int row, q;              // the lane's row and element group in a product
};
constexpr int kTurnCells = 3 * 64;

// E8M0 scales of up to kScaleSteps steps of 16 rows: a row's four bytes of a step are far from
// the next row's, so fetching them step by step would cost as many cache lines as the
// weights; the four lanes of a row fetch four steps at once, and products read them here.
constexpr int kScaleSteps = 16, kScaleRow = kScaleSteps + 1;      // words; the odd stride spreads rows over banks
constexpr int kScaleCells = 16 * kScaleRow / 4;

// A wave's LDS for row fragments 0 .. R - 1, in 16-byte cells.
template <bool MX, int R>
constexpr int wave_cells() { return kTurnCells + (MX ? R * kScaleCells : 0); }
__device__ __forceinline__ Turn turn_of(uint4* scratch) {
  const int lane = threadIdx.x & 63;
  return {scratch, scratch + 64, reinterpret_cast<uint32_t*>(scratch + kTurnCells), cell(lane >> 2, lane & 3),
          lane & 15, lane >> 4};
}

// 16 token columns, one step: lane l loads chunk l & 3 (16 bytes) of column l >> 2.  A column's
// 64-byte pieces are PITCH bytes apart.
template <int PITCH>
struct XStep {
  uint4 v[4];
  __device__ __forceinline__ void load(const uint8_t* p) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = ld16(p + PITCH * j);
  }
  // products 2 s and 2 s + 1
  template <bool MX>
  __device__ __forceinline__ void frags(const Turn& t, int s, bf16x8_t (&o)[2]) const {
    t.x[t.put] = v[2 * s];
    t.x[64 + t.put] = v[2 * s + 1];
#pragma unroll
    for (int u = 0; u < 2; ++u)   // E4M3: elements 64 s + 16 q + 8 u .. are chunk 2 q + u of the eight
      o[u] = __builtin_bit_cast(bf16x8_t, MX ? t.x[(t.q >> 1) * 64 + cell(t.row, 2 * (t.q & 1) + u)]
                                             : t.x[u * 64 + cell(t.row, t.q)]);
  }
  static constexpr int kBytes = 4 * PITCH;
};
constexpr int kXPitch = 64;       // x: rows of consecutive elements
constexpr int kHPitch = 128;      // h: see h_index

// 16 weight rows, one step: lane l loads chunk l & 3 of row l >> 2.
template <bool MX>
struct WStep;
template <>
struct WStep<false> {
  uint4 v[4];
  __device__ __forceinline__ void load(const uint8_t* p) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = ld16(p + 64 * j);
  }
  __device__ __forceinline__ void frags(const Turn& t, int s, int, bf16x8_t (&o)[2]) const {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      t.w[t.put] = v[2 * s + u];
      o[u] = __builtin_bit_cast(bf16x8_t, t.w[cell(t.row, t.q)]);
    }
  }
  static constexpr int kBytes = 2 * kStep;
};
template <>
struct WStep<true> {
  uint4 v[2];
  __device__ __forceinline__ void load(const uint8_t* p) {
    v[0] = ld16(p);
    v[1] = ld16(p + 64);
  }
  // word: the step's place in t.scale (of row 0)
  __device__ __forceinline__ void frags(const Turn& t, int s, int word, bf16x8_t (&o)[2]) const {
    const uint32_t sr = t.scale[word + t.row * kScaleRow];
    t.w[t.put] = v[s];
    const uint4 b = t.w[cell(t.row, t.q)];
    const float scale = __uint_as_float(((sr >> (16 * s + 8 * (t.q >> 1))) & 0xffu) << 23);
    o[0] = decode8(b.x, b.y, scale);
    o[1] = decode8(b.z, b.w, scale);
  }
  __device__ static __forceinline__ bf16x8_t decode8(uint32_t lo, uint32_t hi, float scale) {
    const u32x4_t r = {
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false)),
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true)),
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false)),
        __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true))};
    return __builtin_bit_cast(bf16x8_t, r);
  }
  static constexpr int kBytes = kStep;
};

// acc[g][f] += W_g (16 rows) X_f^T (16 columns) over n steps (MXFP8: at most kScaleSteps).
// w, ws: the loading lane's rows at their first element (scales: the rows' first block); x: the
// loading lane's columns at their first element.  D steps are in flight; the steady loop
// has no conditions.
template <bool MX, int R, int NF, int D, int PITCH>
__device__ __forceinline__ void dot_chunk(const Turn& t, const uint8_t* const (&w)[R], const uint8_t* const (&ws)[R],
                                          const uint8_t* const (&x)[NF], int n, f32x4_t (&acc)[R][NF]) {
  WStep<MX> wr[D][R];
  XStep<PITCH> xr[D][NF];
  auto load = [&](int d, int i) __attribute__((always_inline)) {
#pragma unroll
    for (int g = 0; g < R; ++g) wr[d][g].load(w[g] + (int64_t)i * WStep<MX>::kBytes);
#pragma unroll
    for (int f = 0; f < NF; ++f) xr[d][f].load(x[f] + i * XStep<PITCH>::kBytes);
  };
  auto mul = [&](int d, int i) __attribute__((always_inline)) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      bf16x8_t b[NF][2];
#pragma unroll
      for (int f = 0; f < NF; ++f) xr[d][f].template frags<MX>(t, s, b[f]);
#pragma unroll
      for (int g = 0; g < R; ++g) {
        bf16x8_t a[2];
        wr[d][g].frags(t, s, g * 16 * kScaleRow + i, a);
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int f = 0; f < NF; ++f)
            acc[g][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[u], b[f][u], acc[g][f], 0, 0, 0);
      }
    }
  };
  [[maybe_unused]] uint32_t sc[R][kScaleSteps / 4];
  const int lane = threadIdx.x & 63;
  if constexpr (MX) {
#pragma unroll
    for (int g = 0; g < R; ++g)
#pragma unroll
      for (int m = 0; m < kScaleSteps / 4; ++m) sc[g][m] = ld4(ws[g] + 4 * min(4 * m + (lane & 3), n - 1));
  }
#pragma unroll
  for (int d = 0; d < D; ++d)
    if (d < n) load(d, d);
  if constexpr (MX) {
#pragma unroll
    for (int g = 0; g < R; ++g)
#pragma unroll
      for (int m = 0; m < kScaleSteps / 4; ++m)
        t.scale[(g * 16 + (lane >> 2)) * kScaleRow + 4 * m + (lane & 3)] = sc[g][m];
  }
  int i = 0;
  for (; i + 2 * D <= n; i += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      mul(d, i + d);
      load(d, i + D + d);
      __builtin_amdgcn_sched_barrier(0);   // the next stage's products stay behind these loads
    }
  }
#pragma unroll
  for (int d = 0; d < D; ++d)
    if (i + d < n) {
      mul(d, i + d);
      if (i + D + d < n) load(d, i + D + d);
    }
#pragma unroll
  for (int d = 0; d < D; ++d)
    if (i + D + d < n) mul(d, i + D + d);
}

template <bool MX, int R, int NF, int D, int PITCH>
__device__ __forceinline__ void dot_steps(const Turn& t, const uint8_t* const (&w)[R], const uint8_t* const (&ws)[R],
                                          const uint8_t* const (&x)[NF], int n, f32x4_t (&acc)[R][NF]) {
  if constexpr (!MX) {
    dot_chunk<MX, R, NF, D, PITCH>(t, w, ws, x, n, acc);
  } else {
    const uint8_t *wc[R], *wsc[R], *xc[NF];
    for (int i0 = 0; i0 < n; i0 += kScaleSteps) {
#pragma unroll
      for (int g = 0; g < R; ++g) {
        wc[g] = w[g] + (int64_t)i0 * WStep<MX>::kBytes;
        wsc[g] = ws[g] + i0 * 4;
      }
#pragma unroll
      for (int f = 0; f < NF; ++f) xc[f] = x[f] + (int64_t)i0 * XStep<PITCH>::kBytes;
      dot_chunk<MX, R, NF, D, PITCH>(t, wc, wsc, xc, min(kScaleSteps, n - i0), acc);
    }
  }
}

__device__ __forceinline__ float swiglu(float a, float b, float L) {
  if (L > 0.0f) {   // comparisons that keep a NaN
    a = a > L ? L : a;
    b = b > L ? L : (b < -L ? -L : b);
  }
  return a * sigmoidf_(a) * b;
}

// h's two parts are its rounding to BF16 and what that left (of an infinite or NaN h: 0), 32 upper
// parts and then their 32 lower ones in each 128-byte line.  The second product takes both as columns
// of one fragment, so a load touches each line once, as a whole (parts in two rows, half a line a
// load: 308 us against 291 with 12 tokens for each of 32 BF16 experts of H 7168).
constexpr int kHLower = 32;
__device__ __forceinline__ int64_t h_index(int64_t row, int i, int I) {
  return row * 2 * I + (i >> 5) * 64 + (i & 31);
}

// ---------------------------------------------------------------- FC1 + SwiGLU
// A tile is 8 R intermediate columns of one expert for all its tokens: each fragment of 16 rows is
// 8 gate and 8 up rows in turn, so that a pair ends in one lane's neighbouring sums.  A
// workgroup's 4 waves split the contraction of one tile, or (COLS) take a tile each.
// Grid: [plan] [shared expert's tiles] [min(E, T K) experts' tiles] [gate scores, 4 tokens each].
struct Fc1Shared {
  uint32_t mask[8];
  int16_t raw[kMaxRoutes];         // the table; -2: outside [-1, E)
  int16_t id[kMaxRoutes];          // expert of each route; < 0: none
  int16_t list[kMaxTokens];        // the group's routes
};

// A wave's copy of the routes' experts: lane l has routes 64 u + l.
constexpr int kRouteRegs = kMaxRoutes / 64;
struct Routes {
  int id[kRouteRegs];
};

// Reads the table, drops invalid entries (outside [0, E), or listed before in their row) and
// marks the experts in use.  Returns whether this thread saw an invalid entry.
template <int NT>
__device__ __forceinline__ bool read_table(const Args& a, Fc1Shared& s, Routes& rt) {
  constexpr int U = kMaxRoutes / NT;
  const int tid = threadIdx.x, n = a.T * a.K;
  int e[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int i = tid + u * NT;
    e[u] = i < n ? a.top[i] : -1;
    if (e[u] < -1 || e[u] >= a.E) e[u] = -2;
    s.raw[i] = (int16_t)e[u];
  }
  if (tid < 8) s.mask[tid] = 0;
  __syncthreads();
  bool invalid = false;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int i = tid + u * NT, k = i % a.K;
    bool again = false;
#pragma unroll
    for (int d = 1; d < kMaxTopk; ++d) again |= d <= k && s.raw[d <= k ? i - d : i] == e[u];
    const bool ok = e[u] >= 0 && !again;
    invalid |= e[u] == -2 || (e[u] >= 0 && again);
    s.id[i] = (int16_t)(ok ? e[u] : -1);
    if (ok) atomicOr(&s.mask[e[u] >> 5], 1u << (e[u] & 31));
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kRouteRegs; ++u) rt.id[u] = s.id[64 * u + (tid & 63)];
  return invalid;
}

// Position of set bit g (from 0) of v, which has more than g.
__device__ __forceinline__ int select_bit(uint32_t v, int g) {
  int pos = 0;
#pragma unroll
  for (int h = 16; h > 0; h >>= 1) {
    const int c = __popc(v & ((1u << h) - 1));
    if (g >= c) {
      g -= c;
      v >>= h;
      pos += h;
    }
  }
  return pos;
}

// Expert of group g (ascending; g uniform in the workgroup), or -1 past the last.
__device__ __forceinline__ int group_expert(const Fc1Shared& s, int g) {
  uint32_t m[8], v = 0;
  int word = -1;
#pragma unroll
  for (int w = 0; w < 8; ++w) m[w] = __builtin_amdgcn_readfirstlane(s.mask[w]);
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    const int c = __popc(m[w]);
    if (word < 0) {
      if (g < c) {
        word = w;
        v = m[w];
      } else {
        g -= c;
      }
    }
  }
  return word < 0 ? -1 : 32 * word + select_bit(v, g);
}

// Calls f(u, position) for the routes (64 u + lane) of expert e in order, one lane each;
// returns their number.  One wave.
template <class F>
__device__ __forceinline__ int each_route(const Routes& rt, int n, int e, F&& f) {
  const int lane = threadIdx.x & 63;
  int pos = 0;
#pragma unroll
  for (int u = 0; u < kRouteRegs; ++u) {
    if (64 * u < n) {
      const bool hit = rt.id[u] == e;
      const uint64_t m = __ballot(hit);
      if (hit) f(u, pos + __popcll(m & ((1ull << lane) - 1)));
      pos += __popcll(m);
    }
  }
  return pos;
}

// The same for a table of at most kSmallTable entries, by one wave in registers: the expert of
// group g (here in the order of first appearance: any fixed order serves, as long as every
// workgroup takes the same), its routes to s.list and their number to count.
constexpr int kSmallTable = 32;
__device__ __forceinline__ int small_group(const Args& a, Fc1Shared& s, int g, int& count) {
  const int lane = threadIdx.x & 63, n = a.T * a.K;
  int e = lane < n ? a.top[lane] : -1;
  if (e < 0 || e >= a.E) e = -1;
  const int row0 = lane - lane % a.K;
  bool first = e >= 0, again = false;   // first of its expert; listed again in its row
  for (int j = 0; j < n; ++j) {
    const bool same = j < lane && __builtin_amdgcn_readlane(e, j) == e;
    first &= !same;
    again |= same && j >= row0;
  }
  uint64_t m = __ballot(first);
  if (g >= __popcll(m)) return -1;
  for (; g > 0; --g) m &= m - 1;
  e = __builtin_amdgcn_readlane(e, __ffsll((unsigned long long)m) - 1) == e && !again ? e : -1;
  m = __ballot(e >= 0);
  if (e >= 0) s.list[__popcll(m & ((1ull << lane) - 1))] = (int16_t)lane;
  count = __popcll(m);
  return __builtin_amdgcn_readlane(e, __ffsll((unsigned long long)m) - 1);
}

// The first workgroup leaves the plan for the second kernel, a stable counting sort: each
// wave ranks the routes of its chunks of 64 among the chunk's routes to the same expert
// (eight ballots, one a bit of the expert's number), thread e turns the chunks' counts of expert e
// and those of the experts before it into places, and every route goes to its place.
struct PlanShared {
  int place[kRouteRegs][256];      // of each chunk and expert: the count, then the first place
  int wave[4], invalid;
};
template <int NT>
__device__ __forceinline__ void write_plan(const Args& a, const Fc1Shared& s, bool bad, PlanShared& p) {
  static_assert(NT == 256, "one thread an expert");
  constexpr int C = kRouteRegs / 4;              // chunks of a wave
  const int tid = threadIdx.x, n = a.T * a.K, lane = tid & 63, wave = tid >> 6;
  int id[C], rank[C];
  float w[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = 64 * (wave + 4 * c) + lane;
    id[c] = s.id[i];                             // -1 past the table's end
    w[c] = i < n ? a.rw[i] : 0.0f;
  }
#pragma unroll
  for (int c = 0; c < kRouteRegs; ++c) p.place[c][tid] = 0;
  if (tid == 0) p.invalid = 0;
  for (int i = tid; i < a.tiles2; i += NT) a.arrived[i] = 0;
  __syncthreads();
#pragma unroll
  for (int c = 0; c < C; ++c) {
    uint64_t same = ~0ull;
#pragma unroll
    for (int bit = 0; bit < 8; ++bit) {
      const bool one = (id[c] >> bit) & 1;
      const uint64_t m = __ballot(one);
      same &= one ? m : ~m;
    }
    same &= __ballot(id[c] >= 0);                // -1 has the bits of expert 255, which does not exist
    rank[c] = __popcll(same & ((1ull << lane) - 1));
    if (id[c] >= 0 && rank[c] == 0) p.place[wave + 4 * c][id[c]] = __popcll(same);
  }
  if (bad) p.invalid = 1;
  __syncthreads();
  int count = 0, in_chunk[kRouteRegs];
#pragma unroll
  for (int c = 0; c < kRouteRegs; ++c) {
    in_chunk[c] = p.place[c][tid];
    count += in_chunk[c];
  }
  int before = count;                            // inclusive over the wave, then exclusive over all
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int v = __shfl_up(before, o);
    before += lane >= o ? v : 0;
  }
  if (lane == 63) p.wave[wave] = before;
  __syncthreads();
  before -= count;
  int group = 0, groups = 0, routes = 0;
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    if (v < wave) before += p.wave[v];
    routes += p.wave[v];
  }
#pragma unroll
  for (int v = 0; v < 8; ++v) {
    const uint32_t m = s.mask[v];
    groups += __popc(m);
    group += v < (tid >> 5) ? __popc(m) : (v == (tid >> 5) ? __popc(m & ((1u << (tid & 31)) - 1)) : 0);
  }
  if (tid == 0) {
    a.plan->status = p.invalid ? kRouteInvalid : 0;
    a.plan->groups = groups;
    a.plan->first[groups] = routes;
  }
  if (count > 0) {
    a.plan->expert[group] = tid;
    a.plan->first[group] = before;
  }
#pragma unroll
  for (int c = 0; c < kRouteRegs; ++c) {
    p.place[c][tid] = before;
    before += in_chunk[c];
  }
  __syncthreads();
#pragma unroll
  for (int c = 0; c < C; ++c) {
    if (id[c] >= 0) {
      const int to = p.place[wave + 4 * c][id[c]] + rank[c];
      a.plan->route[to] = 64 * (wave + 4 * c) + lane;
      a.plan->weight[to] = w[c];
    }
  }
}

// Token columns c0 .. c0 + 16 NF - 1 (of `count`) of the tile at i0 (COLS: of wave w's, w tiles
// on).  `cells`: 16-byte cells of lds a wave has.
template <bool MX, int R, int W, int NF, int D, bool COLS>
__device__ __forceinline__ void fc1_tile(const Args& a, const Fc1Shared& s, uint4* lds, int cells, int e, int i0,
                                         int c0, int count) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane >> 2, c4 = 16 * (lane & 3);   // the row and byte this lane loads
  const int steps = a.H / kStep;
  const int s0 = COLS ? 0 : wave * steps / W, s1 = COLS ? steps : (wave + 1) * steps / W;
  if (COLS) i0 += wave * 8 * R;
  const uint8_t *w[R], *ws[R];
#pragma unroll
  for (int g = 0; g < R; ++g) {
    const int row = i0 + 8 * g + (r >> 1);
    ws[g] = nullptr;
    if (e < 0) {
      w[g] = (r & 1 ? a.sup : a.sgate).row(0, row);
    } else {
      const MxRef& m = r & 1 ? a.up : a.gate;
      w[g] = m.data.row(e, row);
      if constexpr (MX) ws[g] = m.scale.row(e, row) + s0 * 4;
    }
    w[g] += (int64_t)s0 * WStep<MX>::kBytes + c4;
  }
  const uint8_t* x[NF];
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    const int c = c0 + 16 * f + r < count ? c0 + 16 * f + r : c0;   // columns past the last repeat one
    const int t = e < 0 ? c : s.list[c] / a.K;
    x[f] = reinterpret_cast<const uint8_t*>(a.x + (int64_t)t * a.H) + (int64_t)s0 * XStep<kXPitch>::kBytes + c4;
  }
  f32x4_t acc[R][NF];
#pragma unroll
  for (int g = 0; g < R; ++g)
#pragma unroll
    for (int f = 0; f < NF; ++f) acc[g][f] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  const Turn turn = turn_of(lds + wave * cells);
  dot_steps<MX, R, NF, D, kXPitch>(turn, w, ws, x, s1 - s0, acc);
  // [wave][column][row]: a lane has rows 4 q .. 4 q + 3 of column r.  Over the turn-round slots
  float* red = reinterpret_cast<float*>(lds);
  if constexpr (COLS) {
    red += (wave * cells - wave * NF * R * 64) * 4;   // the wave's own slots
    wave_lds_fence();
  } else {
    __syncthreads();
  }
#pragma unroll
  for (int g = 0; g < R; ++g)
#pragma unroll
    for (int f = 0; f < NF; ++f)
      *reinterpret_cast<f32x4_t*>(red + ((wave * NF + f) * 16 + turn.row) * (16 * R) + 16 * g + 4 * turn.q) = acc[g][f];
  if constexpr (COLS) wave_lds_fence();
  else __syncthreads();
  const int cols = min(16 * NF, count - c0);
  for (int o = COLS ? lane : threadIdx.x; o < 8 * R * cols; o += COLS ? 64 : 64 * W) {
    const int c = o / (8 * R), p = o % (8 * R);
    float g = 0.0f, u = 0.0f;
#pragma unroll
    for (int v = COLS ? wave : 0; v < (COLS ? wave + 1 : W); ++v) {
      const float2 z = *reinterpret_cast<const float2*>(red + (v * NF * 16 + c) * (16 * R) + 2 * p);
      g += z.x;
      u += z.y;
    }
    const int64_t hrow = e < 0 ? (int64_t)a.T * a.K + c0 + c : s.list[c0 + c];
    const float h = swiglu(g, u, a.limit), hi = bf2f(f2bf(h));
    uint16_t* to = a.h + h_index(hrow, i0 + p, a.I);
    to[0] = (uint16_t)f2bf(h);
    to[kHLower] = (uint16_t)f2bf(fabsf(hi) < __builtin_huge_valf() ? h - hi : 0.0f);
  }
}

// More than 16 tokens: without MANY in passes of 32 over one fragment's weights, which the
// caches then hold; with MANY (two waves a SIMD, so twice the registers) all at once.
template <bool MX, int R, int W, int D, bool MANY, bool COLS>
__device__ __forceinline__ void fc1_group(const Args& a, const Fc1Shared& s, uint4* lds, int cells, int e, int i0,
                                          int count) {
  if (count <= 16) {
    fc1_tile<MX, R, W, 1, D, COLS>(a, s, lds, cells, e, i0, 0, count);
  } else if constexpr (MANY) {
    if (count <= 32) fc1_tile<MX, R, W, 2, 1, COLS>(a, s, lds, cells, e, i0, 0, count);
    else fc1_tile<MX, R, W, 4, 1, COLS>(a, s, lds, cells, e, i0, 0, count);
  } else {
    for (int g = 0; g < R; ++g)
      for (int c0 = 0; c0 < count; c0 += 32) {
        if (!COLS && g + c0) __syncthreads();
        if (COLS) wave_lds_fence();
        fc1_tile<MX, 1, W, 2, 1, COLS>(a, s, lds, cells, e, i0 + (COLS ? 8 * W : 8) * g, c0, count);
      }
  }
}

// Row fragments a workgroup of the shared expert takes: BF16 needs twice the registers.
template <bool MX, int R, bool MANY>
constexpr int shared_frags() { return MX && !MANY ? 1 : R; }

template <bool MX, int R, int W, int D, bool MANY, bool COLS>
__global__ __launch_bounds__(64 * W, MANY ? 2 : 4) void k_decode_fc1(Args a) {
  __shared__ Fc1Shared s;
  // turn-round slots, then the partial sums of up to four column groups
  constexpr int kSums = (MANY ? 4 : 2) * R * 64;
  constexpr int kCells = wave_cells<MX, R>() > kSums ? wave_cells<MX, R>() : kSums;
  __shared__ __align__(16) uint4 lds[W * kCells];
  constexpr int T = COLS ? W : 1;                          // column tiles of a workgroup
  const int tiles = a.I / (8 * R * T);                     // workgroups an expert
  constexpr int RS = shared_frags<MX, R, MANY>();
  const int shared_blocks = a.shared ? a.I / (8 * RS * T) : 0;
  const int routed_blocks = min(a.E, a.T * a.K) * tiles;
  if (blockIdx.x == 0) {
    Routes rt;
    const bool bad = read_table<64 * W>(a, s, rt);
    static_assert(sizeof(PlanShared) <= sizeof(lds), "the plan's scratch");
    write_plan<64 * W>(a, s, bad, *reinterpret_cast<PlanShared*>(lds));
    return;
  }
  int b = blockIdx.x - 1;
  if (b >= shared_blocks + routed_blocks) {   // shared output gate: one wave a token
    const int t = (b - shared_blocks - routed_blocks) * W + (threadIdx.x >> 6), lane = threadIdx.x & 63;
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
    fc1_group<false, RS, W, 2, MANY, COLS>(a, s, lds, kCells, -1, b * 8 * RS * T, a.T);
    return;
  }
  b -= shared_blocks;
  int e, count;   // every wave lists the routes for itself, to the same place with the same values
  if (a.T * a.K <= kSmallTable) {
    e = small_group(a, s, b / tiles, count);
    if (e < 0) return;
  } else {
    Routes rt;
    read_table<64 * W>(a, s, rt);
    e = __builtin_amdgcn_readfirstlane(group_expert(s, b / tiles));
    if (e < 0) return;
    count = each_route(rt, a.T * a.K, e, [&](int u, int p) { s.list[p] = (int16_t)(64 * u + (threadIdx.x & 63)); });
  }
  __builtin_amdgcn_wave_barrier();
  fc1_group<MX, R, W, D, MANY, COLS>(a, s, lds, kCells, e, b % tiles * 8 * R * T, count);
}

// ---------------------------------------------------------------- FC2 + combine
// A workgroup owns 16 R output columns of every token.  Its W waves split the steps of all
// experts in use evenly; each adds w_tk times what it has of an expert's product to an
// accumulator [token][16 R] of its own in LDS, and the waves' accumulators are joined in
// order at the end.  Where H is too short to give every CU a workgroup, `split` workgroups
// share the columns: each leaves its sums in the workspace, and the last one to arrive adds
// them up in order.
struct Fc2Shared {
  int32_t expert[kMaxExperts + 1], first[kMaxExperts + 2];
  int16_t route[kMaxRoutes];
  float weight[kMaxRoutes];
};

// Tokens c0 .. c0 + 8 NF - 1 of one expert (e < 0: the shared one), steps s0 .. s0 + n - 1; row
// fragments g0 .. g0 + R - 1 of the workgroup's RT.  A column fragment is 8 tokens: columns 0 .. 7 are
// the upper parts of their h, 8 .. 15 the lower ones, and their sums are added at the end.
template <bool MX, int R, int RT, int NF, int D>
__device__ __forceinline__ void fc2_part(const Args& a, const Fc2Shared& s, const Turn& turn, float* acc_lds, int g0,
                                         int e, int first, int c0, int count, int s0, int n) {
  const int lane = threadIdx.x & 63, r = lane >> 2, c4 = 16 * (lane & 3);   // the row and byte this lane loads
  const uint8_t *w[R], *ws[R];
#pragma unroll
  for (int g = 0; g < R; ++g) {
    const int row = ((int)blockIdx.x * RT + g0 + g) * 16 + r;
    ws[g] = nullptr;
    if (e < 0) {
      w[g] = a.sdown.row(0, row);
    } else {
      w[g] = a.down.data.row(e, row);
      if constexpr (MX) ws[g] = a.down.scale.row(e, row) + s0 * 4;
    }
    w[g] += (int64_t)s0 * WStep<MX>::kBytes + c4;
  }
  const uint8_t* x[NF];
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    const int c = c0 + 8 * f + (r & 7) < count ? c0 + 8 * f + (r & 7) : c0;
    const int64_t hrow = e < 0 ? (int64_t)a.T * a.K + c : s.route[first + c];
    x[f] = reinterpret_cast<const uint8_t*>(a.h + h_index(hrow, 0, a.I) + (r >> 3) * kHLower) +
           (int64_t)s0 * XStep<kHPitch>::kBytes + c4;
  }
  f32x4_t acc[R][NF];
#pragma unroll
  for (int g = 0; g < R; ++g)
#pragma unroll
    for (int f = 0; f < NF; ++f) acc[g][f] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  dot_steps<MX, R, NF, D, kHPitch>(turn, w, ws, x, n, acc);
#pragma unroll
  for (int g = 0; g < R; ++g)
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[g][f][i] += dpp_f<kDppRor8>(acc[g][f][i]);
#pragma unroll
  for (int f = 0; f < NF; ++f) {
    const int c = c0 + 8 * f + turn.row;
    if (c >= count || turn.row >= 8) continue;
    const int tok = e < 0 ? c : s.route[first + c] / a.K;
    const float wt = e < 0 ? (a.gw ? a.gate_s[c] : 1.0f) : s.weight[first + c];
#pragma unroll
    for (int g = 0; g < R; ++g) {
      f32x4_t* o = reinterpret_cast<f32x4_t*>(acc_lds + (tok * RT + g0 + g) * 16 + 4 * turn.q);   // the wave's own
      f32x4_t v = *o;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += wt * acc[g][f][i];
      *o = v;
    }
  }
}

// All RT fragments of the workgroup together (R at a time up to 8 tokens: the shared expert's
// BF16 rows take more registers than E4M3's).  More than 32 tokens go in passes over the weights,
// which the caches then hold.  MANY: a batch of more than 16 tokens, or short rows.  (Two column
// fragments with two steps in flight: 183 us against 189 with 12 of 64 tokens for each of 32 E4M3
// experts of H 7168.)
template <bool MX, int R, int RT, int D, bool MANY>
__device__ __forceinline__ void fc2_group(const Args& a, const Fc2Shared& s, const Turn& turn, float* acc_lds, int e,
                                          int first, int count, int s0, int n) {
  if (count <= 8) {
    for (int g = 0; g < RT; g += R) fc2_part<MX, R, RT, 1, D>(a, s, turn, acc_lds, g, e, first, 0, count, s0, n);
  } else if (!MANY || count <= 16) {
    fc2_part<MX, RT, RT, 2, MANY ? D : 1>(a, s, turn, acc_lds, 0, e, first, 0, count, s0, n);
  } else {
    for (int c0 = 0; c0 < count; c0 += 32)
      fc2_part<MX, RT, RT, 4, 1>(a, s, turn, acc_lds, 0, e, first, c0, count, s0, n);
  }
}

template <bool MX, int R, bool MANY>
__global__ __launch_bounds__(64 * kFc2Waves, 2) void k_decode_fc2(Args a) {
  constexpr int W = kFc2Waves, D = 2;
  extern __shared__ __align__(16) float acc_all[];   // [W][T][16 R]
  __shared__ Fc2Shared s;
  __shared__ __align__(16) uint4 slots[W * wave_cells<MX, R>()];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // the plan's whole arrays, past their ends too: no load waits for another, and none is
  // waited for before the shared expert is done
  const int routed = a.plan->groups;
  int plan_e = 0, plan_f = 0, plan_r = 0;
  float plan_w = 0.0f;
  if (tid <= kMaxExperts) plan_e = a.plan->expert[tid];
  if (tid < kMaxExperts + 2) plan_f = a.plan->first[tid];
  if (tid < a.T * a.K) {
    plan_r = a.plan->route[tid];
    plan_w = a.plan->weight[tid];
  }
  float* mine = acc_all + wave * a.T * 16 * R;
  for (int i = tid & 63; i < a.T * 4 * R; i += 64) reinterpret_cast<f32x4_t*>(mine)[i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  const Turn turn = turn_of(slots + wave * wave_cells<MX, R>());
  const int steps = a.I / kStep, part = blockIdx.y * W + wave, parts = W * a.split;
  if (a.shared) {   // every wave takes its part: with many tokens these steps cost more than routed ones
    const int s0 = part * steps / parts, s1 = (part + 1) * steps / parts;
    if (s1 > s0) fc2_group<false, 1, R, D, MANY>(a, s, turn, mine, -1, 0, a.T, s0, s1 - s0);
  }
  if (tid <= kMaxExperts) s.expert[tid] = plan_e;
  if (tid < kMaxExperts + 2) s.first[tid] = plan_f;
  if (tid < a.T * a.K) {
    s.route[tid] = (int16_t)plan_r;
    s.weight[tid] = plan_w;
  }
  __syncthreads();
  const int64_t total = (int64_t)routed * steps;
  int64_t p = part * total / parts;
  const int64_t end = (part + 1) * total / parts;
  while (p < end) {   // uniform in the wave
    const int g = (int)(p / steps), s0 = (int)(p % steps);
    const int n = (int)min((int64_t)(steps - s0), end - p);
    const int e = __builtin_amdgcn_readfirstlane(s.expert[g]), first = __builtin_amdgcn_readfirstlane(s.first[g]);
    const int count = __builtin_amdgcn_readfirstlane(s.first[g + 1]) - first;
    fc2_group<MX, R, R, D, MANY>(a, s, turn, mine, e, first, count, s0, n);
    p += n;
  }
  __syncthreads();
  const int outs = a.T * 16 * R;
  auto put = [&](int o, float v) __attribute__((always_inline)) {
    a.out[(int64_t)(o / (16 * R)) * a.H + blockIdx.x * 16 * R + o % (16 * R)] = (uint16_t)f2bf(v);
  };
  float* sums = a.sums + (int64_t)blockIdx.x * a.split * outs;     // [split][T][16 R]
  for (int o = tid; o < outs; o += 64 * W) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) v += acc_all[w * outs + o];
    if (a.split == 1) put(o, v);
    else __hip_atomic_store(sums + (int64_t)blockIdx.y * outs + o, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  if (a.split == 1) return;
  // The sums go through device-scope stores and loads, which the XCDs' caches do not keep to
  // themselves, so all that is needed is that a wave's stores are done before its workgroup is
  // counted.  (Device-scope fences instead would write back a whole L2 in every workgroup: 58 us
  // for a second kernel of 36 tokens at H 512 that takes 17 this way.)
  __shared__ int last;
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (tid == 0) last = __hip_atomic_fetch_add(a.arrived + blockIdx.x, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)
                       == a.split - 1;
  __syncthreads();
  if (!last) return;
  for (int o = tid; o < outs; o += 64 * W) {
    float v = 0.0f;
    for (int y = 0; y < a.split; ++y)
      v += __hip_atomic_load(sums + (int64_t)y * outs + o, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    put(o, v);
  }
}

}  // namespace

// Steps in flight (D) and waves a SIMD fit the register file: four waves leave 128 registers
// each.  Spills and fewer waves cost more than depth gains: one token of BF16 at H 4096
// takes 28.2 us as it is, 30.2 with three steps in flight and 29.1 with eight waves a
// workgroup in the first kernel.
template <bool MX, int R, int D, bool MANY>
void launch_fc1_as(hipStream_t st, const Args& a) {
  constexpr int W = kFc1Waves;
  const int used = a.E < a.T * a.K ? a.E : a.T * a.K;
  // A workgroup's start (reading the table, finding its expert) costs about what 64 KB of
  // weights do, and four waves that split a short contraction have little to add up: up to H
  // 1792 each wave takes columns of its own, as long as that leaves 128 workgroups.  36 tokens over
  // 77 BF16 experts of H 512: 33 us against 41; 64 over 16 E4M3 experts of H 512: 21 against 28;
  // over 64 of H 1664, top-8: 81 against 94.  Longer rows leave too few workgroups to even out (16
  // tokens, 32 BF16 experts of H 2048: 76 against 71), as does a smaller layer (55 tokens, 7 E4M3
  // experts of H 512, I 512: 22 against 20).
  const bool cols = a.H <= 14 * kStep && (int64_t)used * (a.I / (8 * R * W)) >= 128;
  const int T = cols ? W : 1;
  const int tiles = a.I / (8 * R * T);
  const int gate = a.gw ? (a.T + W - 1) / W : 0;
  const int shared = a.shared ? a.I / (8 * shared_frags<MX, R, MANY>() * T) : 0;
  const dim3 grid((unsigned)(1 + shared + used * tiles + gate)), block(64 * W);
  if (cols) hipLaunchKernelGGL((k_decode_fc1<MX, R, W, D, MANY, true>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((k_decode_fc1<MX, R, W, D, MANY, false>), grid, block, 0, st, a);
}
template <bool MX>
void launch_fc1(hipStream_t st, const Args& a) {
  // More than 14 tokens an expert on average (and more than 16 in all): every row fragment
  // takes up to 64 tokens at once, on two waves a SIMD.  64 tokens over 6 BF16 experts of H 4096:
  // 38 us against 54; over 32 experts top-6 (12 each), E4M3: 89 against 80.
  // Otherwise two fragments a workgroup share the tokens' loads with E4M3, where they weigh
  // twice as much as beside BF16: 371 us against 424 (64 tokens, H 7168, E4M3); BF16 loses a
  // little to the coarser grid (151 us against 139, 19 tokens, H 4096).
  if (a.T > 16 && a.T * a.K > 14 * a.E) launch_fc1_as<MX, 2, 1, true>(st, a);
  else launch_fc1_as<MX, MX ? 2 : 1, MX ? 1 : 2, false>(st, a);
}
template <bool MX, int R, bool MANY>
void launch_fc2_as(hipStream_t st, const Args& a) {
  constexpr int W = kFc2Waves;
  static_assert(64 * W >= kMaxRoutes && 64 * W >= kMaxExperts + 2, "the plan in one load a thread");
  hipLaunchKernelGGL((k_decode_fc2<MX, R, MANY>), dim3(a.tiles2, a.split), dim3(64 * W),
                     (size_t)W * a.T * 16 * R * sizeof(float), st, a);
}
template <bool MX>
void launch_fc2(hipStream_t st, const Args& a) {
  // Two fragments for up to 16 tokens leave out what only more need: 146 us against 152 (16 tokens over
  // 32 E4M3 experts of H 5120), 252 against 259 (BF16).  With one fragment that gains nothing.
  if (fc2_shape(a.T, a.H, a.I, a.E, a.K).frags == 1) launch_fc2_as<MX, 1, true>(st, a);
  else if (a.T > 16) launch_fc2_as<MX, 2, true>(st, a);
  else launch_fc2_as<MX, 2, false>(st, a);
}
template void launch_fc1<false>(hipStream_t, const Args&);
template void launch_fc1<true>(hipStream_t, const Args&);
template void launch_fc2<false>(hipStream_t, const Args&);
template void launch_fc2<true>(hipStream_t, const Args&);

}  // namespace decode
}  // namespace moe

// The router's decision: scores from logits, the K best experts of every token, their
// weights, and the gradient back to the logits (C ABI: moe_router_forward / _backward).
//
//   s = softmax(l) over the row, or sigmoid(l) per expert
//   chosen: the K largest of s (+ bias), ties to the lowest expert index
//   w_k = scale s_k / (sum of the chosen s + 1e-20)   or   scale s_k
//
// A row is held by 16 lanes (one DPP row), element e = lane + 16 j in register j, so that
// the K rounds of "largest remaining" are a scan over a few registers and four DPP steps
// each, with no LDS and no barrier, for four rows of a wave at once.
//
// Without a bias the order of the scores is the order of the logits, so the logits
// themselves are compared: no rounding can make or break a tie.  With a bias s + bias is
// compared as in 64 bits: in 32 bits scores near 1 differ by rounding alone and two correct
// programs would choose different experts.  (FP32 keys decide wherever they are far enough
// apart to be sure; FP64 everywhere took 11 us more at 65536 x 64, top-6.)
//
// 65536 x 64 sigmoid scores with a bias, top-6: 12.3 us (4.0 us for its bytes at the rate of a
// large copy); the backward of 65536 x 97 BF16 logits, top-8: 10.3 us (6.0 us).  Bound by vector
// instructions: at 4 clocks a wave, the forward's are most of its time.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "../../include/moe.h"
#include "common.hpp"
#include "host.hpp"
#include "reduce.hpp"

using namespace moe;

namespace {

constexpr int kRouterThreads = 256;
constexpr int kRouterRows = kRouterThreads / 16;   // token rows per workgroup
constexpr float kRouterEps = 1e-20f;

struct RouterArgs {
  const void* logits;
  int64_t ld;
  int64_t tokens;
  int E, K, normalize;
  float scale;
  const float* bias;
  int32_t* top;          // forward: written; backward: read
  float* rw;             // forward: written
  const float* gw;       // backward
  void* dl;              // backward
  int64_t ld_dl;
};

template <bool BF16>
__device__ __forceinline__ float ld_logit(const void* base, int64_t i) {
  if constexpr (BF16) return bf2f(static_cast<const uint16_t*>(base)[i]);
  else return static_cast<const float*>(base)[i];
}

__device__ __forceinline__ float ninf() { return -__builtin_huge_valf(); }

// exp(x) = 2^p (1 + r ln 2), p = x log2(e) rounded and r what that left of it: off by 5 u (u =
// 2^-24; the hardware's 2^p 2 u), a third of the instructions of the library's, which also keeps
// results below 2^-126.  NaN passes; below -150 the result is 0 either way.
__device__ __forceinline__ float exp_(float x) {
  x = x < -150.0f ? -150.0f : x;
  const float p = x * 1.44269504f;
  const float r = fmaf(x, 1.44269504f, -p) + x * 1.92596300e-8f;   // log2(e) in two floats
  const float e = __builtin_amdgcn_exp2f(p);
  return fmaf(e, r * 0.693147181f, e);
}
__device__ __forceinline__ float sigmoid_(float x) {   // 0 where it would not be a normal number; NaN passes
  const float s = __builtin_amdgcn_rcpf(1.0f + exp_(-x));
  return x < -87.0f ? 0.0f : s;
}

// EPL registers of a row: logits (-inf past the last expert).  Every lane loads, past the
// end the last expert's: without branches all loads are under way together.
template <int EPL, bool BF16>
__device__ __forceinline__ void load_row(const RouterArgs& a, int64_t t, int lane, float (&l)[EPL]) {
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = lane + 16 * j;
    const float v = ld_logit<BF16>(a.logits, t * a.ld + min(e, a.E - 1));
    l[j] = e < a.E ? v : ninf();
  }
}

// Row scores in T (float or double).  -inf logits have score 0; a row with nothing else
// keeps zeros (no 0/0).  A NaN logit leaves softmax's whole row NaN.
template <int EPL, bool SOFTMAX, typename T>
__device__ __forceinline__ void row_scores(const float (&l)[EPL], T (&s)[EPL]) {
  if constexpr (SOFTMAX) {
    float m = ninf();
#pragma unroll
    for (int j = 0; j < EPL; ++j) m = fmaxf(m, l[j]);   // ignores NaN
    m = row16_max(m);
    T z = 0;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      if constexpr (std::is_same<T, double>::value) s[j] = l[j] == ninf() ? 0.0 : exp((double)l[j] - (double)m);
      else s[j] = l[j] == ninf() ? 0.0f : exp_(l[j] - m);
      z += s[j];
    }
    z = row16_sum(z);
    const T inv = z == (T)0 ? (T)0 : (T)1 / z;
#pragma unroll
    for (int j = 0; j < EPL; ++j) s[j] *= inv;
  } else {
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      if constexpr (std::is_same<T, double>::value) s[j] = 1.0 / (1.0 + exp(-(double)l[j]));
      else s[j] = sigmoid_(l[j]);
    }
  }
}

// Keys as integers in the same order (-0 becomes +0 first): integer maxima need no
// canonical forms and fold into the DPP instruction.  kNoKey lies below every float's.
constexpr int kNoKey = INT32_MIN;
__device__ __forceinline__ int order_key(float v) {
  const int b = __float_as_int(v + 0.0f);
  return b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float key_value(int k) { return __int_as_float(k ^ ((k >> 31) & 0x7fffffff)); }

// A chosen expert and its score.
struct Entry {
  int e;
  float s;
};

// One round: the largest key left in the row (to `best`); the lane that holds it, for the
// lowest expert if several do, strikes it out and leaves its expert and score in `to` (if
// `write`).  Nothing happens when only `lowest` is left.
template <int EPL, typename T>
__device__ __forceinline__ void take_best(T (&key)[EPL], const float (&s)[EPL], int lane, int rows, T lowest, T& best,
                                          Entry* to, bool write) {
  T m = key[0];
#pragma unroll
  for (int j = 1; j < EPL; ++j) m = key[j] > m ? key[j] : m;
  m = row16_max(m);
  best = m;
  int e = 1 << 20, hits = 0;
  float v = 0.0f;
#pragma unroll
  for (int j = EPL - 1; j >= 0; --j) {
    const bool hit = key[j] == m;
    hits += __popcll(__ballot(hit));
    e = hit ? lane + 16 * j : e;
    v = hit ? s[j] : v;
  }
  if (hits == rows) {   // one in each of the wave's rows: it is known where it is found
    bool own = false;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      const bool hit = key[j] == m;
      own |= hit;
      key[j] = hit ? lowest : key[j];
    }
    if (own && write) *to = Entry{e, v};
  } else {              // the rows agree on the lowest expert
    const bool own = e == row16_min(e) && e < (1 << 20) && m != lowest;
#pragma unroll
    for (int j = 0; j < EPL; ++j) key[j] = own && lane + 16 * j == e ? lowest : key[j];
    if (own && write) *to = Entry{e, v};
  }
}

template <int EPL, bool BF16, bool SOFTMAX, bool BIAS>
__global__ __launch_bounds__(kRouterThreads) void k_router_fwd(RouterArgs a) {
  __shared__ Entry chosen[kRouterRows][kMaxTopk];
  const int lane = threadIdx.x & 15;
  const int64_t t = (int64_t)blockIdx.x * kRouterRows + (threadIdx.x >> 4);
  if (t >= a.tokens) return;   // whole 16-lane rows leave together
  float l[EPL], s[EPL];
  [[maybe_unused]] float bias[EPL];
  load_row<EPL, BF16>(a, t, lane, l);
  if constexpr (BIAS) {
#pragma unroll
    for (int j = 0; j < EPL; ++j) bias[j] = a.bias[min(lane + 16 * j, a.E - 1)];
  }
  int bad = 0;
#pragma unroll
  for (int j = 0; j < EPL; ++j) bad = l[j] != l[j] ? 1 : bad;
  bad = row16_max(bad);
  row_scores<EPL, SOFTMAX, float>(l, s);

  Entry* mine = chosen[threadIdx.x >> 4];
  if (lane < kMaxTopk) mine[lane] = Entry{-1, 0.0f};
  wave_lds_fence();
  const int rows = __popcll(__ballot(true)) >> 4;
  int key[EPL], best[kMaxTopk];
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = lane + 16 * j;
    const float v = BIAS ? s[j] + bias[j] : l[j];
    // an expert whose logit is -inf or NaN, or whose key is -inf or NaN, is never chosen
    key[j] = l[j] > ninf() && v > ninf() ? order_key(v) : kNoKey;
  }
#pragma unroll
  for (int k = 0; k < kMaxTopk; ++k)
    if (k < a.K) take_best<EPL, int>(key, s, lane, rows, kNoKey, best[k], mine + k, true);
  if constexpr (BIAS) {
    // FP32 keys are off by at most 32 u of a softmax score (u = 2^-24: the rounding of l - m
    // times x exp(-x) <= 0.37, the function, the row sum and the division), 8 u of a sigmoid,
    // and u of the key.  Where the keys down to the first one left out are further apart
    // than twice that, FP64 keys have the same order; other rows are decided again in FP64, with
    // the rest of their wave.  Of normally distributed logits that is one row in 1000 to 3000 with
    // sigmoid scores; softmax scores of many experts lie closer: 0.25% of the rows and 1% of the waves
    // at 64 experts, 0.9% and 3.6% at 255.
    int next = key[0];
#pragma unroll
    for (int j = 1; j < EPL; ++j) next = max(next, key[j]);
    // the smallest gap and the largest magnitude; kNoKey is a NaN here, which fminf and fmaxf ignore
    float low = key_value(row16_max(next)), gap = __builtin_huge_valf(), most = fabsf(low);
#pragma unroll
    for (int k = kMaxTopk - 1; k >= 0; --k) {
      if (k < a.K) {
        const float hi = key_value(best[k]);
        gap = fminf(gap, hi - low);
        most = fmaxf(most, fabsf(hi));
        low = hi;
      }
    }
    // (no gap at all: nothing to confuse.  !(>) holds for infinite magnitudes too)
    const bool close = gap < __builtin_huge_valf() && !(gap > (SOFTMAX ? 0x1p-18f : 0x1p-20f) + 0x1p-22f * most);
    if (__any(close)) {
      double dkey[EPL], db;
      const double lowest = -__builtin_huge_val();
      row_scores<EPL, SOFTMAX, double>(l, dkey);
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        const int e = lane + 16 * j;
        dkey[j] = e < a.E ? dkey[j] + (double)bias[j] : lowest;
        if (!(l[j] > ninf()) || dkey[j] != dkey[j]) dkey[j] = lowest;
      }
#pragma unroll
      for (int k = 0; k < kMaxTopk; ++k) {
        if (k < a.K) {
          if (close && lane == 0) mine[k] = Entry{-1, 0.0f};
          wave_lds_fence();
          take_best<EPL, double>(dkey, s, lane, rows, lowest, db, mine + k, close);
        }
      }
    }
  }

  wave_lds_fence();
  const Entry entry = lane < a.K ? mine[lane] : Entry{-1, 0.0f};   // lane k writes entry k
  const int e = entry.e;
  const float w = entry.s;
  const float sum = row16_sum(w);
  const float f = a.normalize ? a.scale / (sum + kRouterEps) : a.scale;
  if (lane < a.K) {
    a.top[t * a.K + lane] = e;
    a.rw[t * a.K + lane] = e < 0 ? 0.0f : (bad ? __builtin_nanf("") : w * f);
  }
}

// Gradient of sum_k gw_k w_k.  With cnt_e the times e stands in the table's row (0 or 1
// for a table of the forward), g_e the sum of its gw, S and G the row sums of cnt s, g s:
//   ds_e = scale g_e                                    (raw scores)
//   ds_e = scale (g_e - cnt_e G / (S + eps)) / (S + eps)  (normalised)
//   softmax: dl_e = s_e (ds_e - sum_j ds_j s_j)     sigmoid: dl_e = ds_e s_e (1 - s_e)
template <int EPL, bool BF16, bool SOFTMAX>
__global__ __launch_bounds__(kRouterThreads) void k_router_bwd(RouterArgs a) {
  __shared__ int tags[kRouterRows * 16 * EPL];
  __shared__ float grads[kRouterRows * 16 * EPL];
  const int lane = threadIdx.x & 15;
  const int64_t t = (int64_t)blockIdx.x * kRouterRows + (threadIdx.x >> 4);
  if (t >= a.tokens) return;
  float l[EPL], s[EPL], g[EPL], cnt[EPL];
  load_row<EPL, BF16>(a, t, lane, l);
  // Lane k holds the row's entry k.  Its position (1 + k) and gradient go to the expert's
  // place in LDS; the lanes then read their experts' places.  A lane that does not find its own
  // position again shares its expert with another entry: such rows add entry by entry.
  int me = lane < a.K ? a.top[t * a.K + lane] : -1;
  const float mg = lane < a.K ? a.gw[t * a.K + lane] : 0.0f;
  if (me >= a.E || me < 0) me = -1;   // skipped
  int* tag = tags + (threadIdx.x >> 4) * (16 * EPL);
  float* grad = grads + (threadIdx.x >> 4) * (16 * EPL);
#pragma unroll
  for (int j = 0; j < EPL; ++j) tag[lane + 16 * j] = 0;
  wave_lds_fence();
  if (me >= 0) {
    tag[me] = lane + 1;
    grad[me] = mg;
  }
  wave_lds_fence();
  const bool twice = me >= 0 && tag[me] != lane + 1;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const bool hit = tag[lane + 16 * j] != 0;
    g[j] = hit ? grad[lane + 16 * j] : 0.0f;
    cnt[j] = hit ? 1.0f : 0.0f;
  }
  if (__any(twice)) {
#pragma unroll
    for (int j = 0; j < EPL; ++j) g[j] = cnt[j] = 0.0f;
    for (int k = 0; k < a.K; ++k) {
      const int e = __shfl(me, k, 16);
      const float v = __shfl(mg, k, 16);
#pragma unroll
      for (int j = 0; j < EPL; ++j) {
        const bool hit = lane + 16 * j == e;
        g[j] += hit ? v : 0.0f;
        cnt[j] += hit ? 1.0f : 0.0f;
      }
    }
  }
  row_scores<EPL, SOFTMAX, float>(l, s);
  if (a.normalize) {
    float S = 0.0f, G = 0.0f;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      S += cnt[j] * s[j];
      G += g[j] * s[j];
    }
    S = row16_sum(S) + kRouterEps;
    G = row16_sum(G) / S;
    const float f = a.scale / S;
#pragma unroll
    for (int j = 0; j < EPL; ++j) g[j] = f * (g[j] - cnt[j] * G);
  } else {
#pragma unroll
    for (int j = 0; j < EPL; ++j) g[j] *= a.scale;
  }
  float dot = 0.0f;
  if constexpr (SOFTMAX) {
#pragma unroll
    for (int j = 0; j < EPL; ++j) dot += g[j] * s[j];
    dot = row16_sum(dot);
  }
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = lane + 16 * j;
    if (e < a.E) {
      // 1 - sigmoid(l) as sigmoid(-l): the difference would cancel near 1
      const float d = SOFTMAX ? s[j] * (g[j] - dot) : g[j] * s[j] * sigmoid_(-l[j]);
      if constexpr (BF16) static_cast<uint16_t*>(a.dl)[t * a.ld_dl + e] = (uint16_t)f2bf(d);
      else static_cast<float*>(a.dl)[t * a.ld_dl + e] = d;
    }
  }
}

moe_status check_router(const moe_router_problem* p) {
  if (!p) return MOE_ERR_NULL;
  if (p->tokens < 0 || p->tokens > ((int64_t)1 << 27)) return MOE_ERR_SHAPE;   // a launch holds 2^32 threads, 16 a row
  if (p->experts < 1 || p->experts > kMaxExperts) return MOE_ERR_SHAPE;
  if (p->topk < 1 || p->topk > kMaxTopk || p->topk > p->experts) return MOE_ERR_SHAPE;
  if (p->logits_dtype != MOE_BF16 && p->logits_dtype != MOE_FP32) return MOE_ERR_DTYPE;
  if (p->score != MOE_ROUTER_SOFTMAX && p->score != MOE_ROUTER_SIGMOID) return MOE_ERR_UNSUPPORTED;
  if (p->flags & ~MOE_ROUTER_NORMALIZE) return MOE_ERR_UNSUPPORTED;
  if (!(p->scale > -3.0e38f && p->scale < 3.0e38f)) return MOE_ERR_UNSUPPORTED;   // NaN, infinite
  if (p->ld_logits < p->experts) return MOE_ERR_LAYOUT;
  return MOE_OK;
}

RouterArgs router_args(const moe_router_problem* p, const void* logits) {
  RouterArgs a{};
  a.logits = logits;
  a.ld = p->ld_logits;
  a.tokens = p->tokens;
  a.E = p->experts; a.K = p->topk;
  a.normalize = (p->flags & MOE_ROUTER_NORMALIZE) != 0;
  a.scale = p->scale;
  return a;
}

// Calls f with the number of registers a row takes per lane, for up to 255 experts.
template <class F>
void with_epl(int E, F&& f) {
  if (E <= 32) f(std::integral_constant<int, 2>{});
  else if (E <= 64) f(std::integral_constant<int, 4>{});
  else if (E <= 128) f(std::integral_constant<int, 8>{});
  else f(std::integral_constant<int, 16>{});
}
template <class F>
void with_bool(bool b, F&& f) {
  if (b) f(std::true_type{});
  else f(std::false_type{});
}

}  // namespace

extern "C" {

moe_status moe_router_forward(const moe_router_problem* p, const void* logits, const float* expert_bias,
                              int32_t* top_experts, float* router_weights, void* stream) {
  MOE_TRY(check_router(p));
  if (p->tokens > 0 && (!logits || !top_experts || !router_weights)) return MOE_ERR_NULL;
  if (!elem_aligned(logits, p->logits_dtype) || !aligned4(expert_bias) || !aligned4(top_experts) ||
      !aligned4(router_weights))
    return MOE_ERR_LAYOUT;
  if (p->tokens == 0) return MOE_OK;
  RouterArgs a = router_args(p, logits);
  a.bias = expert_bias;
  a.top = top_experts;
  a.rw = router_weights;
  const dim3 grid((unsigned)((p->tokens + kRouterRows - 1) / kRouterRows));
  hipStream_t st = static_cast<hipStream_t>(stream);
  return launch("router_fwd", st, [&] {
    with_epl(a.E, [&](auto epl) {
      with_bool(p->logits_dtype == MOE_BF16, [&](auto bf) {
        with_bool(p->score == MOE_ROUTER_SOFTMAX, [&](auto sm) {
          with_bool(a.bias != nullptr, [&](auto bi) {
            hipLaunchKernelGGL((k_router_fwd<epl(), bf(), sm(), bi()>), grid, dim3(kRouterThreads), 0, st, a);
          });
        });
      });
    });
  });
}

moe_status moe_router_backward(const moe_router_problem* p, const void* logits, const int32_t* top_experts,
                               const float* grad_router_weights, void* grad_logits, int64_t ld_grad_logits,
                               void* stream) {
  MOE_TRY(check_router(p));
  if (p->tokens > 0 && (!logits || !top_experts || !grad_router_weights || !grad_logits)) return MOE_ERR_NULL;
  if (ld_grad_logits < p->experts) return MOE_ERR_LAYOUT;
  if (!elem_aligned(logits, p->logits_dtype) || !elem_aligned(grad_logits, p->logits_dtype) ||
      !aligned4(top_experts) || !aligned4(grad_router_weights))
    return MOE_ERR_LAYOUT;
  if (p->tokens == 0) return MOE_OK;
  RouterArgs a = router_args(p, logits);
  a.top = const_cast<int32_t*>(top_experts);
  a.gw = grad_router_weights;
  a.dl = grad_logits;
  a.ld_dl = ld_grad_logits;
  const dim3 grid((unsigned)((p->tokens + kRouterRows - 1) / kRouterRows));
  hipStream_t st = static_cast<hipStream_t>(stream);
  return launch("router_bwd", st, [&] {
    with_epl(a.E, [&](auto epl) {
      with_bool(p->logits_dtype == MOE_BF16, [&](auto bf) {
        with_bool(p->score == MOE_ROUTER_SOFTMAX, [&](auto sm) {
          hipLaunchKernelGGL((k_router_bwd<epl(), bf(), sm()>), grid, dim3(kRouterThreads), 0, st, a);
        });
      });
    });
  });
}

}  // extern "C"

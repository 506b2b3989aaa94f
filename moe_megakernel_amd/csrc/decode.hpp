// The layer's forward for a few tokens (moe_forward_decode): arguments and launchers of its
// two kernels.
#pragma once
#include "common.hpp"

namespace moe {
namespace decode {

constexpr int kMaxTokens = 64;                        // MOE_DECODE_MAX_TOKENS
constexpr int kMaxRoutes = kMaxTokens * kMaxTopk;
constexpr int kRouteInvalid = 9;                      // MOE_ERR_ROUTE_INVALID

// What the first kernel's block 0 leaves for the second: the distinct experts in
// ascending order and each one's routes (t K + k) in ascending order.
struct Plan {
  int32_t status;                                     // 0 or kRouteInvalid
  int32_t groups;                                     // distinct experts
  int32_t expert[kMaxExperts + 1];
  int32_t first[kMaxExperts + 2];                     // into route; first[groups] = routes
  int32_t route[kMaxRoutes];
  float weight[kMaxRoutes];                           // of the routes
};

// The second kernel's launch: row fragments a workgroup (16 output columns each), and workgroups
// that share a workgroup's columns.  Its 8 waves are two a SIMD, which leaves the registers for two
// steps of h's two parts in flight.
//   Up to H 4096 one fragment, at most one workgroup a CU.  Above, two fragments share the tokens'
// loads: 226 us against 283 at H 7168 (64 tokens over 64 E4M3 experts), 66 against 87 (64 over 16
// BF16), 98 against 109 at H 5120 (16 over 32 BF16).
//   A short H is split where that leaves every wave at least 2 steps (56 tokens over 7 BF16 experts
// of H 1280, I 640: 13.4 us against 15.2 with 8).  `split` does not fall as T grows, so a workspace
// sized for T serves every smaller batch.
constexpr int kFc2Waves = 8;
struct Fc2Shape {
  int frags, split;
};
inline Fc2Shape fc2_shape(int64_t T, int64_t H, int64_t I, int64_t E, int64_t K) {
  Fc2Shape f;
  f.frags = H / 16 <= 256 ? 1 : 2;
  const int64_t tiles = H / (16 * f.frags), experts = E < T * K ? E : T * K;
  int64_t split = 256 / tiles;
  const int64_t fed = experts * (I / 128) / (2 * kFc2Waves);
  if (split > fed) split = fed;
  f.split = split < 1 ? 1 : (int)split;
  return f;
}

struct Args {
  const uint16_t* x;          // [T][H]
  const int32_t* top;         // [T][K]
  const float* rw;            // [T][K]
  int T, H, I, E, K;
  int shared;                 // the shared expert takes part
  float limit;                // SwiGLU clamp, 0: none
  MxRef gate, up, down;       // routed weights (scale: MXFP8 only)
  MatRef sgate, sup, sdown;   // shared expert, BF16
  const uint16_t* gw;         // shared output gate's weight [H], or null
  Plan* plan;
  float* gate_s;              // [T] sigmoid(x . gw)
  uint16_t* h;                // [T K + T][2 I]: routed rows by route, then the shared expert's; two parts
  uint16_t* out;              // [T][H]
  int tiles2, split;          // the second kernel's grid
  int32_t* arrived;           // [tiles2], zeroed by the first kernel
  float* sums;                // [tiles2][split][T][16 frags] when split > 1
};

template <bool MX>
void launch_fc1(hipStream_t st, const Args& a);
template <bool MX>
void launch_fc2(hipStream_t st, const Args& a);

}  // namespace decode
}  // namespace moe

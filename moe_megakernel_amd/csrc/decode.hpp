// The layer's forward for a few tokens (moe_forward_decode): arguments and launchers of its
// two kernels.
#pragma once
#include "common.hpp"

namespace moe {
namespace decode {

constexpr int kMaxTokens = 64;                        // MOE_DECODE_MAX_TOKENS
constexpr int kMaxRoutes = kMaxTokens * kMaxTopk;

// What the first kernel's block 0 leaves for the second: the distinct experts in
// ascending order and each one's routes (t K + k) in ascending order.
struct Plan {
  int32_t status;                                     // 0 or MOE_ERR_ROUTE_INVALID
  int32_t groups;                                     // distinct experts
  int32_t expert[kMaxExperts + 1];
  int32_t first[kMaxExperts + 2];                     // into route; first[groups] = routes
  int32_t route[kMaxRoutes];
  float weight[kMaxRoutes];                           // of the routes
};

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
  uint16_t* h;                // [T K + T][I]: routed rows by route, then the shared expert's
  uint16_t* out;              // [T][H]
};

template <bool MX>
void launch_fc1(hipStream_t st, const Args& a);
template <bool MX>
void launch_fc2(hipStream_t st, const Args& a);

}  // namespace decode
}  // namespace moe

// The gated feed-forward block: arguments and launchers of its kernels.
#pragma once
#include "dense.hpp"

namespace moe {
namespace ffn {

enum Act { kSilu = 1, kGelu = 2 };          // moe_ffn_activation
enum Saved { kNone = 0, kBf16 = 1, kInt8 = 4 };   // 0 or moe_dtype

// A BF16 matrix, rows ld elements apart.
struct Mat {
  uint16_t* p;
  int64_t ld;
};

// What the forward keeps of a = x gate^T and b = x up^T: BF16 [T][2I], or codes [T][2I] and scale
// bytes [T][2I / 32]; a at column j, b at I + j.
struct Kept {
  uint8_t* ab;
  uint8_t* scales;
};

// How a product is cut: the tiles, and over how many workgroups each one's contraction is split.
enum Shape { kMedium = 0, kMid = 1, kLarge = 2 };
struct Plan {
  int shape;
  dense::Split split;
};

// h = act(a) b
struct UpArgs {
  Mat x, gate, up, h;
  Kept kept;
  int T, H, I, act, saved;
  Plan plan;
};
// out = h down^T (K = I), or grad_x = dab [gate; up] (K = 2I, b1 the second half's rows)
struct RowsArgs {
  Mat a, b0, b1, c;
  int T, N, K, ksplit;
  Plan plan;
};
// dh = dy down; dab = [da | db]; h again for the weight gradient
struct DhArgs {
  Mat dy, down;
  Kept kept;
  uint16_t* dab;         // [T][2I]
  uint16_t* h;           // [T][I]
  int T, H, I, act, saved;
  Plan plan;
};
// c[m][n] (+)= sum_t a[t][m] b[t][n]; rows m >= msplit go to c1
struct WgradArgs {
  Mat a, b;
  void *c0, *c1;
  int64_t ldc0, ldc1;
  int M, N, T, msplit;
  int fp32, overwrite;
  Plan plan;
};

constexpr int64_t kShapeRows[] = {128, 192, 256}, kShapeCols[] = {128, 256, 256};   // of a Shape's tile

void launch_up(hipStream_t st, const UpArgs& a);
void launch_down(hipStream_t st, const RowsArgs& a);
void launch_dh(hipStream_t st, const DhArgs& a);
void launch_dx(hipStream_t st, const RowsArgs& a);
void launch_wgrad(hipStream_t st, const WgradArgs& a);
// the same for split contractions: the parts' sums added up
void launch_up_sum(hipStream_t st, const UpArgs& a);
void launch_rows_sum(hipStream_t st, const RowsArgs& a);
void launch_dh_sum(hipStream_t st, const DhArgs& a);
void launch_wgrad_sum(hipStream_t st, const WgradArgs& a);

// up to kFewTokens tokens, nothing kept or a and b in BF16 (a block of 32 columns does not end in one workgroup there)
constexpr int kFewTokens = 64;
void launch_up_few(hipStream_t st, const UpArgs& a);   // h in two parts: rows T .. 2T - 1 are the second's
int few_parts(int T, int N, int K);                    // of the contraction of launch_down_few
void launch_down_few(hipStream_t st, const RowsArgs& a);

}  // namespace ffn
}  // namespace moe

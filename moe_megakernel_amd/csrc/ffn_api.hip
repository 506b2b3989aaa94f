// Host side of the gated feed-forward block: checks, the layout of `saved` and the workspaces, and
// the launches.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "../../include/moe.h"
#include "checkpoint.hpp"
#include "ffn.hpp"
#include "host.hpp"

using namespace moe;

static_assert(ffn::kFewTokens == MOE_FFN_FEW_TOKENS, "as the header says");

namespace {

moe_status check_problem(const moe_ffn_problem* p) {
  if (!p) return MOE_ERR_NULL;
  const int64_t T = p->tokens, H = p->hidden, I = p->intermediate, most = 1 << 17;
  if (T < 0 || T > (1 << 24) || H < 64 || H > most || H % 64 || I < 64 || I > most || I % 64) return MOE_ERR_SHAPE;
  if (T * (H + 2 * I) > (int64_t)1 << 38) return MOE_ERR_SHAPE;
  if (p->activation != MOE_FFN_SILU && p->activation != MOE_FFN_GELU) return MOE_ERR_UNSUPPORTED;
  if (p->saved_dtype != 0 && p->saved_dtype != MOE_BF16 && p->saved_dtype != MOE_MXINT8) return MOE_ERR_DTYPE;
  if (p->grad_dtype != MOE_FP32 && p->grad_dtype != MOE_BF16) return MOE_ERR_DTYPE;
  if (p->flags & ~MOE_FFN_OVERWRITE_GRADS) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

struct Offsets {
  size_t total = 0;
  size_t take(size_t bytes) {
    const size_t at = total;
    total = align_up(at + bytes);
    return at;
  }
};

size_t saved_layout(const moe_ffn_problem* p, moe_ffn_saved_layout* L) {
  const size_t T = p->tokens, H = p->hidden, I = p->intermediate;
  *L = moe_ffn_saved_layout{};
  if (!p->saved_dtype) return 0;
  Offsets o;
  const bool i8 = p->saved_dtype == MOE_MXINT8;
  L->ab = o.take(T * 2 * I * (i8 ? 1 : 2));
  if (i8) {
    L->ab_scales = o.take(T * (2 * I / 32));
    L->x = o.take(T * H);
    L->x_scales = o.take(T * (H / 32));
  }
  return o.total > kAlign ? o.total : kAlign;
}

// What a round of `w` workgroups at once takes, in us, for `stages` stages of 32 k each: a start and an end, and a time a stage
// that grows with the CUs at work.  Larger tiles have a CU to themselves (up to 256), so what their ends read
// and write (`bytes` a result element, 2 in the figures) is time in which nothing multiplies; Medium ones (up to 512, two a
// CU) hide most of that behind each other.
double round_us(int shape, int64_t w, double stages, double bytes) {
  const double a = (double)w / 256, end = (bytes - 2.0) * ffn::kShapeRows[shape] * ffn::kShapeCols[shape] * w / 4.9e6;
  if (shape == ffn::kLarge) return (0.57 + 0.20 * a) * stages + 14.0 + end;
  if (shape == ffn::kMid) return (0.50 + 0.19 * a) * stages + 14.0 + end;
  return (w > 256 ? 0.62 * stages + 10.0 : (0.20 + 0.08 * a * a) * stages + 8.0) + 0.1 * end;
}

// How an m x n product over k is cut: the tiles and the parts of the contraction that are expected to end first.  Adding up
// parts costs a launch and their way to memory and back.  Measured, in us, Medium / Mid / Large tiles, the parts in brackets:
// 777 x 24576 over 4096 260 / 176 / 198, 777 x 4096 over 12288 124 [4] / 110 [3] / 100 [4] (one part: 133 / 204 / 230), 777 x 4096 over
// 24576 224 [4] / 202 [3] / 168 [4], 300 x 1024 over 5632 22 [8] / 32 [8] / 37 [8] (45 / 96 / 113), 200 x 1024 over 4096 19 [8] / 29 [8] /
// 34 [8] (37 / 85 / 96), 512 x 1024 over 4096 21 [8] / - / 33 [8] (35 / - / 90), 4096 x 4096 over 4096 173 / - / 118; dh, which ends with
// 10 bytes an element, 4096 x 12288 over 4096 540 / - / 445, 4690 x 5504 over 1024 107 / - / 142.
constexpr int kMaxSplit = 16;
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

ffn::Plan cut(int64_t m, int64_t n, int64_t k, double bytes, bool mid, float* sums) {
  ffn::Plan best{ffn::kMedium, {sums, 1}};
  double least = 1e30;
  for (int s = ffn::kMedium; s <= ffn::kLarge; ++s) {
    if (s == ffn::kMid && !mid) continue;
    const int64_t tiles = ceil_div(m, ffn::kShapeRows[s]) * ceil_div(n, ffn::kShapeCols[s]), most = s == ffn::kMedium ? 512 : 256;
    for (int parts = 1; parts <= kMaxSplit; ++parts) {
      const int64_t w = tiles * parts;
      const double stages = (double)ceil_div(k, 32) / parts, out = parts > 1 ? 4.0 : bytes;
      if (parts > 1 && (w > most || stages < 8)) break;
      double us = (double)(w / most) * round_us(s, most, stages, out) + (w % most ? round_us(s, w % most, stages, out) : 0.0);
      if (parts > 1) us += 4.0 + ((double)parts * 4 + bytes) * (double)(m * n) / 6e6;
      if (us < least) least = us, best.shape = s, best.split.n = parts;
    }
  }
  return best;
}
// Bytes of a split product's sums, no less than what fewer rows or a shorter contraction take: all workgroups of a round
// at most, and all parts of the result.
size_t split_bytes(int64_t m, int64_t n, int64_t k) {
  const int64_t parts = std::min<int64_t>(ceil_div(k, 32) / 8, kMaxSplit), round = (int64_t)256 * 256 * 256 * 4;
  return parts < 2 ? 0 : (size_t)std::min(m * n * 4 * parts, round);
}

struct Fwd {
  size_t h, sums, total;
};
Fwd fwd_layout(const moe_ffn_problem* p) {
  const size_t T = p->tokens, H = p->hidden, I = p->intermediate;
  Offsets o;
  Fwd f;
  f.h = o.take(2 * I * std::max<size_t>(T, 2 * std::min<size_t>(T, ffn::kFewTokens)));   // of few tokens in two parts
  f.sums = o.take(std::max(split_bytes(T, 2 * I, H), split_bytes(T, H, I)));
  f.total = o.total > kAlign ? o.total : kAlign;
  return f;
}
struct Bwd {
  size_t dab, h, x, sums, total;
};
Bwd bwd_layout(const moe_ffn_problem* p) {
  const size_t T = p->tokens, H = p->hidden, I = p->intermediate;
  Offsets o;
  Bwd b;
  b.dab = o.take(4 * T * I);
  b.h = o.take(2 * T * I);
  b.x = o.take(p->saved_dtype == MOE_MXINT8 ? 2 * T * H : 0);
  b.sums = o.take(std::max(std::max(split_bytes(T, I, H), split_bytes(T, H, 2 * I)), split_bytes(2 * I, H, T)));
  b.total = o.total > kAlign ? o.total : kAlign;
  return b;
}

// How each product is cut: bytes a result element at its end, and whether 192 x 256 tiles are built.
bool few(const moe_ffn_problem* p) { return p->tokens <= ffn::kFewTokens && p->saved_dtype != MOE_MXINT8; }
ffn::Plan plan_up(const moe_ffn_problem* p, float* sums) {
  const double ab = p->saved_dtype == 0 ? 0.0 : p->saved_dtype == MOE_BF16 ? 2.0 : 1.0;   // kept of each of a and b
  return cut(p->tokens, 2 * p->intermediate, p->hidden, 1.0 + ab, true, sums);
}
ffn::Plan plan_down(const moe_ffn_problem* p, float* sums) {
  // few: within kMaxSplit and eight stages a part, which split_bytes counts
  if (few(p)) return {0, {sums, ffn::few_parts((int)p->tokens, (int)p->hidden, (int)p->intermediate)}};
  return cut(p->tokens, p->hidden, p->intermediate, 2.0, true, sums);
}
ffn::Plan plan_dh(const moe_ffn_problem* p, float* sums) {
  return cut(p->tokens, p->intermediate, p->hidden, p->saved_dtype == MOE_MXINT8 ? 8.0 : 10.0, true, sums);
}
ffn::Plan plan_dx(const moe_ffn_problem* p, float* sums) {
  return cut(p->tokens, p->hidden, 2 * p->intermediate, 2.0, true, sums);
}
double grad_bytes(const moe_ffn_problem* p) {
  return (p->grad_dtype == MOE_FP32 ? 4.0 : 2.0) * (p->flags & MOE_FFN_OVERWRITE_GRADS ? 1 : 2);
}
ffn::Plan plan_wgrad_down(const moe_ffn_problem* p, float* sums) {
  return cut(p->hidden, p->intermediate, p->tokens, grad_bytes(p), false, sums);
}
ffn::Plan plan_wgrad_up(const moe_ffn_problem* p, float* sums) {
  return cut(2 * p->intermediate, p->hidden, p->tokens, grad_bytes(p), false, sums);
}
moe_ffn_cut shown(const ffn::Plan& c) {
  return {(int32_t)ffn::kShapeRows[c.shape], (int32_t)ffn::kShapeCols[c.shape], c.split.n};
}

// A matrix of `cols` columns that moves in 16-byte pieces.
moe_status check_rows(const moe_rows* m, int64_t cols, int per16) {
  if (!m || !m->base) return MOE_ERR_NULL;
  if (m->ld < cols || m->ld % per16 || m->ld > MOE_FFN_MAX_LD || !aligned16(m->base)) return MOE_ERR_LAYOUT;
  return MOE_OK;
}
moe_status check_bf16(const moe_rows* m, int64_t cols) { return check_rows(m, cols, 8); }

ffn::Mat mat(const moe_rows* m) { return {static_cast<uint16_t*>(m->base), m->ld}; }

ffn::Kept kept(const void* saved, const moe_ffn_saved_layout& L) {
  uint8_t* s = static_cast<uint8_t*>(const_cast<void*>(saved));
  return {s + L.ab, s + L.ab_scales};
}

}  // namespace

extern "C" {

size_t moe_ffn_saved_bytes(const moe_ffn_problem* p) {
  moe_ffn_saved_layout L;
  return check_problem(p) == MOE_OK ? saved_layout(p, &L) : 0;
}

size_t moe_ffn_workspace_bytes(const moe_ffn_problem* p, int for_backward) {
  if (check_problem(p) != MOE_OK || (for_backward && !p->saved_dtype)) return 0;
  return for_backward ? bwd_layout(p).total : fwd_layout(p).total;
}

moe_status moe_ffn_saved_view(const moe_ffn_problem* p, moe_ffn_saved_layout* layout) {
  MOE_TRY(check_problem(p));
  if (!layout) return MOE_ERR_NULL;
  if (!p->saved_dtype) return MOE_ERR_UNSUPPORTED;
  saved_layout(p, layout);
  return MOE_OK;
}

moe_status moe_ffn_plan_view(const moe_ffn_problem* p, moe_ffn_plan* plan) {
  MOE_TRY(check_problem(p));
  if (!plan) return MOE_ERR_NULL;
  *plan = moe_ffn_plan{};
  if (p->tokens == 0) return MOE_OK;
  if (few(p)) {
    plan->up.parts = 1;
    plan->down.parts = plan_down(p, nullptr).split.n;
  } else {
    plan->up = shown(plan_up(p, nullptr));
    plan->down = shown(plan_down(p, nullptr));
  }
  if (!p->saved_dtype) return MOE_OK;
  plan->dh = shown(plan_dh(p, nullptr));
  plan->dx = shown(plan_dx(p, nullptr));
  plan->wgrad_down = shown(plan_wgrad_down(p, nullptr));
  plan->wgrad_up = shown(plan_wgrad_up(p, nullptr));
  return MOE_OK;
}

moe_status moe_ffn_forward(const moe_ffn_problem* p, const moe_rows* x, const moe_rows* gate, const moe_rows* up,
                           const moe_rows* down, const moe_rows* out, void* saved, void* workspace,
                           size_t workspace_bytes, void* stream) {
  MOE_TRY(check_problem(p));
  if (p->tokens == 0) return MOE_OK;
  const int T = (int)p->tokens, H = (int)p->hidden, I = (int)p->intermediate;
  MOE_TRY(check_bf16(x, H));
  MOE_TRY(check_bf16(gate, H));
  MOE_TRY(check_bf16(up, H));
  MOE_TRY(check_bf16(down, I));
  MOE_TRY(check_bf16(out, H));
  if ((saved != nullptr) != (p->saved_dtype != 0)) return MOE_ERR_WORKSPACE;
  const Fwd F = fwd_layout(p);
  if (!workspace || workspace_bytes < F.total) return MOE_ERR_WORKSPACE;
  if (!aligned16(workspace) || (saved && !aligned16(saved))) return MOE_ERR_LAYOUT;
  hipStream_t st = static_cast<hipStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  moe_ffn_saved_layout L;
  saved_layout(p, &L);
  const ffn::Mat h{reinterpret_cast<uint16_t*>(ws + F.h), I};
  // x is read by the checkpoint and the first product alone: out, which the second writes, may take its place
  if (p->saved_dtype == MOE_MXINT8) {
    uint8_t* s = static_cast<uint8_t*>(saved);
    const checkpoint::Args c{static_cast<uint8_t*>(x->base), x->ld, T, H, s + L.x, s + L.x_scales};
    MOE_TRY(launch("checkpoint_store", st, [&] { checkpoint::launch_store(st, c, false); }));
  }
  ffn::UpArgs u{mat(x), mat(gate), mat(up), h, kept(saved, L), T, H, I, p->activation, p->saved_dtype};
  ffn::RowsArgs d{h, mat(down), mat(down), mat(out), T, H, I, I};
  float* sums = reinterpret_cast<float*>(ws + F.sums);
  d.plan = plan_down(p, sums);
  if (few(p)) {
    MOE_TRY(launch("ffn_up_few", st, [&] { ffn::launch_up_few(st, u); }));
    MOE_TRY(launch("ffn_down_few", st, [&] { ffn::launch_down_few(st, d); }));
    if (d.plan.split.n > 1) MOE_TRY(launch("ffn_down_few_sum", st, [&] { ffn::launch_rows_sum(st, d); }));
    return MOE_OK;
  }
  u.plan = plan_up(p, sums);
  MOE_TRY(launch("ffn_up", st, [&] { ffn::launch_up(st, u); }));
  if (u.plan.split.n > 1) MOE_TRY(launch("ffn_up_sum", st, [&] { ffn::launch_up_sum(st, u); }));
  MOE_TRY(launch("ffn_down", st, [&] { ffn::launch_down(st, d); }));
  if (d.plan.split.n > 1) MOE_TRY(launch("ffn_down_sum", st, [&] { ffn::launch_rows_sum(st, d); }));
  return MOE_OK;
}

moe_status moe_ffn_backward(const moe_ffn_problem* p, const moe_rows* grad_out, const moe_rows* x,
                            const moe_rows* gate, const moe_rows* up, const moe_rows* down, const void* saved,
                            const moe_rows* grad_x, const moe_rows* grad_gate, const moe_rows* grad_up,
                            const moe_rows* grad_down, void* workspace, size_t workspace_bytes, void* stream) {
  MOE_TRY(check_problem(p));
  if (!p->saved_dtype) return MOE_ERR_UNSUPPORTED;
  const int T = (int)p->tokens, H = (int)p->hidden, I = (int)p->intermediate;
  const bool i8 = p->saved_dtype == MOE_MXINT8, f32 = p->grad_dtype == MOE_FP32;
  const int per16 = f32 ? 4 : 8;
  if ((grad_gate != nullptr) != (grad_up != nullptr) || (!grad_x && !grad_gate && !grad_down)) return MOE_ERR_NULL;
  if (grad_x && T > 0) MOE_TRY(check_bf16(grad_x, H));
  if (grad_gate) {
    MOE_TRY(check_rows(grad_gate, H, per16));
    MOE_TRY(check_rows(grad_up, H, per16));
  }
  if (grad_down) MOE_TRY(check_rows(grad_down, I, per16));
  const Bwd B = bwd_layout(p);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  if (T > 0) {
    MOE_TRY(check_bf16(grad_out, H));
    if (i8 && x) return MOE_ERR_UNSUPPORTED;
    if (!i8 && grad_gate) MOE_TRY(check_bf16(x, H));
    MOE_TRY(check_bf16(down, I));
    if (grad_x) {
      MOE_TRY(check_bf16(gate, H));
      MOE_TRY(check_bf16(up, H));
    }
    if (!saved || !workspace || workspace_bytes < B.total) return MOE_ERR_WORKSPACE;
    if (!aligned16(workspace) || !aligned16(saved)) return MOE_ERR_LAYOUT;
  }
  hipStream_t st = static_cast<hipStream_t>(stream);
  moe_ffn_saved_layout L;
  saved_layout(p, &L);
  const ffn::Mat dab{reinterpret_cast<uint16_t*>(ws + B.dab), 2 * I}, h{reinterpret_cast<uint16_t*>(ws + B.h), I};
  float* sums = reinterpret_cast<float*>(ws + B.sums);
  if (T > 0) {
    const ffn::DhArgs d{mat(grad_out), mat(down), kept(saved, L), dab.p, h.p, T, H, I, p->activation, p->saved_dtype,
                        plan_dh(p, sums)};
    MOE_TRY(launch("ffn_dh", st, [&] { ffn::launch_dh(st, d); }));
    if (d.plan.split.n > 1) MOE_TRY(launch("ffn_dh_sum", st, [&] { ffn::launch_dh_sum(st, d); }));
  } else if (!(p->flags & MOE_FFN_OVERWRITE_GRADS)) {
    return MOE_OK;
  }
  const int over = (p->flags & MOE_FFN_OVERWRITE_GRADS) ? 1 : 0;
  if (grad_down) {
    const ffn::Mat dy = T > 0 ? mat(grad_out) : ffn::Mat{nullptr, H};
    const ffn::WgradArgs w{dy, h, grad_down->base, nullptr, grad_down->ld, 0, H, I, T, H, f32, over, plan_wgrad_down(p, sums)};
    MOE_TRY(launch("ffn_wgrad_down", st, [&] { ffn::launch_wgrad(st, w); }));
    if (w.plan.split.n > 1) MOE_TRY(launch("ffn_wgrad_down_sum", st, [&] { ffn::launch_wgrad_sum(st, w); }));
  }
  if (grad_gate) {
    ffn::Mat xs{reinterpret_cast<uint16_t*>(ws + B.x), H};
    if (T > 0) {
      if (i8) {
        uint8_t* s = static_cast<uint8_t*>(const_cast<void*>(saved));
        const checkpoint::Args c{ws + B.x, H, T, H, s + L.x, s + L.x_scales};
        MOE_TRY(launch("checkpoint_load", st, [&] { checkpoint::launch_load(st, c, false); }));
      } else {
        xs = mat(x);
      }
    }
    const ffn::WgradArgs w{dab, xs, grad_gate->base, grad_up->base, grad_gate->ld, grad_up->ld, 2 * I, H, T, I, f32,
                           over, plan_wgrad_up(p, sums)};
    MOE_TRY(launch("ffn_wgrad_up", st, [&] { ffn::launch_wgrad(st, w); }));
    if (w.plan.split.n > 1) MOE_TRY(launch("ffn_wgrad_up_sum", st, [&] { ffn::launch_wgrad_sum(st, w); }));
  }
  if (grad_x && T > 0) {                     // last: it may take the place of grad_out or x
    const ffn::RowsArgs r{dab, mat(gate), mat(up), mat(grad_x), T, H, 2 * I, I, plan_dx(p, sums)};
    MOE_TRY(launch("ffn_dx", st, [&] { ffn::launch_dx(st, r); }));
    if (r.plan.split.n > 1) MOE_TRY(launch("ffn_dx_sum", st, [&] { ffn::launch_rows_sum(st, r); }));
  }
  return MOE_OK;
}

}  // extern "C"

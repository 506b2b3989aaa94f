// Host side of the gated feed-forward block: checks, the layout of `saved` and the workspaces, and
// the launches.
#include <hip/hip_runtime.h>

#include "../../include/moe.h"
#include "checkpoint.hpp"
#include "ffn.hpp"
#include "host.hpp"

using namespace moe;

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

struct Fwd {
  size_t h, total;
};
Fwd fwd_layout(const moe_ffn_problem* p) {
  Offsets o;
  Fwd f;
  f.h = o.take((size_t)2 * p->tokens * p->intermediate);
  f.total = o.total > kAlign ? o.total : kAlign;
  return f;
}
struct Bwd {
  size_t dab, h, x, total;
};
Bwd bwd_layout(const moe_ffn_problem* p) {
  const size_t T = p->tokens, H = p->hidden, I = p->intermediate;
  Offsets o;
  Bwd b;
  b.dab = o.take(4 * T * I);
  b.h = o.take(2 * T * I);
  b.x = o.take(p->saved_dtype == MOE_MXINT8 ? 2 * T * H : 0);
  b.total = o.total > kAlign ? o.total : kAlign;
  return b;
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
  if (p->saved_dtype == MOE_MXINT8) {
    uint8_t* s = static_cast<uint8_t*>(saved);
    const checkpoint::Args c{static_cast<uint8_t*>(x->base), x->ld, T, H, s + L.x, s + L.x_scales};
    MOE_TRY(launch("checkpoint_store", st, [&] { checkpoint::launch_store(st, c, false); }));
  }
  const ffn::UpArgs u{mat(x), mat(gate), mat(up), h, kept(saved, L), T, H, I, p->activation, p->saved_dtype};
  const ffn::RowsArgs d{h, mat(down), mat(down), mat(out), T, H, I, I};
  if (T <= ffn::kFewTokens && !p->saved_dtype) {
    MOE_TRY(launch("ffn_up_few", st, [&] { ffn::launch_up_few(st, u); }));
    return launch("ffn_down_few", st, [&] { ffn::launch_down_few(st, d); });
  }
  MOE_TRY(launch("ffn_up", st, [&] { ffn::launch_up(st, u); }));
  return launch("ffn_down", st, [&] { ffn::launch_down(st, d); });
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
  if (T > 0) {
    const ffn::DhArgs d{mat(grad_out), mat(down), kept(saved, L), dab.p, h.p, T, H, I, p->activation, p->saved_dtype};
    MOE_TRY(launch("ffn_dh", st, [&] { ffn::launch_dh(st, d); }));
    if (grad_x) {
      const ffn::RowsArgs r{dab, mat(gate), mat(up), mat(grad_x), T, H, 2 * I, I};
      MOE_TRY(launch("ffn_dx", st, [&] { ffn::launch_dx(st, r); }));
    }
  } else if (!(p->flags & MOE_FFN_OVERWRITE_GRADS)) {
    return MOE_OK;
  }
  const int over = (p->flags & MOE_FFN_OVERWRITE_GRADS) ? 1 : 0;
  if (grad_down) {
    const ffn::Mat dy = T > 0 ? mat(grad_out) : ffn::Mat{nullptr, H};
    const ffn::WgradArgs w{dy, h, grad_down->base, nullptr, grad_down->ld, 0, H, I, T, H, f32, over};
    MOE_TRY(launch("ffn_wgrad_down", st, [&] { ffn::launch_wgrad(st, w); }));
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
                           over};
    MOE_TRY(launch("ffn_wgrad_up", st, [&] { ffn::launch_wgrad(st, w); }));
  }
  return MOE_OK;
}

}  // extern "C"

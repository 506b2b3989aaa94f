"""Python binding of libmoe_mi355x.so, the MI355X post-router MoE layer.

Argument marshalling only: every step of the layer runs in the library's HIP
kernels.  The ctypes structures mirror include/moe.h field for field, and the
functions keep the C names.  Torch is used for device memory and the current
stream; helpers at the bottom turn torch tensors into the C descriptors.

The shared library is built in-tree (python -m moe_megakernel_amd.build); if
it is missing, load() raises instead of falling back to anything else.
"""
from __future__ import annotations

import ctypes as C
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe_mi355x.so")

MOE_OK, MOE_ERR_NULL, MOE_ERR_SHAPE, MOE_ERR_DTYPE, MOE_ERR_LAYOUT = 0, 1, 2, 3, 4
MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_ROUTE_OVERFLOW, MOE_ERR_HIP = 5, 6, 7, 8
MOE_ERR_ROUTE_INVALID = 9
MOE_BF16, MOE_FP32, MOE_MXFP8_E4M3 = 1, 2, 3
MOE_FLAG_HAS_SHARED = 1
MOE_FLAG_RECOMPUTE = 2
MOE_FLAG_TOPK_ROUTING = 4
MOE_FLAG_SHARED_GATE = 8
MOE_ROUTER_SOFTMAX, MOE_ROUTER_SIGMOID = 1, 2
MOE_ROUTER_NORMALIZE = 1
MOE_NORM_LAYER, MOE_NORM_RMS = 1, 2
MOE_NORM_OVERWRITE_GRADS = 1
MOE_NORM_MAX_COLS = 16384

EXPORTED = ("moe_saved_bytes", "moe_workspace_bytes", "moe_saved_view", "moe_forward",
            "moe_forward_topk", "moe_forward_noalloc", "moe_backward", "moe_status_str",
            "moe_kernel_timer_enable", "moe_kernel_timer_read", "moe_mx_staging_view",
            "moe_decode_workspace_bytes", "moe_forward_decode", "moe_router_forward", "moe_router_backward",
            "moe_norm_forward", "moe_norm_backward", "moe_norm_workspace_bytes")
MOE_NOALLOC_SCRATCH_BYTES = 64 << 20
MOE_DECODE_MAX_TOKENS = 64
MOE_DECODE_MAX_INTERMEDIATE = 65536


class moe_problem(C.Structure):
    _fields_ = [("tokens", C.c_int64), ("hidden", C.c_int64), ("intermediate", C.c_int64),
                ("experts", C.c_int32), ("topk", C.c_int32), ("routed_dtype", C.c_int32),
                ("flags", C.c_uint32), ("swiglu_limit", C.c_float)]


class moe_mat(C.Structure):
    _fields_ = [("base", C.c_void_p), ("expert_stride", C.c_int64), ("table", C.c_void_p),
                ("ld", C.c_int64)]


class moe_weight(C.Structure):
    _fields_ = [("dtype", C.c_int32), ("rows", C.c_int64), ("cols", C.c_int64),
                ("row_offset", C.c_int64), ("data", moe_mat), ("scale", moe_mat),
                ("col_data", moe_mat), ("col_scale", moe_mat)]


class moe_weights(C.Structure):
    _fields_ = [(n, moe_weight) for n in ("shared_gate", "shared_up", "shared_down",
                                          "routed_gate", "routed_up", "routed_down", "shared_out_gate")]


class moe_grad(C.Structure):
    _fields_ = [("base", C.c_void_p), ("expert_stride", C.c_int64), ("table", C.c_void_p),
                ("ld", C.c_int64), ("row_offset", C.c_int64), ("dtype", C.c_int32)]


class moe_main_grads(C.Structure):
    _fields_ = [(n, moe_grad) for n in ("shared_gate", "shared_up", "shared_down",
                                        "routed_gate", "routed_up", "routed_down", "shared_out_gate")]


class moe_saved_layout(C.Structure):
    _fields_ = [(n, C.c_size_t) for n in ("top_experts", "router_weights", "counts", "offsets",
                                          "slot_of", "slot_token", "status_word")]


class moe_mx_staging_layout(C.Structure):
    _fields_ = [(n, C.c_size_t) for n in ("x_codes", "x_scales", "h_codes", "h_scales",
                                          "dy_codes", "dy_scales", "dfc1_codes", "dfc1_scales")]


class moe_router_problem(C.Structure):
    _fields_ = [("tokens", C.c_int64), ("experts", C.c_int32), ("topk", C.c_int32), ("score", C.c_int32),
                ("logits_dtype", C.c_int32), ("flags", C.c_uint32), ("scale", C.c_float),
                ("ld_logits", C.c_int64)]


class moe_norm_problem(C.Structure):
    _fields_ = [("rows", C.c_int64), ("cols", C.c_int64), ("kind", C.c_int32), ("dtype", C.c_int32),
                ("param_dtype", C.c_int32), ("grad_dtype", C.c_int32), ("flags", C.c_uint32),
                ("eps", C.c_float)]


class moe_rows(C.Structure):
    _fields_ = [("base", C.c_void_p), ("ld", C.c_int64)]


_lib = None


def load(path: str | None = None):
    """Load the in-tree shared library (raises FileNotFoundError if it was not built)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise FileNotFoundError(f"{p} is missing: build it with `python -m moe_megakernel_amd.build`")
    lib = C.CDLL(p)
    P = C.POINTER
    lib.moe_saved_bytes.argtypes = [P(moe_problem)]
    lib.moe_saved_bytes.restype = C.c_size_t
    lib.moe_workspace_bytes.argtypes = [P(moe_problem), C.c_int]
    lib.moe_workspace_bytes.restype = C.c_size_t
    lib.moe_saved_view.argtypes = [P(moe_problem), P(moe_saved_layout)]
    lib.moe_saved_view.restype = C.c_int
    lib.moe_forward.argtypes = [P(moe_problem), C.c_void_p, C.c_void_p, C.c_void_p, P(moe_weights),
                                C.c_void_p, C.c_void_p, C.c_void_p, C.c_size_t, C.c_void_p]
    lib.moe_forward.restype = C.c_int
    lib.moe_forward_topk.argtypes = lib.moe_forward.argtypes
    lib.moe_forward_topk.restype = C.c_int
    lib.moe_forward_noalloc.argtypes = [P(moe_problem), C.c_void_p, C.c_void_p, C.c_void_p, P(moe_weights),
                                        C.c_void_p, C.c_void_p, C.c_void_p]
    lib.moe_forward_noalloc.restype = C.c_int
    lib.moe_backward.argtypes = [P(moe_problem), C.c_void_p, C.c_void_p, P(moe_weights), C.c_void_p,
                                 C.c_void_p, C.c_void_p, P(moe_main_grads), C.c_void_p, C.c_size_t,
                                 C.c_void_p]
    lib.moe_backward.restype = C.c_int
    lib.moe_status_str.argtypes = [C.c_int]
    lib.moe_status_str.restype = C.c_char_p
    lib.moe_kernel_timer_enable.argtypes = [C.c_int]
    lib.moe_kernel_timer_enable.restype = None
    lib.moe_kernel_timer_read.argtypes = [P(C.c_char_p), P(C.c_int), P(C.c_double), C.c_int]
    lib.moe_kernel_timer_read.restype = C.c_int
    lib.moe_mx_staging_view.argtypes = [P(moe_problem), P(moe_mx_staging_layout)]
    lib.moe_mx_staging_view.restype = C.c_int
    lib.moe_decode_workspace_bytes.argtypes = [P(moe_problem)]
    lib.moe_decode_workspace_bytes.restype = C.c_size_t
    lib.moe_forward_decode.argtypes = [P(moe_problem), C.c_void_p, C.c_void_p, C.c_void_p, P(moe_weights),
                                       C.c_void_p, C.c_void_p, C.c_size_t, C.c_void_p]
    lib.moe_forward_decode.restype = C.c_int
    lib.moe_router_forward.argtypes = [P(moe_router_problem)] + [C.c_void_p] * 5
    lib.moe_router_forward.restype = C.c_int
    lib.moe_router_backward.argtypes = [P(moe_router_problem)] + [C.c_void_p] * 4 + [C.c_int64, C.c_void_p]
    lib.moe_router_backward.restype = C.c_int
    lib.moe_norm_forward.argtypes = [P(moe_norm_problem), P(moe_rows), P(moe_rows), C.c_void_p, C.c_void_p,
                                     P(moe_rows), P(moe_rows), C.c_void_p, C.c_void_p]
    lib.moe_norm_forward.restype = C.c_int
    lib.moe_norm_backward.argtypes = [P(moe_norm_problem), P(moe_rows), P(moe_rows), C.c_void_p, C.c_void_p,
                                      P(moe_rows), P(moe_rows), C.c_void_p, C.c_void_p, C.c_void_p, C.c_size_t,
                                      C.c_void_p]
    lib.moe_norm_backward.restype = C.c_int
    lib.moe_norm_workspace_bytes.argtypes = [P(moe_norm_problem)]
    lib.moe_norm_workspace_bytes.restype = C.c_size_t
    if path is None:
        _lib = lib
    return lib


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: status {status} ({moe_status_str(status)})")
        self.status = status


# ------------------------------------------------------------------ C entry points
def moe_status_str(status: int) -> str:
    return load().moe_status_str(int(status)).decode()


def moe_saved_bytes(p: moe_problem) -> int:
    return int(load().moe_saved_bytes(C.byref(p)))


def moe_workspace_bytes(p: moe_problem, for_backward: bool) -> int:
    return int(load().moe_workspace_bytes(C.byref(p), int(bool(for_backward))))


def moe_saved_view(p: moe_problem) -> moe_saved_layout:
    out = moe_saved_layout()
    st = load().moe_saved_view(C.byref(p), C.byref(out))
    if st != MOE_OK:
        raise MoeError(st, "moe_saved_view")
    return out


def moe_mx_staging_view(p: moe_problem) -> moe_mx_staging_layout:
    out = moe_mx_staging_layout()
    st = load().moe_mx_staging_view(C.byref(p), C.byref(out))
    if st != MOE_OK:
        raise MoeError(st, "moe_mx_staging_view")
    return out


def moe_forward(p, hidden, probs, routing_map, weights, out, saved, workspace, workspace_bytes, stream) -> int:
    """Raw call with integer device addresses; returns the status code."""
    return load().moe_forward(C.byref(p), hidden, probs, routing_map, C.byref(weights), out, saved,
                              workspace, workspace_bytes, stream)


def moe_forward_noalloc(p, hidden, probs, routing_map, weights, out, saved, stream) -> int:
    """Raw call of the allocation-free forward (its scratch is the library's static per-GPU
    array); returns the status code."""
    return load().moe_forward_noalloc(C.byref(p), hidden, probs, routing_map, C.byref(weights), out, saved,
                                      stream)


def moe_forward_topk(p, hidden, top_experts, router_weights, weights, out, saved, workspace, workspace_bytes,
                     stream) -> int:
    """Raw call with integer device addresses (routing as the [T][K] table); returns the status."""
    return load().moe_forward_topk(C.byref(p), hidden, top_experts, router_weights, C.byref(weights), out,
                                   saved, workspace, workspace_bytes, stream)


def moe_backward(p, grad_out, hidden, weights, saved, grad_hidden, grad_probs, main_grads, workspace,
                 workspace_bytes, stream) -> int:
    return load().moe_backward(C.byref(p), grad_out, hidden, C.byref(weights), saved, grad_hidden,
                               grad_probs, C.byref(main_grads), workspace, workspace_bytes, stream)


def moe_decode_workspace_bytes(p: moe_problem) -> int:
    return int(load().moe_decode_workspace_bytes(C.byref(p)))


def moe_forward_decode(p, hidden, top_experts, router_weights, weights, out, workspace, workspace_bytes,
                       stream) -> int:
    """Raw call of the few-token forward with integer device addresses; returns the status."""
    return load().moe_forward_decode(C.byref(p), hidden, top_experts, router_weights, C.byref(weights), out,
                                     workspace, workspace_bytes, stream)


def moe_router_forward(p, logits, expert_bias, top_experts, router_weights, stream) -> int:
    """Raw call with integer device addresses; returns the status."""
    return load().moe_router_forward(C.byref(p), logits, expert_bias, top_experts, router_weights, stream)


def moe_router_backward(p, logits, top_experts, grad_router_weights, grad_logits, ld_grad_logits, stream) -> int:
    """Raw call with integer device addresses; returns the status."""
    return load().moe_router_backward(C.byref(p), logits, top_experts, grad_router_weights, grad_logits,
                                      ld_grad_logits, stream)


def _ref(rows):
    return None if rows is None else C.byref(rows)


def moe_norm_workspace_bytes(p: moe_norm_problem) -> int:
    return int(load().moe_norm_workspace_bytes(C.byref(p)))


def moe_norm_forward(p, x, residual, weight, bias, sum, y, stats, stream) -> int:
    """Raw call: x, residual, sum and y are moe_rows (or None), the rest integer device
    addresses; returns the status."""
    return load().moe_norm_forward(C.byref(p), _ref(x), _ref(residual), weight, bias, _ref(sum), _ref(y), stats,
                                   stream)


def moe_norm_backward(p, grad_y, x, weight, stats, grad_sum, grad_x, grad_weight, grad_bias, workspace,
                      workspace_bytes, stream) -> int:
    """Raw call: grad_y, x, grad_sum and grad_x are moe_rows (or None), the rest integer
    device addresses; returns the status."""
    return load().moe_norm_backward(C.byref(p), _ref(grad_y), _ref(x), weight, stats, _ref(grad_sum), _ref(grad_x),
                                    grad_weight, grad_bias, workspace, workspace_bytes, stream)


def moe_kernel_timer_enable(on: bool) -> None:
    load().moe_kernel_timer_enable(int(bool(on)))


def moe_kernel_timer_read(cap: int = 64) -> dict:
    """{kernel name: (launches, total ms)} since the previous read."""
    names = (C.c_char_p * cap)()
    cnt = (C.c_int * cap)()
    ms = (C.c_double * cap)()
    n = load().moe_kernel_timer_read(names, cnt, ms, cap)
    return {names[i].decode(): (cnt[i], ms[i]) for i in range(min(n, cap))}


# ------------------------------------------------------------------ torch helpers
def problem(tokens, hidden, inter, experts, topk, routed_dtype=MOE_BF16, flags=MOE_FLAG_HAS_SHARED,
            swiglu_limit=0.0) -> moe_problem:
    return moe_problem(tokens, hidden, inter, experts, topk, routed_dtype, flags, swiglu_limit)


def _ptr(t) -> int:
    return 0 if t is None else int(t.data_ptr())


def mat(base=None, expert_stride=0, table=None, ld=0) -> moe_mat:
    """base/table: torch tensors (table: int64 device tensor of per-expert addresses)."""
    return moe_mat(_ptr(base), int(expert_stride), _ptr(table), int(ld))


def weight(dtype, rows, cols, data: moe_mat, row_offset=0, scale=None, col_data=None,
           col_scale=None) -> moe_weight:
    z = moe_mat(0, 0, 0, 0)
    return moe_weight(dtype, rows, cols, row_offset, data, scale or z, col_data or z, col_scale or z)


def grad(base=None, expert_stride=0, table=None, ld=0, row_offset=0, dtype=None) -> moe_grad:
    """main_grad view; dtype defaults to the tensor's (torch.float32 -> MOE_FP32,
    torch.bfloat16 -> MOE_BF16), else MOE_FP32."""
    if dtype is None:
        dtype = MOE_FP32
        t = base if base is not None else None
        if t is not None and hasattr(t, "dtype"):
            import torch
            dtype = MOE_BF16 if t.dtype == torch.bfloat16 else MOE_FP32
    return moe_grad(_ptr(base), int(expert_stride), _ptr(table), int(ld), int(row_offset), int(dtype))


def current_stream() -> int:
    import torch
    return int(torch.cuda.current_stream().cuda_stream)


class Layer:
    """Caller-side convenience: holds the problem, the caller-owned `saved` and
    workspace tensors (allocated once with torch), and issues the two C calls
    on torch's current stream.  Raises MoeError on a non-OK status."""

    def __init__(self, p: moe_problem, device="cuda"):
        import torch
        self.p = p
        self.saved = torch.empty(max(moe_saved_bytes(p), 256), dtype=torch.uint8, device=device)
        fw = max(moe_workspace_bytes(p, False), 256)
        bw = max(moe_workspace_bytes(p, True), 256)
        self.ws_bytes = max(fw, bw)
        self.workspace = torch.empty(self.ws_bytes, dtype=torch.uint8, device=device)
        if moe_saved_bytes(p) == 0:
            raise MoeError(MOE_ERR_SHAPE, "moe_saved_bytes")

    def forward(self, hidden, probs, routing_map, weights: moe_weights, out):
        st = moe_forward(self.p, _ptr(hidden), _ptr(probs), _ptr(routing_map), weights, _ptr(out),
                         _ptr(self.saved), _ptr(self.workspace), self.ws_bytes, current_stream())
        if st != MOE_OK:
            raise MoeError(st, "moe_forward")
        return out

    def forward_noalloc(self, hidden, probs, routing_map, weights: moe_weights, out):
        """moe_forward_noalloc into this layer's `saved` (no workspace is passed)."""
        st = moe_forward_noalloc(self.p, _ptr(hidden), _ptr(probs), _ptr(routing_map), weights, _ptr(out),
                                 _ptr(self.saved), current_stream())
        if st != MOE_OK:
            raise MoeError(st, "moe_forward_noalloc")
        return out

    def forward_topk(self, hidden, top_experts, router_weights, weights: moe_weights, out):
        st = moe_forward_topk(self.p, _ptr(hidden), _ptr(top_experts), _ptr(router_weights), weights,
                              _ptr(out), _ptr(self.saved), _ptr(self.workspace), self.ws_bytes,
                              current_stream())
        if st != MOE_OK:
            raise MoeError(st, "moe_forward_topk")
        return out

    def backward(self, grad_out, hidden, weights: moe_weights, grad_hidden, grad_probs,
                 main_grads: moe_main_grads):
        st = moe_backward(self.p, _ptr(grad_out), _ptr(hidden), weights, _ptr(self.saved),
                          _ptr(grad_hidden), _ptr(grad_probs), main_grads, _ptr(self.workspace),
                          self.ws_bytes, current_stream())
        if st != MOE_OK:
            raise MoeError(st, "moe_backward")

    def routing_state(self):
        """Integer routing state from `saved` as torch views (device)."""
        import torch
        L = moe_saved_view(self.p)
        T, K, E = self.p.tokens, self.p.topk, self.p.experts

        def view(off, n, dt):
            nbytes = n * 4
            return self.saved[off:off + nbytes].view(dt)
        return {
            "top_experts": view(L.top_experts, T * K, torch.int32).view(T, K),
            "router_weights": view(L.router_weights, T * K, torch.float32).view(T, K),
            "counts": view(L.counts, E, torch.int32),
            "offsets": view(L.offsets, E + 1, torch.int32),
            "slot_of": view(L.slot_of, T * K, torch.int32).view(T, K),
            "slot_token": view(L.slot_token, T * K, torch.int32),
            "status_word": view(L.status_word, 1, torch.int32),
        }


# ------------------------------------------------------------------ operators around the layer
def _moe_dtype(dt, where: str) -> int:
    import torch
    code = {torch.bfloat16: MOE_BF16, torch.float32: MOE_FP32}.get(dt)
    if code is None:
        raise MoeError(MOE_ERR_DTYPE, where)
    return code


def _check(where, device, t, dtype, shape):
    """t: a contiguous tensor of this dtype and shape on GPU `device` (an index).  A host
    tensor's address must never reach a kernel."""
    if t is None:
        raise MoeError(MOE_ERR_NULL, where)
    if t.dtype is not dtype:
        raise MoeError(MOE_ERR_DTYPE, where)
    if t.shape != shape:
        raise MoeError(MOE_ERR_SHAPE, where)
    if device < 0 or t.get_device() != device or not t.is_contiguous():
        raise MoeError(MOE_ERR_LAYOUT, where)


def _check_rows(where, device, t, dtype, shape) -> int:
    """As _check for a matrix whose rows may lie apart; returns the elements between rows (of a
    single row: at least its length, its stride means nothing)."""
    if t is None:
        raise MoeError(MOE_ERR_NULL, where)
    if t.dtype is not dtype:
        raise MoeError(MOE_ERR_DTYPE, where)
    if t.shape != shape:
        raise MoeError(MOE_ERR_SHAPE, where)
    if device < 0 or t.get_device() != device:
        raise MoeError(MOE_ERR_LAYOUT, where)
    if t.is_contiguous():
        return shape[1]
    if t.stride(1) != 1 and shape[1] > 1:
        raise MoeError(MOE_ERR_LAYOUT, where)
    return t.stride(0) if shape[0] > 1 else shape[1]


def _device(where, t) -> int:
    """The GPU index of a call's first tensor (-1: not on a GPU), which is a matrix."""
    if t is None:
        raise MoeError(MOE_ERR_NULL, where)
    if t.dim() != 2:
        raise MoeError(MOE_ERR_SHAPE, where)
    return t.get_device()


class _Problems(dict):
    """Problem structs by what of them changes from call to call (the sizes): a call of a size
    met before does not build one again.  Nothing writes to a struct once it is made."""

    def __init__(self, make):
        super().__init__()
        self.make = make

    def __missing__(self, key):
        if len(self) >= 256:
            self.clear()
        p = self[key] = self.make(*key)
        return p


def _call(where, device, fn, *args):
    """fn(*args, stream) on torch's current stream of GPU `device`, with that GPU current."""
    import torch
    if device == torch._C._cuda_getDevice():
        st = fn(*args, torch._C._cuda_getCurrentRawStream(device))
    else:
        with torch.cuda.device(device):
            st = fn(*args, torch._C._cuda_getCurrentRawStream(device))
    if st != MOE_OK:
        raise MoeError(st, where)


class _Fixed:
    """An operator whose options are fixed at construction."""

    @property
    def p(self):
        """A copy of the problem struct."""
        return type(self._p).from_buffer_copy(self._p)


class Router(_Fixed):
    """The router's decision on logits [tokens, experts] (torch tensors, FP32 or BF16): the
    table moe_forward_topk and DecodeLayer take, and the gradient back to the logits.
    Holds options only; every buffer is the caller's."""

    def __init__(self, experts, topk, score="softmax", normalize=False, scale=1.0, dtype=None):
        import torch
        self.dtype = dtype or torch.float32
        kind = {"softmax": MOE_ROUTER_SOFTMAX, "sigmoid": MOE_ROUTER_SIGMOID}.get(score, 0)
        self._p = moe_router_problem(0, experts, topk, kind, _moe_dtype(self.dtype, "Router"),
                                     MOE_ROUTER_NORMALIZE if normalize else 0, scale, experts)
        st = moe_router_forward(self._p, None, None, None, None, None)    # no tokens: checks the options
        if st != MOE_OK:
            raise MoeError(st, "Router")
        self.experts, self.topk, q = experts, topk, self._p
        self._problems = _Problems(lambda T, ld: moe_router_problem(
            T, q.experts, q.topk, q.score, q.logits_dtype, q.flags, q.scale, ld))

    def forward(self, logits, top_experts, router_weights, expert_bias=None):
        """Writes top_experts (int32) and router_weights (float32), both [tokens, topk]."""
        import torch
        where = "moe_router_forward"
        dev, T = _device(where, logits), logits.shape[0]
        ld = _check_rows(where, dev, logits, self.dtype, (T, self.experts))
        table = (T, self.topk)
        _check(where, dev, top_experts, torch.int32, table)
        _check(where, dev, router_weights, torch.float32, table)
        if expert_bias is not None:
            _check(where, dev, expert_bias, torch.float32, (self.experts,))
        _call(where, dev, load().moe_router_forward, self._problems[T, ld], logits.data_ptr(), _ptr(expert_bias),
              top_experts.data_ptr(), router_weights.data_ptr())
        return top_experts, router_weights

    def backward(self, logits, top_experts, grad_router_weights, grad_logits):
        """Writes grad_logits [tokens, experts] in the logits' dtype."""
        import torch
        where = "moe_router_backward"
        dev, T = _device(where, logits), logits.shape[0]
        ld = _check_rows(where, dev, logits, self.dtype, (T, self.experts))
        table = (T, self.topk)
        _check(where, dev, top_experts, torch.int32, table)
        _check(where, dev, grad_router_weights, torch.float32, table)
        ld_grad = _check_rows(where, dev, grad_logits, self.dtype, (T, self.experts))
        _call(where, dev, load().moe_router_backward, self._problems[T, ld], logits.data_ptr(),
              top_experts.data_ptr(), grad_router_weights.data_ptr(), grad_logits.data_ptr(), ld_grad)
        return grad_logits


class Norm(_Fixed):
    """Layer norm (kind "layer") or RMS norm ("rms") of rows [rows, cols].  Holds the options
    and the backward's workspace (its size covers any number of rows); two backward calls
    of one Norm must not overlap on the GPU."""

    def __init__(self, cols, kind="layer", eps=1e-5, dtype=None, param_dtype=None, grad_dtype=None, device="cuda"):
        import torch
        self.dtype = dtype or torch.bfloat16
        self.param_dtype = param_dtype or self.dtype
        self.grad_dtype = grad_dtype or torch.float32
        code = {"layer": MOE_NORM_LAYER, "rms": MOE_NORM_RMS}.get(kind, 0)
        self._p = moe_norm_problem(1 << 30, cols, code, _moe_dtype(self.dtype, "Norm"),
                                   _moe_dtype(self.param_dtype, "Norm"), _moe_dtype(self.grad_dtype, "Norm"), 0, eps)
        self.ws_bytes = moe_norm_workspace_bytes(self._p)
        if self.ws_bytes == 0:      # refused: a call without arguments says why
            raise MoeError(moe_norm_forward(self._p, None, None, None, None, None, None, None, None), "Norm")
        self.workspace = torch.empty(self.ws_bytes, dtype=torch.uint8, device=device)
        self.cols, q = cols, self._p
        self._problems = _Problems(lambda rows, flags: moe_norm_problem(
            rows, q.cols, q.kind, q.dtype, q.param_dtype, q.grad_dtype, flags, q.eps))

    def _rows(self, where, device, t, shape):
        ld = _check_rows(where, device, t, self.dtype, shape)
        return moe_rows(t.data_ptr(), ld)

    def forward(self, x, weight, bias, y, stats=None, residual=None, sum=None):
        """y = norm(x) or, with residual, sum = x + residual and y = norm(sum).  stats: float32
        [rows, 2], what backward needs."""
        import torch
        where = "moe_norm_forward"
        dev, shape = _device(where, x), (x.shape[0], self.cols)
        rx, ry = self._rows(where, dev, x, shape), self._rows(where, dev, y, shape)
        rres = None if residual is None else self._rows(where, dev, residual, shape)
        rsum = None if sum is None else self._rows(where, dev, sum, shape)
        cols = (self.cols,)
        _check(where, dev, weight, self.param_dtype, cols)
        if bias is not None:
            _check(where, dev, bias, self.param_dtype, cols)
        if stats is not None:
            _check(where, dev, stats, torch.float32, (shape[0], 2))
        _call(where, dev, load().moe_norm_forward, self._problems[shape[0], 0], rx, rres, weight.data_ptr(),
              _ptr(bias), rsum, ry, _ptr(stats))
        return y

    def backward(self, grad_y, x, weight, stats, grad_x, grad_weight=None, grad_bias=None, grad_sum=None,
                 overwrite=False):
        """x: what was normalised (the forward's sum if it took a residual).  grad_weight and
        grad_bias [cols] are accumulated, or overwritten."""
        import torch
        where = "moe_norm_backward"
        dev, shape = _device(where, x), (x.shape[0], self.cols)
        rx, rdy, rdx = (self._rows(where, dev, t, shape) for t in (x, grad_y, grad_x))
        rgs = None if grad_sum is None else self._rows(where, dev, grad_sum, shape)
        cols = (self.cols,)
        _check(where, dev, weight, self.param_dtype, cols)
        _check(where, dev, stats, torch.float32, (shape[0], 2))
        for g in (grad_weight, grad_bias):
            if g is not None:
                _check(where, dev, g, self.grad_dtype, cols)
        if self.workspace.get_device() != dev:
            raise MoeError(MOE_ERR_WORKSPACE, where)
        _call(where, dev, load().moe_norm_backward,
              self._problems[shape[0], MOE_NORM_OVERWRITE_GRADS if overwrite else 0], rdy, rx, weight.data_ptr(),
              stats.data_ptr(), rgs, rdx, _ptr(grad_weight), _ptr(grad_bias), self.workspace.data_ptr(), self.ws_bytes)
        return grad_x


class DecodeLayer(_Fixed):
    """The layer's forward for a few tokens.  Holds the problem (its `tokens` is the largest
    batch; a call takes any number up to it) and the workspace; two calls of one DecodeLayer
    must not overlap on the GPU."""

    def __init__(self, p: moe_problem, device="cuda"):
        import torch
        self._p = moe_problem.from_buffer_copy(p)
        self.ws_bytes = moe_decode_workspace_bytes(self._p)
        if self.ws_bytes == 0:      # refused: a call without arguments says why
            raise MoeError(moe_forward_decode(self._p, None, None, None, moe_weights(), None, None, 0, None),
                           "moe_decode_workspace_bytes")
        # zeros: the status word before the first call
        self.workspace = torch.zeros(self.ws_bytes, dtype=torch.uint8, device=device)

        def problem_of(tokens):
            q = moe_problem.from_buffer_copy(self._p)
            q.tokens = tokens
            return q
        self.hidden, self.topk = p.hidden, p.topk
        self._problems = _Problems(problem_of)

    def forward(self, hidden, top_experts, router_weights, weights: moe_weights, out):
        import torch
        where = "moe_forward_decode"
        dev, T = _device(where, hidden), hidden.shape[0]
        if T > self._p.tokens:
            raise MoeError(MOE_ERR_SHAPE, where)
        rows, table = (T, self.hidden), (T, self.topk)
        _check(where, dev, hidden, torch.bfloat16, rows)
        _check(where, dev, top_experts, torch.int32, table)
        _check(where, dev, router_weights, torch.float32, table)
        _check(where, dev, out, torch.bfloat16, rows)
        if self.workspace.get_device() != dev:
            raise MoeError(MOE_ERR_WORKSPACE, where)
        _call(where, dev, load().moe_forward_decode, self._problems[T,], hidden.data_ptr(), top_experts.data_ptr(),
              router_weights.data_ptr(), weights, out.data_ptr(), self.workspace.data_ptr(), self.ws_bytes)
        return out

    def status_word(self):
        """The status word of the last call that had tokens, a device int32 [1]: 0 or
        MOE_ERR_ROUTE_INVALID."""
        import torch
        return self.workspace[:4].view(torch.int32)

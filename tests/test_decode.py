"""The forward of a few tokens (moe_forward_decode) against the layer's formula in 64 bits on
the stored weights (MXFP8 decoded, activations unquantised).

Tolerances.  u = 2^-24.  A product of length n is accumulated in FP32 over at most 32 products
inside a matrix instruction, n / 128 steps and 8 partial sums: (40 + n / 128) u of the sum
of its magnitudes.  The SwiGLU passes errors of a and b on with factors of at most
1.1 |b| and |silu(a)| and adds 32 u |h| (exp and reciprocal).  h may be rounded to BF16 (it is held
closer, which test_h_is_not_rounded_to_bf16 checks): each term
w W h of the output is off by at most 2^-8 of itself, independently, so by
Hoeffding's inequality their sum stays within 6 sqrt(sum of squares) 2^-8 except once in 10^7
elements at the largest possible spread (a rounding error's actual spread is 1/sqrt(3) of it).
The output's own rounding is 2^-8 relative."""
import ctypes as C

import numpy as np
import pytest
import torch

import moe_inputs as gen
import moe_megakernel_amd as mk
from oracle import moe_oracle as O

U = 2.0 ** -24
H8 = 2.0 ** -8
TABLE = mk.MOE_FLAG_TOPK_ROUTING


# ------------------------------------------------------------------ CPU: refusals
PTR = 1 << 20


def _weights(p):
    def w(rows, cols, dt, **kw):
        m = lambda c: mk.moe_mat(PTR, rows * c, 0, c)
        if dt == mk.MOE_BF16:
            return mk.weight(dt, rows, cols, m(cols))
        return mk.weight(dt, rows, cols, m(cols), 0, m(cols // 32), m(cols), m(cols))
    H, I, d = p.hidden, p.intermediate, p.routed_dtype
    b = mk.MOE_BF16
    return mk.moe_weights(w(I, H, b), w(I, H, b), w(H, I, b), w(I, H, d), w(I, H, d), w(H, I, d), w(1, H, b))


def _call(p, w=None, x=PTR, top=PTR, rw=PTR, out=PTR, ws=PTR, nbytes=1 << 40):
    return mk.moe_forward_decode(p, x, top, rw, w or _weights(p), out, ws, nbytes, None)


def _p(tokens=4, hidden=256, inter=128, experts=8, topk=2, dt=mk.MOE_BF16, flags=TABLE | mk.MOE_FLAG_HAS_SHARED, L=0.0):
    return mk.problem(tokens, hidden, inter, experts, topk, dt, flags, L)


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=-1), mk.MOE_ERR_SHAPE), (dict(tokens=mk.MOE_DECODE_MAX_TOKENS + 1), mk.MOE_ERR_SHAPE),
    (dict(hidden=130), mk.MOE_ERR_SHAPE), (dict(inter=64), mk.MOE_ERR_SHAPE),
    (dict(inter=mk.MOE_DECODE_MAX_INTERMEDIATE + 128), mk.MOE_ERR_SHAPE), (dict(experts=256), mk.MOE_ERR_SHAPE),
    (dict(topk=9, experts=16), mk.MOE_ERR_SHAPE), (dict(flags=mk.MOE_FLAG_HAS_SHARED), mk.MOE_ERR_UNSUPPORTED),
    (dict(flags=TABLE | mk.MOE_FLAG_RECOMPUTE), mk.MOE_ERR_UNSUPPORTED),
    (dict(flags=TABLE | mk.MOE_FLAG_SHARED_GATE), mk.MOE_ERR_UNSUPPORTED), (dict(flags=TABLE | 64), mk.MOE_ERR_UNSUPPORTED),
    (dict(dt=mk.MOE_FP32), mk.MOE_ERR_DTYPE), (dict(L=float("nan")), mk.MOE_ERR_UNSUPPORTED),
    (dict(L=-1.0), mk.MOE_ERR_UNSUPPORTED)])
def test_bad_problems_are_refused(kw, status):
    p = _p(**kw)
    assert _call(p, _weights(_p())) == status
    assert mk.moe_decode_workspace_bytes(p) == 0


def test_bad_arguments_are_refused():
    p = _p()
    need = mk.moe_decode_workspace_bytes(p)
    assert need > 0
    assert mk.load().moe_forward_decode(None, PTR, PTR, PTR, C.byref(_weights(p)), PTR, PTR, 1 << 40, None) == mk.MOE_ERR_NULL
    assert mk.load().moe_forward_decode(C.byref(p), PTR, PTR, PTR, None, PTR, PTR, 1 << 40, None) == mk.MOE_ERR_NULL
    for k in ("x", "top", "rw", "out"):
        assert _call(p, **{k: None}) == mk.MOE_ERR_NULL
    assert _call(p, ws=None) == mk.MOE_ERR_WORKSPACE
    assert _call(p, nbytes=need - 1) == mk.MOE_ERR_WORKSPACE
    for k in ("x", "out", "ws"):
        assert _call(p, **{k: PTR + 8}) == mk.MOE_ERR_LAYOUT
    for k in ("top", "rw"):
        assert _call(p, **{k: PTR + 2}) == mk.MOE_ERR_LAYOUT
    w = _weights(p)
    w.routed_up.rows = 64
    assert _call(p, w) == mk.MOE_ERR_SHAPE
    w = _weights(p)
    w.shared_down.dtype = mk.MOE_MXFP8_E4M3
    assert _call(p, w) == mk.MOE_ERR_DTYPE
    assert _call(_p(tokens=0), x=None, top=None, rw=None, out=None) == mk.MOE_OK


def test_workspace_serves_smaller_batches():
    """A DecodeLayer of T tokens calls with fewer: their workspace must not be larger."""
    for H, I, E, K in ((128, 2048, 16, 8), (256, 2304, 20, 4), (4096, 1024, 96, 4), (7168, 2048, 64, 6), (512, 128, 255, 1)):
        for dt in (mk.MOE_BF16, mk.MOE_MXFP8_E4M3):
            need = [mk.moe_decode_workspace_bytes(_p(t, H, I, E, K, dt)) for t in range(65)]
            assert all(n > 0 for n in need) and need == sorted(need)


def test_binding_refuses_host_and_mismatched_tensors():
    p = _p()
    layer = mk.DecodeLayer(p, device="cpu")
    x, top, rw = torch.zeros(4, 256, dtype=torch.bfloat16), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    w = _weights(p)
    for args, status in (((x, top, rw, w, x.clone()), mk.MOE_ERR_LAYOUT), ((x.float(), top, rw, w, x.clone()), mk.MOE_ERR_DTYPE),
                         ((torch.zeros(5, 256, dtype=torch.bfloat16), top, rw, w, x.clone()), mk.MOE_ERR_SHAPE),
                         ((x[:, :128], top, rw, w, x.clone()), mk.MOE_ERR_SHAPE),
                         ((x[0, 0], top, rw, w, x.clone()), mk.MOE_ERR_SHAPE),
                         ((None, top, rw, w, x.clone()), mk.MOE_ERR_NULL)):
        with pytest.raises(mk.MoeError) as ei:
            layer.forward(*args)
        assert ei.value.status == status
    with pytest.raises(mk.MoeError) as ei:
        mk.DecodeLayer(_p(tokens=65), device="cpu")
    assert ei.value.status == mk.MOE_ERR_SHAPE
    with pytest.raises(mk.MoeError) as ei:
        mk.DecodeLayer(_p(flags=0), device="cpu")
    assert ei.value.status == mk.MOE_ERR_UNSUPPORTED


# ------------------------------------------------------------------ reference (64 bits)
def clean_table(top, E):
    """The table with invalid entries dropped (out of range, listed again in the row)."""
    out = top.copy()
    for t in range(top.shape[0]):
        seen = set()
        for k in range(top.shape[1]):
            e = int(top[t, k])
            if e < 0 or e >= E or e in seen:
                out[t, k] = -1
            else:
                seen.add(e)
    return out


def reference(x_bits, top, rw, E, W):
    """(out, tolerance without the output's rounding), float64."""
    x = torch.from_numpy(O.bf16_decode(x_bits))
    T, H = x.shape
    top, rw = torch.from_numpy(top), torch.from_numpy(rw).double()
    out, lin, sq = (torch.zeros(T, H, dtype=torch.float64) for _ in range(3))

    def add(t, w, mats):
        wg, wu, wd = (torch.from_numpy(np.ascontiguousarray(m)) for m in mats)
        I = wg.shape[0]
        a, b = x[t] @ wg.T, x[t] @ wu.T
        ea, eb = (((40 + H / 128) * U) * (x[t].abs() @ m.abs().T) for m in (wg, wu))
        L = W.swiglu_limit
        if L > 0:
            a, b = a.clamp(max=L), b.clamp(-L, L)
        s = a * torch.sigmoid(a)
        h = s * b
        eh = 1.1 * b.abs() * ea + s.abs() * eb + 32 * U * h.abs()
        w = w[:, None]
        out.index_add_(0, t, w * (h @ wd.T))
        mag = h.abs() @ wd.abs().T
        lin.index_add_(0, t, w.abs() * (eh @ wd.abs().T + (48 + I / 128 + E) * U * mag))
        sq.index_add_(0, t, w ** 2 * (h ** 2 @ (wd ** 2).T))

    for e in range(E):
        t, k = (top == e).nonzero(as_tuple=True)
        if t.numel():
            add(t, rw[t, k], W.routed(e))
    if W.shared is not None:
        s = torch.ones(T, dtype=torch.float64)
        if W.shared_gate is not None:
            s = torch.sigmoid(x @ torch.from_numpy(W.shared_gate))
        add(torch.arange(T), s, W.shared)
    return out, lin + 6 * H8 * sq.sqrt()


def test_reference_is_the_layer():
    cfg = gen.custom(5, 256, 6, 3, 128, idx=3)
    s1, s2 = gen.shared_weights(cfg)
    routed = gen.routed_all(cfg)
    W = O.Weights.from_bits(128, s1, s2, lambda e: routed[e], "bf16", swiglu_limit=0.5)
    top, rw = table("short", 5, 6, 3, 0)
    out, _ = reference(gen.hidden(cfg), clean_table(top, 6), rw, 6, W)
    want = O.moe_forward_table(gen.hidden(cfg), clean_table(top, 6), rw, 6, W)
    assert np.allclose(out.numpy(), want, rtol=1e-10, atol=1e-12)


# ------------------------------------------------------------------ GPU
def table(kind, T, E, K, seed):
    rng = np.random.default_rng(seed)
    top = np.stack([rng.permutation(E)[:K] for _ in range(T)]).astype(np.int32)
    rw = rng.random((T, K), dtype=np.float32) - 0.25
    if kind == "short":
        top[rng.random((T, K)) < 0.4] = -1
    elif kind == "none":
        top[:] = -1
    elif kind == "one":                       # every token to expert E - 1, the rest to none
        top[:] = -1
        top[:, rng.integers(K)] = E - 1
    elif kind == "invalid":
        top[::3, 0] = E
        top[1::3, 0] = -5
        if K > 1:
            top[2::3, K - 1] = top[2::3, 0]
    rw[top < 0] = np.nan                      # weights at missing routes are not looked at
    return top, rw


def problem(T, H, I, E, K, routed="bf16", layout="single", kind="random", seed=0, **kw):
    from moe_inputs.device import DeviceProblem
    cfg = gen.custom(T, H, E, K, I, routed=routed, layout=layout, backward=False, idx=200 + seed)
    top, rw = table(kind, T, E, K, seed)
    dp = DeviceProblem(cfg, routing_table=(top, rw), **kw)
    dp.decode = mk.DecodeLayer(dp.p)
    dp.decode.workspace.fill_(0xFF)
    W = O.Weights.from_bits(I, dp.np_s1 if dp.shared else None, dp.np_s2 if dp.shared else None,
                            lambda e: dp.np_routed[e], routed, shared_gate=dp.np_gate, swiglu_limit=dp.swiglu_limit)
    return dp, W


def run(dp):
    return dp.decode.forward(dp.x, dp.top, dp.rw, dp.weights, dp.out)


def check(dp, W, out=None):
    top = clean_table(dp.np_top, dp.cfg.experts)
    ref, tol = reference(dp.np_x, top, np.nan_to_num(dp.np_rw), dp.cfg.experts, W)
    got = (dp.out if out is None else out).cpu().double()
    tol = tol + H8 * (ref.abs() + tol)
    bad = (got - ref).abs() > tol
    assert not bool(bad.any()), (int(bad.sum()), float(((got - ref).abs() / tol.clamp(min=1e-30)).max()))
    invalid = bool(((dp.np_top < -1) | (dp.np_top >= dp.cfg.experts)).any()) or bool(
        ((dp.np_top >= 0) & (dp.np_top < dp.cfg.experts) & (top < 0)).any())
    assert int(dp.decode.status_word().cpu()[0]) == (mk.MOE_ERR_ROUTE_INVALID if invalid else 0)


CASES = [
    # T, H, I, E, K, extra
    dict(T=1, H=128, I=128, E=1, K=1),
    dict(T=1, H=256, I=128, E=8, K=2, layout="table"),
    dict(T=2, H=384, I=256, E=5, K=5, gate=True),
    dict(T=3, H=640, I=384, E=9, K=4, kind="short", shared=False),
    dict(T=7, H=1152, I=128, E=255, K=8, layout="table", pad=32),
    dict(T=16, H=256, I=640, E=6, K=3, kind="one"),
    dict(T=17, H=512, I=256, E=4, K=1, limit=0.4, kind="one"),
    dict(T=16, H=128, I=128, E=3, K=2, kind="none", shared=False),
    dict(T=33, H=256, I=128, E=12, K=4, kind="invalid", gate=True),
    dict(T=48, H=384, I=256, E=4, K=4, kind="random", pad=16),
    dict(T=64, H=256, I=128, E=2, K=1, kind="one"),
    dict(T=64, H=512, I=256, E=40, K=8, kind="short", limit=0.4),
    dict(T=31, H=256, I=1024, E=64, K=6, sep=True),
    dict(T=9, H=4224, I=2304, E=3, K=2, limit=1.0),              # two row fragments; more than 16 steps
    dict(T=37, H=4352, I=128, E=4, K=2, layout="table", gate=True),
    dict(T=64, H=128, I=128, E=255, K=8, kind="invalid", shared=False),
    dict(T=2, H=8448, I=128, E=2, K=1),                          # more than 16 steps a wave in the first product
    dict(T=6, H=256, I=128, E=7, K=4, kind="invalid"),           # tables small enough for registers
    dict(T=8, H=256, I=256, E=30, K=4, kind="short", gate=True),
    dict(T=16, H=256, I=128, E=5, K=2, kind="one"),
    dict(T=50, H=256, I=128, E=5, K=4, kind="invalid", limit=0.4),
    dict(T=20, H=128, I=2048, E=16, K=8, kind="short"),          # second product shared by 4 workgroups a column tile
    dict(T=12, H=256, I=2304, E=20, K=4, gate=True),             # by 2
    dict(T=64, H=384, I=1024, E=12, K=6, layout="table", kind="invalid"),
    dict(T=40, H=256, I=1024, E=40, K=2, kind="one", gate=True),  # short rows: a tile a wave, tokens in passes of 32
    dict(T=18, H=1792, I=512, E=10, K=3, limit=0.4),
]


@pytest.mark.gpu
@pytest.mark.parametrize("routed", ["bf16", "mxfp8"])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_matches_formula(gpu_lib, i, routed):
    c = dict(CASES[i])
    kw = dict(shared=c.pop("shared", True), shared_gate=c.pop("gate", False), swiglu_limit=c.pop("limit", 0.0),
              pad_bytes=c.pop("pad", 0), separate_gate_up=c.pop("sep", False))
    dp, W = problem(routed=routed, seed=i, **c, **kw)
    run(dp)
    torch.cuda.synchronize()
    check(dp, W)
    first = dp.out.clone()
    dp.decode.workspace.fill_(0x5A)
    run(dp)
    torch.cuda.synchronize()
    assert torch.equal(dp.out, first)
    if c.get("kind") == "none" and not dp.shared:
        assert bool((dp.out == 0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("routed", ["bf16", "mxfp8"])
def test_full_width(gpu_lib, routed):
    dp, W = problem(5, 4096, 1024, 10, 4, routed=routed, seed=40)
    run(dp)
    torch.cuda.synchronize()
    check(dp, W)


@pytest.mark.gpu
def test_expert_offsets_past_32_bits(gpu_lib):
    """Experts 2.4 GB apart: byte offsets pass 2^32 from the second expert on."""
    dp, W = problem(9, 256, 128, 3, 2, seed=47)
    gap = 1_200_000_000 // 8 * 8
    for name, rows, cols in (("fc1", 256, 256), ("fc2", 256, 128)):
        big = torch.empty(2 * gap + rows * cols, dtype=torch.bfloat16, device="cuda")
        for e in range(3):
            big[e * gap:e * gap + rows * cols].view(rows, cols).copy_(getattr(dp, name)[e])
        dp._keep.append(big)
        m = mk.mat(base=big, expert_stride=gap, ld=cols)
        if name == "fc1":
            dp.weights.routed_gate.data = dp.weights.routed_up.data = m
        else:
            dp.weights.routed_down.data = m
    run(dp)
    torch.cuda.synchronize()
    check(dp, W)


@pytest.mark.gpu
def test_scales_of_all_sizes(gpu_lib):
    """E8M0 bytes far apart beside each other, and all-zero blocks with byte 0 (2^-127)."""
    dp, W = problem(11, 512, 384, 5, 3, routed="mxfp8", seed=48, swiglu_limit=2.0)
    fc1, fc1s, _, _, fc2, fc2s = dp._keep[:6]
    rng = np.random.default_rng(5)
    for key, t, ts in (("fc1", fc1, fc1s), ("fc2", fc2, fc2s)):
        for e in range(5):
            codes, sc = dp.np_routed[e][key], dp.np_routed[e][key + "_s"]
            sc += rng.integers(-12, 3, sc.shape).astype(np.uint8)
            zero = rng.random(sc.shape) < 0.1
            sc[zero] = 0
            codes[np.repeat(zero, 32, axis=1)] = 0
            t[e].copy_(torch.from_numpy(codes))
            ts[e].copy_(torch.from_numpy(sc))
    run(dp)
    torch.cuda.synchronize()
    check(dp, W)


@pytest.mark.gpu
def test_scales_at_the_ends(gpu_lib):
    """E8M0 bytes 0 (2^-127) and 254 (2^127) beside ordinary ones, and 255, which is NaN."""
    dp, W = problem(5, 256, 128, 3, 3, routed="mxfp8", seed=49, shared=False)
    _, _, _, _, fc2, fc2s = dp._keep[:6]
    for e in range(3):
        codes, sc = dp.np_routed[e]["fc2"], dp.np_routed[e]["fc2_s"]
        codes[7], sc[7] = 0x7E, 0                   # 448 * 2^-127
        codes[9], sc[9] = 0, 127
        codes[9, 40], sc[9, 1] = 0x08, 254          # 2^-6 * 2^127
        fc2[e].copy_(torch.from_numpy(codes))
        fc2s[e].copy_(torch.from_numpy(sc))
    run(dp)
    torch.cuda.synchronize()
    check(dp, W)
    want = dp.out.clone()
    fc2s[1][20, 2] = 255
    run(dp)
    torch.cuda.synchronize()
    keep = [c for c in range(256) if c != 20]
    assert torch.equal(dp.out[:, keep], want[:, keep]) and bool(torch.isnan(dp.out[:, 20]).all())


@pytest.mark.gpu
def test_agrees_with_the_training_forward(gpu_lib):
    """BF16: h and the output are rounded as in moe_forward_topk (each within tol and 2^-8 of
    itself); that one also rounds every expert's output, within 2^-8 of it, before they are added."""
    dp, W = problem(40, 512, 256, 12, 3, seed=41, kind="short", shared_gate=True)
    run(dp)
    got = dp.out.double().cpu()
    dp.forward()
    want = dp.out.double().cpu()
    top, rw = clean_table(dp.np_top, 12), np.nan_to_num(dp.np_rw)
    both, tol = reference(dp.np_x, top, rw, 12, W)
    shared = reference(dp.np_x, np.full_like(top, -1), rw, 12, W)[0]
    each = shared.abs()                                # sum of the magnitudes of the experts' terms
    for k in range(3):
        one = np.full_like(top, -1)
        one[:, k] = top[:, k]
        each += (reference(dp.np_x, one, rw, 12, W)[0] - shared).abs()
    assert bool(((got - want).abs() <= 2 * (tol + H8 * (both.abs() + tol)) + H8 * (each + tol)).all())


@pytest.mark.gpu
def test_smaller_batches_of_one_layer(gpu_lib):
    dp, W = problem(24, 256, 128, 8, 2, seed=42)
    run(dp)
    full = dp.out.clone()
    for T in (1, 2, 15, 16, 17, 24):
        out = torch.full_like(dp.out, float("nan"))
        dp.decode.forward(dp.x[:T], dp.top[:T], dp.rw[:T], dp.weights, out[:T])
        torch.cuda.synchronize()
        assert bool(torch.isnan(out[T:]).all())         # rows behind the last token stay
        top = clean_table(dp.np_top[:T], 8)
        ref, tol = reference(dp.np_x[:T], top, dp.np_rw[:T], 8, W)
        assert bool(((out[:T].cpu().double() - ref).abs() <= tol + H8 * (ref.abs() + tol)).all())
    e = dp.x[:0]
    dp.decode.forward(e, dp.top[:0], dp.rw[:0], dp.weights, dp.out[:0])
    torch.cuda.synchronize()
    assert torch.equal(dp.out, full)


@pytest.mark.gpu
@pytest.mark.parametrize("routed", ["bf16", "mxfp8"])
def test_nonfinite_tokens_stay_in_their_row(gpu_lib, routed):
    dp, W = problem(20, 256, 128, 4, 2, routed=routed, seed=43)
    run(dp)
    want = dp.out.clone()
    dp.x[3, 5] = float("nan")
    dp.x[11] = float("inf")
    dp.rw[7, 0] = float("nan")
    run(dp)
    torch.cuda.synchronize()
    keep = [t for t in range(20) if t not in (3, 7, 11)]
    assert torch.equal(dp.out[keep], want[keep])
    assert bool(torch.isnan(dp.out[[3, 7]]).all()) and not bool(torch.isfinite(dp.out[11].float()).any())


@pytest.mark.gpu
def test_graph_replay_and_side_stream(gpu_lib):
    dp, W = problem(19, 384, 256, 16, 4, seed=44, shared_gate=True)
    run(dp)
    torch.cuda.synchronize()
    want = dp.out.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(dp)
    torch.cuda.synchronize()
    assert torch.equal(dp.out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(dp)
    for i in range(3):                                   # new tokens and a new table each time
        top, rw = table("short", 19, 16, 4, 60 + i)
        dp.top.copy_(torch.from_numpy(top))
        dp.rw.copy_(torch.from_numpy(rw))
        dp.x.copy_(torch.randn(19, 384, device="cuda"))
        run(dp)
        torch.cuda.synchronize()
        want = dp.out.clone()
        dp.out.zero_()
        dp.decode.workspace.fill_(0xA5)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(dp.out, want), i


@pytest.mark.gpu
def test_two_layers_on_two_streams(gpu_lib):
    """Calls with distinct workspaces may overlap."""
    a, Wa = problem(9, 256, 128, 8, 2, seed=45)
    b, Wb = problem(21, 256, 256, 8, 2, seed=46, routed="mxfp8")
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        with torch.cuda.stream(s1):
            run(a)
        with torch.cuda.stream(s2):
            run(b)
    torch.cuda.synchronize()
    check(a, Wa)
    check(b, Wb)


def reference_in_two_parts(x_bits, top, rw, E, W):
    """As reference, for an h that is held in two BF16 parts: the upper one leaves at most 2^-8 of h, and
    the lower one's rounding 2^-8 of that.  (Below 2^-118 the lower part runs out of exponents.)"""
    out, tol = reference(x_bits, top, rw, E, W)
    x = torch.from_numpy(O.bf16_decode(x_bits))
    t_top, t_rw = torch.from_numpy(top), torch.from_numpy(rw).double()
    mag, sq = torch.zeros_like(out), torch.zeros_like(out)

    def add(t, w, mats):
        wg, wu, wd = (torch.from_numpy(np.ascontiguousarray(m)) for m in mats)
        a, b = x[t] @ wg.T, x[t] @ wu.T
        if W.swiglu_limit > 0:
            a, b = a.clamp(max=W.swiglu_limit), b.clamp(-W.swiglu_limit, W.swiglu_limit)
        h = a * torch.sigmoid(a) * b
        mag.index_add_(0, t, w.abs()[:, None] * (h.abs() @ wd.abs().T))
        sq.index_add_(0, t, w[:, None] ** 2 * (h ** 2 @ (wd ** 2).T))

    for e in range(E):
        t, k = (t_top == e).nonzero(as_tuple=True)
        if t.numel():
            add(t, t_rw[t, k], W.routed(e))
    if W.shared is not None:
        s = torch.ones(x.shape[0], dtype=torch.float64)
        if W.shared_gate is not None:
            s = torch.sigmoid(x @ torch.from_numpy(W.shared_gate))
        add(torch.arange(x.shape[0]), s, W.shared)
    return out, tol - 6 * H8 * sq.sqrt() + H8 ** 2 * mag


PARTS = [
    dict(T=1, H=256, I=256, E=4, K=2),
    dict(T=8, H=384, I=640, E=3, K=2, kind="one"),
    dict(T=13, H=384, I=256, E=3, K=3, gate=True),               # 9 to 16 tokens an expert
    dict(T=16, H=4224, I=256, E=3, K=2, limit=0.4),              # two row fragments
    dict(T=24, H=256, I=384, E=4, K=2),
    dict(T=30, H=512, I=256, E=2, K=2, kind="short"),            # 17 to 32
    dict(T=64, H=256, I=1024, E=2, K=1, limit=0.4),
    dict(T=64, H=4224, I=256, E=4, K=3),                         # more than 32, two row fragments
    dict(T=64, H=4224, I=384, E=5, K=2, kind="one", shared=False),
    dict(T=64, H=7168, I=128, E=40, K=4, kind="invalid"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("routed", ["bf16", "mxfp8"])
@pytest.mark.parametrize("i", range(len(PARTS)))
def test_h_is_not_rounded_to_bf16(gpu_lib, i, routed):
    """The output is off by FP32 sums and its own rounding only."""
    c = dict(PARTS[i])
    kw = dict(shared=c.pop("shared", True), shared_gate=c.pop("gate", False), swiglu_limit=c.pop("limit", 0.0))
    dp, W = problem(routed=routed, seed=70 + i, **c, **kw)
    run(dp)
    torch.cuda.synchronize()
    top = clean_table(dp.np_top, c["E"])
    ref, tol = reference_in_two_parts(dp.np_x, top, np.nan_to_num(dp.np_rw), c["E"], W)
    tol = tol + H8 * (ref.abs() + tol)
    off = (dp.out.cpu().double() - ref).abs()
    assert bool((off <= tol).all()), (int((off > tol).sum()), float((off / tol.clamp(min=1e-30)).max()))


def test_layer_names_the_status_of_a_refused_problem():
    """The same status as moe_forward_decode returns for the problem."""
    for kw, status in ((dict(inter=mk.MOE_DECODE_MAX_INTERMEDIATE + 128), mk.MOE_ERR_SHAPE), (dict(hidden=130), mk.MOE_ERR_SHAPE),
                       (dict(tokens=-1), mk.MOE_ERR_SHAPE), (dict(topk=9, experts=16), mk.MOE_ERR_SHAPE),
                       (dict(dt=mk.MOE_FP32), mk.MOE_ERR_DTYPE), (dict(L=-1.0), mk.MOE_ERR_UNSUPPORTED),
                       (dict(flags=TABLE | mk.MOE_FLAG_RECOMPUTE), mk.MOE_ERR_UNSUPPORTED)):
        with pytest.raises(mk.MoeError) as ei:
            mk.DecodeLayer(_p(**kw), device="cpu")
        assert ei.value.status == status, kw

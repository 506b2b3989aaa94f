"""The gated feed-forward block, forward and backward, against its formulas in 64 bits.

Tolerances, elementwise.  u = 2^-24, r = 2^-8 (half a step of BF16, relative).  A product's FP32 sum over n
terms is off by at most 2 n u of the sum of magnitudes (one rounding a term, and the matrix unit's own
alignment).  The activation and its derivative come from a hardware exponential and reciprocal: their
argument is off by a few u of itself, |z| <= 40 wherever they are not 0 or 1 to FP32, so they are off by
2^-16 relative.  h, da and db are rounded to BF16 (r), results once more (r, or u in FP32)."""
import math

import pytest
import torch

import moe_megakernel_amd as mk
from tests.test_checkpoint import reference as int8_reference

PTR = 1 << 20
U, R_BF, ACT = 2.0 ** -24, 2.0 ** -8, 2.0 ** -16
BF = torch.bfloat16


# ------------------------------------------------------------------ reference (64 bits)
def act(a, kind):
    """act(a) and its derivative."""
    z, dz = a, torch.ones_like(a)
    if kind == "gelu":
        k = 2 * math.sqrt(2 / math.pi)
        z, dz = k * (a + 0.044715 * a ** 3), k * (1 + 3 * 0.044715 * a ** 2)
    s = torch.sigmoid(z)
    return a * s, s + a * s * (1 - s) * dz


def ref_forward(x, wg, wu, wd, kind):
    """out and a, b, with bounds of what the kernels' out, a and b may be off by before their own rounding."""
    x, wg, wu, wd = (t.double().cpu() for t in (x, wg, wu, wd))
    H, I = x.shape[1], wg.shape[0]
    a, b = x @ wg.t(), x @ wu.t()
    ea, eb = (2 * H * U * (x.abs() @ w.abs().t()) for w in (wg, wu))
    f, d = act(a, kind)
    ef = 1.2 * ea + ACT * f.abs()              # |act'| <= 1.13
    h = f * b
    eh = (ef * b.abs() + f.abs() * eb + ef * eb) * (1 + R_BF) + R_BF * h.abs()
    out = h @ wd.t()
    return out, eh @ wd.abs().t() + 2 * I * U * ((h.abs() + eh) @ wd.abs().t()), a, b, ea, eb


def ref_backward(dy, x, a, b, wg, wu, wd, kind):
    """(gradients of x, gate, up, down; their bounds before the results' rounding) at a, b, x."""
    dy, x, a, b, wg, wu, wd = (t.double().cpu() for t in (dy, x, a, b, wg, wu, wd))
    T, H = x.shape
    I = wg.shape[0]
    dh, edh = dy @ wd, 2 * H * U * (dy.abs() @ wd.abs())
    f, d = act(a, kind)
    ad, af = ACT * (1 + a.abs()), ACT * f.abs()   # the derivative cancels around its zeros: absolute
    da, db, h = dh * b * d, dh * f, f * b
    eda = (edh * b.abs() * (d.abs() + ad) + dh.abs() * b.abs() * ad) * (1 + R_BF) + R_BF * da.abs()
    edb = (edh * (f.abs() + af) + dh.abs() * af) * (1 + R_BF) + R_BF * db.abs()
    eh = af * b.abs() * (1 + R_BF) + R_BF * h.abs()
    dx = da @ wg + db @ wu
    edx = eda @ wg.abs() + edb @ wu.abs()
    edx = edx + 4 * I * U * (da.abs() @ wg.abs() + db.abs() @ wu.abs() + edx)
    out, bounds = [dx], [edx]
    for g, e, other in ((da, eda, x), (db, edb, x)):
        out.append(g.t() @ other)
        m = e.t() @ other.abs()
        bounds.append(m + 2 * T * U * (g.abs().t() @ other.abs() + m))
    out.append(dy.t() @ h)
    m = dy.abs().t() @ eh
    bounds.append(m + 2 * T * U * (dy.abs().t() @ h.abs() + m))
    return out, bounds


def near(got, ref, bound, half):
    got = got.detach().cpu().double()
    assert torch.isfinite(got).all()
    bad = (got - ref).abs() > bound + half * (ref.abs() + bound)
    assert not bad.any(), (int(bad.sum()), float(((got - ref).abs() - bound).max()))


def test_reference_gradient_matches_autograd_and_differences():
    g = torch.Generator().manual_seed(0)
    rn = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)
    for kind in ("silu", "gelu"):
        x, wg, wu, wd = rn(3, 5).requires_grad_(), rn(4, 5).requires_grad_(), rn(4, 5).requires_grad_(), rn(5, 4).requires_grad_()
        dy = rn(3, 5)
        out, _, a, b, _, _ = ref_forward(x, wg, wu, wd, kind)
        (out * dy).sum().backward()
        got, _ = ref_backward(dy, x.detach(), a.detach(), b.detach(), wg.detach(), wu.detach(), wd.detach(), kind)
        for v, t in zip(got, (x, wg, wu, wd)):
            assert torch.allclose(v, t.grad, rtol=1e-10, atol=1e-12)
        step = 1e-6
        for t, v in ((x, got[0]), (wg, got[1]), (wd, got[3])):
            f = []
            for sign in (1, -1):
                u = [q.detach().clone() for q in (x, wg, wu, wd)]
                next(q for q, o in zip(u, (x, wg, wu, wd)) if o is t)[1, 2] += sign * step
                f.append(float((ref_forward(*u, kind)[0] * dy).sum()))
            assert abs((f[0] - f[1]) / (2 * step) - float(v[1, 2])) < 1e-6
        torch_act = torch.nn.functional.silu(a) if kind == "silu" else torch.nn.functional.gelu(a, approximate="tanh")
        assert torch.allclose(act(a, kind)[0], torch_act, rtol=1e-12)


# ------------------------------------------------------------------ CPU: refusals
def problem(tokens=8, hidden=64, inter=128, activation=mk.MOE_FFN_SILU, saved=mk.MOE_BF16, grad=mk.MOE_FP32, flags=0):
    return mk.moe_ffn_problem(tokens, hidden, inter, activation, saved, grad, flags)


H0, I0 = (PTR, 64), (PTR, 128)       # matrices of 64 and 128 columns


def fwd(p, x=H0, gate=H0, up=H0, down=I0, out=H0, saved=PTR, ws=PTR, n=1 << 40):
    r = lambda m: None if m is None else mk.moe_rows(*m)
    return mk.moe_ffn_forward(p, r(x), r(gate), r(up), r(down), r(out), saved, ws, n, None)


def bwd(p, dy=H0, x=H0, gate=H0, up=H0, down=I0, saved=PTR, gx=H0, gg=H0, gu=H0, gd=I0, ws=PTR, n=1 << 40):
    r = lambda m: None if m is None else mk.moe_rows(*m)
    return mk.moe_ffn_backward(p, r(dy), r(x), r(gate), r(up), r(down), saved, r(gx), r(gg), r(gu), r(gd), ws, n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=-1), mk.MOE_ERR_SHAPE), (dict(tokens=(1 << 24) + 1), mk.MOE_ERR_SHAPE), (dict(hidden=32), mk.MOE_ERR_SHAPE),
    (dict(hidden=100), mk.MOE_ERR_SHAPE), (dict(inter=0), mk.MOE_ERR_SHAPE), (dict(inter=(1 << 17) + 64), mk.MOE_ERR_SHAPE),
    (dict(tokens=1 << 24, hidden=1 << 17), mk.MOE_ERR_SHAPE), (dict(activation=0), mk.MOE_ERR_UNSUPPORTED),
    (dict(activation=3), mk.MOE_ERR_UNSUPPORTED), (dict(saved=mk.MOE_FP32), mk.MOE_ERR_DTYPE),
    (dict(saved=mk.MOE_MXFP8_E4M3), mk.MOE_ERR_DTYPE), (dict(grad=0), mk.MOE_ERR_DTYPE),
    (dict(grad=mk.MOE_MXINT8), mk.MOE_ERR_DTYPE), (dict(flags=2), mk.MOE_ERR_UNSUPPORTED)])
def test_bad_problems_are_refused(kw, status):
    p = problem(**kw)
    assert fwd(p) == status and bwd(p) == status
    assert mk.moe_ffn_saved_bytes(p) == 0
    assert mk.moe_ffn_workspace_bytes(p, False) == 0 and mk.moe_ffn_workspace_bytes(p, True) == 0
    with pytest.raises(mk.MoeError) as e:
        mk.moe_ffn_saved_view(p)
    assert e.value.status == status


def test_bad_arguments_are_refused():
    p = problem()
    assert mk.load().moe_ffn_forward(None, *[None] * 5, None, None, 0, None) == mk.MOE_ERR_NULL
    for kw in (dict(x=None), dict(gate=None), dict(up=(0, 64)), dict(down=None), dict(out=None)):
        assert fwd(p, **kw) == mk.MOE_ERR_NULL, kw
    for kw in (dict(x=(PTR, 56)), dict(x=(PTR, 68)), dict(gate=(PTR + 8, 64)), dict(up=(PTR, 60)), dict(down=(PTR, 64)),
               dict(out=(PTR + 2, 64)), dict(saved=PTR + 8), dict(ws=PTR + 4)):
        assert fwd(p, **kw) == mk.MOE_ERR_LAYOUT, kw
    need = mk.moe_ffn_workspace_bytes(p, False)
    assert fwd(p, ws=None) == fwd(p, n=need - 1) == fwd(p, saved=None) == mk.MOE_ERR_WORKSPACE
    assert fwd(problem(saved=0), saved=PTR) == mk.MOE_ERR_WORKSPACE          # nothing is kept, yet a place for it
    for kw in (dict(dy=None), dict(x=None), dict(gate=None), dict(down=(0, 128)), dict(gg=None), dict(gu=None),
               dict(gx=None, gg=None, gu=None, gd=None)):
        assert bwd(p, **kw) == mk.MOE_ERR_NULL, kw
    for kw in (dict(dy=(PTR, 63)), dict(gx=(PTR + 8, 64)), dict(gg=(PTR, 66)), dict(gd=(PTR, 64)), dict(saved=PTR + 1),
               dict(ws=PTR + 8)):
        assert bwd(p, **kw) == mk.MOE_ERR_LAYOUT, kw
    assert bwd(problem(grad=mk.MOE_BF16), gg=(PTR, 68)) == mk.MOE_ERR_LAYOUT  # 16-byte pieces of BF16
    need = mk.moe_ffn_workspace_bytes(p, True)
    assert bwd(p, ws=None) == bwd(p, n=need - 1) == bwd(p, saved=None) == mk.MOE_ERR_WORKSPACE
    assert bwd(problem(saved=0)) == mk.MOE_ERR_UNSUPPORTED                    # the forward kept nothing
    assert bwd(problem(saved=mk.MOE_MXINT8)) == mk.MOE_ERR_UNSUPPORTED        # x is in `saved`
    # no tokens: nothing to do, whatever else is missing
    e = problem(tokens=0)
    assert fwd(e, x=None, gate=None, out=None, saved=None, ws=None, n=0) == mk.MOE_OK
    assert bwd(e, dy=None, x=None, gate=None, up=None, down=None, saved=None, gx=None, ws=None, n=0) == mk.MOE_OK


def test_sizes_serve_fewer_tokens_and_views_are_ordered():
    for saved in (mk.MOE_BF16, mk.MOE_MXINT8):
        last = (0, 0, 0)
        for T in (0, 1, 2, 63, 64, 65, 1000, 5000):
            p = problem(T, 320, 576, saved=saved)
            now = (mk.moe_ffn_saved_bytes(p), mk.moe_ffn_workspace_bytes(p, False), mk.moe_ffn_workspace_bytes(p, True))
            assert all(n >= l and n > 0 for n, l in zip(now, last))
            last = now
    v = mk.moe_ffn_saved_view(problem(100, 320, 576, saved=mk.MOE_MXINT8))
    assert v.ab == 0 < v.ab_scales < v.x < v.x_scales and all(o % 256 == 0 for o in (v.ab_scales, v.x, v.x_scales))
    # 8 bits and a byte each 32 of 2 I + H values, against 16 bits of 2 I (x stays elsewhere)
    assert mk.moe_ffn_saved_bytes(problem(4096, 4096, 1024, saved=mk.MOE_MXINT8)) == 4096 * (2048 + 4096) * 33 // 32
    assert mk.moe_ffn_saved_bytes(problem(4096, 4096, 1024)) == 4096 * 2048 * 2
    assert mk.moe_ffn_saved_bytes(problem(saved=0)) == 0 == mk.moe_ffn_workspace_bytes(problem(saved=0), True)


def test_binding_refuses_host_and_mismatched_tensors():
    op = mk.FeedForward(64, 128, 8, saved="bf16", device="cpu")
    z = lambda *s, dt=BF: torch.zeros(*s, dtype=dt)
    x, g, d = z(4, 64), z(128, 64), z(64, 128)
    sv = z(op.saved_bytes(4), dt=torch.uint8)

    def status(f, *a, **k):
        with pytest.raises(mk.MoeError) as e:
            f(*a, **k)
        return e.value.status
    assert status(op.forward, x, g, g, d, z(4, 64), sv) == mk.MOE_ERR_LAYOUT            # host memory
    assert status(op.forward, None, g, g, d, z(4, 64), sv) == mk.MOE_ERR_NULL
    assert status(op.forward, z(9, 64), g, g, d, z(9, 64), sv) == mk.MOE_ERR_SHAPE      # more than `tokens`
    assert status(op.forward, z(64), g, g, d, z(64), sv) == mk.MOE_ERR_SHAPE
    assert status(op.backward, x, x, g, g, d, sv, x) == mk.MOE_ERR_LAYOUT
    assert status(mk.FeedForward, 100, 128, 8) == mk.MOE_ERR_SHAPE
    assert status(mk.FeedForward, 64, 128, 8, activation="relu") == mk.MOE_ERR_UNSUPPORTED
    assert status(mk.FeedForward, 64, 128, 8, saved="fp8") == mk.MOE_ERR_DTYPE
    assert status(mk.FeedForward, 64, 128, 8, grad_dtype=torch.float16) == mk.MOE_ERR_DTYPE
    before = op._problems[4, 0].activation
    op.p.activation = mk.MOE_FFN_GELU
    assert op._problems[5, 0].activation == before


# ------------------------------------------------------------------ GPU
def rows(t, pad=0):
    """t with `pad` elements of NaN after each row."""
    buf = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device="cuda")
    buf[:, :t.shape[1]] = t
    return buf[:, :t.shape[1]], buf


def inputs(T, H, I, pad=0, seed=0):
    g = torch.Generator().manual_seed(1000 * seed + T + H + I)
    rn = lambda *s: torch.randn(*s, generator=g)
    w = [(rn(I, H) / H ** 0.5), (rn(I, H) / H ** 0.5), (rn(H, I) / I ** 0.5)]
    return [rows((t * s).to(BF), pad)[0] for t, s in ((rn(T, H), 1.0), (w[0], 2.0), (w[1], 1.0), (w[2], 1.0), (rn(T, H), 1.0))]


def kept(op, saved, T):
    """a, b (and x) as the backward sees them, 64 bits."""
    v = {k: t.cpu() for k, t in op.saved_views(saved, T).items()}
    if op.saved == "bf16":
        return v["ab"].double(), None
    wide = lambda q, s: q.double() * (2.0 ** (s.double() - 133)).repeat_interleave(32, 1)
    return wide(v["ab"], v["ab_scales"]), wide(v["x"], v["x_scales"])


SIZES = [(1, 64, 64), (2, 128, 320), (63, 192, 64), (64, 64, 192), (65, 320, 128), (100, 448, 576), (129, 256, 1024),
         (257, 576, 320), (300, 1088, 704)]


@pytest.mark.gpu
@pytest.mark.parametrize("saved", ["none", "bf16", "int8"])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("T,H,I", SIZES + [(7, 4096, 256), (17, 256, 4096), (33, 1024, 1024), (777, 512, 512)])
def test_forward_matches_formula(gpu_lib, T, H, I, kind, saved):
    pad = 8 * (T % 3)
    x, wg, wu, wd, _ = inputs(T, H, I, pad)
    op = mk.FeedForward(H, I, T, kind, saved)
    out, obuf = rows(torch.zeros(T, H, dtype=BF), pad)
    sv = None if saved == "none" else torch.zeros(op.saved_bytes(T), dtype=torch.uint8, device="cuda")
    op.forward(x, wg, wu, wd, out, sv)
    torch.cuda.synchronize()
    ref, bound, a, b, ea, eb = ref_forward(x, wg, wu, wd, kind)
    near(out, ref, bound, R_BF)
    assert torch.isnan(obuf[:, H:]).all()
    if saved == "none":
        return
    ab, xs = kept(op, sv, T)
    ref, err = torch.cat([a, b], 1), torch.cat([ea, eb], 1)
    if saved == "bf16":
        near(ab, ref, err, R_BF)
    else:       # half a step, and a step is less than 2 / 127 of the block's largest
        top = (ref.abs() + err).view(T, -1, 32).amax(-1).repeat_interleave(32, 1)
        near(ab, ref, err + top / 127, 0.0)
        assert torch.equal(xs, int8_reference(x)[2])


@pytest.mark.gpu
@pytest.mark.parametrize("saved", ["bf16", "int8"])
@pytest.mark.parametrize("gdt", [BF, torch.float32])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("T,H,I", SIZES)
def test_backward_matches_formula(gpu_lib, T, H, I, kind, saved, gdt):
    pad = 8 * (T % 3)
    x, wg, wu, wd, dy = inputs(T, H, I, pad)
    op = mk.FeedForward(H, I, T, kind, saved, grad_dtype=gdt)
    sv = torch.zeros(op.saved_bytes(T), dtype=torch.uint8, device="cuda")
    out = torch.empty(T, H, dtype=BF, device="cuda")
    op.forward(x, wg, wu, wd, out, sv)
    before = sv.clone()
    g = [rows(torch.full(s, 3.0, dtype=dt), pad) for s, dt in (((T, H), BF), ((I, H), gdt), ((I, H), gdt), ((H, I), gdt))]
    op.backward(dy, x if saved == "bf16" else None, wg, wu, wd, sv, *[t for t, _ in g], overwrite=True)
    torch.cuda.synchronize()
    assert torch.equal(sv, before)
    ab, xs = kept(op, sv, T)
    ref, bound = ref_backward(dy, x if xs is None else xs, ab[:, :I], ab[:, I:], wg, wu, wd, kind)
    for (got, buf), r, e in zip(g, ref, bound):
        near(got, r, e, R_BF if got.dtype == BF else U)
        assert torch.isnan(buf[:, got.shape[1]:]).all()
    # added to what is there: a BF16 gradient gets the rounded contribution, one rounding more
    start = [torch.randn(t.shape, generator=torch.Generator().manual_seed(i)).to(t.dtype).cuda() for i, (t, _) in enumerate(g)]
    acc = [rows(s, pad)[0] for s in start]
    op.backward(dy, x if saved == "bf16" else None, wg, wu, wd, sv, *acc)
    torch.cuda.synchronize()
    assert torch.equal(acc[0], g[0][0])
    for a, s, (w, _) in list(zip(acc, start, g))[1:]:
        assert torch.equal(a, (s.float() + w.float()).to(a.dtype))


@pytest.mark.gpu
def test_gradients_that_are_not_asked_for(gpu_lib):
    T, H, I = 70, 128, 192
    x, wg, wu, wd, dy = inputs(T, H, I)
    for saved in ("bf16", "int8"):
        op = mk.FeedForward(H, I, T, saved=saved)
        sv = torch.zeros(op.saved_bytes(T), dtype=torch.uint8, device="cuda")
        op.forward(x, wg, wu, wd, torch.empty_like(x), sv)
        xx = x if saved == "bf16" else None
        z = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt, device="cuda")
        full = [z(T, H, dt=BF), z(I, H), z(I, H), z(H, I)]
        op.backward(dy, xx, wg, wu, wd, sv, *full, overwrite=True)
        for use in ((0,), (1, 2), (3,), (0, 3), (1, 2, 3)):
            part = [torch.zeros_like(t) if i in use else None for i, t in enumerate(full)]
            op.backward(dy, xx, wg, wu, wd, sv, *part, overwrite=True)
            for i in use:
                assert torch.equal(part[i], full[i]), (saved, use)


@pytest.mark.gpu
def test_no_tokens(gpu_lib):
    H, I = 128, 64
    op = mk.FeedForward(H, I, 4, saved="bf16", grad_dtype=BF)
    e, w, d = (torch.ones(*s, dtype=BF, device="cuda") for s in ((0, H), (I, H), (H, I)))
    sv = torch.zeros(op.saved_bytes(0), dtype=torch.uint8, device="cuda")
    op.forward(e, w, w, d, e, sv)
    g = [torch.ones_like(t) for t in (w, w, d)]
    op.backward(e, e, w, w, d, sv, e, *g)
    assert all((t == 1).all() for t in g)
    op.backward(e, e, w, w, d, sv, e, *g, overwrite=True)
    assert all((t == 0).all() for t in g)


@pytest.mark.gpu
@pytest.mark.parametrize("T,saved", [(20, "none"), (60, "none"), (300, "none"), (300, "bf16"), (300, "int8")])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_nonfinite_rows_stay_in_their_row(gpu_lib, T, saved, bad):
    H, I = 192, 320
    x, wg, wu, wd, dy = inputs(T, H, I)
    op = mk.FeedForward(H, I, T, saved=saved)
    sv = None if saved == "none" else torch.zeros(op.saved_bytes(T), dtype=torch.uint8, device="cuda")
    want, got = torch.empty_like(x), torch.empty_like(x)
    op.forward(x, wg, wu, wd, want, sv)
    x2 = x.clone()
    x2[11, 3] = bad
    op.forward(x2, wg, wu, wd, got, sv)
    keep = torch.arange(T) != 11
    assert torch.equal(got[keep], want[keep])
    assert torch.isnan(got[11]).any()
    if saved != "none":
        dx = torch.empty_like(x)
        op.backward(dy, x2 if saved == "bf16" else None, wg, wu, wd, sv, dx)
        assert torch.isfinite(dx[keep]).all() and torch.isnan(dx[11]).any()


@pytest.mark.gpu
def test_gate_and_up_as_views_of_one_tensor(gpu_lib):
    T, H, I = 130, 256, 192
    x, wg, wu, wd, dy = inputs(T, H, I)
    both = torch.cat([wg, wu]).contiguous()
    gboth = torch.zeros(2 * I, H, device="cuda")
    g1, g2 = torch.zeros(I, H, device="cuda"), torch.zeros(I, H, device="cuda")
    op = mk.FeedForward(H, I, T, saved="bf16")
    sv = torch.zeros(op.saved_bytes(T), dtype=torch.uint8, device="cuda")
    o1, o2 = torch.empty_like(x), torch.empty_like(x)
    op.forward(x, wg, wu, wd, o1, sv)
    op.backward(dy, x, wg, wu, wd, sv, None, g1, g2)
    op.forward(x, both[:I], both[I:], wd, o2, sv)
    op.backward(dy, x, both[:I], both[I:], wd, sv, None, gboth[:I], gboth[I:])
    assert torch.equal(o1, o2) and torch.equal(torch.cat([g1, g2]), gboth)


@pytest.mark.gpu
def test_rows_do_not_depend_on_the_batch(gpu_lib):
    """Padding rows change nothing: the same rows in a larger batch of the same kernels give the same bits,
    and one workspace and `saved` of the largest batch serve smaller ones."""
    H, I = 320, 448
    x, wg, wu, wd, dy = inputs(700, H, I)
    op = mk.FeedForward(H, I, 700, saved="int8")
    sv = torch.zeros(op.saved_bytes(700), dtype=torch.uint8, device="cuda")
    full, dfull = torch.empty_like(x), torch.empty_like(x)
    op.forward(x, wg, wu, wd, full, sv)
    op.backward(dy, None, wg, wu, wd, sv, dfull)
    for T in (1, 255, 300):
        out, dx = torch.empty(T, H, dtype=BF, device="cuda"), torch.empty(T, H, dtype=BF, device="cuda")
        op.forward(x[:T], wg, wu, wd, out, sv)
        op.backward(dy[:T], None, wg, wu, wd, sv, dx)
        near(out, full[:T].double().cpu(), torch.zeros(T, H), 2 * R_BF)
        top = dfull[:T].abs().amax().double().cpu()
        assert ((dx - dfull[:T]).abs().double().cpu() <= 2 * R_BF * (dfull[:T].abs().double().cpu() + top)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T,saved", [(9, "none"), (300, "bf16"), (300, "int8")])
def test_captured_on_a_side_stream_and_repeatable(gpu_lib, T, saved):
    H, I = 256, 576
    x, wg, wu, wd, dy = inputs(T, H, I)
    op = mk.FeedForward(H, I, T, "gelu", saved, grad_dtype=torch.float32)
    sv = None if saved == "none" else torch.zeros(op.saved_bytes(T), dtype=torch.uint8, device="cuda")
    out, dx = torch.empty_like(x), torch.empty_like(x)
    g = [torch.zeros(*s, device="cuda") for s in ((I, H), (I, H), (H, I))]

    def step():
        op.forward(x, wg, wu, wd, out, sv)
        if saved != "none":
            op.backward(dy, x if saved == "bf16" else None, wg, wu, wd, sv, dx, *g, overwrite=True)
    outs = [out] + ([dx] + g if saved != "none" else [])
    step()
    torch.cuda.synchronize()
    first = [t.clone() for t in outs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(outs, first))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        x.copy_(torch.randn(T, H, device="cuda"))
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in outs]
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), i


@pytest.mark.gpu
@pytest.mark.parametrize("saved", ["bf16", "int8"])
def test_row_offsets_past_32_bits(gpu_lib, saved):
    T, H, I = 70000, 64, 16384                                 # 2 T I = 2.3e9 values kept
    x, wg, wu, wd, dy = inputs(40, H, I)
    big, bdy = torch.zeros(T, H, dtype=BF, device="cuda"), torch.zeros(T, H, dtype=BF, device="cuda")
    big[-40:], bdy[-40:] = x, dy
    op = mk.FeedForward(H, I, T, saved=saved)
    sv = torch.empty(op.saved_bytes(T), dtype=torch.uint8, device="cuda")
    out, dx, gd = torch.empty_like(big), torch.empty_like(big), torch.empty(H, I, device="cuda")
    op.forward(big, wg, wu, wd, out, sv)
    op.backward(bdy, big if saved == "bf16" else None, wg, wu, wd, sv, dx, grad_down=gd, overwrite=True)
    torch.cuda.synchronize()
    ref, bound, _, _, _, _ = ref_forward(x, wg, wu, wd, "silu")
    near(out[-40:], ref, bound, R_BF)
    v = op.saved_views(sv, T)
    if saved == "bf16":
        ab, xs = v["ab"][-40:].cpu().double(), x
    else:
        wide = lambda q, s: q[-40:].cpu().double() * (2.0 ** (s[-40:].cpu().double() - 133)).repeat_interleave(32, 1)
        ab, xs = wide(v["ab"], v["ab_scales"]), wide(v["x"], v["x_scales"])
    ref, bound = ref_backward(dy, xs, ab[:, :I], ab[:, I:], wg, wu, wd, "silu")
    near(dx[-40:], ref[0], bound[0], R_BF)
    near(gd, ref[3], bound[3], U)
    assert not out[:-40].any() and not dx[:-40].any()


@pytest.mark.gpu
@pytest.mark.parametrize("saved", ["bf16", "int8"])
def test_block_in_a_row_with_the_norm(gpu_lib, saved):
    """norm (with the residual stream) -> block, forward and backward, as a dense layer of the model uses
    them, the norm's input on a checkpoint of its own with 8 bits; against autograd in 64 bits.
    Tolerance: the layer's own bound for BF16 weights, 2e-2 of the largest value, with 8-bit checkpoints
    six roundings of 2^-7 of a block's largest more (x, a, b, the norm's input, and their products)."""
    T, H, I = 200, 256, 512
    x, wg, wu, wd, dy = inputs(T, H, I)
    g = torch.Generator().manual_seed(5)
    res, w = torch.randn(T, H, generator=g).to(BF).cuda(), (1 + 0.1 * torch.randn(H, generator=g)).to(BF).cuda()
    norm, op = mk.Norm(H, kind="rms"), mk.FeedForward(H, I, T, saved=saved)
    s, hid, out = (torch.empty(T, H, dtype=BF, device="cuda") for _ in range(3))
    stats = torch.empty(T, 2, device="cuda")
    sv = torch.zeros(op.saved_bytes(T), dtype=torch.uint8, device="cuda")
    norm.forward(x, w, None, hid, stats, residual=res, sum=s)
    op.forward(hid, wg, wu, wd, out, sv)
    s64 = s.double().cpu()
    if saved == "int8":
        ck = mk.Checkpoint()
        codes = torch.empty(T, H, dtype=torch.int8, device="cuda")
        scales = torch.empty(T, H // 32, dtype=torch.uint8, device="cuda")
        ck.store(s, codes, scales)
        ck.load(codes, scales, s)
    dhid, ds = torch.empty_like(hid), torch.empty_like(hid)
    grads = [torch.zeros(*k, device="cuda") for k in ((I, H), (I, H), (H, I))]
    op.backward(dy, hid if saved == "bf16" else None, wg, wu, wd, sv, dhid, *grads)
    dw = torch.zeros(H, device="cuda")
    norm.backward(dhid, s, w, stats, ds, dw, None, grad_sum=dy)
    torch.cuda.synchronize()
    leaves = [t.double().cpu().requires_grad_() for t in (wg, wu, wd, w)] + [s64.requires_grad_()]
    h64 = s64 / torch.sqrt((s64 ** 2).mean(1, keepdim=True) + 1e-5) * leaves[3]
    o64 = (torch.nn.functional.silu(h64 @ leaves[0].t()) * (h64 @ leaves[1].t())) @ leaves[2].t()
    ((o64 + s64) * dy.double().cpu()).sum().backward()
    tol = 2e-2 + (6 * 2.0 ** -7 if saved == "int8" else 0)
    for got, ref in zip([out, ds, dw] + grads, [o64.detach(), s64.grad, leaves[3].grad] + [t.grad for t in leaves[:3]]):
        err = (got.double().cpu() - ref).abs().max() / ref.abs().max()
        assert err <= tol, float(err)


@pytest.mark.gpu
def test_shared_expert_run_by_the_caller(gpu_lib):
    """Routed-only layer plus the block on the shared expert's weights is the layer with its shared expert."""
    import moe_inputs as gen
    from moe_inputs.device import DeviceProblem
    cfg = gen.custom(300, 256, 8, 2, 128, idx=33)
    both, routed = DeviceProblem(cfg), DeviceProblem(cfg, shared=False)
    both.forward()
    routed.forward()
    I, H = cfg.inter, cfg.hidden
    s1, s2 = both.s1, both.s2
    op = mk.FeedForward(H, I, 300)
    out = torch.empty(300, H, dtype=BF, device="cuda")
    op.forward(both.x, s1[:I], s1[I:], s2, out)
    torch.cuda.synchronize()
    got, ref = routed.out.double() + out.double(), both.out.double()
    assert float((got - ref).abs().max() / ref.abs().max()) <= 2e-2


def test_strides_past_the_limit_are_refused():
    far = mk.MOE_FFN_MAX_LD + 64
    for name in ("x", "gate", "up", "down", "out"):
        assert fwd(problem(), **{name: (PTR, far)}) == mk.MOE_ERR_LAYOUT, name
    for name in ("dy", "x", "gate", "up", "down", "gx", "gg", "gu", "gd"):
        assert bwd(problem(), **{name: (PTR, far)}) == mk.MOE_ERR_LAYOUT, name


# Enough tiles for every CU, few k: the sizes where the products go in larger tiles (up and dh; down and dx; the weights' gradients).
WIDE = [(1101, 64, 8256), (1101, 8256, 64), (70, 3200, 3264), (967, 64, 5440)]


@pytest.mark.gpu
@pytest.mark.parametrize("saved", ["bf16", "int8"])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("T,H,I", WIDE)
def test_wide_forward_matches_formula(gpu_lib, T, H, I, kind, saved):
    test_forward_matches_formula(gpu_lib, T, H, I, kind, saved)


@pytest.mark.gpu
@pytest.mark.parametrize("gdt", [BF, torch.float32])
@pytest.mark.parametrize("T,H,I", WIDE)
def test_wide_backward_matches_formula(gpu_lib, T, H, I, gdt):
    test_backward_matches_formula(gpu_lib, T, H, I, "gelu" if gdt == BF else "silu", "bf16", gdt)


# Few tiles, long contractions: split ones, in tiles of 128 columns (up, dh; down, dx; the weights' gradients) ...
SPLIT = [(67, 1152, 64), (76, 64, 1088), (965, 64, 64), (300, 1024, 704)]
# ... and in larger ones (up; down and dx; dx; dh; up)
SPLIT_WIDE = [(257, 1536, 5568), (1043, 3648, 1856), (129, 3392, 6144), (663, 1536, 5504), (387, 2880, 5504)]


@pytest.mark.gpu
@pytest.mark.parametrize("saved", ["bf16", "int8"])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("T,H,I", SPLIT)
def test_split_forward_matches_formula(gpu_lib, T, H, I, kind, saved):
    test_forward_matches_formula(gpu_lib, T, H, I, kind, saved)


@pytest.mark.gpu
@pytest.mark.parametrize("saved", ["bf16", "int8"])
@pytest.mark.parametrize("gdt", [BF, torch.float32])
@pytest.mark.parametrize("T,H,I", SPLIT)
def test_split_backward_matches_formula(gpu_lib, T, H, I, saved, gdt):
    test_backward_matches_formula(gpu_lib, T, H, I, "silu" if gdt == BF else "gelu", saved, gdt)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,I", SPLIT_WIDE)
def test_split_wide_block_matches_formula(gpu_lib, T, H, I):
    test_forward_matches_formula(gpu_lib, T, H, I, "gelu", "int8")
    test_backward_matches_formula(gpu_lib, T, H, I, "silu", "bf16", torch.float32)


@pytest.mark.gpu
def test_split_gradients_accumulate_repeat_and_capture(gpu_lib):
    """Gradients added to what is there, the same bits in every run, and a captured forward and backward whose
    replays share a workspace with eager calls."""
    T, H, I = 1500, 128, 192
    x, wg, wu, wd, dy = inputs(T, H, I)
    op = mk.FeedForward(H, I, T, "silu", "bf16", grad_dtype=torch.float32)
    sv = torch.zeros(op.saved_bytes(T), dtype=torch.uint8, device="cuda")
    out, dx = torch.empty(T, H, dtype=BF, device="cuda"), torch.empty(T, H, dtype=BF, device="cuda")
    g = [torch.zeros(*s, device="cuda") for s in ((I, H), (I, H), (H, I))]

    def step():
        op.forward(x, wg, wu, wd, out, sv)
        op.backward(dy, x, wg, wu, wd, sv, dx, *g)

    step()
    torch.cuda.synchronize()
    first = [t.clone() for t in [out, dx] + g]
    step()
    torch.cuda.synchronize()
    for t, f in zip([out, dx], first):
        assert torch.equal(t, f)
    for t, f in zip(g, first[2:]):
        assert torch.equal(t, f + f)
    for t in g:
        t.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n in range(1, 4):
        out.zero_(), dx.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for t, f in zip([out, dx], first):
            assert torch.equal(t, f)
        other = torch.empty_like(out)
        op.forward(x, wg, wu, wd, other, sv)             # eager work between the replays, in the same workspace
        torch.cuda.synchronize()
        assert torch.equal(other, first[0])
        want = first[2:]
        total = [f.clone() for f in want]
        for _ in range(n - 1):
            total = [t + f for t, f in zip(total, want)]
        for t, f in zip(g, total):
            assert torch.equal(t, f)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,I", [(16, 192, 4160), (32, 192, 4160), (24, 8256, 64), (48, 192, 2112), (33, 4160, 64), (64, 4160, 2112),
                                   (49, 64, 64), (40, 320, 192)])
def test_few_tokens_of_wide_blocks_match_formula(gpu_lib, T, H, I):
    test_forward_matches_formula(gpu_lib, T, H, I, "silu", "none")
    test_forward_matches_formula(gpu_lib, T, H, I, "gelu", "none")


# Every product in every tile, whole and split: 192 x 256 tiles (down, dx; up; dh), 256 x 256 (down, dx; dh), split 192 x 256 (dh;
# down; up), split 256 x 256 (dh; down; dx; up; the weights' gradients).
TILES = [(1031, 7296, 64), (527, 64, 6592), (1706, 768, 6976), (1729, 6528, 64), (1959, 832, 6272), (527, 2112, 6784),
         (536, 6656, 1984), (259, 1792, 5632), (771, 2432, 4800), (680, 5440, 1920), (673, 5440, 960), (391, 1984, 4224),
         (1965, 448, 4224), (2059, 4160, 960)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,I", TILES)
def test_tiles_match_formula(gpu_lib, T, H, I):
    test_forward_matches_formula(gpu_lib, T, H, I, "silu", "bf16")
    test_backward_matches_formula(gpu_lib, T, H, I, "gelu", "int8" if T % 2 else "bf16", BF)


@pytest.mark.gpu
@pytest.mark.parametrize("saved", ["bf16", "int8"])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_saturated_activations_have_finite_gradients(gpu_lib, kind, saved):
    """Pre-activations of +-2^76, whose square is past FP32: act' is 1 or 0.  Every value is a power of two, so
    the results are exact."""
    T, H, I = 70, 64, 64
    sign = torch.tensor([1.0, -1.0]).repeat(I // 2)[:, None]
    x = torch.full((T, H), 2.0 ** 40).to(BF).cuda()
    wg = (sign * torch.full((I, H), 2.0 ** 30)).to(BF).cuda()
    wu = torch.full((I, H), 2.0 ** -46).to(BF).cuda()
    wd = torch.full((H, I), 2.0 ** -6).to(BF).cuda()
    dy = torch.ones(T, H).to(BF).cuda()
    op = mk.FeedForward(H, I, T, kind, saved, grad_dtype=torch.float32)
    sv = torch.zeros(op.saved_bytes(T), dtype=torch.uint8, device="cuda")
    out, dx = torch.empty(T, H, dtype=BF, device="cuda"), torch.empty(T, H, dtype=BF, device="cuda")
    gg, gu, gd = torch.empty(I, H, device="cuda"), torch.empty(I, H, device="cuda"), torch.empty(H, I, device="cuda")
    op.forward(x, wg, wu, wd, out, sv)
    op.backward(dy, x if saved == "bf16" else None, wg, wu, wd, sv, dx, gg, gu, gd, overwrite=True)
    torch.cuda.synchronize()
    on = (sign > 0).float()                                   # a = 2^76 or -2^76, b = 1, dh = 1
    assert torch.equal(out.cpu(), torch.full((T, H), 2.0 ** 75).to(BF))          # 32 times 2^76 2^-6
    assert torch.equal(dx.cpu(), torch.full((T, H), 2.0 ** 36).to(BF))           # 32 times (2^30 + 2^76 2^-46)
    assert torch.equal(gg.cpu(), (on * (T * 2.0 ** 40)).expand(I, H))            # da = 1 or 0
    assert torch.equal(gu.cpu(), (on * (T * 2.0 ** 116)).expand(I, H))           # db = 2^76 or 0
    assert torch.equal(gd.cpu(), (on * (T * 2.0 ** 76)).t().expand(H, I))


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,I", [(16, 192, 4160), (24, 8256, 64), (33, 4160, 64), (48, 192, 2112), (64, 4160, 2112)])
def test_few_tokens_keep_their_pre_activations(gpu_lib, T, H, I):
    test_forward_matches_formula(gpu_lib, T, H, I, "gelu", "bf16")
    test_backward_matches_formula(gpu_lib, T, H, I, "silu", "bf16", torch.float32)

"""Every kernel of the feed-forward block over many tokens that a call can choose, against the formulas in 64 bits: each product
in each of its tiles, whole and in parts, with each activation, each form of what is kept and each kind of weight gradient.

SIZES are held against the library's own choice (moe_ffn_plan_view): a combination that none of them takes any more is an
error on the CPU.  Tolerances as in tests/test_feed_forward.py; the 64-bit sums are formed on the GPU."""
import itertools

import pytest
import torch

import moe_megakernel_amd as mk
from tests.test_checkpoint import reference as int8_reference
from tests.test_feed_forward import ACT, BF, R_BF, U, act, inputs, kept, problem, rows

KEEP = {"none": 0, "bf16": mk.MOE_BF16, "int8": mk.MOE_MXINT8}
SIZES = [(2718, 3200, 768), (523, 2368, 3456), (3083, 4032, 64), (2526, 2496, 1600), (1425, 3392, 3712), (3214, 1216, 1088),
         (2752, 832, 4608), (3555, 1792, 2432), (776, 4736, 1984)]
ALL_TILES, TWO_TILES = [(128, 128), (192, 256), (256, 256)], [(128, 128), (256, 256)]
GRADS = list(itertools.product((BF, torch.float32), (False, True)))          # type, overwritten


def cuts(T, H, I):
    """What the calls of these sizes run: (product, option, tile, in parts)."""
    out = set()
    at = lambda c: ((c.rows, c.cols), c.parts > 1)
    for name, keep in KEEP.items():
        p = mk.moe_ffn_plan_view(problem(T, H, I, saved=keep))
        out |= {("up", name, *at(p.up)), ("down", None, *at(p.down))}
        if keep:
            out |= {("dh", name, *at(p.dh)), ("dx", None, *at(p.dx))}
    for dt, over in GRADS:
        p = mk.moe_ffn_plan_view(problem(T, H, I, grad=mk.MOE_BF16 if dt is BF else mk.MOE_FP32, flags=int(over)))
        out |= {(n, (dt, over), *at(getattr(p, n))) for n in ("wgrad_down", "wgrad_up")}
    return out


def test_sizes_take_every_tile_whole_and_in_parts():
    want = set()
    for n, options, tiles in (("up", KEEP, ALL_TILES), ("down", [None], ALL_TILES), ("dh", ["bf16", "int8"], ALL_TILES),
                              ("dx", [None], ALL_TILES), ("wgrad_down", GRADS, TWO_TILES), ("wgrad_up", GRADS, TWO_TILES)):
        want |= set(itertools.product([n], options, tiles, (False, True)))
    got = set().union(*[cuts(*s) for s in SIZES])
    assert want <= got, sorted(map(str, want - got))
    assert got <= want, sorted(map(str, got - want))                         # a new tile needs its sizes here


def test_plans_of_few_tokens_of_none_and_refusals():
    zero = lambda c: (c.rows, c.cols, c.parts) == (0, 0, 0)
    for T, parts in ((1, False), (16, False), (17, True), (64, True)):
        for keep in (0, mk.MOE_BF16):
            p = mk.moe_ffn_plan_view(problem(T, 1024, 4096, saved=keep))
            assert (p.up.rows, p.up.cols, p.up.parts) == (0, 0, 1)
            assert (p.down.rows, p.down.cols) == (0, 0) and (p.down.parts > 1) == parts
            assert zero(p.dh) == zero(p.dx) == zero(p.wgrad_down) == zero(p.wgrad_up) == (keep == 0)
    assert mk.moe_ffn_plan_view(problem(64, 1024, 4096, saved=mk.MOE_MXINT8)).up.rows > 0
    p = mk.moe_ffn_plan_view(problem(0))
    assert all(zero(getattr(p, n)) for n, _ in p._fields_)
    with pytest.raises(mk.MoeError) as e:
        mk.moe_ffn_plan_view(problem(hidden=100))
    assert e.value.status == mk.MOE_ERR_SHAPE
    lib = mk.load()
    assert lib.moe_ffn_plan_view(None, mk.moe_ffn_plan()) == mk.MOE_ERR_NULL == lib.moe_ffn_plan_view(problem(), None)


def test_workspace_holds_the_parts():
    """The sums of a product in parts, FP32 [parts][rows][columns], and what lies beside them."""
    for T, H, I in SIZES + [(17, 64, 2048), (64, 4096, 2048), (64, 64, 131072), (40, 1024, 16384), (65, 64, 64), (1, 64, 64),
                            (100, 131072, 64), (100, 64, 131072), (1000, 64, 64), (100000, 64, 64)]:
        for keep in KEEP.values():
            p = problem(T, H, I, saved=keep)
            v, f, b = mk.moe_ffn_plan_view(p), mk.moe_ffn_workspace_bytes(p, False), mk.moe_ffn_workspace_bytes(p, True)
            sums = lambda c, m, n: 4 * c.parts * m * n if c.parts > 1 else 0
            h = 2 * T * I * (2 if v.up.rows == 0 else 1)
            assert f >= h + max(sums(v.up, T, 2 * I), sums(v.down, T, H))
            if keep:
                x = 2 * T * H if keep == mk.MOE_MXINT8 else 0
                assert b >= 6 * T * I + x + max(sums(v.dh, T, I), sums(v.dx, T, H), sums(v.wgrad_down, H, I), sums(v.wgrad_up, 2 * I, H))


# ------------------------------------------------------------------ 64 bits, on the GPU
def near(got, ref, bound, half):
    got = got.double()
    assert torch.isfinite(got).all()
    bad = (got - ref).abs() > bound + half * (ref.abs() + bound)
    assert not bad.any(), (int(bad.sum()), float(((got - ref).abs() - bound).max()))


def forward64(x, wg, wu, wd, kind):
    H, I = x.shape[1], wg.shape[0]
    a, b = x @ wg.t(), x @ wu.t()
    ea, eb = (2 * H * U * (x.abs() @ w.abs().t()) for w in (wg, wu))
    f, _ = act(a, kind)
    ef = 1.2 * ea + ACT * f.abs()
    h = f * b
    eh = (ef * b.abs() + f.abs() * eb + ef * eb) * (1 + R_BF) + R_BF * h.abs()
    return h @ wd.t(), eh @ wd.abs().t() + 2 * I * U * ((h.abs() + eh) @ wd.abs().t()), torch.cat([a, b], 1), torch.cat([ea, eb], 1)


def backward64(dy, x, a, b, wg, wu, wd, kind):
    T, H = x.shape
    I = wg.shape[0]
    dh, edh = dy @ wd, 2 * H * U * (dy.abs() @ wd.abs())
    f, d = act(a, kind)
    ad, af = ACT * (1 + a.abs()), ACT * f.abs()
    da, db, h = dh * b * d, dh * f, f * b
    eda = (edh * b.abs() * (d.abs() + ad) + dh.abs() * b.abs() * ad) * (1 + R_BF) + R_BF * da.abs()
    edb = (edh * (f.abs() + af) + dh.abs() * af) * (1 + R_BF) + R_BF * db.abs()
    eh = af * b.abs() * (1 + R_BF) + R_BF * h.abs()
    edx = eda @ wg.abs() + edb @ wu.abs()
    edx = edx + 4 * I * U * (da.abs() @ wg.abs() + db.abs() @ wu.abs() + edx)
    out = [(da @ wg + db @ wu, edx)]
    for g, e, other, eo in ((da, eda, x, None), (db, edb, x, None), (dy, None, h, eh)):
        m = e.t() @ other.abs() if eo is None else g.abs().t() @ eo
        out.append((g.t() @ other, m + 2 * T * U * (g.abs().t() @ other.abs() + m)))
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("saved", list(KEEP))
@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("T,H,I", SIZES)
def test_every_kernel_matches_formula(gpu_lib, T, H, I, kind, saved):
    x, wg, wu, wd, dy = inputs(T, H, I)
    x64, wg64, wu64, wd64, dy64 = (t.double() for t in (x, wg, wu, wd, dy))
    op = mk.FeedForward(H, I, T, kind, saved)
    op.workspace.fill_(0xff)                                                 # NaN, were it read
    sv = None if saved == "none" else torch.full((op.saved_bytes(T),), 0xff, dtype=torch.uint8, device="cuda")
    out, obuf = rows(torch.zeros(T, H, dtype=BF), 8)
    op.forward(x, wg, wu, wd, out, sv)
    ref, bound, ab64, eab = forward64(x64, wg64, wu64, wd64, kind)
    near(out, ref, bound, R_BF)
    assert torch.isnan(obuf[:, H:]).all()
    if saved == "none":
        return
    if saved == "bf16":
        ab, xs = op.saved_views(sv, T)["ab"].double(), x64
        near(ab, ab64, eab, R_BF)
    else:
        ab, xs = (t.cuda() for t in kept(op, sv, T))                          # decoded on the CPU, whose powers of two are exact
        top = (ab64.abs() + eab).view(T, -1, 32).amax(-1).repeat_interleave(32, 1)
        near(ab, ab64, eab + top / 127, 0.0)
        assert torch.equal(xs.cpu(), int8_reference(x)[2])
    ref = backward64(dy64, xs, ab[:, :I], ab[:, I:], wg64, wu64, wd64, kind)
    before = sv.clone()
    for gdt, over in GRADS:
        op = mk.FeedForward(H, I, T, kind, saved, grad_dtype=gdt)
        op.workspace.fill_(0xff)
        start = [torch.randn(*s, device="cuda").to(gdt) for s in ((I, H), (I, H), (H, I))]
        got = [rows(t, 8) for t in [torch.zeros(T, H, dtype=BF)] + start]
        op.backward(dy, x if saved == "bf16" else None, wg, wu, wd, sv, *[t for t, _ in got], overwrite=over)
        near(got[0][0], *ref[0], R_BF)
        for (t, _), s, (r, e) in zip(got[1:], start, ref[1:]):
            half = R_BF if gdt is BF else U
            if over:
                near(t, r, e, half)
            else:                     # in BF16 the contribution is rounded before it is added
                s = s.double()
                near(t, r + s, e + (half * (r.abs() + e) if gdt is BF else 0.0), half)
        assert all(torch.isnan(buf[:, t.shape[1]:]).all() for t, buf in got)
    assert torch.equal(sv, before)

"""Layer norm and RMS norm, forward and backward, against the formulas in 64 bits.

Tolerances.  u = 2^-24 is half a step of FP32.  A row sum runs over at most 16 elements a
thread, 6 steps across the wave and 16 waves, so a mean of terms t is off by at most
38 u mean|t|; with the rounding of each term 40 u.  The forward centres twice, so its mean
is off by 40 u mean|d| <= 40 u / rstd and (x - mean) rstd by 40 u + 3 u |xh| plus rstd's own
45 u |xh|: 64 u (1 + |xh|) |w| + 2 u |y| covers it.  The backward's stats are inputs, xh is off by
3 u |xh| and the two means by 44 u: 64 u of the sum of magnitudes.  Results stored in BF16
add half a step, 2^-8 relative.  Column sums add rows in at most rows / 256 + 64 steps."""
import ctypes as C

import pytest
import torch

import moe_megakernel_amd as mk

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}


# ------------------------------------------------------------------ reference (64 bits)
def ref_forward(x, w, b, kind, eps):
    x, w = x.double(), w.double()
    mu = x.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(x[:, :1])
    rstd = 1.0 / torch.sqrt(((x - mu) ** 2).mean(1, keepdim=True) + eps)
    xh = (x - mu) * rstd
    y = xh * w + (0 if b is None else b.double())
    return y, xh, mu, rstd


def ref_backward(dy, x, w, stats, kind, gsum):
    dy, w, st = dy.double(), w.double(), stats.double()
    rstd = st[:, 1:]
    xh = (x.double() - st[:, :1]) * rstd
    g = dy * w
    m1 = g.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(rstd)
    m2 = (g * xh).mean(1, keepdim=True)
    dx = rstd * (g - m1 - xh * m2) + (0 if gsum is None else gsum.double())
    mag = rstd * (g.abs() + g.abs().mean(1, keepdim=True) + xh.abs() * (g * xh).abs().mean(1, keepdim=True))
    if gsum is not None:
        mag = mag + gsum.double().abs()
    return dx, mag, dy * xh


def padded(t, pad, offset=0):
    """t with rows `pad` elements longer, starting `offset` elements into its storage; the rest
    NaN, so that reading it shows and writing it can be seen."""
    R, N = t.shape
    buf = torch.full((R * (N + pad) + offset,), float("nan"), dtype=t.dtype, device=t.device)
    v = buf[offset:].view(R, N + pad)[:, :N]
    v.copy_(t)
    return v, buf


def untouched(view, buf, offset=0):
    """Every element of buf outside the view is still NaN."""
    R, N = view.shape
    pad = buf[offset:].view(R, -1)[:, N:]
    return bool(torch.isnan(buf[:offset]).all()) and bool(torch.isnan(pad).all())


# ------------------------------------------------------------------ CPU: the reference itself
def test_reference_gradient_matches_autograd_and_differences():
    g = torch.Generator().manual_seed(0)
    for kind in ("layer", "rms"):
        x = torch.randn(3, 7, generator=g, dtype=torch.float64, requires_grad=True)
        w = torch.randn(7, generator=g, dtype=torch.float64, requires_grad=True)
        b = torch.randn(7, generator=g, dtype=torch.float64, requires_grad=True)
        dy = torch.randn(3, 7, generator=g, dtype=torch.float64)
        y, _, mu, rstd = ref_forward(x, w, b, kind, 1e-5)
        (y * dy).sum().backward()
        stats = torch.cat([mu, rstd], 1).detach()
        dx, _, terms = ref_backward(dy, x.detach(), w.detach(), stats, kind, None)
        assert torch.allclose(dx, x.grad, rtol=1e-10, atol=1e-12)
        assert torch.allclose(terms.sum(0), w.grad, rtol=1e-10, atol=1e-12)
        assert torch.allclose(dy.sum(0), b.grad, rtol=1e-12)
        h = 1e-6
        for i in ((0, 0), (1, 3), (2, 6)):
            xp, xm = x.detach().clone(), x.detach().clone()
            xp[i] += h
            xm[i] -= h
            f = lambda q: float((ref_forward(q, w.detach(), b.detach(), kind, 1e-5)[0] * dy).sum())
            assert abs((f(xp) - f(xm)) / (2 * h) - float(dx[i])) < 1e-7


# ------------------------------------------------------------------ CPU: refusals
def _problem(rows=4, cols=64, kind=mk.MOE_NORM_LAYER, dtype=mk.MOE_BF16, param=mk.MOE_BF16, grad=mk.MOE_FP32,
             flags=0, eps=1e-5):
    return mk.moe_norm_problem(rows, cols, kind, dtype, param, grad, flags, eps)


PTR = 1 << 20     # 16-byte aligned; refused calls never touch it


def _fwd(p, x=(PTR, 64), res=None, w=PTR, b=None, sum=None, y=(PTR, 64), stats=None):
    r = lambda v: None if v is None else mk.moe_rows(*v)
    return mk.moe_norm_forward(p, r(x), r(res), w, b, r(sum), r(y), stats, None)


def _bwd(p, dy=(PTR, 64), x=(PTR, 64), w=PTR, stats=PTR, gsum=None, dx=(PTR, 64), gw=PTR, gb=None, ws=PTR,
         nbytes=1 << 40):
    r = lambda v: None if v is None else mk.moe_rows(*v)
    return mk.moe_norm_backward(p, r(dy), r(x), w, stats, r(gsum), r(dx), gw, gb, ws, nbytes, None)


BAD_PROBLEMS = [
    (dict(rows=-1), mk.MOE_ERR_SHAPE), (dict(rows=(1 << 30) + 1), mk.MOE_ERR_SHAPE), (dict(cols=0), mk.MOE_ERR_SHAPE),
    (dict(cols=mk.MOE_NORM_MAX_COLS + 1), mk.MOE_ERR_SHAPE), (dict(kind=0), mk.MOE_ERR_UNSUPPORTED),
    (dict(kind=3), mk.MOE_ERR_UNSUPPORTED), (dict(dtype=mk.MOE_MXFP8_E4M3), mk.MOE_ERR_DTYPE),
    (dict(param=0), mk.MOE_ERR_DTYPE), (dict(grad=7), mk.MOE_ERR_DTYPE), (dict(flags=2), mk.MOE_ERR_UNSUPPORTED),
    (dict(eps=-1e-9), mk.MOE_ERR_UNSUPPORTED), (dict(eps=float("nan")), mk.MOE_ERR_UNSUPPORTED),
    (dict(eps=float("inf")), mk.MOE_ERR_UNSUPPORTED),
]


@pytest.mark.parametrize("kw,status", BAD_PROBLEMS)
def test_bad_problems_are_refused(kw, status):
    p = _problem(**kw)
    assert _fwd(p) == status
    assert _bwd(p) == status
    assert mk.moe_norm_workspace_bytes(p) == 0


def test_bad_arguments_are_refused():
    p = _problem()
    assert mk.load().moe_norm_forward(None, None, None, None, None, None, None, None, None) == mk.MOE_ERR_NULL
    assert _fwd(p, x=None) == mk.MOE_ERR_NULL
    assert _fwd(p, x=(0, 64)) == mk.MOE_ERR_NULL
    assert _fwd(p, y=None) == mk.MOE_ERR_NULL
    assert _fwd(p, w=None) == mk.MOE_ERR_NULL
    assert _fwd(p, x=(PTR, 63)) == mk.MOE_ERR_LAYOUT
    assert _fwd(p, x=(PTR + 1, 64)) == mk.MOE_ERR_LAYOUT
    assert _fwd(p, y=(PTR, 0)) == mk.MOE_ERR_LAYOUT
    assert _fwd(p, res=(PTR, 64)) == mk.MOE_ERR_NULL            # residual without sum
    assert _fwd(p, sum=(PTR, 64)) == mk.MOE_ERR_LAYOUT          # sum without residual
    assert _fwd(p, res=(PTR, 64), sum=(PTR, 8)) == mk.MOE_ERR_LAYOUT
    assert _fwd(p, res=(PTR, 64), sum=(2 * PTR, 64), y=(2 * PTR, 64)) == mk.MOE_ERR_LAYOUT
    assert _fwd(p, w=PTR + 1) == mk.MOE_ERR_LAYOUT
    assert _fwd(p, b=PTR + 1) == mk.MOE_ERR_LAYOUT
    assert _fwd(p, stats=PTR + 4) == mk.MOE_ERR_LAYOUT
    assert _bwd(p, dy=None) == mk.MOE_ERR_NULL
    assert _bwd(p, dx=None) == mk.MOE_ERR_NULL
    assert _bwd(p, stats=None) == mk.MOE_ERR_NULL
    assert _bwd(p, gsum=(PTR, 8)) == mk.MOE_ERR_LAYOUT
    assert _bwd(p, gw=PTR + 2) == mk.MOE_ERR_LAYOUT
    assert _bwd(p, ws=None) == mk.MOE_ERR_WORKSPACE
    assert _bwd(p, nbytes=mk.moe_norm_workspace_bytes(p) - 1) == mk.MOE_ERR_WORKSPACE
    assert _bwd(p, ws=PTR + 8) == mk.MOE_ERR_LAYOUT
    assert _fwd(_problem(rows=0)) == mk.MOE_OK                  # nothing to do, nothing launched
    assert _fwd(_problem(rows=0), x=(0, 64), y=(0, 64)) == mk.MOE_OK


def test_workspace_does_not_grow_with_rows():
    big = mk.moe_norm_workspace_bytes(_problem(rows=1 << 30, cols=4096))
    assert big == mk.moe_norm_workspace_bytes(_problem(rows=1 << 20, cols=4096))
    for rows in (1, 2, 17, 1023, 4097):
        assert 0 < mk.moe_norm_workspace_bytes(_problem(rows=rows, cols=4096)) <= big


def test_workspace_serves_smaller_batches():
    """A workspace sized for some rows takes a call with fewer of them."""
    for cols in (1, 96, 1000, 1024, 2055, 4096, 7168, 8200, 16384):
        for dtype in (mk.MOE_BF16, mk.MOE_FP32):
            need = [mk.moe_norm_workspace_bytes(_problem(rows=r, cols=cols, dtype=dtype)) for r in
                    [*range(1100), 2047, 2048, 2049, 5000, 1 << 15, 1 << 20, 1 << 30]]
            assert all(n > 0 for n in need) and need == sorted(need), (cols, dtype)


def test_binding_refuses_host_and_mismatched_tensors():
    n = mk.Norm(64, device="cpu")
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.ones(64, dtype=torch.bfloat16)
    for args, status in (((x, w, None, x.clone()), mk.MOE_ERR_LAYOUT),               # host memory
                         ((x.float(), w, None, x.clone()), mk.MOE_ERR_DTYPE),
                         ((x[:, :32], w, None, x.clone()), mk.MOE_ERR_SHAPE),
                         ((x[0], w, None, x.clone()), mk.MOE_ERR_SHAPE),
                         ((None, w, None, x.clone()), mk.MOE_ERR_NULL)):
        with pytest.raises(mk.MoeError) as ei:
            n.forward(*args)
        assert ei.value.status == status
    for kw, status in ((dict(cols=0), mk.MOE_ERR_SHAPE), (dict(cols=64, kind="batch"), mk.MOE_ERR_UNSUPPORTED),
                       (dict(cols=64, dtype=torch.float16), mk.MOE_ERR_DTYPE)):
        with pytest.raises(mk.MoeError) as ei:
            mk.Norm(device="cpu", **kw)
        assert ei.value.status == status


# ------------------------------------------------------------------ GPU
def make(R, N, dtype, pdtype, seed=0, offset=0.0):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)
    x = (rn(R, N) * torch.exp(0.5 * rn(R, 1)) + 0.3 * rn(R, 1) + offset).to(dtype)
    return (x, (1 + 0.2 * rn(N)).to(pdtype), (0.3 * rn(N)).to(pdtype), rn(R, N).to(dtype), rn(R, N).to(dtype))


def check_forward(x, w, b, y, stats, kind, eps=1e-5):
    ref, xh, mu, rstd = ref_forward(x, w, b, kind, eps)
    tol = 64 * U * (1 + xh.abs()) * w.double().abs() + 2 * U * ref.abs()
    if b is not None:
        tol = tol + U * b.double().abs()
    tol = tol + HALF[y.dtype] * (ref.abs() + tol)
    assert bool(((y.double() - ref).abs() <= tol).all())
    if stats is not None:
        d = (x.double() - mu).abs().mean(1, keepdim=True)
        assert bool(((stats[:, :1].double() - mu).abs() <= 48 * U * d + 2 * U * mu.abs()).all())
        assert bool(((stats[:, 1:].double() / rstd - 1).abs() <= 64 * U).all())


def check_backward(dy, x, w, stats, kind, gsum, dx, dw, db):
    ref, mag, terms = ref_backward(dy, x, w, stats, kind, gsum)
    tol = 64 * U * mag
    tol = tol + HALF[dx.dtype] * (ref.abs() + tol)
    assert bool(((dx.double() - ref).abs() <= tol).all())
    steps = (x.shape[0] // 256 + 68) * U
    if dw is not None:
        assert bool(((dw.double() - terms.sum(0)).abs() <= steps * terms.abs().sum(0) + 1e-30).all())
    if db is not None:
        assert bool(((db.double() - dy.double().sum(0)).abs() <= steps * dy.double().abs().sum(0) + 1e-30).all())


BF, F32 = torch.bfloat16, torch.float32
SIZES = [(1, 1), (1, 8), (3, 2), (5, 7), (1, 4096), (2, 63), (17, 64), (33, 65), (16, 1024), (17, 1032), (9, 1023),
         (300, 128), (1025, 384), (7, 7168), (40, 260), (3, 12300), (513, 4096), (3, 16384), (4, 16383), (2, 8200), (260, 2055),
         (77, 200), (600, 256), (129, 249), (2000, 100), (20000, 72),                   # rows that share a wave
         (50, 134), (9, 4095), (65, 1038), (6, 14), (300, 4098)]                    # a last piece of 2, 4, 6 and 3 elements


def _run_forward(n, x, w, b, res, kind, pad, offset):
    dev = "cuda"
    R, N = x.shape
    xv, xb = padded(x.to(dev), pad, offset)
    yv, yb = padded(torch.zeros(R, N, dtype=x.dtype, device=dev), pad, offset)
    stats = torch.full((R, 2), float("nan"), device=dev)
    rv = sv = None
    if res is not None:
        rv, _ = padded(res.to(dev), pad, offset)
        sv, sb = padded(torch.zeros(R, N, dtype=x.dtype, device=dev), pad, offset)
    n.forward(xv, w.to(dev), None if b is None else b.to(dev), yv, stats, residual=rv, sum=sv)
    torch.cuda.synchronize()
    assert untouched(yv, yb, offset) and (sv is None or untouched(sv, sb, offset))
    return yv.cpu(), stats.cpu(), None if sv is None else sv.cpu()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dtype,pdtype", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
def test_forward_matches_formula(gpu_lib, kind, dtype, pdtype):
    for i, (R, N) in enumerate(SIZES):
        x, w, b, res, _ = make(R, N, dtype, pdtype, seed=i)
        n = mk.Norm(N, kind=kind, dtype=dtype, param_dtype=pdtype)
        pad, offset = [(0, 0), (8, 0), (3, 0), (8, 8), (0, 1)][i % 5]
        y, stats, _ = _run_forward(n, x, w, b if i % 2 else None, None, kind, pad, offset)
        check_forward(x, w, b if i % 2 else None, y, stats, kind)
        y, stats, s = _run_forward(n, x, w, b, res, kind, pad, offset)
        assert torch.equal(s, (x.float() + res.float()).to(dtype)), (R, N)
        check_forward(s, w, b, y, stats, kind)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dtype,pdtype", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
def test_backward_matches_formula(gpu_lib, kind, dtype, pdtype):
    dev = "cuda"
    for i, (R, N) in enumerate(SIZES):
        x, w, _, dy, gs = make(R, N, dtype, pdtype, seed=100 + i)
        pad, offset = [(0, 0), (8, 0), (3, 0), (8, 8), (0, 1)][i % 5]
        gs = gs if i % 2 else None
        _, _, mu, rstd = ref_forward(x, w, None, kind, 1e-5)
        stats = torch.cat([mu, rstd], 1).float()
        n = mk.Norm(N, kind=kind, dtype=dtype, param_dtype=pdtype)
        xv, dyv = padded(x.to(dev), pad, offset)[0], padded(dy.to(dev), pad, offset)[0]
        gsv = None if gs is None else padded(gs.to(dev), pad, offset)[0]
        dxv, dxb = padded(torch.zeros(R, N, dtype=dtype, device=dev), pad, offset)
        for want in ("wb", "w", "b", ""):
            dw = torch.full((N,), float("nan"), device=dev) if "w" in want else None
            db = torch.full((N,), float("nan"), device=dev) if "b" in want else None
            n.backward(dyv, xv, w.to(dev), stats.to(dev), dxv, dw, db, grad_sum=gsv, overwrite=True)
            torch.cuda.synchronize()
            assert untouched(dxv, dxb, offset)
            check_backward(dy, x, w, stats, kind, gs, dxv.cpu(), *(None if t is None else t.cpu() for t in (dw, db)))
            dxv.zero_()


@pytest.mark.gpu
@pytest.mark.parametrize("gdtype", [F32, BF])
def test_main_grad_accumulates(gpu_lib, gdtype):
    R, N = 700, 1024
    x, w, _, dy, _ = make(R, N, BF, BF, seed=5)
    x, w, dy = x.cuda(), w.cuda(), dy.cuda()
    n = mk.Norm(N, grad_dtype=gdtype)
    y, dx, stats = torch.empty_like(x), torch.empty_like(x), torch.empty(R, 2, device="cuda")
    n.forward(x, w, None, y, stats)
    fresh = [torch.empty(N, dtype=gdtype, device="cuda") for _ in range(2)]
    n.backward(dy, x, w, stats, dx, *fresh, overwrite=True)
    start = [torch.linspace(-50, 50, N, device="cuda").to(gdtype) for _ in range(2)]
    acc = [s.clone() for s in start]
    for _ in range(2):
        n.backward(dy, x, w, stats, dx, *acc)
    for f, s, a in zip(fresh, start, acc):      # one rounding of the contribution, one of each sum
        once = (s.float() + f.float()).to(gdtype)
        assert torch.equal(a, (once.float() + f.float()).to(gdtype))


@pytest.mark.gpu
def test_no_rows(gpu_lib):
    n = mk.Norm(96)
    e = torch.empty(0, 96, dtype=BF, device="cuda")
    w, st = torch.ones(96, dtype=BF, device="cuda"), torch.empty(0, 2, device="cuda")
    n.forward(e, w, None, e.clone(), st)
    dw = torch.full((96,), 3.0, device="cuda")
    n.backward(e, e, w, st, e.clone(), dw)
    assert bool((dw == 3.0).all())
    n.backward(e, e, w, st, e.clone(), dw, overwrite=True)
    assert bool((dw == 0.0).all())


@pytest.mark.gpu
def test_large_offset_keeps_the_centred_values(gpu_lib):
    """Rows of mean 1000 and spread 1 in FP32: the twice-centred statistics stay within the
    bound, which has no term in the offset."""
    x, w, b, _, _ = make(33, 4096, F32, F32, seed=8, offset=1000.0)
    y, stats, _ = _run_forward(mk.Norm(4096, dtype=F32), x, w, b, None, "layer", 0, 0)
    check_forward(x, w, b, y, stats, "layer")


@pytest.mark.gpu
def test_nonfinite_rows_stay_in_their_row(gpu_lib):
    x, w, b, _, _ = make(6, 1500, F32, F32, seed=9)
    x[1, 700] = float("nan")
    x[3, 2] = float("inf")
    y, stats, _ = _run_forward(mk.Norm(1500, dtype=F32), x, w, b, None, "layer", 0, 0)
    assert bool(torch.isnan(y[1]).all()) and bool(torch.isnan(y[3]).all())
    keep = [0, 2, 4, 5]
    check_forward(x[keep], w, b, y[keep], stats[keep], "layer")
    # a constant row: centred values are exactly zero
    x[0] = 0.1
    y, _, _ = _run_forward(mk.Norm(1500, dtype=F32), x, w, b, None, "layer", 0, 0)
    assert float((y[0] - b).abs().max()) <= 2.0 ** -20     # |x - mean| <= u |x|, times rstd = 316: 2^-24 * 0.1 * 316


@pytest.mark.gpu
def test_sum_in_place(gpu_lib):
    x, w, b, res, _ = make(40, 4096, BF, BF, seed=10)
    want_y, _, want_s = _run_forward(mk.Norm(4096), x, w, b, res, "layer", 0, 0)
    for which in (0, 1):
        t = [x.cuda(), res.cuda()]
        y = torch.empty_like(t[0])
        mk.Norm(4096).forward(t[0], w.cuda(), b.cuda(), y, residual=t[1], sum=t[which])
        assert torch.equal(t[which].cpu(), want_s) and torch.equal(y.cpu(), want_y)


@pytest.mark.gpu
@pytest.mark.parametrize("R,N", [(1, 64), (70, 4096), (1030, 264), (300, 2055), (5, 16384)])
def test_outputs_in_place_of_inputs(gpu_lib, R, N):
    """y over x, grad_x over grad_y, x or grad_sum: the same bits as into memory of their own."""
    x, w, b, dy, gs = (t.cuda() for t in make(R, N, BF, BF, seed=13))
    n = mk.Norm(N)
    y, stats, dx, dw, db = (torch.empty_like(x), torch.empty(R, 2, device="cuda"), torch.empty_like(x),
                            torch.empty(N, device="cuda"), torch.empty(N, device="cuda"))
    n.forward(x, w, b, y, stats)
    t = x.clone()
    n.forward(t, w, b, t)
    assert torch.equal(t, y)
    n.backward(dy, x, w, stats, dx, dw, db, grad_sum=gs, overwrite=True)
    for i in range(3):
        c = [dy.clone(), x.clone(), gs.clone()]
        dw2, db2 = torch.empty_like(dw), torch.empty_like(db)
        n.backward(c[0], c[1], w, stats, c[i], dw2, db2, grad_sum=c[2], overwrite=True)
        assert torch.equal(c[i], dx) and torch.equal(dw2, dw) and torch.equal(db2, db)


@pytest.mark.gpu
def test_row_offsets_past_32_bits(gpu_lib):
    """Five rows a gigabyte apart: byte offsets pass 2^32."""
    N, ld = 264, (1 << 29) + 8
    x, w, b, dy, _ = make(5, N, BF, BF, seed=11)
    store = torch.empty(2, 4 * ld + N, dtype=BF, device="cuda")
    xv, yv = (store[i].as_strided((5, N), (ld, 1), store[i].storage_offset()) for i in (0, 1))
    xv.copy_(x)
    stats = torch.empty(5, 2, device="cuda")
    n = mk.Norm(N)
    n.forward(xv, w.cuda(), b.cuda(), yv, stats)
    check_forward(x, w, b, yv.cpu(), stats.cpu(), "layer")
    dw, db = torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
    n.backward(dy.cuda(), xv, w.cuda(), stats, yv, dw, db, overwrite=True)
    check_backward(dy, x, w, stats.cpu(), "layer", None, yv.cpu(), dw.cpu(), db.cpu())


@pytest.mark.gpu
def test_graph_replay_side_stream_and_repeatability(gpu_lib):
    R, N = 1000, 4096
    x, w, b, dy, gs = (t.cuda() for t in make(R, N, BF, BF, seed=12))
    n = mk.Norm(N)
    y, dx, stats = torch.empty_like(x), torch.empty_like(x), torch.empty(R, 2, device="cuda")
    dw, db = torch.empty(N, device="cuda"), torch.empty(N, device="cuda")

    def step():
        n.forward(x, w, b, y, stats)
        n.backward(dy, x, w, stats, dx, dw, db, grad_sum=gs, overwrite=True)

    outs = (y, dx, stats, dw, db)
    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(outs, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        x2 = torch.randn_like(x.float()).to(BF)
        x.copy_(x2)
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in outs]
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(outs, want)), i


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("N", [1000, 1003, 1500, 3584, 7168, 12300])
def test_constant_rows_far_from_zero(gpu_lib, N, dtype):
    """Rows of one value c, far above the spread that eps allows for.  The first mean is off by at
    most 40 u c (and half a step of c), so d = c - mean is exact, a multiple of half a step of c and at
    most 81 of those: the sum of N of them is exact (81 N < 2^24) and so is its Nth, which is d
    itself.  What is left is a variance of 0: y is the bias, the mean c and rstd 1 / sqrt(eps),
    off by the rounding of the root and of the quotient, u each."""
    g = torch.Generator().manual_seed(N)
    R, eps = 256, 1e-12
    c = torch.exp(torch.empty(R).uniform_(9.2, 11.6, generator=g))         # 1e4 .. 1.1e5
    c[:4] = torch.tensor([11572.6005859375, 31307.4, 26514.5, -20000.3])
    x = c.to(dtype)[:, None].expand(R, N).contiguous()
    w, b = 1 + 0.2 * torch.randn(N, generator=g), 0.3 * torch.randn(N, generator=g)
    y, stats, _ = _run_forward(mk.Norm(N, eps=eps, dtype=dtype, param_dtype=F32), x, w, b, None, "layer", 0, 0)
    assert torch.equal(y, b.to(dtype)[None].expand(R, N))
    assert torch.equal(stats[:, 0], x[:, 0].float())
    want = 1.0 / float(torch.tensor(eps, dtype=F32).double().sqrt())
    assert bool((stats[:, 1].double() / want - 1).abs().max() <= 3 * U)


@pytest.mark.gpu
@pytest.mark.parametrize("N", [1000, 1003, 3584, 7168, 12300])
def test_rows_of_two_neighbouring_values(gpu_lib, N):
    """c and the next number above it, a step (2 u c at most) apart, half of each or a few among the rest.
    As for constant rows all differences and their sum are exact, |delta| <= 81 half steps; its
    division is off by u |delta| <= 41 u steps and each centred value by that and u of itself.
    The variance is then off by its sum's 40 u and twice those 41 u steps over its root, at most."""
    g = torch.Generator().manual_seed(N + 1)
    R, eps = 64, 1e-12
    c = torch.exp(torch.empty(R, 1).uniform_(9.3, 10.3, generator=g))      # 1.1e4 .. 3e4
    step = torch.exp2(torch.floor(torch.log2(c)) - 23)
    share = torch.tensor([0.5, 0.02])[torch.arange(R) % 2][:, None]
    on = torch.rand(R, N, generator=g) < share
    on[:, 0] = True
    x = c + step * on
    assert bool(((x == c) | on).all()) and bool((x[:, 0] > c[:, 0]).all())
    w, b = 1 + 0.2 * torch.randn(N, generator=g), 0.3 * torch.randn(N, generator=g)
    y, stats, _ = _run_forward(mk.Norm(N, eps=eps, dtype=F32), x, w, b, None, "layer", 0, 0)
    ref, xh, mu, rstd = ref_forward(x, w, b, "layer", float(torch.tensor(eps, dtype=F32)))
    off = 41 * U * step.double() * rstd                       # of (x - mean) rstd
    rel = 64 * U + 2 * off + off ** 2                         # of rstd
    assert bool(((stats[:, 1:].double() / rstd - 1).abs() <= rel).all())
    assert bool(((stats[:, :1].double() - mu).abs() <= 41 * U * step.double() + 2 * U * mu.abs()).all())
    tol = (off + (rel + 4 * U) * xh.abs()) * w.double().abs() + 2 * U * (ref.abs() + b.double().abs())
    assert bool(((y.double() - ref).abs() <= tol).all())


@pytest.mark.gpu
@pytest.mark.parametrize("N", [97, 200, 1000, 1003, 1400, 1900, 3584, 7168])
def test_constant_rows_beside_ordinary_ones(gpu_lib, N):
    """Rows that share a wave or a workgroup with rows of one value (and with one that holds a
    NaN) get the results they get beside others, bit for bit; every second of them has a spread of a
    few steps of its mean."""
    R, eps = 96, 1e-12
    x, w, b, _, _ = make(R, N, F32, F32, seed=21)
    n = mk.Norm(N, eps=eps, dtype=F32)
    y, stats, _ = _run_forward(n, x, w, b, None, "layer", 0, 0)
    check_forward(x, w, b, y, stats, "layer", eps=eps)
    g = torch.Generator().manual_seed(N)
    x[1::2] = 20000 + torch.randint(0, 16, (R // 2, N), generator=g) * torch.rand(R // 2, 1, generator=g) * 2.0 ** -9   # steps
    alone, stats, _ = _run_forward(n, x, w, b, None, "layer", 0, 0)
    flat = torch.rand(R, generator=g) < 0.4
    c = torch.exp(torch.empty(R, 1).uniform_(9.3, 11.5, generator=g))
    mixed = torch.where(flat[:, None], c, x)
    mixed[5, N // 2], flat[5] = float("nan"), True
    y, st, _ = _run_forward(n, mixed, w, b, None, "layer", 0, 0)
    assert bool(torch.isnan(y[5]).all())
    assert torch.equal(y[~flat], alone[~flat]) and torch.equal(st[~flat], stats[~flat])
    flat[5] = False
    assert torch.equal(y[flat], b[None].expand(int(flat.sum()), N))


LAYOUTS = [
    # R, N, pad, offset: rows of whole 16-byte pieces that are 4-byte aligned only (BF16)
    (1, 8, 2, 2), (37, 64, 2, 0), (130, 128, 6, 2), (600, 256, 2, 2), (70, 384, 2, 4), (65, 1032, 2, 2), (300, 4096, 2, 2),
    (5, 7168, 6, 2),
    # more than 8192 columns: contiguous, 4-byte aligned, by elements
    (3, 8200, 0, 0), (300, 8208, 0, 0), (5, 12304, 0, 0), (4, 16384, 0, 0), (4, 12304, 2, 2), (6, 16384, 2, 0),
    (3, 8201, 0, 0), (270, 9001, 1, 0), (3, 16383, 3, 1), (4, 16384, 1, 1),
]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dtype,pdtype", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("i", range(len(LAYOUTS)))
def test_layouts_match_formula(gpu_lib, i, dtype, pdtype, kind):
    dev, (R, N, pad, offset) = "cuda", LAYOUTS[i]
    x, w, b, dy, gs = make(R, N, dtype, pdtype, seed=200 + i)
    n = mk.Norm(N, kind=kind, dtype=dtype, param_dtype=pdtype)
    y, stats, _ = _run_forward(n, x, w, b, None, kind, pad, offset)
    check_forward(x, w, b, y, stats, kind)
    y, stats, s = _run_forward(n, x, w, None, dy, kind, pad, offset)
    assert torch.equal(s, (x.float() + dy.float()).to(dtype))
    check_forward(s, w, None, y, stats, kind)
    _, _, mu, rstd = ref_forward(x, w, None, kind, 1e-5)
    stats = torch.cat([mu, rstd], 1).float()
    xv, dyv, gsv = (padded(t.to(dev), pad, offset)[0] for t in (x, dy, gs))
    for gsum in (None, gs):
        dxv, dxb = padded(torch.zeros(R, N, dtype=dtype, device=dev), pad, offset)
        dw, db = (torch.full((N,), float("nan"), device=dev) for _ in range(2))
        n.backward(dyv, xv, w.to(dev), stats.to(dev), dxv, dw, db, grad_sum=None if gsum is None else gsv, overwrite=True)
        torch.cuda.synchronize()
        assert untouched(dxv, dxb, offset)
        check_backward(dy, x, w, stats, kind, gsum, dxv.cpu(), dw.cpu(), db.cpu())


def test_norm_names_the_status_of_refused_options():
    """The same status as moe_norm_forward returns for them."""
    for kw, status in ((dict(eps=-1.0), mk.MOE_ERR_UNSUPPORTED), (dict(eps=float("nan")), mk.MOE_ERR_UNSUPPORTED),
                       (dict(cols=mk.MOE_NORM_MAX_COLS + 1), mk.MOE_ERR_SHAPE), (dict(cols=-1), mk.MOE_ERR_SHAPE)):
        with pytest.raises(mk.MoeError) as ei:
            mk.Norm(**{"cols": 64, "device": "cpu", **kw})
        assert ei.value.status == status, kw

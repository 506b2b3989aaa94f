"""The 8-bit product with a scale for each block of 128 and its quantiser, against their
formulas in 64 bits.

Quantiser, tolerance: none for BF16 values.  448 v / m with 8-bit v and m is a tie of E4M3 or at
least 2^-14 of itself away from one, and the FP32 quotient is within 2^-23; the scale is one correctly rounded
division.  For FP32 values a code is the nearest up to 2^-22 of the quotient.

Product: u = 2^-24.  With an FP32 result the codes' products are exact, a block is a sum of 128, K / 128
scaled blocks follow (their scale a product of two): off by at most 2 (128 + K / 128 + 8) u of the sum
of magnitudes.  With a BF16 result the 8-bit instruction keeps 2^-16 of its largest product: 2^-15 of the sum of
magnitudes covers two partial sums, and the result's rounding is 2^-8 of itself."""
import pytest
import torch

import moe_megakernel_amd as mk

PTR = 1 << 20
U = 2.0 ** -24
F8 = torch.float8_e4m3fn


# ------------------------------------------------------------------ references
def blocks(v, kind):
    """m of each block, broadcast over v's padded shape: (padded v, m [same shape], m by block)."""
    P, Q = v.shape
    rb = 1 if kind == "rows" else 128
    p = torch.nn.functional.pad(v, (0, -Q % 128, 0, -P % rb))
    t = p.view(p.shape[0] // rb, rb, -1, 128)
    m = t.abs().amax(-1).amax(1)
    return p, m.repeat_interleave(rb, 0).repeat_interleave(128, 1), m


def ref_quantize(x, kind, transpose):
    v = x.detach().cpu().double()
    if transpose:
        v = v.t().contiguous()
    P, Q = v.shape
    p, m, by = blocks(v, kind)
    bad = ~torch.isfinite(by)
    q = torch.where(m > 0, 448.0 * p / m, torch.zeros_like(p))[:P, :Q]
    scale = torch.where(by > 0, (by.float() / 448.0), torch.ones_like(by).float())
    scale = torch.where(bad, torch.full_like(scale, float("nan")), scale)
    return q, (scale.t().contiguous() if kind == "rows" else scale)


def nearest_e4m3(q):
    """The E4M3 value nearest to each q (64 bits, |q| <= 448), ties to even."""
    e = torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6)))
    e = torch.where(2.0 ** e > q.abs().clamp(min=2.0 ** -6), e - 1, e)
    step = 2.0 ** (e.clamp(min=-6) - 3)
    return torch.round(q / step) * step


def values(q, s, kind):
    q = q.detach().cpu().double()
    s = s.detach().cpu().double()
    if kind == "rows":
        return q * s.t().repeat_interleave(128, 1)[:, :q.shape[1]]
    return q * s.repeat_interleave(128, 0)[:q.shape[0]].repeat_interleave(128, 1)[:, :q.shape[1]]


def test_reference_codes_match_the_type():
    q = torch.cat([torch.linspace(-448, 448, 10001, dtype=torch.float64), torch.tensor([2.0 ** -10, 3 * 2.0 ** -10], dtype=torch.float64)])
    assert torch.equal(nearest_e4m3(q), q.float().to(F8).double())


# ------------------------------------------------------------------ CPU: refusals
@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), mk.MOE_ERR_SHAPE), (dict(rows=(1 << 31) + 1), mk.MOE_ERR_SHAPE), (dict(cols=0), mk.MOE_ERR_SHAPE),
    (dict(cols=(1 << 24) + 1), mk.MOE_ERR_SHAPE), (dict(rows=1 << 31, cols=1 << 20), mk.MOE_ERR_SHAPE),
    (dict(kind=0), mk.MOE_ERR_UNSUPPORTED), (dict(kind=3), mk.MOE_ERR_UNSUPPORTED),
    (dict(dtype=mk.MOE_MXINT8), mk.MOE_ERR_DTYPE), (dict(flags=2), mk.MOE_ERR_UNSUPPORTED)])
def test_bad_quantizer_problems_are_refused(kw, status):
    d = dict(rows=4, cols=64, kind=mk.MOE_FP8_ROWS, dtype=mk.MOE_BF16, flags=0)
    d.update(kw)
    p = mk.moe_block_quantize_problem(d["rows"], d["cols"], d["kind"], d["dtype"], d["flags"])
    assert mk.moe_block_quantize(p, mk.moe_rows(PTR, max(d["cols"], 1)), PTR, PTR, None) == status


def test_bad_quantizer_arguments_are_refused():
    p = mk.moe_block_quantize_problem(4, 64, mk.MOE_FP8_TILES, mk.MOE_FP32, 0)
    ok = mk.moe_rows(PTR, 64)
    assert mk.moe_block_quantize(p, None, PTR, PTR, None) == mk.MOE_ERR_NULL
    assert mk.moe_block_quantize(p, ok, None, PTR, None) == mk.MOE_ERR_NULL
    assert mk.moe_block_quantize(p, ok, PTR, None, None) == mk.MOE_ERR_NULL
    assert mk.moe_block_quantize(p, mk.moe_rows(PTR, 63), PTR, PTR, None) == mk.MOE_ERR_LAYOUT
    assert mk.moe_block_quantize(p, mk.moe_rows(PTR + 2, 64), PTR, PTR, None) == mk.MOE_ERR_LAYOUT
    assert mk.moe_block_quantize(p, ok, PTR + 8, PTR, None) == mk.MOE_ERR_LAYOUT
    assert mk.moe_block_quantize(p, ok, PTR, PTR + 2, None) == mk.MOE_ERR_LAYOUT


def _mm(rows=4, cols=32, depth=64, groups=1, scales=mk.MOE_FP8_TILES, out=mk.MOE_BF16, flags=0):
    return mk.moe_block_matmul_problem(rows, cols, depth, groups, scales, out, flags)


def _call(p, a=(PTR, 64), sa=PTR, b=(PTR, 2048, 0, 64), sb=PTR, off=None, out=(PTR, 32)):
    return mk.moe_block_matmul(p, a and mk.moe_rows(*a), sa, b and mk.moe_mat(*b), sb, off, out and mk.moe_rows(*out), None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), mk.MOE_ERR_SHAPE), (dict(rows=(1 << 24) + 1), mk.MOE_ERR_SHAPE), (dict(cols=0), mk.MOE_ERR_SHAPE),
    (dict(depth=24), mk.MOE_ERR_SHAPE), (dict(depth=0), mk.MOE_ERR_SHAPE), (dict(groups=0), mk.MOE_ERR_SHAPE),
    (dict(groups=257), mk.MOE_ERR_SHAPE), (dict(rows=1 << 24, cols=1 << 20), mk.MOE_ERR_SHAPE),
    (dict(scales=0), mk.MOE_ERR_UNSUPPORTED), (dict(scales=mk.MOE_FP8_ROWS, groups=2), mk.MOE_ERR_UNSUPPORTED),
    (dict(out=mk.MOE_MXINT8), mk.MOE_ERR_DTYPE), (dict(flags=1), mk.MOE_ERR_UNSUPPORTED)])
def test_bad_product_problems_are_refused(kw, status):
    assert _call(_mm(**kw), off=PTR) == status


def test_bad_product_arguments_are_refused():
    p = _mm()
    for kw in (dict(a=None), dict(a=(0, 64)), dict(sa=None), dict(b=None), dict(b=(0, 0, 0, 64)), dict(sb=None),
               dict(out=None), dict(out=(0, 32))):
        assert _call(p, **kw) == mk.MOE_ERR_NULL, kw
    for kw in (dict(a=(PTR, 48)), dict(a=(PTR, 72)), dict(a=(PTR + 8, 64)), dict(sa=PTR + 1), dict(b=(PTR, 0, PTR, 64)),
               dict(b=(PTR, 0, 0, 60)), dict(b=(PTR + 4, 0, 0, 64)), dict(sb=PTR + 2), dict(out=(PTR, 31)),
               dict(out=(PTR + 1, 32)), dict(off=PTR + 2)):
        assert _call(p, **kw) == mk.MOE_ERR_LAYOUT, kw
    assert _call(_mm(groups=2)) == mk.MOE_ERR_NULL               # several groups need offsets
    assert _call(_mm(groups=2), b=(PTR, 24, 0, 64), off=PTR) == mk.MOE_ERR_LAYOUT
    assert _call(_mm(rows=0), a=None, sa=None, b=None, sb=None, out=None) == mk.MOE_OK


def test_binding_refuses_host_and_mismatched_tensors():
    q, mm = mk.Fp8Quantizer(), mk.Fp8Matmul()
    x, c, s = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, 64, dtype=F8), torch.zeros(1, 4)

    def status(f, *a, **k):
        with pytest.raises(mk.MoeError) as e:
            f(*a, **k)
        return e.value.status
    assert status(q.forward, x, c, s) == mk.MOE_ERR_LAYOUT
    assert status(q.forward, x.float(), c, s) == mk.MOE_ERR_DTYPE
    assert status(q.forward, x[:, :0], c, s) == mk.MOE_ERR_SHAPE
    w, ws, out = torch.zeros(32, 64, dtype=F8), torch.zeros(1, 1), torch.zeros(4, 32, dtype=torch.bfloat16)
    assert status(mm.forward, c, s, w, ws, out) == mk.MOE_ERR_LAYOUT
    assert status(mm.forward, c, s, w[:, :48], ws, out) == mk.MOE_ERR_SHAPE
    assert status(mm.forward, c, s, None, ws, out) == mk.MOE_ERR_NULL
    assert status(mk.Fp8Matmul, "cols") == mk.MOE_ERR_UNSUPPORTED
    assert status(mk.Fp8Quantizer, "cols") == mk.MOE_ERR_UNSUPPORTED
    assert status(mk.Fp8Quantizer, dtype=torch.float16) == mk.MOE_ERR_DTYPE
    assert mk.Fp8Quantizer("tiles", transpose=True).shapes(130, 77) == ((77, 144), (1, 2))
    assert mk.Fp8Quantizer("rows").shapes(130, 77) == ((130, 80), (1, 130))


# ------------------------------------------------------------------ GPU: quantiser
def gpu_quantize(x, kind, transpose, pad=0):
    op = mk.Fp8Quantizer(kind, transpose, x.dtype)
    R, C = x.shape
    buf = torch.full((R, C + pad), float("nan"), dtype=x.dtype, device="cuda")
    buf[:, :C] = x
    qs, ss = op.shapes(R, C)
    codes = torch.full(qs, 0x7f, dtype=torch.uint8, device="cuda").view(F8)
    scales = torch.full(ss, float("inf"), device="cuda")
    op.forward(buf[:, :C], codes, scales)
    return codes, scales


def check_quantize(x, kind, transpose, pad=0):
    codes, scales = gpu_quantize(x, kind, transpose, pad)
    q, s = ref_quantize(x, kind, transpose)
    P, Q = q.shape
    assert torch.equal(scales.cpu().nan_to_num(-1), s.nan_to_num(-1))
    got = codes.cpu().double()
    assert not got[:, Q:].any()                               # the padding
    got = got[:, :Q]
    dead = torch.isnan(values(torch.ones(P, Q), s, kind))
    want = torch.where(dead, torch.zeros_like(q), q)
    if x.dtype == torch.bfloat16:
        assert torch.equal(got, nearest_e4m3(want.nan_to_num(0.0)))
    else:
        best = nearest_e4m3(want.nan_to_num(0.0))
        assert ((got - want).abs() <= (best - want).abs() + 2.0 ** -22 * want.abs()).all()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["rows", "tiles"])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("R,C,pad,dtype", [(1, 1, 0, torch.bfloat16), (1, 128, 0, torch.bfloat16), (5, 127, 1, torch.float32),
                                           (128, 128, 0, torch.float32), (129, 136, 8, torch.bfloat16), (70, 1000, 0, torch.bfloat16),
                                           (300, 77, 3, torch.float32), (257, 640, 0, torch.bfloat16), (33, 2056, 8, torch.float32)])
def test_quantizer_is_the_definition(gpu_lib, kind, transpose, R, C, pad, dtype):
    g = torch.Generator().manual_seed(R + C)
    x = torch.randn(R, C, generator=g) * torch.exp(3 * torch.randn(R, 1, generator=g))
    check_quantize(x.to(dtype), kind, transpose, pad)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["rows", "tiles"])
@pytest.mark.parametrize("transpose", [False, True])
def test_quantizer_on_zeros_extremes_and_nonfinite_values(gpu_lib, kind, transpose):
    x = torch.randn(260, 300)
    x[:140] = 0.0
    x[200, 250] = 3.0e38
    check_quantize(x.to(torch.bfloat16), kind, transpose)
    check_quantize(torch.randn(9, 200) * 1e-38, kind, transpose)
    for bad in (float("nan"), float("inf")):
        y = torch.randn(260, 300)
        y[130, 5] = bad
        y[0, 299] = -bad
        check_quantize(y, kind, transpose)


# ------------------------------------------------------------------ GPU: product
def operands(M, N, K, G, scales, seed):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)
    a, sa = gpu_quantize((rn(M, K) * torch.exp(rn(M, 1))).cuda(), "rows", False)
    b = torch.empty(G, N, K, dtype=F8, device="cuda")
    sbs = []
    for e in range(G):
        be, s = gpu_quantize((rn(N, K) * 0.05).cuda(), scales, False)
        b[e] = be
        sbs.append(s)
    sb = sbs[0] if scales == "rows" else torch.stack(sbs)
    return a, sa, b, sb


def check_product(M, N, K, G=1, ends=None, scales="tiles", out_dtype=torch.bfloat16, accumulate=False, pad=0, seed=0):
    a, sa, b, sb = operands(M, N, K, G, scales, seed)
    ends = ends or [0, M]
    use_offsets = G > 1 or ends != [0, M]
    offsets = torch.tensor(ends, dtype=torch.int32, device="cuda") if use_offsets else None
    inside = torch.zeros(M, dtype=torch.bool)
    for lo, hi in zip(ends, ends[1:]):
        inside[lo:hi] = True
    # rows outside every group: NaN codes and scales
    a.view(torch.uint8)[~inside.cuda()] = 0x7f
    sa[:, ~inside.cuda()] = float("nan")
    buf = torch.randn(M, N + pad, generator=torch.Generator().manual_seed(seed + 1)).to(out_dtype).cuda()
    before = buf.clone()
    mk.Fp8Matmul(scales, out_dtype, accumulate).forward(a, sa, b, sb, buf[:, :N], offsets=offsets)
    torch.cuda.synchronize()
    av = values(a, sa, "rows")
    ref, mag = torch.zeros(M, N, dtype=torch.float64), torch.zeros(M, N, dtype=torch.float64)
    for e, (lo, hi) in enumerate(zip(ends, ends[1:])):
        bv = values(b[e], sb if scales == "rows" else sb[e], scales)
        ref[lo:hi] = av[lo:hi] @ bv.t()
        mag[lo:hi] = av[lo:hi].abs() @ bv.abs().t()
    old = before[:, :N].cpu().double()
    half = 2.0 ** -8 if out_dtype == torch.bfloat16 else U
    tol = (2.0 ** -15 if out_dtype == torch.bfloat16 else 2 * (128 + K / 128 + 8) * U) * mag + half * ref.abs()
    if accumulate:
        tol = tol + half * (ref.abs() + old.abs() + tol)
        ref = ref + old
    got = buf[:, :N].cpu().double()
    assert torch.isfinite(got[inside]).all()
    assert ((got - ref).abs()[inside] <= tol[inside]).all()
    assert torch.equal(buf[:, N:], before[:, N:])
    assert torch.equal(buf[~inside.cuda()], before[~inside.cuda()])


@pytest.mark.gpu
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("scales", ["tiles", "rows"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 16), (1, 16, 128), (16, 17, 144), (33, 130, 1040), (64, 256, 4096), (65, 128, 128),
                                   (66, 5, 272), (200, 515, 1040), (257, 384, 640), (513, 100, 2048), (700, 1024, 512)])
def test_product_matches_formula(gpu_lib, out_dtype, scales, M, N, K):
    check_product(M, N, K, scales=scales, out_dtype=out_dtype, seed=M + N + K)


@pytest.mark.gpu
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("ends", [[0, 0, 0, 40], [3, 10, 10, 37], [0, 64, 64, 64], [0, 300, 301, 600], [7, 200, 560, 597],
                                  [600, 600, 600, 600], [0, 0, 600, 600]])
def test_groups_take_their_own_weight_and_leave_other_rows(gpu_lib, out_dtype, ends):
    M = 64 if ends[-1] <= 64 else 600
    check_product(M, 200, 400, G=3, ends=ends, out_dtype=out_dtype, pad=4, seed=ends[1] + ends[2])


@pytest.mark.gpu
def test_many_groups(gpu_lib):
    G = 256
    g = torch.Generator().manual_seed(3)
    n = torch.randint(0, 6, (G,), generator=g)
    ends = [2] + (2 + torch.cumsum(n, 0)).tolist()
    check_product(ends[-1] + 9, 64, 144, G=G, ends=ends, seed=4)
    one = [0] + [0] * 100 + [50] * 156
    check_product(60, 64, 144, G=G, ends=one, seed=5)


@pytest.mark.gpu
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,pad", [(30, 50, 0), (300, 260, 4), (300, 259, 1)])
def test_accumulation_and_strides(gpu_lib, out_dtype, M, N, pad):
    check_product(M, N, 528, out_dtype=out_dtype, accumulate=True, pad=pad, seed=N)
    check_product(M, N, 528, scales="rows", out_dtype=out_dtype, accumulate=True, pad=pad, seed=N)
    check_product(M, N, 528, out_dtype=out_dtype, pad=pad, seed=N)


@pytest.mark.gpu
def test_offset_entries_outside_the_rows_stay_inside(gpu_lib):
    """Entries below 0 or above M count as the nearest end."""
    for M in (40, 300):
        a, sa, b, sb = operands(M, 96, 256, 2, "tiles", 8)
        out, want = torch.zeros(M, 96, dtype=torch.bfloat16, device="cuda"), torch.zeros(M, 96, dtype=torch.bfloat16, device="cuda")
        mm = mk.Fp8Matmul()
        mm.forward(a, sa, b, sb, want, offsets=torch.tensor([0, 17, M], dtype=torch.int32, device="cuda"))
        mm.forward(a, sa, b, sb, out, offsets=torch.tensor([-5, 17, M + 99], dtype=torch.int32, device="cuda"))
        assert torch.equal(out, want)


@pytest.mark.gpu
def test_nan_scale_stays_in_its_row_and_column(gpu_lib):
    for M in (20, 300):
        a, sa, b, sb = operands(M, 300, 512, 1, "tiles", 9)
        sa[2, 5] = float("nan")
        sb[0, 1, 0] = float("inf")
        out = torch.zeros(M, 300, dtype=torch.bfloat16, device="cuda")
        mk.Fp8Matmul().forward(a, sa, b, sb, out)
        bad = ~torch.isfinite(out).cpu()
        assert bad[5].all()
        assert bad[:, 128:256].all()
        bad[5] = False
        bad[:, 128:256] = False
        assert not bad.any()


@pytest.mark.gpu
def test_row_offsets_past_32_bits(gpu_lib):
    M, N, K = 140000, 16, 16384                                # 2.3e9 codes
    a = torch.zeros(M, K, dtype=torch.uint8, device="cuda").view(F8)
    sa = torch.ones(K // 128, M, device="cuda")
    t, st, b, sb = operands(5, N, K, 1, "tiles", 10)
    a.view(torch.uint8)[-5:] = t.view(torch.uint8)
    sa[:, -5:] = st
    out = torch.ones(M, N, dtype=torch.float32, device="cuda")
    mk.Fp8Matmul(out_dtype=torch.float32).forward(a, sa, b, sb, out)
    ref = values(t, st, "rows") @ values(b[0], sb[0], "tiles").t()
    mag = values(t, st, "rows").abs() @ values(b[0], sb[0], "tiles").abs().t()
    assert ((out[-5:].cpu().double() - ref).abs() <= 2 * (128 + 128 + 8) * U * mag + U * ref.abs()).all()
    assert not out[:-5].any()


@pytest.mark.gpu
def test_training_step_of_a_projection(gpu_lib):
    """y = x W^T, dx = dy W and dW += dy^T x, each from the quantiser's codes, against the products
    of the values that the codes stand for; with autograd's as the formula of the three."""
    T, N, K = 333, 256, 384
    g = torch.Generator().manual_seed(11)
    bf = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()
    x, w, dy = bf(T, K), bf(N, K), bf(T, N)
    xq, wq, wt = gpu_quantize(x, "rows", False), gpu_quantize(w, "tiles", False), gpu_quantize(w, "tiles", True)
    dq, dt, xt = gpu_quantize(dy, "rows", False), gpu_quantize(dy, "rows", True), gpu_quantize(x, "rows", True)
    y, dx = torch.empty(T, N, dtype=torch.bfloat16, device="cuda"), torch.empty(T, K, dtype=torch.bfloat16, device="cuda")
    start = torch.randn(N, K, generator=g)
    dw = start.cuda()
    mk.Fp8Matmul().forward(*xq, *wq, y)
    mk.Fp8Matmul().forward(*dq, *wt, dx)
    mk.Fp8Matmul("rows", torch.float32, accumulate=True).forward(*dt, *xt, dw)
    assert torch.equal(values(*wq, "tiles"), values(*wt, "tiles").t())
    # the weight gradient's operands: the same matrix in blocks along its other side
    xv, wv, dv = values(*xq, "rows").requires_grad_(True), values(*wq, "tiles").requires_grad_(True), values(*dq, "rows")
    yv = xv @ wv.t()
    (yv * dv).sum().backward()
    dtv, xtv = values(*dt, "rows")[:, :T], values(*xt, "rows")[:, :T]
    dwv = dtv @ xtv.t()

    def near(got, ref, mag, half, f):
        assert ((got.detach().cpu().double() - ref).abs() <= f * mag + half * ref.abs()).all()
    near(y, yv.detach(), xv.detach().abs() @ wv.detach().abs().t(), 2.0 ** -8, 2.0 ** -15)
    near(dx, xv.grad, dv.abs() @ wv.detach().abs(), 2.0 ** -8, 2.0 ** -15)
    near(dw, dwv + start.double(), dtv.abs() @ xtv.abs().t() + start.double().abs(), U, 2 * (128 + 3 + 8) * U)
    # and the 8-bit gradient is the formula's up to its operands' roundings: both sides are within 2^-4 of
    # the same value, so a product of two is within (17 / 15)^2 - 1 < 0.29 of the other's; codes below
    # 2^-6 have steps of their own, 2^-10 of 448 at most
    mag = dv.abs().t() @ xv.detach().abs()
    assert ((dwv - wv.grad).abs() <= 0.29 * mag + 2.0 ** -8 * mag.max()).all()


@pytest.mark.gpu
@pytest.mark.parametrize("M", [20, 300])
def test_captured_and_on_another_stream(gpu_lib, M):
    N, K = 256, 512
    g = torch.Generator().manual_seed(12)
    x = torch.randn(M, K, generator=g).to(torch.bfloat16).cuda()
    w = torch.randn(N, K, generator=g).to(torch.bfloat16).cuda()
    wq = gpu_quantize(w, "tiles", False)
    q = mk.Fp8Quantizer()
    qs, ss = q.shapes(M, K)
    codes, scales = torch.empty(qs, dtype=F8, device="cuda"), torch.empty(ss, device="cuda")
    out, mm = torch.empty(M, N, dtype=torch.bfloat16, device="cuda"), mk.Fp8Matmul()
    offsets = torch.tensor([1, M - 2], dtype=torch.int32, device="cuda")

    def step():
        q.forward(x, codes, scales)
        mm.forward(codes, scales, *wq, out, offsets=offsets)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        x.copy_(torch.randn(M, K, generator=g))
        out.zero_()
        step()
        torch.cuda.synchronize()
        want = out.clone()
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), i


def test_products_past_the_limits_are_refused():
    far = mk.MOE_FP8_MAX_LD + 16
    assert _call(_mm(), a=(PTR, far)) == mk.MOE_ERR_LAYOUT
    assert _call(_mm(), b=(PTR, 0, 0, far)) == mk.MOE_ERR_LAYOUT
    assert _call(_mm(depth=(1 << 22) + 16), a=(PTR, 1 << 23), b=(PTR, 0, 0, 1 << 23)) == mk.MOE_ERR_SHAPE


# Enough tiles for every CU: the sizes where the product goes in large tiles, of two and of nine blocks of k.
@pytest.mark.gpu
@pytest.mark.parametrize("scales", ["tiles", "rows"])
@pytest.mark.parametrize("K", [144, 1040])
@pytest.mark.parametrize("accumulate,pad", [(False, 1), (True, 6)])
def test_wide_product_matches_formula(gpu_lib, scales, K, accumulate, pad):
    check_product(1050, 5130, K, scales=scales, accumulate=accumulate, pad=pad, seed=K)


@pytest.mark.gpu
@pytest.mark.parametrize("ends", [[0, 0, 129, 1200], [5, 500, 1100, 1150]])
def test_wide_product_in_groups_matches_formula(gpu_lib, ends):
    check_product(1200, 5130, 1040, G=3, ends=ends, seed=ends[1])

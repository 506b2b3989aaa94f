"""The router's decision and its gradient, against the formulas in 64 bits.

Tolerances.  u = 2^-24.  exp(l - m) in FP32 is off by (|l - m| + 4) u relative (the rounding
of its argument and 2 ulp of the function), the row sum by 20 u more and the divisions by 1 u
each, so scores, chosen sums and weights are within (range + 64) u of themselves, range being
the largest |l - m| of the row (|l| for sigmoid).  A gradient is that far off in each of its terms.
Tables are compared exactly: logits are compared as they are and scores with a bias in 64 bits."""
import pytest
import torch

import moe_megakernel_amd as mk

U = 2.0 ** -24
NINF = float("-inf")


# ------------------------------------------------------------------ reference (64 bits)
def ref_scores(l, score):
    l = l.double()
    if score == "sigmoid":
        return torch.sigmoid(l)
    m = l.amax(1, keepdim=True)
    p = torch.exp(l - torch.where(torch.isfinite(m), m, torch.zeros_like(m)))
    z = p.sum(1, keepdim=True)
    return p / torch.where(z == 0, torch.ones_like(z), z)


def ref_forward(l, K, score, normalize, scale, bias=None):
    s = ref_scores(l, score)
    key = l.double() if bias is None else s + bias.double()
    key = torch.where(l.double() == NINF, torch.full_like(key, NINF), key)
    top = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :K]
    gone = key.gather(1, top) == NINF
    w = s.gather(1, top).masked_fill(gone, 0.0)
    if normalize:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    return top.masked_fill(gone, -1).to(torch.int32), w * scale


def ref_weights(l, top, score, normalize, scale):
    """Differentiable weights of a given table (-1 and out-of-range entries: 0)."""
    s = ref_scores(l, score)
    ok = (top >= 0) & (top < l.shape[1])
    w = s.gather(1, top.clamp(0, l.shape[1] - 1).long()) * ok
    if normalize:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    return w * scale


def ref_backward(l, top, gw, score, normalize, scale):
    l = l.double().clone().requires_grad_(True)
    ok = (top >= 0) & (top < l.shape[1])
    w = ref_weights(l, top, score, normalize, scale)
    (w * torch.where(ok, gw.double(), torch.zeros_like(gw.double()))).sum().backward()
    return torch.nan_to_num(l.grad, nan=0.0)     # 0 * inf at -inf logits: the gradient there is 0


# ------------------------------------------------------------------ CPU
def test_reference_gradient_matches_differences():
    g = torch.Generator().manual_seed(3)
    l = torch.randn(4, 9, generator=g, dtype=torch.float64)
    gw = torch.randn(4, 3, generator=g, dtype=torch.float64)
    for score in ("softmax", "sigmoid"):
        for norm in (False, True):
            top, _ = ref_forward(l, 3, score, norm, 1.7)
            dl = ref_backward(l, top, gw, score, norm, 1.7)
            f = lambda q: float((ref_weights(q, top, score, norm, 1.7) * gw).sum())
            for i in ((0, 0), (1, 4), (3, 8), (2, int(top[2, 0]))):
                p, m = l.clone(), l.clone()
                p[i] += 1e-6
                m[i] -= 1e-6
                assert abs((f(p) - f(m)) / 2e-6 - float(dl[i])) < 1e-7


PTR = 1 << 20


def _problem(tokens=4, experts=8, topk=2, score=mk.MOE_ROUTER_SOFTMAX, dtype=mk.MOE_FP32, flags=0, scale=1.0, ld=None):
    return mk.moe_router_problem(tokens, experts, topk, score, dtype, flags, scale, experts if ld is None else ld)


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=-1), mk.MOE_ERR_SHAPE), (dict(tokens=(1 << 27) + 1), mk.MOE_ERR_SHAPE), (dict(experts=0), mk.MOE_ERR_SHAPE),
    (dict(experts=256), mk.MOE_ERR_SHAPE), (dict(topk=0), mk.MOE_ERR_SHAPE), (dict(topk=9, experts=16), mk.MOE_ERR_SHAPE),
    (dict(topk=5, experts=4), mk.MOE_ERR_SHAPE), (dict(score=0), mk.MOE_ERR_UNSUPPORTED), (dict(score=3), mk.MOE_ERR_UNSUPPORTED),
    (dict(dtype=mk.MOE_MXFP8_E4M3), mk.MOE_ERR_DTYPE), (dict(flags=2), mk.MOE_ERR_UNSUPPORTED),
    (dict(scale=float("nan")), mk.MOE_ERR_UNSUPPORTED), (dict(scale=float("inf")), mk.MOE_ERR_UNSUPPORTED),
    (dict(ld=7), mk.MOE_ERR_LAYOUT)])
def test_bad_problems_are_refused(kw, status):
    p = _problem(**kw)
    assert mk.moe_router_forward(p, PTR, None, PTR, PTR, None) == status
    assert mk.moe_router_backward(p, PTR, PTR, PTR, PTR, 256, None) == status


def test_bad_arguments_are_refused():
    p = _problem()
    f, b = mk.moe_router_forward, mk.moe_router_backward
    assert mk.load().moe_router_forward(None, None, None, None, None, None) == mk.MOE_ERR_NULL
    for i in range(3):
        a = [PTR, PTR, PTR]
        a[i] = None
        assert f(p, a[0], None, a[1], a[2], None) == mk.MOE_ERR_NULL
    for i in range(4):
        a = [PTR] * 4
        a[i] = None
        assert b(p, *a, 8, None) == mk.MOE_ERR_NULL
    assert f(p, PTR + 2, None, PTR, PTR, None) == mk.MOE_ERR_LAYOUT
    assert f(p, PTR, PTR + 2, PTR, PTR, None) == mk.MOE_ERR_LAYOUT
    assert f(p, PTR, None, PTR + 1, PTR, None) == mk.MOE_ERR_LAYOUT
    assert f(_problem(dtype=mk.MOE_BF16), PTR + 1, None, PTR, PTR, None) == mk.MOE_ERR_LAYOUT
    assert b(p, PTR, PTR, PTR, PTR, 7, None) == mk.MOE_ERR_LAYOUT
    assert b(p, PTR, PTR, PTR, PTR + 2, 8, None) == mk.MOE_ERR_LAYOUT
    assert f(_problem(tokens=0), None, None, None, None, None) == mk.MOE_OK
    assert b(_problem(tokens=0), None, None, None, None, 8, None) == mk.MOE_OK


def test_binding_refuses_host_and_mismatched_tensors():
    r = mk.Router(8, 2)
    l, top, w = torch.zeros(3, 8), torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, 2)
    for args, status in (((l, top, w), mk.MOE_ERR_LAYOUT), ((l.double(), top, w), mk.MOE_ERR_DTYPE),
                         ((l[:, :7], top, w), mk.MOE_ERR_SHAPE), ((l[0], top, w), mk.MOE_ERR_SHAPE),
                         ((None, top, w), mk.MOE_ERR_NULL)):
        with pytest.raises(mk.MoeError) as ei:
            r.forward(*args)
        assert ei.value.status == status
    for kw, status in ((dict(experts=300, topk=2), mk.MOE_ERR_SHAPE), (dict(experts=8, topk=9), mk.MOE_ERR_SHAPE),
                       (dict(experts=8, topk=2, score="relu"), mk.MOE_ERR_UNSUPPORTED),
                       (dict(experts=8, topk=2, dtype=torch.float16), mk.MOE_ERR_DTYPE)):
        with pytest.raises(mk.MoeError) as ei:
            mk.Router(**kw)
        assert ei.value.status == status


# ------------------------------------------------------------------ GPU
SIZES = [(1, 1, 1), (1, 8, 8), (5, 2, 2), (17, 3, 1), (33, 16, 4), (100, 17, 8), (64, 32, 5), (1000, 33, 3), (257, 64, 6),
         (96, 65, 8), (4096, 96, 4), (31, 127, 7), (16, 128, 8), (77, 129, 2), (300, 255, 8)]


def logits_of(T, E, dtype, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    l = torch.randn(T, E, generator=g) * 2
    l = l.to(dtype)
    if T > 2:
        l[T // 2] = l[T // 2, 0]                     # a row of ties
        l[T // 3, ::2] = NINF                        # unavailable experts
        l[T - 1] = NINF                              # nothing available
    if T > 20:
        l[7, 1:] = NINF                              # one expert left
        l[9, 0], l[9, 1:2] = 0.0, -0.0               # signed zeros tie
    buf = torch.full((T, E + pad), float("nan"), dtype=dtype)
    buf[:, :E] = l
    return l, buf.cuda()[:, :E]


def rng_of(l, score):
    f = torch.where(torch.isfinite(l), l.float(), torch.zeros_like(l.float())).double()
    return (f.amax(1, keepdim=True) - f.amin(1, keepdim=True)) if score == "softmax" else f.abs().amax(1, keepdim=True)


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("with_bias", [False, True])
def test_forward_matches_formula(gpu_lib, score, dtype, with_bias):
    for i, (T, E, K) in enumerate(SIZES):
        normalize, scale, pad = i % 2 == 0, [1.0, 2.5][i % 2], [0, 3, 0][i % 3]
        l, lv = logits_of(T, E, dtype, seed=i, pad=pad)
        bias = 0.1 * torch.randn(E, generator=torch.Generator().manual_seed(50 + i)) if with_bias else None
        top = torch.full((T + 1, K), -7, dtype=torch.int32, device="cuda")
        w = torch.full((T + 1, K), float("nan"), device="cuda")
        mk.Router(E, K, score=score, normalize=normalize, scale=scale, dtype=dtype).forward(
            lv, top[:T], w[:T], expert_bias=None if bias is None else bias.cuda())
        torch.cuda.synchronize()
        rt, rw = ref_forward(l, K, score, normalize, scale, bias)
        assert torch.equal(top[:T].cpu(), rt), (T, E, K)
        tol = (rng_of(l, score) + 64) * U * rw.abs() + 1e-30
        assert bool(((w[:T].cpu().double() - rw).abs() <= tol).all()), (T, E, K)
        assert bool((top[T] == -7).all()) and bool(torch.isnan(w[T]).all())     # behind the last row


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("normalize", [False, True])
def test_backward_matches_formula(gpu_lib, score, dtype, normalize):
    half = 2.0 ** -8 if dtype == torch.bfloat16 else U
    for i, (T, E, K) in enumerate(SIZES):
        scale, pad = [1.0, 2.5][i % 2], [0, 5, 0][i % 3]
        l, lv = logits_of(T, E, dtype, seed=20 + i, pad=pad)
        top, _ = ref_forward(l, K, score, normalize, scale)
        gw = torch.randn(T, K, generator=torch.Generator().manual_seed(i))
        if T > 30 and K > 1:
            top[3, 0] = -1
            top[4, 1] = top[4, 0]            # listed twice: both gradients
            top[5, 0] = E + 3                # outside: skipped
            gw[3, 0] = gw[5, 0] = float("nan")
        out = torch.full((T + 1, E + pad), float("nan"), dtype=dtype, device="cuda")
        mk.Router(E, K, score=score, normalize=normalize, scale=scale, dtype=dtype).backward(
            lv, top.cuda(), gw.cuda(), out[:T, :E])
        torch.cuda.synchronize()
        ref = ref_backward(l, top, gw, score, normalize, scale)
        # magnitudes of the terms that are added up in each element
        s = ref_scores(l, score)
        ok = (top >= 0) & (top < E)
        ga = torch.where(ok, gw.abs().double(), torch.zeros(T, K, dtype=torch.float64)) * scale
        ds = torch.zeros(T, E, dtype=torch.float64).scatter_add_(1, top.clamp(0, E - 1).long(), ga)
        cnt = torch.zeros(T, E, dtype=torch.float64).scatter_add_(1, top.clamp(0, E - 1).long(), ok.double())
        if normalize:
            S = (cnt * s).sum(1, keepdim=True) + 1e-20
            ds = (ds + cnt * (ds * s).sum(1, keepdim=True) / S) / S
        mag = s * (ds + ds.mul(s).sum(1, keepdim=True)) if score == "softmax" else ds * s * (1 - s)
        tol = (4 * rng_of(l, score) + 192) * U * mag + 1e-30
        tol = tol + half * (ref.abs() + tol)
        got = out[:T, :E].cpu().double()
        assert bool(((got - ref).abs() <= tol).all()), (T, E, K)
        assert bool(torch.isnan(out[T]).all()) and bool(torch.isnan(out[:, E:]).all())


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_close_keys_are_compared_in_64_bits(gpu_lib, score):
    """Keys s + bias that FP32 cannot tell apart: the bias is chosen as -s rounded to FP32, so the
    keys are the rounding errors (1e-8 and less) of every expert, in 64 bits all different."""
    E, K = 40, 6
    g = torch.Generator().manual_seed(4)
    base = torch.randn(1, E, generator=g)
    bias = -ref_scores(base, score)[0].float()
    l = torch.cat([base, torch.randn(60, E, generator=g), base, base])
    l[3] = 0.0                                        # equal scores: the bias decides, in order
    l[-1, 5:9] = l[-1, 5]                             # some equal logits beside unequal biases
    for b in (bias, torch.zeros(E), bias + 0.25):
        rt, _ = ref_forward(l, K, score, True, 1.0, b)
        top, w = torch.empty(63, K, dtype=torch.int32, device="cuda"), torch.empty(63, K, device="cuda")
        mk.Router(E, K, score=score, normalize=True).forward(l.cuda(), top, w, expert_bias=b.cuda())
        assert torch.equal(top.cpu(), rt)


@pytest.mark.gpu
def test_nan_rows(gpu_lib):
    l = torch.randn(4, 40, generator=torch.Generator().manual_seed(1))
    l[1, 5] = float("nan")
    l[2] = float("nan")
    for score in ("softmax", "sigmoid"):
        for bias in (None, torch.zeros(40, device="cuda")):
            top = torch.empty(4, 3, dtype=torch.int32, device="cuda")
            w = torch.empty(4, 3, device="cuda")
            mk.Router(40, 3, score=score).forward(l.cuda(), top, w, expert_bias=bias)
            top, w = top.cpu(), w.cpu()
            rt, _ = ref_forward(l[[0, 3]], 3, score, False, 1.0)
            assert torch.equal(top[[0, 3]], rt) and bool(torch.isfinite(w[[0, 3]]).all())
            chosen = top[1] >= 0
            assert 5 not in top[1].tolist() and bool(torch.isnan(w[1][chosen]).all())
            if bias is None or score == "sigmoid":
                assert bool(chosen.all())
            assert bool((top[2] == -1).all()) and bool((w[2] == 0).all())


@pytest.mark.gpu
def test_graph_replay_and_side_stream(gpu_lib):
    T, E, K = 300, 96, 4
    l = torch.randn(T, E, device="cuda")
    gw = torch.randn(T, K, device="cuda")
    top, w, dl = (torch.empty(T, K, dtype=torch.int32, device="cuda"), torch.empty(T, K, device="cuda"),
                  torch.empty(T, E, device="cuda"))
    r = mk.Router(E, K, normalize=True)

    def step():
        r.forward(l, top, w)
        r.backward(l, top, gw, dl)

    outs = (top, w, dl)
    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        l.normal_()
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in outs]
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))

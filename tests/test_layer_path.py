"""The operators in a row, as a transformer block uses them around the layer: norm (with the
residual stream) -> router -> experts, forward and backward for training, and the few-token
forward for serving.

Training is compared with torch autograd of the same chain in 64 bits.  Tolerance: the layer's
own bound for BF16 weights is 2e-2 of the largest value; the norm's output and input gradient, the
logits' input and the sum of the two gradients that reach it are rounded to BF16 once each, 2^-8."""
import numpy as np
import pytest
import torch

import moe_inputs as gen
import moe_megakernel_amd as mk
from oracle import moe_oracle as O
from tests.gpu_parity_util import BF16_TOL, rel_err

CHAIN_TOL = BF16_TOL + 4 * 2.0 ** -8
SCALE = 1.5


def build(T, H, E, K, I, seed=70, **kw):
    from moe_inputs.device import DeviceProblem
    cfg = gen.custom(T, H, E, K, I, backward=True, idx=seed)
    top = np.zeros((T, K), np.int32) - 1
    dp = DeviceProblem(cfg, routing_table=(top, np.zeros((T, K), np.float32)), **kw)
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)
    t = dict(x=rn(T, H), res=rn(T, H), w=1 + 0.1 * rn(H), b=0.1 * rn(H))
    t = {k: v.to(torch.bfloat16).cuda() for k, v in t.items()}
    t["wr"] = (rn(E, H) * 0.1).cuda()                           # router weight, FP32
    return dp, t


def expert_weights(dp):
    I = dp.cfg.inter
    W = O.Weights.from_bits(I, dp.np_s1, dp.np_s2, lambda e: dp.np_routed[e], "bf16")
    f = lambda mats: [torch.from_numpy(np.ascontiguousarray(m)) for m in mats]
    return f(W.shared), [f(W.routed(e)) for e in range(dp.cfg.experts)]


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_training_step(gpu_lib, score):
    T, H, E, K, I = 96, 256, 8, 2, 128
    dp, t = build(T, H, E, K, I)
    norm, router = mk.Norm(H), mk.Router(E, K, score=score, normalize=True, scale=SCALE)
    bf = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")
    s, hidden, stats = bf(T, H), bf(T, H), torch.empty(T, 2, device="cuda")
    top, rw = torch.empty(T, K, dtype=torch.int32, device="cuda"), torch.empty(T, K, device="cuda")
    norm.forward(t["x"], t["w"], t["b"], hidden, stats, residual=t["res"], sum=s)
    logits = hidden.float() @ t["wr"].T
    router.forward(logits, top, rw)
    dp.layer.forward_topk(hidden, top, rw, dp.weights, dp.out)
    # the block's output is s + experts(norm(s)); its gradient dy reaches both
    dy = dp.dy
    dp.layer.backward(dy, hidden, dp.weights, dp.dx, dp.dprobs, dp.main_grads)
    dlogits = torch.empty_like(logits)
    router.backward(logits, top, dp.dprobs, dlogits)
    dhidden = (dp.dx.float() + dlogits @ t["wr"]).to(torch.bfloat16)
    dwr = dlogits.T @ hidden.float()
    ds, dw, db = bf(T, H), torch.zeros(H, device="cuda"), torch.zeros(H, device="cuda")
    norm.backward(dhidden, s, t["w"], stats, ds, dw, db, grad_sum=dy)
    torch.cuda.synchronize()

    d = {k: v.double().cpu().requires_grad_(True) for k, v in t.items() if k not in ("x", "res")}
    s64 = s.double().cpu().requires_grad_(True)
    mu, var = s64.mean(1, keepdim=True), s64.var(1, unbiased=False, keepdim=True)
    h64 = (s64 - mu) / torch.sqrt(var + 1e-5) * d["w"] + d["b"]
    l64 = h64 @ d["wr"].T
    sc = torch.softmax(l64, 1) if score == "softmax" else torch.sigmoid(l64)
    chosen = top.cpu().long()
    w64 = sc.gather(1, chosen)
    w64 = SCALE * w64 / w64.sum(1, keepdim=True)
    shared, routed = expert_weights(dp)
    ffn = lambda rows, m: (torch.nn.functional.silu(rows @ m[0].T) * (rows @ m[1].T)) @ m[2].T
    out = ffn(h64, shared)
    for e in range(E):
        r, k = (chosen == e).nonzero(as_tuple=True)
        out = out.index_add(0, r, w64[r, k][:, None] * ffn(h64[r], routed[e]))
    ((out + s64) * dy.double().cpu()).sum().backward()

    got = dict(out=(dp.out, out), weights=(rw, w64), ds=(ds, s64.grad), dw=(dw, d["w"].grad), db=(db, d["b"].grad),
               dwr=(dwr, d["wr"].grad))
    for name, (a, b) in got.items():
        assert rel_err(a.detach().double().cpu().numpy(), b.detach().numpy()) <= CHAIN_TOL, name


@pytest.mark.gpu
def test_serving_step_captured(gpu_lib):
    """norm -> router -> few-token forward in one graph, replayed on new tokens."""
    T, H, E, K, I = 5, 384, 16, 4, 256
    dp, t = build(T, H, E, K, I, seed=71)
    norm, router, layer = mk.Norm(H, kind="rms"), mk.Router(E, K, score="sigmoid", normalize=True), mk.DecodeLayer(dp.p)
    s, hidden = torch.empty_like(t["x"]), torch.empty_like(t["x"])
    top, rw = torch.empty(T, K, dtype=torch.int32, device="cuda"), torch.empty(T, K, device="cuda")
    logits, out = torch.empty(T, E, device="cuda"), torch.empty_like(t["x"])
    bias = torch.linspace(-0.1, 0.1, E, device="cuda")
    wrt = t["wr"].T.contiguous()

    def step():
        norm.forward(t["x"], t["w"], None, hidden, residual=t["res"], sum=s)
        torch.mm(hidden.float(), wrt, out=logits)
        router.forward(logits, top, rw, expert_bias=bias)
        layer.forward(hidden, top, rw, dp.weights, out)

    step()
    torch.cuda.synchronize()
    # the training forward on the same table agrees
    dp.layer.forward_topk(hidden, top, rw, dp.weights, dp.out)
    torch.cuda.synchronize()
    assert rel_err(out.double().cpu().numpy(), dp.out.double().cpu().numpy()) <= BF16_TOL
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        t["x"].copy_(torch.randn(T, H, device="cuda"))
        step()
        torch.cuda.synchronize()
        want = [v.clone() for v in (s, hidden, top, rw, out)]
        for v in (s, hidden, top, rw, out):
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((s, hidden, top, rw, out), want)), i
        assert int(layer.status_word()) == 0


def test_options_are_fixed_at_construction():
    """What a caller writes into `p` of an operator changes no call, of a size met before or not."""
    def decode():
        return mk.DecodeLayer(mk.problem(8, 256, 128, 8, 2, flags=mk.MOE_FLAG_TOPK_ROUTING), device="cpu")

    for op, first, later, field in ((decode(), (2,), (3,), "swiglu_limit"), (mk.Norm(64, device="cpu"), (2, 0), (3, 0), "eps"),
                                    (mk.Router(8, 2), (2, 8), (3, 8), "scale")):
        before = getattr(op._problems[first], field)
        setattr(op.p, field, 7.0)
        assert getattr(op._problems[first], field) == getattr(op._problems[later], field) == before
        assert getattr(op.p, field) == before

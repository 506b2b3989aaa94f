"""Measured cases of the operators around the post-router MoE layer: the layer for a few
tokens (serving), the norm in front of it (forward and backward) and the router's choice of
experts (forward and backward).

`run` computes a case in its plain form, elementary torch operations in 32 bits (64 for
router scores that are compared with each other), or, where `own` is true, through the
library's entry points.  `exact` is the operator's definition in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
_ROUTER_EPS = 1e-20


# ------------------------------------------------------------------------- cases
def listed():
    return [
        # one token of a chat: the 4096-wide 96-expert top-4 layer with its shared expert
        _decode("decode_1_bf16", T=1, H=4096, I=1024, E=96, K=4, routed="bf16", layout="single", shared=True),
        # a handful of streams, MXFP8 experts in allocations of their own, gated shared expert
        _decode("decode_7_mxfp8", T=7, H=4096, I=1024, E=96, K=4, routed="mxfp8", layout="table", shared=True,
                gate=True, clamp=1.5),
        # a ragged batch in which some routes were dropped, routed experts only
        _decode("decode_19_bf16_short", T=19, H=4096, I=1024, E=96, K=4, routed="bf16", layout="single",
                shared=False, missing=0.1),
        # the largest batch on the wide 64-expert top-6 layer
        _decode("decode_64_mxfp8_wide", T=64, H=7168, I=2048, E=64, K=6, routed="mxfp8", layout="single",
                shared=True),
        # one generated token: the norm's latency
        _norm("norm_fwd_1", "norm_fwd", rows=1, cols=4096, kind="layer", dtype="bf16", param="bf16", bias=True),
        # training forward: residual added on the way, 8192 x 7168
        _norm("norm_fwd_8192_residual", "norm_fwd", rows=8192, cols=7168, kind="rms", dtype="bf16", param="bf16",
              residual=True),
        # training backward of the 4096-token layer, weight and bias gradients included
        _norm("norm_bwd_4096", "norm_bwd", rows=4096, cols=4096, kind="layer", dtype="bf16", param="bf16", bias=True),
        # FP32 rows of an odd length at an odd stride
        _norm("norm_bwd_odd_fp32", "norm_bwd", rows=1023, cols=2055, kind="layer", dtype="fp32", param="fp32",
              bias=True, pad=2, residual=True),
        # one step of a small serving batch: the router's latency
        _router("router_fwd_19", "router_fwd", tokens=19, experts=96, topk=4, score="softmax", dtype="fp32",
                normalize=True),
        # sigmoid scores with a balancing bias, several sequences at once
        _router("router_fwd_65536", "router_fwd", tokens=65536, experts=64, topk=6, score="sigmoid", dtype="fp32",
                normalize=True, bias=True, scale=2.5),
        # training backward of the 4096-token layer's router
        _router("router_bwd_4096", "router_bwd", tokens=4096, experts=96, topk=4, score="softmax", dtype="fp32",
                normalize=True),
        # BF16 logits, raw softmax probabilities as weights, an odd expert count at a padded stride
        _router("router_bwd_65536_bf16", "router_bwd", tokens=65536, experts=97, topk=8, score="softmax",
                dtype="bf16", pad=3),
    ]


def _decode(name, *, T, H, I, E, K, routed, layout, shared, gate=False, clamp=0.0, missing=0.0):
    return dict(name=name, op="decode", T=T, H=H, I=I, E=E, K=K, routed=routed, layout=layout, shared=shared,
                gate=gate, clamp=clamp, missing=missing)


def _norm(name, op, *, rows, cols, kind, dtype, param, bias=False, residual=False, pad=0):
    return dict(name=name, op=op, rows=rows, cols=cols, kind=kind, dtype=dtype, param=param, bias=bias,
                residual=residual, pad=pad)


def _router(name, op, *, tokens, experts, topk, score, dtype, normalize=False, bias=False, scale=1.0, pad=0):
    return dict(name=name, op=op, tokens=tokens, experts=experts, topk=topk, score=score, dtype=dtype,
                normalize=normalize, bias=bias, scale=scale, pad=pad)


def _log_int(rng, lo, hi):
    return int(min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))))))


def draw(rng):
    op = rng.choice(["decode", "decode", "norm_fwd", "norm_bwd", "router_fwd", "router_bwd"])
    if op == "decode":
        most = max(work(c)["bytes"] for c in listed() if c["op"] == "decode")
        while True:
            E = _log_int(rng, 4, 128)
            shared = rng.random() < 0.7
            c = _decode("", T=_log_int(rng, 1, 64), H=128 * _log_int(rng, 2, 56), I=128 * _log_int(rng, 1, 16), E=E,
                        K=rng.randint(1, min(8, E)), routed=rng.choice(["bf16", "mxfp8"]),
                        layout=rng.choice(["single", "table"]), shared=shared, gate=shared and rng.random() < 0.3,
                        clamp=rng.choice([0.0, 0.0, 1.5]), missing=rng.choice([0.0, 0.0, 0.15]))
            if work(c)["bytes"] <= most and c["E"] * c["I"] * c["H"] <= 64 * 2048 * 7168:
                break
    elif op.startswith("norm"):
        while True:
            c = _norm("", op, rows=_log_int(rng, 1, 16384), cols=_log_int(rng, 8, 10240),
                      kind=rng.choice(["layer", "rms"]), dtype=rng.choice(["bf16", "fp32"]),
                      param=rng.choice(["bf16", "fp32"]), bias=rng.random() < 0.5, residual=rng.random() < 0.4,
                      pad=rng.choice([0, 0, 1, 8]))
            if rng.random() < 0.5:      # widths of real models are multiples of 128
                c["cols"] = 128 * max(1, c["cols"] // 128)
            if c["rows"] * c["cols"] * (2 if c["dtype"] == "fp32" else 1) <= 8192 * 7168:
                break
    else:
        E = _log_int(rng, 2, 255)
        c = _router("", op, tokens=_log_int(rng, 1, 65536), experts=E, topk=rng.randint(1, min(8, E)),
                    score=rng.choice(["softmax", "sigmoid"]), dtype=rng.choice(["fp32", "bf16"]),
                    normalize=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]), pad=rng.choice([0, 0, 3]))
        c["bias"] = op == "router_fwd" and rng.random() < 0.4
        c["normalize"] &= c["topk"] > 1     # a single normalised weight is constant
        if c["tokens"] * c["experts"] > 65536 * 97:
            c["tokens"] = 65536 * 97 // c["experts"]
    del c["name"]
    return c


# ------------------------------------------------------------------------- inputs
_TORCH = {"bf16": torch.bfloat16, "fp32": torch.float32}
_SIZE = {"bf16": 2, "fp32": 4}


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _mx_quantize(w):
    """[rows][cols] floats -> E4M3 codes and E8M0 scale bytes, blocks of 32 along cols: the
    smallest exponent that brings a block's largest magnitude to at most 448."""
    b = w.view(w.shape[0], -1, 32)
    m, e = torch.frexp(b.abs().amax(-1))                 # amax = m 2^e, m in [0.5, 1)
    e = e - 9 + (m > 0.875).to(e.dtype)                  # 448 = 0.875 2^9
    q = (b * torch.ldexp(torch.ones_like(m), -e)[..., None]).to(torch.float8_e4m3fn)
    return q.view(w.shape).view(torch.uint8), (e + 127).to(torch.uint8)


def _prepare_decode(c, seed):
    T, H, I, E, K = c["T"], c["H"], c["I"], c["E"], c["K"]
    g = _gen(seed)
    rn = lambda *s: torch.randn(*s, device=DEV, generator=g)
    st = {"case": c, "x": rn(T, H).to(torch.bfloat16)}
    top_w, top = torch.softmax(rn(T, E), -1).topk(K, dim=-1)
    top_w = top_w / top_w.sum(-1, keepdim=True)
    gone = torch.rand(T, K, device=DEV, generator=g) < c["missing"]
    st["top"] = torch.where(gone, torch.full_like(top, -1), top).to(torch.int32).contiguous()
    st["rw"] = top_w.contiguous()
    if c["routed"] == "bf16":
        st["w1"] = torch.empty(E, 2 * I, H, dtype=torch.bfloat16, device=DEV)
        st["w2"] = torch.empty(E, H, I, dtype=torch.bfloat16, device=DEV)
        for e in range(E):
            st["w1"][e] = rn(2 * I, H) * 0.02
            st["w2"][e] = rn(H, I) * 0.02
    else:
        st["w1"] = torch.empty(E, 2 * I, H, dtype=torch.uint8, device=DEV)
        st["w2"] = torch.empty(E, H, I, dtype=torch.uint8, device=DEV)
        st["s1"] = torch.empty(E, 2 * I, H // 32, dtype=torch.uint8, device=DEV)
        st["s2"] = torch.empty(E, H, I // 32, dtype=torch.uint8, device=DEV)
        for e in range(E):
            st["w1"][e], st["s1"][e] = _mx_quantize(rn(2 * I, H) * 0.02)
            st["w2"][e], st["s2"][e] = _mx_quantize(rn(H, I) * 0.02)
    if c["shared"]:
        st["sw1"] = (rn(2 * I, H) * 0.02).to(torch.bfloat16)
        st["sw2"] = (rn(H, I) * 0.02).to(torch.bfloat16)
        if c["gate"]:
            st["gate"] = (rn(H) * 0.02).to(torch.bfloat16)
    if own:
        import moe_megakernel_amd as mk
        mx = c["routed"] == "mxfp8"
        dt = mk.MOE_MXFP8_E4M3 if mx else mk.MOE_BF16
        keep = []

        def routed(t):
            if t is None:
                return None
            if c["layout"] == "single":
                return mk.mat(base=t, expert_stride=t.shape[1] * t.shape[2], ld=t.shape[2])
            tab = torch.tensor([int(t[e].data_ptr()) for e in range(E)], dtype=torch.int64, device=DEV)
            keep.append(tab)
            return mk.mat(table=tab, ld=t.shape[2])

        m1, m2 = routed(st["w1"]), routed(st["w2"])
        z1, z2 = routed(st.get("s1")), routed(st.get("s2"))
        w = mk.moe_weights()
        w.routed_gate = mk.weight(dt, I, H, m1, row_offset=0, scale=z1)
        w.routed_up = mk.weight(dt, I, H, m1, row_offset=I, scale=z1)
        w.routed_down = mk.weight(dt, H, I, m2, scale=z2)
        flags = mk.MOE_FLAG_TOPK_ROUTING
        if c["shared"]:
            flags |= mk.MOE_FLAG_HAS_SHARED
            w.shared_gate = mk.weight(mk.MOE_BF16, I, H, mk.mat(base=st["sw1"], ld=H))
            w.shared_up = mk.weight(mk.MOE_BF16, I, H, mk.mat(base=st["sw1"], ld=H), row_offset=I)
            w.shared_down = mk.weight(mk.MOE_BF16, H, I, mk.mat(base=st["sw2"], ld=I))
            if c["gate"]:
                flags |= mk.MOE_FLAG_SHARED_GATE
                w.shared_out_gate = mk.weight(mk.MOE_BF16, 1, H, mk.mat(base=st["gate"], ld=H))
        st["keep"], st["weights"] = keep, w
        st["layer"] = mk.DecodeLayer(mk.problem(T, H, I, E, K, dt, flags=flags, swiglu_limit=c["clamp"]), device=DEV)
        st["out"] = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    return st


def _rows(t, pad):
    """t with `pad` unused elements after every row."""
    if not pad:
        return t.contiguous()
    buf = torch.zeros(t.shape[0], t.shape[1] + pad, dtype=t.dtype, device=t.device)
    buf[:, :t.shape[1]] = t
    return buf[:, :t.shape[1]]


def _prepare_norm(c, seed):
    R, N, dt, pt = c["rows"], c["cols"], _TORCH[c["dtype"]], _TORCH[c["param"]]
    g = _gen(seed)
    rn = lambda *s: torch.randn(*s, device=DEV, generator=g)
    st = {"case": c, "eps": 1e-5}
    # a residual stream: each row with a scale and an offset of its own
    st["x"] = _rows((rn(R, N) * torch.exp(0.5 * rn(R, 1)) + 0.3 * rn(R, 1)).to(dt), c["pad"])
    st["w"] = (1.0 + 0.1 * rn(N)).to(pt)
    st["b"] = (0.1 * rn(N)).to(pt) if c["bias"] else None
    st["res"] = st["gsum"] = None
    if c["op"] == "norm_fwd":
        if c["residual"]:
            st["res"] = _rows(rn(R, N).to(dt), c["pad"])
    else:
        st["dy"] = _rows(rn(R, N).to(dt), c["pad"])
        if c["residual"]:
            st["gsum"] = _rows(rn(R, N).to(dt), c["pad"])
        x = st["x"].float()
        mu = x.mean(-1, keepdim=True) if c["kind"] == "layer" else torch.zeros(R, 1, device=DEV)
        st["stats"] = torch.cat([mu, torch.rsqrt(((x - mu) ** 2).mean(-1, keepdim=True) + st["eps"])], 1).contiguous()
    if own:
        import moe_megakernel_amd as mk
        st["op"] = mk.Norm(N, kind=c["kind"], eps=st["eps"], dtype=dt, param_dtype=pt, device=DEV)
        if c["op"] == "norm_fwd":
            st["y"] = _rows(torch.empty(R, N, dtype=dt, device=DEV), c["pad"])
            st["sum"] = _rows(torch.empty(R, N, dtype=dt, device=DEV), c["pad"]) if c["residual"] else None
            st["stats"] = torch.empty(R, 2, dtype=torch.float32, device=DEV)
        else:
            st["dx"] = _rows(torch.empty(R, N, dtype=dt, device=DEV), c["pad"])
            st["dw"] = torch.empty(N, dtype=torch.float32, device=DEV)
            st["db"] = torch.empty(N, dtype=torch.float32, device=DEV) if c["bias"] else None
    return st


def _prepare_router(c, seed):
    T, E, K = c["tokens"], c["experts"], c["topk"]
    g = _gen(seed)
    logits = torch.randn(T, E, device=DEV, generator=g) * 1.5
    st = {"case": c, "logits": _rows(logits.to(_TORCH[c["dtype"]]), c["pad"])}
    st["bias"] = 0.05 * torch.randn(E, device=DEV, generator=g) if c["bias"] else None
    if c["op"] == "router_bwd":
        st["top"] = _choose(st["logits"].float(), K).to(torch.int32).contiguous()
        st["gw"] = torch.randn(T, K, device=DEV, generator=g)
    if own:
        import moe_megakernel_amd as mk
        st["op"] = mk.Router(E, K, score=c["score"], normalize=c["normalize"], scale=c["scale"],
                             dtype=_TORCH[c["dtype"]])
        if c["op"] == "router_fwd":
            st["top"] = torch.empty(T, K, dtype=torch.int32, device=DEV)
            st["rw"] = torch.empty(T, K, dtype=torch.float32, device=DEV)
        else:
            st["dl"] = _rows(torch.empty(T, E, dtype=_TORCH[c["dtype"]], device=DEV), c["pad"])
    return st


def prepare(case, seed):
    op = case["op"]
    if op == "decode":
        return _prepare_decode(case, seed)
    return _prepare_norm(case, seed) if op.startswith("norm") else _prepare_router(case, seed)


# ------------------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    return {"decode": _run_decode, "norm_fwd": _run_norm_fwd, "norm_bwd": _run_norm_bwd,
            "router_fwd": _run_router_fwd, "router_bwd": _run_router_bwd}[op](state)


def _mx_decode(codes, scale):
    """E4M3 codes and E8M0 scales -> float32 (exact: scales lie well inside the exponent range)."""
    v = codes.view(torch.float8_e4m3fn).float()
    s = (scale.to(torch.int32) << 23).view(torch.float32)
    return (v.view(*scale.shape, 32) * s[..., None]).view(v.shape)


def _swiglu(ab, I, L):
    a, b = ab[..., :I], ab[..., I:]
    if L > 0:
        a, b = a.clamp(max=L), b.clamp(-L, L)
    return a / (1.0 + torch.exp(-a)) * b


def _run_decode(st):
    c = st["case"]
    if own:
        return st["layer"].forward(st["x"], st["top"], st["rw"], st["weights"], st["out"])
    T, I, E, K, L = c["T"], c["I"], c["E"], c["K"], c["clamp"]
    mx = c["routed"] == "mxfp8"
    x = st["x"].float()
    out = torch.zeros(T, c["H"], device=DEV)

    def pick(key, skey, idx):
        w = st[key][idx] if isinstance(idx, int) else st[key].index_select(0, idx)[0]
        if not mx:
            return w.float()
        return _mx_decode(w, st[skey][idx] if isinstance(idx, int) else st[skey].index_select(0, idx)[0])

    if T * K < E:       # fewer routes than experts: fetch each route's expert
        for t in range(T):
            for k in range(K):
                e = st["top"][t, k:k + 1].long()
                w = torch.where(e < 0, torch.zeros_like(st["rw"][t, k:k + 1]), st["rw"][t, k:k + 1])
                e = e.clamp(min=0)
                h = _swiglu(x[t:t + 1] @ pick("w1", "s1", e).T, I, L)
                out[t:t + 1] += w * (h @ pick("w2", "s2", e).T)
    else:               # every expert on every token, masked by its weight
        for e in range(E):
            w = (st["rw"] * (st["top"] == e)).sum(-1, keepdim=True)
            h = _swiglu(x @ pick("w1", "s1", e).T, I, L)
            out += w * (h @ pick("w2", "s2", e).T)
    if c["shared"]:
        s = _swiglu(x @ st["sw1"].float().T, I, L) @ st["sw2"].float().T
        if c["gate"]:
            s = s / (1.0 + torch.exp(-(x @ st["gate"].float())))[:, None]
        out += s
    return out.to(torch.bfloat16)


def _run_norm_fwd(st):
    c = st["case"]
    if own:
        st["op"].forward(st["x"], st["w"], st["b"], st["y"], st["stats"], residual=st["res"], sum=st["sum"])
        return [st["y"], st["stats"]] + ([st["sum"]] if st["sum"] is not None else [])
    x, outs = st["x"].float(), []
    if st["res"] is not None:
        s = (x + st["res"].float()).to(st["x"].dtype)
        outs, x = [s], s.float()
    mu = x.mean(-1, keepdim=True) if c["kind"] == "layer" else torch.zeros(c["rows"], 1, device=DEV)
    d = x - mu
    rstd = 1.0 / torch.sqrt((d * d).mean(-1, keepdim=True) + st["eps"])
    y = d * rstd * st["w"].float()
    if st["b"] is not None:
        y = y + st["b"].float()
    return [y.to(st["x"].dtype), torch.cat([mu, rstd], 1)] + outs


def _run_norm_bwd(st):
    c = st["case"]
    if own:
        st["op"].backward(st["dy"], st["x"], st["w"], st["stats"], st["dx"], st["dw"], st["db"],
                          grad_sum=st["gsum"], overwrite=True)
        return [st["dx"], st["dw"]] + ([st["db"]] if st["db"] is not None else [])
    dy, mu, rstd = st["dy"].float(), st["stats"][:, :1], st["stats"][:, 1:]
    xh = (st["x"].float() - mu) * rstd
    g = dy * st["w"].float()
    dx = g - xh * (g * xh).mean(-1, keepdim=True)
    if c["kind"] == "layer":
        dx = dx - g.mean(-1, keepdim=True)
    dx = dx * rstd
    if st["gsum"] is not None:
        dx = dx + st["gsum"].float()
    out = [dx.to(st["x"].dtype), (dy * xh).sum(0)]
    return out + ([dy.sum(0)] if st["b"] is not None else [])


def _choose(key, K):
    """Indices of the K largest of each row, descending, ties to the lowest index."""
    return torch.sort(key, dim=-1, descending=True, stable=True).indices[:, :K]


def _scores(l, score):
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    p = torch.exp(l - l.amax(-1, keepdim=True))
    return p / p.sum(-1, keepdim=True)


def _run_router_fwd(st):
    c = st["case"]
    if own:
        st["op"].forward(st["logits"], st["top"], st["rw"], expert_bias=st["bias"])
        return [st["top"], st["rw"]]
    l = st["logits"].float()
    # the order of the scores is that of the logits; with a bias they are compared in 64 bits
    key = l if st["bias"] is None else _scores(l.double(), c["score"]) + st["bias"].double()
    top = _choose(key, c["topk"])
    w = _scores(l, c["score"]).gather(-1, top)
    if c["normalize"]:
        w = w / (w.sum(-1, keepdim=True) + _ROUTER_EPS)
    return [top.to(torch.int32), w * c["scale"]]


def _run_router_bwd(st):
    c = st["case"]
    if own:
        return st["op"].backward(st["logits"], st["top"], st["gw"], st["dl"])
    s, top = _scores(st["logits"].float(), c["score"]), st["top"].long()
    sk, g = s.gather(-1, top), st["gw"] * c["scale"]
    if c["normalize"]:
        S = sk.sum(-1, keepdim=True) + _ROUTER_EPS
        g = (g - (g * sk).sum(-1, keepdim=True) / S) / S
    ds = torch.zeros_like(s).scatter_(-1, top, g)
    dl = s * (ds - (ds * s).sum(-1, keepdim=True)) if c["score"] == "softmax" else ds * s * (1.0 - s)
    return dl.to(st["logits"].dtype)


# ------------------------------------------------------------------------- floor
def work(case):
    c = case
    if c["op"] == "decode":
        T, H, I, E, K = c["T"], c["H"], c["I"], c["E"], c["K"]
        kept = K * (1.0 - c["missing"])
        hit = E * (1.0 - (1.0 - kept / E) ** T)      # distinct experts expected
        per = 3 * H * I * (2 if c["routed"] == "bf16" else 1 + 1 / 32)
        b = hit * per + 4 * T * H + 8 * T * K + (6 * H * I if c["shared"] else 0) + (2 * H if c["gate"] else 0)
        return {"bytes": int(b), "flops": int(6 * H * I * T * (kept + (1 if c["shared"] else 0)))}
    if c["op"].startswith("norm"):
        R, N, z, p = c["rows"], c["cols"], _SIZE[c["dtype"]], _SIZE[c["param"]]
        if c["op"] == "norm_fwd":
            b = R * N * z * (4 if c["residual"] else 2) + N * p * (2 if c["bias"] else 1) + 8 * R
            return {"bytes": b, "flops": 8 * R * N}
        b = R * N * z * (4 if c["residual"] else 3) + N * p + 4 * N * (2 if c["bias"] else 1) + 8 * R
        return {"bytes": b, "flops": 13 * R * N}
    T, E, K, z = c["tokens"], c["experts"], c["topk"], _SIZE[c["dtype"]]
    if c["op"] == "router_fwd":
        return {"bytes": T * E * z + 8 * T * K + (4 * E if c["bias"] else 0), "flops": T * E * (4 + K)}
    return {"bytes": 2 * T * E * z + 8 * T * K, "flops": 8 * T * E}


# ------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    global own
    mine, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = mine
    op = case["op"]
    return {"decode": _exact_decode, "norm_fwd": _exact_norm_fwd, "norm_bwd": _exact_norm_bwd,
            "router_fwd": _exact_router_fwd, "router_bwd": _exact_router_bwd}[op](case, st)


def _exact_decode(c, st):
    x = st["x"].double()
    out = torch.zeros(c["T"], c["H"], dtype=torch.float64, device=DEV)

    def ffn(rows, w1, w2):
        gate, up = rows.matmul(w1[:c["I"]].t()), rows.matmul(w1[c["I"]:].t())
        if c["clamp"] > 0:
            gate, up = gate.minimum(torch.full_like(gate, c["clamp"])), up.clamp(-c["clamp"], c["clamp"])
        return (gate * torch.sigmoid(gate) * up).matmul(w2.t())

    def wide(key, skey, e):
        if c["routed"] == "bf16":
            return st[key][e].double()
        v = st[key][e].view(torch.float8_e4m3fn).double()
        s = torch.pow(torch.full_like(st[skey][e], 2, dtype=torch.float64), st[skey][e].double() - 127.0)
        return v * s.repeat_interleave(32, dim=-1)

    for e in range(c["E"]):
        t, k = (st["top"] == e).nonzero(as_tuple=True)
        if t.numel():
            out.index_add_(0, t, st["rw"][t, k].double()[:, None] * ffn(x[t], wide("w1", "s1", e), wide("w2", "s2", e)))
    if c["shared"]:
        s = ffn(x, st["sw1"].double(), st["sw2"].double())
        out += s * torch.sigmoid(x.matmul(st["gate"].double()))[:, None] if c["gate"] else s
    return out


def _exact_norm_fwd(c, st):
    x, outs = st["x"].double(), []
    if st["res"] is not None:       # the stored sum is what is normalised
        x = (x + st["res"].double()).to(st["x"].dtype).double()
        outs = [x]
    mu = x.sum(1) / c["cols"] if c["kind"] == "layer" else torch.zeros(c["rows"], dtype=torch.float64, device=DEV)
    var = (x - mu[:, None]).square().sum(1) / c["cols"]
    rstd = (var + st["eps"]).pow(-0.5)
    y = (x - mu[:, None]) * rstd[:, None] * st["w"].double()[None]
    if st["b"] is not None:
        y += st["b"].double()[None]
    return [y, torch.stack([mu, rstd], 1)] + outs


def _exact_norm_bwd(c, st):
    x, dy, n = st["x"].double(), st["dy"].double(), c["cols"]
    mu, rstd = st["stats"].double().unbind(1)
    xh = (x - mu[:, None]) * rstd[:, None]
    g = dy * st["w"].double()[None]
    inner = (g * xh).sum(1) / n
    mean = g.sum(1) / n if c["kind"] == "layer" else torch.zeros_like(inner)
    dx = rstd[:, None] * (g - mean[:, None] - xh * inner[:, None])
    if st["gsum"] is not None:
        dx = dx + st["gsum"].double()
    out = [dx, torch.einsum("rn,rn->n", dy, xh)]
    return out + ([dy.sum(0)] if st["b"] is not None else [])


def _exact_router_fwd(c, st):
    l = st["logits"].double()
    s = torch.sigmoid(l) if c["score"] == "sigmoid" else torch.softmax(l, -1)
    key = l if st["bias"] is None else s + st["bias"].double()
    top = torch.argsort(key, dim=-1, descending=True, stable=True)[:, :c["topk"]]
    w = torch.take_along_dim(s, top, 1)
    if c["normalize"]:
        w = w / (w.sum(1, keepdim=True) + _ROUTER_EPS)
    return [top.to(torch.int32), w * c["scale"]]


def _exact_router_bwd(c, st):
    l = st["logits"].double()
    s = torch.sigmoid(l) if c["score"] == "sigmoid" else torch.softmax(l, -1)
    chosen = torch.zeros_like(s).scatter_(1, st["top"].long(), 1.0)
    g = torch.zeros_like(s).scatter_(1, st["top"].long(), st["gw"].double()) * c["scale"]
    if c["normalize"]:
        S = (s * chosen).sum(1, keepdim=True) + _ROUTER_EPS
        g = chosen * (g / S - (g * s).sum(1, keepdim=True) / S ** 2)
    if c["score"] == "sigmoid":
        return g * s * (1.0 - s)
    return s * g - s * (s * g).sum(1, keepdim=True)

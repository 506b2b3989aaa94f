"""Measured cases of the dense operators next to the post-router MoE layer: the gated
feed-forward block (forward and backward), activation checkpoints in 8 bits and what the
block's backward makes of them, and the 8-bit matrix product with a scale for each block of
128 with its quantiser.

`run` computes a case in its plain form, elementary torch operations in 32 bits, or, where
`own` is true, through the library's entry points.  `exact` is the operator's definition in
64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------------- cases
def listed():
    return [
        # one generated token through a shared expert that the caller runs itself
        _ffn("ffn_fwd_1", "ffn_fwd", T=1, H=4096, I=1024),
        # a ragged serving batch through the wide layer's shared expert
        _ffn("ffn_fwd_37_wide", "ffn_fwd", T=37, H=7168, I=2048),
        # a short training micro-batch of a dense layer, its pre-activations kept in BF16
        _ffn("ffn_fwd_777_saved", "ffn_fwd", T=777, H=4096, I=12288, act="gelu", saved="bf16"),
        # training backward of a dense layer at 4096 tokens
        _ffn("ffn_bwd_4096", "ffn_bwd", T=4096, H=4096, I=12288, saved="bf16"),
        # a whole training step of the wide layer's shared expert on 8-bit checkpoints
        _ffn("ffn_step_8192_int8", "ffn_step", T=8192, H=7168, I=2048, saved="int8"),
        # a few rows put away and fetched: the calls' latency
        _ckpt("ckpt_19", rows=19, cols=4096, dtype="bf16"),
        # the wide layer's hidden states put away in the forward and fetched in the backward
        _ckpt("ckpt_8192", rows=8192, cols=7168, dtype="bf16"),
        # activations on their way into an 8-bit product
        _quant("fp8_quantize_8192", rows=8192, cols=7168, kind="rows", transpose=False),
        # a weight's transposed copy, for the data gradient, after an optimiser step
        _quant("fp8_quantize_weight_t", rows=4096, cols=7168, kind="tiles", transpose=True),
        # a small serving batch through one projection
        _matmul("fp8_matmul_19", M=19, N=7168, K=2048),
        # a projection of a long training batch
        _matmul("fp8_matmul_8192", M=8192, N=4096, K=7168),
        # the tokens of 96 experts, sorted by expert, some rows unused behind the last
        _matmul("fp8_matmul_96_groups", M=16384, N=2048, K=4096, groups=96, spare=37),
    ]


def _ffn(name, op, *, T, H, I, act="silu", saved="none"):
    return dict(name=name, op=op, T=T, H=H, I=I, act=act, saved=saved)


def _ckpt(name, *, rows, cols, dtype, pad=0):
    return dict(name=name, op="ckpt", rows=rows, cols=cols, dtype=dtype, pad=pad)


def _quant(name, *, rows, cols, kind, transpose, dtype="bf16"):
    return dict(name=name, op="quant", rows=rows, cols=cols, kind=kind, transpose=transpose, dtype=dtype)


def _matmul(name, *, M, N, K, groups=1, spare=0, scales="tiles", out="bf16"):
    return dict(name=name, op="matmul", M=M, N=N, K=K, groups=groups, spare=spare, scales=scales, out=out)


def _log_int(rng, lo, hi):
    return int(min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))))))


def draw(rng):
    op = rng.choice(["ffn_fwd", "ffn_fwd", "ffn_bwd", "ffn_step", "ckpt", "quant", "matmul", "matmul"])
    if op.startswith("ffn"):
        most = work(_ffn("", "ffn_bwd", T=4096, H=4096, I=12288))["flops"]
        while True:
            c = _ffn("", op, T=_log_int(rng, 1, 16384), H=64 * _log_int(rng, 4, 112), I=64 * _log_int(rng, 4, 192),
                     act=rng.choice(["silu", "gelu"]), saved=rng.choice(["bf16", "int8"]))
            if op == "ffn_fwd":
                c["saved"] = rng.choice(["none", "none", "bf16"])
                if rng.random() < 0.4:
                    c["T"] = _log_int(rng, 1, 64)
            if work(c)["flops"] <= most and c["H"] * c["I"] <= 4096 * 12288:
                break
    elif op == "ckpt":
        while True:
            c = _ckpt("", rows=_log_int(rng, 1, 32768), cols=_log_int(rng, 16, 12288), dtype=rng.choice(["bf16", "fp32"]),
                      pad=rng.choice([0, 0, 8, 1]))
            if rng.random() < 0.5:
                c["cols"] = 32 * max(1, c["cols"] // 32)
            if c["rows"] * c["cols"] * (2 if c["dtype"] == "fp32" else 1) <= 8192 * 7168:
                break
    elif op == "quant":
        while True:
            c = _quant("", rows=_log_int(rng, 1, 16384), cols=_log_int(rng, 16, 8192), kind=rng.choice(["rows", "tiles"]),
                       transpose=rng.random() < 0.5, dtype=rng.choice(["bf16", "bf16", "fp32"]))
            if rng.random() < 0.5:
                c["cols"] = 128 * max(1, c["cols"] // 128)
            if c["rows"] * c["cols"] * (2 if c["dtype"] == "fp32" else 1) <= 8192 * 7168:
                break
    else:
        while True:
            G = rng.choice([1, 1, _log_int(rng, 2, 96)])
            c = _matmul("", M=_log_int(rng, 1, 16384), N=_log_int(rng, 64, 8192), K=16 * _log_int(rng, 8, 512), groups=G,
                        spare=rng.choice([0, 0, 5]), scales="tiles" if G > 1 else rng.choice(["tiles", "tiles", "rows"]),
                        out=rng.choice(["bf16", "bf16", "fp32"]))
            if rng.random() < 0.5:      # widths of real models
                c["N"], c["K"] = 64 * max(1, c["N"] // 64), 128 * max(1, c["K"] // 128)
            if c["M"] * c["N"] * c["K"] <= 8192 * 4096 * 7168 and G * c["N"] * c["K"] <= 96 * 2048 * 4096:
                break
    del c["name"]
    return c


# ------------------------------------------------------------------------- formats
_TORCH = {"bf16": torch.bfloat16, "fp32": torch.float32}
_SIZE = {"bf16": 2, "fp32": 4}


def _up(n, k):
    return -(-n // k)


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _pow2(e):
    """2^e in 64 bits, exactly (torch's exp2 and pow on the GPU may be off by a rounding, which
    moves ties)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _int8(v):
    """Rows of floats -> 8-bit codes and exponent bytes in blocks of 32: the smallest exponent
    e in [-127, 127] that brings a block's largest magnitude to at most 127 2^(e - 6)."""
    R, N = v.shape
    b = torch.nn.functional.pad(v, (0, -N % 32)).view(R, -1, 32)
    m, e = torch.frexp(b.abs().amax(-1))                 # amax = m 2^e, m in [0.5, 1)
    e = torch.where(m == 0, torch.full_like(e, -127), e - 1 + (m > 127 / 128).to(e.dtype)).clamp(-127, 127)
    q = torch.round(b.double() * _pow2(6 - e)[..., None]).clamp(-127, 127)
    return q.to(torch.int8).view(R, -1)[:, :N].contiguous(), (e + 127).to(torch.uint8)


def _int8_values(codes, scales):
    """The values that codes and exponent bytes stand for, FP32 (exact)."""
    R, N = codes.shape
    s = _pow2(scales.to(torch.int64) - 133).float()
    return codes.float() * s.repeat_interleave(32, dim=1)[:, :N]


def _e4m3(v, kind, real=torch.float32):
    """Floats [R][C] -> E4M3 codes [R][C] of 448 v / (largest magnitude) and FP32 scales, that
    magnitude / 448, of each 128 columns of a row ([C / 128][R]) or of each 128 x 128 tile
    ([R / 128][C / 128])."""
    R, C = v.shape
    rb = 1 if kind == "rows" else 128
    p = torch.nn.functional.pad(v.to(real), (0, -C % 128, 0, -R % rb))
    p = p.view(_up(R, rb), rb, -1, 128)
    amax = p.abs().amax(-1).amax(1)
    amax = torch.where(amax == 0, torch.full_like(amax, 448.0), amax)
    s = amax / 448.0
    q = (p * 448.0 / amax[:, None, :, None]).reshape(_up(R, rb) * rb, -1)[:R, :C].to(torch.float8_e4m3fn)
    return q, (s.t().contiguous() if kind == "rows" else s.contiguous()).float()


def _e4m3_values(q, s, kind, real=torch.float32):
    """The values of _e4m3's codes [R][>= C] and scales."""
    R, C = q.shape
    if kind == "rows":
        return q.to(real) * s.to(real).t().repeat_interleave(128, dim=1)[:, :C]
    return q.to(real) * s.to(real).repeat_interleave(128, dim=0)[:R].repeat_interleave(128, dim=1)[:, :C]


def _rows(t, pad):
    """t with `pad` unused elements after every row."""
    if not pad:
        return t.contiguous()
    buf = torch.zeros(t.shape[0], t.shape[1] + pad, dtype=t.dtype, device=t.device)
    buf[:, :t.shape[1]] = t
    return buf[:, :t.shape[1]]


# ------------------------------------------------------------------------- inputs
def _prepare_ffn(c, seed):
    T, H, I, bf = c["T"], c["H"], c["I"], torch.bfloat16
    g = _gen(seed)
    rn = lambda *s: torch.randn(*s, device=DEV, generator=g)
    st = {"case": c, "x": rn(T, H).to(bf), "gate": (rn(I, H) * 0.02).to(bf), "up": (rn(I, H) * 0.02).to(bf),
          "down": (rn(H, I) * 0.02).to(bf)}
    if c["op"] != "ffn_fwd":
        st["dy"] = rn(T, H).to(bf)
    if c["op"] == "ffn_bwd":        # what the forward kept
        x = st["x"]
        ab = torch.cat([x @ st["gate"].t(), x @ st["up"].t()], 1)
        if c["saved"] == "bf16":
            st["ab"] = ab
        else:
            st["ab"], st["ab_s"] = _int8(ab.float())
            st["xq"], st["xq_s"] = _int8(x.float())
    if own:
        import moe_megakernel_amd as mk
        op = st["op"] = mk.FeedForward(H, I, T, activation=c["act"], saved=c["saved"], grad_dtype=bf, device=DEV)
        if c["saved"] != "none":
            st["saved"] = torch.zeros(op.saved_bytes(T), dtype=torch.uint8, device=DEV)
            st["views"] = v = op.saved_views(st["saved"], T)
            if c["op"] == "ffn_bwd":
                v["ab"].copy_(st["ab"])
                if c["saved"] == "int8":
                    v["ab_scales"].copy_(st["ab_s"])
                    v["x"].copy_(st["xq"])
                    v["x_scales"].copy_(st["xq_s"])
        st["out"], st["dx"] = torch.empty(T, H, dtype=bf, device=DEV), torch.empty(T, H, dtype=bf, device=DEV)
        st["dgate"], st["dup"] = (torch.empty(I, H, dtype=bf, device=DEV) for _ in range(2))
        st["ddown"] = torch.empty(H, I, dtype=bf, device=DEV)
    return st


def _prepare_ckpt(c, seed):
    g = _gen(seed)
    R, N, dt = c["rows"], c["cols"], _TORCH[c["dtype"]]
    # hidden states: each row with a scale of its own, a few columns far larger than the others
    v = torch.randn(R, N, device=DEV, generator=g) * torch.exp(torch.randn(R, 1, device=DEV, generator=g))
    v[:, ::97] *= 20.0
    st = {"case": c, "x": _rows(v.to(dt), c["pad"])}
    if own:
        import moe_megakernel_amd as mk
        st["op"] = mk.Checkpoint(dtype=dt)
        st["codes"] = torch.empty(R, N, dtype=torch.int8, device=DEV)
        st["scales"] = torch.empty(R, _up(N, 32), dtype=torch.uint8, device=DEV)
        st["y"] = _rows(torch.empty(R, N, dtype=dt, device=DEV), c["pad"])
    return st


def _prepare_quant(c, seed):
    g = _gen(seed)
    R, C, dt = c["rows"], c["cols"], _TORCH[c["dtype"]]
    st = {"case": c, "x": (torch.randn(R, C, device=DEV, generator=g) *
                           torch.exp(torch.randn(R, 1, device=DEV, generator=g))).to(dt)}
    if own:
        import moe_megakernel_amd as mk
        op = st["op"] = mk.Fp8Quantizer(kind=c["kind"], transpose=c["transpose"], dtype=dt)
        qs, ss = op.shapes(R, C)
        st["codes"] = torch.empty(*qs, dtype=torch.float8_e4m3fn, device=DEV)
        st["scales"] = torch.empty(*ss, dtype=torch.float32, device=DEV)
    return st


def _prepare_matmul(c, seed):
    g = _gen(seed)
    M, N, K, G = c["M"], c["N"], c["K"], c["groups"]
    rn = lambda *s: torch.randn(*s, device=DEV, generator=g)
    st = {"case": c}
    st["a"], st["sa"] = _e4m3(rn(M, K) * torch.exp(0.5 * rn(M, 1)), "rows")
    st["b"] = torch.empty(G, N, K, dtype=torch.float8_e4m3fn, device=DEV)
    if c["scales"] == "rows":
        st["b"][0], st["sb"] = _e4m3(rn(N, K) * 0.02, "rows")
    else:
        st["sb"] = torch.empty(G, _up(N, 128), _up(K, 128), device=DEV)
        for e in range(G):
            st["b"][e], st["sb"][e] = _e4m3(rn(N, K) * 0.02, "tiles")
    used = max(1, M - c["spare"])
    share = torch.rand(G, generator=torch.Generator().manual_seed(seed)) ** 2 + 1e-3     # uneven groups
    ends = torch.round(torch.cumsum(share, 0) / share.sum() * used).to(torch.int64).tolist()
    st["ends"] = [0] + ends[:-1] + [used]
    st["offsets"] = torch.tensor(st["ends"], dtype=torch.int32, device=DEV) if G > 1 or c["spare"] else None
    if own:
        import moe_megakernel_amd as mk
        st["op"] = mk.Fp8Matmul(scales=c["scales"], out_dtype=_TORCH[c["out"]], device=DEV)
        # rows behind the last group are left as they are: here zeros
        st["out"] = torch.zeros(M, N, dtype=_TORCH[c["out"]], device=DEV)
    return st


def prepare(case, seed):
    op = case["op"].split("_")[0]
    return {"ffn": _prepare_ffn, "ckpt": _prepare_ckpt, "quant": _prepare_quant, "matmul": _prepare_matmul}[op](case, seed)


# ------------------------------------------------------------------------- one pass
def run(state):
    return {"ffn_fwd": _run_ffn_fwd, "ffn_bwd": _run_ffn_bwd, "ffn_step": _run_ffn_step, "ckpt": _run_ckpt,
            "quant": _run_quant, "matmul": _run_matmul}[state["case"]["op"]](state)


def _act(a, kind):
    """The activation and its derivative."""
    if kind == "silu":
        s = 1.0 / (1.0 + torch.exp(-a))
        return a * s, s * (1.0 + a * (1.0 - s))
    k = math.sqrt(2.0 / math.pi)
    t = torch.tanh(k * (a + 0.044715 * a * a * a))
    return 0.5 * a * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * a * (1.0 - t * t) * k * (1.0 + 3 * 0.044715 * a * a)


def _plain_fwd(st):
    c = st["case"]
    x = st["x"].float()
    a, b = x @ st["gate"].float().t(), x @ st["up"].float().t()
    out = (_act(a, c["act"])[0] * b) @ st["down"].float().t()
    return out.to(torch.bfloat16), torch.cat([a, b], 1)


def _plain_bwd(st, ab, x):
    c, I = st["case"], st["case"]["I"]
    a, b, dy = ab[:, :I], ab[:, I:], st["dy"].float()
    dh = dy @ st["down"].float()
    h, dact = _act(a, c["act"])
    da, db = dh * b * dact, dh * h
    dx = da @ st["gate"].float() + db @ st["up"].float()
    return [v.to(torch.bfloat16) for v in (dx, da.t() @ x, db.t() @ x, dy.t() @ (h * b))]


def _own_bwd(st):
    x = st["x"] if st["case"]["saved"] == "bf16" else None
    st["op"].backward(st["dy"], x, st["gate"], st["up"], st["down"], st["saved"], st["dx"], st["dgate"], st["dup"],
                      st["ddown"], overwrite=True)
    return [st["dx"], st["dgate"], st["dup"], st["ddown"]]


def _run_ffn_fwd(st):
    keep = st["case"]["saved"] == "bf16"
    if own:
        st["op"].forward(st["x"], st["gate"], st["up"], st["down"], st["out"], st.get("saved"))
        return [st["out"]] + ([st["views"]["ab"]] if keep else [])
    out, ab = _plain_fwd(st)
    return [out] + ([ab.to(torch.bfloat16)] if keep else [])


def _run_ffn_bwd(st):
    if own:
        return _own_bwd(st)
    if st["case"]["saved"] == "bf16":
        return _plain_bwd(st, st["ab"].float(), st["x"].float())
    return _plain_bwd(st, _int8_values(st["ab"], st["ab_s"]), _int8_values(st["xq"], st["xq_s"]))


def _run_ffn_step(st):
    if own:
        st["op"].forward(st["x"], st["gate"], st["up"], st["down"], st["out"], st["saved"])
        return [st["out"]] + _own_bwd(st)
    out, ab = _plain_fwd(st)
    x = st["x"].float()
    if st["case"]["saved"] == "int8":       # the backward sees what was kept
        ab, x = _int8_values(*_int8(ab)), _int8_values(*_int8(x))
    else:
        ab = ab.to(torch.bfloat16).float()
    return [out] + _plain_bwd(st, ab, x)


def _run_ckpt(st):
    if own:
        st["op"].store(st["x"], st["codes"], st["scales"])
        return st["op"].load(st["codes"], st["scales"], st["y"])
    return _int8_values(*_int8(st["x"].float())).to(st["x"].dtype)


def _padded_codes(q, s):
    """Codes, their rows padded with zero codes to a multiple of 16, and scales."""
    q = torch.nn.functional.pad(q.view(torch.uint8), (0, -q.shape[1] % 16))
    return [q.contiguous().view(torch.float8_e4m3fn), s]


def _run_quant(st):
    c = st["case"]
    if own:
        st["op"].forward(st["x"], st["codes"], st["scales"])
        return [st["codes"], st["scales"]]
    x = st["x"].float()
    q, s = _e4m3(x.t() if c["transpose"] else x, c["kind"])
    return _padded_codes(q, s)


def _run_matmul(st):
    c = st["case"]
    if own:
        st["op"].forward(st["a"], st["sa"], st["b"], st["sb"], st["out"], offsets=st["offsets"])
        return st["out"]
    out = torch.zeros(c["M"], c["N"], device=DEV)
    a = _e4m3_values(st["a"], st["sa"], "rows")
    for e in range(c["groups"]):
        m0, m1 = st["ends"][e], st["ends"][e + 1]
        if m1 > m0:
            b = _e4m3_values(st["b"][e], st["sb"] if c["scales"] == "rows" else st["sb"][e], c["scales"])
            out[m0:m1] = a[m0:m1] @ b.t()
    return out.to(_TORCH[c["out"]])


# ------------------------------------------------------------------------- floor
def work(case):
    c = case
    if c["op"].startswith("ffn"):
        T, H, I = c["T"], c["H"], c["I"]
        keep = {"none": 0, "bf16": 4 * T * I, "int8": int(33 / 32 * T * (2 * I + H))}[c["saved"]]
        fwd = 4 * T * H + 6 * H * I + keep
        x = 0 if c["saved"] == "int8" else 2 * T * H
        bwd = 4 * T * H + x + keep + 12 * H * I       # dy, dx, x or its codes, weights and their gradients
        n = {"ffn_fwd": (fwd, 6), "ffn_bwd": (bwd, 12), "ffn_step": (fwd + bwd, 18)}[c["op"]]
        return {"bytes": n[0], "flops": n[1] * T * H * I}
    if c["op"] == "ckpt":
        n, z = c["rows"] * c["cols"], _SIZE[c["dtype"]]
        return {"bytes": int(2 * n * (z + 33 / 32)), "flops": 5 * n}
    if c["op"] == "quant":
        R, C = c["rows"], c["cols"]
        blocks = _up(C, 128) * (R if c["kind"] == "rows" else _up(R, 128))
        return {"bytes": R * C * (_SIZE[c["dtype"]] + 1) + 4 * blocks, "flops": 3 * R * C}
    M, N, K, G = c["M"], c["N"], c["K"], c["groups"]
    used = max(1, M - c["spare"])
    kb = _up(K, 128)
    sb = N * kb if c["scales"] == "rows" else G * _up(N, 128) * kb
    return {"bytes": used * K + min(G, used) * N * K + used * N * _SIZE[c["out"]] + 4 * (used * kb + sb),
            "flops": 2 * used * N * K}


# ------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    global own
    mine, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = mine
    op = case["op"].split("_")[0]
    return {"ffn": _exact_ffn, "ckpt": _exact_ckpt, "quant": _exact_quant, "matmul": _exact_matmul}[op](case, st)


def _near8(v):
    """v (64 bits) as its 8-bit checkpoint gives it back, by the definition: a power of two for
    each 32 values of a row, found by its logarithm, and the nearest of 255 multiples."""
    R, N = v.shape
    b = torch.nn.functional.pad(v, (0, -N % 32)).view(R, -1, 32)
    top = b.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(top.clamp(min=1e-290) / 127.0))
    e = torch.where(top > 127.0 * _pow2(e), e + 1, torch.where(top <= 127.0 * _pow2(e - 1), e - 1, e))
    step = _pow2(e.clamp(-133, 121))
    return (torch.clamp(torch.round(b / step), -127, 127) * step).view(R, -1)[:, :N]


def _exact_ffn(c, st):
    x, wg, wu, wd = (st[k].double() for k in ("x", "gate", "up", "down"))

    def act(a):
        if c["act"] == "silu":
            return a * torch.sigmoid(a)
        return a * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (a + 0.044715 * a.pow(3)))

    outs = []
    if c["op"] != "ffn_bwd":
        a, b = x.matmul(wg.t()), x.matmul(wu.t())
        outs = [(act(a) * b).matmul(wd.t())]
        if c["op"] == "ffn_fwd":
            return outs + ([torch.cat([a, b], 1)] if c["saved"] == "bf16" else [])
        if c["saved"] == "int8":
            a, b, x = _near8(a), _near8(b), _near8(x)
        else:
            a, b = a.to(torch.bfloat16).double(), b.to(torch.bfloat16).double()
    elif c["saved"] == "bf16":
        a, b = st["ab"].double().split(c["I"], 1)
    else:
        wide = lambda q, s: q.double() * _pow2(s.long() - 133).repeat_interleave(32, 1)[:, :q.shape[1]]
        (a, b), x = wide(st["ab"], st["ab_s"]).split(c["I"], 1), wide(st["xq"], st["xq_s"])
    dy = st["dy"].double()
    a = a.detach().requires_grad_(True)
    with torch.enable_grad():
        ha = act(a)
    dh = dy.matmul(wd)
    da, = torch.autograd.grad(ha, a, dh * b)
    ha = ha.detach()
    db = dh * ha
    return outs + [da.matmul(wg) + db.matmul(wu), da.t().matmul(x), db.t().matmul(x), dy.t().matmul(ha * b)]


def _exact_ckpt(c, st):
    return _near8(st["x"].double())


def _exact_quant(c, st):
    x = st["x"].double()
    q, s = _e4m3(x.t() if c["transpose"] else x, c["kind"], torch.float64)
    q = torch.nn.functional.pad(q.double(), (0, -q.shape[1] % 16))
    return [q, s.double()]


def _exact_matmul(c, st):
    out = torch.zeros(c["M"], c["N"], dtype=torch.float64, device=DEV)
    wide = lambda s, n: torch.repeat_interleave(s.double(), 128, dim=1)[:, :n]
    K, N = c["K"], c["N"]
    a = st["a"].double().mul_(wide(st["sa"].t(), K))
    for e, (m0, m1) in enumerate(zip(st["ends"], st["ends"][1:])):
        if m0 == m1:
            continue
        if c["scales"] == "rows":
            b = st["b"][0].double() * wide(st["sb"].t(), K)
        else:
            b = st["b"][e].double() * wide(st["sb"][e], K).repeat_interleave(128, dim=0)[:N]
        torch.mm(a[m0:m1], b.t(), out=out[m0:m1])
    return out

"""Activation checkpoints in 8 bits, against the format's definition in 64 bits.

No tolerance: the step is a power of two, so the scaled value, its rounding to the nearest code and
the decoded value are exact in FP32, and the values agree bit for bit."""
import pytest
import torch

import moe_megakernel_amd as mk

PTR = 1 << 20     # 16-byte aligned; refused calls never touch it


# ------------------------------------------------------------------ reference (64 bits, CPU)
def reference(x):
    """(codes, scale bytes, values) of the definition: the smallest s in [0, 254] with the
    block's largest magnitude <= 127 2^(s - 133), found by trying."""
    v = x.detach().cpu().double()
    R, N = v.shape
    nb = (N + 31) // 32
    b = torch.zeros(R, nb * 32, dtype=torch.float64)
    b[:, :N] = v
    b = b.view(R, nb, 32)
    top = b.abs().amax(-1)
    bad = ~torch.isfinite(b).all(-1)
    steps = 2.0 ** (torch.arange(255, dtype=torch.float64) - 133)
    s = torch.searchsorted(127.0 * steps, top.clamp(max=1e300).nan_to_num(0.0, 0.0, 0.0)).clamp(max=254)
    step = steps[s]
    q = torch.round(b.nan_to_num(0.0, 0.0, 0.0) / step[..., None]).clamp(-127, 127)
    q = torch.where(bad[..., None], torch.zeros_like(q), q)
    val = torch.where(bad[..., None], torch.full_like(q, float("nan")), q * step[..., None])
    s = torch.where(bad, torch.full_like(s, 255), s)
    return q.view(R, -1)[:, :N].to(torch.int8), s.to(torch.uint8), val.view(R, -1)[:, :N]


def test_reference_is_within_half_a_step():
    g = torch.Generator().manual_seed(0)
    x = torch.randn(5, 77, generator=g) * torch.exp(3 * torch.randn(5, 1, generator=g))
    q, s, v = reference(x)
    step = (2.0 ** (s.double() - 133)).repeat_interleave(32, 1)[:, :77]
    assert ((v - x.double()).abs() <= step / 2).all()
    assert torch.equal(v, q.double() * step)
    # one step smaller would not hold the largest
    top = torch.nn.functional.pad(x, (0, 19)).view(5, 3, 32).abs().amax(-1).double()
    assert (top > 127 * 2.0 ** (s.double() - 134)).all()


# ------------------------------------------------------------------ CPU: refusals
@pytest.mark.parametrize("rows,cols,dtype,status", [
    (-1, 8, mk.MOE_BF16, mk.MOE_ERR_SHAPE), ((1 << 31) + 1, 8, mk.MOE_BF16, mk.MOE_ERR_SHAPE),
    (4, 0, mk.MOE_BF16, mk.MOE_ERR_SHAPE), (4, mk.MOE_CHECKPOINT_MAX_COLS + 1, mk.MOE_BF16, mk.MOE_ERR_SHAPE),
    (1 << 31, 4096, mk.MOE_BF16, mk.MOE_ERR_SHAPE),        # more threads than a launch holds
    (4, 8, mk.MOE_MXFP8_E4M3, mk.MOE_ERR_DTYPE), (4, 8, 0, mk.MOE_ERR_DTYPE)])
def test_bad_problems_are_refused(rows, cols, dtype, status):
    p = mk.moe_checkpoint_problem(rows, cols, dtype)
    x = mk.moe_rows(PTR, max(cols, 1))
    assert mk.moe_checkpoint_store(p, x, PTR, PTR, None) == status
    assert mk.moe_checkpoint_load(p, PTR, PTR, x, None) == status


def test_bad_arguments_are_refused():
    p = mk.moe_checkpoint_problem(4, 64, mk.MOE_FP32)
    for x, c, s, status in ((None, PTR, PTR, mk.MOE_ERR_NULL), ((0, 64), PTR, PTR, mk.MOE_ERR_NULL),
                            ((PTR, 64), None, PTR, mk.MOE_ERR_NULL), ((PTR, 64), PTR, None, mk.MOE_ERR_NULL),
                            ((PTR, 63), PTR, PTR, mk.MOE_ERR_LAYOUT), ((PTR + 2, 64), PTR, PTR, mk.MOE_ERR_LAYOUT)):
        r = None if x is None else mk.moe_rows(*x)
        assert mk.moe_checkpoint_store(p, r, c, s, None) == status
        assert mk.moe_checkpoint_load(p, c, s, r, None) == status
    empty = mk.moe_checkpoint_problem(0, 64, mk.MOE_BF16)
    assert mk.moe_checkpoint_store(empty, None, None, None, None) == mk.MOE_OK


def test_binding_refuses_host_and_mismatched_tensors():
    op = mk.Checkpoint()
    x, c, s = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4, 2, dtype=torch.uint8)

    def status(*a):
        with pytest.raises(mk.MoeError) as e:
            op.store(*a)
        with pytest.raises(mk.MoeError) as f:
            op.load(a[1], a[2], a[0])
        assert e.value.status == f.value.status
        return e.value.status
    assert status(x, c, s) == mk.MOE_ERR_LAYOUT                  # host memory
    assert status(x.float(), c, s) == mk.MOE_ERR_DTYPE
    assert status(x[0], c, s) == mk.MOE_ERR_SHAPE
    assert status(None, c, s) == mk.MOE_ERR_NULL
    assert status(x[:, :0], c, s) == mk.MOE_ERR_SHAPE
    with pytest.raises(mk.MoeError) as e:
        mk.Checkpoint(dtype=torch.float16)
    assert e.value.status == mk.MOE_ERR_DTYPE


# ------------------------------------------------------------------ GPU
def placed(t, pad, offset):
    """t with `pad` elements after each row, `offset` elements into its storage, NaN around."""
    R, N = t.shape
    buf = torch.full((R * (N + pad) + offset,), float("nan"), dtype=t.dtype, device="cuda")
    v = buf[offset:].view(R, N + pad)[:, :N]
    v.copy_(t)
    return v, buf


def check(x, pad=0, offset=0):
    R, N = x.shape
    op = mk.Checkpoint(dtype=x.dtype)
    xv, _ = placed(x, pad, offset)
    guard = 64
    cbuf = torch.full((R * N + guard,), 77, dtype=torch.int8, device="cuda")
    sbuf = torch.full((R * ((N + 31) // 32) + guard,), 77, dtype=torch.uint8, device="cuda")
    codes, scales = cbuf[:R * N].view(R, N), sbuf[:-guard].view(R, -1)
    op.store(xv, codes, scales)
    y, ybuf = placed(torch.zeros_like(x), pad, offset)
    op.load(codes, scales, y)
    torch.cuda.synchronize()
    q, s, v = reference(x)
    assert torch.equal(codes.cpu(), q)
    assert torch.equal(scales.cpu(), s)
    assert torch.equal(y.cpu().double().nan_to_num(7.0), v.to(x.dtype).double().nan_to_num(7.0))
    assert torch.equal(torch.isnan(y.cpu()), torch.isnan(v))
    assert (cbuf[R * N:] == 77).all() and (sbuf[-guard:] == 77).all()
    if pad:
        assert torch.isnan(ybuf[offset:].view(R, N + pad)[:, N:]).all()
    assert torch.isnan(ybuf[:offset]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R,N,pad,offset", [(1, 1, 0, 0), (1, 32, 0, 0), (3, 31, 0, 0), (5, 33, 1, 1), (7, 40, 0, 0),
                                            (2, 1000, 8, 8), (257, 96, 0, 0), (19, 4096, 0, 0), (64, 2055, 3, 5),
                                            (300, 72, 4, 0), (1025, 8, 0, 0)])
def test_round_trip_is_the_definition(gpu_lib, dtype, R, N, pad, offset):
    g = torch.Generator().manual_seed(R * 1000 + N)
    x = torch.randn(R, N, generator=g) * torch.exp(4 * torch.randn(R, 1, generator=g))
    x[:, ::37] *= 30
    check(x.to(dtype), pad, offset)


@pytest.mark.gpu
def test_ties_zeros_and_the_ends_of_the_range(gpu_lib):
    one = torch.zeros(1, 32)
    rows = []
    for top in (127.0, 126.5, 127.0 / 128, 1.984375, 1.9921875, 2.0 ** -126, 2.0 ** -133, 3.3895e38, 2.0 ** 121, 1.0):
        r = one.clone()
        r[0, 0] = top
        r[0, 1:32] = top * (torch.arange(31) + 0.5) / 127     # halves of a step among them
        rows.append(r)
        rows.append(-r)
    rows += [one, -one]
    x = torch.cat(rows)
    check(x)
    check(x.to(torch.bfloat16))
    tiny = torch.full((3, 32), 2.0 ** -149)                   # FP32 below half the smallest step
    tiny[1] = 2.0 ** -134
    tiny[2] = (127.0 * 2.0 ** -133) * (1 + 2.0 ** -7)
    check(tiny)


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_nonfinite_values_mark_their_block_only(gpu_lib, bad):
    for dtype in (torch.bfloat16, torch.float32):
        x = torch.randn(4, 100).to(dtype)
        x[1, 40] = bad
        x[2, 99] = bad
        check(x)


@pytest.mark.gpu
def test_no_rows(gpu_lib):
    op = mk.Checkpoint()
    e = lambda n, dt: torch.empty(0, n, dtype=dt, device="cuda")
    op.store(e(40, torch.bfloat16), e(40, torch.int8), e(2, torch.uint8))
    op.load(e(40, torch.int8), e(2, torch.uint8), e(40, torch.bfloat16))


@pytest.mark.gpu
def test_offsets_past_32_bits(gpu_lib):
    R, N = 70000, 32768                                       # 2.3e9 values
    x = torch.zeros(R, N, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(3, N).to(torch.bfloat16)
    x[-3:] = tail.cuda()
    op = mk.Checkpoint()
    codes = torch.empty(R, N, dtype=torch.int8, device="cuda")
    scales = torch.empty(R, N // 32, dtype=torch.uint8, device="cuda")
    op.store(x, codes, scales)
    q, s, v = reference(tail)
    assert torch.equal(codes[-3:].cpu(), q) and torch.equal(scales[-3:].cpu(), s)
    x.fill_(1.0)
    op.load(codes, scales, x)
    assert torch.equal(x[-3:].cpu().double(), v)
    assert not x[:-3].any()


@pytest.mark.gpu
def test_captured_and_on_another_stream(gpu_lib):
    op = mk.Checkpoint()
    x = torch.randn(33, 520, device="cuda").to(torch.bfloat16)
    codes, scales = torch.empty(33, 520, dtype=torch.int8, device="cuda"), torch.empty(33, 17, dtype=torch.uint8, device="cuda")
    y = torch.empty_like(x)

    def step():
        op.store(x, codes, scales)
        op.load(codes, scales, y)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y.cpu().double(), reference(x)[2])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        x.copy_(torch.randn(33, 520, device="cuda"))
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y.cpu().double(), reference(x)[2])

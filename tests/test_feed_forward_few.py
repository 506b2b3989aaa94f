"""The feed-forward block's forward for up to 64 tokens: nothing but the output is rounded to BF16.

Tolerance: that of many tokens (tests/test_feed_forward.py) with h off by 2^-16 of itself (two BF16 parts, each
half a step of 2^-8 relative: 2^-8 2^-8) in the place of 2^-8."""
import pytest
import torch

import moe_megakernel_amd as mk
from tests.test_feed_forward import ACT, BF, R_BF, U, act, inputs, near

H_PARTS = 2.0 ** -16


def reference(x, wg, wu, wd, kind):
    x, wg, wu, wd = (t.double().cpu() for t in (x, wg, wu, wd))
    H, I = x.shape[1], wg.shape[0]
    a, b = x @ wg.t(), x @ wu.t()
    ea, eb = (2 * H * U * (x.abs() @ w.abs().t()) for w in (wg, wu))
    f, _ = act(a, kind)
    ef = 1.2 * ea + ACT * f.abs()
    h = f * b
    eh = (ef * b.abs() + f.abs() * eb + ef * eb) * (1 + H_PARTS) + H_PARTS * h.abs()
    return h @ wd.t(), eh @ wd.abs().t() + 2 * 2 * I * U * ((h.abs() + eh) @ wd.abs().t())


@pytest.mark.gpu
@pytest.mark.parametrize("kind,saved", [("silu", "none"), ("gelu", "bf16")])
@pytest.mark.parametrize("T,H,I", [(1, 64, 64), (1, 4096, 64), (5, 320, 192), (8, 192, 64), (9, 64, 128), (16, 128, 64), (17, 192, 192),
                                   (32, 64, 64), (33, 320, 64), (40, 4160, 64), (48, 64, 192), (49, 192, 64), (64, 64, 64),
                                   (24, 8256, 64), (64, 4160, 128), (12, 4160, 64),
                                   (20, 128, 2048), (40, 64, 4160), (64, 320, 2112), (33, 4096, 2048)])    # in parts
def test_only_the_output_is_rounded(gpu_lib, T, H, I, kind, saved):
    x, wg, wu, wd, _ = inputs(T, H, I)
    op = mk.FeedForward(H, I, T, kind, saved)
    sv = None if saved == "none" else torch.zeros(op.saved_bytes(T), dtype=torch.uint8, device="cuda")
    out = torch.empty(T, H, dtype=BF, device="cuda")
    op.forward(x, wg, wu, wd, out, sv)
    torch.cuda.synchronize()
    near(out, *reference(x, wg, wu, wd, kind), R_BF)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 12, 64])
def test_h_at_the_end_of_the_range(gpu_lib, T):
    """h = (2 - 2^-8) 2^127 is finite in FP32 and in one BF16 value infinite: so is the output, and not NaN."""
    H = I = 64
    x = torch.zeros(T, H, dtype=BF, device="cuda")
    x[:, 0], x[:, 1] = 2.0 ** 60, 2.0 ** 60
    wg, wu = torch.zeros(I, H, dtype=BF, device="cuda"), torch.zeros(I, H, dtype=BF, device="cuda")
    wg[0, 0] = 1.0                                                   # a = 2^60, act(a) = a
    wu[0, 0], wu[0, 1] = 2.0 ** 8, -2.0 ** -1                        # b = (2^8 - 2^-1) 2^60, h = (2 - 2^-8) 2^127
    wd = torch.zeros(H, I, dtype=BF, device="cuda")
    wd[:, 0] = 1.0
    op = mk.FeedForward(H, I, T)
    out = torch.empty(T, H, dtype=BF, device="cuda")
    op.forward(x, wg, wu, wd, out)
    torch.cuda.synchronize()
    assert torch.equal(out, torch.full_like(out, float("inf")))

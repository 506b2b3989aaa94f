"""The feed-forward block's rows are each other's business nowhere: the same rows among other ones, NaN among them, give
the same bits, and so does a smaller call in a workspace of a larger one."""
import pytest
import torch

import moe_megakernel_amd as mk
from tests.test_feed_forward import BF, inputs

# few tokens, a tile or two, contractions in parts
SIZES = [(40, 320, 448), (300, 320, 448), (300, 1024, 704)]


@pytest.mark.gpu
@pytest.mark.parametrize("saved", ["bf16", "int8"])
@pytest.mark.parametrize("T,H,I", SIZES)
@pytest.mark.parametrize("other", [0.5, float("nan"), float("inf")])
def test_rows_do_not_depend_on_the_other_rows(gpu_lib, T, H, I, saved, other):
    x, wg, wu, wd, dy = inputs(T, H, I)
    keep = torch.arange(T) % 3 != 1
    x2, dy2 = x.clone(), dy.clone()
    x2[~keep], dy2[~keep] = other, other
    outs = []
    for most in (T, 2 * T + 100):
        for xs, ys in ((x, dy), (x2, dy2)):
            op = mk.FeedForward(H, I, most, saved=saved)
            op.workspace.fill_(0xff)                                 # NaN, were it read
            sv = torch.full((op.saved_bytes(most),), 0xff, dtype=torch.uint8, device="cuda")
            out, dx = torch.empty_like(x), torch.empty_like(x)
            op.forward(xs, wg, wu, wd, out, sv)
            op.backward(ys, xs if saved == "bf16" else None, wg, wu, wd, sv, dx)
            outs.append((out[keep], dx[keep]))
    torch.cuda.synchronize()
    for out, dx in outs:
        assert torch.isfinite(out).all() and torch.isfinite(dx).all()
        assert torch.equal(out, outs[0][0]) and torch.equal(dx, outs[0][1])

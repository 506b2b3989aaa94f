"""The gated feed-forward block at the ends of FP32's range."""
import pytest
import torch

import moe_megakernel_amd as mk
from tests.test_feed_forward import BF


@pytest.mark.gpu
@pytest.mark.parametrize("saved", ["bf16", "int8"])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("T,H,I", [(70, 64, 64), (70, 1152, 64)])       # one part, several
def test_switched_off_units_take_no_gradient_however_large(gpu_lib, T, H, I, kind, saved):
    """a = -256: act and act' are below 2^-350, so da, db and h are 0 in FP32 although dh b = 2^140 is past it."""
    op = mk.FeedForward(H, I, T, kind, saved)
    sv = torch.zeros(op.saved_bytes(T), dtype=torch.uint8, device="cuda")
    v = op.saved_views(sv, T)
    x = torch.ones(T, H, dtype=BF, device="cuda")
    if saved == "bf16":
        v["ab"][:, :I], v["ab"][:, I:] = -256.0, 2.0 ** 70
    else:                                    # code 2^(s - 133)
        v["ab"][:, :I], v["ab"][:, I:] = -64, 64
        v["ab_scales"][:, :I // 32], v["ab_scales"][:, I // 32:] = 135, 197
        v["x"][:], v["x_scales"][:] = 64, 127
    w = torch.ones(I, H, dtype=BF, device="cuda")
    wd = torch.full((H, I), 2.0 ** 30 / H, dtype=BF, device="cuda")     # dh = 2^70
    dy = torch.full((T, H), 2.0 ** 40, dtype=BF, device="cuda")
    dx = torch.empty_like(x)
    g = [torch.ones(*s, device="cuda") for s in ((I, H), (I, H), (H, I))]
    op.backward(dy, x if saved == "bf16" else None, w, w, wd, sv, dx, *g, overwrite=True)
    torch.cuda.synchronize()
    for t in [dx] + g:
        assert (t == 0).all()

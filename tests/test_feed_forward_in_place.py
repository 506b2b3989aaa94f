"""The gated feed-forward block with results that take the place of inputs: the same bits as in places of
their own."""
import pytest
import torch

import moe_megakernel_amd as mk
from tests.test_feed_forward import BF, inputs

# few tokens, a tile or two, contractions in parts
SIZES = [(7, 64, 128), (130, 256, 192), (1500, 128, 192)]


@pytest.mark.gpu
@pytest.mark.parametrize("saved,where", [("bf16", "grad_out"), ("bf16", "x"), ("int8", "grad_out")])
@pytest.mark.parametrize("T,H,I", SIZES)
def test_input_gradient_in_the_place_of_an_input(gpu_lib, T, H, I, saved, where):
    x, wg, wu, wd, dy = inputs(T, H, I)
    op = mk.FeedForward(H, I, T, saved=saved)
    sv = torch.zeros(op.saved_bytes(T), dtype=torch.uint8, device="cuda")
    op.forward(x, wg, wu, wd, torch.empty_like(x), sv)
    xx = x if saved == "bf16" else None
    grads = lambda: [torch.zeros(*s, device="cuda") for s in ((I, H), (I, H), (H, I))]
    want, dx = grads(), torch.empty_like(x)
    op.backward(dy, xx, wg, wu, wd, sv, dx, *want)
    got = grads()
    place = dy if where == "grad_out" else x
    op.backward(dy, xx, wg, wu, wd, sv, place, *got)
    torch.cuda.synchronize()
    assert torch.equal(place, dx)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("saved", ["none", "bf16", "int8"])
@pytest.mark.parametrize("T,H,I", SIZES + [(20, 128, 2048), (300, 1024, 704)])
def test_output_in_the_place_of_the_input(gpu_lib, T, H, I, saved):
    x, wg, wu, wd, _ = inputs(T, H, I)
    op = mk.FeedForward(H, I, T, saved=saved)
    kept = [None if saved == "none" else torch.zeros(op.saved_bytes(T), dtype=torch.uint8, device="cuda") for _ in range(2)]
    out = torch.empty_like(x)
    op.forward(x, wg, wu, wd, out, kept[0])
    op.forward(x, wg, wu, wd, x, kept[1])
    torch.cuda.synchronize()
    assert torch.equal(out, x)
    assert saved == "none" or torch.equal(*kept)

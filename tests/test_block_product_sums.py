"""What the 8-bit product's sums keep: products of 2^17.6 that cancel beside products of 1.

A block with n products that are not 0.  FP32 results, and any of up to 64 rows: FP32 sums, off by at most 2 n u of the sum of
magnitudes (u = 2^-24, one rounding a term and the unit's alignment).  BF16 results of more rows: a block to 2^-15 of its sum
of magnitudes (2^-16 of its largest product in each of two partial sums).  A BF16 result's rounding is 2^-8 of itself."""
import pytest
import torch

import moe_megakernel_amd as mk

F8, U = torch.float8_e4m3fn, 2.0 ** -24


@pytest.mark.gpu
@pytest.mark.parametrize("scales", ["tiles", "rows"])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M", [20, 300])
@pytest.mark.parametrize("K", [128, 1024])
def test_cancelling_products_keep_what_is_stated(gpu_lib, M, K, out_dtype, scales):
    N, kb = 48, K // 128
    a, b = torch.zeros(M, K), torch.zeros(N, K)
    g = torch.Generator().manual_seed(M + K)
    at = [torch.randperm(128, generator=g) + 128 * i for i in range(kb)]
    for p in at:
        a[:, p[:2]] = 448.0
        b[:, p[0]], b[:, p[1]] = 448.0, -448.0
        a[:, p[2:6]] = 1.0
        b[:, p[2:6]] = torch.randint(1, 4, (N, 4), generator=g).float()
    sa = 2.0 ** torch.randint(-3, 4, (kb, M), generator=g).float()
    sb = torch.ones(kb, N) if scales == "rows" else torch.ones(1, 1, kb)
    out = torch.empty(M, N, dtype=out_dtype, device="cuda")
    mk.Fp8Matmul(scales, out_dtype).forward(a.to(F8).cuda(), sa.cuda(), b[None].to(F8).cuda(), sb.cuda(), out)
    torch.cuda.synchronize()
    av = a.double() * sa.double().t().repeat_interleave(128, 1)
    ref, mag = av @ b.double().t(), av.abs() @ b.double().abs().t()
    fp32 = out_dtype == torch.float32 or M <= 64
    sums = (2 * (6 + kb) * U if fp32 else 2.0 ** -15) * mag
    assert (ref > 0).all() and (not fp32 or (sums < ref / 2).all())
    assert ((out.cpu().double() - ref).abs() <= sums + (2.0 ** -8 if out_dtype == torch.bfloat16 else U) * (ref.abs() + sums)).all()

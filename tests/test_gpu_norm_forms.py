"""The norm's forms that rows, parameters and values choose: rows whose squares
pass the largest float."""

import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [96, 768, 2880, 8192, 20000, 1001])
def test_rows_whose_squares_overflow(gpu_lib, d, dtype):
    # (x - mean)^2 is inf in 32 bits, and r = inf^-1/2 = 0: xh is 0 and y is beta,
    # whatever the width
    for T in (3, 700):
        x = torch.randn(T, d, device="cuda")
        x[1] = 0.0
        x[1, :7] = 1e25
        x = x.to(dtype)
        gamma = torch.randn(d, device="cuda").to(dtype)
        beta = torch.randn(d, device="cuda").to(dtype)
        for center in (True, False):
            y, mean, rstd, _ = gpu_lib.norm_forward(x, gamma, beta, center=center)
            assert rstd[1] == 0 and torch.equal(y[1], beta)
            keep = [t for t in range(T) if t != 1]
            alone = gpu_lib.norm_forward(x[keep].contiguous(), gamma, beta, center=center)
            assert torch.equal(y[keep], alone[0]) and torch.isfinite(y).all()
            dx, dg, _ = gpu_lib.norm_backward(torch.ones_like(x), x, mean, rstd, gamma)
            assert not dx[1].any() and torch.isfinite(dg).all()

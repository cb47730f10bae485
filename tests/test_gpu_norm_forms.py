"""The norm's forms that rows, parameters and values choose: widths around the
vectors a thread holds, rows whose squares pass the largest float.  Tolerances
are those of test_gpu_norm.py."""

import pytest
import torch

import ops_ref
from test_gpu_norm import _check_backward, _check_forward, _make, _np

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


@pytest.mark.parametrize("d", [520, 776, 1280, 1288, 1536, 2048, 2056, 2560, 2568, 3080, 4104, 6152,
                               8200, 10248, 12296])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_many_rows_at_every_count_of_vectors(gpu_lib, d, dtype):
    # one to four vectors (fp32: eight) a thread, and what three would be in bf16
    x, gamma, beta, dy = _make(1300, d, dtype, seed=21)
    _, mean, rstd, kept = _check_forward(gpu_lib, x, gamma, beta, True, checkpoint=True)
    _check_backward(gpu_lib, dy, x, _np(x), mean, rstd, gamma)
    _check_backward(gpu_lib, dy, kept, ops_ref.act8(_np(x))[2], mean, rstd, gamma)


@pytest.mark.parametrize("T,d", [(1, 16392), (65, 20000), (300, 17000), (4200, 16385), (300, 16384),
                                 (200, 9001), (161, 1001), (1300, 4096)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_workspace_of_just_the_size(gpu_lib, T, d, dtype):
    x, gamma, beta, dy = _make(T, d, dtype, seed=22)
    n = gpu_lib.norm_workspace_bytes(T, d)
    buf = torch.full((n + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
    _, mean, rstd, kept = gpu_lib.norm_forward(x, gamma, beta, checkpoint=True)
    for src in (x, kept):
        ref = gpu_lib.norm_backward(dy, src, mean, rstd, gamma, bias=True)
        got = gpu_lib.norm_backward(dy, src, mean, rstd, gamma, bias=True, workspace=buf[:n])
        assert all(torch.equal(a, b) for a, b in zip(ref, got))
        assert (buf[n:] == 0xA5).all()
    with pytest.raises(gpu_lib.CklError):
        gpu_lib.norm_backward(dy, x, mean, rstd, gamma, workspace=buf[:n - 16])

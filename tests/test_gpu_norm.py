"""The norm's forward and backward pass and 8-bit activations against 64-bit
plain forms.

Tolerances, with u = 2^-24 and h half a step of the output's type: a sum over a
row is at most 32 adds in a thread, 5 in a warp and 32 over the warps, so it is
off by at most 72 u times the sum of magnitudes; the handful of further
operations an element goes through leaves every term below within 100 u of the
magnitudes it is made of.  A column's sum over T rows is a chain of at most
T / 64 + 128 adds.
"""

import numpy as np
import pytest
import torch

import ops_ref
from ops_ref import HALF, U32

pytestmark = pytest.mark.gpu

C = 100 * U32
BF, F32 = torch.bfloat16, torch.float32
# the widths at which the kernels change (warps a row, vectors a thread, whole
# vectors or single elements), and some between
WIDTHS = [1, 7, 8, 31, 32, 33, 40, 256, 264, 1001, 1024, 2880, 4096, 8192, 8200, 8201, 16384,
          16400, 32767, 32768, 100003]


def _make(T, d, dtype, seed=0, pdtype=None, offset=0.3):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1000 * T + d)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    chan = 1 + 20 * (torch.rand(1, d, generator=g, device="cuda") < 0.05)
    x = (r(T, d) * chan + offset).to(dtype)
    pdtype = pdtype or dtype
    return x, (1 + 0.2 * r(d)).to(pdtype), (0.3 * r(d)).to(pdtype), r(T, d).to(dtype)


def _np(t):
    return None if t is None else t.double().cpu().numpy()


def _close(got, ref, tol):
    got, ref = _np(got), np.asarray(ref)
    assert got.shape == ref.shape
    err = np.abs(got - ref)
    assert (err <= tol).all(), (float((err / np.maximum(tol, 1e-300)).max()), float(err.max()))


def _same(got, ref, equal_nan=False):
    got = got.cpu().numpy() if isinstance(got, torch.Tensor) else got
    assert got.shape == ref.shape
    bad = np.argwhere(~((got == ref) | (equal_nan & (got != got) & (ref != ref))))
    assert len(bad) == 0, (len(bad), [(tuple(i), got[tuple(i)], ref[tuple(i)]) for i in bad[:8]])


def _check_forward(ckl, x, gamma, beta, center, eps=1e-5, **kw):
    y, mean, rstd, kept = ckl.norm_forward(x, gamma, beta, eps, center, **kw)
    xs, g, b = _np(x), _np(gamma), _np(beta)
    ry, rmu, rr, xh = ops_ref.norm(xs, g, b, eps, center)
    g1 = np.ones(x.shape[1]) if g is None else np.abs(g)
    b1 = 0.0 if b is None else np.abs(b)
    size = np.abs(xs).mean(1)[:, None]
    if center:
        _close(mean, rmu, C * size[:, 0] + 1e-300)
    else:
        assert mean is None
    # the mean's error moves x - mean and, to second order, the variance
    dr = C * (1 + (size[:, 0] * rr) * (1 if center else 0))
    _close(rstd, rr, dr * rr)
    mag = g1 * (np.abs(xh) * (1 + dr[:, None]) + (size * rr[:, None] if center else 0)) + b1
    _close(y, ry, 1.01 * HALF[x.dtype] * np.abs(ry) + 2 * C * mag + dr[:, None] * np.abs(xh) * g1)
    return y, mean, rstd, kept


def _check_backward(ckl, dy, x, xv, mean, rstd, gamma, bias=True, **kw):
    """xv: the values (float64) that x, a tensor or its 8 bits, stands for."""
    dx, dg, db = ckl.norm_backward(dy, x, mean, rstd, gamma, bias=bias, **kw)
    T = dy.shape[0]
    d, g, r = _np(dy), _np(gamma), _np(rstd)
    mu = 0.0 if mean is None else _np(mean)[:, None]
    xh = (xv - mu) * r[:, None]
    rdx, rdg, rdb = ops_ref.norm_grads(d, xh, r, g, mean is not None)
    a = np.abs(d if g is None else d * g)
    mag = a + a.mean(1, keepdims=True) + np.abs(xh) * (a * np.abs(xh)).mean(1, keepdims=True)
    _close(dx, rdx, 1.01 * HALF[dy.dtype] * np.abs(rdx) + C * r[:, None] * mag)
    n = (T / 64 + 128 + 8) * U32
    if g is not None:
        _close(dg, rdg, n * np.abs(d * xh).sum(0) + 1e-300)
    else:
        assert dg is None
    if bias:
        _close(db, rdb, n * np.abs(d).sum(0) + 1e-300)
    else:
        assert db is None
    return dx, dg, db


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", WIDTHS)
def test_forward_and_backward_at_every_width(gpu_lib, d, dtype):
    for T, center in ((3, True), (5, False)):
        x, gamma, beta, dy = _make(T, d, dtype)
        if not center:
            beta = None
        _, mean, rstd, kept = _check_forward(gpu_lib, x, gamma, beta, center, checkpoint=True)
        _check_backward(gpu_lib, dy, x, _np(x), mean, rstd, gamma, bias=center)
        q, e, val = ops_ref.act8(_np(x))
        _same(kept[0], q)
        _same(kept[1], e)
        _check_backward(gpu_lib, dy, kept, val, mean, rstd, gamma, bias=center)


@pytest.mark.parametrize("T,d", [(1, 4096), (149, 2880), (1500, 64), (5000, 8), (3000, 1001),
                                 (700, 4096), (640, 16384), (300, 20000), (300, 9001), (1300, 2880),
                                 (1205, 5120), (1190, 8192), (1300, 2568), (1200, 7168), (1200, 7176)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_many_rows(gpu_lib, T, d, dtype):
    x, gamma, beta, dy = _make(T, d, dtype, seed=1)
    _, mean, rstd, kept = _check_forward(gpu_lib, x, gamma, beta, True, checkpoint=True)
    first = _check_backward(gpu_lib, dy, x, _np(x), mean, rstd, gamma)
    again = gpu_lib.norm_backward(dy, x, mean, rstd, gamma, bias=True)
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    _check_backward(gpu_lib, dy, kept, ops_ref.act8(_np(x))[2], mean, rstd, gamma)


@pytest.mark.parametrize("pdtype", [BF, F32])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_parameter_types_and_absent_parameters(gpu_lib, dtype, pdtype):
    for d in (72, 73):
        x, gamma, beta, dy = _make(9, d, dtype, seed=2, pdtype=pdtype)
        for g, b in ((gamma, beta), (gamma, None), (None, beta), (None, None)):
            _, mean, rstd, _ = _check_forward(gpu_lib, x, g, b, True)
            _check_backward(gpu_lib, dy, x, _np(x), mean, rstd, g, bias=b is not None)


def test_unaligned_arrays(gpu_lib):
    # a multiple of 8 wide, but no 16-byte rows: single elements
    for d in (64, 16384):
        x, gamma, beta, dy = _make(4, d, BF, seed=3)

        def off(t):
            b = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape)
            return b.copy_(t)

        for xs, gs, ds in ((off(x), gamma, dy), (x, off(gamma), off(dy))):
            _, mean, rstd, kept = _check_forward(gpu_lib, xs, gs, beta, True, checkpoint=True)
            _check_backward(gpu_lib, ds, xs, _np(x), mean, rstd, gs)
            _check_backward(gpu_lib, ds, kept, ops_ref.act8(_np(x))[2], mean, rstd, gs)


def test_large_means_constant_rows_and_eps(gpu_lib):
    x, gamma, beta, dy = _make(6, 512, F32, seed=4, offset=3000.0)
    x[1] = 7.0                                      # no variance at all
    x[2] = 0.0
    for eps in (1e-5, 0.1):
        _, mean, rstd, _ = _check_forward(gpu_lib, x, gamma, beta, True, eps)
        _check_backward(gpu_lib, dy, x, _np(x), mean, rstd, gamma)
    y, _, rstd, _ = gpu_lib.norm_forward(x[2:3], None, None, 0.0, True)
    assert torch.isinf(rstd).all()                  # 0 / 0 of the formula
    assert torch.isnan(y).all()


def test_a_bad_row_stays_alone(gpu_lib):
    x, gamma, beta, dy = _make(5, 300, BF, seed=5)
    x[1, 7] = float("nan")
    x[3, 299] = float("inf")
    y, mean, rstd, kept = gpu_lib.norm_forward(x, gamma, beta, checkpoint=True)
    good = [0, 2, 4]
    ref = ops_ref.norm(_np(x[good]), _np(gamma), _np(beta), 1e-5, True)[0]
    assert np.abs(_np(y[good]) - ref).max() < 0.1 and torch.isnan(y[1]).all()
    for src in (x, kept):
        dx = gpu_lib.norm_backward(dy, src, mean, rstd, gamma)[0]
        assert torch.isfinite(dx[good]).all() and torch.isnan(dx[1]).all()


def test_empty_batches_accumulation_and_given_buffers(gpu_lib):
    x, gamma, beta, dy = _make(37, 136, BF, seed=6)
    _, mean, rstd, _ = gpu_lib.norm_forward(x, gamma, beta)
    dx, dg, db = gpu_lib.norm_backward(dy, x, mean, rstd, gamma, bias=True)
    ws = torch.empty(gpu_lib.norm_workspace_bytes(37, 136), dtype=torch.uint8, device="cuda")
    g2, b2 = dg.clone(), db.clone()
    gpu_lib.norm_backward(dy, x, mean, rstd, gamma, bias=True, dgamma=g2, dbeta=b2,
                          accumulate=True, workspace=ws)
    assert torch.equal(g2, dg + dg) and torch.equal(b2, db + db)
    # no rows: nothing to add, zero otherwise
    e, em = x[:0], mean[:0]
    y0, m0, r0, k0 = gpu_lib.norm_forward(e, gamma, beta, checkpoint=True)
    assert y0.shape == (0, 136) and m0.shape == (0,) and k0[1].shape == (0, 5)
    gpu_lib.norm_backward(e, e, em, em, gamma, bias=True, dgamma=g2, dbeta=b2, accumulate=True)
    assert torch.equal(g2, dg + dg)
    _, g0, b0 = gpu_lib.norm_backward(e, e, em, em, gamma, bias=True)
    assert not g0.any() and not b0.any()
    # in place
    a, b = x.clone(), dy.clone()
    y = gpu_lib.norm_forward(x, gamma, beta)[0]
    assert torch.equal(gpu_lib.norm_forward(a, gamma, beta, out=a)[0], y) and torch.equal(a, y)
    assert torch.equal(gpu_lib.norm_backward(b, x, mean, rstd, gamma, out_dx=b)[0], dx)


@pytest.mark.parametrize("T,d", [(1, 31), (3, 31), (5, 64), (130, 257), (600, 8), (2000, 40)])
def test_nothing_behind_the_workspace_or_the_outputs_is_written(gpu_lib, T, d):
    x, gamma, beta, dy = _make(T, d, BF, seed=12)
    n = gpu_lib.norm_workspace_bytes(T, d)
    ws = torch.full((n + 4096,), 0xA5, dtype=torch.uint8, device="cuda")

    def guarded(dtype, *shape):
        k = int(np.prod(shape))
        t = torch.full((k + 64,), 77, dtype=dtype, device="cuda")
        return t, t[:k].view(shape)

    y_, y = guarded(BF, T, d)
    dx_, dx = guarded(BF, T, d)
    dg_, dg = guarded(F32, d)
    db_, db = guarded(F32, d)
    _, mean, rstd, _ = gpu_lib.norm_forward(x, gamma, beta, out=y)
    gpu_lib.norm_backward(dy, x, mean, rstd, gamma, bias=True, dgamma=dg, dbeta=db,
                          workspace=ws[:n], out_dx=dx)
    assert (ws[n:] == 0xA5).all()
    for t in (y_, dx_, dg_, db_):
        assert (t[-64:] == 77).all()


def test_leading_dimensions(gpu_lib):
    x, gamma, beta, dy = _make(24, 48, BF, seed=7)
    y, mean, rstd, kept = gpu_lib.norm_forward(x, gamma, beta, checkpoint=True)
    x3, dy3 = x.view(2, 3, 4, 48), dy.view(2, 3, 4, 48)
    y3, mean3, rstd3, kept3 = gpu_lib.norm_forward(x3, gamma, beta, checkpoint=True)
    assert torch.equal(y3.view(24, 48), y) and mean3.shape == (2, 3, 4)
    assert kept3[1].shape == (2, 3, 4, 2)
    a = gpu_lib.norm_backward(dy, kept, mean, rstd, gamma, bias=True)
    b = gpu_lib.norm_backward(dy3, kept3, mean3, rstd3, gamma, bias=True)
    assert torch.equal(b[0].view(24, 48), a[0]) and torch.equal(a[1], b[1])


def test_other_streams_and_graphs(gpu_lib):
    x, gamma, beta, dy = _make(300, 520, BF, seed=8)
    ref_f = gpu_lib.norm_forward(x, gamma, beta, checkpoint=True)
    ref_b = gpu_lib.norm_backward(dy, ref_f[3], ref_f[1], ref_f[2], gamma, bias=True)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    f = gpu_lib.norm_forward(x, gamma, beta, checkpoint=True, stream=s)
    b = gpu_lib.norm_backward(dy, f[3], f[1], f[2], gamma, bias=True, stream=s)
    s.synchronize()
    assert torch.equal(f[0], ref_f[0]) and all(torch.equal(p, q) for p, q in zip(b, ref_b))
    # captured: the replay reads what the buffers then hold
    xs, ds = torch.zeros_like(x), torch.zeros_like(dy)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        f = gpu_lib.norm_forward(xs, gamma, beta, checkpoint=True)
        b = gpu_lib.norm_backward(ds, f[3], f[1], f[2], gamma, bias=True)
    for _ in range(2):
        xs.copy_(x)
        ds.copy_(dy)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(f[0], ref_f[0]) and all(torch.equal(p, q) for p, q in zip(b, ref_b))


def test_two_streams_at_once(gpu_lib):
    x, gamma, beta, dy = _make(2000, 1024, BF, seed=13)
    f = gpu_lib.norm_forward(x, gamma, beta)
    ref = gpu_lib.norm_backward(dy, x, f[1], f[2], gamma, bias=True)
    torch.cuda.synchronize()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = [gpu_lib.norm_backward(dy, x, f[1], f[2], gamma, bias=True, stream=t) for t in s]
        torch.cuda.synchronize()
        for g in got:
            assert all(torch.equal(a, b) for a, b in zip(g, ref))


@pytest.mark.parametrize("checkpoint", [False, True])
def test_autograd(gpu_lib, checkpoint):
    x, gamma, beta, dy = _make(40, 96, F32, seed=9)
    for center in (True, False):
        leaves = [x.clone().requires_grad_(), gamma.clone().requires_grad_()]
        if center:
            leaves.append(beta.clone().requires_grad_())
            y = gpu_lib.layer_norm(*leaves, checkpoint=checkpoint)
        else:
            y = gpu_lib.rms_norm(*leaves, checkpoint=checkpoint)
        (y * dy).sum().backward()
        eps = 1e-5 if center else 1e-6
        xv = ops_ref.act8(_np(x))[2] if checkpoint else _np(x)
        _, mu, r, _ = ops_ref.norm(_np(x), None, None, eps, center)
        xh = (xv - mu[:, None]) * r[:, None]
        ref = ops_ref.norm_grads(_np(dy), xh, r, _np(gamma), center)
        for leaf, g in zip(leaves, ref):
            assert np.abs(_np(leaf.grad) - g).max() <= 1e-4 * np.abs(g).max()
        with pytest.raises(RuntimeError):           # no second derivative
            y = gpu_lib.rms_norm(leaves[0], leaves[1])
            (dx,) = torch.autograd.grad(y.sum(), leaves[0], create_graph=True)
            dx.sum().backward()
    # only what needs a gradient
    g = gamma.clone().requires_grad_()
    gpu_lib.layer_norm(x, g, beta).sum().backward()
    assert g.grad is not None


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,d", [(1, 1), (3, 31), (5, 32), (4, 33), (7, 40), (1000, 1001),
                                 (333, 2880), (3, 100000)])
def test_act8_is_exactly_the_definition(gpu_lib, T, d, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(T * d)
    x = torch.randn(T, d, generator=g, device="cuda")
    x *= torch.exp2(torch.randint(-40, 40, (T, 1), generator=g, device="cuda").float())
    x = x.to(dtype)
    q, e = gpu_lib.act8_pack(x)
    rq, re, val = ops_ref.act8(_np(x))
    _same(q, rq)
    _same(e, re)
    for out in (BF, F32):
        _same(_np(gpu_lib.act8_unpack(q, e, out)), val)


@pytest.mark.parametrize("d", [64, 65])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_act8_extremes(gpu_lib, dtype, d):
    x = torch.zeros(8, d, dtype=F32, device="cuda")
    tiny = 2.0 ** -133 if dtype == BF else 2.0 ** -149   # the type's smallest
    x[1, 3] = tiny
    x[2, 3] = -3 * tiny
    x[2, 4] = 2.0 ** -126
    x[3, 3] = torch.finfo(dtype).max
    x[3, 40] = 1.9921875                                 # rounds to 128: the next power
    x[4, 3], x[4, 4] = float("inf"), 1.5
    x[5, 3], x[5, 4] = float("nan"), -2.5
    x[6, :32] = float("-inf")
    x[7, 3], x[7, 5] = 1.984375, -1.984375
    x = x.to(dtype)
    q, e = gpu_lib.act8_pack(x)
    rq, re, val = ops_ref.act8(_np(x))
    _same(q, rq)
    _same(e, re)
    for out in (BF, F32):
        _same(_np(gpu_lib.act8_unpack(q, e, out)), val, True)
    assert gpu_lib.act8_unpack(q, e)[3, 3] == 127 * 2.0 ** 121  # the largest floats clamp


def test_act8_past_2_31_elements(gpu_lib):
    T, d = 66000, 32768
    x = torch.zeros(T, d, dtype=BF, device="cuda")
    x[-2:] = _make(2, d, BF, seed=10)[0]
    q, e = gpu_lib.act8_pack(x)
    rq, re, val = ops_ref.act8(_np(x[-2:]))
    _same(q[-2:], rq)
    _same(e[-2:], re)
    back = gpu_lib.act8_unpack(q, e)
    assert np.array_equal(_np(back[-2:]), val) and not back[:10].any()


@pytest.mark.parametrize("T,d", [(66000, 32768), (530000, 4096)])
def test_norm_past_2_31_elements(gpu_lib, T, d):
    x = torch.zeros(T, d, dtype=BF, device="cuda")
    last, gamma, beta, dy = _make(2, d, BF, seed=11)
    x[-2:] = last
    y, mean, rstd, kept = gpu_lib.norm_forward(x, gamma, beta, checkpoint=True)
    small = gpu_lib.norm_forward(last, gamma, beta, checkpoint=True)
    assert torch.equal(y[-2:], small[0]) and torch.equal(kept[0][-2:], small[3][0])
    y.zero_()
    y[-2:] = dy                                     # the gradient of the last two rows
    dx, dg, _ = gpu_lib.norm_backward(y, kept, mean, rstd, gamma, out_dx=y)
    sx, sg, _ = gpu_lib.norm_backward(dy, small[3], small[1], small[2], gamma)
    assert torch.equal(dx[-2:], sx)
    assert (dg - sg).abs().max() <= 1e-5 * sg.abs().max()


def test_refusals(gpu_lib):
    x, gamma, beta, dy = _make(4, 64, BF)
    _, mean, rstd, kept = gpu_lib.norm_forward(x, gamma, beta, checkpoint=True)
    with pytest.raises(TypeError):
        gpu_lib.norm_forward(x.half(), gamma)
    with pytest.raises(ValueError):
        gpu_lib.norm_forward(x.t(), gamma)
    with pytest.raises(ValueError):
        gpu_lib.norm_forward(x, gamma[:32])
    with pytest.raises(TypeError):
        gpu_lib.norm_forward(x, gamma, beta.float())
    with pytest.raises(gpu_lib.CklError):
        gpu_lib.norm_forward(x, gamma, eps=-1.0)
    with pytest.raises(TypeError):
        gpu_lib.norm_backward(dy, x.float(), mean, rstd, gamma)
    with pytest.raises(ValueError):
        gpu_lib.norm_backward(dy, x, mean, rstd[:3], gamma)
    with pytest.raises(ValueError):
        gpu_lib.norm_backward(dy, (kept[0], kept[1][:, :1]), mean, rstd, gamma)
    with pytest.raises(ValueError):
        gpu_lib.norm_backward(dy, x, mean, rstd, None, dgamma=torch.zeros(64, device="cuda"))
    with pytest.raises(ValueError):
        gpu_lib.norm_backward(dy, x, mean, rstd, gamma, accumulate=True)
    with pytest.raises(gpu_lib.CklError):
        gpu_lib.norm_backward(dy, x, mean, rstd, gamma,
                              workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(TypeError):
        gpu_lib.act8_unpack(*kept, dtype=torch.float16)

"""The norm's forms that rows, parameters and values choose: widths around the
vectors a thread holds, rows whose squares pass the largest float.  Tolerances
are those of test_gpu_norm.py."""

import pytest
import torch

import ops_ref
import test_gpu_norm
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


@pytest.mark.parametrize("d", [64, 65])
def test_act8_of_subnormal_groups(gpu_lib, d):
    g = torch.Generator(device="cuda").manual_seed(d)
    x = torch.rand(300, d, generator=g, device="cuda", dtype=torch.float64) * 2 - 1
    x *= torch.exp2(-149 + 29 * torch.rand(300, 1, generator=g, device="cuda", dtype=torch.float64))
    x = x.to(F32)
    q, e = gpu_lib.act8_pack(x)
    rq, re, val = ops_ref.act8(_np(x))
    assert (q.cpu().numpy() == rq).all() and (e.cpu().numpy() == re).all()
    for out in (BF, F32):
        assert (_np(gpu_lib.act8_unpack(q, e, out)) == val).all()
    # around the largest that b = 0 holds, 127.5 of its steps, and b = 1's: in bf16
    # every value is one of the steps, and comes back as it is
    step = torch.tensor([126.0, 127.0, 127.25, 127.5, 127.75, 128.0, 254.0, 254.5, 255.0, 256.0])
    x = (step.double()[:, None] * 2.0 ** -133).repeat(1, d).cuda()
    x[:, 1::3] *= -1
    for dtype in (BF, F32):
        for center in (None, True, False):               # alone, and kept by a norm's forward
            xt = x.to(dtype)
            if center is None:
                q, e = gpu_lib.act8_pack(xt)
            else:
                q, e = gpu_lib.norm_forward(xt, center=center, checkpoint=True)[3]
            rq, re, val = ops_ref.act8(_np(xt))
            assert (q.cpu().numpy() == rq).all() and (e.cpu().numpy() == re).all()
            if dtype == BF:
                small = (xt[:, 0] < 2.0 ** -126).nonzero()[:, 0]
                back = gpu_lib.act8_unpack(q, e)
                assert len(small) and torch.equal(back[small], xt[small])


def test_act8_at_every_largest_magnitude(gpu_lib):
    # every finite bf16 as a group's largest, and fp32's around where a scale ends
    bits = torch.arange(0x7F80, dtype=torch.int32, device="cuda")
    tops = (bits << 16).view(F32)
    mant = torch.tensor([0, 1, 0x400000, 0x7EFFFF, 0x7F0000, 0x7F0001, 0x7F7FFF, 0x7F8000, 0x7F8001,
                         0x7FFFFF], dtype=torch.int32, device="cuda")
    fine = ((torch.arange(255, dtype=torch.int32, device="cuda")[:, None] << 23) | mant).view(-1)
    for top, dtype in ((tops, BF), (fine.view(F32), F32)):
        part = torch.linspace(-1, 1, 40, device="cuda", dtype=torch.float64)
        x = (top.double()[:, None] * part).to(dtype)
        x[:, 5] = top.to(dtype)
        q, e = gpu_lib.act8_pack(x)
        rq, re, val = ops_ref.act8(_np(x))
        assert (q.cpu().numpy() == rq).all() and (e.cpu().numpy() == re).all()
        assert (_np(gpu_lib.act8_unpack(q, e, dtype)) == val).all()


def _unused(*a, **kw):
    raise AssertionError("not asked for")


@pytest.mark.parametrize("T,d", [(9, 72), (700, 2880), (1300, 4096), (300, 1001), (70, 20000)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_weight_that_is_not_trained(gpu_lib, monkeypatch, T, d, dtype):
    # only what is asked for: no sums over the rows, no memory for them
    x, gamma, beta, dy = _make(T, d, dtype, seed=23)
    y, mean, rstd, kept = gpu_lib.norm_forward(x, gamma, beta, checkpoint=True)
    for src in (x, kept):
        dx, dg, db = gpu_lib.norm_backward(dy, src, mean, rstd, gamma, bias=True)
        only = gpu_lib.norm_backward(dy, src, mean, rstd, gamma, bias=True, weight=False)
        assert torch.equal(only[0], dx) and only[1] is None and torch.equal(only[2], db)
    with pytest.raises(ValueError):
        gpu_lib.norm_backward(dy, x, mean, rstd, gamma, dgamma=torch.zeros(d, device="cuda"),
                              weight=False)
    dx = gpu_lib.norm_backward(dy, x, mean, rstd, gamma)[0]
    monkeypatch.setattr(gpu_lib._ops, "norm_workspace_bytes", _unused)
    alone = gpu_lib.norm_backward(dy, x, mean, rstd, gamma, weight=False)
    assert torch.equal(alone[0], dx) and alone[1:] == (None, None)
    xs = x.clone().requires_grad_()
    gpu_lib.layer_norm(xs, gamma, beta).backward(dy)      # gamma and beta are no leaves
    assert torch.equal(xs.grad, dx) and gamma.grad is None


def test_norm_kl_loss_makes_what_needs_a_gradient(gpu_lib, monkeypatch):
    x, gamma, beta, _ = _make(60, 128, BF, seed=24)
    W = (torch.randn(500, 128, device="cuda") * 0.1).to(BF)
    idx = torch.randint(0, 500, (60, 8), device="cuda", dtype=torch.int32)
    logp = torch.zeros(60, 8, device="cuda")
    full = [t.clone().requires_grad_() for t in (x, gamma, beta, W)]
    gpu_lib.norm_kl_loss(*full, idx, logp).backward()
    for need in ((0,), (1,), (0, 3), (2, 3), (3,)):
        leaves = [t.clone().requires_grad_(i in need) for i, t in enumerate((x, gamma, beta, W))]
        with monkeypatch.context() as m:
            if need == (3,):                              # the head alone: no norm behind it
                m.setattr(gpu_lib._ops, "norm_backward", _unused)
            if not {1, 2} & set(need):
                m.setattr(gpu_lib._ops, "norm_workspace_bytes", _unused)
            gpu_lib.norm_kl_loss(*leaves, idx, logp).backward()
        for i, (a, b) in enumerate(zip(leaves, full)):
            if i not in need:
                assert a.grad is None
            else:
                # the head's fp32 sums (500 terms: 2^-14 of the largest) may be taken
                # in another order, and a bf16 rounding with them (2^-7 of the value)
                p, q = a.grad.double(), b.grad.double()
                assert ((p - q).abs() <= 2.0 ** -7 * q.abs() + 2.0 ** -14 * q.abs().max()).all()


@pytest.mark.parametrize("T,d", [(400, 72), (400, 2880), (1300, 1280), (1300, 4096), (310, 7176),
                                 (310, 16384), (400, 1001), (1300, 17), (320, 17000), (300, 8300),
                                 (300, 9001)])
@pytest.mark.parametrize("dtype,pdtype", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)])
def test_many_rows_without_centring_and_with_other_parameters(gpu_lib, T, d, dtype, pdtype):
    # more rows than keep the parameters in registers: from shared memory, and
    # where there are none
    x, gamma, beta, dy = _make(T, d, dtype, seed=25, pdtype=pdtype)
    val = ops_ref.act8(_np(x))[2]
    for center, g, b in ((False, gamma, None), (False, None, None), (True, gamma, None),
                         (True, None, beta), (True, None, None), (False, gamma, beta)):
        _, mean, rstd, kept = _check_forward(gpu_lib, x, g, b, center, checkpoint=g is not None)
        _check_backward(gpu_lib, dy, x, _np(x), mean, rstd, g, bias=b is not None)
        if kept is not None:
            _check_backward(gpu_lib, dy, kept, val, mean, rstd, g, bias=b is not None)


@pytest.mark.parametrize("T,d", [(5000, 8), (3000, 1001), (2000, 96), (1300, 2880), (1300, 2560),
                                 (1300, 20000), (1300, 9001), (700, 16384), (3000, 64)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_in_place_with_many_rows_a_group(gpu_lib, T, d, dtype):
    # rows fetched ahead while earlier ones are overwritten
    x, gamma, beta, dy = _make(T, d, dtype, seed=26)
    for kept8 in (False, True):
        y, mean, rstd, kept = gpu_lib.norm_forward(x, gamma, beta, checkpoint=kept8)
        a = x.clone()
        got = gpu_lib.norm_forward(a, gamma, beta, checkpoint=kept8, out=a)
        assert got[0] is a and torch.equal(a, y)
        assert torch.equal(got[1], mean) and torch.equal(got[2], rstd)
        if kept8:
            assert torch.equal(got[3][0], kept[0]) and torch.equal(got[3][1], kept[1])
        src = kept if kept8 else x
        ref = gpu_lib.norm_backward(dy, src, mean, rstd, gamma, bias=True)
        b = dy.clone()
        got = gpu_lib.norm_backward(b, src, mean, rstd, gamma, bias=True, out_dx=b)
        assert got[0] is b and all(torch.equal(p, q) for p, q in zip(got, ref))


@pytest.mark.parametrize("d", [32767, 65536, 100003])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_very_long_rows(gpu_lib, monkeypatch, d, dtype):
    # a thread adds d / 512 values of a row in a chain, beside the 40 adds over
    # the block and the further operations of test_gpu_norm.py's bound
    monkeypatch.setattr(test_gpu_norm, "C", (-(-d // 512) + 100) * ops_ref.U32)
    x, gamma, beta, dy = _make(70, d, dtype, seed=27)
    for center in (True, False):
        _, mean, rstd, kept = _check_forward(gpu_lib, x, gamma, beta, center, checkpoint=True)
        _check_backward(gpu_lib, dy, x, _np(x), mean, rstd, gamma)
        _check_backward(gpu_lib, dy, kept, ops_ref.act8(_np(x))[2], mean, rstd, gamma)


@pytest.mark.parametrize("center", [True, False])
def test_norm_kl_loss_captured(gpu_lib, center):
    # each replay gives the gradients of what the buffers then hold
    x, gamma, beta, _ = _make(200, 128, BF, seed=28)
    W = (torch.randn(1000, 128, device="cuda") * 0.1).to(BF)
    idx = torch.randint(0, 1000, (200, 16), device="cuda", dtype=torch.int32)
    logp = torch.log_softmax(torch.randn(200, 16, device="cuda"), 1)

    def step(*t):
        leaves = [v.requires_grad_() for v in t]
        xs, gs, Ws = leaves[0], leaves[1], leaves[-1]
        loss = gpu_lib.norm_kl_loss(xs, gs, leaves[2] if center else None, Ws, idx, logp,
                                    center=center, chunk=64)
        return [loss.detach()] + list(torch.autograd.grad(loss, leaves))

    data = (x, gamma, beta, W) if center else (x, gamma, W)
    ref = step(*[t.clone() for t in data])
    held = [torch.zeros_like(t) for t in data]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step(*[t.detach() for t in held])
    for _ in range(2):
        for h, t in zip(held, data):
            h.copy_(t)
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, ref):
            a, b = a.double(), b.double()
            assert ((a - b).abs() <= 2.0 ** -7 * b.abs() + 2.0 ** -14 * b.abs().max()).all()


def test_one_row_without_leading_dimensions_and_three(gpu_lib):
    x, gamma, beta, dy = _make(6, 48, F32, seed=29)
    for shape in ((2, 1, 3, 48), (6, 48)):
        xs, gs, bs = (t.clone().requires_grad_() for t in (x.view(shape), gamma, beta))
        y = gpu_lib.layer_norm(xs, gs, bs)
        y.backward(dy.view(shape))
        if shape == (2, 1, 3, 48):
            first = (y, xs.grad, gs.grad, bs.grad)
    assert all(torch.equal(a.reshape(b.shape), b)
               for a, b in zip(first, (y, xs.grad, gs.grad, bs.grad)))
    one = x[0].clone().requires_grad_()
    y1 = gpu_lib.rms_norm(one, gamma, checkpoint=True)
    y1.backward(dy[0])
    assert one.grad.shape == (48,)
    y2, _, r, kept = gpu_lib.norm_forward(x[:1], gamma, None, 1e-6, False, True)
    assert torch.equal(y1, y2[0])
    dx = gpu_lib.norm_backward(dy[:1], kept, None, r, gamma)[0]
    assert torch.equal(one.grad, dx[0])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 4096, 16384, 20000])
def test_arrays_at_any_element(gpu_lib, d, dtype):
    # whole vectors of elements at addresses that no vector has
    x, gamma, beta, dy = _make(7, d, dtype, seed=30)

    def at(t, k):
        b = torch.empty(t.numel() + k, dtype=t.dtype, device="cuda")[k:].view(t.shape)
        return b.copy_(t)

    q, e = gpu_lib.act8_pack(x)
    q1, e1 = gpu_lib.act8_pack(at(x, 1))
    assert torch.equal(q, q1) and torch.equal(e, e1)
    y, mean, rstd, kept = gpu_lib.norm_forward(x, gamma, beta, checkpoint=True)
    assert torch.equal(kept[0], q) and torch.equal(kept[1], e)
    for k in (1, 3, 4):
        qs, es = at(q, k), at(e, k)
        for out in (BF, F32):
            assert torch.equal(gpu_lib.act8_unpack(qs, es, out), gpu_lib.act8_unpack(q, e, out))
        _check_backward(gpu_lib, dy, (qs, es), ops_ref.act8(_np(x))[2], mean, rstd, gamma)
        _check_backward(gpu_lib, dy, at(x, k), _np(x), mean, rstd, gamma)
        _check_forward(gpu_lib, x, at(gamma, k), beta, True, checkpoint=True)
        _check_forward(gpu_lib, x, gamma, beta, True, out=at(torch.zeros_like(x), k))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [40, 17, 33, 320, 1280])
def test_backward_of_a_large_constant_row(gpu_lib, d, dtype):
    # mean r passes the largest float; the row's own x - mean is 0, so xh is 0 and
    # dx = r (a - mean(a)); what stands behind the row must not count
    for T in (3, 700):
        x, gamma, beta, dy = _make(T, d, dtype, seed=31)
        x[1] = 2.0 ** 110
        _, mean, rstd, kept = gpu_lib.norm_forward(x, gamma, beta, eps=1e-12, checkpoint=True)
        assert mean[1] == 2.0 ** 110 and rstd[1] > 9e5
        r, a = _np(rstd)[1], _np(dy)[1] * _np(gamma)
        ref = r * (a - a.mean())
        for src in (x, kept):
            dx, dg, db = gpu_lib.norm_backward(dy, src, mean, rstd, gamma, bias=True)
            tol = 1.01 * ops_ref.HALF[dtype] * abs(ref) + 100 * ops_ref.U32 * r * (abs(a) + abs(a).mean())
            assert (abs(_np(dx)[1] - ref) <= tol).all()
            assert torch.isfinite(dx).all() and torch.isfinite(dg).all()

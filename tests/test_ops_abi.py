"""The operators' C ABI and binding without a GPU: exported symbols and the
arguments that are refused on the host."""

import ctypes
import os
import re

import numpy as np
import pytest
import torch

import ops_ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4097)
N = None


@pytest.fixture(scope="module")
def ckl():
    import chunked_kl_loss_ckl_b200 as m
    return m


def test_header_declares_and_library_exports(ckl):
    src = open(os.path.join(ROOT, "include", "ckl_ops.h")).read()
    names = sorted(set(re.findall(r"CKL_API\s+[\w\s\*]+?\b(ckl_\w+)\s*\(", src)))
    assert names == ["ckl_act8_pack", "ckl_act8_unpack", "ckl_norm_backward", "ckl_norm_forward",
                     "ckl_norm_workspace_bytes", "ckl_sample"]
    raw = ctypes.CDLL(ckl.LIB_PATH)
    for name in names:
        assert hasattr(raw, name), name
    for name, value in re.findall(r"#define CKL_(ACT8_GROUP|SAMPLE_BAD_INPUT) (\d+)", src):
        assert getattr(ckl, name) == int(value)


def test_act8_refusals(ckl):
    f, g = ckl.lib.ckl_act8_pack, ckl.lib.ckl_act8_unpack
    assert f(F, 0, -1, 8, F, F, N) == 1
    assert f(F, 0, 4, 0, F, F, N) == 1
    assert f(F, 2, 4, 8, F, F, N) == 1               # no such dtype
    assert f(F, 0, 1 << 61, 8, F, F, N) == 1         # T d out of range
    assert f(N, 0, 4, 8, F, F, N) == 1
    assert f(F, 0, 4, 8, N, F, N) == 1
    assert f(F, 0, 4, 8, F, N, N) == 1
    assert f(ODD, 0, 4, 8, F, F, N) == 1
    assert g(F, N, 4, 8, 0, F, N) == 1
    assert g(F, F, 4, 8, 3, F, N) == 1
    assert g(F, F, 4, 8, 1, ctypes.c_void_p(4098), N) == 1


def test_norm_refusals(ckl):
    f, b = ckl.lib.ckl_norm_forward, ckl.lib.ckl_norm_backward
    w = ckl.lib.ckl_norm_workspace_bytes
    ok = [F, 0, F, F, 0, 4, 64, 1e-5, F, F, F, N, N, N]

    def fwd(**kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return f(*a)

    assert fwd(_1=2) == 1 and fwd(_4=-1) == 1
    assert fwd(_5=-1) == 1 and fwd(_6=0) == 1
    assert fwd(_6=1 << 31) == 1 and fwd(_5=1 << 55) == 1
    assert fwd(_7=-1.0) == 1 and fwd(_7=float("nan")) == 1 and fwd(_7=float("inf")) == 1
    assert fwd(_0=N) == 1 and fwd(_8=N) == 1 and fwd(_10=N) == 1
    assert fwd(_11=F) == 1 and fwd(_12=F) == 1         # q and exponents go together
    assert fwd(_0=ODD) == 1 and fwd(_2=ODD) == 1 and fwd(_9=ctypes.c_void_p(4098)) == 1
    okb = [F, 0, F, N, N, F, F, F, 0, 4, 64, F, F, F, 0, F, 1 << 20, N]

    def bwd(**kw):
        a = list(okb)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return b(*a)

    assert bwd(_0=N) == 1 and bwd(_6=N) == 1 and bwd(_11=N) == 1
    assert bwd(_2=N) == 1 and bwd(_2=N, _3=F) == 1     # neither x nor both of q, exponents
    assert bwd(_15=N) == 1 and bwd(_15=ctypes.c_void_p(4104)) == 1
    assert bwd(_16=w(4, 64) - 1) == 3
    assert bwd(_10=1 << 31) == 1
    assert w(-1, 64) == 0 and w(4, 0) == 0 and w(4, 1 << 31) == 0
    assert w(0, 64) > 0 and w(4, 64) == 4 * 64 * 8
    assert w(1 << 30, 4096) <= 592 * 4096 * 8          # does not grow with T for ever


def test_sample_refusals(ckl):
    f = ckl.lib.ckl_sample
    #      z  ld  T  V  u  N  temp k  p    mp   rows          ids logp st stream
    ok = [F, 64, 4, 64, F, 1, 1.0, 0, 1.0, 0.0, N, N, N, N, F, F, N, N]

    def s(**kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return f(*a)

    assert s(_1=63) == 1 and s(_2=-1) == 1 and s(_3=0) == 1 and s(_5=0) == 1
    assert s(_2=1 << 30, _5=4) == 1                    # T N out of range
    assert s(_1=1 << 60, _2=16) == 1
    assert s(_0=N) == 1 and s(_4=N) == 1 and s(_14=N) == 1
    assert s(_0=ODD) == 1 and s(_4=ctypes.c_void_p(4098)) == 1 and s(_16=ODD) == 1
    for bad in (-1.0, float("nan"), float("inf")):
        assert s(_6=bad) == 1
    for bad in (0.0, -0.5, float("nan")):
        assert s(_8=bad) == 1
    for bad in (-0.1, 1.5, float("nan")):
        assert s(_9=bad) == 1
    assert s(_1=1 << 23, _3=(1 << 21) + 1) == 2


def test_binding_refuses_cpu_tensors(ckl):
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        ckl.norm_forward(x)
    with pytest.raises(ValueError):
        ckl.norm_backward(x, x, None, torch.zeros(4))
    with pytest.raises(ValueError):
        ckl.act8_pack(x)
    with pytest.raises(ValueError):
        ckl.act8_unpack(x.to(torch.int8), torch.zeros(4, 2, dtype=torch.uint8))
    with pytest.raises(ValueError):
        ckl.sample(x.to(torch.bfloat16), torch.zeros(4))


def test_reference_act8_is_within_its_bound():
    rng = np.random.default_rng(0)
    x = rng.normal(0, 1, (64, 70)) * np.exp(rng.uniform(-30, 30, (64, 1)))
    q, e, val = ops_ref.act8(x)
    pad = np.pad(np.abs(x), ((0, 0), (0, 26))).reshape(64, 3, 32).max(2)
    assert (np.abs(val - x) <= np.repeat(pad, 32, 1)[:, :70] / 127 + 1e-300).all()
    # the smallest scale that holds the largest: half of it would not
    assert (np.abs(q.astype(int)).max(1) >= 64).all()


def test_reference_norm_gradients_match_differences():
    rng = np.random.default_rng(1)
    for center in (True, False):
        x, dy = rng.normal(0.5, 1, (3, 11)), rng.normal(0, 1, (3, 11))
        g, b = rng.normal(1, 0.1, 11), rng.normal(0, 0.1, 11)
        f = lambda x, g, b: (ops_ref.norm(x, g, b, 1e-5, center)[0] * dy).sum()  # noqa: E731
        _, _, r, xh = ops_ref.norm(x, g, b, 1e-5, center)
        dx, dg, db = ops_ref.norm_grads(dy, xh, r, g, center)
        h = 1e-6
        for (i, j) in ((0, 0), (1, 5), (2, 10)):
            e = np.zeros_like(x)
            e[i, j] = h
            assert abs((f(x + e, g, b) - f(x - e, g, b)) / (2 * h) - dx[i, j]) < 1e-7
            e = np.zeros(11)
            e[j] = h
            assert abs((f(x, g + e, b) - f(x, g - e, b)) / (2 * h) - dg[j]) < 1e-7
            assert abs((f(x, g, b + e) - f(x, g, b - e)) / (2 * h) - db[j]) < 1e-7


def test_sample_takes_every_count_of_draws_that_the_header_names(ckl):
    # T N < 2^31; a vocabulary past the largest is refused next, before anything
    # is launched
    f = ckl.lib.ckl_sample

    def s(T, draws):
        return f(F, 1 << 23, T, (1 << 21) + 1, F, draws, 1.0, 0, 1.0, 0.0, N, N, N, N, F, F, N, N)

    top = 2 ** 31 - 1
    for T, draws in ((1, top), (top, 1), (1, 1 << 30), (2, (1 << 30) - 1), (2, 800_000_000),
                     (3, 715_827_882), (7, 306_783_378)):
        assert s(T, draws) == 2, (T, draws)
    for T, draws in ((1 << 31, 1), (2, 1 << 30), (3, 715_827_883), (top, 2), (46341, 46341)):
        assert s(T, draws) == 1, (T, draws)


def test_norm_workspace_is_what_the_sums_take(ckl):
    # 2 d floats a part: a part an SM (160 at most), and for rows that no thread
    # holds (d > 16384) a part for 64 rows, 64 at most
    w = ckl.lib.ckl_norm_workspace_bytes
    for d in (1, 64, 4096, 16384):
        for T in (1, 7, 148, 160, 161, 8192, 1 << 30):
            assert w(T, d) == min(T, 160) * d * 8
    for d in (16385, 20000, 1 << 20):
        for T in (1, 64, 65, 1000, 4096, 4097, 1 << 30):
            assert w(T, d) == min(-(-T // 64), 64) * d * 8
    assert w(0, 64) == 64 * 8 and w(0, 20000) == 20000 * 8


def test_reference_act8_bound_of_subnormal_groups():
    # b = 0 has the smallest step, 2^-133: fp32 groups below 2^-127 are off by up to
    # half of it, which is more than largest / 127
    rng = np.random.default_rng(2)
    x = rng.uniform(-1, 1, (400, 32)) * np.exp2(rng.uniform(-149, -120, (400, 1)))
    x = x.astype(np.float32).astype(np.float64)
    x[0] = 1.4 * 2.0 ** -134
    x[1] = 2.0 ** -134                               # half a step: to even, 0
    q, e, val = ops_ref.act8(x)
    top, err = np.abs(x).max(1, keepdims=True), np.abs(val - x)
    assert (err <= np.maximum(top / 127, 2.0 ** -134)).all()
    assert (err[0] > 0.4 * x[0]).all() and not val[1].any()
    assert (e[top[:, 0] < 2.0 ** -127] == 0).all()

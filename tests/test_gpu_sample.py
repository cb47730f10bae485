"""Sampling from logits against a 64-bit plain form: the ids are equal (weights
and sums are fp64 on both sides), the log-probs are within fp32's half step."""

import numpy as np
import pytest
import torch

import ops_ref
from ops_ref import U32

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
LAST = 1.0 - 2.0 ** -24   # the largest number below 1


def _z(T, V, seed, scale=2.0):
    rng = np.random.default_rng(seed)
    z = rng.normal(0, scale, (T, V))
    k = min(V, 20)
    for t in range(T):
        z[t, rng.choice(V, k, replace=False)] += rng.uniform(0, 10, k)
    return torch.from_numpy(z).to(BF), rng


def _num(v, t):
    return v if not isinstance(v, torch.Tensor) else v[t].item()


def _check(ckl, z, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, rows=None, status=0):
    zd = z if z.is_cuda else z.cuda()
    ud = torch.as_tensor(u, dtype=torch.float32).cuda()
    par = [p.cuda() if isinstance(p, torch.Tensor) else p for p in (temperature, top_k, top_p, min_p)]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ids, logp = ckl.sample(zd, ud, *par, status=st)
    assert ids.shape == ud.shape and logp.shape == ud.shape
    assert st.item() == status
    T = z.shape[0]
    ids, logp = ids.view(T, -1).cpu().numpy(), logp.view(T, -1).double().cpu().numpy()
    un = ud.view(T, -1).double().cpu().numpy()
    for t in (range(T) if rows is None else rows):
        ri, rl = ops_ref.sample(z[t].double().cpu().numpy(), un[t], _num(temperature, t),
                                int(_num(top_k, t)), _num(top_p, t), _num(min_p, t))
        assert np.array_equal(ids[t], ri), (t, ids[t], ri)
        assert np.array_equal(np.isnan(logp[t]), np.isnan(rl))
        ok = ~np.isnan(rl)
        # both are rounded from 64 bits: half a step, and 64-bit noise near 0
        assert (np.abs(logp[t] - rl)[ok] <= 1.01 * U32 * np.abs(rl[ok]) + 1e-12).all()
    return ids, logp


FILTERS = [dict(), dict(temperature=0.7), dict(temperature=1.7), dict(temperature=0.0),
           dict(top_k=1), dict(top_k=7), dict(top_k=1000, temperature=1.3), dict(top_p=0.9),
           dict(top_p=1e-6), dict(top_p=0.5, top_k=40), dict(min_p=0.05), dict(min_p=1.0),
           dict(min_p=1e-9), dict(temperature=0.8, top_k=50, top_p=0.95, min_p=0.02),
           dict(temperature=30.0), dict(temperature=1e-3), dict(temperature=1e-320)]


@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 33, 256, 257, 1001, 2048, 2049, 4096, 4097, 50257])
def test_every_filter_at_every_size(gpu_lib, V):
    for i, f in enumerate(FILTERS):
        z, rng = _z(5, V, 10 * V + i)
        _check(gpu_lib, z, rng.random(5), **f)
        _check(gpu_lib, z, rng.random((5, 3)), **f)


@pytest.mark.parametrize("T", [1, 2, 9, 20, 40, 200])
def test_teacher_sized_rows(gpu_lib, T):
    z, rng = _z(T, 128256, T)
    rows = range(min(T, 6))
    for f in (dict(), dict(temperature=0.7, top_k=50, top_p=0.95), dict(top_p=0.8)):
        _check(gpu_lib, z, rng.random(T), rows=rows, **f)


@pytest.mark.parametrize("N", [2, 63, 64, 65, 130])
@pytest.mark.parametrize("V", [5, 999, 4099, 128256])
def test_many_draws_a_row(gpu_lib, N, V):
    z, rng = _z(3, V, N)
    ids, _ = _check(gpu_lib, z, rng.random((3, N)))
    assert V == 5 or len(np.unique(ids)) > 3
    _check(gpu_lib, z, rng.random((3, N)), temperature=1.2, top_p=0.9)
    _check(gpu_lib, z, np.full((3, N), 0.25))               # one value many times


def test_rows_far_more_than_blocks(gpu_lib):
    z, rng = _z(3000, 517, 1)
    _check(gpu_lib, z, rng.random(3000), top_p=0.95)
    z, rng = _z(1500, 300, 2)
    _check(gpu_lib, z, rng.random((1500, 5)))
    z, rng = _z(1000, 4500, 3)
    _check(gpu_lib, z, rng.random(1000), top_p=0.95, rows=range(0, 1000, 3))
    _check(gpu_lib, z, rng.random((1000, 3)), rows=range(0, 1000, 3))


@pytest.mark.parametrize("V", [1024, 8192])
def test_ties_and_borders(gpu_lib, V):
    # equal logits: u = k / V is the border of two tokens and draws the second
    z = torch.full((3, V), 0.5, dtype=BF)
    z[1] = 0.0
    z[1, ::2] = -0.0                                          # equal to +0
    z[2, :V // 2] = -1.0
    u = np.arange(V) / V
    ids, logp = _check(gpu_lib, z, np.stack([u, u, u]))
    assert np.array_equal(ids[0], np.arange(V)) and np.array_equal(ids[1], np.arange(V))
    assert (ids[2, 0] == V // 2) and np.allclose(logp[0], -np.log(V))
    # top-k and top-p cut inside a tie: the lowest ids stay
    ids, _ = _check(gpu_lib, z, np.stack([u, u, u]), top_k=3)
    assert set(ids[0]) == {0, 1, 2} and set(ids[2]) == {V // 2, V // 2 + 1, V // 2 + 2}
    ids, _ = _check(gpu_lib, z, np.stack([u, u, u]), top_p=0.25)
    assert set(ids[0]) == set(range(V // 4))
    rng = np.random.default_rng(3)
    grid = torch.from_numpy(np.round(rng.normal(0, 2, (40, 2 * V)) * 2) / 2).to(BF)
    for f in (dict(), dict(top_k=11), dict(top_p=0.6), dict(min_p=0.1)):
        _check(gpu_lib, grid, rng.random((40, 4)), **f)


@pytest.mark.parametrize("V", [2000, 6000])
def test_ends_of_the_unit_interval(gpu_lib, V):
    z, _ = _z(4, V, 5)
    u = np.tile([0.0, 2.0 ** -149, LAST], (4, 1))
    for f in FILTERS:
        _check(gpu_lib, z, u, **f)


@pytest.mark.parametrize("V", [1003, 5003])
def test_masked_rows(gpu_lib, V):
    z, rng = _z(8, V, 6)
    inf, low = float("-inf"), torch.finfo(BF).min
    z[0, 1:] = inf                       # one token left
    z[1] = inf                           # none left
    z[2, ::2] = low
    z[3, :] = low
    z[3, 77] = -3.0                      # one token above the type's lowest value
    z[4] = low                           # all of them equal, and lowest
    z[5, 100:] = inf
    z[6, :] = -1e4
    z[6, 3:9] = 2.0
    z[7, V - 1] = inf
    for f in (dict(), dict(top_p=0.9, temperature=0.6), dict(top_k=5), dict(min_p=0.1),
              dict(temperature=0.0), dict(temperature=1e4), dict(temperature=1e38)):
        _check(gpu_lib, z, rng.random(8), **f)
        ids, _ = _check(gpu_lib, z, rng.random((8, 3)), **f)
        assert (ids[0] == 0).all() and (ids[1] == -1).all()


@pytest.mark.parametrize("V", [1501, 5001])
def test_values_of_any_size(gpu_lib, V):
    # beyond the counters' range: tiny, huge, both, and all of the type
    rng = np.random.default_rng(7)
    z = torch.from_numpy(rng.normal(0, 1, (8, V))).to(BF)
    z[0, 5] = 1e-20
    z[1] = torch.from_numpy(rng.normal(0, 1, V) * 1e-30).to(BF)
    z[2] = torch.from_numpy(rng.normal(0, 1, V) * 1e30).to(BF)
    z[3] = torch.from_numpy(rng.normal(0, 1, V) + 300).to(BF)
    z[4] = torch.from_numpy(rng.normal(0, 1, V) - 300).to(BF)
    z[5] = torch.from_numpy(np.exp(rng.uniform(-80, 80, V))
                            * rng.choice([-1, 1], V)).to(BF)
    z[6, ::3] = -260.0
    z[7, 0] = 256.0
    z[7, 1] = 2.0 ** -133
    for f in (dict(), dict(top_k=9), dict(top_p=0.7), dict(min_p=0.01), dict(temperature=0.0),
              dict(temperature=20.0), dict(temperature=1e30, top_p=0.5),
              dict(temperature=0.9, top_k=100, top_p=0.9, min_p=0.001)):
        _check(gpu_lib, z, rng.random(8), **f)
        _check(gpu_lib, z, rng.random((8, 4)), **f)


@pytest.mark.parametrize("V", [700, 9001])
def test_bad_numbers(gpu_lib, V):
    z, rng = _z(6, V, 8)
    z[1, 13] = float("nan")
    z[2, V - 1] = float("inf")
    u = rng.random((6, 3))
    u[3, 1], u[4, 0], u[5, 2] = 1.0, -1e-9, np.nan
    ids, _ = _check(gpu_lib, z, u, status=16)
    assert (ids[1] == -1).all() and (ids[2] == -1).all() and (ids[3] >= 0).tolist() == [1, 0, 1]
    _check(gpu_lib, z, u[:, 2], status=16)
    z, _ = _z(6, V, 9)
    bad = float("nan")
    _check(gpu_lib, z, rng.random(6), status=16,
           temperature=torch.tensor([1.0, -1.0, bad, float("inf"), 1.0, 0.0]))
    _check(gpu_lib, z, rng.random(6), status=16, top_p=torch.tensor([1.0, 0.0, -1.0, bad, 2.0, 0.5]))
    _check(gpu_lib, z, rng.random(6), status=16, min_p=torch.tensor([0.0, -0.1, 1.1, bad, 1.0, 0.5]))


@pytest.mark.parametrize("V", [1700, 7001])
def test_parameters_per_row(gpu_lib, V):
    z, rng = _z(24, V, 10)
    pick = lambda v, dt: torch.tensor(rng.choice(v, 24), dtype=dt)  # noqa: E731
    for _ in range(3):
        _check(gpu_lib, z, rng.random((24, 2)),
               temperature=pick([0.0, 0.5, 1.0, 2.0], torch.float32),
               top_k=pick([-1, 0, 1, 50, 5000], torch.int32),
               top_p=pick([0.3, 0.9, 1.0, 3.0], torch.float32),
               min_p=pick([0.0, 0.05, 0.5], torch.float32))


@pytest.mark.parametrize("V", [1003, 5003])
def test_strided_rows_bit_types_and_repeats(gpu_lib, V):
    z, rng = _z(13, V, 11)
    wide = torch.full((13, V + 6), 50.0, dtype=BF, device="cuda")  # beside the rows: large
    for at in (0, 1, 5):
        v = wide[:, at:at + V]
        v.copy_(z)
        u = torch.from_numpy(rng.random((13, 9))).float()
        _check(gpu_lib, v, u)
        _check(gpu_lib, v, u[:, 0])
        wide.fill_(50.0)
    zc, u = z.cuda(), torch.rand(13, 9, device="cuda")
    a = gpu_lib.sample(zc, u)
    for dt in (torch.int16, torch.uint16):
        b = gpu_lib.sample(zc.view(dt), u)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    one = gpu_lib.sample(zc, u[:, 4].contiguous())
    assert torch.equal(one[0], a[0][:, 4]) and torch.equal(one[1], a[1][:, 4])


def test_wide_rows_and_far_offsets(gpu_lib):
    z, rng = _z(2, 300007, 12)                        # more than one step a tile
    _check(gpu_lib, z, rng.random(2))
    _check(gpu_lib, z, rng.random((2, 70)), top_p=0.95)
    z = torch.zeros(2, 1 << 21, dtype=BF)             # the widest, all equal: full counters
    z[1, 5] = 9.0
    _check(gpu_lib, z, rng.random(2))
    _check(gpu_lib, z, rng.random((2, 5)))
    big = torch.empty(18 * (1 << 27), dtype=BF, device="cuda").view(18, 1 << 27)
    for V in (1000, 5000):
        v = big[:, 7:7 + V]                           # row 17 starts past 2^31 elements
        z, rng = _z(18, V, 13)
        v.copy_(z)
        _check(gpu_lib, v, rng.random(18))


def test_streams_and_graphs(gpu_lib):
    z, _ = _z(50, 5000, 14)
    z, u = z.cuda(), torch.rand(50, 3, device="cuda")
    ref = gpu_lib.sample(z, u, top_p=0.9)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = gpu_lib.sample(z, u, top_p=0.9, stream=s)
    s.synchronize()
    assert torch.equal(got[0], ref[0])
    zs, us = torch.zeros_like(z), torch.zeros_like(u)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = gpu_lib.sample(zs, us, top_p=0.9)
        one = gpu_lib.sample(zs, us[:, 0].contiguous(), top_p=0.9)
    for _ in range(2):
        zs.copy_(z)
        us.copy_(u)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[0], ref[0]) and torch.equal(one[0], ref[0][:, 0])


def test_two_streams_at_once(gpu_lib):
    # nothing is shared between calls: both draw what they draw alone
    z, _ = _z(300, 20000, 16)
    z, u = z.cuda(), torch.rand(300, 70, device="cuda")
    ref = gpu_lib.sample(z, u, top_p=0.9), gpu_lib.sample(z, u[:, 0].contiguous(), top_k=7)
    torch.cuda.synchronize()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    one = u[:, 0].contiguous()
    torch.cuda.synchronize()
    for _ in range(5):
        a = gpu_lib.sample(z, u, top_p=0.9, stream=s[0])
        b = gpu_lib.sample(z, one, top_k=7, stream=s[1])
        torch.cuda.synchronize()
        assert torch.equal(a[0], ref[0][0]) and torch.equal(b[0], ref[1][0])


def test_frequencies_follow_the_distribution(gpu_lib):
    # 20000 draws: counts within six standard deviations of their means
    z = torch.linspace(0, 3, 17).to(BF)[None].cuda()
    n = 20000
    u = torch.rand(1, n, device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    ids, logp = gpu_lib.sample(z, u)
    p = torch.softmax(z.double(), 1)[0]
    cnt = torch.bincount(ids[0].long(), minlength=17).double()
    assert ((cnt - n * p).abs() <= 6 * (n * p * (1 - p)).sqrt()).all()
    assert (logp[0].double() - p.log()[ids[0].long()]).abs().max() < 1e-6


def test_empty_batch_and_refusals(gpu_lib):
    z, _ = _z(4, 64, 15)
    z = z.cuda()
    u = torch.rand(4, device="cuda")
    ids, logp = gpu_lib.sample(z[:0], u[:0])
    assert ids.shape == (0,) and logp.shape == (0,)
    with pytest.raises(TypeError):
        gpu_lib.sample(z.float(), u)
    with pytest.raises(ValueError):
        gpu_lib.sample(z[0], u)
    with pytest.raises(ValueError):
        gpu_lib.sample(z.t(), torch.rand(64, device="cuda"))
    with pytest.raises(ValueError):
        gpu_lib.sample(z[:1].expand(4, 64), u)
    with pytest.raises(ValueError):
        gpu_lib.sample(z, u[:3])
    with pytest.raises(TypeError):
        gpu_lib.sample(z, u.double())
    with pytest.raises(ValueError):
        gpu_lib.sample(z, u, temperature=torch.ones(3, device="cuda"))
    with pytest.raises(TypeError):
        gpu_lib.sample(z, u, top_k=torch.ones(4, device="cuda"))
    with pytest.raises(gpu_lib.CklError):
        gpu_lib.sample(z, u, temperature=-1.0)
    with pytest.raises(gpu_lib.CklError):
        gpu_lib.sample(z, torch.empty(4, 0, device="cuda"))


def test_counts_past_32_bits_do_not_wrap(gpu_lib):
    z = _z(3, 5000, 77)[0].cuda()
    u = torch.rand(3, device="cuda")
    every = gpu_lib.sample(z, u)
    for k in (2 ** 31, 2 ** 32 + 1, -1, -2 ** 32 + 1):
        got = gpu_lib.sample(z, u, top_k=k)
        assert torch.equal(got[0], every[0]) and torch.equal(got[1], every[1])

"""Sampling where rows share a block or a block is shared by rows: every number of
blocks a row, many draws, rows of other values and rows without an answer among
ordinary ones.  Compared with the 64-bit plain form as in test_gpu_sample.py."""

import threading

import numpy as np
import pytest
import torch

from test_gpu_sample import _check, _z

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.mark.parametrize("T", [3, 12, 13, 30, 33, 60, 74, 80, 148, 310])
def test_many_draws_at_every_number_of_blocks_a_row(gpu_lib, T):
    # 64 draws and more: 8, 4, 2 blocks a row, one, and several rows a block
    z, rng = _z(T, 50257, T)
    rows = sorted(set(range(0, T, max(1, T // 6))) | {T - 1})
    _check(gpu_lib, z, rng.random((T, 64)), rows=rows)
    _check(gpu_lib, z, rng.random((T, 130)), rows=rows[:3], temperature=1.1, top_p=0.9)
    _check(gpu_lib, z, np.tile(rng.random((T, 1)), (1, 70)), rows=rows[-3:], top_k=40)


@pytest.mark.parametrize("T", [2, 12, 40, 74, 220, 700])
@pytest.mark.parametrize("N", [1, 5])
def test_rows_of_every_kind_beside_each_other(gpu_lib, T, N):
    V = 6007
    z, rng = _z(T, V, 100 + T)
    kind = np.arange(T) % 9
    inf = float("inf")
    for t in range(T):
        k = kind[t]
        if k == 1:
            z[t, 5] = 2.0 ** -60                     # below the counters' range
        elif k == 2:
            z[t] += 260.0                            # above it
        elif k == 3:
            z[t, rng.integers(V)] = float("nan")
        elif k == 4:
            z[t] = -inf
        elif k == 5:
            z[t, 11:] = -inf
        elif k == 6:
            z[t] = z[t, 0]                           # one value
        elif k == 7:
            z[t, ::2] = torch.finfo(BF).min
        elif k == 8:
            z[t, V - 3:] = inf
    u = rng.random((T, N)) if N > 1 else rng.random(T)
    some = sorted(set(range(min(T, 18))) | set(range(max(0, T - 18), T)))
    bad = 16 if (kind == 3).any() or (kind == 8).any() else 0
    for f in (dict(), dict(temperature=0.0), dict(temperature=8.0, top_k=300),
              dict(top_p=0.8, min_p=0.01)):
        _check(gpu_lib, z, u, rows=some, status=bad, **f)


@pytest.mark.parametrize("V", [128256, 300007])
def test_other_values_in_long_rows(gpu_lib, V):
    z, rng = _z(3, V, 9)
    z[0, V - 1] = 2.0 ** -100
    z[1] += 300.0
    z[2, ::5] = -1e30
    _check(gpu_lib, z, rng.random(3))
    _check(gpu_lib, z, rng.random((3, 3)), top_p=0.9, temperature=30.0)


def test_two_host_threads(gpu_lib):
    work = []
    for i, (T, V, N) in enumerate(((40, 20000, 64), (300, 9000, 1))):
        z, rng = _z(T, V, i)
        z, u = z.cuda(), torch.from_numpy(rng.random((T, N))).float().cuda()
        work.append((z, u, gpu_lib.sample(z, u, top_p=0.9), torch.cuda.Stream()))
    torch.cuda.synchronize()
    bad = []

    def loop(z, u, ref, st):
        try:
            for _ in range(50):
                ids, logp = gpu_lib.sample(z, u, top_p=0.9, stream=st)
                st.synchronize()
                if not (torch.equal(ids, ref[0]) and torch.equal(logp, ref[1])):
                    bad.append("another result")
        except Exception as e:
            bad.append(repr(e))

    threads = [threading.Thread(target=loop, args=w) for w in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad[:3]

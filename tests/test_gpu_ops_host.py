"""What the operators' host side has to hold whatever else the process does:
calls from several threads, and errors of other calls."""

import ctypes
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def test_two_host_threads_at_different_widths(gpu_lib):
    # the same kernels with another amount of shared memory each
    ckl = gpu_lib
    work = []
    for d in (2880, 4096):
        x = torch.randn(1300, d, device="cuda").to(BF)
        gamma, beta = torch.randn(d, device="cuda").to(BF), torch.randn(d, device="cuda").to(BF)
        y, mean, rstd, _ = ckl.norm_forward(x, gamma, beta)
        dx = ckl.norm_backward(y, x, mean, rstd, gamma)[0]
        work.append((x, gamma, beta, y, mean, rstd, dx, torch.cuda.Stream(), torch.empty_like(x),
                     torch.empty_like(x), torch.empty_like(mean), torch.empty_like(rstd)))
    torch.cuda.synchronize()
    start, bad = threading.Barrier(2), []

    def loop(x, gamma, beta, y, mean, rstd, dx, st, y1, dx1, mean1, rstd1):
        T, d = x.shape
        p = [t.data_ptr() for t in (x, gamma, beta, y1, mean1, rstd1, y, dx1)]
        start.wait()
        for _ in range(3000):
            rc = (ckl.lib.ckl_norm_forward(p[0], 0, p[1], p[2], 0, T, d, 1e-5, *p[3:6], None, None,
                                           st.cuda_stream),
                  ckl.lib.ckl_norm_backward(p[6], 0, p[0], None, None, p[4], p[5], p[1], 0, T, d,
                                            p[7], None, None, 0, None, 0, st.cuda_stream))
            if any(rc):
                bad.append((d, rc))
        st.synchronize()
        if not (torch.equal(y, y1) and torch.equal(dx, dx1)):
            bad.append((d, "another result"))

    threads = [threading.Thread(target=loop, args=w) for w in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, (len(bad), bad[:4])


class _RefusedLaunches:
    """Within it a launch into the default stream fails on the host: another
    stream that waits for that one is being captured."""

    def __init__(self):
        self.rt = ctypes.CDLL("libcudart.so.12")     # torch's, loaded already
        self.st, self.graph = ctypes.c_void_p(), ctypes.c_void_p()
        assert self.rt.cudaStreamCreate(ctypes.byref(self.st)) == 0

    def __enter__(self):
        assert self.rt.cudaStreamBeginCapture(self.st, 2) == 0

    def __exit__(self, *exc):
        self.rt.cudaStreamEndCapture(self.st, ctypes.byref(self.graph))
        self.rt.cudaGetLastError()                   # torch's own copy of the error
        assert self.rt.cudaStreamDestroy(self.st) == 0


@pytest.mark.parametrize("what", ["sample", "short", "norm", "reduce", "act8", "duplicates"])
def test_a_failed_call_is_no_later_call_s_error(gpu_lib, what):
    ckl = gpu_lib
    x = torch.randn(6, 8192, device="cuda").to(BF)
    dy = torch.randn_like(x)
    gamma = torch.ones(8192, dtype=BF, device="cuda")
    u = torch.rand(6, device="cuda")
    idx = torch.zeros(6, 4, dtype=torch.int32, device="cuda")
    first = torch.zeros(1, dtype=torch.int32, device="cuda")
    y, mean, rstd, _ = ckl.norm_forward(x, gamma)
    dx, dg, _ = ckl.norm_backward(dy, x, mean, rstd, gamma)
    q, e = ckl.act8_pack(x)
    ids, logp = ckl.sample(x, u)
    ckl.sample(x[:, :500], u)
    ws = torch.empty(ckl.norm_workspace_bytes(6, 8192), dtype=torch.uint8, device="cuda")
    p = {k: v.data_ptr() for k, v in dict(x=x, dy=dy, g=gamma, u=u, idx=idx, first=first, mean=mean,
                                          rstd=rstd, q=q, e=e, ids=ids, logp=logp, ws=ws, dx=dx,
                                          dg=dg, y=y).items()}
    call = {
        "sample": lambda: ckl.lib.ckl_sample(p["x"], 8192, 6, 8192, p["u"], 1, 1.0, 0, 1.0, 0.0,
                                             None, None, None, None, p["ids"], p["logp"], None,
                                             None),
        "short": lambda: ckl.lib.ckl_sample(p["x"], 8192, 6, 500, p["u"], 1, 1.0, 0, 1.0, 0.0, None,
                                            None, None, None, p["ids"], p["logp"], None, None),
        "norm": lambda: ckl.lib.ckl_norm_forward(p["x"], 0, p["g"], None, 0, 6, 8192, 1e-5, p["y"],
                                                 p["mean"], p["rstd"], None, None, None),
        "reduce": lambda: ckl.lib.ckl_norm_backward(p["dy"], 0, p["x"], None, None, p["mean"],
                                                    p["rstd"], p["g"], 0, 0, 8192, p["dx"], p["dg"],
                                                    None, 0, p["ws"], ws.numel(), None),
        "act8": lambda: ckl.lib.ckl_act8_pack(p["x"], 0, 6, 8192, p["q"], p["e"], None),
        "duplicates": lambda: ckl.lib.ckl_find_duplicate_ids(p["idx"], 6, 4, p["first"], None),
    }[what]
    torch.cuda.synchronize()
    with _RefusedLaunches():
        assert call() == 4
    # valid calls, each the first one after the failed call
    a = ckl.act8_pack(x)
    assert torch.equal(a[0], q)
    with _RefusedLaunches():
        assert call() == 4
    assert torch.equal(ckl.norm_forward(x, gamma)[0], y)
    with _RefusedLaunches():
        assert call() == 4
    assert torch.equal(ckl.sample(x, u)[0], ids)
    with _RefusedLaunches():
        assert call() == 4
    got = ckl.sample(x[:, :500], u)
    assert got[0].max() < 500
    assert call() == 0
    torch.cuda.synchronize()

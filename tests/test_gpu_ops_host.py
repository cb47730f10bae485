"""What the operators' host side has to hold whatever else the process does:
calls from several threads."""

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

"""The operators as a distillation step uses them: final norm, head loss against
a teacher cache (sampled or top-K), its backward, the norm's backward (from x
or from its 8 bits), against 64-bit plain forms of the whole step."""

import numpy as np
import pytest
import torch

import ops_ref
import oracle
from gpu_util import GRAD_RFRO, LOSS_RTOL, rel_fro

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _bits(t):
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


def _problem(T=200, d=128, V=1000, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = (3 * r(T, d) + 0.5).to(BF)
    gamma, beta = (1 + 0.2 * r(d)).to(BF), (0.1 * r(d)).to(BF)
    W = (r(V, d) * d ** -0.5).to(BF)
    teacher = (2 * r(T, V)).to(BF)
    mask = (torch.rand(T, generator=g, device="cuda") > 0.1).to(torch.uint8)
    u = torch.rand(T, 24, generator=g, device="cuda")
    return x, gamma, beta, W, teacher, mask, u


def _reference(x, gamma, beta, W, idx, logp, mask, H, xv):
    """Loss and gradients: the head's from the H the GPU made (its rounding is
    the norm's own, tested elsewhere), the norm's through xv."""
    ref = oracle.dense(_bits(H), _bits(W), idx.cpu().numpy(), logp.cpu().numpy(),
                       mask.cpu().numpy())
    n = lambda t: t.double().cpu().numpy()  # noqa: E731
    _, mu, r, _ = ops_ref.norm(n(x), None, None, 1e-5, True)
    xh = (xv - mu[:, None]) * r[:, None]
    dx, dg, db = ops_ref.norm_grads(ref["dH"], xh, r, n(gamma), True)
    return ref["loss"], dx, dg, db, ref["dW"]


@pytest.mark.parametrize("cache", ["topk", "sampled"])
@pytest.mark.parametrize("how", ["ops", "checkpoint", "norm_kl_loss"])
def test_distillation_step(gpu_lib, cache, how):
    ckl = gpu_lib
    x, gamma, beta, W, teacher, mask, u = _problem()
    if cache == "topk":
        idx, logp, _ = ckl.topk_cache(teacher, 24)
    else:
        idx, _ = ckl.sample(teacher, u)
        logp = torch.zeros_like(u)                 # equal weights, repeats as they are
    leaves = [t.clone().requires_grad_() for t in (x, gamma, beta, W)]
    if how == "norm_kl_loss":
        loss = ckl.norm_kl_loss(*leaves, idx, logp, mask, chunk=64)
    else:
        H = ckl.layer_norm(*leaves[:3], checkpoint=how == "checkpoint")
        loss = ckl.chunked_kl_loss(H, leaves[3], idx, logp, mask, chunk=64)
    loss.backward()
    torch.cuda.synchronize()
    H = ckl.norm_forward(x, gamma, beta)[0]
    xv = x.double().cpu().numpy()
    if how == "checkpoint":
        xv = ops_ref.act8(xv)[2]
    ref = _reference(x, gamma, beta, W, idx, logp, mask, H, xv)
    assert abs(loss.item() - ref[0]) <= LOSS_RTOL * abs(ref[0])
    for leaf, g in zip(leaves, ref[1:]):
        # the gradients' bf16 rounding adds 2^-8 to the loss's own bound
        assert rel_fro(leaf.grad.double().cpu().numpy(), g) <= GRAD_RFRO + 2.0 ** -8


def test_both_forms_of_the_loss_agree_to_the_bit(gpu_lib):
    ckl = gpu_lib
    x, gamma, beta, W, teacher, mask, _ = _problem(seed=1)
    idx, logp, _ = ckl.topk_cache(teacher, 16)
    out = []
    for path in (0, 1):
        leaves = [t.clone().requires_grad_() for t in (x, gamma, beta, W)]
        if path:
            loss = ckl.norm_kl_loss(*leaves, idx, logp, mask, chunk=64)
        else:
            loss = ckl.chunked_kl_loss(ckl.layer_norm(*leaves[:3]), leaves[3], idx, logp, mask, 64)
        loss.backward()
        out.append([loss] + [t.grad for t in leaves])
    assert all(torch.equal(a, b) for a, b in zip(*out))


def test_rms_norm_head_and_sampling_from_the_student(gpu_lib):
    ckl = gpu_lib
    x, gamma, _, W, teacher, mask, u = _problem(seed=2)
    idx, logp, _ = ckl.topk_cache(teacher, 16)
    leaves = [t.clone().requires_grad_() for t in (x, gamma, W)]
    loss = ckl.norm_kl_loss(leaves[0], leaves[1], None, leaves[2], idx, logp, mask, center=False)
    loss.backward()
    assert all(torch.isfinite(t.grad).all() for t in leaves)
    # the student's own tokens: ids and log-probs of its logits
    H = ckl.norm_forward(x, gamma, center=False)[0]
    z = (H.float() @ W.float().t()).to(BF)
    ids, lp = ckl.sample(z, u[:, 0].contiguous())
    ref = torch.log_softmax(z.double(), 1).gather(1, ids.long()[:, None])[:, 0]
    assert (lp.double() - ref).abs().max() < 1e-5


@pytest.mark.parametrize("checkpoint", [False, True])
def test_both_passes_captured_by_autograd(gpu_lib, checkpoint):
    """Forward and backward of the chain in one graph: each replay gives the
    gradients of what the buffers then hold.  The order of fp32 sums may differ
    from the eager call's (1000 terms: 2^-14 of the largest), and with it a
    bf16 rounding (2^-7 of the value)."""
    ckl = gpu_lib
    x, gamma, beta, W, teacher, mask, u = _problem(seed=3)
    idx, logp, _ = ckl.topk_cache(teacher, 24)

    def step(x, gamma, beta, W):
        leaves = [t.requires_grad_() for t in (x, gamma, beta, W)]
        H = ckl.layer_norm(*leaves[:3], checkpoint=checkpoint)
        loss = ckl.chunked_kl_loss(H, leaves[3], idx, logp, mask, chunk=64)
        return torch.autograd.grad(loss, leaves)

    ref = step(*[t.clone() for t in (x, gamma, beta, W)])
    held = [torch.zeros_like(t) for t in (x, gamma, beta, W)]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step(*[t.detach() for t in held])
    for _ in range(2):
        for h, t in zip(held, (x, gamma, beta, W)):
            h.copy_(t)
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, ref):
            a, b = a.double(), b.double()
            assert ((a - b).abs() <= 2.0 ** -7 * b.abs() + 2.0 ** -14 * b.abs().max()).all()


def test_norm_kl_loss_refusals(gpu_lib):
    ckl = gpu_lib
    x, gamma, beta, W, teacher, mask, u = _problem(T=8, V=64)
    idx, logp, _ = ckl.topk_cache(teacher, 4)
    for bad in ((x.float(), gamma, beta, W, idx, logp, mask),
                (x, gamma.half(), beta, W, idx, logp, mask)):
        with pytest.raises(TypeError):
            ckl.norm_kl_loss(*bad)
    for bad in ((x.cpu(), gamma, beta, W, idx, logp, mask),
                (x, gamma, beta, W.cpu(), idx, logp, mask),
                (x, gamma, beta, W, idx, logp, mask.cpu()),
                (x, gamma[:-1].contiguous(), beta, W, idx, logp, mask),
                (x.t(), gamma, beta, W, idx, logp, mask),
                (x, gamma, beta, W[:, :-8].contiguous(), idx, logp, mask)):
        with pytest.raises(ValueError):
            ckl.norm_kl_loss(*bad)
    assert torch.isfinite(ckl.norm_kl_loss(x, gamma, beta, W, idx, logp, mask))

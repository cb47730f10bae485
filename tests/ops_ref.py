"""Plain 64-bit forms of the operators around the loss, for the tests."""

from __future__ import annotations

import numpy as np
import torch

U32 = 2.0 ** -24   # half a step of fp32, relative
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def act8(x):
    """(q, exponents, values) of float64 rows [T, d], element by element as the
    header defines them."""
    x = np.asarray(x, np.float64)
    T, d = x.shape
    G = -(-d // 32)
    q = np.zeros((T, d), np.int8)
    e = np.zeros((T, G), np.uint8)
    val = np.empty((T, d))
    for g in range(G):
        s = slice(32 * g, min(d, 32 * g + 32))
        part = x[:, s]
        fin = np.isfinite(part)
        top = np.where(fin, np.abs(part), 0.0).max(1)
        ex = np.frexp(top)[1] - 1            # floor(log2), 0 for 0 handled below
        b = np.where(top >= 2.0 ** -126, ex + 127, 0)
        b = b + (np.rint(top * 2.0 ** (133.0 - b)) > 127)
        b = np.minimum(b, 254)
        scale = 2.0 ** (b[:, None] - 133.0)
        with np.errstate(invalid="ignore", over="ignore"):
            r = np.clip(np.rint(part / scale), -127, 127)
        qq = np.where(fin, np.nan_to_num(r), -128)
        q[:, s], e[:, g] = qq, b
        val[:, s] = np.where(fin, qq * scale, np.nan)
    return q, e, val


def norm(x, gamma, beta, eps, center):
    """(y, mean, rstd, xh) in float64 (numpy)."""
    mu = x.mean(1) if center else np.zeros(x.shape[0])
    r = 1.0 / np.sqrt(((x - mu[:, None]) ** 2).mean(1) + eps)
    xh = (x - mu[:, None]) * r[:, None]
    y = xh * (1.0 if gamma is None else gamma) + (0.0 if beta is None else beta)
    return y, mu, r, xh


def norm_grads(dy, xh, r, gamma, center):
    a = dy if gamma is None else dy * gamma
    dx = a - xh * (a * xh).mean(1, keepdims=True)
    if center:
        dx = dx - a.mean(1, keepdims=True)
    return dx * r[:, None], (dy * xh).sum(0), dy.sum(0)


def sample(z, u, temperature, top_k, top_p, min_p):
    """(ids, logp) of one row: z float64 [V], u float64 [N]."""
    N = len(u)
    ids, logp = np.full(N, -1, np.int64), np.full(N, np.nan)
    if np.isnan(z).any() or np.isposinf(z).any() or not np.isfinite(z).any():
        return ids, logp
    ok = temperature >= 0 and np.isfinite(temperature) and top_p > 0 and 0 <= min_p <= 1
    if not ok:
        return ids, logp
    order = np.argsort(-z, kind="stable")
    order = order[np.isfinite(z[order])]
    zs = z[order]
    if temperature == 0:
        w = np.ones(1)
    else:
        with np.errstate(over="ignore"):
            w = np.exp((zs - zs[0]) / temperature)
        L = len(w)
        if 0 < top_k < L:
            L = top_k
        cum = np.cumsum(w[:L])
        keep = L
        if top_p < 1:
            keep = min(keep, int((cum < top_p * cum[-1]).sum()) + 1)
        if min_p > 0:
            keep = min(keep, max(1, int((w >= min_p).sum())))
        w = w[:keep]
    cum = np.cumsum(w)
    for n in range(N):
        if not 0 <= u[n] < 1:
            continue
        k = min(int(np.searchsorted(cum, u[n] * cum[-1], side="right")), len(w) - 1)
        ids[n] = order[k]
        logp[n] = np.log(w[k] / cum[-1])
    return ids, logp

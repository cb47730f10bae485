"""The operators around the loss (``include/ckl_ops.h``): the norm that makes
the hidden states, 8-bit activations, sampling.  Imported by the package, which
offers every name of ``__all__`` as its own."""

from __future__ import annotations

import ctypes
import functools

import torch
from torch.autograd.function import once_differentiable

from . import CKL_OK, LIB_PATH, CklError, backward, forward, lib

__all__ = [
    "ACT8_GROUP", "SAMPLE_BAD_INPUT", "act8_pack", "act8_unpack", "norm_forward",
    "norm_backward", "norm_workspace_bytes", "layer_norm", "rms_norm", "norm_kl_loss", "sample",
]

ACT8_GROUP = 32
SAMPLE_BAD_INPUT = 16

_DTYPES = {torch.bfloat16: 0, torch.float32: 1}
_INT32_MAX = 2 ** 31 - 1


def _bind(L):
    if not hasattr(L, "ckl_sample"):
        raise ImportError(f"{LIB_PATH} lacks ckl_sample: it is older than its sources; rebuild "
                          "with `python -c 'import __graft_entry__ as g; g.build()'`")
    vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
    f32, f64 = ctypes.c_float, ctypes.c_double
    for name, args in (
            ("ckl_act8_pack", [vp, i32, i64, i64, vp, vp, vp]),
            ("ckl_act8_unpack", [vp, vp, i64, i64, i32, vp, vp]),
            ("ckl_norm_forward", [vp, i32, vp, vp, i32, i64, i64, f32, vp, vp, vp, vp, vp, vp]),
            ("ckl_norm_backward", [vp, i32, vp, vp, vp, vp, vp, vp, i32, i64, i64, vp, vp, vp,
                                   i32, vp, sz, vp]),
            ("ckl_sample", [vp, i64, i64, i64, vp, i32, f64, i32, f64, f64, vp, vp, vp, vp, vp,
                            vp, vp, vp])):
        f = getattr(L, name)
        f.argtypes = args
        f.restype = ctypes.c_int
    L.ckl_norm_workspace_bytes.argtypes = [i64, i64]
    L.ckl_norm_workspace_bytes.restype = sz


_bind(lib)


# The raw handle of a device's current stream: building a torch.cuda.Stream
# for it takes longer than launching a small kernel.
_raw_stream = torch._C._cuda_getCurrentRawStream


def _on(t, stream, call):
    """call(stream handle) with t's device current and, when one is given,
    ``stream`` current too, so that what the call allocates belongs to it."""
    dev = t.get_device()
    if stream is None and dev == torch.cuda.current_device():
        return call(_raw_stream(dev))
    if stream is not None and stream.device != t.device:
        raise ValueError(f"the stream is on {stream.device}, the tensors are on {t.device}")
    with torch.cuda.device(dev):
        if stream is None:
            return call(_raw_stream(dev))
        with torch.cuda.stream(stream):
            return call(stream.cuda_stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _check(name, t, dtypes, shape=None, like=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {tuple(dtypes)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if like is not None and t.get_device() != like.get_device():
        raise ValueError(f"{name} is on {t.device}, expected {like.device}")


def _rows(name, t):
    """(T, d) of a tensor taken as rows of its last dimension."""
    if t.dim() < 1 or t.shape[-1] == 0:
        raise ValueError(f"{name} must have a last dimension of at least 1")
    d = t.shape[-1]
    return t.numel() // d, d


def _kept_shapes(shape):
    return tuple(shape), tuple(shape[:-1]) + (-(-shape[-1] // ACT8_GROUP),)


# ---------------------------------------------------------- 8-bit activations
def act8_pack(x, stream=None):
    """x [..., d] (bf16 or fp32) in 8 bits: (q int8 [..., d], exponents uint8
    [..., ceil(d / 32)]), each group of 32 elements with its own power-of-two
    scale (ckl_act8_pack)."""
    _check("x", x, _DTYPES)
    T, d = _rows("x", x)
    qs, es = _kept_shapes(x.shape)

    def call(st):
        q = x.new_empty(qs, dtype=torch.int8)
        e = x.new_empty(es, dtype=torch.uint8)
        rc = lib.ckl_act8_pack(_ptr(x), _DTYPES[x.dtype], T, d, _ptr(q), _ptr(e), st)
        if rc != CKL_OK:
            raise CklError(rc, "ckl_act8_pack")
        return q, e

    return _on(x, stream, call)


def _check_kept(q, exponents):
    _check("q", q, (torch.int8,))
    T, d = _rows("q", q)
    _check("exponents", exponents, (torch.uint8,), _kept_shapes(q.shape)[1], like=q)
    return T, d


def act8_unpack(q, exponents, dtype=torch.bfloat16, stream=None):
    """The values of ``act8_pack``'s result, as bf16 or fp32 (exact in both)."""
    T, d = _check_kept(q, exponents)
    if dtype not in _DTYPES:
        raise TypeError(f"dtype must be one of {tuple(_DTYPES)}")

    def call(st):
        x = torch.empty_like(q, dtype=dtype)
        rc = lib.ckl_act8_unpack(_ptr(q), _ptr(exponents), T, d, _DTYPES[dtype], _ptr(x), st)
        if rc != CKL_OK:
            raise CklError(rc, "ckl_act8_unpack")
        return x

    return _on(q, stream, call)


# ----------------------------------------------------------------------- norm
def _param_dtype(gamma, beta, d, x):
    dt = None
    for name, t in (("gamma", gamma), ("beta", beta)):
        if t is not None:
            _check(name, t, _DTYPES, (d,), like=x)
            if dt is not None and t.dtype != dt:
                raise TypeError("gamma and beta must have one dtype")
            dt = t.dtype
    return 0 if dt is None else _DTYPES[dt]


def norm_forward(x, gamma=None, beta=None, eps: float = 1e-5, center: bool = True,
                 checkpoint: bool = False, stream=None, out=None):
    """Layer norm (``center``) or RMS norm of x [..., d], bf16 or fp32.

    Returns (y, mean, rstd, kept) for ``norm_backward``: mean (None without
    centring) and rstd are fp32 [...]; ``kept`` is x in 8 bits, (q, exponents)
    as ``act8_pack`` makes them, with ``checkpoint``, else None.  A caller that
    hands ``kept`` to the backward need not keep x.
    """
    _check("x", x, _DTYPES)
    T, d = _rows("x", x)
    pd = _param_dtype(gamma, beta, d, x)
    if out is not None:
        _check("out", out, (x.dtype,), x.shape, like=x)

    def call(st):
        y = out if out is not None else torch.empty_like(x)
        rstd = x.new_empty(x.shape[:-1], dtype=torch.float32)
        mean = torch.empty_like(rstd) if center else None
        q = e = kept = None
        if checkpoint:
            qs, es = _kept_shapes(x.shape)
            q = x.new_empty(qs, dtype=torch.int8)
            e = x.new_empty(es, dtype=torch.uint8)
            kept = (q, e)
        rc = lib.ckl_norm_forward(_ptr(x), _DTYPES[x.dtype], _ptr(gamma), _ptr(beta), pd, T, d,
                                  eps, _ptr(y), _ptr(mean), _ptr(rstd), _ptr(q), _ptr(e), st)
        if rc != CKL_OK:
            raise CklError(rc, "ckl_norm_forward")
        return y, mean, rstd, kept

    return _on(x, stream, call)


@functools.lru_cache(maxsize=1024)
def norm_workspace_bytes(T: int, d: int) -> int:
    n = lib.ckl_norm_workspace_bytes(T, d)
    if n == 0:
        raise CklError(1, "ckl_norm_workspace_bytes")
    return int(n)


def norm_backward(dy, x, mean, rstd, gamma=None, bias: bool = False, dgamma=None, dbeta=None,
                  accumulate: bool = False, workspace=None, stream=None, out_dx=None,
                  weight: bool = True):
    """(dx, dgamma, dbeta) of ``norm_forward``, from its mean and rstd.

    ``x`` is the forward's input, or what it kept of it, (q, exponents).
    dgamma (None without gamma, or without ``weight``: a gamma that is not
    trained) and dbeta (with ``bias``, else None) are fp32 [d]; given ones are
    written, or added to with ``accumulate``.
    """
    _check("dy", dy, _DTYPES)
    T, d = _rows("dy", dy)
    q = e = None
    if isinstance(x, (tuple, list)):
        q, e = x
        _check("q", q, (torch.int8,), dy.shape, like=dy)
        _check("exponents", e, (torch.uint8,), _kept_shapes(q.shape)[1], like=dy)
        x = None
    else:
        _check("x", x, (dy.dtype,), dy.shape, like=dy)
    pd = _param_dtype(gamma, None, d, dy)
    _check("rstd", rstd, (torch.float32,), dy.shape[:-1], like=dy)
    if mean is not None:
        _check("mean", mean, (torch.float32,), dy.shape[:-1], like=dy)
    for name, t in (("dgamma", dgamma), ("dbeta", dbeta)):
        if t is not None:
            _check(name, t, (torch.float32,), (d,), like=dy)
    weight = weight and gamma is not None
    if dgamma is not None and not weight:
        raise ValueError("dgamma without gamma, or without weight")
    if dbeta is not None and not bias:
        raise ValueError("dbeta without bias")
    if accumulate and ((weight and dgamma is None) or (bias and dbeta is None)):
        raise ValueError("accumulate needs the gradients that are added to")
    if workspace is not None and (not workspace.is_cuda or workspace.device != dy.device
                                  or workspace.dtype != torch.uint8
                                  or not workspace.is_contiguous()):
        raise ValueError("workspace must be a contiguous uint8 tensor on dy's device")
    if out_dx is not None:
        _check("out_dx", out_dx, (dy.dtype,), dy.shape, like=dy)

    def call(st):
        dx = out_dx if out_dx is not None else torch.empty_like(dy)
        dg = dgamma
        if dg is None and weight:
            dg = rstd.new_empty(d)
        db = dbeta
        if db is None and bias:
            db = rstd.new_empty(d)
        ws, n = workspace, 0
        if dg is not None or db is not None:
            if ws is None:
                ws = dy.new_empty(norm_workspace_bytes(T, d), dtype=torch.uint8)
            n = ws.numel()
        rc = lib.ckl_norm_backward(_ptr(dy), _DTYPES[dy.dtype], _ptr(x), _ptr(q), _ptr(e),
                                   _ptr(mean), _ptr(rstd), _ptr(gamma), pd, T, d, _ptr(dx),
                                   _ptr(dg), _ptr(db), int(bool(accumulate)), _ptr(ws), n, st)
        if rc != CKL_OK:
            raise CklError(rc, "ckl_norm_backward")
        return dx, dg, db

    return _on(dy, stream, call)


class _Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gamma, beta, eps, center, checkpoint):
        y, mean, rstd, kept = norm_forward(x, gamma, beta, eps, center, checkpoint)
        ctx.kept8 = kept is not None
        ctx.bias = None if beta is None else beta.dtype
        ctx.save_for_backward(*(kept if kept is not None else (x,)), mean, rstd, gamma)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        *x, mean, rstd, gamma = ctx.saved_tensors
        x = tuple(x) if ctx.kept8 else x[0]
        bias = ctx.bias is not None and ctx.needs_input_grad[2]
        dx, dg, db = norm_backward(dy.contiguous(), x, mean, rstd, gamma, bias=bias,
                                   weight=ctx.needs_input_grad[1])
        return (dx, None if dg is None else dg.to(gamma.dtype),
                db.to(ctx.bias) if bias else None, None, None, None)


def layer_norm(x, gamma=None, beta=None, eps: float = 1e-5, checkpoint: bool = False):
    """Differentiable layer norm over the last dimension.  With ``checkpoint``
    the backward pass reads x from 8 bits, and x itself is not kept.

    To capture both passes into a CUDA graph, take the gradients by
    ``torch.autograd.grad``, of leaves that no other live autograd graph holds.
    """
    return _Norm.apply(x, gamma, beta, eps, True, checkpoint)


def rms_norm(x, gamma=None, eps: float = 1e-6, checkpoint: bool = False):
    """Differentiable RMS norm over the last dimension (see ``layer_norm``)."""
    return _Norm.apply(x, gamma, None, eps, False, checkpoint)


class _NormKL(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gamma, beta, W, idx, logp, mask, eps, center, chunk):
        H, mean, rstd, _ = norm_forward(x, gamma, beta, eps, center)
        loss, lse = forward(H, W, idx, logp, mask, chunk)
        ctx.save_for_backward(x, gamma, beta, W, idx, logp, mask, mean, rstd, lse)
        ctx.eps, ctx.center, ctx.chunk = eps, center, chunk
        return loss.reshape(())

    @staticmethod
    @once_differentiable
    def backward(ctx, g):
        x, gamma, beta, W, idx, logp, mask, mean, rstd, lse = ctx.saved_tensors
        # the same call on the same x: the forward's H, bit for bit
        H = norm_forward(x, gamma, beta, ctx.eps, ctx.center)[0]
        gl = g.reshape(1).to(torch.float32).contiguous()
        dH, dW = backward(H, W, idx, logp, mask, lse, grad_loss=gl, chunk=ctx.chunk)
        del H
        dx = dg = db = None
        bias = beta is not None and ctx.needs_input_grad[2]
        if any(ctx.needs_input_grad[:3]):
            dx, dg, db = norm_backward(dH, x, mean, rstd, gamma, bias=bias, out_dx=dH,
                                       weight=ctx.needs_input_grad[1])
        return (dx, None if dg is None else dg.to(gamma.dtype), db.to(beta.dtype) if bias else None,
                dW.to(W.dtype) if ctx.needs_input_grad[3] else None, None, None, None, None, None,
                None)


def norm_kl_loss(x, gamma, beta, W, idx, logp, mask=None, eps: float = 1e-5, center: bool = True,
                 chunk: int = 1024):
    """``chunked_kl_loss`` of H = norm(x), x and W in bf16, differentiable in x,
    gamma, beta and W.  Between the passes it keeps x alone: the backward makes H
    again, as it makes the logits again, so T x d hidden states are not held
    twice.  (``layer_norm`` says what a capture of both passes needs.)"""
    _check("x", x, (torch.bfloat16,))
    for name, t in (("W", W), ("topk_idx", idx), ("topk_logp", logp), ("mask", mask)):
        if t is not None and t.get_device() != x.get_device():
            raise ValueError(f"{name} is on {t.device}, expected {x.device}")
    with torch.cuda.device(x.get_device()):
        return _NormKL.apply(x, gamma, beta, W, idx, logp, mask, eps, center, chunk)


# ------------------------------------------------------------------- sampling
def sample(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, stream=None, status=None):
    """Token ids drawn from rows of logits [T, V] (bf16, or its bits as int16 /
    uint16; rows may be further apart than V) by uniform numbers u, fp32 [T] or
    [T, N] in [0, 1): (ids int32, log-probs fp32), both of u's shape.

    ``temperature`` (0: the most likely token), ``top_k`` (0: off), ``top_p``
    and ``min_p`` are numbers or per-row CUDA tensors [T] (fp32; top_k int32);
    ckl_sample in ``include/ckl_ops.h`` defines their order.  The log-prob is
    the token's under the distribution drawn from.  A row with a NaN or +inf
    logit or a parameter out of range, a draw whose number is, and a row
    without a finite logit give id -1 and log-prob NaN; the first two also set
    SAMPLE_BAD_INPUT in ``status`` (an int32 [1] tensor that the caller
    cleared), when given.  Rows with logits of 256 and more, or other than 0
    below 2^-40 in magnitude, are far slower (``include/ckl_ops.h``).

    N draws a row are a teacher cache: ``forward(H, W, ids, zeros, ...)``.
    """
    if not logits.is_cuda or logits.dim() != 2:
        raise ValueError("logits must be a 2-D CUDA tensor")
    if logits.dtype not in (torch.bfloat16, torch.int16, torch.uint16):
        raise TypeError("logits must be bf16 (or its bits as int16/uint16)")
    T, V = logits.shape
    if V > 1 and logits.stride(1) != 1:
        raise ValueError("a row of logits must be contiguous")
    ld = logits.stride(0) if T > 1 else V
    if ld < V:
        raise ValueError("rows of logits must not overlap")
    _check("u", u, (torch.float32,), like=logits)
    if u.dim() not in (1, 2) or u.shape[0] != T:
        raise ValueError("u must have shape [T] or [T, N]")
    N = 1 if u.dim() == 1 else u.shape[1]
    if T * N > _INT32_MAX:
        raise ValueError("u must have fewer than 2^31 numbers")
    if isinstance(top_k, int):  # more than a row has is all of it
        top_k = max(0, min(top_k, _INT32_MAX))
    numbers, rows = [], []
    for name, v, dt, off in (("temperature", temperature, torch.float32, 1.0),
                             ("top_k", top_k, torch.int32, 0),
                             ("top_p", top_p, torch.float32, 1.0),
                             ("min_p", min_p, torch.float32, 0.0)):
        if isinstance(v, torch.Tensor):
            _check(name, v, (dt,), (T,), like=logits)
            numbers.append(off)
            rows.append(_ptr(v))
        else:
            numbers.append(v)
            rows.append(None)
    if status is not None:
        _check("status", status, (torch.int32,), (1,), like=logits)

    def call(st):
        ids = torch.empty_like(u, dtype=torch.int32)
        logp = torch.empty_like(u)
        rc = lib.ckl_sample(_ptr(logits), ld, T, V, _ptr(u), N, *numbers, *rows, _ptr(ids),
                            _ptr(logp), _ptr(status), st)
        if rc != CKL_OK:
            raise CklError(rc, "ckl_sample")
        return ids, logp

    return _on(logits, stream, call)

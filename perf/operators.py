"""Measured cases of the operators around the loss: the norm that makes its hidden
states (forward, backward, and a step whose backward reads 8-bit activations),
the 8-bit activation format itself, and sampling from logits.

``run`` computes an operator in its plain form (elementary torch operations)
or, with ``own`` set, through the library's public calls.
"""

import math

import torch

own = False

GROUP = 32  # elements of a row that share an 8-bit scale
EPS = 1e-5


# --------------------------------------------------------------------- cases
def _norm(name, op, T, d, dtype="bf16", center=True):
    return {"name": name, "op": op, "T": T, "d": d, "dtype": dtype, "center": center}


def _sample(name, T, V, N, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, rows=False,
            masked=False):
    return {"name": name, "op": "sample", "T": T, "V": V, "N": N, "temperature": temperature,
            "top_k": top_k, "top_p": top_p, "min_p": min_p, "rows": rows, "masked": masked}


def listed():
    return [
        # the head's input for a few tokens being generated: launch latency
        _norm("norm_fwd_tokens", "norm_fwd", 4, 2880, center=False),
        # one sequence of hidden states before the head
        _norm("norm_fwd_8k", "norm_fwd", 8192, 4096),
        # a small fp32 model with a row length no vector width divides
        _norm("norm_bwd_ragged_f32", "norm_bwd", 777, 1001, dtype="f32"),
        # the same sequence's backward, with the weight's and the bias' gradients
        _norm("norm_bwd_8k", "norm_bwd", 8192, 4096),
        # a short batch's step from 8-bit activations
        _norm("norm_ckpt_small", "norm_ckpt", 512, 2880, center=False),
        # a long context's step: the forward keeps x in 8 bits, the backward reads it
        _norm("norm_ckpt_32k", "norm_ckpt", 32768, 4096),
        # keeping and restoring any activation in 8 bits
        _norm("act8_32k", "act8", 32768, 2880),
        _norm("act8_ragged_f32", "act8", 1000, 1001, dtype="f32"),
        # one sequence being generated, the usual filters
        _sample("sample_one", 1, 128256, 1, temperature=0.7, top_k=50, top_p=0.95),
        # a serving batch, each row with its own parameters, some rows greedy
        _sample("sample_batch", 96, 201088, 1, rows=True),
        # guided generation: most of the vocabulary masked, odd vocabulary
        _sample("sample_guided", 333, 50257, 1, temperature=1.2, min_p=0.02, masked=True),
        # a sampled teacher cache: 64 draws a position from the whole distribution
        _sample("sample_cache", 4096, 128256, 64),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "norm_ckpt", "act8", "sample", "sample"])
    if op != "sample":
        d = _log_int(rng, 16, 16384)
        if rng.random() < 0.5:
            d = max(16, d // 8 * 8)
        T = min(_log_int(rng, 1, 32768), 32768 * 4096 // d)
        return {"op": op, "T": T, "d": d, "dtype": rng.choice(["bf16", "bf16", "f32"]),
                "center": rng.random() < 0.5}
    V = _log_int(rng, 1000, 201088)
    if rng.random() < 0.5:
        V = V // 8 * 8
    T = min(_log_int(rng, 1, 4096), 4096 * 128256 // V)
    case = {"op": op, "T": T, "V": V, "N": rng.choice([1, 1, 1, 2, 7, 32, 64]),
            "temperature": 1.0, "top_k": 0, "top_p": 1.0, "min_p": 0.0, "rows": False,
            "masked": rng.random() < 0.25}
    kind = rng.choice(["plain", "top_k", "top_p", "min_p", "all", "rows"])
    if kind != "plain":
        case["temperature"] = rng.choice([0.6, 0.8, 1.0, 1.3])
    if kind in ("top_k", "all"):
        case["top_k"] = _log_int(rng, 1, 1000)
    if kind in ("top_p", "all"):
        case["top_p"] = rng.choice([0.5, 0.8, 0.9, 0.95, 0.99])
    if kind in ("min_p", "all"):
        case["min_p"] = rng.choice([0.01, 0.05, 0.1])
    case["rows"] = kind == "rows"
    return case


# -------------------------------------------------------------------- inputs
def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def rand(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    s = dict(case)
    if case["op"] != "sample":
        T, d, dt = case["T"], case["d"], _dtype(case)
        # a residual stream: rows of different size, a few channels far larger
        chan = 1.0 + 20.0 * (rand(1, d) < 0.01)
        x = randn(T, d).mul_(chan).mul_(0.5 + 2.0 * rand(T, 1)).add_(0.3).to(dt)
        s["x"] = x
        if case["op"] == "act8":
            return s
        s["gamma"] = (1.0 + 0.1 * randn(d)).to(dt)
        s["beta"] = (0.1 * randn(d)).to(dt) if case["center"] else None
        if case["op"] != "norm_fwd":
            s["dy"] = randn(T, d).to(dt)
        if case["op"] == "norm_bwd":
            xd = x.double()
            mean = xd.mean(1, keepdim=True) if case["center"] else torch.zeros_like(xd[:, :1])
            var = (xd - mean).square_().mean(1)
            s["mean"] = mean[:, 0].float() if case["center"] else None
            s["rstd"] = (var + EPS).rsqrt_().float()
        return s
    T, V, N = case["T"], case["V"], case["N"]
    # logits of a language model: a broad body and a few likely tokens a row
    z = randn(T, V).mul_(2.0)
    at = torch.randint(0, V, (T, 48), generator=g, device="cuda")
    z.scatter_add_(1, at, 3.0 + 2.5 * rand(T, 48) - 1.5 * torch.log(rand(T, 48).clamp_min_(1e-6)))
    if case["masked"]:
        z.masked_fill_(rand(T, V) < 0.9, float("-inf"))
        z[:, V // 2] = 1.0
    s["logits"] = z.to(torch.bfloat16)
    s["u"] = rand(T) if N == 1 else rand(T, N)
    if case["rows"]:
        pick = torch.randint(0, 4, (T,), generator=g, device="cuda")
        s["temperature"] = torch.tensor([0.0, 0.7, 1.0, 1.3], device="cuda")[pick]
        pick = torch.randint(0, 4, (T,), generator=g, device="cuda")
        s["top_k"] = torch.tensor([0, 1, 40, 500], dtype=torch.int32, device="cuda")[pick]
        pick = torch.randint(0, 3, (T,), generator=g, device="cuda")
        s["top_p"] = torch.tensor([1.0, 0.9, 0.95], device="cuda")[pick]
        pick = torch.randint(0, 3, (T,), generator=g, device="cuda")
        s["min_p"] = torch.tensor([0.0, 0.0, 0.05], device="cuda")[pick]
    return s


# -------------------------------------------------------------- plain forms
def _pow2(k):
    """2^k as float32, for int32 k of normal numbers."""
    return ((k + 127) << 23).to(torch.int32).view(torch.float32)


def _groups(x):
    """x as float32 [T, groups, GROUP], the last group filled up with zeros."""
    T, d = x.shape
    pad = -d % GROUP
    xf = x.float()
    if pad:
        xf = torch.cat([xf, torch.zeros(T, pad, device=x.device)], 1)
    return xf.view(T, -1, GROUP)


def _act8(x):
    """The values that x has in 8 bits (float32): per group an integer of
    -127..127 times a power of two, the smallest one that holds the largest."""
    xg = _groups(x)
    a = xg.abs().amax(2, keepdim=True)
    E = torch.frexp(a)[1] - 1
    E = torch.where(a > 0, E, torch.zeros_like(E))
    E = E + (torch.round(a * _pow2(6 - E)) > 127).to(torch.int32)
    q = torch.round(xg * _pow2(6 - E))
    return (q * _pow2(E - 6)).view(x.shape[0], -1)[:, :x.shape[1]]


def _plain_forward(x, gamma, beta, center):
    xf = x.float()
    mean = xf.mean(1, keepdim=True) if center else None
    xc = xf - mean if center else xf
    rstd = torch.rsqrt(xc.square().mean(1, keepdim=True) + EPS)
    y = xc * rstd * gamma.float()
    if beta is not None:
        y = y + beta.float()
    return y.to(x.dtype), None if mean is None else mean[:, 0], rstd[:, 0]


def _plain_backward(dy, x, mean, rstd, gamma, center):
    g = dy.float()
    xf = x.float()
    xh = (xf - mean[:, None] if center else xf) * rstd[:, None]
    a = g * gamma.float()
    dx = a - xh * (a * xh).mean(1, keepdim=True)
    if center:
        dx = dx - a.mean(1, keepdim=True)
    dx = dx * rstd[:, None]
    dgamma = (g * xh).sum(0)
    dbeta = g.sum(0) if center else None
    return dx.to(dy.dtype), dgamma, dbeta


def _column(v, like):
    """A parameter as a float64 column: one number or one a row."""
    if isinstance(v, torch.Tensor):
        return v.double()[:, None]
    return torch.full((like.shape[0], 1), float(v), dtype=torch.float64, device=like.device)


def _plain_sample(logits, u, temperature, top_k, top_p, min_p):
    T, V = logits.shape
    z, order = torch.sort(logits.float(), dim=1, descending=True, stable=True)
    temp = _column(temperature, logits)
    greedy = temp == 0
    # 64 bits: a draw next to the border of two tokens must fall on the right one
    w = torch.exp((z.double() - z[:, :1].double()) / torch.where(greedy, 1.0, temp))
    cum = torch.cumsum(w, 1)
    k = _column(top_k, logits).long()
    k = torch.where(k <= 0, V, k.clamp(max=V))
    p = _column(top_p, logits)
    mp = _column(min_p, logits)
    kept = k
    mass = p * torch.gather(cum, 1, k - 1)
    kept_p = (cum < mass).sum(1, keepdim=True) + 1
    kept = torch.where(p < 1, torch.minimum(kept, kept_p), kept)
    kept = torch.minimum(kept, (w >= mp).sum(1, keepdim=True))
    kept = torch.where(greedy, 1, kept)
    total = torch.gather(cum, 1, kept - 1)
    uu = u.double().view(T, -1)
    pos = torch.searchsorted(cum, uu * total, right=True)
    pos = torch.minimum(pos, kept - 1)
    ids = torch.gather(order, 1, pos).to(torch.int32)
    logp = torch.log(torch.gather(w, 1, pos) / total).float()
    return ids.view(u.shape), logp.view(u.shape)


# ----------------------------------------------------------------------- run
def run(s):
    if own:
        return _run_own(s)
    op = s["op"]
    if op == "norm_fwd":
        y, mean, rstd = _plain_forward(s["x"], s["gamma"], s["beta"], s["center"])
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "norm_bwd":
        dx, dg, db = _plain_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["gamma"],
                                     s["center"])
        return {"dx": dx, "dgamma": dg, "dbeta": db}
    if op == "norm_ckpt":
        y, mean, rstd = _plain_forward(s["x"], s["gamma"], s["beta"], s["center"])
        dx, dg, db = _plain_backward(s["dy"], _act8(s["x"]), mean, rstd, s["gamma"], s["center"])
        return {"y": y, "dx": dx, "dgamma": dg, "dbeta": db}
    if op == "act8":
        return {"x": _act8(s["x"]).to(s["x"].dtype)}
    ids, logp = _plain_sample(s["logits"], s["u"], s["temperature"], s["top_k"], s["top_p"],
                              s["min_p"])
    return {"ids": ids, "logp": logp}


def _run_own(s):
    import chunked_kl_loss_ckl_b200 as ckl

    op = s["op"]
    if op == "norm_fwd":
        y, mean, rstd, _ = ckl.norm_forward(s["x"], s["gamma"], s["beta"], eps=EPS,
                                            center=s["center"])
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "norm_bwd":
        dx, dg, db = ckl.norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["gamma"],
                                       bias=s["center"])
        return {"dx": dx, "dgamma": dg, "dbeta": db}
    if op == "norm_ckpt":
        y, mean, rstd, kept = ckl.norm_forward(s["x"], s["gamma"], s["beta"], eps=EPS,
                                               center=s["center"], checkpoint=True)
        dx, dg, db = ckl.norm_backward(s["dy"], kept, mean, rstd, s["gamma"], bias=s["center"])
        return {"y": y, "dx": dx, "dgamma": dg, "dbeta": db}
    if op == "act8":
        q, e = ckl.act8_pack(s["x"])
        return {"x": ckl.act8_unpack(q, e, dtype=s["x"].dtype)}
    ids, logp = ckl.sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"],
                           top_p=s["top_p"], min_p=s["min_p"])
    return {"ids": ids, "logp": logp}


# ---------------------------------------------------------------------- work
def work(case):
    if case["op"] == "sample":
        T, V, N = case["T"], case["V"], case["N"]
        # the logits once, a number and (id, log-prob) a draw; per logit its
        # difference, its exponential and its place in the sum
        return {"bytes": 2 * T * V + 12 * T * N + (16 * T if case["rows"] else 0),
                "flops": 3 * T * V}
    T, d = case["T"], case["d"]
    n, b = T * d, 4 if case["dtype"] == "f32" else 2
    kept = n + T * -(-d // GROUP)             # 8-bit values and their scales
    stats = 4 * T * (2 if case["center"] else 1)
    params = d * b * (2 if case["center"] else 1)
    grads = 4 * d * (2 if case["center"] else 1)
    if case["op"] == "norm_fwd":
        return {"bytes": 2 * n * b + stats + params, "flops": 7 * n}
    if case["op"] == "norm_bwd":
        return {"bytes": 3 * n * b + stats + d * b + grads, "flops": 12 * n}
    if case["op"] == "norm_ckpt":
        return {"bytes": 4 * n * b + 2 * kept + 2 * stats + params + d * b + grads,
                "flops": 23 * n}
    return {"bytes": 2 * n * b + 2 * kept, "flops": 4 * n}


# --------------------------------------------------------------------- exact
def _exact_act8(x):
    x = x.double()
    T, d = x.shape
    out = torch.empty_like(x)
    whole = d // GROUP * GROUP
    spans = [(0, whole, GROUP)] if whole else []
    if d > whole:
        spans.append((whole, d, d - whole))
    for b, e, width in spans:
        part = x[:, b:e].reshape(-1, width)
        top = part.abs().max(1, keepdim=True).values
        step = torch.exp2(torch.floor(torch.log2(top.clamp_min(1e-30))) - 6).float().double()
        step = torch.where(top / step >= 128, step * 2, step)   # log2 just below a power
        step = torch.where(torch.round(top / step) >= 128, step * 2, step)
        out[:, b:e] = (torch.round(part / step) * step).view(T, e - b)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "act8":
        return {"x": _exact_act8(s["x"])}
    if case["op"] == "sample":
        return _exact_sample(s)
    x = s["x"].double()
    gamma = s["gamma"].double()
    d = x.shape[1]
    if case["op"] == "norm_bwd":
        mean, rstd = s["mean"], s["rstd"].double()[:, None]
        mean = mean.double()[:, None] if mean is not None else 0.0
    else:
        mean = x.sum(1, keepdim=True) / d if case["center"] else 0.0
        rstd = 1.0 / torch.sqrt((x * x).sum(1, keepdim=True) / d - mean * mean + EPS)
    out = {}
    if case["op"] != "norm_bwd":
        y = (x - mean) * rstd * gamma
        if s["beta"] is not None:
            y += s["beta"].double()
        out["y"] = y
    if case["op"] == "norm_fwd":
        out["mean"] = mean[:, 0] if case["center"] else None
        out["rstd"] = rstd[:, 0]
        return out
    xh = (_exact_act8(s["x"]) if case["op"] == "norm_ckpt" else x).sub_(mean).mul_(rstd)
    dy = s["dy"].double()
    out["dgamma"] = torch.einsum("td,td->d", dy, xh)
    out["dbeta"] = dy.sum(0) if case["center"] else None
    # the Jacobian of the normalisation applied to dy * gamma
    a = dy.mul_(gamma)
    along = (a * xh).sum(1, keepdim=True) / d
    shift = a.sum(1, keepdim=True) / d if case["center"] else 0.0
    out["dx"] = rstd * (a - shift - along * xh)
    return out


def _exact_sample(s):
    z = s["logits"]
    T, V = z.shape
    u = s["u"].view(T, -1)
    ids = torch.empty(u.shape, dtype=torch.int32, device=z.device)
    logp = torch.empty(u.shape, dtype=torch.float64, device=z.device)

    def row_of(name, t0, t1):
        v = s[name]
        if isinstance(v, torch.Tensor):
            return v[t0:t1].double().view(-1, 1)
        return torch.full((t1 - t0, 1), v, dtype=torch.float64, device=z.device)

    index = torch.arange(V, device=z.device)
    for t0 in range(0, T, 512):
        t1 = min(T, t0 + 512)
        zz = z[t0:t1].double()
        # one whole number orders the tokens: the logit's place among all
        # bf16 values, then the lowest id
        bits = z[t0:t1].view(torch.int16).long()
        place = torch.where(bits < 0, -(bits & 0x7FFF), bits)
        first = (-place * (1 << 20) + index).sort(1).values % (1 << 20)
        zz = zz.gather(1, first)
        temp, k = row_of("temperature", t0, t1), row_of("top_k", t0, t1)
        p, mp = row_of("top_p", t0, t1), row_of("min_p", t0, t1)
        rank = index.double()[None] + 1
        w = torch.exp((zz - zz[:, :1]) / temp.clamp_min(1e-30))
        w = torch.where((k > 0) & (rank > k), 0.0, w)
        before = torch.cat([torch.zeros_like(w[:, :1]), w.cumsum(1)[:, :-1]], 1)
        out = (p < 1) & (before >= p * w.sum(1, keepdim=True))
        out |= torch.exp((zz - zz[:, :1]) / temp.clamp_min(1e-30)) < mp
        out |= (temp == 0) & (rank > 1)
        w = w.masked_fill(out, 0.0)
        upto = w.cumsum(1)
        total = upto[:, -1:]
        pos = torch.searchsorted(upto / total, u[t0:t1].double(), right=True)
        pos = torch.minimum(pos, (w > 0).sum(1, keepdim=True) - 1)
        ids[t0:t1] = first.gather(1, pos).to(torch.int32)
        logp[t0:t1] = torch.log(w.gather(1, pos) / total)
    return {"ids": ids.view(s["u"].shape), "logp": logp.view(s["u"].shape)}

"""Cases for the tensor-product operators: dense products with a fused
epilogue, products grouped by expert, and the orthogonalised update.

Three operators, each forward and (for the two products) backward:

  linear          y = act(x w^T + bias) + residual, optionally with the
                  pre-activation kept for the backward pass
  grouped_linear  the same product where row t of x meets the weight of its
                  own expert; rows are sorted by expert, offsets[e] is the
                  first row of expert e
  orthogonalize   Newton-Schulz iteration on a (batch of) gradient matrices:
                  x0 = g / |g|_F, then steps times
                  A = x x^T, x <- a x + (b A + c A A) x

``own`` selects the framework's kernels; otherwise everything is computed
with elementary torch operations in 32 bits and rounded once at the end.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
NS = (3.4445, -4.7750, 2.0315)     # a, b, c of the quintic iteration
NS_STEPS = 5
NS_EPS = 1e-7


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one new token through an output projection that adds to the residual
        # stream: the weight is read once, nothing else matters
        {"name": "linear one token", "op": "linear", "m": 1, "n": 4096, "k": 4096, "dtype": "bf16", "act": "none",
         "bias": False, "residual": True, "preact": False},
        # a small decoding batch through an up-projection
        {"name": "linear decode batch", "op": "linear", "m": 37, "n": 8192, "k": 2048, "dtype": "f16", "act": "gelu",
         "bias": True, "residual": False, "preact": False},
        # a short prompt against an output width that is no multiple of anything
        {"name": "linear prompt odd width", "op": "linear", "m": 1001, "n": 5003, "k": 2056, "dtype": "bf16",
         "act": "silu", "bias": True, "residual": True, "preact": False},
        # a training micro-batch through an up-projection, pre-activation kept
        {"name": "linear train forward", "op": "linear", "m": 8192, "n": 8192, "k": 4096, "dtype": "bf16",
         "act": "gelu", "bias": True, "residual": False, "preact": True},
        # its backward pass: gradients of input, weight and bias
        {"name": "linear train backward", "op": "linear_backward", "m": 4096, "n": 4096, "k": 4096, "dtype": "bf16",
         "act": "gelu", "bias": True},
        # the backward pass of a small layer on a ragged batch
        {"name": "linear backward ragged", "op": "linear_backward", "m": 777, "n": 1544, "k": 1032, "dtype": "f16",
         "act": "relu", "bias": True},
        # three tokens, eight experts each: few rows, most experts idle
        {"name": "experts decode", "op": "grouped", "t": 24, "e": 64, "n": 2048, "k": 1024, "dtype": "bf16",
         "act": "silu", "bias": False, "preact": False, "skew": 0.5},
        # a prefill's tokens over unevenly loaded experts, some of them empty
        {"name": "experts prefill ragged", "op": "grouped", "t": 8190, "e": 32, "n": 4096, "k": 2048, "dtype": "bf16",
         "act": "gelu", "bias": True, "preact": False, "skew": 0.7},
        # training backward over ragged experts
        {"name": "experts backward ragged", "op": "grouped_backward", "t": 8191, "e": 16, "n": 2048, "k": 2048,
         "dtype": "f16", "act": "silu", "bias": True, "skew": 0.7},
        # the update of one small projection (per-head or low-rank matrices)
        {"name": "orthogonalize small", "op": "ortho", "batch": 1, "p": 128, "q": 128, "dtype": "bf16"},
        # a tall f32 gradient as an F32 AllReduce leaves it, odd sizes
        {"name": "orthogonalize tall odd", "op": "ortho", "batch": 1, "p": 2737, "q": 1001, "dtype": "f32"},
        # the stacked gradients of several layers of one shape
        {"name": "orthogonalize batch", "op": "ortho", "batch": 4, "p": 2048, "q": 4096, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, int(round(v / step)) * step)


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_backward", "grouped", "grouped", "grouped_backward", "ortho",
                     "ortho"])
    dtype = rng.choice(["bf16", "f16"])
    act = rng.choice(["none", "relu", "gelu", "silu"])
    most = 8192 * 8192 * 4096          # multiply-adds of the largest listed product
    if op in ("linear", "linear_backward"):
        n = _log_int(rng, 256, 8192, 8) + rng.choice([0, 0, 0, 1, 3])
        k = _log_int(rng, 256, 8192, 8)
        m = _log_int(rng, 1, 8192)
        m = max(1, min(m, most // (2 * n * k)))
        c = {"op": op, "m": m, "n": n, "k": k, "dtype": dtype, "act": act, "bias": rng.random() < 0.5}
        if op == "linear":
            c |= {"residual": rng.random() < 0.5, "preact": rng.random() < 0.3}
        return c
    if op in ("grouped", "grouped_backward"):
        e = rng.choice([4, 8, 16, 32, 64])
        n, k = _log_int(rng, 256, 4096, 8), _log_int(rng, 256, 4096, 8)
        t = max(1, min(_log_int(rng, 8, 8192), most // (8 * n * k)))
        c = {"op": op, "t": t, "e": e, "n": n, "k": k, "dtype": dtype, "act": act, "bias": rng.random() < 0.5,
             "skew": rng.choice([0.0, 0.4, 0.8])}
        if op == "grouped":
            c["preact"] = rng.random() < 0.3
        return c
    p, q = _log_int(rng, 64, 4096), _log_int(rng, 64, 4096)
    batch = rng.choice([1, 1, 2, 4])
    while batch > 1 and batch * p * q > 4 * 2048 * 2048:
        batch //= 2
    if p * q * min(p, q) > 2048 * 4096 * 2048:
        p //= 2
    return {"op": "ortho", "batch": batch, "p": p, "q": q, "dtype": rng.choice(["bf16", "f32"])}


# ----------------------------------------------------------------- inputs
def _counts(t, e, skew, seed):
    """Rows of every expert: a multinomial draw over unequal loads; with a
    skew, every fifth expert gets nothing."""
    g = torch.Generator().manual_seed(seed * 7919 + 13)
    load = torch.exp(skew * 1.5 * torch.randn(e, generator=g))
    if skew > 0:
        load[4::5] = 0
    pick = torch.multinomial(load / load.sum(), t, replacement=True, generator=g)
    return torch.bincount(pick, minlength=e)


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def randn(*shape, scale=1.0, dtype=dt):
        t = torch.empty(shape, device=dev, dtype=dtype)
        return t.normal_(0.0, scale, generator=g)

    s = {"case": case}
    if case["op"] == "ortho":
        b, p, q = case["batch"], case["p"], case["q"]
        # a few strong directions over a broad floor, as gradients have
        r = min(8, p, q)
        u, v = randn(b, p, r, dtype=torch.float32), randn(b, r, q, dtype=torch.float32)
        s["g"] = ((u @ v) * 0.5 + randn(b, p, q, dtype=torch.float32)).mul_(1e-3).to(dt)
        return s
    n, k = case["n"], case["k"]
    if case["op"] in ("linear", "linear_backward"):
        rows, lead = case["m"], ()
    else:
        rows, lead = case["t"], (case["e"],)
        counts = _counts(case["t"], case["e"], case["skew"], seed)
        offs = torch.zeros(case["e"] + 1, dtype=torch.int32)
        offs[1:] = torch.cumsum(counts, 0)
        s["offsets"] = offs.to(dev)
        s["ends"] = offs.tolist()      # a program that exchanged the rows knows the counts
    s["x"] = randn(rows, k)
    s["w"] = randn(*lead, n, k, scale=k ** -0.5)
    if case["op"].endswith("backward"):
        s["dy"] = randn(rows, n)
        s["z"] = randn(rows, n)        # pre-activations as the forward pass kept them
        return s
    s["bias"] = randn(*lead, n, scale=0.5) if case["bias"] else None
    s["residual"] = randn(rows, n) if case.get("residual") else None
    return s


# ----------------------------------------------------------- plain forms
def _act(z, act):
    if act == "relu":
        return torch.clamp(z, min=0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.tanh(0.7978845608028654 * (z + 0.044715 * z * z * z)))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    if act == "gelu":
        c = 0.7978845608028654
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _plain_linear(s):
    c = s["case"]
    z = s["x"].float() @ s["w"].float().t()
    if s["bias"] is not None:
        z = z + s["bias"].float()
    y = _act(z, c["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    dt = s["x"].dtype
    return {"y": y.to(dt), "z": z.to(dt)} if c["preact"] else {"y": y.to(dt)}


def _plain_linear_backward(s):
    c, dt = s["case"], s["x"].dtype
    dz = s["dy"].float()
    if c["act"] != "none":
        dz = dz * _act_grad(s["z"].float(), c["act"])
    out = {"dx": (dz @ s["w"].float()).to(dt), "dw": (dz.t() @ s["x"].float()).to(dt)}
    if c["bias"]:
        out["db"] = dz.sum(0).to(dt)
    return out


def _by_expert(s, a, b):
    """a[rows of e] @ b[e] for every expert, one row range after another."""
    ends = s["ends"]
    return torch.cat([a[i:j] @ b[e] for e, (i, j) in enumerate(zip(ends, ends[1:])) if j > i])


def _by_expert_padded(s, a, b):
    """The same as one batched product over ranges padded to the longest: fewer
    launches where the ranges are short."""
    ends = s["ends"]
    e, at = _rows_by_expert(s)
    p = torch.zeros((b.shape[0], max(j - i for i, j in zip(ends, ends[1:])), a.shape[1]), device=a.device)
    p[e, at] = a
    return torch.bmm(p, b)[e, at]


def _rows_by_expert(s):
    """Expert of every row and the row's place within it."""
    t = torch.arange(s["x"].shape[0], device=s["x"].device)
    e = torch.searchsorted(s["offsets"][1:], t.int(), right=True)
    return e, t - s["offsets"][e]


def _products(s, a, b):
    few = a.shape[0] < 16 * b.shape[0]
    return _by_expert_padded(s, a, b) if few else _by_expert(s, a, b)


def _plain_grouped(s):
    c, dt = s["case"], s["x"].dtype
    z = _products(s, s["x"].float(), s["w"].float().transpose(1, 2))
    if s["bias"] is not None:
        z = z + s["bias"].float()[_rows_by_expert(s)[0]]
    y = _act(z, c["act"]).to(dt)
    return {"y": y, "z": z.to(dt)} if c["preact"] else {"y": y}


def _plain_grouped_backward(s):
    c, dt = s["case"], s["x"].dtype
    dz, x, ends = s["dy"].float(), s["x"].float(), s["ends"]
    if c["act"] != "none":
        dz = dz * _act_grad(s["z"].float(), c["act"])
    out = {"dx": _products(s, dz, s["w"].float()).to(dt),
           "dw": torch.stack([dz[i:j].t() @ x[i:j] for i, j in zip(ends, ends[1:])]).to(dt)}
    if c["bias"]:
        out["db"] = torch.stack([dz[i:j].sum(0) for i, j in zip(ends, ends[1:])]).to(dt)
    return out


def _plain_ortho(s):
    g = s["g"].float()
    tall = g.shape[1] > g.shape[2]
    x = g.transpose(1, 2) if tall else g
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + NS_EPS)
    a, b, c = NS
    for _ in range(NS_STEPS):
        m = torch.bmm(x, x.transpose(1, 2))
        x = a * x + torch.bmm(b * m + c * torch.bmm(m, m), x)
    return (x.transpose(1, 2) if tall else x).to(torch.bfloat16)


# ------------------------------------------------------------------- run
def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        if op == "linear":
            return _plain_linear(s)
        if op == "linear_backward":
            return _plain_linear_backward(s)
        if op == "grouped":
            return _plain_grouped(s)
        if op == "grouped_backward":
            return _plain_grouped_backward(s)
        return _plain_ortho(s)
    import collective_communication_schedule_gb300 as ccl
    if op == "ortho":
        return ccl.orthogonalize(s["g"], steps=NS_STEPS, coeffs=NS, eps=NS_EPS)
    act = {"none": ccl.ACT_NONE, "relu": ccl.ACT_RELU, "gelu": ccl.ACT_GELU, "silu": ccl.ACT_SILU}[c["act"]]
    if op.endswith("backward"):
        z = s["z"] if act != ccl.ACT_NONE else None
        if op == "linear_backward":
            dx, dw, db = ccl.linear_backward(s["dy"], s["x"], s["w"], preact=z, act=act, bias=c["bias"])
        else:
            dx, dw, db = ccl.grouped_linear_backward(s["dy"], s["x"], s["w"], s["offsets"], preact=z, act=act,
                                                     bias=c["bias"])
        return {"dx": dx, "dw": dw, "db": db} if c["bias"] else {"dx": dx, "dw": dw}
    if op == "linear":
        r = ccl.linear(s["x"], s["w"], bias=s["bias"], residual=s["residual"], act=act, preact=c["preact"])
    else:
        r = ccl.grouped_linear(s["x"], s["w"], s["offsets"], bias=s["bias"], act=act, preact=c["preact"])
    return {"y": r[0], "z": r[1]} if c["preact"] else {"y": r}


# ------------------------------------------------------------------ work
def work(case):
    if case["op"] == "ortho":
        b, p, q = case["batch"], min(case["p"], case["q"]), max(case["p"], case["q"])
        es = 4 if case["dtype"] == "f32" else 2
        # x x^T and A A are symmetric: half of each is enough
        return {"bytes": b * p * q * (es + 2), "flops": NS_STEPS * b * (p * p * q + p * p * p + 2 * p * p * q)}
    n, k = case["n"], case["k"]
    if case["op"] in ("linear", "linear_backward"):
        rows, mats = case["m"], 1
    else:
        rows, mats = case["t"], min(case["e"], case["t"])
    if case["op"].endswith("backward"):
        mats_out = 1 if case["op"] == "linear_backward" else case["e"]
        read = rows * (n * (2 if case["act"] != "none" else 1) + k) + mats * n * k
        wrote = rows * k + mats_out * n * k + (mats_out * n if case["bias"] else 0)
        return {"bytes": 2 * (read + wrote), "flops": 4 * rows * n * k}
    read = rows * k + mats * n * k + (mats * n if case["bias"] else 0) + (rows * n if case.get("residual") else 0)
    wrote = rows * n * (2 if case["preact"] else 1)
    return {"bytes": 2 * (read + wrote), "flops": 2 * rows * n * k}


# ----------------------------------------------------------------- exact
def _gelu64(z):
    u = math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
    return z * torch.sigmoid(2 * u)


def _gelu64_grad(z):
    r = math.sqrt(2 / math.pi)
    p = torch.sigmoid(2 * r * (z + 0.044715 * z ** 3))
    return p + z * p * (1 - p) * 2 * r * (1 + 0.134145 * z ** 2)


_ACT64 = {"none": lambda z: z, "relu": lambda z: z.relu(), "silu": lambda z: z * z.sigmoid(), "gelu": _gelu64}
_GRAD64 = {"none": torch.ones_like, "relu": lambda z: torch.heaviside(z, torch.zeros_like(z)),
           "silu": lambda z: z.sigmoid() * (1 + z * (-z).sigmoid()), "gelu": _gelu64_grad}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "ortho":
        a, b, c = NS
        outs = []
        for g in s["g"].double():
            x = g / (torch.linalg.norm(g) + NS_EPS)
            for _ in range(NS_STEPS):
                if x.shape[0] <= x.shape[1]:
                    m = x @ x.T
                    x = a * x + b * (m @ x) + c * (m @ (m @ x))
                else:
                    m = x.T @ x
                    x = a * x + b * (x @ m) + c * ((x @ m) @ m)
            outs.append(x)
        return torch.stack(outs)
    x, w = s["x"].double(), s["w"].double()
    if case["op"] in ("linear", "linear_backward"):
        ends, w = [0, x.shape[0]], w[None]
    else:
        ends = s["ends"]
    spans = list(zip(range(len(w)), ends[:-1], ends[1:]))
    if case["op"].endswith("backward"):
        dz = s["dy"].double() * _GRAD64[case["act"]](s["z"].double())
        out = {"dx": torch.cat([dz[i:j] @ w[e] for e, i, j in spans]),
               "dw": torch.stack([dz[i:j].T @ x[i:j] for e, i, j in spans])}
        if case["bias"]:
            out["db"] = torch.stack([dz[i:j].sum(0) for e, i, j in spans])
        if case["op"] == "linear_backward":
            out = {n: v if n == "dx" else v[0] for n, v in out.items()}
        return out
    bias = s["bias"].double().reshape(len(w), 1, -1) if case["bias"] else torch.zeros(len(w), 1, 1, device=x.device)
    z = torch.cat([x[i:j] @ w[e].T + bias[e] for e, i, j in spans])
    y = _ACT64[case["act"]](z)
    if case.get("residual"):
        y = y + s["residual"].double()
    return {"y": y, "z": z} if case["preact"] else {"y": y}

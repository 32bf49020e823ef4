"""Cases for the operators between and around the tensor products of a layer of
experts: the router, the rows' way to their experts and back, the norm in front
and the loss behind.

  route       scores of every token for every expert, the k best experts (with
              a bias for balance and groups of experts), their weights, and the
              places that sort the rows by expert; and its gradient
  dispatch    rows of tokens to the places of their experts; combine: the
              weighted sum of what the experts made of them; gradients of both
  layer_norm  forward with the statistics kept, and backward
  loss        softmax cross entropy of x w^T against target classes without
              keeping the logits, forward and backward

``own`` selects the framework's kernels; otherwise everything is computed with
elementary torch operations in 32 bits and rounded once at the end (the
router's selection in 64 bits: which expert comes first is decided there).
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
IGNORE = -100
EPS = 1e-5


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one new token through a router with a balancing bias and groups: latency
        {"name": "route one token", "op": "route", "rows": 1, "experts": 64, "k": 6, "dtype": "f32", "score": "sigmoid",
         "bias": True, "groups": 8, "top_groups": 3, "group_best": 2, "renormalize": True, "masked": False},
        # a prefill's tokens over many experts, with the order of the rows
        {"name": "route prefill", "op": "route", "rows": 8190, "experts": 256, "k": 8, "dtype": "f32", "score": "sigmoid",
         "bias": True, "groups": 8, "top_groups": 4, "group_best": 2, "renormalize": True, "masked": False},
        # gradient of softmax weights that were not renormalised: dense over the experts
        {"name": "route backward", "op": "route_backward", "rows": 8191, "experts": 128, "k": 4, "dtype": "bf16",
         "score": "softmax", "renormalize": False, "masked": True},
        # a decoding batch's way home, added to the residual stream
        {"name": "combine decode", "op": "combine", "rows": 24, "experts": 64, "k": 8, "h": 2048, "dtype": "bf16",
         "residual": True, "skew": 0.5, "dropped": 0.0},
        # a prefill's rows to their experts
        {"name": "dispatch prefill", "op": "dispatch", "rows": 8190, "experts": 32, "k": 4, "h": 2048, "dtype": "bf16",
         "skew": 0.7, "dropped": 0.0},
        # training over experts some of which live elsewhere: part of the choices has no row here
        {"name": "combine backward ragged", "op": "combine_backward", "rows": 4097, "experts": 16, "k": 6, "h": 1544,
         "dtype": "f16", "skew": 0.7, "dropped": 0.2},
        # the norm of a training micro-batch of odd length and width
        {"name": "norm train forward odd", "op": "norm", "rows": 8191, "n": 2057, "dtype": "bf16", "wtype": "f32"},
        # its gradient, with those of weight and bias, at an ordinary width
        {"name": "norm train backward", "op": "norm_backward", "rows": 8192, "n": 4096, "dtype": "bf16", "wtype": "bf16"},
        # scoring a few tokens: the projection to the vocabulary is read once
        {"name": "loss few rows", "op": "loss", "rows": 37, "vocab": 32003, "k": 2048, "dtype": "bf16"},
        # a training micro-batch over a large vocabulary
        {"name": "loss train forward", "op": "loss", "rows": 8192, "vocab": 131072, "k": 2048, "dtype": "bf16"},
        # a small ragged batch's gradient, with one of the log-sum too
        {"name": "loss backward ragged", "op": "loss_backward", "rows": 777, "vocab": 32003, "k": 1032, "dtype": "f16",
         "dlse": True},
        # a training micro-batch's gradient
        {"name": "loss train backward", "op": "loss_backward", "rows": 4096, "vocab": 65536, "k": 4096, "dtype": "bf16",
         "dlse": False},
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, int(round(v / step)) * step)


def draw(rng):
    op = rng.choice(["route", "route", "route_backward", "dispatch", "combine", "combine_backward", "norm", "norm_backward",
                     "loss", "loss", "loss_backward"])
    if op.startswith("route"):
        e = rng.choice([8, 16, 60, 64, 128, 160, 256, 384])
        c = {"op": op, "rows": _log_int(rng, 1, 16384), "experts": e, "k": rng.randint(1, 8),
             "dtype": rng.choice(["f32", "bf16", "f16"]), "score": rng.choice(["softmax", "sigmoid"]),
             "renormalize": rng.random() < 0.5, "masked": rng.random() < 0.3}
        if op == "route":
            g = rng.choice([1, 1, 4, 8]) if e % 8 == 0 else 1
            best = rng.choice([1, 2]) if g > 1 and e // g > 1 else 1
            c |= {"bias": rng.random() < 0.5, "groups": g, "group_best": best,
                  "top_groups": rng.randint((c["k"] * g + e - 1) // e, g)}
        return c
    if op.startswith("norm"):
        n = _log_int(rng, 64, 16384) if rng.random() < 0.3 else _log_int(rng, 64, 16384, 8)
        rows = max(1, min(_log_int(rng, 1, 32768), 8192 * 4096 // n))
        dt = rng.choice(["bf16", "f16", "f32"])
        return {"op": op, "rows": rows, "n": n, "dtype": dt, "wtype": rng.choice([dt, "f32"])}
    dt = rng.choice(["bf16", "f16"])
    if op.startswith("loss"):
        v, k = _log_int(rng, 500, 131072), _log_int(rng, 128, 4096, 8)
        most = 4096 * 65536 * 4096 // 2
        c = {"op": op, "rows": max(1, min(_log_int(rng, 1, 8192), most // (v * k))), "vocab": v, "k": k, "dtype": dt}
        if op == "loss_backward":
            c["dlse"] = rng.random() < 0.3
        return c
    k, h = rng.randint(1, 8), _log_int(rng, 64, 8192, 8) + rng.choice([0, 0, 0, 1])
    rows = max(1, min(_log_int(rng, 1, 16384), 8190 * 4 * 2048 // (k * h)))
    c = {"op": op, "rows": rows, "experts": rng.choice([8, 16, 32, 64, 128]), "k": k, "h": h, "dtype": dt,
         "skew": rng.choice([0.0, 0.4, 0.8]), "dropped": rng.choice([0.0, 0.0, 0.3])}
    if op == "combine":
        c["residual"] = rng.random() < 0.5
    return c


# ----------------------------------------------------------------- inputs
def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    c, op, rows, dt = case, case["op"], case["rows"], DTYPES[case["dtype"]]

    def randn(*shape, scale=1.0, dtype=dt):
        return torch.empty(shape, device=dev, dtype=dtype).normal_(0.0, scale, generator=g)

    def rand(*shape):
        return torch.rand(shape, device=dev, generator=g)

    s = {"case": case}
    if op.startswith("route"):
        e = c["experts"]
        # unequally loaded experts; with a mask, some experts are closed to some rows, and all of them to a few (padding)
        s["logits"] = (randn(rows, e, scale=1.5, dtype=torch.float32) + randn(e, scale=0.7, dtype=torch.float32)).to(dt)
        if c["masked"]:
            closed = (rand(rows, e) < 0.4) & (rand(rows, 1) < 0.3) | (rand(rows, 1) < 0.02)
            s["logits"].masked_fill_(closed, -math.inf)
        if op == "route":
            s["bias"] = randn(e, scale=0.05, dtype=torch.float32) if c["bias"] else None
        else:
            s["chosen"] = _choose(s["logits"].double(), c["k"])
            s["dweights"] = randn(rows, c["k"], dtype=torch.float32)
        return s
    if op.startswith("norm"):
        n, wt = c["n"], DTYPES[c["wtype"]]
        s["x"] = randn(rows, n) + randn(rows, 1)
        s["w"] = 1 + randn(n, scale=0.1, dtype=wt)
        s["b"] = randn(n, scale=0.1, dtype=wt)
        if op == "norm_backward":
            s["dy"] = randn(rows, n)
            x = s["x"].double()                # statistics as the forward pass keeps them
            s["mean"] = x.mean(1).float()
            s["rstd"] = (x.var(1, unbiased=False) + EPS).rsqrt().float()
        return s
    if op.startswith("loss"):
        v, k = c["vocab"], c["k"]
        s["w"] = randn(v, k, scale=2 * k ** -0.5)
        t = torch.randint(0, v, (rows,), device=dev, generator=g)
        # a model that has learned something: the target's logit stands out
        s["x"] = (randn(rows, k, dtype=torch.float32) + 2 * s["w"][t].float()).to(dt)
        ignored = rand(rows) < 0.1
        s["target"] = torch.where(ignored, IGNORE, t)
        if op == "loss_backward":
            # the mean over the tokens that count; f16 gradients are scaled up, as training in f16 does
            scale = 4096.0 if c["dtype"] == "f16" else 1.0
            s["dloss"] = torch.full((rows,), scale / rows, device=dev)
            s["dlse"] = 0.1 * scale / rows * rand(rows) if c["dlse"] else None
            s["lse"] = torch.cat([torch.logsumexp(a.float() @ s["w"].float().t(), 1) for a in s["x"].split(1024)])
            s["lse"].masked_fill_(ignored, 0)
        return s
    # distinct experts for every row, unequal loads
    e, k, h = c["experts"], c["k"], c["h"]
    load = c["skew"] * randn(e, dtype=torch.float32)
    chosen = (randn(rows, e, dtype=torch.float32) + load).topk(k, 1).indices
    dropped = rand(rows, k) < c["dropped"]
    chosen = torch.where(dropped, e, chosen)                    # (behind all others)
    s["place"] = _places(chosen, e)
    s["count"] = rows * k
    if op == "dispatch":
        s["x"] = randn(rows, h)
        s["out"] = torch.zeros(rows * k, h, dtype=dt, device=dev)
        return s
    s["r"] = randn(rows * k, h)
    s["weights"] = torch.softmax(randn(rows, k, dtype=torch.float32), 1)
    if op == "combine":
        s["residual"] = randn(rows, h) if c["residual"] else None
    else:
        s["dy"] = randn(rows, h)
        s["out"] = torch.zeros(rows * k, h, dtype=dt, device=dev)
    return s


# ----------------------------------------------------------- plain forms
def _choose(value, k):
    """The k largest values of every row, ties to the lower index, -1 where only -inf is left."""
    best, at = torch.sort(value, dim=1, descending=True, stable=True)
    return torch.where(best[:, :k] == -math.inf, -1, at[:, :k]).int()


def _places(chosen, e):
    """Where every slot goes when slots are sorted by expert (stable); -1 for slots of none."""
    flat = chosen.reshape(-1).long()
    flat = torch.where(flat < 0, e, flat)
    order = torch.sort(flat, stable=True).indices
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=order.device)
    return torch.where(flat < e, place, -1).view(chosen.shape).int()


def _scores(logits, score):
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-logits))
    p = torch.exp(logits - logits.amax(1, keepdim=True).clamp(min=-3e38))
    return p / p.sum(1, keepdim=True).clamp(min=1e-30)


def _plain_route(s):
    c, e, k = s["case"], s["case"]["experts"], s["case"]["k"]
    l64 = s["logits"].double()
    # without a bias scores order the experts as the logits do; sums of two need the scores themselves
    scored = s["bias"] is not None or c["group_best"] == 2
    value = _scores(l64, c["score"]) if scored else l64
    if s["bias"] is not None:
        value = value + s["bias"].double()
    value = value.masked_fill(l64 == -math.inf, -math.inf)
    if c["groups"] > 1:
        of = torch.sort(value.view(-1, c["groups"], e // c["groups"]), dim=2, descending=True).values
        if c["group_best"] == 2:               # of one open expert: its value alone
            of = of[..., 0] + of[..., 1].masked_fill(of[..., 1] == -math.inf, 0)
        else:
            of = of[..., 0]
        keep = torch.sort(of, dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        open_ = torch.zeros_like(of, dtype=torch.bool).scatter_(1, keep, True)
        value = value.masked_fill(~open_.repeat_interleave(e // c["groups"], 1), -math.inf)
    chosen = _choose(value, k)
    w = _scores(s["logits"].float(), c["score"]).gather(1, chosen.clamp(min=0).long())
    w = w.masked_fill(chosen < 0, 0)
    if c["renormalize"]:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-30)
    counts = (chosen.reshape(-1, 1) == torch.arange(e, device=w.device, dtype=torch.int32)).sum(0)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int()
    return {"weights": w, "chosen": chosen, "offsets": offsets, "place": _places(chosen, e)}


def _plain_route_backward(s):
    c, none = s["case"], s["chosen"] < 0
    at = s["chosen"].clamp(min=0).long()
    p = _scores(s["logits"].float(), c["score"])
    g = s["dweights"].masked_fill(none, 0)
    w = p.gather(1, at).masked_fill(none, 0)
    if c["renormalize"]:
        total = w.sum(1, keepdim=True).clamp(min=1e-30)
        g = (g - (g * w).sum(1, keepdim=True) / total) / total
    dp = torch.zeros_like(p).scatter_add_(1, at, g.masked_fill(none, 0))
    dl = dp * p * (1 - p) if c["score"] == "sigmoid" else p * (dp - (dp * p).sum(1, keepdim=True))
    return dl.to(s["logits"].dtype)


def _plain_dispatch(s):
    x, place, n = s["x"], s["place"], s["count"]
    out = torch.zeros(n + 1, x.shape[1], dtype=x.dtype, device=x.device)       # one row more, for slots of none
    out[torch.where(place < 0, n, place).long()] = x[:, None]
    return out[:n]


def _gathered(s):
    return s["r"].float()[s["place"].clamp(min=0).long()]


def _plain_combine(s):
    w = s["weights"].masked_fill(s["place"] < 0, 0)
    y = (w[..., None] * _gathered(s)).sum(1)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(s["r"].dtype)


def _plain_combine_backward(s):
    dy, place, n, dt = s["dy"].float(), s["place"], s["count"], s["r"].dtype
    dr = torch.zeros(n + 1, dy.shape[1], dtype=dt, device=dy.device)
    dr[torch.where(place < 0, n, place).long()] = (s["weights"][..., None] * dy[:, None]).to(dt)
    dw = (_gathered(s) * dy[:, None]).sum(2).masked_fill(place < 0, 0)
    return {"dr": dr[:n], "dweights": dw}


def _plain_norm(s):
    x = s["x"].float()
    mean = x.mean(1, keepdim=True)
    rstd = 1 / ((x - mean).square().mean(1, keepdim=True) + EPS).sqrt()
    y = (x - mean) * rstd * s["w"].float() + s["b"].float()
    return {"y": y.to(s["x"].dtype), "mean": mean[:, 0], "rstd": rstd[:, 0]}


def _plain_norm_backward(s):
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xh = (s["x"].float() - s["mean"][:, None]) * rstd
    g = dy * s["w"].float()
    dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    wt = s["w"].dtype
    return {"dx": dx.to(s["x"].dtype), "dw": (dy * xh).sum(0).to(wt), "db": dy.sum(0).to(wt)}


def _plain_loss(s):
    logits = s["x"].float() @ s["w"].float().t()
    top = logits.amax(1, keepdim=True)
    lse = top[:, 0] + torch.exp(logits - top).sum(1).log()
    none = s["target"] == IGNORE
    loss = lse - logits.gather(1, s["target"].clamp(min=0)[:, None])[:, 0]
    return {"loss": loss.masked_fill(none, 0), "lse": lse.masked_fill(none, 0)}


def _plain_loss_backward(s):
    x, w, dt = s["x"].float(), s["w"].float(), s["x"].dtype
    none = s["target"] == IGNORE
    b = s["dloss"].masked_fill(none, 0)
    a = b if s["dlse"] is None else b + s["dlse"].masked_fill(none, 0)
    dl = (x @ w.t()).sub_(s["lse"][:, None]).exp_().mul_(a[:, None]).masked_fill_(none[:, None], 0)
    dl.scatter_add_(1, s["target"].clamp(min=0)[:, None], -b[:, None])
    return {"dx": (dl @ w).to(dt), "dw": (dl.t() @ x).to(dt)}


PLAIN = {"route": _plain_route, "route_backward": _plain_route_backward, "dispatch": _plain_dispatch,
         "combine": _plain_combine, "combine_backward": _plain_combine_backward, "norm": _plain_norm,
         "norm_backward": _plain_norm_backward, "loss": _plain_loss, "loss_backward": _plain_loss_backward}


# ------------------------------------------------------------------- run
def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        return PLAIN[op](s)
    import collective_communication_schedule_gb300 as ccl
    if op.startswith("route"):
        score = ccl.SCORE_SIGMOID if c["score"] == "sigmoid" else ccl.SCORE_SOFTMAX
        if op == "route_backward":
            return ccl.route_backward(s["dweights"], s["logits"], s["chosen"], score=score, renormalize=c["renormalize"])
        w, chosen, offsets, place = ccl.route(s["logits"], c["k"], score=score, bias=s["bias"], groups=c["groups"],
                                              top_groups=c["top_groups"], group_best=c["group_best"],
                                              renormalize=c["renormalize"], order=True)
        return {"weights": w, "chosen": chosen, "offsets": offsets, "place": place}
    if op == "dispatch":
        return ccl.dispatch(s["x"], s["place"], out=s["out"])
    if op == "combine":
        return ccl.combine(s["r"], s["place"], s["weights"], residual=s["residual"])
    if op == "combine_backward":
        dr, dw = ccl.combine_backward(s["dy"], s["r"], s["place"], s["weights"], out=s["out"])
        return {"dr": dr, "dweights": dw}
    if op == "norm":
        y, mean, rstd = ccl.layer_norm(s["x"], s["w"], s["b"], eps=EPS, stats=True)
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "norm_backward":
        dx, dw, db = ccl.layer_norm_backward(s["dy"], s["x"], s["w"], s["mean"], s["rstd"], bias=True)
        return {"dx": dx, "dw": dw, "db": db}
    if op == "loss":
        loss, lse = ccl.linear_cross_entropy(s["x"], s["w"], s["target"], ignore_index=IGNORE)
        return {"loss": loss, "lse": lse}
    dx, dw = ccl.linear_cross_entropy_backward(s["dloss"], s["x"], s["w"], s["target"], s["lse"], dlse=s["dlse"],
                                               ignore_index=IGNORE)
    return {"dx": dx, "dw": dw}


# ------------------------------------------------------------------ work
def work(case):
    c, op, rows = case, case["op"], case["rows"]
    es = 4 if c["dtype"] == "f32" else 2
    if op == "route":
        return {"bytes": rows * c["experts"] * es + rows * c["k"] * 12 + c["experts"] * 8, "flops": 8 * rows * c["experts"]}
    if op == "route_backward":
        return {"bytes": 2 * rows * c["experts"] * es + rows * c["k"] * 8, "flops": 8 * rows * c["experts"]}
    if op.startswith("norm"):
        n, ws = c["n"], 4 if c["wtype"] == "f32" else 2
        if op == "norm":
            return {"bytes": 2 * rows * n * es + 8 * rows + 2 * n * ws, "flops": 8 * rows * n}
        return {"bytes": 3 * rows * n * es + 8 * rows + 3 * n * ws, "flops": 14 * rows * n}
    if op.startswith("loss"):
        v, k = c["vocab"], c["k"]
        if op == "loss":
            return {"bytes": 2 * k * (rows + v) + 16 * rows, "flops": 2 * rows * v * k}
        return {"bytes": 4 * k * (rows + v) + 20 * rows, "flops": 6 * rows * v * k}
    k, h = c["k"], c["h"]
    slots = round(rows * k * (1 - c["dropped"]))
    if op == "dispatch":
        return {"bytes": es * h * (rows + slots) + 4 * rows * k, "flops": 0}
    if op == "combine":
        return {"bytes": es * h * (rows * (2 if c["residual"] else 1) + slots) + 8 * rows * k, "flops": 2 * slots * h}
    return {"bytes": es * h * (rows + 2 * slots) + 12 * rows * k, "flops": 3 * slots * h}


# ----------------------------------------------------------------- exact
def _weights64(logits, at, none, c):
    """Weights of given choices, for values and (by autograd) gradients."""
    dead = (logits == -math.inf).all(1, keepdim=True)
    logits = torch.where(dead, 0.0, logits)
    p = torch.sigmoid(logits) if c["score"] == "sigmoid" else torch.softmax(logits, 1)
    w = torch.where(none, 0.0, p.gather(1, at))
    return w / torch.where(none.all(1, keepdim=True), 1.0, w.sum(1, keepdim=True)) if c["renormalize"] else w


def _exact_route(s, c):
    l64, k, e = s["logits"].double(), c["k"], c["experts"]
    p = torch.sigmoid(l64) if c["score"] == "sigmoid" else torch.softmax(l64, 1).nan_to_num(0)
    scored = c["bias"] or c["group_best"] == 2
    value = (p if scored else l64) + (s["bias"].double() if c["bias"] else 0)
    value[l64 == -math.inf] = -math.inf
    if c["groups"] > 1:
        best = value.view(-1, c["groups"], e // c["groups"]).topk(c["group_best"], 2).values
        of = torch.where(best == -math.inf, 0, best).sum(2)
        of[best[..., 0] == -math.inf] = -math.inf
        # a group's rank: those that are better, and those before it that are as good
        before = torch.ones(c["groups"], c["groups"], device=of.device).tril(-1).bool()
        rank = ((of[:, None, :] > of[:, :, None]) | (of[:, None, :] == of[:, :, None]) & before).sum(2)
        value = torch.where((rank < c["top_groups"]).repeat_interleave(e // c["groups"], 1), value, -math.inf)
    best, at = value.topk(k, 1)
    return {"weights": _weights64(l64, at, best == -math.inf, c), "chosen": None, "offsets": None, "place": None}


def exact(case, seed):
    s, c, op = prepare(case, seed), case, case["op"]
    if op == "route":
        return _exact_route(s, c)
    if op == "route_backward":
        l64 = s["logits"].double().requires_grad_(True)
        none = s["chosen"] < 0
        w = _weights64(l64, s["chosen"].clamp(min=0).long(), none, c)
        (w * s["dweights"].double()).sum().backward()
        return l64.grad
    if op == "dispatch":
        out = torch.zeros_like(s["out"], dtype=torch.float64)
        for j in range(c["k"]):
            here = s["place"][:, j] >= 0
            out[s["place"][here, j].long()] = s["x"][here].double()
        return out
    if op in ("combine", "combine_backward"):
        place = s["place"].long()
        live = (place >= 0).double()
        w = s["weights"].double() * live
        y = s["residual"].double() if op == "combine" and c["residual"] else 0
        dr = torch.zeros(s["count"], c["h"], dtype=torch.float64, device=place.device)
        dw = torch.zeros_like(w)
        for j in range(c["k"]):
            at, here = place[:, j].clamp(min=0), live[:, j:j + 1]
            r = s["r"].double()[at]
            if op == "combine":
                y = y + w[:, j:j + 1] * r
            else:
                dr.index_add_(0, at, w[:, j:j + 1] * s["dy"].double())
                dw[:, j:j + 1] = (r * s["dy"].double()).sum(1, keepdim=True) * here
        return y if op == "combine" else {"dr": dr, "dweights": dw}
    if op.startswith("norm"):
        x = s["x"].double().requires_grad_(True)
        w, b = s["w"].double().requires_grad_(True), s["b"].double().requires_grad_(True)
        mean, var = x.mean(1, keepdim=True), x.var(1, unbiased=False, keepdim=True)
        rstd = (var + EPS) ** -0.5
        y = (x - mean) * rstd * w + b
        if op == "norm":
            return {"y": y.detach(), "mean": mean[:, 0].detach(), "rstd": rstd[:, 0].detach()}
        (y * s["dy"].double()).sum().backward()
        return {"dx": x.grad, "dw": w.grad, "db": b.grad}
    # the loss, some rows at a time
    w, none = s["w"].double(), s["target"] < 0
    out = {"loss": [], "lse": [], "dx": []}
    dw = torch.zeros_like(w) if op == "loss_backward" else None
    step = max(16, 2 ** 27 // c["vocab"])
    for i in range(0, c["rows"], step):
        rows = slice(i, i + step)
        x, t, off = s["x"][rows].double(), s["target"][rows].clamp(min=0)[:, None], none[rows, None]
        logits = x @ w.T
        if op == "loss":
            lse = torch.logsumexp(logits, 1, keepdim=True)
            out["lse"].append(torch.where(off, 0, lse)[:, 0])
            out["loss"].append(torch.where(off, 0, lse - logits.gather(1, t))[:, 0])
            continue
        b = torch.where(off, 0, s["dloss"][rows, None].double())
        a = b if s["dlse"] is None else b + torch.where(off, 0, s["dlse"][rows, None].double())
        dl = torch.softmax(logits, 1) * a
        dl.scatter_add_(1, t, -b)
        out["dx"].append(dl @ w)
        dw += dl.T @ x
    if op == "loss":
        return {"loss": torch.cat(out["loss"]), "lse": torch.cat(out["lse"])}
    return {"dx": torch.cat(out["dx"]), "dw": dw}

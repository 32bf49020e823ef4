"""One training step of a routed layer of experts and its loss, data-parallel
over virtual ranks.

Every rank has its own tokens and all weights.  Forward: layer norm, router
(sigmoid scores, a balancing bias, groups of experts), rows to the places of
their experts, two expert products, the weighted sum on top of the residual
stream, cross entropy of the projection to the vocabulary without its logits.
Backward: the same in reverse.  Ring AllReduces sum the gradients of the
vocabulary projection and of the router over the ranks, and the bias moves
towards experts that got fewer rows than others.

    python examples/routed_step.py            # prints the losses and what a step computes
"""
from __future__ import annotations

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import collective_communication_schedule_gb300 as ccl

RANKS, EXPERTS, CHOICES, HIDDEN, INNER, VOCAB = 2, 16, 4, 256, 512, 1000
ROUTING = dict(score=ccl.SCORE_SIGMOID, renormalize=True, scale=2.0)


def make(tokens=120, seed=0):
    """Tokens and targets of all ranks, and the weights they share."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rnd(*shape, scale=1.0, dtype=torch.bfloat16):
        return torch.empty(shape, device="cuda", dtype=dtype).normal_(0, scale, generator=g)

    target = [torch.randint(0, VOCAB, (tokens + 9 * r,), device="cuda", generator=g) for r in range(RANKS)]
    for t in target:
        t[::11] = -100                       # padding
    return {"x": [rnd(tokens + 9 * r, HIDDEN) for r in range(RANKS)], "target": target,
            "gain": 1 + rnd(HIDDEN, scale=0.1), "shift": rnd(HIDDEN, scale=0.1),
            "router": rnd(EXPERTS, HIDDEN, scale=HIDDEN ** -0.5),
            "bias": rnd(EXPERTS, scale=0.02, dtype=torch.float32),
            "up": rnd(EXPERTS, INNER, HIDDEN, scale=HIDDEN ** -0.5),
            "down": rnd(EXPERTS, HIDDEN, INNER, scale=INNER ** -0.5),
            "vocab": rnd(VOCAB, HIDDEN, scale=2 * HIDDEN ** -0.5)}


def rank_step(p, r, tokens_in_all):
    """What rank r computes: losses, choices, gradients of its tokens and of the weights."""
    x, target = p["x"][r], p["target"][r]
    # forward
    h, mean, rstd = ccl.layer_norm(x, p["gain"], p["shift"], stats=True)
    logits = ccl.linear(h, p["router"])
    weights, chosen, offsets, place = ccl.route(logits, CHOICES, bias=p["bias"], groups=4, top_groups=2, group_best=2,
                                                order=True, **ROUTING)
    rows = ccl.dispatch(h, place)
    inner, z = ccl.grouped_linear(rows, p["up"], offsets, act=ccl.ACT_GELU, preact=True)
    outs = ccl.grouped_linear(inner, p["down"], offsets)
    y = ccl.combine(outs, place, weights, residual=x)
    loss, lse = ccl.linear_cross_entropy(y, p["vocab"], target)

    # backward, of the mean over all ranks' tokens
    dloss = torch.full_like(loss, 1.0 / tokens_in_all)
    dy, dvocab = ccl.linear_cross_entropy_backward(dloss, y, p["vocab"], target, lse)
    douts, dweights = ccl.combine_backward(dy, outs, place, weights)
    dinner, ddown, _ = ccl.grouped_linear_backward(douts, inner, p["down"], offsets)
    drows, dup, _ = ccl.grouped_linear_backward(dinner, rows, p["up"], offsets, preact=z, act=ccl.ACT_GELU)
    dlogits = ccl.route_backward(dweights, logits, chosen, **ROUTING)
    dh_router, drouter, _ = ccl.linear_backward(dlogits, h, p["router"])
    dh = ccl.combine(drows, place, residual=dh_router)
    dx, dgain, dshift = ccl.layer_norm_backward(dh, x, p["gain"], mean, rstd, bias=True)
    return {"loss": loss, "weights": weights, "chosen": chosen, "counts": offsets.diff(), "dx": dx + dy, "dvocab": dvocab,
            "dup": dup, "ddown": ddown, "drouter": drouter, "dgain": dgain, "dshift": dshift}


def step(p):
    live = sum(int((t != -100).sum()) for t in p["target"])
    out = [rank_step(p, r, live) for r in range(RANKS)]
    total = {}
    for name, rows in (("dvocab", VOCAB), ("drouter", EXPERTS)):
        n = rows * HIDDEN // RANKS
        plan = ccl.Plan(ccl.Schedule.builtin(ccl.RING_ALLREDUCE, RANKS), n, ccl.BF16, channels=1)
        sums = [torch.empty((rows, HIDDEN), dtype=torch.bfloat16, device="cuda") for _ in range(RANKS)]
        plan.execute([o[name].view(torch.int16) for o in out], [t.view(torch.int16) for t in sums])
        torch.cuda.synchronize()
        plan.status()
        total[name] = sums[0]
    counts = sum(o["counts"] for o in out)
    total["bias"] = p["bias"] + 0.01 * torch.sign(counts.float().mean() - counts)
    total["loss"] = sum(o["loss"].sum() for o in out) / live
    ccl.tensor_status()
    return out, total


if __name__ == "__main__":
    ranks, total = step(make())
    print("loss", f"{total['loss'].item():.4f}", "rows by expert", sum(o["counts"] for o in ranks).tolist())
    for name in ("dx", "dup", "ddown", "dgain", "dshift"):
        print(name, " ".join(f"{o[name].float().norm().item():.3e}" for o in ranks))
    print("dvocab", f"{total['dvocab'].float().norm().item():.3e}", "drouter", f"{total['drouter'].float().norm().item():.3e}")

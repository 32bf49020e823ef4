"""One training step of a layer of experts over virtual ranks.

Four ranks hold their own tokens and two experts each.  A chunk program (one
chunk per token row) carries every rank's rows to the ranks that own their
experts and places them there by expert, so the expert products run on them as
they arrive; its mirror image brings the results back.  A dense projection adds
the result to the residual stream.  In the backward pass the same two programs
carry the gradients, a ring AllReduce sums the projection's gradient over the
ranks, and the update taken from the sum is orthogonalised.

    python examples/expert_step.py            # prints the norms of what a step computes
"""
from __future__ import annotations

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import collective_communication_schedule_gb300 as ccl

RANKS, EXPERTS, HIDDEN, INNER = 4, 8, 256, 512
PER = EXPERTS // RANKS                      # experts of a rank


def words(t):
    """The plans move 16-bit words whatever they mean."""
    return t.view(torch.int16)


class Exchange:
    """Rows of every rank to the owners of their experts and back.

    counts[r][e]: rows that rank r sends to expert e (each rank's rows are in
    expert order).  Rank d receives them sorted by expert, then by source."""

    def __init__(self, counts):
        self.counts = counts
        rows_in = max(sum(c) for c in counts)
        ends = [[0] for _ in range(RANKS)]
        ops = []
        for d in range(RANKS):
            at = 0
            for e in range(d * PER, (d + 1) * PER):
                for r in range(RANKS):
                    n, start = counts[r][e], sum(counts[r][:e])
                    if n:
                        ops.append((ccl.COPY, r, ccl.IN, start, d, ccl.OUT, at, n))
                    at += n
                ends[d].append(at)
        rows_out = max(e[-1] for e in ends)
        back = [(o, d, ccl.IN, doff, s, ccl.OUT, soff, n) for o, s, _, soff, d, _, doff, n in ops]
        self.offsets = [torch.tensor(e, dtype=torch.int32, device="cuda") for e in ends]
        self.rows_in, self.rows_out = max(1, rows_in), max(1, rows_out)
        kw = dict(channels=1, link_mode=ccl.LINK_DIRECT, tb_alloc=ccl.TB_BALANCED)
        there = ccl.Schedule.compile(ops, RANKS, (self.rows_in, self.rows_out, 0))
        self.there = ccl.Plan(there, HIDDEN, ccl.BF16, **kw)
        home = ccl.Schedule.compile(back, RANKS, (self.rows_out, self.rows_in, 0))
        self.home = ccl.Plan(home, HIDDEN, ccl.BF16, **kw)

    def _run(self, plan, rows, tensors):
        ins = [torch.nn.functional.pad(t, (0, 0, 0, n - t.shape[0])) for t, n in zip(tensors, rows[0])]
        outs = [torch.zeros((n, HIDDEN), dtype=torch.bfloat16, device="cuda") for n in rows[1]]
        plan.execute([words(t) for t in ins], [words(t) for t in outs])
        return outs

    def to_experts(self, tensors):
        return self._run(self.there, ([self.rows_in] * RANKS, [self.rows_out] * RANKS), tensors)

    def from_experts(self, tensors):
        outs = self._run(self.home, ([self.rows_out] * RANKS, [self.rows_in] * RANKS), tensors)
        return [t[:sum(c)] for t, c in zip(outs, self.counts)]


def make(tokens=96, seed=0):
    """Tokens, weights and output gradients of all ranks."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rnd(*shape, scale=1.0):
        return torch.empty(shape, device="cuda", dtype=torch.bfloat16).normal_(0, scale, generator=g)

    return {"x": [rnd(tokens + 7 * r, HIDDEN) for r in range(RANKS)],
            "router": rnd(HIDDEN, EXPERTS),
            "up": [rnd(PER, INNER, HIDDEN, scale=HIDDEN ** -0.5) for _ in range(RANKS)],
            "down": [rnd(PER, HIDDEN, INNER, scale=INNER ** -0.5) for _ in range(RANKS)],
            "proj": rnd(HIDDEN, HIDDEN, scale=HIDDEN ** -0.5),
            "dy": [rnd(tokens + 7 * r, HIDDEN) for r in range(RANKS)]}


def step(p):
    """Outputs, gradients and the projection's update of one step."""
    expert = [(x.float() @ p["router"].float()).argmax(1) for x in p["x"]]
    order = [torch.argsort(e, stable=True) for e in expert]
    ex = Exchange([torch.bincount(e, minlength=EXPERTS).tolist() for e in expert])

    # forward: rows to their experts, two products there, home, projection and residual
    rows = ex.to_experts([x[o] for x, o in zip(p["x"], order)])
    inner, kept, mixed = [], [], []
    for d in range(RANKS):
        h, z = ccl.grouped_linear(rows[d], p["up"][d], ex.offsets[d], act=ccl.ACT_GELU, preact=True)
        inner.append(h)
        kept.append(z)
        mixed.append(ccl.grouped_linear(h, p["down"][d], ex.offsets[d]))
    home = ex.from_experts(mixed)
    y = [ccl.linear(t, p["proj"], residual=x[o]) for t, x, o in zip(home, p["x"], order)]

    # backward: projection, rows to their experts again, two products, home
    dhome, dproj = [], []
    for r in range(RANKS):
        dx, dw, _ = ccl.linear_backward(p["dy"][r], home[r], p["proj"])
        dhome.append(dx)
        dproj.append(dw)
    drows = ex.to_experts(dhome)
    dup, ddown, dout = [], [], []
    for d in range(RANKS):
        dh, dw, _ = ccl.grouped_linear_backward(drows[d], inner[d], p["down"][d], ex.offsets[d])
        ddown.append(dw)
        dx, dw, _ = ccl.grouped_linear_backward(dh, rows[d], p["up"][d], ex.offsets[d], preact=kept[d],
                                                act=ccl.ACT_GELU)
        dup.append(dw)
        dout.append(dx)
    dtokens = [a + b for a, b in zip(ex.from_experts(dout), p["dy"])]

    # the projection is shared: sum its gradient over the ranks, update along its orthogonal factor
    n = HIDDEN * HIDDEN
    reduce = ccl.Plan(ccl.Schedule.builtin(ccl.RING_ALLREDUCE, RANKS), n // RANKS, ccl.BF16, channels=2)
    total = [torch.empty((HIDDEN, HIDDEN), dtype=torch.bfloat16, device="cuda") for _ in range(RANKS)]
    reduce.execute([words(t) for t in dproj], [words(t) for t in total])
    update = ccl.orthogonalize(total[0])
    torch.cuda.synchronize()
    for plan in (ex.there, ex.home, reduce):
        plan.status()
    ccl.tensor_status()
    return {"order": order, "expert": expert, "y": y, "dtokens": dtokens, "dup": dup, "ddown": ddown, "dproj": total[0],
            "update": update}


if __name__ == "__main__":
    out = step(make())
    for name in ("y", "dtokens", "dup", "ddown"):
        print(name, " ".join(f"{t.float().norm().item():.3f}" for t in out[name]))
    print("dproj", f"{out['dproj'].float().norm().item():.3f}", "update", f"{out['update'].float().norm().item():.3f}")

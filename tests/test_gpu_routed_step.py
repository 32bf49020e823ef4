"""The example's step -- norm, router, dispatch, expert products, combine, loss
and all their gradients over two virtual ranks -- against the whole computation
in 64 bits with the choices that the step made.

Every intermediate is bf16 (relative 2^-9).  Outputs pass through up to six
roundings and gradients through up to twelve; errors of independent terms add in
quadrature, so 2^-9 sqrt(12) ~ 0.7 % of the norm is expected and 2 % allowed.  The
router's gradient is a difference of terms of one size (g - sum g w), of which
about a third of the size is left here: 4 %."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import routed_step
    yield routed_step
    sys.path.remove(os.path.join(ROOT, "examples"))


def gelu(z):
    return 0.5 * z * (1 + torch.tanh((2 / torch.pi) ** 0.5 * (z + 0.044715 * z ** 3)))


@pytest.mark.parametrize("tokens,seed", [(120, 0), (1, 1), (401, 2)])
def test_step_against_64_bits(example, tokens, seed):
    p = example.make(tokens, seed)
    ranks, total = example.step(p)
    leaf = lambda t: t.double().requires_grad_(True)  # noqa: E731
    w = {n: leaf(p[n]) for n in ("gain", "shift", "router", "up", "down", "vocab")}
    xs = [leaf(x) for x in p["x"]]
    live = sum(int((t != -100).sum()) for t in p["target"])
    losses, wide = [], []
    for r, x in enumerate(xs):
        chosen, target = ranks[r]["chosen"].long(), p["target"][r]
        mean, var = x.mean(1, keepdim=True), x.var(1, unbiased=False, keepdim=True)
        h = (x - mean) * (var + 1e-5) ** -0.5 * w["gain"] + w["shift"]
        score = torch.sigmoid(h @ w["router"].T)
        c = score.detach() + p["bias"].double()
        # the choices are what the definition says for some scores within their roundings
        # (2^-9 of h and of the logits: 0.02 of a score covers them)
        groups = c.view(-1, 4, example.EXPERTS // 4).topk(2, 2).values.sum(2)
        kept = groups.topk(2, 1).values[:, 1:]
        assert bool((groups.gather(1, chosen // (example.EXPERTS // 4)) >= kept - 0.08).all())
        picked = c.gather(1, chosen)
        assert bool((picked[:, :-1] >= picked[:, 1:] - 0.04).all())
        s = score.gather(1, chosen)
        weights = 2.0 * s / s.sum(1, keepdim=True)
        assert (weights.detach() - ranks[r]["weights"].double()).norm() <= 0.02 * weights.detach().norm()
        y = x
        for j in range(example.CHOICES):
            e = chosen[:, j]
            inner = gelu(torch.einsum("tik,tk->ti", w["up"][e], h))
            y = y + weights[:, j:j + 1] * torch.einsum("tki,ti->tk", w["down"][e], inner)
        logits = y @ w["vocab"].T
        loss = torch.logsumexp(logits, 1) - logits.gather(1, target.clamp(min=0)[:, None])[:, 0]
        loss = torch.where(target == -100, 0.0, loss)
        # values are off by the roundings of y (2^-9 of its norm, against rows of norm 2) and of what went into it
        wide.append(4 * 2 * 2.0 ** -8 * y.detach().norm(dim=1).max().item())
        assert bool(((loss.detach() - ranks[r]["loss"].double()).abs() <= wide[-1]).all())
        losses.append(loss.sum())
    (sum(losses) / live).backward()
    assert abs(total["loss"].item() - (sum(losses) / live).item()) <= max(wide)

    def near(a, b, what, most=0.02):
        rel = ((a.double() - b).norm() / b.norm().clamp(min=1e-30)).item()
        assert rel < most, (what, rel)

    for r in range(example.RANKS):
        near(ranks[r]["dx"], xs[r].grad, f"dx {r}")
        assert int(ranks[r]["counts"].sum()) == p["x"][r].shape[0] * example.CHOICES
    for name, got in (("up", "dup"), ("down", "ddown"), ("gain", "dgain"), ("shift", "dshift")):
        near(sum(o[got].double() for o in ranks), w[name].grad, got)
    near(total["dvocab"], w["vocab"].grad, "dvocab")
    near(total["drouter"], w["router"].grad, "drouter", 0.04)
    counts = sum(o["counts"] for o in ranks)
    moved = total["bias"] - p["bias"]
    assert bool((moved[counts.float() > counts.float().mean()] < 0).all())

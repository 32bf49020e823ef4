"""The example's step over four virtual ranks -- rows exchanged by chunk
programs, expert products, dense projection, gradients, AllReduce,
orthogonalised update -- against the whole computation in 64 bits.

Every intermediate is bf16 (relative 2^-9): the outputs pass through four
roundings, the gradients through at most eight; errors of independent terms
add in quadrature, so 2^-9 x sqrt(8) ~ 0.6 % of the norm is expected and 2 %
allowed.  The summed projection gradient is rounded at every hop of the ring as
well; the update sits behind it and multiplies its error by up to the first
slope of the iteration where directions are weak, so it is compared with the
update of the gradient that the step itself computed."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import expert_step
    yield expert_step
    sys.path.remove(os.path.join(ROOT, "examples"))


def gelu(z):
    return 0.5 * z * (1 + torch.tanh((2 / torch.pi) ** 0.5 * (z + 0.044715 * z ** 3)))


@pytest.mark.parametrize("tokens,seed", [(96, 0), (1, 1), (33, 2)])
def test_step_against_64_bits(example, tokens, seed):
    p = example.make(tokens, seed)
    got = example.step(p)
    leaf = lambda t: t.double().requires_grad_(True)  # noqa: E731
    xs, up, down, proj = [leaf(x) for x in p["x"]], [leaf(w) for w in p["up"]], [leaf(w) for w in p["down"]], leaf(p["proj"])
    loss, ys = 0, []
    for r, x in enumerate(xs):
        rows = x[got["order"][r]]
        expert = got["expert"][r][got["order"][r]]
        outs = []
        for t, e in zip(rows, expert.tolist()):
            d, i = divmod(e, example.PER)
            outs.append(down[d][i] @ gelu(up[d][i] @ t))
        y = torch.stack(outs) @ proj.T + rows
        ys.append(y.detach())
        loss = loss + (y * p["dy"][r].double()).sum()
    loss.backward()

    def near(a, b, what):
        rel = ((a.double() - b).norm() / b.norm().clamp(min=1e-30)).item()
        assert rel < 0.02, (what, rel)

    for r in range(example.RANKS):
        near(got["y"][r], ys[r], f"y {r}")
        near(got["dtokens"][r], xs[r].grad[got["order"][r]], f"dx {r}")
    for d in range(example.RANKS):
        for i in range(example.PER):
            for name, ref in (("dup", up[d].grad[i]), ("ddown", down[d].grad[i])):
                if bool(ref.any()):
                    near(got[name][d][i], ref, name)
                else:
                    assert not got[name][d][i].any()
    near(got["dproj"], proj.grad, "dproj")
    g = got["dproj"].double()
    x = g / g.norm()
    for _ in range(5):
        m = x @ x.T
        x = 3.4445 * x + (-4.7750 * m + 2.0315 * (m @ m)) @ x
    near(got["update"], x, "update")

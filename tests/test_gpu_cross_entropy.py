"""Softmax cross entropy of x w^T and its gradients against 64 bits.

Tolerances, element by element.  A value (logit) is a sum of k products in 32
bits in any order: within k 2^-23 S of the exact one (S: the same product of
absolute values).  exp2 is within 2^-22, its argument rounds to 2^-24 of itself
(twice) and of the largest value's; the longest chain of additions of the sum of
exponentials is 64 in a tile, one per tile and 16 group, and a few joins.  The
derivative dl = a p - b [target] is rounded to the element type (half a step,
eps / 2; f16 is scaled so that it holds 2^-38 of the largest row's factor to half
a unit) and enters products of `vocab` or `rows` terms, each within 2^-23 times
their number of the sum of absolute values; the result is rounded once more."""
import ctypes
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DT = [torch.bfloat16, torch.float16]
IDS = ["bf16", "f16"]


@pytest.fixture(scope="module")
def ccl():
    import collective_communication_schedule_gb300 as m
    yield m
    m.tensor_status()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rnd(g, *shape, dtype=torch.float32, scale=1.0):
    return torch.empty(shape, device="cuda", dtype=torch.float32).normal_(0, scale, generator=g).to(dtype)


def close(got, want, slack, what=""):
    tiny = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}.get(got.dtype, 2.0 ** -150)
    d = (got.double() - want).abs()
    tol = slack + torch.finfo(got.dtype).eps / 2 * (want.abs() + slack) + tiny
    assert bool((d <= tol).all()), f"{what}: worst {(d / tol).max().item():.3g} of the tolerance, {int((~(d <= tol)).sum())} off"


def make(g, rows, vocab, k, dtype, sharp=2.0, ignored=0.15, bits=64):
    w = rnd(g, vocab, k, dtype=dtype, scale=sharp * k ** -0.5)
    t = torch.randint(0, vocab, (rows,), device="cuda", generator=g)
    x = (rnd(g, rows, k) + w[t].float()).to(dtype)
    t = torch.where(torch.rand(rows, device="cuda", generator=g) < ignored, -100, t)
    return x, w, t if bits == 64 else t.int()


def values64(x, w):
    x, w = x.double(), w.double()
    return x @ w.T, x.shape[1] * 2.0 ** -23 * (x.abs() @ w.abs().T)


def check_loss(ccl, x, w, t, ignore=-100):
    loss, lse = ccl.linear_cross_entropy(x, w, t, ignore_index=ignore)
    ccl.tensor_status()
    assert loss.dtype == lse.dtype == torch.float32 and loss.shape == lse.shape == t.shape
    v, e = values64(x, w)
    live = t != ignore
    want = torch.logsumexp(v, 1)
    e_t = e.gather(1, t.long().clamp(min=0)[:, None])[:, 0]
    own = v.gather(1, t.long().clamp(min=0)[:, None])[:, 0]
    far = (v.amax(1) - v.amin(1)).clamp(max=60)
    slack = e.amax(1) + 2.0 ** -22 + (80 + w.shape[0] / 4096 + 2 * far) * 2.0 ** -24 + 2.0 ** -22 * v.amax(1).abs()
    close(lse, torch.where(live, want, 0.0), slack + 2.0 ** -23 * want.abs(), "lse")
    close(loss, torch.where(live, want - own, 0.0), slack + e_t + 2.0 ** -22 * (v.amax(1) - own).abs(), "loss")
    assert not loss[~live].any() and not lse[~live].any()
    return loss, lse


def check_grad(ccl, x, w, t, dloss, dlse, lse=None, ignore=-100, chunk=None):
    rows, vocab, dtype = x.shape[0], w.shape[0], x.dtype
    if lse is None:
        lse = torch.where(t != ignore, torch.logsumexp(x.double() @ w.double().T, 1), 0.0).float()
    got = ccl.linear_cross_entropy_backward(dloss, x, w, t, lse, dlse=dlse, ignore_index=ignore)
    ccl.tensor_status()
    live = t != ignore
    b = torch.where(live, dloss.double(), 0.0)
    a = b + torch.where(live, dlse.double(), 0.0) if dlse is not None else b
    v, e = values64(x, w)
    p = torch.where(live[:, None], torch.exp(v - lse.double()[:, None]), 0.0)
    hot = torch.zeros_like(p).scatter_(1, t.long().clamp(min=0)[:, None], torch.where(live, 1.0, 0.0).double()[:, None])
    dl = a[:, None] * p - b[:, None] * hot
    # exp's argument: the value's error, and roundings of the products with log2 e and of the difference
    rel = torch.expm1((e + 2.0 ** -22 + 2.0 ** -23 * (v.abs() + lse.double()[:, None].abs())).clamp(max=50))
    off = (a.abs()[:, None] * p) * rel + 2.0 ** -23 * (a.abs() + b.abs())[:, None] * (p + hot)
    off = off + torch.finfo(dtype).eps / 2 * (dl.abs() + off)
    # an exponential below the smallest normal number of 32 bits counts as 0, and so may the product with its factor
    off = off + torch.where(live, 2.0 ** -126 * (1 + a.abs()), 0.0)[:, None]
    if dtype == torch.float16:
        off = off + torch.maximum(a.abs(), b.abs()).max() * 2.0 ** -38
        off[~live] = 0
    size = dl.abs() + off
    xz = torch.where((a != 0)[:, None] | (b != 0)[:, None], x.double(), 0.0)
    close(got[0], dl @ w.double(), off @ w.double().abs() + vocab * 2.0 ** -23 * (size @ w.double().abs()), "dx")
    close(got[1], dl.T @ xz, off.T @ xz.abs() + rows * 2.0 ** -23 * (size.T @ xz.abs()), "dw")
    assert not got[0][~live].any()
    return got


SIZES = [(1, 1, 1), (1, 2, 8), (2, 31, 63), (37, 129, 72), (128, 256, 64), (129, 257, 264), (300, 500, 1000), (5, 1003, 1032),
         (700, 5000, 200), (1, 33001, 520), (260, 2050, 2048), (1500, 1000, 136)]


@pytest.mark.parametrize("dtype", DT, ids=IDS)
@pytest.mark.parametrize("rows,vocab,k", SIZES)
def test_loss(ccl, rows, vocab, k, dtype):
    for bits in (64, 32):
        check_loss(ccl, *make(gen(rows + vocab), rows, vocab, k, dtype, bits=bits))


@pytest.mark.parametrize("dtype", DT, ids=IDS)
@pytest.mark.parametrize("rows,vocab,k", [(1, 40001, 8), (32, 40001, 72), (33, 40001, 72), (100, 40000, 40), (128, 45001, 64),
                                          (129, 40001, 72), (200, 60000, 40), (256, 60001, 136)])
def test_loss_of_few_rows_over_several_tiles(ccl, rows, vocab, k, dtype):
    """More tiles than SMs, all rows in each of them: statistics are carried from one tile to the next."""
    g = gen(rows + vocab)
    x, w, t = make(g, rows, vocab, k, dtype)
    t[0] = vocab - 1
    t[-1] = 0 if rows > 1 else vocab - 1
    loss, lse = check_loss(ccl, x, w, t)
    other = check_loss(ccl, x, w, t.int())
    assert torch.equal(other[0], loss) and torch.equal(other[1], lse)
    check_grad(ccl, x, w, t, rnd(g, rows) / rows, rnd(g, rows) / rows, lse)


@pytest.mark.parametrize("dtype", DT, ids=IDS)
@pytest.mark.parametrize("rows,vocab,k", SIZES)
def test_loss_backward(ccl, rows, vocab, k, dtype):
    g = gen(rows + vocab)
    x, w, t = make(g, rows, vocab, k, dtype)
    dloss = rnd(g, rows) / rows
    dx, dw = check_grad(ccl, x, w, t, dloss, None)
    check_grad(ccl, x, w, t.int(), dloss, rnd(g, rows) / rows)
    lse = torch.where(t != -100, torch.logsumexp(x.double() @ w.double().T, 1), 0.0).float()
    only = ccl.linear_cross_entropy_backward(dloss, x, w, t, lse, need_dw=False)
    assert only[1] is None and ((only[0].double() - dx.double()).norm() <= 2.0 ** -7 * dx.double().norm())
    only = ccl.linear_cross_entropy_backward(dloss, x, w, t, lse, need_dx=False)
    assert only[0] is None and ((only[1].double() - dw.double()).norm() <= 2.0 ** -7 * dw.double().norm())


@pytest.mark.parametrize("rows,vocab,k,dtype", [(2100, 70001, 72, torch.bfloat16), (4100, 33000, 264, torch.float16),
                                                (3000, 100000, 33, torch.bfloat16)])
def test_pieces_of_the_vocabulary(ccl, rows, vocab, k, dtype):
    """More derivatives than the workspace holds at a time: the last piece is narrower, dx grows over the pieces."""
    g = gen(vocab)
    x, w, t = make(g, rows, vocab, k, dtype)
    t[::97] = vocab - 1
    t[1::97] = 0
    check_loss(ccl, x, w, t)
    dloss = torch.full((rows,), 1024.0 / rows, device="cuda")
    dx, dw = check_grad(ccl, x, w, t, dloss, None)
    lse = torch.where(t != -100, torch.cat([torch.logsumexp(c.double() @ w.double().T, 1) for c in x.split(500)]), 0.0).float()
    again = ccl.linear_cross_entropy_backward(dloss, x, w, t, lse)
    assert torch.equal(again[0], ccl.linear_cross_entropy_backward(dloss, x, w, t, lse, need_dw=False)[0])
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)
    only = ccl.linear_cross_entropy_backward(dloss, x, w, t, lse, need_dx=False)[1]
    assert ((only.double() - dw.double()).norm() <= 2.0 ** -7 * dw.double().norm())


@pytest.mark.parametrize("dtype", DT, ids=IDS)
def test_views_and_odd_strides(ccl, dtype):
    g = gen(3)
    for lead, pitch, k in ((8, 16, 72), (3, 5, 72), (0, 1, 65)):
        big_x, big_w = rnd(g, 62, k + pitch + lead, dtype=dtype), rnd(g, 310, k + pitch + lead, dtype=dtype, scale=0.2)
        x, w = big_x[1::1, lead:lead + k][:60], big_w[5:305, lead:lead + k]
        t = torch.randint(0, 300, (60,), device="cuda", generator=g)
        loss, lse = check_loss(ccl, x, w, t)
        flat = ccl.linear_cross_entropy(x.contiguous(), w.contiguous(), t)
        assert torch.equal(flat[0], loss) and torch.equal(flat[1], lse)
        d = rnd(g, 60)
        got = check_grad(ccl, x, w, t, d, None, lse)
        want = ccl.linear_cross_entropy_backward(d, x.contiguous(), w.contiguous(), t, lse)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def c_grad(ccl, **kw):
    a = ccl.CrossEntropyGrad(**kw)
    size = ctypes.c_int64()
    assert ccl.lib.ccl_cross_entropy_grad_workspace(ctypes.byref(a), ctypes.byref(size)) == 0
    ws = torch.full((size.value + 512,), 0x7f, dtype=torch.uint8, device="cuda")
    at = ws.data_ptr() + 255 & ~255
    assert ccl.lib.ccl_cross_entropy_grad(ctypes.byref(a), at, size.value, torch.cuda.current_stream().cuda_stream) == 0, \
        ccl.lib.ccl_last_error_detail()
    torch.cuda.synchronize()
    assert bool((ws[at - ws.data_ptr() + size.value:] == 0x7f).all())


@pytest.mark.parametrize("rows,vocab,k,lead", [(70, 300, 72, 8), (70, 300, 72, 3), (2100, 70001, 40, 8), (2100, 70001, 40, 1)])
def test_writes_only_its_outputs(ccl, rows, vocab, k, lead):
    g = gen(rows + lead)
    x, w, t = make(g, rows, vocab, k, torch.bfloat16)
    lse = ccl.linear_cross_entropy(x, w, t)[1]
    d = rnd(g, rows)
    want = ccl.linear_cross_entropy_backward(d, x, w, t, lse)
    held = [torch.full((n + 2, k + 16 + lead), 7.0, dtype=torch.bfloat16, device="cuda") for n in (rows, vocab)]
    dx, dw = (h[1:-1, lead:lead + k] for h in held)
    c_grad(ccl, rows=rows, vocab=vocab, k=k, dtype=ccl.BF16, target_bits=64, ignore_index=-100, x=x.data_ptr(), w=w.data_ptr(),
           target=t.data_ptr(), dloss=d.data_ptr(), lse=lse.data_ptr(), dx=dx.data_ptr(), dw=dw.data_ptr(), lddx=dx.stride(0),
           lddw=dw.stride(0))
    assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])
    dx.fill_(7)
    dw.fill_(7)
    assert all(bool((h == 7).all()) for h in held)


@pytest.mark.parametrize("dtype", DT, ids=IDS)
@pytest.mark.parametrize("rows,vocab,k", [(40, 300, 72), (700, 1500, 264), (2100, 70000, 40)])
def test_ignored_rows_may_hold_anything(ccl, rows, vocab, k, dtype):
    g = gen(rows)
    x, w, t = make(g, rows, vocab, k, dtype, ignored=0.3)
    t[:3] = -100
    dead = t == -100
    zero = torch.where(dead[:, None], torch.zeros_like(x), x)
    bad = x.clone()
    bad[dead] = math.nan
    bad[0, 0], bad[1] = math.inf, 1.0
    loss, lse = ccl.linear_cross_entropy(zero, w, t)
    other = ccl.linear_cross_entropy(bad, w, t)
    assert torch.equal(loss, other[0]) and torch.equal(lse, other[1])
    d = rnd(g, rows)
    want = ccl.linear_cross_entropy_backward(d, zero, w, t, lse)
    d = torch.where(dead, math.nan, d)
    got = ccl.linear_cross_entropy_backward(d, bad, w, t, torch.where(dead, math.nan, lse), dlse=torch.where(dead, math.inf, 0.0))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    clean = ccl.linear_cross_entropy_backward(d, x, w, t, lse)
    assert torch.equal(clean[0], want[0]) and bool(clean[1].isfinite().all())
    only = ccl.linear_cross_entropy_backward(d, bad, w, t, lse, need_dx=False)[1]
    assert bool(only.isfinite().all())
    # nothing but ignored rows
    none = torch.full_like(t, -100)
    loss, lse = ccl.linear_cross_entropy(bad, w, none)
    dx, dw = ccl.linear_cross_entropy_backward(d, bad, w, none, lse)
    assert not loss.any() and not lse.any() and not dx.any() and not dw.any()
    # another index to ignore, within the vocabulary
    t = torch.where(dead, 5, t)
    check_loss(ccl, x, w, t, ignore=5)


def test_no_rows(ccl):
    w = torch.ones(20, 16, dtype=torch.bfloat16, device="cuda")
    x, t, z = w[:0], torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, device="cuda")
    loss, lse = ccl.linear_cross_entropy(x, w, t)
    assert loss.shape == (0,)
    dx, dw = ccl.linear_cross_entropy_backward(z, x, w, t, z)
    assert dx.shape == (0, 16) and dw.shape == (20, 16) and not dw.any()


def test_targets_out_of_range_count_as_ignored_and_are_reported(ccl):
    g = gen(4)
    x, w, t = make(g, 50, 200, 64, torch.bfloat16, ignored=0.0)
    none, bad = t.clone(), t.clone()
    none[[3, 7, 9, 11]] = -100
    bad[3], bad[7], bad[9], bad[11] = 200, -1, 2 ** 40, -2 ** 63
    d = rnd(g, 50)
    want = ccl.linear_cross_entropy(x, w, none)
    grads = ccl.linear_cross_entropy_backward(d, x, w, none, want[1])
    ccl.tensor_status()
    got = ccl.linear_cross_entropy(x, w, bad)
    with pytest.raises(ccl.CclError, match="target"):
        ccl.tensor_status()
    other = ccl.linear_cross_entropy_backward(d, x, w, bad, got[1])
    with pytest.raises(ccl.CclError, match="target"):
        ccl.tensor_status()
    ccl.tensor_status()
    for a, b in zip((*got, *other), (*want, *grads)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", DT, ids=IDS)
def test_large_values_and_sure_predictions(ccl, dtype):
    g = gen(5)
    x, w, t = make(g, 150, 700, 64, dtype)
    x = (x.float() * 30).to(dtype)                       # values to +-500, most targets far above the rest
    loss, lse = check_loss(ccl, x, w, t)
    check_grad(ccl, x, w, t, rnd(g, 150), None, lse)
    # a target whose share is all but 1: the loss keeps its digits
    w = torch.zeros(300, 8, dtype=dtype, device="cuda")
    w[7, 0] = 1
    x = torch.zeros(4, 8, dtype=dtype, device="cuda")
    x[:, 0] = torch.tensor([8.0, 12.0, 14.0, 15.0])
    t = torch.full((4,), 7, device="cuda")
    loss, _ = ccl.linear_cross_entropy(x, w, t)
    want = torch.log1p(299 * torch.exp(-x[:, 0].double()))
    # the sum is 1 and 299 small terms: each addition rounds to 2^-24, 4 of them in a group of 16, 4 groups of a warp,
    # 3 joins of warps, one a tile (at most 10) and 16 joins at the end
    close(loss, want, (4 + 4 + 3 + 10 + 16) * 2.0 ** -24 * torch.ones_like(want))


def test_values_that_are_not_finite_stay_in_their_rows(ccl):
    g = gen(6)
    x, w, t = make(g, 140, 600, 72, torch.bfloat16, ignored=0.0)
    loss, lse = ccl.linear_cross_entropy(x, w, t)
    bad = x.clone()
    bad[5, 3], bad[131] = math.nan, math.nan
    other, other_lse = ccl.linear_cross_entropy(bad, w, t)
    keep = [i for i in range(140) if i not in (5, 131)]
    assert bool(other[[5, 131]].isnan().all()) and torch.equal(other[keep], loss[keep]) and torch.equal(other_lse[keep], lse[keep])
    dx, dw = ccl.linear_cross_entropy_backward(torch.ones(140, device="cuda"), bad, w, t, other_lse)
    want, _ = ccl.linear_cross_entropy_backward(torch.ones(140, device="cuda"), x, w, t, lse)
    assert bool(dx[[5, 131]].isnan().all()) and torch.equal(dx[keep], want[keep]) and bool(dw.isnan().all())


@pytest.mark.parametrize("dtype", DT, ids=IDS)
def test_factors_of_any_size(ccl, dtype):
    """dloss from tiny (a mean over many tokens) to large, and of very different sizes side by side: powers of two
    of it change nothing but the exponent."""
    g = gen(7)
    x, w, t = make(g, 90, 400, 136, dtype, ignored=0.1)
    lse = ccl.linear_cross_entropy(x, w, t)[1]
    d = rnd(g, 90)
    for e in (-12, 6) if dtype == torch.float16 else (-100, -30, 60):
        check_grad(ccl, x, w, t, d * 2.0 ** e, None, lse)
    mixed = d * 2.0 ** (-torch.arange(90, device="cuda") / 4).floor()
    check_grad(ccl, x, w, t, mixed, None, lse)
    check_grad(ccl, x, w, t, mixed, mixed.flip(0) * 3, lse)
    zero = torch.zeros(90, device="cuda")
    check_grad(ccl, x, w, t, zero, d, lse)               # of the log-sums alone
    dx, dw = ccl.linear_cross_entropy_backward(zero, x, w, t, lse)
    assert not dx.any() and not dw.any()
    minus = ccl.linear_cross_entropy_backward(d, x, w, t, lse, dlse=-d)
    p = torch.zeros(90, 400, dtype=torch.float64, device="cuda")
    live = t != -100
    p[live, t[live]] = -d[live].double()
    close(minus[0], p @ w.double(), 2.0 ** -8 * (p.abs() @ w.double().abs()))


def test_gradients_against_differences(ccl):
    """The loss sum(dloss loss + dlse lse) in 64 bits along random directions of x and w.  dl is rounded to bf16
    (2^-9 of each term, independent): in quadrature over the terms of the derivative; the difference is off by h^2
    times third derivatives below 4 |v|^3 a value."""
    g = gen(8)
    x, w, t = make(g, 40, 150, 64, torch.bfloat16)
    live = t != -100
    d, e = rnd(g, 40), rnd(g, 40)
    lse = ccl.linear_cross_entropy(x, w, t)[1]
    dx, dw = ccl.linear_cross_entropy_backward(d, x, w, t, lse, dlse=e)

    def f(x, w):
        v = x @ w.T
        s = torch.logsumexp(v, 1)
        own = v.gather(1, t.clamp(min=0)[:, None])[:, 0]
        return (torch.where(live, d.double() * (s - own) + e.double() * s, 0.0)).sum()

    h = 1e-5
    for which, grad in enumerate((dx, dw)):
        v = rnd(g, *grad.shape).double()
        at = lambda s: f(x.double() + (s * h * v if which == 0 else 0), w.double() + (s * h * v if which else 0))  # noqa: E731
        slope, along = (at(1) - at(-1)) / (2 * h), (grad.double() * v).sum()
        size = (grad.double() * v).norm() + (grad.double().abs().sum(1) if which == 0 else grad.double().abs().sum(0)).norm()
        assert abs(slope - along) <= 6 * 2.0 ** -8 * size + 1e-6 * slope.abs(), (slope.item(), along.item(), size.item())


def test_weights_past_32_bits(ccl):
    """Rows of w and dw beyond 2^31 elements."""
    vocab, k = 270000, 8200                                              # 2.2e9 elements, 4.4 GB
    g = gen(9)
    w = torch.empty(vocab, k, dtype=torch.bfloat16, device="cuda").normal_(0, k ** -0.5, generator=g)
    t = torch.tensor([vocab - 1, 3, 262000], device="cuda")
    x = (rnd(g, 3, k) + w[t].float()).to(torch.bfloat16)
    loss, lse = ccl.linear_cross_entropy(x, w, t)
    v = torch.cat([x.double() @ c.double().T for c in w.split(20000)], 1)
    want = torch.logsumexp(v, 1)
    # values: the sum of absolute products is about 0.64 |x| |w| sqrt(k): k 2^-23 of it
    slack = k * 2.0 ** -23 * x.double().abs().sum(1) * k ** -0.5 * 2
    close(lse, want, slack)
    close(loss, want - v.gather(1, t[:, None])[:, 0], 2 * slack)
    d = torch.ones(3, device="cuda")
    dx, dw = ccl.linear_cross_entropy_backward(d, x, w, t, lse)
    p = torch.exp(v - lse.double()[:, None])
    p.scatter_add_(1, t[:, None], -torch.ones(3, 1, dtype=torch.float64, device="cuda"))
    for rows in (slice(0, 100), slice(261950, 262050), slice(vocab - 100, vocab)):
        ref = p[:, rows].T @ x.double()
        close(dw[rows], ref, 2.0 ** -7 * (p[:, rows].abs().T @ x.double().abs()))
    ref = sum(p[:, i:i + 20000] @ w[i:i + 20000].double() for i in range(0, vocab, 20000))
    assert (dx.double() - ref).norm() <= 2.0 ** -7 * ref.norm()
    ccl.tensor_status()


@pytest.mark.parametrize("rows,vocab,k,dtype", [(50, 3001, 136, torch.float16), (2100, 66000, 64, torch.bfloat16)])
def test_results_repeat_bit_for_bit_on_other_streams_and_in_graphs(ccl, rows, vocab, k, dtype):
    def everything(x, w, t, d, **kw):
        loss, lse = ccl.linear_cross_entropy(x, w, t, **kw)
        return [loss, lse, *ccl.linear_cross_entropy_backward(d, x, w, t, lse, dlse=d, **kw)]

    g = gen(rows)
    sets = []
    for _ in range(2):
        x, w, t = make(g, rows, vocab, k, dtype)
        x[t == -100] = math.nan
        sets.append((x, w, t, rnd(g, rows)))
    want = [everything(*s) for s in sets]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = everything(*sets[0], stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[0]))
    held = [[t.clone() for t in sets[0]] for _ in range(2)]
    graphs, outs = [], []
    for h in held:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(everything(*h))
        graphs.append(graph)
    for a, b in zip(held[1], sets[1]):
        a.copy_(b)
    for _ in range(2):
        graphs[0].replay()
        graphs[1].replay()
    torch.cuda.synchronize()
    for o, u in zip(outs, want):
        assert all(torch.equal(a, b) for a, b in zip(o, u))
    ccl.tensor_status()

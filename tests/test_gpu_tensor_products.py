"""Dense and expert-grouped products, their gradients and the orthogonalised
update, against plain implementations in 64 bits.

Tolerances, element by element: a product of k terms summed in 32 bits in any
order is within k 2^-23 S of the exact one (S: the same product of absolute
values; 2^-23 covers sums that truncate); an activation multiplies that by
at most 1.13 (the largest slope of gelu; silu's is 1.10) and adds its own
error, below 2^-16 of |z| (the fast exponential's 2^-21 and a few operations);
rounding to the output type adds half a unit, 2^-9 of the value for bf16, 2^-12
and 2^-25 absolute for f16 -- taken once more (doubled) for sums that sit on a
rounding boundary.
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

UNIT = {torch.bfloat16: (2.0 ** -8, 2.0 ** -130), torch.float16: (2.0 ** -10, 2.0 ** -24)}
DT = [torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def ccl():
    import collective_communication_schedule_gb300 as m
    yield m
    m.tensor_status()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rnd(g, *shape, dtype, scale=1.0):
    return torch.empty(shape, device="cuda", dtype=dtype).normal_(0, scale, generator=g)


def act64(z, act):
    return {0: lambda: z, 1: lambda: z.clamp(min=0),
            2: lambda: 0.5 * z * (1 + torch.tanh((2 / torch.pi) ** 0.5 * (z + 0.044715 * z ** 3))),
            3: lambda: z * torch.sigmoid(z)}[act]()


def act_grad64(z, act):
    if act == 0:
        return torch.ones_like(z)
    z = z.clone().requires_grad_(True)
    act64(z, act).sum().backward()
    return z.grad * (z.detach() > 0) if act == 1 else z.grad


def close(got, want, slack, dtype):
    """|got - want| <= slack + the rounding of `dtype`, everywhere."""
    rel, tiny = UNIT[dtype]
    d = (got.double() - want).abs()
    tol = slack + rel * want.abs() + tiny
    assert bool((d <= tol).all()), f"worst {(d / tol).max().item():.3g} of the tolerance, {int((d > tol).sum())} off"


def product_slack(absprod, k):
    return absprod * (k * 2.0 ** -23)


def check_linear(ccl, rows, n, k, dtype, act, bias, residual, preact, x=None, w=None):
    g = gen(rows * 31 + n * 7 + k)
    x = rnd(g, rows, k, dtype=dtype) if x is None else x
    w = rnd(g, n, k, dtype=dtype, scale=k ** -0.5) if w is None else w
    b = rnd(g, n, dtype=dtype) if bias else None
    r = rnd(g, rows, n, dtype=dtype) if residual else None
    got = ccl.linear(x, w, bias=b, residual=r, act=act, preact=preact)
    y, zk = got if preact else (got, None)
    z = x.double() @ w.double().T
    slack = product_slack(x.double().abs() @ w.double().abs().T, k)
    if bias:
        z = z + b.double()
    want = act64(z, act)
    ys = 1.13 * slack + 2.0 ** -16 * z.abs()
    if residual:
        want = want + r.double()
    ys = ys + 2.0 ** -22 * (z.abs() + want.abs())
    close(y, want, ys, dtype)
    if preact:
        close(zk, z, slack + 2.0 ** -22 * z.abs(), dtype)


SIZES = [(1, 8, 8), (1, 1, 1), (3, 5, 7), (1, 256, 4096), (17, 130, 72), (33, 128, 64), (64, 1000, 520),
         (129, 257, 65), (200, 384, 1032), (257, 640, 200), (513, 1111, 328), (1500, 2050, 136)]


@pytest.mark.parametrize("dtype", DT, ids=["bf16", "f16"])
@pytest.mark.parametrize("rows,n,k", SIZES)
def test_linear_plain(ccl, rows, n, k, dtype):
    check_linear(ccl, rows, n, k, dtype, ccl.ACT_NONE, False, False, False)


@pytest.mark.parametrize("dtype", DT, ids=["bf16", "f16"])
@pytest.mark.parametrize("act", [0, 1, 2, 3])
@pytest.mark.parametrize("rows,n,k,bias,residual,preact", [
    (1, 72, 264, True, True, False), (40, 203, 96, True, False, True), (300, 520, 328, False, True, True),
    (129, 1031, 64, True, True, True)])
def test_linear_epilogue(ccl, rows, n, k, bias, residual, preact, act, dtype):
    check_linear(ccl, rows, n, k, dtype, act, bias, residual, preact)


@pytest.mark.parametrize("k", [1, 2, 8, 9, 63, 64, 65, 127, 128, 1024, 5000])
def test_linear_reduction_lengths(ccl, k):
    check_linear(ccl, 70, 140, k, torch.bfloat16, ccl.ACT_NONE, True, False, False)


def test_linear_strided_and_unaligned_operands(ccl):
    g = gen(5)
    big = rnd(g, 90, 400, dtype=torch.bfloat16)
    for x in (big[:, :136], big[:, 8:144], big[:, 3:139], big[1::2, 5:69], big.view(-1)[1:1 + 80 * 136].view(80, 136)):
        check_linear(ccl, *(x.shape[0], 96, x.shape[1]), torch.bfloat16, ccl.ACT_SILU, True, True, True, x=x)
    w = rnd(g, 70, 300, dtype=torch.bfloat16)[:, 7:143]
    check_linear(ccl, 50, 70, 136, torch.bfloat16, ccl.ACT_NONE, False, False, False, w=w)


def test_linear_writes_only_its_output(ccl):
    g = gen(6)
    for n, off in ((130, 0), (131, 3), (64, 8)):
        x, w = rnd(g, 45, 72, dtype=torch.float16), rnd(g, n, 72, dtype=torch.float16)
        whole = torch.full((47, n + 16), 9.0, dtype=torch.float16, device="cuda")
        out = whole[1:46, off:off + n]
        ccl.linear(x, w, out=out)
        assert torch.equal(out, ccl.linear(x, w))
        mask = torch.ones_like(whole, dtype=torch.bool)
        mask[1:46, off:off + n] = False
        assert bool((whole[mask] == 9).all())


def test_rows_far_apart(ccl):
    """Row strides that take offsets past 32 bits (a slice of a long cache)."""
    rows, stride = 40000, 60000
    g = gen(31)
    cache = torch.empty(rows * stride, dtype=torch.bfloat16, device="cuda")      # 4.8 GB
    wide = cache.view(rows, stride)
    x, out, r = wide[:, 8:72], wide[:, 1000:1040], wide[:, 5000:5040]
    x.normal_(0, 1, generator=g)
    r.normal_(0, 1, generator=g)
    w = rnd(g, 40, 64, dtype=torch.bfloat16)
    want = x.double() @ w.double().T + r.double()
    ccl.linear(x, w, residual=r, out=out)
    close(out, want, product_slack(x.double().abs() @ w.double().abs().T, 64) + 2.0 ** -22 * want.abs(), torch.bfloat16)
    dy, z = wide[:, 5000:5040], wide[:, 1000:1040]
    got = ccl.linear_backward(dy, x, w, preact=z, act=ccl.ACT_SILU, bias=True)
    check_grads(got, dy, x, w, z, 3, [(0, rows)], torch.bfloat16)
    del cache


def test_linear_adds_to_the_residual_in_place(ccl):
    g = gen(7)
    x, w, r = rnd(g, 33, 64, dtype=torch.bfloat16), rnd(g, 200, 64, dtype=torch.bfloat16), rnd(g, 33, 200,
                                                                                              dtype=torch.bfloat16)
    want = ccl.linear(x, w, residual=r)
    ccl.linear(x, w, residual=r, out=r)
    assert torch.equal(r, want)


def test_linear_keeps_infinities_and_nan_where_they_belong(ccl):
    g = gen(8)
    x, w = rnd(g, 70, 100, dtype=torch.bfloat16), rnd(g, 150, 100, dtype=torch.bfloat16)
    base = ccl.linear(x, w)
    x[3, 5] = float("nan")
    x[68, 99] = float("inf")
    y = ccl.linear(x, w)
    assert bool(y[3].isnan().all()) and bool((y[68].isinf()).all())
    keep = [i for i in range(70) if i not in (3, 68)]
    assert torch.equal(y[keep], base[keep])
    assert bool(ccl.linear(x, w, act=ccl.ACT_RELU)[3].isnan().all())


def test_no_rows(ccl):
    x, w = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(8, 64, dtype=torch.bfloat16,
                                                                               device="cuda")
    assert ccl.linear(x, w).shape == (0, 8)
    dx, dw, db = ccl.linear_backward(torch.empty(0, 8, dtype=torch.bfloat16, device="cuda"), x, w, bias=True)
    assert dx.shape == (0, 64) and not dw.any() and not db.any()
    offs = torch.zeros(4, dtype=torch.int32, device="cuda")
    w3 = w.repeat(3, 1, 1)
    assert ccl.grouped_linear(x, w3, offs).shape == (0, 8)
    dx, dw, db = ccl.grouped_linear_backward(torch.empty(0, 8, dtype=torch.bfloat16, device="cuda"), x, w3, offs,
                                             bias=True)
    assert dw.shape == (3, 8, 64) and not dw.any() and not db.any()


# ------------------------------------------------------------- gradients
def check_grads(got, dy, x, w, z, act, spans, dtype):
    """Against the formula in 64 bits.  dz is rounded to the type once more
    (relative 2^-9 or 2^-12 of each term) before the products; the bias
    gradient sums it unrounded."""
    dx, dw, db = got
    unit = UNIT[dtype][0]
    dz = dy.double()
    if act:
        dz = dz * act_grad64(z.double(), act)
    own = 2.0 ** -14 * (1 + (z.double().abs() if act else 0)) * dy.double().abs() if act else 0 * dz
    size = dz.abs() + own
    wd, xd = w.double(), x.double()
    wd = wd if wd.dim() == 3 else wd[None]
    rounding = (unit if act else 0) + x.shape[0] * 2.0 ** -23
    for e, (i, j) in enumerate(spans):
        a = dz[i:j]
        if dx is not None:
            slack = size[i:j] @ wd[e].abs() * ((unit if act else 0) + w.shape[-2] * 2.0 ** -23) + own[i:j] @ wd[e].abs()
            close(dx[i:j], a @ wd[e], slack, dtype)
        if dw is not None:
            d = dw if dw.dim() == 2 else dw[e]
            close(d, a.T @ xd[i:j], size[i:j].T @ xd[i:j].abs() * rounding + own[i:j].T @ xd[i:j].abs(), dtype)
        if db is not None:
            d = db if db.dim() == 1 else db[e]
            close(d, a.sum(0), own[i:j].sum(0) + size[i:j].sum(0) * (x.shape[0] * 2.0 ** -23), dtype)


@pytest.mark.parametrize("dtype", DT, ids=["bf16", "f16"])
@pytest.mark.parametrize("act", [0, 1, 2, 3])
@pytest.mark.parametrize("rows,n,k", [(1, 8, 8), (1, 300, 72), (5, 3, 7), (65, 129, 200), (333, 264, 520),
                                      (700, 131, 72)])
def test_linear_backward(ccl, rows, n, k, act, dtype):
    g = gen(rows + n + k)
    dy, x, w, z = (rnd(g, *s, dtype=dtype) for s in ((rows, n), (rows, k), (n, k), (rows, n)))
    got = ccl.linear_backward(dy, x, w, preact=z, act=act, bias=True)
    check_grads(got, dy, x, w, z, act, [(0, rows)], dtype)


@pytest.mark.parametrize("act", [2, 3])
def test_gradients_against_differences(ccl, act):
    """The whole path (forward keeps z, backward uses it) against central
    differences of the loss sum(dy * y) in 64 bits along random directions:
    the kept z and dz are bf16 (2^-8 each with the output's rounding), so a
    directional derivative is within 3 x 2^-8 of the sum of its terms' sizes,
    taken in quadrature over the independent roundings, plus the difference
    quotient's h^2."""
    dtype = torch.bfloat16
    g = gen(77)
    rows, n, k = 40, 72, 56
    x, w, b, dy = (rnd(g, *s, dtype=dtype) for s in ((rows, k), (n, k), (n,), (rows, n)))
    w = (w.float() * k ** -0.5).to(dtype)
    y, z = ccl.linear(x, w, bias=b, act=act, preact=True)
    grads = ccl.linear_backward(dy, x, w, preact=z, act=act, bias=True)

    def loss(xx, ww, bb):
        return (dy.double() * act64(xx @ ww.T + bb, act)).sum()

    base = [t.double() for t in (x, w, b)]
    for i, grad in enumerate(grads):
        v = torch.randn(base[i].shape, device="cuda", dtype=torch.float64, generator=g)
        h = 1e-4
        up, down = list(base), list(base)
        up[i], down[i] = base[i] + h * v, base[i] - h * v
        want = (loss(*up) - loss(*down)) / (2 * h)
        got = (grad.double() * v).sum()
        spread = (grad.double() * v).square().sum().sqrt()
        assert abs(got - want) <= 3 * 2.0 ** -8 * 6 * spread + 1e-6, (i, got.item(), want.item(), spread.item())


def test_backward_computes_only_what_is_asked(ccl):
    g = gen(9)
    dt = torch.bfloat16
    dy, x, w = (rnd(g, *s, dtype=dt) for s in ((70, 48), (70, 40), (48, 40)))
    full = ccl.linear_backward(dy, x, w, bias=True)
    for dx, dw, db in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 0, 1)):
        part = ccl.linear_backward(dy, x, w, bias=bool(db), need_dx=bool(dx), need_dw=bool(dw))
        for asked, p, f in zip((dx, dw, db), part, full):
            assert (p is None) == (not asked)
            if asked:
                assert torch.equal(p, f)


# --------------------------------------------------------------- experts
COUNTS = [[5], [0, 7, 0], [1, 0, 64, 65, 0, 130, 3], [63, 64, 65, 1], [0, 0, 300, 0], [17] * 40,
          [1] * 9 + [0] * 20 + [257]]


def offsets_of(counts, first=0):
    o = [first]
    for c in counts:
        o.append(o[-1] + c)
    return o


@pytest.mark.parametrize("dtype", DT, ids=["bf16", "f16"])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}x{sum(c)}")
@pytest.mark.parametrize("n,k,act,bias,preact", [(136, 72, 0, False, False), (257, 65, 3, True, True)])
def test_grouped_linear(ccl, counts, n, k, act, bias, preact, dtype):
    first, tail = 3, 4          # rows before and after the experts' own
    offs = offsets_of(counts, first)
    rows, e = offs[-1] + tail, len(counts)
    g = gen(rows + n)
    x, w = rnd(g, rows, k, dtype=dtype), rnd(g, e, n, k, dtype=dtype, scale=k ** -0.5)
    x[:first] = float("nan")
    x[offs[-1]:] = float("inf")
    b = rnd(g, e, n, dtype=dtype) if bias else None
    o = torch.tensor(offs, dtype=torch.int32, device="cuda")
    out = torch.full((rows, n), 5.0, dtype=dtype, device="cuda")
    got = ccl.grouped_linear(x, w, o, bias=b, act=act, preact=preact, out=out)
    y = got[0] if preact else got
    assert y is out
    assert bool((y[:first] == 5).all()) and bool((y[offs[-1]:] == 5).all())
    for i in range(e):
        s = slice(offs[i], offs[i + 1])
        z = x[s].double() @ w[i].double().T
        slack = product_slack(x[s].double().abs() @ w[i].double().abs().T, k)
        if bias:
            z = z + b[i].double()
        close(y[s], act64(z, act), 1.13 * slack + 2.0 ** -15 * z.abs(), dtype)
        if preact:
            close(got[1][s], z, slack + 2.0 ** -22 * z.abs(), dtype)


@pytest.mark.parametrize("dtype", DT, ids=["bf16", "f16"])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}x{sum(c)}")
@pytest.mark.parametrize("n,k,act", [(136, 72, 0), (131, 200, 2)])
def test_grouped_backward(ccl, counts, n, k, act, dtype):
    first, tail = 2, 3
    offs = offsets_of(counts, first)
    rows, e = offs[-1] + tail, len(counts)
    g = gen(rows + n)
    dy, x, z = rnd(g, rows, n, dtype=dtype), rnd(g, rows, k, dtype=dtype), rnd(g, rows, n, dtype=dtype)
    w = rnd(g, e, n, k, dtype=dtype)
    # rows that no expert owns never reach a gradient
    x[:first] = float("nan")
    dy[offs[-1]:] = float("inf")
    x[offs[-1]:] = float("nan")
    o = torch.tensor(offs, dtype=torch.int32, device="cuda")
    got = ccl.grouped_linear_backward(dy, x, w, o, preact=z, act=act, bias=True)
    check_grads(got, dy, x, w, z, act, list(zip(offs[:-1], offs[1:])), dtype)


@pytest.mark.parametrize("counts", [[3, 70, 0, 65, 1, 127, 200, 33] * 5, [900, 1, 1300, 77], [64] * 24],
                         ids=lambda c: f"{len(c)}x{sum(c)}")
def test_grouped_backward_with_many_tiles_per_threadblock(ccl, counts):
    """Several experts' tiles pass through each threadblock's ring of stages,
    with the cleared last slices of more than one in flight."""
    offs = offsets_of(counts)
    rows, e, n, k, dtype = offs[-1], len(counts), 1032, 1288, torch.bfloat16
    g = gen(rows)
    dy, x = rnd(g, rows, n, dtype=dtype), rnd(g, rows, k, dtype=dtype)
    w = rnd(g, e, n, k, dtype=dtype)
    o = torch.tensor(offs, dtype=torch.int32, device="cuda")
    got = ccl.grouped_linear_backward(dy, x, w, o, bias=True)
    ccl.tensor_status()
    check_grads(got, dy, x, w, None, 0, list(zip(offs[:-1], offs[1:])), dtype)


@pytest.mark.parametrize("rows,n,k", [(4100, 4104, 520), (16, 5000, 4096), (1, 3000, 6000), (300, 512, 8192),
                                      (2048, 2048, 2056)])
def test_linear_large_and_split(ccl, rows, n, k):
    check_linear(ccl, rows, n, k, torch.bfloat16, ccl.ACT_NONE, True, True, False)
    ccl.tensor_status()


def test_grouped_with_one_expert_equals_the_dense_product(ccl):
    g = gen(11)
    x, w = rnd(g, 77, 96, dtype=torch.bfloat16), rnd(g, 1, 200, 96, dtype=torch.bfloat16)
    o = torch.tensor([0, 77], dtype=torch.int32, device="cuda")
    d = (ccl.grouped_linear(x, w, o).double() - ccl.linear(x, w[0]).double()).abs()
    assert bool((d <= 2.0 ** -7 * ccl.linear(x, w[0]).double().abs() + 1e-3).all())


def test_bad_offsets_stay_inside_the_rows_and_are_reported(ccl):
    g = gen(12)
    x, w = rnd(g, 60, 64, dtype=torch.bfloat16), rnd(g, 3, 40, 64, dtype=torch.bfloat16)
    for offs in ([0, 20, 10, 60], [0, 10, 20, 61], [-5, 10, 20, 60]):
        ccl.tensor_status()
        o = torch.tensor(offs, dtype=torch.int32, device="cuda")
        ccl.grouped_linear(x, w, o)
        with pytest.raises(ccl.CclError) as e:
            ccl.tensor_status()
        assert e.value.code == 1 and "offsets" in e.value.detail
        ccl.grouped_linear_backward(x[:, :40].contiguous(), x, w, o, bias=True)
        with pytest.raises(ccl.CclError):
            ccl.tensor_status()
    ccl.tensor_status()


# -------------------------------------------------------- orthogonalising
def ns64(g, steps, coeffs, eps=1e-7):
    a, b, c = coeffs
    x = g / (g.norm() + eps)
    for _ in range(steps):
        m = x @ x.T if x.shape[0] <= x.shape[1] else x.T @ x
        r = b * m + c * (m @ m)
        x = a * x + (r @ x if x.shape[0] <= x.shape[1] else x @ r)
    return x


MUON = (3.4445, -4.7750, 2.0315)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32], ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", [(1, 1, 1), (1, 5, 300), (1, 64, 64), (1, 128, 128), (3, 100, 77), (2, 129, 520),
                                   (1, 700, 33), (1, 513, 1000), (2, 1000, 384)])
def test_orthogonalize(ccl, shape, dtype):
    """Each step rounds three matrices to f16: 2^-12 / sqrt(3) relative in the
    2-norm each, 15 roundings in quadrature 5.5e-4; a rounding made early
    grows against the directions it does not share by at most the slope
    3.4445 per step, but only until those reach size 1 themselves (two or
    three steps for these spectra): a factor of about 10, 5.5e-3, and the
    update's own rounding 2^-9 / sqrt(3) on top of it."""
    g = rnd(gen(sum(shape)), *shape, dtype=torch.float32).mul_(0.02).to(dtype)
    out = ccl.orthogonalize(g)
    assert out.dtype == torch.bfloat16 and out.shape == g.shape
    for i in range(shape[0]):
        want = ns64(g[i].double(), 5, MUON)
        rel = ((out[i].double() - want).norm() / want.norm()).item()
        assert rel <= 8e-3, rel


@pytest.mark.parametrize("shape", [(1, 128, 384), (1, 385, 128), (2, 100, 900), (1, 2000, 77), (3, 128, 2048), (1, 60, 1025),
                                   (40, 64, 257), (1, 2049, 128), (2, 127, 511), (1, 3, 2000)])
def test_orthogonalize_with_a_short_side(ccl, shape):
    """One threadblock or a cluster per matrix; same tolerance as above."""
    g = rnd(gen(sum(shape)), *shape, dtype=torch.float32).mul_(3.0)
    out = torch.full((shape[0], shape[1] + 1, shape[2] + 5), 7.0, dtype=torch.bfloat16, device="cuda")
    view = out[:, :-1, 2:-3]
    ccl.orthogonalize(g, out=view)
    ccl.tensor_status()
    mask = torch.ones_like(out, dtype=torch.bool)
    mask[:, :-1, 2:-3] = False
    assert bool((out[mask] == 7).all())
    for i in range(shape[0]):
        want = ns64(g[i].double(), 5, MUON)
        rel = ((view[i].double() - want).norm() / want.norm()).item()
        assert rel <= 8e-3, rel


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32], ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("shape", [(1, 128, 2049), (1, 4096, 128), (2, 77, 3333), (1, 3001, 5), (1, 128, 4097), (9, 16, 4095),
                                   (33, 40, 2500), (150, 24, 700)])
def test_orthogonalize_with_a_long_side_and_in_batches(ccl, shape, dtype):
    """The largest clusters, and batches that go around them or leave them to
    the general products; same tolerance as above."""
    g = rnd(gen(sum(shape)), *shape, dtype=torch.float32).mul_(0.1).to(dtype)
    out = ccl.orthogonalize(g)
    ccl.tensor_status()
    assert torch.equal(out, ccl.orthogonalize(g))
    for i in {0, shape[0] // 2, shape[0] - 1}:
        want = ns64(g[i].double(), 5, MUON)
        rel = ((out[i].double() - want).norm() / want.norm()).item()
        assert rel <= 8e-3, rel


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32], ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("p,q", [(128, 385), (65, 130), (127, 1001), (385, 7), (3, 2047), (90, 64)])
def test_orthogonalize_loads_the_same_from_any_alignment(ccl, p, q, dtype):
    """Rows on 16-byte boundaries and off them, and in place, with nothing but
    NaN around the matrix: the same bits."""
    g = rnd(gen(p + q), p, q, dtype=torch.float32).to(dtype)
    want = ccl.orthogonalize(g, out=torch.empty(p, q, dtype=torch.bfloat16, device="cuda"))
    for lead, pitch in ((8, -(-q // 8) * 8 + 16), (1, q + 1), (3, q + 7)):
        held = torch.full((p + 2, pitch + lead), float("nan"), dtype=dtype, device="cuda")
        view = held[1:-1, lead:lead + q]
        view.copy_(g)
        assert torch.equal(ccl.orthogonalize(view), want)
        if dtype == torch.bfloat16:
            ccl.orthogonalize(view, out=view)
            assert torch.equal(view, want)
            held[1:-1, lead:lead + q] = float("nan")
            assert bool(held.isnan().all())


def test_orthogonalize_options(ccl):
    g = rnd(gen(3), 96, 160, dtype=torch.float32)
    cubic = (1.5, -0.5, 0.0)
    for steps in (1, 2, 7):
        for scale in (1.0, 0.2):
            out = torch.empty(96, 170, dtype=torch.float16, device="cuda")[:, :160]
            assert ccl.orthogonalize(g, steps=steps, coeffs=cubic, scale=scale, eps=1e-3, out=out) is out
            want = scale * ns64(g.double(), steps, cubic, 1e-3)
            assert ((out.double() - want).norm() / want.norm()).item() <= 8e-3


def test_orthogonalize_strided_view_and_scale_invariance(ccl):
    big = rnd(gen(4), 3, 70, 200, dtype=torch.bfloat16)
    view = big[:, 1:60, 3:150]
    assert torch.equal(ccl.orthogonalize(view), ccl.orthogonalize(view.contiguous()))
    # a power of two of a bf16 gradient changes neither its rounding nor its direction
    for e in (-30, 20):
        assert torch.equal(ccl.orthogonalize((view.float() * 2.0 ** e).to(torch.bfloat16).contiguous(), eps=0.0),
                           ccl.orthogonalize(view.contiguous(), eps=0.0))


def test_orthogonalize_of_zero_is_zero(ccl):
    assert not ccl.orthogonalize(torch.zeros(2, 40, 130, device="cuda")).any()


# ------------------------------------------------------ streams and calls
def test_results_repeat_bit_for_bit_on_other_streams_and_in_graphs(ccl):
    g = gen(21)
    dt = torch.bfloat16
    x, dy, z = rnd(g, 300, 264, dtype=dt), rnd(g, 300, 136, dtype=dt), rnd(g, 300, 136, dtype=dt)
    w = rnd(g, 5, 136, 264, dtype=dt)
    o = torch.tensor([0, 100, 100, 163, 290, 300], dtype=torch.int32, device="cuda")

    def everything(**kw):
        return [ccl.linear(x, w[0], act=ccl.ACT_GELU, **kw), ccl.grouped_linear(x, w, o, **kw),
                *ccl.grouped_linear_backward(dy, x, w, o, preact=z, act=ccl.ACT_SILU, bias=True, **kw),
                ccl.orthogonalize(w, **kw)]

    want = everything()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = everything(stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = everything()
    for t in held:
        t.zero_()
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, held))


# ---------------------------------------------- experts through the C entry
def c_call(ccl, name, args):
    """A call of the C interface with the workspace it asks for, on the current stream."""
    import ctypes
    size = ctypes.c_int64()
    fail = getattr(ccl.lib, name + "_workspace")(ctypes.byref(args), ctypes.byref(size))
    assert fail == 0, ccl.lib.ccl_last_error_detail().decode()
    ws = torch.empty(max(size.value, 1), dtype=torch.uint8, device="cuda")
    fail = getattr(ccl.lib, name)(ctypes.byref(args), ws.data_ptr(), size.value, torch.cuda.current_stream().cuda_stream)
    assert fail == 0, ccl.lib.ccl_last_error_detail().decode()


@pytest.mark.parametrize("in_place", [False, True], ids=["apart", "in place"])
@pytest.mark.parametrize("dtype", DT, ids=["bf16", "f16"])
@pytest.mark.parametrize("counts", [[100], [70, 0, 65, 300, 255, 129, 97], [250, 17, 1], [68] * 12, [5, 16, 0, 33]],
                         ids=lambda c: f"{len(c)}x{sum(c)}")
@pytest.mark.parametrize("n,k,act", [(136, 64, 0), (1024, 264, 0), (131, 72, 0), (136, 64, 2)])
def test_experts_with_a_residual(ccl, n, k, act, counts, dtype, in_place):
    """Every row gets its own row of the residual, also the last rows of an
    expert whose tile does not end with a block of 16."""
    first, tail = 3, 4          # rows before and after the experts' own
    offs = offsets_of(counts, first)
    rows, e = offs[-1] + tail, len(counts)
    g = gen(rows + n)
    x, w = rnd(g, rows, k, dtype=dtype), rnd(g, e, n, k, dtype=dtype, scale=k ** -0.5)
    r = rnd(g, rows, n, dtype=dtype, scale=4.0)
    o = torch.tensor(offs, dtype=torch.int32, device="cuda")
    out = r.clone() if in_place else torch.full((rows, n), 5.0, dtype=dtype, device="cuda")
    before = out.clone()
    c_call(ccl, "ccl_linear", ccl.Linear(
        rows=rows, n=n, k=k, dtype=ccl.BF16 if dtype == torch.bfloat16 else ccl.F16, act=act, experts=e, x=x.data_ptr(),
        w=w.data_ptr(), residual=(out if in_place else r).data_ptr(), offsets=o.data_ptr(), y=out.data_ptr()))
    ccl.tensor_status()
    assert torch.equal(out[:first], before[:first]) and torch.equal(out[offs[-1]:], before[offs[-1]:])
    for i in range(e):
        s = slice(offs[i], offs[i + 1])
        z = x[s].double() @ w[i].double().T
        want = act64(z, act) + r[s].double()
        slack = 1.13 * product_slack(x[s].double().abs() @ w[i].double().abs().T, k) + 2.0 ** -16 * z.abs()
        close(out[s], want, slack + 2.0 ** -22 * (z.abs() + want.abs()), dtype)


@pytest.mark.parametrize("dtype", DT, ids=["bf16", "f16"])
@pytest.mark.parametrize("act", [2, 3])
def test_activation_gradients_at_the_ends_of_the_range(ccl, act, dtype):
    """The slope is 0 far below zero and 1 far above, up to the largest finite
    value and at the infinities that a kept z can overflow to; NaN stays."""
    big = [100.0, 1000.0, 6e4] + ([1e10, 1.8e19, 2e19, 1e30, 3e38] if dtype == torch.bfloat16 else []) + [float("inf")]
    z = torch.tensor([[-v for v in big] + big + [float("nan")]], dtype=dtype, device="cuda")
    want = torch.tensor([[0.0] * len(big) + [1.0] * len(big)], dtype=dtype, device="cuda")
    n = z.shape[1]
    one, x = torch.ones_like(z), torch.ones(1, 8, dtype=dtype, device="cuda")
    dx, dw, db = ccl.linear_backward(one, x, torch.ones(n, 8, dtype=dtype, device="cuda"), preact=z, act=act, bias=True)
    assert torch.equal(db[None, :-1], want) and bool(db[-1].isnan())
    assert torch.equal(dw[:-1], want.T.expand(-1, 8)) and bool(dw[-1].isnan().all())
    for i in range(n - 1):          # an element's own product
        dx, _, _ = ccl.linear_backward(one[:, :1], x, torch.ones(1, 8, dtype=dtype, device="cuda"), preact=z[:, i:i + 1],
                                       act=act, need_dw=False)
        assert bool((dx == want[0, i]).all()), z[0, i]


@pytest.mark.parametrize("counts", [None, [600, 0, 2400, 514, 66]], ids=["dense", "experts"])
@pytest.mark.parametrize("n,k", [(200, 136), (131, 72), (520, 264)])
def test_bias_gradient_does_not_depend_on_what_else_is_asked(ccl, n, k, counts):
    """Many chunks of rows, whose sums cancel but for the roundings of the
    additions: what is left shows the order, which the sizes alone give."""
    rows, dt = 3580, torch.bfloat16
    g = gen(rows + n)
    dy, x = rnd(g, rows, n, dtype=dt), rnd(g, rows, k, dtype=dt)
    offs = offsets_of(counts or [rows])
    for i, j in zip(offs[:-1], offs[1:]):
        dy[(i + j) // 2:j] = -dy[i:(i + j) // 2]
    if counts:
        w = rnd(g, len(counts), n, k, dtype=dt)
        o = torch.tensor(offs, dtype=torch.int32, device="cuda")

        def call(**kw):
            return ccl.grouped_linear_backward(dy, x, w, o, bias=True, **kw)[2]
    else:
        w = rnd(g, n, k, dtype=dt)

        def call(**kw):
            return ccl.linear_backward(dy, x, w, bias=True, **kw)[2]
    want = call()
    for dx, dw in ((0, 0), (1, 0), (0, 1)):
        assert torch.equal(call(need_dx=bool(dx), need_dw=bool(dw)), want), (dx, dw)


@pytest.mark.parametrize("offs,sound", [([0, 20, 10, 60], [(0, 0, 10), (2, 20, 60)]),
                                        ([0, 10, 20, 61], [(0, 0, 10), (1, 10, 20), (2, 20, 60)]),
                                        ([-5, 10, 20, 60], [(0, 0, 10), (1, 10, 20), (2, 20, 60)]),
                                        ([70, 80, 90, 100], []),
                                        ([0, 2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1], [])])
@pytest.mark.parametrize("n", [40, 37])
def test_bad_offsets_write_nothing_around_the_outputs(ccl, offs, sound, n):
    """Outputs lie inside larger tensors whose rest stays as it is; rows of
    ranges that overlap no other (expert, first, end) are right."""
    rows, k, e, dt = 60, 64, 3, torch.bfloat16
    g = gen(13)
    x, dy, z = rnd(g, rows, k, dtype=dt), rnd(g, rows, n, dtype=dt), rnd(g, rows, n, dtype=dt)
    w = rnd(g, e, n, k, dtype=dt, scale=k ** -0.5)
    o = torch.tensor(offs, dtype=torch.int32, device="cuda")

    def inside(*shape):
        """A packed view with a matrix's worth of other memory on both sides."""
        size = 1
        for v in shape:
            size *= v
        held = torch.full((3 * size + 16,), 7.0, dtype=dt, device="cuda")
        lead = size + -size % 8
        return held, lead, size, held[lead:lead + size].view(shape)

    held = {name: inside(*s) for name, s in (("y", (rows, n)), ("z", (rows, n)), ("dx", (rows, k)), ("dw", (e, n, k)),
                                             ("db", (e, n)))}
    at = {name: h[3].data_ptr() for name, h in held.items()}
    ccl.tensor_status()
    common = dict(rows=rows, n=n, k=k, dtype=ccl.BF16, experts=e, x=x.data_ptr(), w=w.data_ptr(), offsets=o.data_ptr())
    c_call(ccl, "ccl_linear", ccl.Linear(act=ccl.ACT_SILU, y=at["y"], z=at["z"], **common))
    with pytest.raises(ccl.CclError):
        ccl.tensor_status()
    c_call(ccl, "ccl_linear_grad", ccl.LinearGrad(act=ccl.ACT_SILU, dy=dy.data_ptr(), z=z.data_ptr(), dx=at["dx"],
                                                  dw=at["dw"], db=at["db"], **common))
    with pytest.raises(ccl.CclError):
        ccl.tensor_status()
    for name, (whole, lead, size, _) in held.items():
        assert bool((whole[:lead] == 7).all()) and bool((whole[lead + size:] == 7).all()), name
    dz = dy.double() * act_grad64(z.double(), 3)
    for i, a, b in sound:
        s = slice(a, b)
        v = x[s].double() @ w[i].double().T
        slack = product_slack(x[s].double().abs() @ w[i].double().abs().T, k)
        close(held["z"][3][s], v, slack + 2.0 ** -22 * v.abs(), dt)
        close(held["y"][3][s], act64(v, 3), 1.13 * slack + 2.0 ** -15 * v.abs(), dt)
        own = 2.0 ** -14 * (1 + z[s].double().abs()) * dy[s].double().abs()
        slack = (dz[s].abs() + own) @ w[i].double().abs() * (2.0 ** -8 + n * 2.0 ** -23) + own @ w[i].double().abs()
        close(held["dx"][3][s], dz[s] @ w[i].double(), slack, dt)


@pytest.mark.parametrize("lead", [8, 3], ids=["on 16 bytes", "off 16 bytes"])
def test_stacks_of_experts_apart(ccl, lead):
    """Weights, biases and their gradients as slices of larger stacks (row and
    matrix strides that are not packed): the bits of packed ones, and nothing
    written beside the gradients."""
    e, n, k, dt = 4, 136, 72, torch.bfloat16
    offs = offsets_of([70, 0, 33, 150])
    rows = offs[-1]
    g = gen(lead)
    x, dy = rnd(g, rows, k, dtype=dt), rnd(g, rows, n, dtype=dt)
    w = rnd(g, e, n + 5, k + 24, dtype=dt)[:, 2:2 + n, lead:lead + k]
    b = rnd(g, e, n + 16, dtype=dt)[:, lead:lead + n]
    o = torch.tensor(offs, dtype=torch.int32, device="cuda")
    assert torch.equal(ccl.grouped_linear(x, w, o, bias=b, act=ccl.ACT_SILU),
                       ccl.grouped_linear(x, w.contiguous(), o, bias=b.contiguous(), act=ccl.ACT_SILU))
    dx, dw, db = ccl.grouped_linear_backward(dy, x, w, o, bias=True)
    want = ccl.grouped_linear_backward(dy, x, w.contiguous(), o, bias=True)
    assert all(torch.equal(p, q) for p, q in zip((dx, dw, db), want))
    whole = torch.full((e, n + 5, k + 24), 7.0, dtype=dt, device="cuda")
    sums = torch.full((e, n + 16), 7.0, dtype=dt, device="cuda")
    dw, db = whole[:, 2:2 + n, lead:lead + k], sums[:, lead:lead + n]
    c_call(ccl, "ccl_linear_grad", ccl.LinearGrad(
        rows=rows, n=n, k=k, dtype=ccl.BF16, experts=e, dy=dy.data_ptr(), x=x.data_ptr(), offsets=o.data_ptr(),
        dw=dw.data_ptr(), db=db.data_ptr(), lddw=dw.stride(1), dw_stride=dw.stride(0), db_stride=db.stride(0)))
    only = ccl.grouped_linear_backward(dy, x, w, o, bias=True, need_dx=False)
    assert torch.equal(dw, only[1]) and torch.equal(db, only[2])
    dw.fill_(7.0)
    db.fill_(7.0)
    assert bool((whole == 7).all()) and bool((sums == 7).all())


def test_bad_offsets_are_reported_whatever_is_asked(ccl):
    g = gen(14)
    dt = torch.bfloat16
    dy, x, w = rnd(g, 60, 40, dtype=dt), rnd(g, 60, 64, dtype=dt), rnd(g, 3, 40, 64, dtype=dt)
    for offs, sound in (([0, 20, 10, 60], False), ([0, 10, 20, 61], False), ([-5, 10, 20, 60], False), ([3, 3, 20, 59], True)):
        o = torch.tensor(offs, dtype=torch.int32, device="cuda")
        for dx, dw, bias in ((0, 0, 1), (1, 0, 0), (0, 1, 0), (1, 0, 1), (0, 1, 1), (1, 1, 0)):
            ccl.tensor_status()
            ccl.grouped_linear_backward(dy, x, w, o, bias=bool(bias), need_dx=bool(dx), need_dw=bool(dw))
            if sound:
                ccl.tensor_status()
            else:
                with pytest.raises(ccl.CclError, match="offsets"):
                    ccl.tensor_status()

"""Router, order by expert, rows to their experts and back, and layer norm,
against plain implementations in 64 bits.

Tolerances, element by element, from the operations of the formulas: a sum of
terms in 32 bits whose longest chain of additions is d long is within d 2^-24 of
the sum S of absolute values; the exponential is within 2 units (2^-22), a
division, product or sum within 2^-24 of its result; rounding to the output type
adds half a step, eps / 2 of the value (and half of the smallest number of f16,
2^-25)."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

TYPES = [torch.float32, torch.bfloat16, torch.float16]
IDS = ["f32", "bf16", "f16"]
INF = math.inf


@pytest.fixture(scope="module")
def ccl():
    import collective_communication_schedule_gb300 as m
    yield m
    m.tensor_status()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rnd(g, *shape, dtype=torch.float32, scale=1.0):
    return torch.empty(shape, device="cuda", dtype=torch.float32).normal_(0, scale, generator=g).to(dtype)


def close(got, want, slack, dtype=None):
    """|got - want| <= slack + the rounding to `dtype` of what lies within it."""
    dtype = dtype or got.dtype
    tiny = {torch.float16: 2.0 ** -25}.get(dtype, 2.0 ** -134 if dtype == torch.bfloat16 else 2.0 ** -150)
    d = (got.double() - want).abs()
    tol = slack + torch.finfo(dtype).eps / 2 * (want.abs() + slack) + tiny
    assert bool((d <= tol).all()), f"worst {(d / tol).max().item():.3g} of the tolerance, {int((~(d <= tol)).sum())} off"


# ---------------------------------------------------------------- router
def route64(logits, k, score, bias, groups, top, best, renorm, scale=1.0):
    """Choices and weights from the definition, in 64 bits."""
    l = logits.double()
    rows, e = l.shape
    p = torch.sigmoid(l) if score else torch.softmax(torch.where((l == -INF).all(1, keepdim=True), 0.0, l), 1)
    scored = bias is not None or (groups > 1 and best == 2)
    c = p if scored else l
    if bias is not None:
        c = c + bias.double()
    c = torch.where(l == -INF, -INF, c)
    if groups > 1:
        s = c.view(rows, groups, e // groups).sort(2, descending=True).values
        v = s[..., 0]
        if best == 2 and e // groups > 1:
            v = v + torch.where(s[..., 1] == -INF, 0.0, s[..., 1])
        kept = torch.sort(v, dim=1, descending=True, stable=True).indices[:, :top]
        open_ = torch.zeros_like(v, dtype=torch.bool).scatter_(1, kept, True)
        if bias is None:   # scores grow with the logits, though two of 64 bits may round to one value
            c = torch.where(l == -INF, -INF, l)
        c = torch.where(open_.repeat_interleave(e // groups, 1), c, -INF)
    v, at = torch.sort(c, dim=1, descending=True, stable=True)
    chosen = torch.where(v[:, :k] == -INF, -1, at[:, :k])
    return chosen, weights64(l, chosen, score, renorm, scale)


def weights64(l, chosen, score, renorm, scale=1.0):
    on, at = chosen >= 0, chosen.clamp(min=0).long()
    if renorm:         # by differences of logarithms: no sum that underflows
        log = (torch.nn.functional.logsigmoid(l) if score else l).gather(1, at)
        log = torch.where(on, log, -INF)
        top = torch.where(on.any(1, keepdim=True), log.detach().amax(1, keepdim=True), 0.0)
        w = torch.exp(log - top)
        w = w / torch.where(on.any(1, keepdim=True), w.sum(1, keepdim=True), 1.0)
    else:
        dead = (l == -INF).all(1, keepdim=True)
        w = (torch.sigmoid(l) if score else torch.softmax(torch.where(dead, 0.0, l), 1)).gather(1, at)
    return scale * torch.where(on, w, 0.0)


def order64(chosen, e):
    flat = chosen.reshape(-1).long().cpu()
    offsets = [0]
    place = torch.full_like(flat, -1)
    for i in range(e):
        at = (flat == i).nonzero()[:, 0]
        place[at] = torch.arange(offsets[-1], offsets[-1] + len(at))
        offsets.append(offsets[-1] + len(at))
    return torch.tensor(offsets), place.view(chosen.shape)


# scores: exp within 2^-22 and its argument off by 2^-24 |l - max| (here up to 60), sums of up to 37 terms in a
# chain, two divisions: 2^-24 (60 + 8 + 2 * 37 + 4) < 2^-16.7
WEIGHT_TOL = 2.0 ** -16.5


def check_route(ccl, logits, k, score=0, bias=None, groups=1, top=1, best=1, renorm=True, scale=1.0, order=True):
    want, w = route64(logits, k, score, bias, groups, top, best, renorm, scale)
    got = ccl.route(logits, k, score=score, bias=bias, groups=groups, top_groups=top, group_best=best, renormalize=renorm,
                    scale=scale, order=order)
    ccl.tensor_status()
    assert got[1].dtype == torch.int32 and got[0].dtype == torch.float32
    assert torch.equal(got[1].long(), want.long())
    close(got[0], w, WEIGHT_TOL * w.abs() + 2.0 ** -126 * abs(scale))
    if order:
        offsets, place = order64(want, logits.shape[1])
        assert torch.equal(got[2].cpu().long(), offsets) and torch.equal(got[3].cpu().long(), place)
    return got


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("score", [0, 1], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("rows,e,k", [(1, 1, 1), (1, 5, 5), (3, 32, 1), (32, 33, 8), (33, 60, 6), (1, 64, 8), (200, 160, 6),
                                      (1500, 256, 8), (40, 1000, 31), (37, 1024, 32), (2500, 8, 2)])
def test_route(ccl, rows, e, k, score, dtype):
    g = gen(rows + e)
    logits = rnd(g, rows, e, dtype=dtype, scale=2.0)
    bias = rnd(g, e, scale=0.1)
    for renorm in (False, True):
        check_route(ccl, logits, k, score, None, renorm=renorm, scale=1.0 if renorm else 2.5)
        check_route(ccl, logits, k, score, bias, renorm=renorm)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("score", [0, 1], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("rows,e,k,groups,top", [(70, 64, 6, 8, 3), (300, 256, 8, 8, 4), (5, 32, 2, 32, 2), (33, 96, 12, 2, 1),
                                                 (64, 160, 6, 5, 5), (20, 1024, 32, 16, 3), (9, 8, 1, 8, 1)])
def test_route_groups(ccl, rows, e, k, groups, top, score, dtype):
    g = gen(rows + groups)
    logits = rnd(g, rows, e, dtype=dtype, scale=1.5)
    for bias in (None, rnd(g, e, scale=0.05), torch.zeros(e, device="cuda")):
        for best in (1, 2):
            check_route(ccl, logits, k, score, bias, groups, top, best)


def test_route_decides_near_values_in_64_bits(ccl):
    """Biases that bring all scores of a row together to within a rounding of 32 bits, and scores that 32 bits
    round to 1."""
    for seed in range(6):
        g = gen(seed)
        row = rnd(g, 1, 128, scale=1.0)
        for score in (0, 1):
            p = torch.sigmoid(row.double()) if score else torch.softmax(row.double(), 1)
            bias = (0.7 - p[0]).float()
            check_route(ccl, row.repeat(50, 1), 8, score, bias)
            check_route(ccl, row.repeat(3, 1), 32, score, bias)
            check_route(ccl, row, 8, score, bias, groups=8, top=2, best=2)
            check_route(ccl, row, 8, score, bias, groups=4, top=3, best=1)
        flat = 18 + 8 * torch.rand(40, 64, device="cuda", generator=g)
        check_route(ccl, flat, 6, 1, torch.zeros(64, device="cuda"))
        check_route(ccl, flat, 6, 1, None, groups=8, top=4, best=2)


def test_route_groups_by_near_best_values(ccl):
    """Groups whose largest values lie within a rounding of 32 bits of each other and of others of their own."""
    for seed in range(6):
        g = gen(100 + seed)
        for e, groups in ((1024, 2), (1024, 16), (500, 10), (96, 4), (64, 16)):
            flat = 18 + 8 * torch.rand(200, e, device="cuda", generator=g)
            for bias in (torch.zeros(e, device="cuda"), None):
                for best in (1, 2):
                    check_route(ccl, flat, 6, 1, bias, groups, max(1, groups // 4, -(-6 * groups // e)), best)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
def test_route_ties_go_to_the_lower_expert(ccl, dtype):
    g = gen(3)
    logits = torch.randint(-2, 3, (100, 96), device="cuda", generator=g).to(dtype)
    zero = torch.zeros(96, device="cuda")
    for score in (0, 1):
        for bias in (None, zero):
            check_route(ccl, logits, 9, score, bias)
            check_route(ccl, logits, 9, score, bias, groups=8, top=3, best=1)
            check_route(ccl, logits, 9, score, bias, groups=8, top=3, best=2)
    assert torch.equal(ccl.route(torch.zeros(2, 40, device="cuda"), 5)[1].cpu(), torch.arange(5).int().repeat(2, 1))


def test_route_closed_experts(ccl):
    """-Inf closes an expert, a row of them has no choices, and so do closed experts beyond the open ones."""
    g = gen(4)
    for rows in (30, 700):
        logits = rnd(g, rows, 64, scale=1.5)
        logits[torch.rand(rows, 64, device="cuda", generator=g) < 0.5] = -INF
        logits[::7] = -INF
        logits[3, 5:] = -INF
        logits[4, :63] = -INF
        for score in (0, 1):
            for bias in (None, rnd(g, 64, scale=0.1)):
                for groups, top, best in ((1, 1, 1), (8, 3, 1), (8, 3, 2), (32, 9, 2)):
                    for renorm in (True, False):
                        w, chosen, offsets, place = check_route(ccl, logits, 8, score, bias, groups, top, best, renorm)
                        assert bool((chosen[0] == -1).all()) and not w[0].any()
    # a bias of -Inf closes an expert in every row
    bias = torch.zeros(64, device="cuda")
    bias[::2] = -INF
    chosen = ccl.route(rnd(g, 50, 64), 40 - 8, bias=bias)[1]
    assert bool((chosen % 2 == 1).all()) and bool((chosen.sort(1).values == torch.arange(1, 64, 2, device="cuda")).all())


def test_route_keeps_choices_sound_with_nan_and_inf(ccl):
    g = gen(5)
    logits = rnd(g, 40, 32)
    logits[3, 7] = math.nan
    logits[5] = math.nan
    logits[6, 2] = INF
    logits[8, 9], logits[8, 10] = -3.4028234663852886e38, 3.4028234663852886e38
    clean = [i for i in range(40) if i not in (3, 5, 6, 8)]
    for score in (0, 1):
        for bias in (None, rnd(g, 32, scale=0.1)):
            w, chosen, offsets, place = ccl.route(logits, 6, score=score, bias=bias, order=True)
            want, ww = route64(logits[clean], 6, score, bias, 1, 1, 1, True)
            assert torch.equal(chosen[clean].long(), want)
            close(w[clean], ww, WEIGHT_TOL * ww)
            # always distinct experts in range, so that the rows' order stays whole
            assert bool((chosen >= 0).all()) and bool((chosen < 32).all())
            assert bool((chosen.sort(1).values.diff(dim=1) > 0).all())
            assert bool((place.reshape(-1).sort().values == torch.arange(240, device="cuda")).all())
            assert 7 not in chosen[3].tolist() or bias is not None
            assert torch.equal(w[3].isnan(), torch.full((6,), score == 0, device="cuda"))
            assert bool(w[5].isnan().all())
            if bias is None:
                assert chosen[6, 0] == 2 and chosen[8, 0] == 10
    # far below what 32 bits can hold, weights are still shares of the chosen
    low = rnd(g, 20, 16) - 200
    check_route(ccl, low, 4, 1, renorm=True)
    check_route(ccl, low, 4, 0, renorm=True)


@pytest.mark.parametrize("dtype", TYPES[:2], ids=IDS[:2])
@pytest.mark.parametrize("rows,e,k,groups,top", [(11000, 64, 6, 1, 1), (11000, 256, 8, 8, 4), (11000, 384, 3, 1, 1), (6000, 512, 8, 16, 4),
                                                 (6000, 1000, 5, 1, 1)])
def test_route_more_rows_than_warps(ccl, rows, e, k, groups, top, dtype):
    """With the order, a warp takes a second row and more, and its choices count with those of the block."""
    g = gen(rows + e)
    logits = rnd(g, rows, e, dtype=dtype, scale=1.5)
    for score, bias in ((0, None), (1, rnd(g, e, scale=0.05))):
        w, chosen, _, _ = check_route(ccl, logits, k, score, bias, groups, top, min(2, groups))
        alone = ccl.route(logits, k, score=score, bias=bias, groups=groups, top_groups=top, group_best=min(2, groups))
        assert torch.equal(alone[0], w) and torch.equal(alone[1], chosen)


def choices_with_nan(l, k, score, bias, groups, top):
    """Choices in 64 bits by groups of two largest values, a NaN being the lowest finite number, and so a sum below it."""
    low = torch.finfo(torch.float64).min
    l = l.double()
    rows, e = l.shape
    p = torch.sigmoid(l) if score else torch.softmax(l, 1)
    c = p + bias.double() if bias is not None else p
    c = torch.where(l == -INF, -INF, torch.where(c.isnan(), low, c))
    s = c.view(rows, groups, e // groups).sort(2, descending=True).values
    v = s[..., 0] + torch.where(s[..., 1] == -INF, 0.0, s[..., 1])
    v = torch.where(s[..., 0] == -INF, -INF, v.clamp(min=low))
    kept = torch.sort(v, dim=1, descending=True, stable=True).indices[:, :top]
    open_ = torch.zeros_like(v, dtype=torch.bool).scatter_(1, kept, True).repeat_interleave(e // groups, 1)
    if bias is None:
        c = torch.where(l == -INF, -INF, torch.where(l.isnan(), low, l))
    v, at = torch.sort(torch.where(open_, c, -INF), dim=1, descending=True, stable=True)
    return torch.where(v[:, :k] == -INF, -1, at[:, :k])


@pytest.mark.parametrize("score", [0, 1], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("e,groups", [(64, 8), (60, 4), (256, 8), (96, 32), (1024, 16)])
def test_route_groups_of_nan_or_lowest_values_stay_open(ccl, e, groups, score):
    """A group whose two best are NaN, or as low as a type goes, is behind the others but in front of a closed one."""
    g = gen(e)
    size = e // groups
    k = min(4, 2 * size)
    logits = rnd(g, 60, e)
    for row in range(60):
        own = logits[row].view(groups, size)
        if row % 5 == 1:
            own[groups - 1, 0] = math.nan                                  # one: with softmax all scores are NaN
        elif row % 5 == 2:
            own[1:] = math.nan
        elif row % 5 == 3:
            own[1:, 1:] = math.nan                                         # one number a group
        elif row % 5 == 4:
            own[2:] = math.nan                                             # one group of numbers
        own[0] = -INF
        if row % 2:
            own[groups - 1, -1] = -INF
    lowest = torch.full((e,), -3.4028234663852886e38, device="cuda")
    some = rnd(g, e, scale=0.1)
    some[size:2 * size] = lowest[0]
    for bias in (None, rnd(g, e, scale=0.1), some, lowest):
        for top in (1, 2, groups - 1):
            if top * size < k:
                continue
            want = choices_with_nan(logits, k, score, bias, groups, top)
            w, chosen, offsets, place = ccl.route(logits, k, score=score, bias=bias, groups=groups, top_groups=top, group_best=2,
                                                  order=True)
            assert torch.equal(chosen.long(), want)
            assert bool((chosen[chosen >= 0] >= size).all()) and bool((chosen[:, 0] >= 0).all())
            assert bool((w[chosen < 0] == 0).all())
            at, where = order64(want, e)
            assert torch.equal(offsets.cpu().long(), at) and torch.equal(place.cpu().long(), where)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("score", [0, 1], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True], ids=["as they are", "renormalised"])
@pytest.mark.parametrize("rows,e,k", [(1, 1, 1), (9, 33, 5), (65, 64, 8), (300, 256, 8), (17, 1024, 32)])
def test_route_backward(ccl, rows, e, k, renorm, score, dtype):
    """Against the derivative of the 64-bit weights, and against differences of the 64-bit weights along a
    direction.  Every factor of the formulas is within 2^-16.5 as the weights are, and there are at most four of
    them in a term; the terms' absolute values bound their sum."""
    g = gen(rows + k)
    held = rnd(g, rows, e + 3, dtype=dtype, scale=1.5)
    logits = held[:, :e]
    if rows > 8:
        logits[2] = -INF
        logits[3, : e // 2 + 1] = -INF
    chosen = ccl.route(logits, k, score=score)[1]
    dw = rnd(g, rows, k)
    got = ccl.route_backward(dw, logits, chosen, score=score, renormalize=renorm, scale=1.5)
    assert got.dtype == dtype and got.shape == logits.shape
    l = logits.double()
    leaf = l.clone().requires_grad_(True)
    (weights64(leaf, chosen, score, renorm, 1.5) * dw.double()).sum().backward()
    want = leaf.grad.nan_to_num(0) * (l != -INF)
    w = weights64(l, chosen, score, renorm, 1.5)
    most = (dw.double().abs() * w).sum(1, keepdim=True)               # sum of |g| w, with which every weight meets
    at = torch.where(chosen < 0, 0, chosen).long()
    own = torch.zeros_like(l).scatter_add_(1, at, torch.where(chosen < 0, 0.0, dw.double().abs() * w))
    share = torch.zeros_like(l).scatter_add_(1, at, w / 1.5)
    if not score and not renorm:
        dead = (l == -INF).all(1, keepdim=True)
        share = torch.softmax(torch.where(dead, 0.0, l), 1) * ~dead
    close(got, want, 4 * WEIGHT_TOL * (own + share * most) + 1e-30)
    # differences: the 64-bit weights along a direction, (f(+h) - f(-h)) / 2h, off by h^2 times the third derivative
    # (below 8 sum |dw| w |v|^3 for these functions) and by 2^-52 / h of the sum
    v = rnd(g, rows, e).double()
    h = 1e-4
    f = lambda s: (weights64(torch.where(l == -INF, l, l + s * h * v), chosen, score, renorm, 1.5) * dw.double()).sum()  # noqa: E731
    slope, along = (f(1) - f(-1)) / (2 * h), (got.double() * v).sum()
    size = (dw.double().abs() * 1.5).sum()
    rounding = torch.finfo(dtype).eps / 2 * (got.double() * v).abs().sum()
    assert abs(slope - along) <= 8 * h * h * size * 64 + 1e-10 * size + rounding + \
        (4 * WEIGHT_TOL * (own + share * most) * v.abs()).sum()


def test_route_backward_sums_choices_of_one_expert(ccl):
    logits, dw = rnd(gen(6), 5, 16), rnd(gen(7), 5, 4)
    chosen = torch.tensor([[3, 3, 0, -1]] * 5, dtype=torch.int32, device="cuda")
    got = ccl.route_backward(dw, logits, chosen, score=1, renormalize=False)
    s = torch.sigmoid(logits.double())
    want = torch.zeros(5, 16, dtype=torch.float64, device="cuda")
    want[:, 3] = (dw[:, 0] + dw[:, 1]).double()
    want[:, 0] = dw[:, 2].double()
    want *= s * (1 - s)
    close(got, want, 2.0 ** -18 * (want.abs() + 4))
    bad = chosen.clone()
    bad[2, 1] = 16
    ccl.tensor_status()
    out = ccl.route_backward(dw, logits, bad, score=1, renormalize=False)
    with pytest.raises(ccl.CclError, match="expert"):
        ccl.tensor_status()
    assert torch.equal(out[[0, 1, 3, 4]], got[[0, 1, 3, 4]])


@pytest.mark.parametrize("slots,e", [(1, 1), (31, 4), (500, 1024), (2048, 7), (2049, 64), (70001, 256), (400000, 33)])
def test_expert_order(ccl, slots, e):
    g = gen(slots)
    chosen = torch.randint(-1, e, (slots,), device="cuda", generator=g, dtype=torch.int32)
    chosen[slots // 2:slots // 2 + 40] = e - 1                     # a run of one expert
    offsets, place = ccl.expert_order(chosen, e)
    want, at = order64(chosen, e)
    assert torch.equal(offsets.cpu().long(), want) and torch.equal(place.cpu().long(), at)
    ccl.tensor_status()


def test_expert_order_edges(ccl):
    empty = torch.empty(0, 3, dtype=torch.int32, device="cuda")
    offsets, place = ccl.expert_order(empty, 5)
    assert not offsets.any() and offsets.shape == (6,) and place.shape == (0, 3)
    none = torch.full((70, 2), -1, dtype=torch.int32, device="cuda")
    offsets, place = ccl.expert_order(none, 5)
    assert not offsets.any() and bool((place == -1).all())
    for slots in (64, 9000):
        chosen = torch.zeros(slots, dtype=torch.int32, device="cuda")
        chosen[7], chosen[9] = 5, 2 ** 31 - 1
        ccl.tensor_status()
        offsets, place = ccl.expert_order(chosen, 5)
        with pytest.raises(ccl.CclError, match="expert"):
            ccl.tensor_status()
        assert offsets[-1] == slots - 2 and place[7] == -1 and place[9] == -1
        assert bool((place[place >= 0] == torch.arange(slots - 2, device="cuda")).all())
    w, chosen, offsets, place = ccl.route(torch.empty(0, 8, device="cuda"), 2, order=True)
    assert w.shape == (0, 2) and not offsets.any()


# ------------------------------------------------------------- row moves
def some_places(g, rows, k, count, dropped):
    """Distinct places below count (>= rows * k), some choices without one."""
    p = torch.randperm(count, device="cuda", generator=g)[:rows * k].view(rows, k).int()
    return torch.where(torch.rand(rows, k, device="cuda", generator=g) < dropped, -1, p)


def check_moves(ccl, rows, k, h, dtype, dropped=0.2, extra=3, pitch=0, lead=0):
    g = gen(rows * 7 + h)
    count = rows * k + extra
    place = some_places(g, rows, k, count, dropped)

    def mat(n, fill=None):
        held = torch.full((n + 2, h + lead + pitch), 9.0, dtype=dtype, device="cuda")
        view = held[1:-1, lead:lead + h]
        if fill is not None:
            view.copy_(fill)
        return held, view

    x, dy, res = (mat(rows, rnd(g, rows, h))[1] for _ in range(3))
    named = torch.zeros(count, dtype=torch.bool, device="cuda")
    named[place[place >= 0].long()] = True
    tok = torch.zeros(count, dtype=torch.long, device="cuda")
    tok[place[place >= 0].long()] = torch.arange(rows, device="cuda")[:, None].expand(rows, k)[place >= 0]
    # there
    held, out = mat(count)
    assert ccl.dispatch(x, place, out=out) is out
    assert torch.equal(out[named], x[tok[named]]) and bool((out[~named] == 9).all())
    out[~named] = math.nan                               # what no place names is not read
    mask = torch.ones_like(held, dtype=torch.bool)
    mask[1:-1, lead:lead + h] = False
    assert bool((held[mask] == 9).all())
    # and back
    r = mat(count, rnd(g, count, h))[1]
    r[~named] = math.nan
    weights = rnd(g, rows, k)
    live = (place >= 0)[..., None]
    rr = torch.where(live, r.double()[place.clamp(min=0).long()], 0.0)
    for w, s in ((weights, res), (weights, None), (None, res), (None, None)):
        held, y = mat(rows)
        ccl.combine(r, place, w, residual=s, out=y)
        ww = w.double()[..., None] if w is not None else 1.0
        want = (ww * rr).sum(1) + (s.double() if s is not None else 0)
        size = (ww * rr).abs().sum(1) + (s.double().abs() if s is not None else 0)
        close(y, want, (k + 1) * 2.0 ** -24 * size)
        mask = torch.ones_like(held, dtype=torch.bool)
        mask[1:-1, lead:lead + h] = False
        assert bool((held[mask] == 9).all())
    got = ccl.dispatch_backward(r, place)
    close(got, rr.sum(1), k * 2.0 ** -24 * rr.abs().sum(1))
    # gradients: a chain of at most h / 32 products a lane, then 5 additions
    held, dr = mat(count)
    out, dw = ccl.combine_backward(dy, r, place, weights, out=dr)
    want = torch.full((count, h), 9.0, dtype=torch.float64, device="cuda")
    at = place[place >= 0].long()
    want[at] = (weights.double()[..., None] * dy.double()[:, None])[place >= 0]
    close(dr, want, 2.0 ** -24 * want.abs())
    assert bool((dr[~named] == 9).all()) and out is dr
    terms = rr * dy.double()[:, None]
    close(dw, terms.sum(2), (h / 32 + 8) * 2.0 ** -24 * terms.abs().sum(2))
    assert not dw[place < 0].any()
    only = ccl.combine_backward(dy, r, place, weights, need_dr=False)
    assert only[0] is None and torch.equal(only[1], dw)
    only = ccl.combine_backward(dy, r, place, None, need_dweights=False)
    assert only[1] is None and torch.equal(only[0][at], dy[tok[at]])
    ccl.tensor_status()


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("rows,k,h", [(1, 1, 1), (1, 8, 2048), (3, 2, 7), (24, 8, 520), (33, 32, 65), (200, 4, 1032),
                                      (513, 6, 256), (70, 1, 8192), (1000, 3, 130)])
def test_rows_there_and_back(ccl, rows, k, h, dtype):
    check_moves(ccl, rows, k, h, dtype)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("lead,pitch", [(0, 8), (8, 8), (1, 0), (3, 5)])
def test_rows_of_any_stride(ccl, lead, pitch, dtype):
    check_moves(ccl, 50, 3, 264, dtype, lead=lead, pitch=pitch)


def check_many_choices(ccl, rows, k, h, dtype, lead=0, pitch=0):
    """Gradients of more choices of short rows than are taken a warp each.  A lane has 8 products at most, then up to 5
    additions over the lanes of a row."""
    g = gen(rows + h)
    count = rows * k + 5
    place = some_places(g, rows, k, count, 0.2)
    dy = rnd(g, rows, h + lead + pitch, dtype=dtype)[:, lead:lead + h]
    r = rnd(g, count, h + lead + pitch, dtype=dtype)[:, lead:lead + h]
    live = place >= 0
    at = place[live].long()
    named = torch.zeros(count, dtype=torch.bool, device="cuda")
    named[at] = True
    r[~named] = math.nan
    weights = rnd(g, rows, k)
    held = torch.full((count + 2, h + lead + pitch), 9.0, dtype=dtype, device="cuda")
    dr = held[1:-1, lead:lead + h]
    out, dw = ccl.combine_backward(dy, r, place, weights, out=dr)
    assert out is dr
    want = torch.full((count, h), 9.0, dtype=torch.float64, device="cuda")
    want[at] = (weights.double()[..., None] * dy.double()[:, None])[live]
    close(dr, want, 2.0 ** -24 * want.abs())
    assert bool((dr[~named] == 9).all())
    terms = torch.where(live[..., None], r.double()[place.clamp(min=0).long()], 0.0) * dy.double()[:, None]
    close(dw, terms.sum(2), 13 * 2.0 ** -24 * terms.abs().sum(2))
    assert not dw[~live].any()
    only = ccl.combine_backward(dy, r, place, weights, need_dr=False)
    assert only[0] is None and torch.equal(only[1], dw)
    only = ccl.combine_backward(dy, r, place, None, need_dweights=False)
    assert only[1] is None and torch.equal(only[0][at], dy[:, None].expand(rows, k, h)[live])
    only = ccl.combine_backward(dy, r, place, weights, need_dweights=False)
    assert only[1] is None and torch.equal(only[0][at], dr[at])
    dr.fill_(9)
    assert bool((held == 9).all())
    ccl.tensor_status()
    # places out of range do as much as none, and are reported
    bad, none = place.clone(), place.clone()
    for t, j, p in ((0, 0, count), (rows // 2, k - 1, 2 ** 31 - 1), (rows - 1, k - 1, count + 1)):
        bad[t, j], none[t, j] = p, -1
    want = ccl.combine_backward(dy, r, none, weights, out=torch.full_like(want, 9.0, dtype=dtype))
    ccl.tensor_status()
    got = ccl.combine_backward(dy, r, bad, weights, out=dr)
    with pytest.raises(ccl.CclError, match="place"):
        ccl.tensor_status()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("rows,k,h", [(2731, 7, 8), (5501, 3, 24), (16387, 1, 40), (1030, 16, 128), (2731, 7, 128), (520, 32, 256),
                                      (5501, 3, 256), (2731, 7, 136)])
def test_gradients_of_many_short_rows(ccl, rows, k, h, dtype):
    """1 to 32 lanes a row, some of them beyond its end, and last groups of one to four choices."""
    if h * torch.finfo(dtype).bits // 8 > 512:
        h = 128
    check_many_choices(ccl, rows, k, h, dtype)


@pytest.mark.parametrize("dtype", TYPES, ids=IDS)
@pytest.mark.parametrize("lead,pitch", [(0, 8), (8, 8), (1, 0), (3, 5)])
def test_gradients_of_many_short_rows_of_any_stride(ccl, lead, pitch, dtype):
    check_many_choices(ccl, 2731, 7, 72, dtype, lead, pitch)


def test_moves_without_places_or_rows(ccl):
    x = rnd(gen(1), 6, 40, dtype=torch.bfloat16)
    none = torch.full((6, 2), -1, dtype=torch.int32, device="cuda")
    out = torch.full((12, 40), 3.0, dtype=torch.bfloat16, device="cuda")
    ccl.dispatch(x, none, out=out)
    assert bool((out == 3).all())
    assert not ccl.combine(out, none).any() and torch.equal(ccl.combine(out, none, residual=x), x)
    assert torch.equal(ccl.combine(out[:0], none, residual=x), x)
    dr, dw = ccl.combine_backward(x, out, none, torch.ones(6, 2, device="cuda"))
    assert not dw.any()
    empty = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    assert ccl.dispatch(x[:0], empty).shape == (0, 40) and ccl.combine(out, empty).shape == (0, 40)


def test_shapes_that_disagree_are_refused(ccl):
    x = torch.zeros(4, 8, device="cuda")
    i, w = torch.zeros(4, 2, device="cuda", dtype=torch.int32), torch.zeros(4, 2, device="cuda")
    for place in (i[0, 0], i[0], i[:3], i[None], i.long(), i.t().contiguous().t(), i.cpu()):
        for call in (lambda: ccl.dispatch(x, place), lambda: ccl.combine_backward(x, x, place, w), lambda: ccl.combine(x, place, w)):
            with pytest.raises(ValueError):
                call()
    for call in (lambda: ccl.combine(x, i, w, out=x[:, :7]), lambda: ccl.combine(x, i, w, residual=x[:3]),
                 lambda: ccl.combine(x, i, w.t().contiguous().t()), lambda: ccl.dispatch(x, i, out=x[:, :7]),
                 lambda: ccl.route_backward(w[:3], x, i), lambda: ccl.layer_norm(x, w[0]), lambda: ccl.layer_norm(x, out=x[:3]),
                 lambda: ccl.layer_norm_backward(x, x, None, w[:, 0], w[:, 0]), lambda: ccl.route(x, 2, bias=w[0])):
        with pytest.raises(ValueError):
            call()


def test_residual_in_place(ccl):
    g = gen(2)
    r, res = rnd(g, 60, 264, dtype=torch.bfloat16), rnd(g, 20, 264, dtype=torch.bfloat16)
    place = some_places(g, 20, 3, 60, 0.1)
    want = ccl.combine(r, place, residual=res)
    assert ccl.combine(r, place, residual=res, out=res) is res and torch.equal(res, want)


def test_places_beyond_the_rows_are_passed_over_and_reported(ccl):
    g = gen(3)
    x, r = rnd(g, 9, 72, dtype=torch.float16), rnd(g, 18, 72, dtype=torch.float16)
    good = some_places(g, 9, 2, 18, 0.0)
    bad, none = good.clone(), good.clone()
    bad[4, 1], bad[8, 0] = 18, 2 ** 31 - 1
    none[4, 1], none[8, 0] = -1, -2 ** 31
    w = rnd(g, 9, 2)
    held = torch.full((3, 18, 72), 5.0, dtype=torch.float16, device="cuda")
    for call in (lambda p: ccl.dispatch(x, p, out=held[1].fill_(5)), lambda p: ccl.combine(r, p, w),
                 lambda p: ccl.combine_backward(x, r, p, w, out=held[1].fill_(5))):
        ccl.tensor_status()
        want = call(none)
        want = [t.clone() for t in (want if isinstance(want, tuple) else (want,))]
        ccl.tensor_status()
        got = call(bad)
        with pytest.raises(ccl.CclError, match="place"):
            ccl.tensor_status()
        assert all(torch.equal(a, b) for a, b in zip(got if isinstance(got, tuple) else (got,), want))
        assert bool((held[0] == 5).all()) and bool((held[2] == 5).all())
    for call in (lambda p: ccl.dispatch(x, p, out=held[1, :0]), lambda p: ccl.combine(r[:0], p, w),
                 lambda p: ccl.combine_backward(x, r[:0], p, w)):       # no rows to place them in at all
        call(torch.full_like(good, -1))
        ccl.tensor_status()
        call(torch.zeros_like(good))
        with pytest.raises(ccl.CclError, match="place"):
            ccl.tensor_status()
    ccl.tensor_status()


def test_rows_past_32_bits(ccl):
    """Places whose rows begin beyond 2^31 elements (and 2^32 bytes)."""
    h, count = 4104, 600000                                              # 2.5e9 elements, 4.9 GB
    r = torch.empty(count, h, dtype=torch.bfloat16, device="cuda")
    place = torch.tensor([[count - 1, 0], [count - 2, 523300], [5, count - 3]], dtype=torch.int32, device="cuda")
    g = gen(4)
    x, w = rnd(g, 3, h, dtype=torch.bfloat16), rnd(g, 3, 2)
    ccl.dispatch(x, place, out=r)
    for t in range(3):
        for j in range(2):
            assert torch.equal(r[place[t, j].item()], x[t])
    y = ccl.combine(r, place, w)
    want = w.double().sum(1, keepdim=True) * x.double()
    close(y, want, 3 * 2.0 ** -24 * w.double().abs().sum(1, keepdim=True) * x.double().abs())
    dr, dw = ccl.combine_backward(x, r, place, w)
    assert torch.equal(dr[count - 1], (w[0, 0] * x[0].float()).to(torch.bfloat16))
    close(dw, (x.double() ** 2).sum(1, keepdim=True).expand(3, 2), (h / 32 + 8) * 2.0 ** -24 * h * 4)
    ccl.tensor_status()


# ------------------------------------------------------------------ norm
NORM_TYPES = [(torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
              (torch.float16, torch.float16), (torch.float16, torch.float32)]
NORM_IDS = ["f32", "bf16", "bf16+f32", "f16", "f16+f32"]


def chain(n):
    """The longest chain of additions of a row's sum: at most 32 in a thread (n / 1024 in long rows), 5 in the warp,
    32 over the warps."""
    return max(32, n / 1024 + 1) + 5 + 32


def norm64(x, w, b, eps):
    x = x.double()
    mean = x.mean(1, keepdim=True)
    rstd = (x.var(1, unbiased=False, keepdim=True) + eps) ** -0.5
    xh = (x - mean) * rstd
    return mean, rstd, xh, xh * (w.double() if w is not None else 1) + (b.double() if b is not None else 0)


def check_norm(ccl, x, w, b, eps=1e-5):
    mean, rstd, xh, want = norm64(x, w, b, eps)
    y, m, r = ccl.layer_norm(x, w, b, eps=eps, stats=True)
    d, n = chain(x.shape[1]) * 2.0 ** -24, x.shape[1]
    xa = x.double().abs()
    em = (d + 2.0 ** -23) * xa.mean(1, keepdim=True)                      # the mean
    close(m[:, None], mean, em)
    # the variance: each difference off by em + 2^-24 of it, their squares' sum by its chain; em^2 for the shift
    dx = (x.double() - mean).abs()
    ev = (2 * dx * (em + 2.0 ** -24 * dx)).mean(1, keepdim=True) + em ** 2 + (d + 2.0 ** -22) * (dx ** 2).mean(1, keepdim=True)
    er = 0.5 * ev * rstd ** 3 + 2.0 ** -22 * rstd
    close(r[:, None], rstd, 1.1 * er)
    wa = w.double().abs() if w is not None else 1.0
    slack = wa * (rstd * (em + 2.0 ** -24 * xa) + 1.1 * er * dx) + 2.0 ** -22 * (wa * xh.abs() + want.abs())
    close(y, want, slack)
    assert torch.equal(ccl.layer_norm(x, w, b, eps=eps), y)
    return y, m, r


@pytest.mark.parametrize("t,tw", NORM_TYPES, ids=NORM_IDS)
@pytest.mark.parametrize("rows,n", [(1, 1), (2, 7), (5, 64), (33, 255), (3, 256), (4, 512), (130, 1000), (7, 1032), (65, 2057),
                                    (3, 4096), (2, 4104), (5, 8192), (2, 9001), (3, 16384), (2, 16392), (2, 40001)])
def test_layer_norm(ccl, rows, n, t, tw):
    g = gen(rows + n)
    x = rnd(g, rows, n, dtype=t) + rnd(g, rows, 1, dtype=t)
    w, b = rnd(g, n, dtype=tw), rnd(g, n, dtype=tw)
    check_norm(ccl, x, w, b)
    check_norm(ccl, x, w, None)
    check_norm(ccl, x, None, None, eps=0.5)


def test_layer_norm_of_rows_far_from_zero(ccl):
    """The variance is summed over differences from the mean: a mean 1e4 times the spread costs no more than its
    own rounding."""
    g = gen(1)
    for n in (300, 4096, 20000):
        x = rnd(g, 6, n) + 1e4
        check_norm(ccl, x, None, None)
        x[2] = 3.0                                                        # a row without spread
        y, m, r = check_norm(ccl, x, None, None)
        assert not y[2].any() and m[2] == 3


@pytest.mark.parametrize("t", TYPES, ids=IDS)
def test_layer_norm_strides_and_in_place(ccl, t):
    g = gen(2)
    for n, lead, pitch in ((264, 8, 8), (264, 1, 0), (257, 0, 3), (2048, 0, 16)):
        held = torch.full((22, n + lead + pitch), 7.0, dtype=t, device="cuda")
        x = held[1:-1, lead:lead + n]
        x.copy_(rnd(g, 20, n))
        w, b = rnd(g, n, dtype=t), rnd(g, n, dtype=t)
        want = ccl.layer_norm(x.contiguous(), w, b)
        check_norm(ccl, x, w, b)
        if lead % 8 == 0 and pitch % 8 == 0:
            assert torch.equal(ccl.layer_norm(x, w, b), want)
        # (weights off 16 bytes take the way of single elements)
        wide = torch.empty(n + 1, dtype=t, device="cuda")[1:]
        wide.copy_(w)
        check_norm(ccl, x, wide, b)
        want = ccl.layer_norm(x, w, b)
        ccl.layer_norm(x, w, b, out=x)
        assert torch.equal(x, want)
        x.fill_(7.0)
        assert bool((held == 7).all())


SHIFTED = [(15000, 131), (15000, 517), (3700, 2057), (1900, 4097), (1400, 9001)]


@pytest.mark.parametrize("t,tw", NORM_TYPES[1:], ids=NORM_IDS[1:])
@pytest.mark.parametrize("rows,n", SHIFTED)
def test_layer_norm_of_more_rows_off_16_bytes_than_are_taken_at_once(ccl, rows, n, t, tw):
    """Three turns of every group of threads, each with another distance to 16 bytes, y at the distance of x or not."""
    g = gen(n)
    x = rnd(g, rows, n, dtype=t) + rnd(g, rows, 1, dtype=t)
    w, b = rnd(g, n, dtype=tw), rnd(g, n, dtype=tw)
    y = check_norm(ccl, x, w, b)[0]
    for lead, pitch in ((1, 0), (0, 4), (5, 3)):
        held = torch.full((rows + 2, n + lead + pitch), 7.0, dtype=t, device="cuda")
        out = held[1:-1, lead:lead + n]
        assert ccl.layer_norm(x, w, b, out=out) is out and torch.equal(out, y)
        out.copy_(x)
        want = check_norm(ccl, out, w, b)[0]
        ccl.layer_norm(out, w, b, out=out)
        assert torch.equal(out, want)
        out.fill_(7.0)
        assert bool((held == 7).all())


def check_norm_grad(ccl, dy, x, w, mean, rstd, tw, bias=True):
    rows, n = x.shape
    got = ccl.layer_norm_backward(dy, x, w, mean, rstd, bias=bias)
    m, r, g0 = mean.double()[:, None], rstd.double()[:, None], dy.double()
    xh = (x.double() - m) * r
    g = g0 * (w.double() if w is not None else 1)
    a, b = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    want = r * (g - a - xh * b)
    d = chain(n) * 2.0 ** -24
    ea = (d + 2.0 ** -23) * g.abs().mean(1, keepdim=True)
    eb = (d + 2.0 ** -21) * (g * xh).abs().mean(1, keepdim=True)
    close(got[0], want, r * (ea + xh.abs() * eb + 2.0 ** -21 * (g.abs() + a.abs() + (xh * b).abs())))
    # a sum over rows in any order
    s = (rows + 8) * 2.0 ** -24
    terms = g0 * xh
    close(got[1], terms.sum(0), (s + 2.0 ** -21) * terms.abs().sum(0), tw)
    if bias:
        close(got[2], g0.sum(0), s * g0.abs().sum(0), tw)
    assert got[1].dtype == tw
    return got


@pytest.mark.parametrize("t,tw", NORM_TYPES, ids=NORM_IDS)
@pytest.mark.parametrize("rows,n", [(1, 1), (2, 7), (700, 64), (33, 255), (9, 256), (300, 1000), (7, 1032), (65, 2057),
                                    (900, 4096), (2, 8192), (3, 9001), (5, 16384), (2, 16392), (40, 20001)])
def test_layer_norm_backward(ccl, rows, n, t, tw):
    g = gen(rows + n)
    x, dy, w = rnd(g, rows, n, dtype=t), rnd(g, rows, n, dtype=t), rnd(g, n, dtype=tw)
    mean, rstd, _, _ = norm64(x, w, None, 1e-5)
    mean, rstd = mean[:, 0].float(), rstd[:, 0].float()
    got = check_norm_grad(ccl, dy, x, w, mean, rstd, tw)
    check_norm_grad(ccl, dy, x, None, mean, rstd, t)
    again = ccl.layer_norm_backward(dy, x, w, mean, rstd, bias=False)
    assert torch.equal(again[0], got[0]) and torch.equal(again[1], got[1]) and again[2] is None
    only = ccl.layer_norm_backward(dy, x, w, mean, rstd, bias=True, need_dx=False, need_dw=False)
    assert only[0] is None and only[1] is None and torch.equal(only[2], got[2])
    alone = ccl.layer_norm_backward(dy, x, w, mean, rstd, need_dw=False)
    assert torch.equal(alone[0], got[0]) and alone[1] is None


@pytest.mark.parametrize("t,tw", NORM_TYPES, ids=NORM_IDS)
@pytest.mark.parametrize("rows,n", [(15000, 64), (15000, 131), (3700, 517), (3700, 1000), (1900, 1101), (1900, 2000),
                                    (1000, 2057), (500, 4097), (470, 7001), (470, 8192), (470, 12288), (470, 16384)])
def test_layer_norm_backward_of_more_rows_than_are_taken_at_once(ccl, rows, n, t, tw):
    """Three turns and a part of one of every group of threads, by elements and by 16 bytes."""
    g = gen(n)
    for lead in (0, 3) if n % 8 == 0 and n < 5000 else (0,):
        x, dy = (rnd(g, rows, n + lead, dtype=t)[:, lead:] for _ in range(2))
        w = rnd(g, n, dtype=tw)
        mean, rstd, _, _ = norm64(x, w, None, 1e-5)
        mean, rstd = mean[:, 0].float(), rstd[:, 0].float()
        got = check_norm_grad(ccl, dy, x, w, mean, rstd, tw)
        alone = ccl.layer_norm_backward(dy, x, w, mean, rstd, need_dw=False)
        assert torch.equal(alone[0], got[0])
        sums = ccl.layer_norm_backward(dy, x, w, mean, rstd, bias=True, need_dx=False)
        assert torch.equal(sums[1], got[1]) and torch.equal(sums[2], got[2])


def test_layer_norm_backward_of_views(ccl):
    g = gen(5)
    for t in TYPES:
        for n, lead in ((264, 8), (264, 3), (131, 1)):
            x, dy = (rnd(g, 30, n + 16, dtype=t)[:, lead:lead + n] for _ in range(2))
            w = rnd(g, n, dtype=t)
            mean, rstd, _, _ = norm64(x, w, None, 1e-5)
            check_norm_grad(ccl, dy, x, w, mean[:, 0].float(), rstd[:, 0].float(), t)


def test_layer_norm_backward_against_differences(ccl):
    """The loss sum(dy * y) in 64 bits along random directions of x, w and b: the difference (f(+h) - f(-h)) / 2h is
    off by about h^2 of the size; the gradients are f32, the slope of dx is checked through the statistics too."""
    g = gen(6)
    x, dy, w, b = rnd(g, 12, 96), rnd(g, 12, 96), rnd(g, 96), rnd(g, 96)
    _, m, r = ccl.layer_norm(x, w, b, stats=True)
    dx, dw, db = ccl.layer_norm_backward(dy, x, w, m, r, bias=True)
    f = lambda x, w, b: (norm64(x, w, b, 1e-5)[3] * dy.double()).sum()  # noqa: E731
    h = 1e-4
    for which, grad in enumerate((dx, dw, db)):
        v = [torch.zeros_like(t).double() for t in (x, w, b)]
        v[which] = rnd(g, *grad.shape).double()
        at = lambda s: f(*(t.double() + s * h * d for t, d in zip((x, w, b), v)))  # noqa: E731
        slope, along = (at(1) - at(-1)) / (2 * h), (grad.double() * v[which]).sum()
        # 96 x 12 terms of size about 1: rounding of the gradients 2^-20 each, h^2 times third derivatives of about 50
        assert abs(slope - along) <= 96 * 12 * (2.0 ** -20 + 50 * h * h)


def test_layer_norm_without_rows(ccl):
    x = torch.empty(0, 40, device="cuda")
    w = torch.ones(40, device="cuda")
    y, m, r = ccl.layer_norm(x, w, w, stats=True)
    assert y.shape == (0, 40) and m.shape == (0,)
    dx, dw, db = ccl.layer_norm_backward(x, x, w, m, r, bias=True)
    assert dx.shape == (0, 40) and not dw.any() and not db.any()


def test_layer_norm_past_32_bits(ccl):
    n, rows = 4104, 600000
    x = torch.zeros(rows, n, dtype=torch.bfloat16, device="cuda")
    last = rnd(gen(7), 3, n, dtype=torch.bfloat16)
    x[-3:] = last
    y, m, r = ccl.layer_norm(x, stats=True, out=torch.empty_like(x))
    want, wm, wr = ccl.layer_norm(last, stats=True)
    assert torch.equal(y[-3:], want) and torch.equal(m[-3:], wm) and not y[:-3:1000].any()
    dx, dw, db = ccl.layer_norm_backward(y, x, None, m, r, bias=True)
    wdx = ccl.layer_norm_backward(want, last, None, wm, wr)[0]
    assert torch.equal(dx[-3:], wdx)


# ----------------------------------------------------- streams and graphs
def everything(ccl, t, stream=None):
    kw = {} if stream is None else {"stream": stream}
    w, chosen, offsets, place = ccl.route(t["logits"], 4, score=1, bias=t["bias"], groups=8, top_groups=4, group_best=2,
                                          order=True, **kw)
    o2, p2 = ccl.expert_order(chosen, 64, **kw)
    y, m, r = ccl.layer_norm(t["x"], t["w"], t["w"], stats=True, **kw)
    rows = ccl.dispatch(y, place, **kw)
    z = ccl.combine(rows, place, w, residual=t["x"], **kw)
    dr, dw = ccl.combine_backward(t["x"], rows, place, w, **kw)
    dl = ccl.route_backward(dw, t["logits"], chosen, score=1, **kw)
    dy = ccl.dispatch_backward(dr, place, **kw)
    dx, dg, db = ccl.layer_norm_backward(dy, t["x"], t["w"], m, r, bias=True, **kw)
    return [w, chosen, offsets, place, o2, p2, y, m, r, rows, z, dr, dw, dl, dy, dx, dg, db]


@pytest.mark.parametrize("rows", [20, 700])
def test_results_repeat_bit_for_bit_on_other_streams_and_in_graphs(ccl, rows):
    g = gen(rows)
    make = lambda: {"logits": rnd(g, rows, 64), "bias": rnd(g, 64, scale=0.1), "x": rnd(g, rows, 264, dtype=torch.bfloat16),  # noqa: E731
                    "w": rnd(g, 264, dtype=torch.bfloat16)}
    a, b = make(), make()
    want, other = everything(ccl, a), everything(ccl, b)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = everything(ccl, a, stream=s)
    with torch.cuda.stream(s):
        more = everything(ccl, a)
    s.synchronize()
    for p, q, u in zip(got, more, want):
        assert torch.equal(p, u) and torch.equal(q, u)
    # two captured graphs over inputs that change, replayed in turn
    ins = [{n: t.clone() for n, t in a.items()} for _ in range(2)]
    graphs, outs = [], []
    for held in ins:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(everything(ccl, held))
        graphs.append(graph)
    for n in a:
        ins[1][n].copy_(b[n])
    for _ in range(2):
        graphs[0].replay()
        graphs[1].replay()
    torch.cuda.synchronize()
    for p, q, u, v in zip(outs[0], outs[1], want, other):
        assert torch.equal(p, u) and torch.equal(q, v)
    ccl.tensor_status()

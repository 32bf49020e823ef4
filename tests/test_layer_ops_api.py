"""Refusals, workspace sizes and struct layouts of the router, the row moves, the
norm and the cross entropy (no GPU needed: arguments are checked before any device is touched)."""
import ctypes
import os
import shutil
import subprocess

import pytest

import collective_communication_schedule_gb300 as ccl

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 20                # stands for device addresses: never read here
INVALID, UNSUPPORTED = 1, 5


def maker(cls, **base):
    def make(**kw):
        a = cls(**base)
        for k, v in kw.items():
            setattr(a, k, v)
        return a
    return make


route = maker(ccl.Route, rows=40, experts=16, k=4, dtype=ccl.F32, score=0, scale=1.0, logits=A, weights=2 * A, chosen=3 * A)
route_grad = maker(ccl.RouteGrad, rows=4, experts=16, k=4, dtype=ccl.F32, scale=1.0, logits=A, chosen=2 * A, dweights=3 * A,
                   dlogits=4 * A)
order = maker(ccl.ExpertOrder, slots=100000, experts=16, chosen=A, offsets=2 * A, place=3 * A)
dispatch = maker(ccl.Dispatch, rows=4, count=8, h=32, k=2, dtype=ccl.BF16, x=A, place=2 * A, out=3 * A)
combine = maker(ccl.Combine, rows=4, count=8, h=32, k=2, dtype=ccl.BF16, r=A, place=2 * A, weights=3 * A, y=4 * A)
combine_grad = maker(ccl.CombineGrad, rows=4, count=8, h=32, k=2, dtype=ccl.F16, dy=A, r=2 * A, place=3 * A, weights=4 * A,
                     dr=5 * A, dweights=6 * A)
norm = maker(ccl.LayerNorm, rows=4, n=32, dtype=ccl.BF16, wdtype=ccl.F32, eps=1e-5, x=A, w=2 * A, b=3 * A, y=4 * A)
norm_grad = maker(ccl.LayerNormGrad, rows=4, n=32, dtype=ccl.BF16, wdtype=ccl.BF16, dy=A, x=2 * A, w=3 * A, mean=4 * A,
                  rstd=5 * A, dx=6 * A, dw=7 * A, db=8 * A)
ce = maker(ccl.CrossEntropy, rows=40, vocab=100, k=32, dtype=ccl.BF16, target_bits=64, ignore_index=-100, x=A, w=2 * A,
           target=3 * A, loss=4 * A, lse=5 * A)
ce_grad = maker(ccl.CrossEntropyGrad, rows=40, vocab=100, k=32, dtype=ccl.F16, target_bits=32, ignore_index=-100, x=A, w=2 * A,
                target=3 * A, dloss=4 * A, lse=5 * A, dx=6 * A, dw=7 * A)
WITH_WORKSPACE = {"ccl_route", "ccl_expert_order", "ccl_layer_norm_grad", "ccl_cross_entropy", "ccl_cross_entropy_grad"}


def code(name, a, ws=64 * A, size=1 << 40):
    fn = getattr(ccl.lib, name)
    return fn(ctypes.byref(a), ws, size, None) if name in WITH_WORKSPACE else fn(ctypes.byref(a), None)


REFUSED = [
    ("ccl_route", route(dtype=ccl.I32), UNSUPPORTED, "f32, bf16 and f16"),
    ("ccl_route", route(experts=0), INVALID, "experts"),
    ("ccl_route", route(experts=1025), INVALID, "experts"),
    ("ccl_route", route(k=0), INVALID, "choices"),
    ("ccl_route", route(k=17), INVALID, "choices"),
    ("ccl_route", route(experts=64, k=33), INVALID, "choices"),
    ("ccl_route", route(rows=-1), INVALID, "rows"),
    ("ccl_route", route(rows=1 << 30), INVALID, "rows"),
    ("ccl_route", route(score=2), INVALID, "score"),
    ("ccl_route", route(groups=3, top_groups=1, group_best=1), INVALID, "groups"),
    ("ccl_route", route(groups=33, experts=66, top_groups=20, group_best=1), INVALID, "groups"),
    ("ccl_route", route(groups=-1), INVALID, "groups"),
    ("ccl_route", route(groups=4, top_groups=5, group_best=1), INVALID, "top_groups"),
    ("ccl_route", route(groups=4, top_groups=0, group_best=1), INVALID, "top_groups"),
    ("ccl_route", route(groups=4, top_groups=2, group_best=3), INVALID, "group_best"),
    ("ccl_route", route(groups=8, top_groups=1, group_best=1), INVALID, "more choices"),
    ("ccl_route", route(ld=15), INVALID, "logits stride"),
    ("ccl_route", route(logits=None), INVALID, "logits is null"),
    ("ccl_route", route(logits=A + 2), INVALID, "not aligned"),
    ("ccl_route", route(offsets=5 * A), INVALID, "together"),
    ("ccl_route", route(place=5 * A), INVALID, "together"),
    ("ccl_route", route(weights=A), INVALID, "also"),
    ("ccl_route", route(chosen=2 * A), INVALID, "also"),
    ("ccl_route", route(place=3 * A, offsets=4 * A), INVALID, "also"),
    ("ccl_route_grad", route_grad(k=17), INVALID, "choices"),
    ("ccl_route_grad", route_grad(chosen=None), INVALID, "chosen is null"),
    ("ccl_route_grad", route_grad(ldd=8), INVALID, "dlogits stride"),
    ("ccl_route_grad", route_grad(dlogits=A), INVALID, "also"),
    ("ccl_expert_order", order(experts=0), INVALID, "experts"),
    ("ccl_expert_order", order(slots=1 << 31), INVALID, "slots"),
    ("ccl_expert_order", order(place=A), INVALID, "also"),
    ("ccl_expert_order", order(offsets=None), INVALID, "offsets is null"),
    ("ccl_dispatch", dispatch(dtype=ccl.I32), UNSUPPORTED, "f32, bf16 and f16"),
    ("ccl_dispatch", dispatch(k=0), INVALID, "choices"),
    ("ccl_dispatch", dispatch(h=0), INVALID, "sizes"),
    ("ccl_dispatch", dispatch(count=1 << 31), INVALID, "sizes"),
    ("ccl_dispatch", dispatch(rows=1 << 31), INVALID, "sizes"),
    ("ccl_dispatch", dispatch(ldo=31), INVALID, "out stride"),
    ("ccl_dispatch", dispatch(place=None), INVALID, "place is null"),
    ("ccl_dispatch", dispatch(x=A + 1), INVALID, "not aligned"),
    ("ccl_dispatch", dispatch(out=A), INVALID, "also"),
    ("ccl_combine", combine(y=A), INVALID, "also"),
    ("ccl_combine", combine(residual=4 * A, lds=40), INVALID, "stride"),
    ("ccl_combine", combine(weights=3 * A + 2), INVALID, "not aligned"),
    ("ccl_combine", combine(ldr=8), INVALID, "r stride"),
    ("ccl_combine_grad", combine_grad(dr=A), INVALID, "also"),
    ("ccl_combine_grad", combine_grad(dr=2 * A), INVALID, "also"),
    ("ccl_combine_grad", combine_grad(dweights=4 * A), INVALID, "also"),
    ("ccl_combine_grad", combine_grad(r=None), INVALID, "r is null"),
    ("ccl_layer_norm", norm(dtype=ccl.I32), UNSUPPORTED, "f32, bf16 and f16"),
    ("ccl_layer_norm", norm(wdtype=ccl.F16), UNSUPPORTED, "type of x"),
    ("ccl_layer_norm", norm(n=0), INVALID, "sizes"),
    ("ccl_layer_norm", norm(n=(1 << 24) + 1), INVALID, "sizes"),
    ("ccl_layer_norm", norm(eps=-1.0), INVALID, "eps"),
    ("ccl_layer_norm", norm(eps=float("nan")), INVALID, "eps"),
    ("ccl_layer_norm", norm(ldx=31), INVALID, "x stride"),
    ("ccl_layer_norm", norm(y=2 * A), INVALID, "also"),
    ("ccl_layer_norm", norm(y=A, ldy=40), INVALID, "stride"),
    ("ccl_layer_norm", norm(x=None), INVALID, "x is null"),
    ("ccl_layer_norm", norm(mean=A + 2), INVALID, "not aligned"),
    ("ccl_layer_norm_grad", norm_grad(mean=None), INVALID, "mean is null"),
    ("ccl_layer_norm_grad", norm_grad(dx=A), INVALID, "also"),
    ("ccl_layer_norm_grad", norm_grad(dx=2 * A), INVALID, "also"),
    ("ccl_layer_norm_grad", norm_grad(dw=8 * A), INVALID, "also"),
    ("ccl_layer_norm_grad", norm_grad(dw=3 * A), INVALID, "also"),
    ("ccl_cross_entropy", ce(dtype=ccl.F32), UNSUPPORTED, "bf16 and f16"),
    ("ccl_cross_entropy", ce(rows=-1), INVALID, "sizes"),
    ("ccl_cross_entropy", ce(vocab=0), INVALID, "sizes"),
    ("ccl_cross_entropy", ce(vocab=(1 << 30) + 1), INVALID, "sizes"),
    ("ccl_cross_entropy", ce(k=0), INVALID, "sizes"),
    ("ccl_cross_entropy", ce(target_bits=16), INVALID, "32 nor 64"),
    ("ccl_cross_entropy", ce(ldw=31), INVALID, "w stride"),
    ("ccl_cross_entropy", ce(x=None), INVALID, "x is null"),
    ("ccl_cross_entropy", ce(target=None), INVALID, "target is null"),
    ("ccl_cross_entropy", ce(target=3 * A + 4), INVALID, "not aligned"),
    ("ccl_cross_entropy", ce(loss=None), INVALID, "loss is null"),
    ("ccl_cross_entropy", ce(loss=5 * A), INVALID, "also"),
    ("ccl_cross_entropy", ce(lse=3 * A), INVALID, "also"),
    ("ccl_cross_entropy_grad", ce_grad(dtype=ccl.F32), UNSUPPORTED, "bf16 and f16"),
    ("ccl_cross_entropy_grad", ce_grad(lse=None), INVALID, "lse is null"),
    ("ccl_cross_entropy_grad", ce_grad(dloss=None), INVALID, "dloss is null"),
    ("ccl_cross_entropy_grad", ce_grad(dlse=A + 2), INVALID, "not aligned"),
    ("ccl_cross_entropy_grad", ce_grad(dx=A), INVALID, "also"),
    ("ccl_cross_entropy_grad", ce_grad(dw=2 * A), INVALID, "also"),
    ("ccl_cross_entropy_grad", ce_grad(dw=6 * A), INVALID, "also"),
    ("ccl_cross_entropy_grad", ce_grad(lddw=16), INVALID, "dw stride"),
]


@pytest.mark.parametrize("name,a,want,word", REFUSED, ids=range(len(REFUSED)))
def test_refusals(name, a, want, word):
    assert code(name, a) == want
    assert word in ccl.lib.ccl_last_error_detail().decode()


def test_workspaces_are_asked_for_and_checked():
    def need(name, a):
        n = ctypes.c_int64(-1)
        assert getattr(ccl.lib, name + "_workspace")(ctypes.byref(a), ctypes.byref(n)) == 0
        return n.value

    assert need("ccl_route", route()) == 0
    assert need("ccl_route", route(offsets=4 * A, place=5 * A)) >= 3 * 16 * 4      # counts of three blocks of 16 rows
    assert need("ccl_route", route(offsets=4 * A, place=5 * A, rows=16)) == 0
    assert need("ccl_expert_order", order()) > 0 and need("ccl_expert_order", order(slots=100)) == 0
    assert need("ccl_layer_norm_grad", norm_grad()) >= 2 * 32 * 4
    assert need("ccl_layer_norm_grad", norm_grad(dw=None, db=None)) == 0
    assert need("ccl_cross_entropy", ce()) >= 40 * 8
    assert need("ccl_cross_entropy", ce(rows=0)) == 0 and need("ccl_cross_entropy_grad", ce_grad(rows=0)) == 0
    assert need("ccl_cross_entropy_grad", ce_grad(dx=None, dw=None)) == 0
    assert need("ccl_cross_entropy", ce(k=33)) >= need("ccl_cross_entropy", ce(k=40)) + 140 * 40 * 2
    # the derivatives of a piece of the vocabulary, and dx's sum: never those of all of it
    size = dict(rows=8192, vocab=1 << 20, k=1024)
    assert need("ccl_cross_entropy_grad", ce_grad(**size)) < (256 << 20) + 8192 * (1024 * 6 + 64) + (1 << 20)
    assert code("ccl_cross_entropy_grad", ce_grad(), ws=None, size=0) == INVALID
    assert "workspace" in ccl.lib.ccl_last_error_detail().decode()
    assert code("ccl_expert_order", order(), ws=None, size=0) == INVALID
    assert "workspace" in ccl.lib.ccl_last_error_detail().decode()
    assert code("ccl_layer_norm_grad", norm_grad(), ws=64 * A + 16) == INVALID
    assert ccl.lib.ccl_route_workspace(None, ctypes.byref(ctypes.c_int64())) == INVALID
    assert ccl.lib.ccl_route_workspace(ctypes.byref(route()), None) == INVALID


def test_empty_calls_need_no_device():
    assert code("ccl_route", route(rows=0, logits=None, weights=None, chosen=None)) == 0
    assert code("ccl_route_grad", route_grad(rows=0)) == 0
    assert code("ccl_dispatch", dispatch(rows=0)) == 0
    assert code("ccl_dispatch", dispatch(rows=0, x=None, out=None, place=None)) == 0
    assert code("ccl_combine", combine(rows=0)) == 0
    assert code("ccl_combine_grad", combine_grad(dr=None, dweights=None)) == 0
    assert code("ccl_layer_norm", norm(rows=0)) == 0
    assert code("ccl_cross_entropy", ce(rows=0)) == 0
    assert code("ccl_cross_entropy_grad", ce_grad(dx=None, dw=None)) == 0
    assert code("ccl_layer_norm_grad", norm_grad(dx=None, dw=None, db=None)) == 0
    for name in ("ccl_route", "ccl_route_grad", "ccl_expert_order", "ccl_dispatch", "ccl_combine", "ccl_combine_grad",
                 "ccl_layer_norm", "ccl_layer_norm_grad", "ccl_cross_entropy", "ccl_cross_entropy_grad"):
        fn = getattr(ccl.lib, name)
        assert (fn(None, None, 0, None) if name in WITH_WORKSPACE else fn(None, None)) == INVALID


def test_structs_match_the_header_layout(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if not cc:
        pytest.skip("no C compiler")
    pairs = [(ccl.Route, "ccl_route_t"), (ccl.RouteGrad, "ccl_route_grad_t"), (ccl.ExpertOrder, "ccl_expert_order_t"),
             (ccl.Dispatch, "ccl_dispatch_t"), (ccl.Combine, "ccl_combine_t"), (ccl.CombineGrad, "ccl_combine_grad_t"),
             (ccl.LayerNorm, "ccl_layer_norm_t"), (ccl.LayerNormGrad, "ccl_layer_norm_grad_t"),
             (ccl.CrossEntropy, "ccl_cross_entropy_t"), (ccl.CrossEntropyGrad, "ccl_cross_entropy_grad_t")]
    lines, want = ["#include <stddef.h>", "#include <stdio.h>", '#include "ccl.h"', "int main(void) {"], []
    for cls, name in pairs:
        lines.append(f'    printf("%zu\\n", sizeof({name}));')
        want.append(ctypes.sizeof(cls))
        for f in cls._fields_:
            lines.append(f'    printf("%zu\\n", offsetof({name}, {f[0]}));')
            want.append(getattr(cls, f[0]).offset)
    (tmp_path / "l.c").write_text("\n".join(lines + ["    return 0;", "}"]) + "\n")
    exe = str(tmp_path / "l")
    subprocess.run([cc, "-std=c11", "-I", os.path.join(ROOT, "include"), str(tmp_path / "l.c"), "-o", exe], check=True)
    assert [int(v) for v in subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split()] == want


def test_python_refusals():
    torch = pytest.importorskip("torch")
    x, i = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(4, 2, dtype=torch.int32)
    w, v = torch.zeros(4, 2), torch.zeros(4)
    calls = [lambda: ccl.route(x, 2), lambda: ccl.route(x[0], 2), lambda: ccl.route_backward(w, x, i),
             lambda: ccl.expert_order(i, 4), lambda: ccl.dispatch(x, i), lambda: ccl.combine(x, i, w),
             lambda: ccl.combine_backward(x, x, i, w), lambda: ccl.dispatch_backward(x, i), lambda: ccl.layer_norm(x),
             lambda: ccl.linear_cross_entropy(x, x, v.long()), lambda: ccl.linear_cross_entropy(x, x, v),
             lambda: ccl.linear_cross_entropy_backward(v, x, x, v.long(), v), lambda: ccl.layer_norm(x[0]), lambda: ccl.layer_norm_backward(x, x, None, v, v)]
    for call in calls:
        with pytest.raises(ValueError):
            call()


def test_operands_that_want_gradients_are_refused():
    """No autograd graph is recorded: the gradient would be lost without a word."""
    torch = pytest.importorskip("torch")
    x, i, w = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    n = torch.zeros(8)
    calls = [lambda t: ccl.route(t(x), 2), lambda t: ccl.route(x, 2, bias=t(n)), lambda t: ccl.dispatch(t(x), i),
             lambda t: ccl.combine(t(x), i, w), lambda t: ccl.combine(x, i, t(w)), lambda t: ccl.combine(x, i, w, residual=t(x)),
             lambda t: ccl.linear_cross_entropy(t(x), x, i[:, 0].contiguous()),
             lambda t: ccl.linear_cross_entropy(x, t(x), i[:, 0].contiguous()), lambda t: ccl.layer_norm(t(x)), lambda t: ccl.layer_norm(x, t(n)), lambda t: ccl.layer_norm(x, n, t(n))]
    for call in calls:
        with pytest.raises(ValueError, match="autograd"):
            call(lambda t: t.clone().requires_grad_(True))
        with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
            call(lambda t: t.clone().requires_grad_(True))

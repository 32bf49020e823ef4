"""Refusals, workspace sizes and struct layouts of the tensor products (no GPU
needed: arguments are checked before any device is touched)."""
import ctypes
import os
import shutil
import subprocess

import pytest

import collective_communication_schedule_gb300 as ccl

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 1 << 20                # stands for device addresses: never read here


def linear(**kw):
    a = ccl.Linear(rows=4, n=16, k=32, dtype=ccl.BF16, x=A, w=2 * A, y=3 * A)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def grad(**kw):
    a = ccl.LinearGrad(rows=4, n=16, k=32, dtype=ccl.F16, dy=A, x=2 * A, w=3 * A, dx=4 * A, dw=5 * A)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def ortho(**kw):
    a = ccl.Ortho(batch=1, p=16, q=32, dtype=ccl.F32, out_dtype=ccl.BF16, steps=5, a=3.4, b=-4.7, c=2.0, eps=1e-7,
                  scale=1.0, g=A, out=2 * A)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def code(name, a, ws=64 * A, size=1 << 40):
    return getattr(ccl.lib, name)(ctypes.byref(a), ws, size, None)


INVALID, UNSUPPORTED = 1, 5


@pytest.mark.parametrize("name,a,want,word", [
    ("ccl_linear", linear(dtype=ccl.F32), UNSUPPORTED, "bf16 and f16"),
    ("ccl_linear", linear(dtype=ccl.I32), UNSUPPORTED, "bf16 and f16"),
    ("ccl_linear", linear(rows=-1), INVALID, "sizes"),
    ("ccl_linear", linear(k=0), INVALID, "sizes"),
    ("ccl_linear", linear(n=0), INVALID, "sizes"),
    ("ccl_linear", linear(rows=1 << 31), INVALID, "sizes"),
    ("ccl_linear", linear(act=4), INVALID, "activation"),
    ("ccl_linear", linear(act=-1), INVALID, "activation"),
    ("ccl_linear", linear(ldx=31), INVALID, "x stride"),
    ("ccl_linear", linear(ldw=-32), INVALID, "w stride"),
    ("ccl_linear", linear(ldy=15), INVALID, "y stride"),
    ("ccl_linear", linear(x=None), INVALID, "x is null"),
    ("ccl_linear", linear(y=None), INVALID, "y is null"),
    ("ccl_linear", linear(w=A + 1), INVALID, "not aligned"),
    ("ccl_linear", linear(y=A), INVALID, "also an operand"),
    ("ccl_linear", linear(experts=3), INVALID, "offsets"),
    ("ccl_linear", linear(experts=1025, offsets=A), INVALID, "experts outside"),
    ("ccl_linear", linear(experts=3, offsets=A, w_stride=100), INVALID, "w expert stride"),
    ("ccl_linear_grad", grad(dtype=ccl.F32), UNSUPPORTED, "bf16 and f16"),
    ("ccl_linear_grad", grad(act=ccl.ACT_GELU), INVALID, "z is null"),
    ("ccl_linear_grad", grad(dy=None), INVALID, "dy is null"),
    ("ccl_linear_grad", grad(lddx=8), INVALID, "dx stride"),
    ("ccl_linear_grad", grad(dx=A), INVALID, "also an operand"),
    ("ccl_orthogonalize", ortho(dtype=ccl.I32), UNSUPPORTED, "gradients"),
    ("ccl_orthogonalize", ortho(out_dtype=ccl.F32), UNSUPPORTED, "update"),
    ("ccl_orthogonalize", ortho(p=0), INVALID, "sizes"),
    ("ccl_orthogonalize", ortho(batch=-1), INVALID, "sizes"),
    ("ccl_orthogonalize", ortho(steps=0), INVALID, "steps"),
    ("ccl_orthogonalize", ortho(eps=-1.0), INVALID, "eps"),
    ("ccl_orthogonalize", ortho(eps=float("nan")), INVALID, "eps"),
    ("ccl_orthogonalize", ortho(g=None), INVALID, "null"),
    ("ccl_orthogonalize", ortho(ldg=31), INVALID, "g stride"),
    ("ccl_orthogonalize", ortho(g=A + 2), INVALID, "not aligned"),
])
def test_refusals(name, a, want, word):
    assert code(name, a) == want
    assert word in ccl.lib.ccl_last_error_detail().decode()


def test_workspaces_are_asked_for_and_checked():
    def need(name, a):
        n = ctypes.c_int64(-1)
        assert getattr(ccl.lib, name + "_workspace")(ctypes.byref(a), ctypes.byref(n)) == 0
        return n.value

    assert need("ccl_linear", linear()) == 0
    assert need("ccl_linear", linear(k=33)) >= (4 + 16) * 40 * 2        # both operands copied to padded rows
    assert need("ccl_linear", linear(x=A + 2)) >= 4 * 32 * 2
    assert need("ccl_linear_grad", grad()) == 0
    assert need("ccl_linear_grad", grad(act=ccl.ACT_RELU, z=A)) >= 4 * 16 * 2
    assert need("ccl_orthogonalize", ortho()) > 2 * 16 * 32 * 2
    assert code("ccl_linear", linear(k=33), ws=None, size=0) == INVALID
    assert "workspace" in ccl.lib.ccl_last_error_detail().decode()
    assert code("ccl_orthogonalize", ortho(), ws=64 * A, size=16) == INVALID
    assert code("ccl_orthogonalize", ortho(), ws=64 * A + 16) == INVALID
    assert ccl.lib.ccl_linear_workspace(None, ctypes.byref(ctypes.c_int64())) == INVALID
    assert ccl.lib.ccl_linear_workspace(ctypes.byref(linear()), None) == INVALID


def test_empty_calls_need_no_device():
    assert code("ccl_linear", linear(rows=0, x=None, w=None, y=None)) == 0
    assert code("ccl_orthogonalize", ortho(batch=0)) == 0


def test_structs_match_the_header_layout(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if not cc:
        pytest.skip("no C compiler")
    pairs = [(ccl.Linear, "ccl_linear_t"), (ccl.LinearGrad, "ccl_linear_grad_t"), (ccl.Ortho, "ccl_ortho_t")]
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
    x, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(6, 8, dtype=torch.bfloat16)
    for call in (lambda: ccl.linear(x, w), lambda: ccl.orthogonalize(x), lambda: ccl.linear(x[0], w),
                 lambda: ccl.linear_backward(x, x, w, act=ccl.ACT_GELU), lambda: ccl.orthogonalize(x[0])):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("a", [
    grad(dx=2 * A),                              # over x, which dw reads
    grad(dw=3 * A),                              # over w, which dx reads
    grad(dx=6 * A, dw=6 * A),
    grad(db=A), grad(db=2 * A), grad(db=3 * A), grad(db=4 * A), grad(db=5 * A),
    grad(act=ccl.ACT_GELU, z=6 * A, dx=2 * A),
    grad(experts=2, offsets=7 * A, dw=3 * A),
    grad(x=2 * A + 2, dx=2 * A + 2),             # copied to the workspace first, but refused all the same
], ids=range(11))
def test_gradients_over_operands_are_refused(a):
    """The two products run at one time: neither may write what the other reads."""
    assert code("ccl_linear_grad", a) == INVALID
    assert "also" in ccl.lib.ccl_last_error_detail().decode()


@pytest.mark.parametrize("a", [
    linear(z=A), linear(z=2 * A), linear(z=3 * A),
    linear(residual=4 * A, z=4 * A),                          # z is stored before the residual is read
    linear(bias=4 * A, z=4 * A), linear(bias=3 * A),
    linear(residual=3 * A, ldr=24),                           # y over a residual with other strides
    linear(residual=3 * A, ldy=24),
    linear(experts=2, offsets=5 * A, residual=4 * A, z=4 * A),
], ids=range(9))
def test_products_over_operands_are_refused(a):
    assert code("ccl_linear", a) == INVALID
    assert "operand" in ccl.lib.ccl_last_error_detail().decode() or "stride" in ccl.lib.ccl_last_error_detail().decode()


@pytest.mark.parametrize("a", [ortho(batch=2, out=A),                                    # f32 over bf16: matrices apart
                               ortho(batch=2, dtype=ccl.BF16, out=A, out_stride=1024),
                               ortho(batch=3, dtype=ccl.F16, out=A, ldg=40),
                               ortho(batch=2, p=64, q=5000, dtype=ccl.F32, out=A)], ids=range(4))
def test_updates_over_gradients_of_other_strides_are_refused(a):
    """A matrix may be written while another one of the batch is read."""
    assert code("ccl_orthogonalize", a) == INVALID
    assert "in place" in ccl.lib.ccl_last_error_detail().decode()


def test_gradients_ask_for_no_more_than_they_use():
    def need(a):
        n = ctypes.c_int64(-1)
        assert ccl.lib.ccl_linear_grad_workspace(ctypes.byref(a), ctypes.byref(n)) == 0
        return n.value

    rows, n, k = 3200, 136, 33                       # k = 33: x and w are copied to padded rows for a product
    size = dict(rows=rows, n=n, k=k)
    sums = (rows // 32 + 1) * 192 * 4 + 256          # one row of 32-bit sums for every 32 rows
    for act, z in ((ccl.ACT_NONE, None), (ccl.ACT_GELU, 6 * A)):
        alone = dict(size, act=act, z=z, dx=None, dw=None)
        assert need(grad(**alone)) == 0
        assert code("ccl_linear_grad", grad(**alone), ws=None, size=0) == 0          # nothing to do
        assert 0 < need(grad(db=7 * A, **alone)) <= sums
        assert 0 < need(grad(db=7 * A, experts=3, offsets=8 * A, **alone)) <= sums + 2 * 192 * 4
        assert 0 < need(grad(db=7 * A, dy=A + 2, **alone)) <= sums
    # the operand of a product that is not asked for is not copied
    apart = need(grad(dw=None, **size)), need(grad(dx=None, **size))
    assert apart[0] == -(-n * 40 * 2 // 256) * 256 and apart[1] == rows * 40 * 2
    assert need(grad(experts=2, offsets=8 * A, dx=None, n=7, k=40, lddw=40)) == need(grad(dx=None, n=7, k=40))
    assert need(grad(experts=2, offsets=8 * A, dx=None, n=7, k=40, ldw=44, w_stride=308)) == need(grad(dx=None, n=7, k=40))


def test_operands_that_want_gradients_are_refused():
    """The products record no autograd graph: the gradient would be lost without a word."""
    torch = pytest.importorskip("torch")
    plain = dict(dtype=torch.bfloat16)
    x, w, b, r = torch.zeros(4, 8, **plain), torch.zeros(6, 8, **plain), torch.zeros(6, **plain), torch.zeros(4, 6, **plain)
    offs = torch.zeros(3, dtype=torch.int32)
    calls = [lambda t: ccl.linear(t(x), w), lambda t: ccl.linear(x, t(w)), lambda t: ccl.linear(x, w, bias=t(b)),
             lambda t: ccl.linear(x, w, residual=t(r)), lambda t: ccl.grouped_linear(x, t(w).expand(2, 6, 8), offs),
             lambda t: ccl.orthogonalize(t(w))]
    for call in calls:
        with pytest.raises(ValueError, match="autograd"):
            call(lambda t: t.clone().requires_grad_(True))
        with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
            call(lambda t: t.clone().requires_grad_(True))
        with pytest.raises(ValueError, match="CUDA"):
            call(lambda t: t)

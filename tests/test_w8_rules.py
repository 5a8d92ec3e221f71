"""8-bit layer and block norms without a GPU: the rounding rule, the gradient
formulas against differences, and the refusals of the C API and of the binding."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest
import torch

import gemv_w4a16_groupwise_b200 as w4
import w8_reference as ref


def test_rounding_rule_is_the_exact_quotient_half_to_even():
    """rint(v * inv) equals the exact 127 v / max rounded half to even for every bf16
    significand pair and distance that can matter, at both ends of what inv may be:
    127 / max itself and 2^-21 above it (exactly 127 / max where that is a power of two)."""
    i, d = np.meshgrid(np.arange(256), np.arange(11))
    for b in range(128, 256):
        inside = i <= b * 2 ** d
        num, den = 127 * i[inside], b * 2 ** d[inside]
        lo, rem2 = num // den, 2 * (num % den)
        want = lo + ((rem2 > den) | ((rem2 == den) & (lo % 2 == 1)))
        exact = np.float64(127) / b
        up = np.nextafter(exact, 2.0) if Fraction(float(exact)) < Fraction(127, b) else exact
        for inv in ([exact] if b == 254 else [up, exact * (1 + 2.0 ** -21)]):
            got = np.rint(i[inside] * 2.0 ** -d[inside] * inv)     # an fma onto 1.5 * 2^23 rounds the exact product
            assert (got == want).all(), b


def _loss(x, y, pre, post, gate, alpha, off, cn, cr):
    f = ref.norm_forward(x, y, pre, post, gate, alpha, off, 1e-5)
    n, _ = ref.norm_of(f["residual"], pre, off, 1e-5)
    return (n * cn).sum() + (f["residual"] * cr).sum()


@pytest.mark.parametrize("post,gate", [(False, None), (True, None), (False, "channel"), (True, "token"),
                                       (True, "channel")])
def test_gradient_formulas_against_differences(post, gate):
    gen = torch.Generator().manual_seed(11)
    rnd = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)  # noqa: E731
    M, C, alpha, off = 3, 5, 0.7, 1.0
    v = {"x": rnd(M, C), "y": rnd(M, C), "pre": rnd(C), "post": rnd(C) if post else None,
         "gate": {None: None, "channel": rnd(C), "token": rnd(M, C)}[gate]}
    cn, cr = rnd(M, C), rnd(M, C)
    f = ref.norm_forward(v["x"], v["y"], v["pre"], v["post"], v["gate"], alpha, off, 1e-5)
    _, rr = ref.norm_of(f["residual"], v["pre"], off, 1e-5)
    ry = f["rstd_y"] if post else torch.zeros(M, dtype=torch.float64)
    g = ref.norm_backward(cn, cr, f["residual"], torch.stack([ry, rr]), v["y"], v["pre"], v["post"], v["gate"],
                          alpha, off)
    for name, out in (("x", "d_x"), ("y", "d_y"), ("pre", "d_pre_weight"), ("post", "d_post_weight"),
                      ("gate", "d_gate")):
        if v[name] is None:
            assert out not in g
            continue
        for at in range(v[name].numel()):
            h = 1e-5
            step = torch.zeros_like(v[name]).view(-1)
            step[at] = h
            step = step.view_as(v[name])
            plus, minus = ({**v, name: v[name] + s} for s in (step, -step))
            diff = (_loss(**plus, alpha=alpha, off=off, cn=cn, cr=cr)
                    - _loss(**minus, alpha=alpha, off=off, cn=cn, cr=cr)) / (2 * h)
            # central differences: h^2 f''' / 6 and 2^-53 |f| / h, both under 1e-8 here
            assert abs(diff - g[out][0].reshape(-1)[at]) < 1e-7, (name, at)


FAKE = 1 << 20      # never dereferenced: validation fails before any CUDA call


def test_quantize_rows_refusals():
    f = w4.library().w8_quantize_rows
    assert f(FAKE, 0, 8, None, FAKE, 16, FAKE, None) == 1
    assert f(FAKE, 4, 0, None, FAKE, 16, FAKE, None) == 1
    assert f(FAKE, 4, 17, None, FAKE, 16, FAKE, None) == 1          # ld < C
    assert f(None, 4, 8, None, FAKE, 16, FAKE, None) == 1
    assert f(FAKE, 4, 8, None, None, 16, FAKE, None) == 1
    assert f(FAKE, 4, 8, None, FAKE, 16, None, None) == 1
    assert f(FAKE + 2, 4, 8, None, FAKE, 16, FAKE, None) == 3
    assert f(FAKE, 4, 8, FAKE + 4, FAKE, 16, FAKE, None) == 3
    assert f(FAKE, 4, 8, None, FAKE, 24, FAKE, None) == 3
    assert f(FAKE, 4, (1 << 30) + 16, None, FAKE, 1 << 31, FAKE, None) == 2


def _gemm_args(**k):
    d = dict(A=FAKE, lda=64, a_s=FAKE, M=4, N=32, K=64, W=FAKE, ldw=64, w_s=FAKE, bias=None, tr=0, Y=FAKE, ws=None,
             nws=0, st=None)
    d.update(k)
    return tuple(d.values())


@pytest.mark.parametrize("want,change", [
    (1, dict(M=0)), (1, dict(N=-1)), (1, dict(K=0)), (1, dict(ldw=48)), (1, dict(lda=48)), (1, dict(W=None)),
    (1, dict(A=None)), (1, dict(a_s=None)), (1, dict(Y=None)), (1, dict(w_s=None)), (1, dict(tr=1)),
    (2, dict(K=131072, lda=131072, ldw=131072)), (2, dict(M=(1 << 30) + 1)), (2, dict(N=(1 << 30) + 1)), (2, dict(tr=1, N=131072, w_s=None, lda=131072)),
    (3, dict(lda=72)), (3, dict(ldw=72)), (3, dict(A=FAKE + 8)), (3, dict(bias=FAKE + 2)), (3, dict(Y=FAKE + 4))])
def test_gemm_refusals(want, change):
    assert w4.library().w8a8_gemm(*_gemm_args(**change)) == want


@pytest.mark.parametrize("want,change", [
    (1, dict(M=0)), (1, dict(w_s=None)), (1, dict(ldw=48)), (2, dict(K=131072, ldw=131072)),
    (2, dict(tr=1, N=131072)), (3, dict(A=FAKE + 2)), (3, dict(w_s=FAKE + 4)), (4, dict(M=40)),
    (4, dict(M=40, ws=FAKE, nws=64)), (3, dict(M=40, ws=FAKE + 8, nws=1 << 30))])
def test_linear_refusals(want, change):
    d = dict(A=FAKE, M=4, N=32, K=64, W=FAKE, ldw=64, w_s=FAKE, bias=None, tr=0, Y=FAKE, ws=None, nws=0, st=None)
    d.update(change)
    assert w4.library().w8a8_linear(*d.values()) == want


def _norm_args(**k):
    d = dict(x=FAKE, y=FAKE, M=2, C=8, post=None, gate=None, kind=0, alpha=1.0, pre=FAKE, off=0.0, eps=1e-5, r=FAKE,
             n=FAKE, ld=16, scales=None, rstd=None, st=None)
    d.update(k)
    return tuple(d.values())


@pytest.mark.parametrize("want,change", [
    (1, dict(M=0)), (1, dict(C=0)), (2, dict(C=16385)), (2, dict(M=(1 << 30) + 1)), (1, dict(kind=3, gate=FAKE)), (1, dict(kind=1)),
    (1, dict(gate=FAKE)), (1, dict(eps=0.0)), (1, dict(eps=-1.0)), (1, dict(eps=float("nan"))),
    (1, dict(eps=float("inf"))), (1, dict(x=None)), (1, dict(pre=None)), (1, dict(n=None)), (1, dict(r=None)),
    (1, dict(y=None)), (1, dict(y=None, r=None, post=FAKE)), (1, dict(y=None, r=None, gate=FAKE, kind=1)),
    (1, dict(scales=FAKE, C=24)), (3, dict(scales=FAKE, ld=24)), (3, dict(x=FAKE + 2)), (3, dict(rstd=FAKE + 4))])
def test_block_norm_refusals(want, change):
    assert w4.library().w4_block_norm(*_norm_args(**change)) == want


@pytest.mark.parametrize("want,change", [
    (1, dict(M=0)), (2, dict(C=16385)), (1, dict(dn=None)), (1, dict(rstd=None)), (1, dict(dy=None)),
    (1, dict(y=None)), (1, dict(post=FAKE)), (1, dict(dgate=FAKE)), (1, dict(gate=FAKE, kind=1)),
    (3, dict(dx=FAKE + 2)), (3, dict(dres=FAKE + 2)), (4, dict())])
def test_block_norm_backward_refusals(want, change):
    d = dict(dn=FAKE, dres=None, r=FAKE, rstd=FAKE, y=FAKE, M=2, C=8, post=None, gate=None, kind=0, alpha=1.0,
             pre=FAKE, off=0.0, dx=FAKE, dy=FAKE, dpre=FAKE, dpost=None, dgate=None, ws=None, nws=0, st=None)
    d.update(change)
    assert w4.library().w4_block_norm_backward(*d.values()) == want


def test_binding_refuses_host_tensors_and_wrong_types():
    x = torch.zeros(2, 16, dtype=torch.bfloat16)
    q, s = torch.zeros(4, 16, dtype=torch.int8), torch.ones(4)
    for call in (lambda: w4.w8_quantize_rows(x), lambda: w4.w8a8_linear(x, q, s),
                 lambda: w4.w8a8_gemm(q, s, q, s), lambda: w4.w4_block_norm(x, pre_weight=x[0]),
                 lambda: w4.w4_block_norm_backward(x, x, s, pre_weight=x[0])):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError):
        w4.w8a8_gemm(q, s, q, s, transposed=True)      # the scales belong in A's rows
    with pytest.raises(ValueError):
        w4.w8a8_gemm(q, s, q)
    with pytest.raises(TypeError):
        w4.w8_quantize_rows([1.0])


def test_native_calls_leave_what_they_do_not_take():
    """The native module answers None, and raises nothing, for host tensors and odd arguments."""
    native = w4._native()
    x, q, s = torch.zeros(2, 16, dtype=torch.bfloat16), torch.zeros(4, 16, dtype=torch.int8), torch.ones(4)
    assert native.quantize_rows(x, None) is None
    assert native.quantize_rows(3, None) is None and native.quantize_rows(x) is None
    assert native.gemm(q, s, q, s, None, False, None) is None and native.gemm(None, 1, 2, 3, 4, 5, 6) is None
    assert native.linear(x, q, s, None, False, None) is None and native.linear(x) is None
    assert native.norm(x, x, x[0], None, None, 1.0, 0.0, 1e-5, False, False, None) is None
    assert native.norm_backward(x, x, s, None, None, x[0], None, None, 1.0, 0.0) is None
    with pytest.raises(TypeError):
        native.bind(1)


def test_header_and_binding_agree_on_the_new_symbols():
    lib = ctypes.CDLL(w4.library_path())
    for name in ("w8_quantize_rows", "w8a8_gemm", "w8a8_linear", "w8a8_workspace_bytes",
                 "w8a8_linear_workspace_bytes", "w4_block_norm", "w4_block_norm_backward",
                 "w4_block_norm_workspace_bytes"):
        assert hasattr(lib, name), name

"""The 8-bit layer and the block norms where the binding's native part cannot be built or loaded: the same
checks, the same kernels, the same bits."""
import subprocess
import warnings

import pytest
import torch

import gemv_w4a16_groupwise_b200 as w4
from gemv_w4a16_groupwise_b200 import build


def _fail(error):
    def build_binding(*args, **kwargs):
        raise error
    return build_binding


@pytest.fixture(params=[subprocess.CalledProcessError(1, ["g++"]), FileNotFoundError("g++"), PermissionError("tree"),
                        ImportError("undefined symbol")], ids=lambda e: type(e).__name__)
def no_native(request, monkeypatch):
    monkeypatch.setattr(build, "build_binding", _fail(request.param))
    monkeypatch.setattr(w4._Torch, "torch", None)
    monkeypatch.setattr(w4._Torch, "native", None)


def test_checks_still_speak(no_native):
    x = torch.zeros(2, 16, dtype=torch.bfloat16)
    q, s = torch.zeros(4, 16, dtype=torch.int8), torch.ones(4)
    with pytest.warns(RuntimeWarning, match="native"):
        with pytest.raises(ValueError):
            w4.w8_quantize_rows(x)
    with warnings.catch_warnings():
        warnings.simplefilter("error")           # it is said once
        for call in (lambda: w4.w8a8_linear(x, q, s), lambda: w4.w8a8_gemm(q, s, q, s),
                     lambda: w4.w4_block_norm(x, pre_weight=x[0]),
                     lambda: w4.w4_block_norm_backward(x, x, s, pre_weight=x[0])):
            with pytest.raises(ValueError):
                call()


def _step(dev):
    g = torch.Generator(device=dev).manual_seed(1)
    r = lambda *s: torch.randn(s, generator=g, device=dev).to(torch.bfloat16)  # noqa: E731
    out = []
    for M, N, K in ((1, 96, 64), (5, 200, 333), (70, 640, 512)):
        W, ws = w4.w8_quantize_rows(r(N, K))
        x, b = r(M, K), r(N)
        a, a_s = w4.w8_quantize_rows(x)
        d, d_s = w4.w8_quantize_rows(r(M, N), channel_scales=ws)
        out += [W, ws, a, a_s, d, d_s, w4.w8a8_gemm(a, a_s, W, ws, bias=b), w4.w8a8_gemm(d, d_s, W, transposed=True),
                w4.w8a8_linear(x, W, ws, bias=b), w4.w8a8_linear(r(M, N), W, ws, transposed=True)]
        for gate in (None, r(K), r(M, K)):
            k = dict(pre_weight=r(K), post_weight=r(K), gate=gate, residual_scale=0.5, weight_offset=1.0)
            y = r(M, K)
            f = w4.w4_block_norm(x, y, keep_rstd=True, **k)
            out += [*f, *w4.w4_block_norm(x, y, quantize=True, **k)]
            out += w4.w4_block_norm_backward(r(M, K), f.residual, f.rstd, y, d_residual=r(M, K), **k)
        out += w4.w4_block_norm(x, pre_weight=r(K))
    assert w4.w4_device_error() == 0
    return out


@pytest.mark.gpu
def test_the_same_bits(cuda_device, monkeypatch):
    want = _step(cuda_device)
    monkeypatch.setattr(build, "build_binding", _fail(FileNotFoundError("g++")))
    monkeypatch.setattr(w4._Torch, "torch", None)
    monkeypatch.setattr(w4._Torch, "native", None)
    with pytest.warns(RuntimeWarning, match="native"):
        got = _step(cuda_device)
    assert w4._Torch.native is w4._NoNative and len(got) == len(want)
    for a, b in zip(got, want):
        assert (a is None and b is None) or (torch.equal(a, b) and a.shape == b.shape and a.stride() == b.stride())

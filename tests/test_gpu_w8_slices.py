"""Part of a batch, or of the channels, at any row: codes and scales as slices of larger tensors."""
import ctypes

import pytest
import torch

import gemv_w4a16_groupwise_b200 as w4

FAKE = 1 << 20      # never dereferenced: validation fails before any CUDA call


def test_scales_off_four_bytes_are_refused():
    f = w4.library().w8a8_gemm
    args = lambda a_s, w_s: (FAKE, 64, a_s, 4, 32, 64, FAKE, 64, w_s, None, 0, FAKE, None, 0, None)  # noqa: E731
    assert f(*args(FAKE + 2, FAKE)) == 3 and f(*args(FAKE, FAKE + 2)) == 3
    assert w4.library().w8_quantize_rows(FAKE, 4, 8, None, FAKE, 16, ctypes.c_void_p(FAKE + 1), None) == 3


@pytest.mark.gpu
@pytest.mark.parametrize("M", [4, 30, 300])
@pytest.mark.parametrize("lo", [1, 2, 3, 4])
@pytest.mark.parametrize("tr", [False, True])
def test_product_of_a_part(cuda_device, M, lo, tr):
    dev = cuda_device
    N, K = 520, 640
    g = torch.Generator(device=dev).manual_seed(M + lo)
    rows = lambda *s: torch.randn(s, generator=g, device=dev).to(torch.bfloat16)  # noqa: E731
    W, ws = w4.w8_quantize_rows(rows(N, K))
    a, a_s = w4.w8_quantize_rows(rows(M + 8, N if tr else K), channel_scales=ws if tr else None)
    whole = w4.w8a8_gemm(a, a_s, W, None if tr else ws, transposed=tr)
    part = w4.w8a8_gemm(a[lo:lo + M], a_s[lo:lo + M], W, None if tr else ws, transposed=tr)
    assert torch.equal(part, whole[lo:lo + M])
    if not tr:
        part = w4.w8a8_gemm(a[lo:lo + M], a_s[lo:lo + M], W[lo:lo + 512], ws[lo:lo + 512])
        assert torch.equal(part, whole[lo:lo + M, lo:lo + 512])


@pytest.mark.gpu
@pytest.mark.parametrize("C", [64, 999, 40000])
@pytest.mark.parametrize("lo", [1, 2, 3])
def test_rows_quantized_into_a_part(cuda_device, C, lo):
    dev = cuda_device
    X = torch.randn(9, C, device=dev).to(torch.bfloat16)
    codes, scales = w4.w8_quantize_rows(X)
    buf = torch.full((16, (C + 15) // 16 * 16), 99, dtype=torch.int8, device=dev)
    sc = torch.full((16,), 7.0, device=dev)
    w4.w8_quantize_rows(X, out=(buf[lo:lo + 9, :C], sc[lo:lo + 9]))
    assert torch.equal(buf[lo:lo + 9, :C], codes) and torch.equal(sc[lo:lo + 9], scales)
    assert (buf[:lo] == 99).all() and (buf[lo + 9:] == 99).all() and (sc[:lo] == 7).all() and (sc[lo + 9:] == 7).all()

"""The codes of fp32 rows (rows times channel factors, normed rows): those of fp32 arithmetic, and how near
they are to the exact quotients.

Bound.  127 v and its quotient by max |v| are rounded to fp32, half a step (2^-24) each, before the rounding to
a whole number: |code - 127 v / max |v|| <= 0.5 + 127 (2^-23 + 2^-48).  The quotients here are taken in 64 bits
of the same fp32 values (127 * 2^-52 off at most).

bf16 rows multiply by inv, the least fp32 number that is not below 127 / max |v|."""
import numpy as np
import pytest
import torch

import gemv_w4a16_groupwise_b200 as w4

F, WIDE = np.float32, np.longdouble
NEAR = 0.5 + 127 * (2.0 ** -23 + 2.0 ** -48 + 2.0 ** -52)


def _inv(top, r):
    """The kernels' steps on a maximum and a reciprocal of it, each rounded once."""
    i = F(127) * r
    left = (WIDE(127) - i.astype(WIDE) * top.astype(WIDE)).astype(F)
    i = (left.astype(WIDE) * r.astype(WIDE) + i.astype(WIDE)).astype(F)
    low = WIDE(127) - i.astype(WIDE) * top.astype(WIDE) > 0
    return np.where(low, np.nextafter(i, F(np.inf)), i)


@pytest.mark.parametrize("ulp", [-1, 0, 1])
def test_inv_is_the_least_that_is_not_below(ulp):
    """Every eighth significand and all of bf16's, with a reciprocal that is off by an ulp either way."""
    top = (np.arange(0, 1 << 23, 8, dtype=np.uint32) | np.uint32(0x3F800000)).view(F)
    top = np.concatenate([top, np.nextafter(top, F(4)), np.arange(128, 256).astype(F)])
    r = (WIDE(1) / top.astype(WIDE)).astype(F)
    if ulp:
        r = np.nextafter(r, F(np.inf * ulp))
    inv = _inv(top, r)
    assert (inv.astype(WIDE) * top.astype(WIDE) >= 127).all()
    assert (np.nextafter(inv, F(0)).astype(WIDE) * top.astype(WIDE) < 127).all()


def _exact(v):
    v = v.double()
    return v * 127 / v.abs().amax(1, keepdim=True)


def _near(codes, v):
    assert torch.equal(codes.float(), torch.round(v * 127 / v.abs().amax(1, keepdim=True)))
    off = (codes.double() - _exact(v)).abs()
    assert (off <= NEAR).all(), f"{int((off > NEAR).sum())} codes of {off.numel()}, the worst off by {off.max().item():.9f}"


@pytest.mark.gpu
@pytest.mark.parametrize("R,C", [(2000, 1024), (1500, 999), (700, 4096), (300, 6001), (300, 8192), (200, 11008),
                                 (100, 14336), (100, 16383), (40, 33000), (21, 40001)])
def test_rows_times_channel_factors(cuda_device, R, C):
    dev = cuda_device
    g = torch.Generator(device=dev).manual_seed(R + C)
    X = torch.randn(R, C, generator=g, device=dev).to(torch.bfloat16)
    f = torch.rand(C, generator=g, device=dev) * 0.002 + 1e-4
    codes, _ = w4.w8_quantize_rows(X, channel_scales=f)
    _near(codes, X.float() * f)


@pytest.mark.gpu
@pytest.mark.parametrize("M,C", [(2000, 1024), (1500, 999), (700, 4096), (300, 6001), (200, 16384)])
def test_normed_rows(cuda_device, M, C):
    """The normed values are four fp32 products and sums of tensors at hand, formed here in the same order."""
    dev = cuda_device
    g = torch.Generator(device=dev).manual_seed(M + C)
    x = torch.randn(M, C, generator=g, device=dev).to(torch.bfloat16)
    pre = (0.1 * torch.randn(C, generator=g, device=dev)).to(torch.bfloat16)
    f = w4.w4_block_norm(x, pre_weight=pre, weight_offset=1.0, quantize=True, keep_rstd=True)
    _near(f.normed, (x.float() * f.rstd[1][:, None]) * (pre.float() + 1.0))


@pytest.mark.gpu
@pytest.mark.parametrize("R,C", [(500, 4096), (300, 11008), (300, 1001)])
def test_gradients_times_the_scales_of_quantized_weights(cuda_device, R, C):
    """Scales that are bf16 values over 127: quotients of two products of bf16 values, ties among them."""
    dev = cuda_device
    g = torch.Generator(device=dev).manual_seed(C)
    _, ws = w4.w8_quantize_rows((0.02 * torch.randn(C, 512, generator=g, device=dev)).to(torch.bfloat16))
    X = torch.randn(R, C, generator=g, device=dev).to(torch.bfloat16)
    codes, _ = w4.w8_quantize_rows(X, channel_scales=ws)
    _near(codes, X.float() * ws)


@pytest.mark.gpu
@pytest.mark.parametrize("C", [24, 999, 4096])
def test_extreme_fp32_rows(cuda_device, C):
    """Rows times factors that leave fp32's middle range, where the row is scaled by a power of two first; rows of
    zeros; poisoned rows."""
    dev = cuda_device
    g = torch.Generator(device=dev).manual_seed(C)
    X = torch.randn(6, C, generator=g, device=dev).to(torch.bfloat16)
    X[1] = 0
    X[2, C // 2] = float("inf")
    X[3, 0] = float("nan")
    for factor in (1e-35, 1e-30, 1.0, 1e29, 1e33):
        f = (torch.rand(C, generator=g, device=dev) + 0.5) * factor
        codes, scales = w4.w8_quantize_rows(X, channel_scales=f)
        fine = [0, 4, 5]
        v = (X.float() * f)[fine]
        power = 2.0 ** -round(torch.log2(v.abs().max()).item())      # exact, so that 127 v stays in range
        _near(codes[fine], (v.double() * power).float())
        assert not codes[1:4].any() and scales[1] == 0 and torch.isnan(scales[2:4]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("C", [64, 999, 4096, 11008, 40000])
def test_one_factor_for_all_channels(cuda_device, C):
    """A common factor fills rows with quotients that are ties but for a rounding; a power of two leaves every code."""
    dev = cuda_device
    g = torch.Generator(device=dev).manual_seed(C)
    X = torch.randn(257, C, generator=g, device=dev).to(torch.bfloat16)
    X[:, C // 2] = X.abs().amax(1) / 2
    X[:, 0] = X.abs().amax(1)
    X[:, 1] = -X[:, 0] / 2
    plain, scales = w4.w8_quantize_rows(X)
    for factor in (0.3, 0.0123, 7.7e-5, 1.9):
        f = torch.full((C,), factor, device=dev)
        codes, _ = w4.w8_quantize_rows(X, channel_scales=f)
        _near(codes, X.float() * f)
        assert (codes[:, 0] == 127).all()
    for factor in (1.0, 0.125, 2.0 ** -20):
        codes, s = w4.w8_quantize_rows(X, channel_scales=torch.full((C,), factor, device=dev))
        assert torch.equal(codes, plain) and torch.equal(s, scales * factor)

"""How near the codes of fp32 rows are to the exact quotients: rows times channel factors, normed rows.

Bound.  The kernels multiply by inv, the least fp32 number that is not below 127 / max |v|, so above it by
less than 2^-23 of it, in one fma whose result is the rounded integer: |code - 127 v / max |v|| <= 0.5 +
127 * 2^-23.  The quotients here are taken in 64 bits of the same fp32 values (127 * 2^-52 off at most)."""
import numpy as np
import pytest
import torch

import gemv_w4a16_groupwise_b200 as w4

F, WIDE = np.float32, np.longdouble
NEAR = 0.5 + 127 * 2.0 ** -23 + 127 * 2.0 ** -52


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
@pytest.mark.parametrize("C", [64, 999, 4096, 11008, 40000])
def test_one_factor_for_all_channels(cuda_device, C):
    """A common factor leaves half of the maximum at 63.5, which is 64; a power of two leaves every code."""
    dev = cuda_device
    g = torch.Generator(device=dev).manual_seed(C)
    X = torch.randn(257, C, generator=g, device=dev).to(torch.bfloat16)
    X[:, C // 2] = X.abs().amax(1) / 2
    X[:, 0] = X.abs().amax(1)
    X[:, 1] = -X[:, 0] / 2
    plain, scales = w4.w8_quantize_rows(X)
    for factor in (0.3, 0.0123, 7.7e-5, 1.9):
        codes, _ = w4.w8_quantize_rows(X, channel_scales=torch.full((C,), factor, device=dev))
        assert (codes[:, 0] == 127).all() and (codes[:, 1] == -64).all()
    for factor in (1.0, 0.125, 2.0 ** -20):
        codes, s = w4.w8_quantize_rows(X, channel_scales=torch.full((C,), factor, device=dev))
        assert torch.equal(codes, plain) and torch.equal(s, scales * factor)

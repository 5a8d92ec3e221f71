"""64-bit references of the 8-bit layer and the block norms (not a test module).

Plain torch in float64 on whatever device the inputs are on; shares nothing
with the library.  Each norm reference also gives, per output, the sum of the
magnitudes that enter it, from which the tests derive their bounds."""
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def quantize_rows(v64):
    """(unrounded quotients 127 v / max|v|, scales) of float64 rows."""
    top = v64.abs().amax(1, keepdim=True)
    q = torch.where(top > 0, v64 * 127 / torch.where(top > 0, top, 1.0), 0.0)
    return q, top[:, 0] / 127


def product(A, a_scales, W, w_scales, bias, transposed):
    """(Y, magnitude of its terms) in float64; the integer sums are exact there."""
    a, w = A.double(), W.double()
    acc = a @ (w if transposed else w.t())
    y = acc * a_scales.double()[:, None]
    if w_scales is not None:
        y = y * w_scales.double()
    big = y.abs()
    if bias is not None:
        y = y + bias.double()
        big = big + bias.double().abs()
    return y, big


def norm_forward(x, y, pre, post, gate, alpha, off, eps):
    """float64 inputs -> dict of residual (before its rounding) and its magnitude, rstd_y."""
    if y is None:
        return {"residual": x, "big": x.abs(), "rstd_y": None}
    t, ry = y, None
    if post is not None:
        ry = 1 / torch.sqrt((y * y).mean(1) + eps)
        t = t * ry[:, None] * (post + off)
    if gate is not None:
        t = t * gate
    return {"residual": x + alpha * t, "big": x.abs() + (alpha * t).abs(), "rstd_y": ry}


def norm_of(r, pre, off, eps):
    rr = 1 / torch.sqrt((r * r).mean(1) + eps)
    return r * rr[:, None] * (pre + off), rr


def norm_backward(dn, dres, r, rstd, y, pre, post, gate, alpha, off):
    """float64 inputs -> {name: (gradient, magnitude of its terms)}."""
    C = r.shape[1]
    rr = rstd[1][:, None]
    xh, w = r * rr, pre + off
    dh = dn * w
    dr = rr * (dh - xh * (dh * xh).sum(1, keepdim=True) / C)
    A = rr * (dn.abs() * w.abs() + xh.abs() * (dh * xh).abs().sum(1, keepdim=True) / C)
    if dres is not None:
        dr, A = dr + dres, A + dres.abs()
    out = {"d_x": (dr, A), "d_pre_weight": ((dn * xh).sum(0), (dn * xh).abs().sum(0))}
    if y is None:
        return out
    dt, D = alpha * dr, abs(alpha) * A
    yh = y * rstd[0][:, None] if post is not None else y
    if gate is not None:
        u = yh * (post + off) if post is not None else y
        g, G = dt * u, D * u.abs()
        out["d_gate"] = (g.sum(0), G.sum(0)) if gate.dim() == 1 else (g, G)
        dt, D = dt * gate, D * gate.abs()
    if post is not None:
        out["d_post_weight"] = ((dt * yh).sum(0), (D * yh.abs()).sum(0))
        dt, D = dt * (post + off), D * (post + off).abs()
        ry = rstd[0][:, None]
        dt = ry * (dt - yh * (dt * yh).sum(1, keepdim=True) / C)
        D = ry * (D + yh.abs() * (D * yh.abs()).sum(1, keepdim=True) / C)
    out["d_y"] = (dt, D)
    return out


def assert_within(got, want, bound, what):
    """|got - want| <= bound per element; infinities and NaN in the same places."""
    got = got.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    fine = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), fine), f"{what}: finite in other places"
    over = (got - want).abs()[fine] - bound[fine]
    if over.numel() and over.max() > 0:
        i = int(over.argmax())
        raise AssertionError(f"{what}: {int((over > 0).sum())} of {over.numel()} outside; worst "
                             f"got {got[fine][i].item():.9g} want {want[fine][i].item():.9g} "
                             f"bound {bound[fine][i].item():.3g}")

"""Block norms whose blocks walk over several rows of odd width (rows begin at either half of a word), and the
overlaps of outputs with inputs that the header allows.

Bounds as in test_gpu_block_norm: statistics within 64 * 2^-24, what is formed from them within 128 * 2^-24 of
the magnitudes that enter, column sums (rows + 128) * 2^-24, and the rounding to bf16."""
import pytest
import torch

import gemv_w4a16_groupwise_b200 as w4
from test_gpu_block_norm import BF, _backward, _call, _case, _check_backward, _check_forward

pytestmark = pytest.mark.gpu

# blocks on 148 SMs: forward 1184 to 1024, 592 to 4096, 296 to 8192, 148 beyond; backward half as many at most
SHAPES = [(5000, 65), (3001, 999), (2000, 2047), (1500, 4095), (1001, 8191), (700, 16383), (4000, 1), (3000, 7)]


@pytest.mark.parametrize("M,C", SHAPES)
@pytest.mark.parametrize("gate", [None, "channel", "token"])
@pytest.mark.parametrize("post", [False, True])
def test_many_odd_rows(cuda_device, M, C, gate, post):
    s = _case(M, C, post, gate, cuda_device)
    f = _call(s, 0.5, 0.0, keep_rstd=True)
    _check_forward(s, f, 0.5, 0.0)
    q = _call(s, 0.5, 0.0, quantize=True)
    assert torch.equal(q.residual, f.residual)
    _check_forward(s, q, 0.5, 0.0)
    for dres in (True, False):
        g = _backward(s, f, 0.5, 0.0, dres=dres)
        _check_backward(s, f, g, 0.5, 0.0, dres=dres)
        for a, b in zip(g, _backward(s, f, 0.5, 0.0, dres=dres)):
            assert (a is None and b is None) or torch.equal(a, b)


@pytest.mark.parametrize("M,C", SHAPES + [(2000, 1024), (900, 4096)])
@pytest.mark.parametrize("where", ["x", "y"])
@pytest.mark.parametrize("quantize", [False, True])
def test_residual_in_place(cuda_device, M, C, where, quantize):
    s = _case(M, C, True, "token", cuda_device)
    want = _call(s, 0.5, 0.0, quantize=quantize)
    f = _call(s, 0.5, 0.0, quantize=quantize, residual_out=s[where])
    assert f.residual is s[where] and torch.equal(f.residual, want.residual) and torch.equal(f.normed, want.normed)
    assert not quantize or torch.equal(f.scales, want.scales)


def _backward_into(s, f, d_x, d_y):
    """The C function with outputs of the caller's."""
    lib = w4.library()
    M, C = d_x.shape
    kind = {1: 1, 2: 2}[s["gate"].dim()]
    d_pre, d_post, d_gate = torch.empty_like(s["pre"]), torch.empty_like(s["post"]), torch.empty_like(s["gate"])
    ws = torch.empty(lib.w4_block_norm_workspace_bytes(M, C), dtype=torch.uint8, device=d_x.device)
    p = lambda t: t.data_ptr()  # noqa: E731
    st = lib.w4_block_norm_backward(p(s["dn"]), p(s["dres"]), p(f.residual), p(f.rstd), p(s["y"]), M, C, p(s["post"]),
                                    p(s["gate"]), kind, 0.5, p(s["pre"]), 0.0, p(d_x), p(d_y), p(d_pre), p(d_post),
                                    p(d_gate), p(ws), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert st == 0
    return d_x, d_y, d_pre, d_post, d_gate


@pytest.mark.parametrize("M,C", SHAPES + [(2000, 1024), (900, 4096), (500, 16384)])
@pytest.mark.parametrize("gate", ["channel", "token"])
def test_gradients_in_place(cuda_device, M, C, gate):
    s = _case(M, C, True, gate, cuda_device)
    f = _call(s, 0.5, 0.0, keep_rstd=True)
    want = _backward(s, f, 0.5, 0.0)
    for x_at, y_at in (("dres", None), ("dn", None), (None, "y"), ("dres", "y"), ("dn", "y")):
        t = {k: (v.clone() if torch.is_tensor(v) else v) for k, v in s.items()}
        d_x = t[x_at] if x_at else torch.empty(M, C, dtype=BF, device=cuda_device)
        d_y = t[y_at] if y_at else torch.empty(M, C, dtype=BF, device=cuda_device)
        for a, b in zip(_backward_into(t, f, d_x, d_y), want):
            assert torch.equal(a, b), (x_at, y_at)

"""Block norms on the GPU against 64 bits, and a run of block norm, 8-bit and
4-bit products as a model uses them.

Bounds.  Row sums of C squares (or products) are fp32 sums of at most 16 terms
in a thread, 5 shuffles and 32 warps: 53 half steps at most, so a statistic is
within 64 * 2^-24 and everything formed from it within 128 * 2^-24 of the
magnitudes that enter, plus the rounding to bf16.  Column sums run over the
rows: (rows + 128) * 2^-24 of the magnitudes."""
import pytest
import torch

import gemv_w4a16_groupwise_b200 as w4
import w8_reference as ref

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
U = 2.0 ** -24


def _case(M, C, post, gate, dev, off=0.0, seed=0):
    g = torch.Generator(device=dev)
    g.manual_seed(M * 31 + C + seed)
    r = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
    return {"x": (r(M, C) * 2).to(BF), "y": (r(M, C) * 3).to(BF), "pre": (1 - off + 0.2 * r(C)).to(BF),
            "post": (1 - off + 0.2 * r(C)).to(BF) if post else None,
            "gate": {None: None, "channel": r(C).to(BF), "token": r(M, C).to(BF)}[gate],
            "dn": r(M, C).to(BF), "dres": r(M, C).to(BF)}


def _d(t):
    return None if t is None else t.double()


def _call(s, alpha, off, eps=1e-5, **k):
    return w4.w4_block_norm(s["x"], s["y"], pre_weight=s["pre"], post_weight=s["post"], gate=s["gate"],
                            residual_scale=alpha, weight_offset=off, eps=eps, **k)


def _check_forward(s, f, alpha, off, eps=1e-5):
    y = s["y"]
    want = ref.norm_forward(_d(s["x"]), _d(y), _d(s["pre"]), _d(s["post"]), _d(s["gate"]), alpha, off, eps)
    ref.assert_within(f.residual, want["residual"], 2.0 ** -8 * want["residual"].abs() + 128 * U * want["big"],
                      "residual")
    n, rr = ref.norm_of(f.residual.double(), _d(s["pre"]), off, eps)
    if f.scales is None:
        ref.assert_within(f.normed, n, (2.0 ** -8 + 128 * U) * n.abs(), "normed")
    else:
        q, sc = ref.quantize_rows(n)
        assert ((f.scales.double() - sc).abs() <= 128 * U * sc).all()
        # the values and their maximum are within 128 steps each
        assert ((f.normed.double() - q).abs() <= 0.5 + 256 * U * 127).all()
    if f.rstd is not None:
        ref.assert_within(f.rstd[1], rr, 64 * U * rr, "rstd")
        if s["post"] is not None:
            ref.assert_within(f.rstd[0], want["rstd_y"], 64 * U * want["rstd_y"], "rstd of y")
        else:
            assert (f.rstd[0] == 0).all()


def _check_backward(s, f, g, alpha, off, dres=True):
    M = s["dn"].shape[0]
    want = ref.norm_backward(_d(s["dn"]), _d(s["dres"]) if dres else None, _d(f.residual), _d(f.rstd), _d(s["y"]),
                             _d(s["pre"]), _d(s["post"]), _d(s["gate"]), alpha, off)
    for name, value in g._asdict().items():
        assert (value is None) == (name not in want), name
        if value is None:
            continue
        w, big = want[name]
        steps = M + 128 if w.dim() == 1 else 128
        assert value.dtype == BF
        ref.assert_within(value, w, 2.0 ** -8 * w.abs() + 2 * steps * U * big, name)


def _backward(s, f, alpha, off, dres=True):
    return w4.w4_block_norm_backward(s["dn"], f.residual, f.rstd, s["y"], d_residual=s["dres"] if dres else None,
                                     pre_weight=s["pre"], post_weight=s["post"], gate=s["gate"],
                                     residual_scale=alpha, weight_offset=off)


KINDS = [(False, None), (True, None), (False, "channel"), (True, "channel"), (False, "token"), (True, "token")]
WIDTHS = [1, 7, 8, 64, 129, 1000, 1023, 1024, 1032, 2047, 2048, 2056, 4096, 4099, 5120, 8192, 8200, 12001, 16383,
          16384]


@pytest.mark.parametrize("C", WIDTHS)
@pytest.mark.parametrize("k", range(len(KINDS)))
def test_forward_and_backward(cuda_device, C, k):
    post, gate = KINDS[k]
    M = (1, 3, 40, 300, 5, 2)[(k + WIDTHS.index(C)) % 6]
    alpha, off = ((1.0, 0.0), (0.22, 1.0))[(k + C) % 2]
    s = _case(M, C, post, gate, cuda_device, off)
    f = _call(s, alpha, off, keep_rstd=True)
    assert f.scales is None
    _check_forward(s, f, alpha, off)
    q = _call(s, alpha, off, quantize=True)
    assert q.rstd is None and torch.equal(q.residual, f.residual)
    _check_forward(s, q, alpha, off)
    g = _backward(s, f, alpha, off)
    _check_backward(s, f, g, alpha, off)
    for a, b in zip(g, _backward(s, f, alpha, off)):       # the same bits again
        assert (a is None and b is None) or torch.equal(a, b)
    _check_backward(s, f, _backward(s, f, alpha, off, dres=False), alpha, off, dres=False)


@pytest.mark.parametrize("M,C", [(1000, 64), (5000, 256), (2000, 2048), (900, 4100)])
def test_many_rows(cuda_device, M, C):
    s = _case(M, C, True, "channel", cuda_device)
    f = _call(s, 0.5, 0.0, keep_rstd=True)
    _check_forward(s, f, 0.5, 0.0)
    _check_backward(s, f, _backward(s, f, 0.5, 0.0), 0.5, 0.0)


@pytest.mark.parametrize("C", [9, 512, 4096])
def test_without_a_block_before(cuda_device, C):
    s = _case(6, C, False, None, cuda_device)
    s["y"] = None
    f = w4.w4_block_norm(s["x"], pre_weight=s["pre"], keep_rstd=True)
    assert f.residual is s["x"]
    _check_forward(s, f, 1.0, 0.0)
    _check_backward(s, f, _backward(s, f, 1.0, 0.0), 1.0, 0.0)


@pytest.mark.parametrize("where", ["x", "y"])
@pytest.mark.parametrize("C", [100, 4096])
def test_in_place(cuda_device, where, C):
    s = _case(33, C, True, "token", cuda_device)
    want = _call(s, 0.5, 0.0)
    f = _call(s, 0.5, 0.0, residual_out=s[where])
    assert f.residual is s[where]
    assert torch.equal(f.residual, want.residual) and torch.equal(f.normed, want.normed)


@pytest.mark.parametrize("C", [24, 4096])
def test_zero_and_poisoned_rows(cuda_device, C):
    s = _case(6, C, True, "channel", cuda_device)
    s["x"][0] = 0
    s["y"][0] = 0                       # residual 0: norm of a zero row is 0
    s["x"][1, C // 2] = float("nan")
    s["y"][2, 0] = float("inf")
    s["y"][3] = 0
    f, q = _call(s, 1.0, 0.0), _call(s, 1.0, 0.0, quantize=True)
    assert (f.residual[0] == 0).all() and (f.normed[0] == 0).all() and q.scales[0] == 0 and not q.normed[0].any()
    for r in (1, 2):
        assert torch.isnan(f.normed[r]).any() and torch.isnan(q.scales[r]) and not q.normed[r].any()
    for r in (3, 4, 5):
        assert torch.isfinite(f.normed[r]).all() and torch.isfinite(q.scales[r])
    keep = [3, 4, 5]
    one = {k: (v[keep].contiguous() if k in ("x", "y") else v) for k, v in s.items()}
    again = _call(one, 1.0, 0.0)
    assert torch.equal(again.normed, f.normed[keep]) and torch.equal(again.residual, f.residual[keep])


@pytest.mark.parametrize("C", [8192, 8191])
def test_offsets_past_32_bits(cuda_device, C):
    """More than 2^31 values in a tensor: rows at the end are what they are alone."""
    dev = cuda_device
    M = 2 ** 31 // C + 300
    M += (M % 2) ^ 1                   # odd, so that odd rows begin at either half of a word
    s = _case(8, C, True, "channel", dev)
    big = {**s, **{k: s[k].repeat((M + 7) // 8, 1)[:M].contiguous() for k in ("x", "y", "dn", "dres")}}
    f, q = _call(big, 0.5, 0.0, keep_rstd=True), _call(big, 0.5, 0.0, quantize=True)
    g = _backward(big, f, 0.5, 0.0)
    one = {**s, **{k: big[k][:8].contiguous() for k in ("x", "y", "dn", "dres")}}
    f1, q1 = _call(one, 0.5, 0.0, keep_rstd=True), _call(one, 0.5, 0.0, quantize=True)
    g1 = _backward(one, f1, 0.5, 0.0)
    for lo in (0, 8 * (M // 16), (M // 8 - 1) * 8):
        at = slice(lo, lo + 8)
        assert torch.equal(f.residual[at], f1.residual) and torch.equal(f.normed[at], f1.normed)
        assert torch.equal(q.normed[at], q1.normed) and torch.equal(q.scales[at], q1.scales)
        assert torch.equal(g.d_x[at], g1.d_x) and torch.equal(g.d_y[at], g1.d_y)


def test_zero_scale_leaves_the_residual(cuda_device):
    s = _case(4, 320, True, "token", cuda_device)
    assert torch.equal(_call(s, 0.0, 0.0).residual, s["x"])


def test_graph_of_a_training_step(cuda_device):
    """Forward, products and backward in one captured graph, replayed on new inputs, twice side by side."""
    dev = cuda_device
    M, C, N = 70, 512, 640
    s = _case(M, C, True, "channel", dev)
    W, ws = w4.w8_quantize_rows((torch.randn(N, C, device=dev) * 0.05).to(BF))
    dY = torch.randn(M, N, device=dev).to(BF)

    def step():
        f = _call(s, 0.5, 0.0, quantize=True, keep_rstd=True)
        y = w4.w8a8_gemm(f.normed, f.scales, W, ws)
        dn = w4.w8a8_linear(dY, W, ws, transposed=True)
        g = w4.w4_block_norm_backward(dn, f.residual, f.rstd, s["y"], pre_weight=s["pre"], post_weight=s["post"],
                                      gate=s["gate"], residual_scale=0.5)
        return [f.residual, y, *g]

    step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step()
        graphs.append((g, out))
    for turn in range(3):
        s["x"].copy_(torch.randn(M, C, device=dev).to(BF))
        dY.copy_(torch.randn(M, N, device=dev).to(BF))
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream(dev) for _ in graphs]
        for (g, out), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for _, out in graphs:
            for a, b in zip(out, want):
                assert torch.equal(a, b)


@pytest.mark.parametrize("M", [1, 5, 33, 260])
def test_blocks_in_a_row(cuda_device, M):
    """norm -> 8-bit products -> norm after and before -> 4-bit product, and the way back, each
    link against the 64-bit value of the link on the tensors that the link before gave."""
    dev = cuda_device
    C, H = 768, 1280
    s = _case(M, C, True, "channel", dev)
    g = torch.Generator(device=dev)
    g.manual_seed(M)
    r = lambda *z: torch.randn(z, generator=g, device=dev)  # noqa: E731
    up, up_s = w4.w8_quantize_rows((r(H, C) * 0.04).to(BF))
    down, down_s = w4.w8_quantize_rows((r(C, H) * 0.03).to(BF))
    bias = (r(H) * 0.01).to(BF)
    packed, scales, zeros = w4.w4_quantize_pack((r(512, C) * 0.02).to(BF), "groupwise", 128)

    first = w4.w4_block_norm(s["x"], pre_weight=s["pre"], quantize=True, keep_rstd=True)
    h = w4.w8a8_gemm(first.normed, first.scales, up, up_s, bias=bias)
    want, big = ref.product(first.normed, first.scales, up, up_s, bias, False)
    ref.assert_within(h, want, 2.0 ** -8 * want.abs() + 8 * U * big, "up")
    y = w4.w8a8_linear(h, down, down_s)
    hq, hs = w4.w8_quantize_rows(h)
    want, big = ref.product(hq, hs, down, down_s, None, False)
    ref.assert_within(y, want, 2.0 ** -8 * want.abs() + 8 * U * big, "down")
    s["y"] = y
    second = _call(s, 0.5, 0.0, keep_rstd=True)
    _check_forward(s, second, 0.5, 0.0)
    mm = w4.w4a16_gemm
    out = mm(second.normed, packed, scales, zeros, "groupwise", 128, N=512, K=C)
    assert torch.isfinite(out).all() and out.shape == (M, 512)

    dout = r(M, 512).to(BF)
    s["dn"] = mm(dout, packed, scales, zeros, "groupwise", 128, N=512, K=C, transposed=True)
    grad = _backward(s, second, 0.5, 0.0)
    _check_backward(s, second, grad, 0.5, 0.0)
    dh = w4.w8a8_linear(grad.d_y, down, down_s, transposed=True)
    q, qs = w4.w8_quantize_rows(grad.d_y, channel_scales=down_s)
    want, big = ref.product(q, qs, down, None, None, True)
    ref.assert_within(dh, want, 2.0 ** -8 * want.abs() + 8 * U * big, "down transposed")
    dn = w4.w8a8_linear(dh, up, up_s, transposed=True)
    last = w4.w4_block_norm_backward(dn, s["x"], first.rstd, d_residual=grad.d_x, pre_weight=s["pre"])
    s0 = {**s, "y": None, "post": None, "gate": None, "dn": dn, "dres": grad.d_x}
    _check_backward(s0, first, last, 1.0, 0.0)
    assert w4.w4_device_error() == 0


def test_arguments_the_native_call_leaves(cuda_device):
    """Whole-number scales and offsets go through the Python checks to the same kernel."""
    s = _case(9, 200, True, "token", cuda_device)
    a, b = _call(s, 1.0, 0.0, keep_rstd=True), _call(s, 1, 0, keep_rstd=True)
    for p, q in zip(a, b):
        assert (p is None and q is None) or torch.equal(p, q)
    for p, q in zip(_backward(s, a, 1.0, 0.0), _backward(s, b, 1, 0)):
        assert torch.equal(p, q)
    w = torch.nn.Parameter(s["pre"])
    assert torch.equal(w4.w4_block_norm(s["x"], s["y"], pre_weight=w).normed,
                       w4.w4_block_norm(s["x"], s["y"], pre_weight=s["pre"]).normed)


def test_binding_refusals(cuda_device):
    dev = cuda_device
    s = _case(4, 64, True, "channel", dev)
    with pytest.raises(ValueError):
        w4.w4_block_norm(s["x"], pre_weight=s["pre"], gate=s["gate"])
    with pytest.raises(ValueError):
        w4.w4_block_norm(s["x"], s["y"][:3].contiguous(), pre_weight=s["pre"])
    with pytest.raises(ValueError):
        w4.w4_block_norm(s["x"], s["y"], pre_weight=s["pre"][:32])
    with pytest.raises(ValueError):
        w4.w4_block_norm(s["x"], s["y"], pre_weight=s["pre"], gate=s["dn"][:, :32])
    with pytest.raises(TypeError):
        w4.w4_block_norm(s["x"].float(), s["y"], pre_weight=s["pre"])
    with pytest.raises(TypeError):
        w4.w4_block_norm(s["x"], s["y"], pre_weight=s["pre"].float())
    with pytest.raises(ValueError):
        w4.w4_block_norm(s["x"].t(), s["y"], pre_weight=s["pre"])
    with pytest.raises(ValueError):
        w4.w4_block_norm(s["x"], s["y"], pre_weight=s["pre"].cpu())
    with pytest.raises(ValueError):
        w4.w4_block_norm(s["x"], pre_weight=s["pre"], residual_out=s["y"])
    with pytest.raises(w4.W4Error):
        w4.w4_block_norm(s["x"], s["y"], pre_weight=s["pre"], eps=0.0)
    with pytest.raises(w4.W4Error):
        w4.w4_block_norm(torch.zeros(1, 16392, dtype=BF, device=dev), pre_weight=torch.zeros(16392, dtype=BF, device=dev))
    f = _call(s, 1.0, 0.0, keep_rstd=True)
    with pytest.raises(ValueError):
        w4.w4_block_norm_backward(s["dn"], f.residual, f.rstd[:1], s["y"], pre_weight=s["pre"])
    with pytest.raises(ValueError):
        w4.w4_block_norm_backward(s["dn"], f.residual, f.rstd, pre_weight=s["pre"], post_weight=s["post"])

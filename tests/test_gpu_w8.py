"""8-bit rows, products and the linear layer on the GPU against 64 bits.

Bounds.  Codes of bf16 rows are exact.  Scales: one division, half a step
(2^-24).  A product's integer sum is exact; its conversion to fp32, the product
of the two scales, the fma and the rounding to bf16 are one half step each:
2^-8 of the result and 4 * 2^-24 of the terms (doubled here for the second
order)."""
import pytest
import torch

import gemv_w4a16_groupwise_b200 as w4
import w8_reference as ref

pytestmark = pytest.mark.gpu


def _gen(seed, dev):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return g


def _codes(R, C, seed, dev, pad=0):
    """Random int8 rows over the whole range, rows 16-byte strided, garbage behind each row."""
    ld = (C + 15) // 16 * 16 + pad
    q = torch.randint(-128, 128, (R, ld), generator=_gen(seed, dev), device=dev, dtype=torch.int32).to(torch.int8)
    return q[:, :C]


def _bound(y, big):
    return 2.0 ** -8 * y.abs() + 8 * 2.0 ** -24 * big


def _check_product(M, N, K, tr, dev, bias=True, seed=0, pad=0):
    g = _gen(1000 + seed, dev)
    A, W = _codes(M, N if tr else K, seed + 1, dev, pad), _codes(N, K, seed + 2, dev, pad)
    a_s = torch.rand(M, generator=g, device=dev) + 0.01
    w_s = None if tr else torch.rand(N, generator=g, device=dev) * 0.1
    out_len = K if tr else N
    b = torch.randn(out_len, generator=g, device=dev).to(torch.bfloat16) if bias else None
    y = w4.w8a8_gemm(A, a_s, W, w_s, bias=b, transposed=tr)
    want, big = ref.product(A, a_s, W, w_s, b, tr)
    ref.assert_within(y, want, _bound(want, big), f"product {M}x{N}x{K} tr={tr}")
    return A, a_s, W, w_s, b, y


# ------------------------------------------------------------- quantize
def test_codes_are_the_exact_quotients_for_every_significand(cuda_device):
    """One row per significand of the maximum, holding every bf16 value of the ten binades below it."""
    rows = []
    for b in range(128, 256):
        bits = [(127 - d) << 7 | s for d in range(0, 11) for s in range(128)]
        v = torch.tensor(bits, dtype=torch.int16).view(torch.bfloat16).double()
        v = torch.where(v <= b / 128, v, torch.zeros_like(v))
        rows.append(torch.cat([torch.tensor([b / 128], dtype=torch.float64), v, -v]))
    X = torch.stack(rows)
    codes, scales = w4.w8_quantize_rows(X.to(cuda_device).to(torch.bfloat16))
    # in units of 2^-17 both sides are whole numbers: exact halves to even
    num, den = (X * 2 ** 17).long() * 127, (X[:, :1] * 2 ** 17).long()
    mag, lo = num.abs(), num.abs() // den
    rem2 = 2 * (mag % den)
    want = (lo + ((rem2 > den) | ((rem2 == den) & (lo % 2 == 1))).long()) * num.sign()
    assert torch.equal(codes.cpu().long(), want)
    s64 = X[:, 0] / 127
    assert ((scales.cpu().double() - s64).abs() <= 2.0 ** -24 * s64).all()


@pytest.mark.parametrize("R,C", [(1, 1), (3, 7), (2, 16), (5, 100), (4, 1001), (7, 2048), (3, 4096), (2, 8200),
                                 (3, 14336), (2, 28672), (2, 33000), (1, 128256), (700, 64), (2000, 4096), (7200, 999),
                                 (1800, 6001), (1000, 8192)])
@pytest.mark.parametrize("folded", [False, True])
def test_quantize_rows(cuda_device, R, C, folded):
    dev = cuda_device
    g = _gen(R * 7 + C, dev)
    X = (torch.randn(R, C, generator=g, device=dev) * 3).to(torch.bfloat16)
    ch = torch.rand(C, generator=g, device=dev) * 0.1 if folded else None
    codes, scales = w4.w8_quantize_rows(X, channel_scales=ch)
    assert codes.shape == (R, C) and codes.stride(0) % 16 == 0
    v = X.float() * ch if folded else X.float()
    q, s = ref.quantize_rows(v.double())
    # inv is within 2^-21 of 127 / max: at most 127 * 2^-21 beyond half a code; bf16 rows are exact
    assert ((codes.double() - q).abs() <= 0.5 + (127 * 2.0 ** -21 if folded else 0)).all()
    if not folded:
        assert torch.equal(codes.double(), torch.round(q))
    assert ((scales.double() - s).abs() <= 2.0 ** -24 * s).all()


@pytest.mark.parametrize("C", [5, 64, 4096, 40000])
def test_quantize_rows_extremes(cuda_device, C):
    dev = cuda_device
    X = torch.randn(9, C, generator=_gen(C, dev), device=dev)
    X[0] = 0
    X[1] = X[1].clamp(-1, 1) * 3.3e38
    X[2] *= 1e-38
    X[3] = 0
    X[3, C // 2] = 9.2e-41          # the smallest bf16 subnormal
    X[4, C - 1] = float("inf")
    X[5, 0] = float("nan")
    X[6, C // 2] = float("-inf")
    X[7] = -0.0
    X[8, 0] = 1e30                   # the others round to 0
    X = X.to(torch.bfloat16)
    codes, scales = w4.w8_quantize_rows(X)
    for r in (4, 5, 6):
        assert torch.isnan(scales[r]) and not codes[r].any()
    fine = [0, 1, 2, 3, 7, 8]
    q, s = ref.quantize_rows(X[fine].double())
    assert torch.equal(codes[fine].double(), torch.round(q))
    # a scale below fp32's normal range is off by up to half of 2^-149
    assert ((scales[fine].double() - s).abs() <= 2.0 ** -24 * s + 2.0 ** -150).all()
    W, ws = w4.w8_quantize_rows(torch.randn(32, C, device=dev).to(torch.bfloat16))
    y = w4.w8a8_linear(X, W, ws)
    assert torch.isnan(y[[4, 5, 6]]).all() and (y[[0, 7]] == 0).all() and torch.isfinite(y[[2, 3, 8]]).all()


def test_quantize_writes_only_its_rows(cuda_device):
    dev = cuda_device
    R, C = 5, 37
    buf = torch.full((R + 2, 64), 99, dtype=torch.int8, device=dev)
    sc = torch.full((R + 4,), 7.0, device=dev)
    X = torch.randn(R, C, device=dev).to(torch.bfloat16)
    w4.w8_quantize_rows(X, out=(buf[:R, :C], sc[:R]))
    c, s = w4.w8_quantize_rows(X)
    assert torch.equal(buf[:R, :C], c) and torch.equal(sc[:R], s)
    assert (buf[R:] == 99).all() and (buf[:, 48:] == 99).all() and (sc[R:] == 7).all()


# ------------------------------------------------------------- product
SHAPES = [(1, 1, 1), (1, 64, 64), (2, 33, 100), (4, 512, 2048), (1, 6144, 4096), (3, 4099, 1001), (7, 1000, 4096),
          (8, 256, 16384), (9, 2048, 2048), (16, 4096, 512), (17, 130, 144), (31, 96, 5000), (32, 1024, 1024),
          (33, 4099, 1001), (63, 512, 640), (64, 2048, 8192), (65, 300, 300), (100, 2048, 2048), (127, 257, 129),
          (128, 512, 2048), (129, 1024, 1023), (255, 4096, 256), (300, 700, 900), (513, 6144, 1024), (777, 4099, 1001),
          (1024, 512, 4096), (2050, 1028, 516), (4100, 70, 80), (70000, 40, 48)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("tr", [False, True])
def test_product(cuda_device, M, N, K, tr):
    _check_product(M, N, K, tr, cuda_device, bias=(M + N + K) % 2 == 0, seed=M + N + K)


@pytest.mark.parametrize("M", [1, 20, 200])
@pytest.mark.parametrize("tr", [False, True])
def test_product_longest_sum_does_not_overflow(cuda_device, M, tr):
    """All codes -128 over the longest sum that is taken: 2^14 * 131071 < 2^31."""
    dev = cuda_device
    L, O = 131071, 48
    N, K = (L, O) if tr else (O, L)
    A = torch.full((M, 131072), -128, dtype=torch.int8, device=dev)[:, :L]
    W = torch.full((N, (K + 15) // 16 * 16), -128, dtype=torch.int8, device=dev)[:, :K]
    a_s = torch.full((M,), 2.0 ** -31, device=dev)
    y = w4.w8a8_gemm(A, a_s, W, None if tr else torch.ones(N, device=dev), transposed=tr)
    want = torch.full((M, O), 16384.0 * L * 2.0 ** -31, dtype=torch.float64, device=dev)
    ref.assert_within(y, want, _bound(want, want), "longest sum")


@pytest.mark.parametrize("M", [1, 5, 40, 300])
@pytest.mark.parametrize("tr", [False, True])
def test_product_of_views_leaves_the_rest_alone(cuda_device, M, tr):
    """Rows inside a wider tensor, garbage behind them, an output inside guard rows."""
    dev = cuda_device
    N, K = 200, 333
    A, a_s, W, w_s, b, y = _check_product(M, N, K, tr, dev, seed=M, pad=48)
    guard = torch.full((M + 2, y.shape[1]), 3.0, dtype=torch.bfloat16, device=dev)
    # a row offset that keeps 16-byte alignment is not given for odd widths: use the first rows
    w4.w8a8_gemm(A, a_s, W, w_s, bias=b, transposed=tr, out=guard[:M])
    assert torch.equal(guard[:M], y) and (guard[M:] == 3).all()


def test_a_row_does_not_depend_on_the_rows_beside_it(cuda_device):
    dev = cuda_device
    N, K = 640, 1024
    X = torch.randn(300, K, device=dev).to(torch.bfloat16)
    W, ws = w4.w8_quantize_rows(torch.randn(N, K, device=dev).to(torch.bfloat16))
    whole = w4.w8a8_linear(X, W, ws)
    for lo, hi in ((0, 1), (3, 6), (0, 20), (100, 170), (150, 300)):
        assert torch.equal(w4.w8a8_linear(X[lo:hi], W, ws), whole[lo:hi])
    X2 = X.clone()
    X2[7] = float("nan")
    y = w4.w8a8_linear(X2, W, ws)
    keep = torch.arange(300, device=dev) != 7
    assert torch.isnan(y[7]).all() and torch.equal(y[keep], whole[keep])


# ------------------------------------------------------------- linear
@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("tr", [False, True])
def test_linear_is_quantize_then_product(cuda_device, M, N, K, tr):
    dev = cuda_device
    g = _gen(M + 3 * N + 5 * K, dev)
    A = torch.randn(M, N if tr else K, generator=g, device=dev).to(torch.bfloat16)
    W, ws = w4.w8_quantize_rows((torch.randn(N, K, generator=g, device=dev) * 0.02).to(torch.bfloat16))
    b = torch.randn(K if tr else N, generator=g, device=dev).to(torch.bfloat16)
    y = w4.w8a8_linear(A, W, ws, bias=b, transposed=tr)
    a, a_s = w4.w8_quantize_rows(A, channel_scales=ws if tr else None)
    assert torch.equal(y, w4.w8a8_gemm(a, a_s, W, None if tr else ws, bias=b, transposed=tr))


def test_transposed_is_the_adjoint(cuda_device):
    """<dY, X W^T> = <dY W, X> up to the quantization of tokens, which is bounded per element:
    half a code of each row, summed over the row against the other operand's magnitudes."""
    dev = cuda_device
    M, N, K = 40, 300, 500
    g = _gen(5, dev)
    X = torch.randn(M, K, generator=g, device=dev).to(torch.bfloat16)
    dY = torch.randn(M, N, generator=g, device=dev).to(torch.bfloat16)
    W, ws = w4.w8_quantize_rows(torch.randn(N, K, generator=g, device=dev).to(torch.bfloat16))
    w = W.double() * ws.double()[:, None]
    y, dx = w4.w8a8_linear(X, W, ws).double(), w4.w8a8_linear(dY, W, ws, transposed=True).double()
    sx = X.double().abs().amax(1, keepdim=True) / 127
    sd = (dY.double() * ws.double()).abs().amax(1, keepdim=True) / 127
    by = 0.5 * sx * w.abs().sum(1) + 2.0 ** -7 * y.abs()
    # codes stand for dY * ws: half a code there is half a code over ws of dY
    bx = 0.5 * sd * W.double().abs().sum(0) + 2.0 ** -7 * dx.abs()
    true = (dY.double() * (X.double() @ w.t())).sum()
    assert abs((dY.double() * y).sum() - true) <= (dY.double().abs() * by).sum()
    assert abs((dx * X.double()).sum() - true) <= (X.double().abs() * bx).sum()


@pytest.mark.parametrize("M", [1, 2, 3, 4, 6])
@pytest.mark.parametrize("K", [64, 1000, 4096])
def test_poisoned_and_zero_tokens_of_a_small_batch(cuda_device, M, K):
    """A token with a NaN or an infinity is NaN throughout and its neighbours are what they are
    alone; a token of zeros gives the bias; weights with scale 0 or NaN reach their channel only."""
    dev = cuda_device
    N = 100
    g = _gen(M + K, dev)
    X = torch.randn(M, K, generator=g, device=dev).to(torch.bfloat16)
    Wb = torch.randn(N, K, generator=g, device=dev).to(torch.bfloat16)
    Wb[7] = 0
    Wb[9, K - 1] = float("nan")
    W, ws = w4.w8_quantize_rows(Wb)
    b = torch.randn(N, generator=g, device=dev).to(torch.bfloat16)
    clean = w4.w8a8_linear(X, W, ws, bias=b)
    assert torch.isnan(clean[:, 9]).all() and torch.equal(clean[:, 7], b[7].expand(M))
    fine = [n for n in range(N) if n != 9]
    assert torch.isfinite(clean[:, fine]).all()
    for bad in (float("nan"), float("inf"), float("-inf"), 0.0):
        X2 = X.clone()
        if bad == 0.0:
            X2[M - 1] = 0
        else:
            X2[M - 1, K // 2] = bad
        y = w4.w8a8_linear(X2, W, ws, bias=b)
        assert torch.equal(y[:M - 1, fine], clean[:M - 1, fine])
        if bad == 0.0:
            assert torch.equal(y[M - 1, fine], b[fine])
        else:
            assert torch.isnan(y[M - 1]).all()


@pytest.mark.parametrize("M,N,K,tr", [(40, 4096, 14336, False), (5, 3000, 130000, False), (20, 120000, 256, True),
                                      (130, 512, 20000, False), (600, 1024, 9000, True)])
def test_product_with_a_cut_reduction(cuda_device, M, N, K, tr):
    """Long sums over few tiles, whose reduction is shared by many blocks."""
    _check_product(M, N, K, tr, cuda_device, seed=M)


def test_offsets_past_32_bits(cuda_device):
    """More than 2^31 values in the tokens, their codes and the output: rows at the end are what
    they are alone."""
    dev = cuda_device
    M, N, K = 70000, 32000, 32000            # 2.24e9 elements each
    g = _gen(3, dev)
    X = torch.empty(M, K, dtype=torch.bfloat16, device=dev)
    for lo in range(0, M, 10000):
        X[lo:lo + 10000] = torch.randn(min(10000, M - lo), K, generator=g, device=dev)
    W, ws = w4.w8_quantize_rows(torch.randn(N, K, generator=g, device=dev).to(torch.bfloat16))
    codes, scales = w4.w8_quantize_rows(X)
    y = w4.w8a8_gemm(codes, scales, W, ws)
    for lo in (0, 33000, 67100, 69990):       # 67109 rows of 32000 are 2^31 values
        rows = X[lo:lo + 10].clone()
        c, s = w4.w8_quantize_rows(rows)
        assert torch.equal(codes[lo:lo + 10], c) and torch.equal(scales[lo:lo + 10], s)
        assert torch.equal(y[lo:lo + 10], w4.w8a8_gemm(c, s, W, ws))
    del y, codes
    d = w4.w8a8_linear(X, W, ws, transposed=True)
    for lo in (0, 69990):
        assert torch.equal(d[lo:lo + 10], w4.w8a8_linear(X[lo:lo + 10].clone(), W, ws, transposed=True))


# ------------------------------------------------------------- use
def test_graph_replays_and_two_streams(cuda_device):
    dev = cuda_device
    N, K = 1536, 2048
    W, ws = w4.w8_quantize_rows((torch.randn(N, K, device=dev) * 0.02).to(torch.bfloat16))
    xs = [torch.randn(M, K, device=dev).to(torch.bfloat16) for M in (1, 12, 130)]
    want = [w4.w8a8_linear(x, W, ws) for x in xs]
    grads = [torch.randn(x.shape[0], N, device=dev).to(torch.bfloat16) for x in xs]
    want_t = [w4.w8a8_linear(d, W, ws, transposed=True) for d in grads]
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):           # two graphs of the same calls: nothing is shared between them
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = [w4.w8a8_linear(x, W, ws) for x in xs] + [w4.w8a8_linear(d, W, ws, transposed=True) for d in grads]
        graphs.append((g, out))
    streams = [torch.cuda.Stream(dev) for _ in graphs]
    for _ in range(3):
        for (g, out), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                for o in out:
                    o.zero_()
                g.replay()
        torch.cuda.synchronize()
        for _, out in graphs:
            for o, w in zip(out, want + want_t):
                assert torch.equal(o, w)
    x2 = [x * 2 for x in xs]
    for x, y in zip(xs, x2):
        x.copy_(y)
    graphs[0][0].replay()
    torch.cuda.synchronize()
    for o, x in zip(graphs[0][1], x2):
        assert torch.equal(o, w4.w8a8_linear(x, W, ws))
    assert w4.w4_device_error() == 0


def test_first_calls_of_a_process_can_be_captured(cuda_device):
    """A fresh process whose first calls are made under stream capture."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(w4.__file__)))
    code = """
import torch, gemv_w4a16_groupwise_b200 as w4
x = torch.randn(20, 512, device="cuda").to(torch.bfloat16)
w = torch.randn(640, 512, device="cuda").to(torch.bfloat16)
pre = torch.ones(512, device="cuda", dtype=torch.bfloat16)
def calls():
    W, ws = w4.w8_quantize_rows(w)
    f = w4.w4_block_norm(x, x, pre_weight=pre, quantize=True, keep_rstd=True)
    y = w4.w8a8_gemm(f.normed, f.scales, W, ws)
    d = w4.w8a8_linear(y, W, ws, transposed=True)
    return [y, w4.w8a8_linear(x[:2], W, ws), *w4.w4_block_norm_backward(d, f.residual, f.rstd, x, pre_weight=pre)[:3]]
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    out = calls()
g.replay()
torch.cuda.synchronize()
for a, b in zip(out, calls()):
    assert torch.equal(a, b)
assert w4.w4_device_error() == 0
print("captured")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_weights_written_right_before_the_product(cuda_device):
    """Weights quantized by the call before, again and again into the same storage: a product
    never sees older ones."""
    dev = cuda_device
    N, K = 2048, 1024
    ws = [(torch.randn(N, K, device=dev) * 0.02).to(torch.bfloat16) for _ in range(4)]
    xs = [torch.randn(M, K, device=dev).to(torch.bfloat16) for M in (1, 8, 200)]
    want = [[w4.w8a8_linear(x, *w4.w8_quantize_rows(w)) for x in xs] for w in ws]
    torch.cuda.synchronize()
    codes = torch.empty(N, K, dtype=torch.int8, device=dev)
    scales = torch.empty(N, device=dev)
    got = []
    for w in ws:
        row = []
        for x in xs:
            codes.zero_()
            w4.w8_quantize_rows(w, out=(codes, scales))
            row.append(w4.w8a8_linear(x, codes, scales))
        got.append(row)
    for a, b in zip(want, got):
        for p, q in zip(a, b):
            assert torch.equal(p, q)


def test_parameters_out_and_odd_arguments(cuda_device):
    """What the native calls take, leave to the Python checks, and give back."""
    dev = cuda_device
    X = torch.nn.Parameter(torch.randn(5, 96, device=dev).to(torch.bfloat16))
    W, ws = w4.w8_quantize_rows(torch.randn(40, 96, device=dev).to(torch.bfloat16))
    y = w4.w8a8_linear(X, W, ws)
    assert type(y) is torch.Tensor and not y.requires_grad and y.is_contiguous()
    out = torch.empty_like(y)
    assert w4.w8a8_linear(X, W, ws, out=out) is out and torch.equal(out, y)
    a, a_s = w4.w8_quantize_rows(X)
    assert w4.w8a8_gemm(a, a_s, W, ws, out=out) is out and torch.equal(out, y)
    assert torch.equal(w4.w8a8_linear(X, W, ws, transposed=0), y)
    one, one_s = w4.w8_quantize_rows(torch.randn(1, 96, device=dev).to(torch.bfloat16))   # a single weight row
    got = w4.w8a8_linear(X, one, one_s)
    wide = torch.cat([one, one])
    assert torch.equal(got, w4.w8a8_linear(X, wide, one_s.repeat(2))[:, :1])
    with torch.inference_mode():
        assert torch.equal(w4.w8a8_linear(X, W, ws), y)
    strided = torch.zeros(5, 200, dtype=torch.bfloat16, device=dev)[:, :96]
    with pytest.raises(ValueError):
        w4.w8a8_linear(strided, W, ws)


def test_binding_refusals(cuda_device):
    dev = cuda_device
    q, s = torch.zeros(4, 32, dtype=torch.int8, device=dev), torch.ones(4, device=dev)
    x = torch.zeros(2, 32, dtype=torch.bfloat16, device=dev)
    with pytest.raises(ValueError):
        w4.w8a8_linear(x, torch.zeros(4, 24, dtype=torch.int8, device=dev), s)       # rows off 16 bytes
    with pytest.raises(ValueError):
        w4.w8a8_linear(x[:, :24].contiguous(), torch.zeros(1, 24, dtype=torch.int8, device=dev)[:, :24],
                       torch.ones(2, device=dev))
    with pytest.raises(ValueError):
        w4.w8a8_linear(x, q.t().contiguous().t(), s)
    with pytest.raises(TypeError):
        w4.w8a8_linear(x, q.to(torch.uint8), s)
    with pytest.raises(TypeError):
        w4.w8a8_linear(x.float(), q, s)
    with pytest.raises(TypeError):
        w4.w8a8_linear(x, q, s.half())
    with pytest.raises(ValueError):
        w4.w8a8_linear(x, q, s.cpu())
    with pytest.raises(ValueError):
        w4.w8a8_linear(x, q, s[:3])
    with pytest.raises(ValueError):
        w4.w8a8_linear(x, q, s, bias=torch.zeros(5, dtype=torch.bfloat16, device=dev))
    with pytest.raises(ValueError):
        w4.w8a8_linear(x, q, s, out=torch.zeros(3, 4, dtype=torch.bfloat16, device=dev))
    with pytest.raises(ValueError):
        w4.w8a8_linear(x, torch.empty_strided((4, 17), (16, 1), dtype=torch.int8, device=dev), s)
    # a last row that could not be read in 16-byte pieces
    tight = torch.zeros(3 * 32 + 20, dtype=torch.int8, device=dev).as_strided((4, 20), (32, 1))
    with pytest.raises(ValueError):
        w4.w8a8_linear(torch.zeros(2, 20, dtype=torch.bfloat16, device=dev), tight, s)
    with pytest.raises(w4.W4Error):
        w4.w8_quantize_rows(torch.zeros(0, 8, dtype=torch.bfloat16, device=dev))
    with pytest.raises(w4.W4Error):
        w4.w8a8_linear(x[:0], q, s)

"""The bounded waits of the 8-bit product's pair kernel, made to run out without a GPU fault.

Every producer stops before its first or its second tile (nothing of the rest is issued, but for the weights of
a linear call that are asked for ahead, which land) and the limit is 1 ms: both CTAs of a pair have to give up,
report it, and leave the output of the tiles that were not finished alone.  No tile of these problems is shared
between pairs."""
import pytest
import torch

import gemv_w4a16_groupwise_b200 as w4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K,first", [(20, 2048, 512, 0), (200, 4096, 1024, 0), (600, 2048, 4096, 0),
                                         (2048, 6144, 512, 0), (2048, 6144, 512, 1)])
@pytest.mark.parametrize("tr", [False, True])
@pytest.mark.parametrize("call", ["gemm", "linear"])
def test_both_ctas_of_a_pair_give_up(cuda_device, M, N, K, first, tr, call):
    dev = cuda_device
    if tr:
        N, K = K, N
    g = torch.Generator(device=dev).manual_seed(M + N)
    W, ws = w4.w8_quantize_rows(torch.randn(N, K, generator=g, device=dev).to(torch.bfloat16))
    A = torch.randn(M, N if tr else K, generator=g, device=dev).to(torch.bfloat16)
    a, a_s = w4.w8_quantize_rows(A, channel_scales=ws if tr else None)
    out = torch.full((M, K if tr else N), float("nan"), dtype=torch.bfloat16, device=dev)
    assert w4.library().w8a8_workspace_bytes(M, N, K, int(tr)) == 0      # whole tiles only

    def run(o):
        if call == "linear":
            return w4.w8a8_linear(A, W, ws, transposed=tr, out=o)
        return w4.w8a8_gemm(a, a_s, W, None if tr else ws, transposed=tr, out=o)

    want = run(None).clone()
    assert w4.w4_device_error() == 0
    try:
        w4.w4_debug_set_wait_limit(1_000_000)
        w4.w4_debug_withhold_stage(first)
        run(out)
        torch.cuda.synchronize()
        code = w4.w4_device_error()
    finally:
        w4.w4_debug_withhold_stage(-1)
        w4.w4_debug_set_wait_limit(0)
    assert code in (1, 3, 4), code
    untouched = torch.isnan(out)
    if first == 0:
        assert untouched.all()
    else:       # pairs that got as far as their second tile had stored their first
        assert untouched.any() and torch.equal(out[~untouched], want[~untouched])
    assert w4.w4_device_error() == 0
    for _ in range(3):
        assert torch.equal(run(out), want)
    assert w4.w4_device_error() == 0

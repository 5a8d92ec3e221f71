"""First calls of the 8-bit layer on several threads at once."""
import threading
import time

import pytest
import torch

import gemv_w4a16_groupwise_b200 as w4
from gemv_w4a16_groupwise_b200 import build


def test_the_binding_is_built_once(monkeypatch):
    real, builds = build.build_binding, []

    def slow(*args, **kwargs):
        builds.append(threading.get_ident())
        time.sleep(0.3)
        return real(*args, **kwargs)

    monkeypatch.setattr(build, "build_binding", slow)
    monkeypatch.setattr(w4._Torch, "torch", None)
    monkeypatch.setattr(w4._Torch, "native", None)
    x, q, s = torch.zeros(2, 16, dtype=torch.bfloat16), torch.zeros(4, 16, dtype=torch.int8), torch.ones(4)
    calls = [lambda: w4.w8_quantize_rows(x), lambda: w4.w8_quantize_rows(x, out=(q, s)),
             lambda: w4.w8a8_linear(x, q, s), lambda: w4.w4_block_norm(x, pre_weight=x[0])] * 2
    start, seen = threading.Barrier(len(calls)), []

    def work(call):
        start.wait()
        try:
            call()
        except Exception as e:      # noqa: BLE001 -- host tensors are refused, by a ValueError
            seen.append(type(e))

    threads = [threading.Thread(target=work, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join(30)
    assert seen == [ValueError] * len(calls)
    assert len(builds) == 1
    assert w4._Torch.native is not None


@pytest.mark.gpu
def test_threads_with_streams_of_their_own(cuda_device, monkeypatch):
    """First calls on four threads, each on its stream, give what one thread gives."""
    dev = cuda_device
    g = torch.Generator(device=dev).manual_seed(0)
    W, ws = w4.w8_quantize_rows(torch.randn(640, 512, generator=g, device=dev).to(torch.bfloat16))
    xs = [torch.randn(m, 512, generator=g, device=dev).to(torch.bfloat16) for m in (1, 7, 40, 300)]
    want = [w4.w8a8_linear(x, W, ws) for x in xs]
    torch.cuda.synchronize()
    monkeypatch.setattr(w4._Torch, "torch", None)
    monkeypatch.setattr(w4._Torch, "native", None)
    start, got = threading.Barrier(4), [None] * 4

    def work(i):
        stream = torch.cuda.Stream(dev)
        start.wait()
        with torch.cuda.stream(stream):
            out = [w4.w8a8_linear(xs[i], W, ws) for _ in range(20)]
        stream.synchronize()
        got[i] = out

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    for out, y in zip(got, want):
        assert out is not None and all(torch.equal(o, y) for o in out)

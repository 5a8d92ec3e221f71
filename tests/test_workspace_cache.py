"""The sizes of workspaces that the binding remembers stay few, whatever shapes a program goes through."""
import pytest
import torch

import gemv_w4a16_groupwise_b200 as w4


@pytest.mark.gpu
def test_norm_backward_of_many_shapes(cuda_device, monkeypatch):
    monkeypatch.setattr(w4, "_ws_cache", {("filled", i): 0 for i in range(4097)})
    x = torch.randn(3, 8, device=cuda_device).to(torch.bfloat16)
    f = w4.w4_block_norm(x, x, pre_weight=x[0], keep_rstd=True)
    # a whole-number scale goes through the Python checks, which look the size up
    w4.w4_block_norm_backward(x, f.residual, f.rstd, x, pre_weight=x[0], residual_scale=1)
    assert len(w4._ws_cache) == 1

"""The layer's backward belongs to the forward that it follows, whatever the caller's ScoredRouter holds by then."""

import pytest
import torch

from gpu_util import note

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("change", [dict(scale=7.0), dict(renormalize=False), dict(score="softmax")], ids=str)
def test_settings_changed_between_forward_and_backward(change):
    from expert_ffn_layer_top_amd import layer
    from test_gpu_layer_fp8b import Case
    c = Case(100, 128, 192, 8, 2)
    x, dy = c.tensors()
    w = c.weights()
    note(f"layer router {change}")
    grads = []
    for late in ({}, change):
        router, _ = c.router("scored")
        ctx = layer.forward(x, w, c.k, fp8b=True, router=router)
        for name, value in late.items():
            setattr(router, name, value)
        grads.append(layer.backward(ctx, w, dy))
    torch.cuda.synchronize()
    for key in ("dx", "d_logits", "dw_r"):
        assert torch.equal(grads[0][key], grads[1][key]), key

"""The layer's refusals of options that do not go together (before any GPU call)."""

import pytest
import torch

from expert_ffn_layer_top_amd import layer


def _args():
    w = layer.Weights(*(torch.zeros(2, 64, 64, dtype=torch.bfloat16) for _ in range(3)))
    return torch.zeros(4, 64, dtype=torch.bfloat16), w, 1


@pytest.mark.parametrize("kw,what", [
    (dict(mxfp8=True, fp8b=True), "choose one"),
    (dict(serving=True), "serving"),
    (dict(serving=True, mxfp8=True), "serving"),
    (dict(serving=True, fp8b=True, recompute=True), "serving"),
    (dict(fp8b="yes"), "quantize_fp8b"),
    (dict(fp8b={}), "must hold"),
    (dict(fp8b=dict(wg=0, wu=0, wd=0)), "transposed"),
    (dict(router=layer.ScoredRouter(), balance_weight=0.1), "balance_weight"),
    (dict(router=layer.ScoredRouter(), want_probs=True), "want_probs"),
], ids=str)
def test_refusals(kw, what):
    x, w, k = _args()
    with pytest.raises(ValueError, match=what):
        layer.forward(x, w, k, logits=torch.zeros(4, 2), **kw)


def test_backward_of_a_serving_forward_is_refused():
    _, w, _ = _args()
    with pytest.raises(ValueError, match="serving"):
        layer.backward(dict(serving=True), w, None)

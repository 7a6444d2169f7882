"""More of the layer with adapters: what a frozen layer's forward keeps, the events around its calls."""

import pytest
import torch

from gpu_util import note
from test_gpu_layer_adapter import GRADS, Case, mods

pytestmark = pytest.mark.gpu

FORMATS = pytest.mark.parametrize("fmt", [{}, dict(mxfp8=True), dict(fp8b=True)], ids=["bf16", "mxfp8", "fp8b"])
PERMUTED = ("xp", "xq", "xpq", "xps")


@FORMATS
def test_a_frozen_forward_keeps_nothing_for_the_weights(fmt):
    """The permuted input only where recompute reads it, no token blocks of A; without adapters neither x nor A.  The backward
    gives the same bits as that of a layer that is trained whole."""
    layer, _ = mods()
    note(f"layer frozen keeps {fmt}")
    c = Case(T=150, d=256, f=128)
    for with_adapters in (True, False):
        kw = dict(adapters=c.ad, adapter_ids=c.ids) if with_adapters else {}
        whole = layer.forward(c.x, c.w, c.k, logits=c.logits, **kw, **fmt)
        want = layer.backward(whole, c.w, c.dy)
        held = [name for name in PERMUTED if name in whole]
        assert held and whole["a"] is not None and whole["x"] is c.x
        for recompute in (False, True):
            ctx = layer.forward(c.x, c.w, c.k, logits=c.logits, frozen=True, recompute=recompute, **kw, **fmt)
            assert [name for name in PERMUTED if name in ctx] == (held if recompute else [])
            assert "aT" not in ctx and "aTs" not in ctx
            assert (ctx["x"] is not None) == with_adapters and (ctx["a"] is not None) == (with_adapters and not recompute)
            out = layer.backward(ctx, c.w, c.dy)
            assert torch.equal(ctx["y"], whole["y"])
            assert not any(name.startswith("dw_") for name in out)
            for name in GRADS:
                # (without adapters the MXFP8 backward of a layer trained whole quantises dYexp from fp32, not from bf16)
                if name in out and (with_adapters or "mxfp8" not in fmt or name == "d_logits"):
                    assert torch.equal(out[name], want[name]), (with_adapters, recompute, name)


@FORMATS
def test_events_bracket_every_call_of_the_adapters(fmt):
    layer, _ = mods()
    note(f"layer adapters events {fmt}")
    c = Case(T=150, d=256, f=128)
    events = {name: tuple(torch.cuda.Event(enable_timing=True) for _ in range(2)) for name in layer.ADAPTER_CALLS}
    ctx = layer.forward(c.x, c.w, c.k, logits=c.logits, adapters=c.ad, adapter_ids=c.ids, events=events, **fmt)
    layer.backward(ctx, c.w, c.dy, events=events)
    torch.cuda.synchronize()
    for name, (start, end) in events.items():
        assert start.elapsed_time(end) > 0, name            # (an event that was not recorded raises)


@FORMATS
def test_a_frozen_layer_that_owns_its_router_needs_no_x(fmt):
    layer, _ = mods()
    note(f"layer frozen with its router {fmt}")
    c = Case(T=150, d=256, f=128)
    g = torch.Generator(device="cuda").manual_seed(2)
    w = layer.Weights(c.w.w_gate, c.w.w_up, c.w.w_down, w_r=torch.randn((256, c.E), generator=g, device="cuda", dtype=torch.float32) / 16)
    for kw in ({}, dict(adapters=c.ad, adapter_ids=c.ids)):
        want = layer.backward(layer.forward(c.x, w, c.k, **kw, **fmt), w, c.dy)
        out = layer.backward(layer.forward(c.x, w, c.k, frozen=True, **kw, **fmt), w, c.dy)
        assert "dw_r" in want and not any(name.startswith("dw_") for name in out)
        for name in ("d_logits", "dx"):
            if kw or "mxfp8" not in fmt or name == "d_logits":
                assert torch.equal(out[name], want[name]), name

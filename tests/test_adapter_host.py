"""Refusals of the adapters' and the dropout's calls, on the host: the torch wrappers (CPU tensors; a consistent call stops
at the device check), the layer's options, and the C entry points (every call fails its argument checks, so
nothing is launched)."""

import ctypes

import pytest
import torch

from expert_ffn_layer_top_amd import _lib, layer, ops

bf, i32, f32, i64 = torch.bfloat16, torch.int32, torch.float32, torch.int64
T, k, E, L, d, f, r = 8, 2, 4, 3, 192, 128, 16
n = T * k


def z(*shape, dt=bf):
    return torch.zeros(shape, dtype=dt)


def consistent(fn, *args, **kw):
    with pytest.raises(ValueError, match="GPU"):
        fn(*args, **kw)


def refused(match, fn, *args, exc=(ValueError, TypeError), **kw):
    with pytest.raises(exc, match=match):
        fn(*args, **kw)


def drop(p=0.1, site=0, rng=None):
    return ops.Dropout(p, z(2, dt=i64) if rng is None else rng, site)


def test_dropout():
    gate, dest = z(T, k, dt=f32), z(T, k, dt=i32)
    consistent(ops.dropout, z(T, d), drop())
    consistent(ops.dropout, z(T, d), drop(), residual=z(T, d))
    consistent(ops.unpermute_combine_dropout, z(n, d), gate, dest, drop())
    consistent(ops.unpermute_combine_dropout, z(n, d), gate, dest, None, residual=z(T, d))
    consistent(ops.unpermute_combine_dropout_bwd, z(T, d), z(n, d), gate, dest, drop())
    for p in (-0.1, 1.0, 1.5, float("nan"), 1 - 2.0 ** -18):
        refused("p = ", ops.dropout, z(T, d), drop(p))
    refused("site", ops.dropout, z(T, d), drop(site=16))
    refused("rng", ops.dropout, z(T, d), drop(rng=z(2, dt=i32)))
    refused("rng", ops.dropout, z(T, d), drop(rng=z(3, dt=i64)))
    refused("Dropout", ops.dropout, z(T, d), 0.1)
    refused("x", ops.dropout, z(T, d, dt=f32), drop())
    refused("x", ops.dropout, z(d, T).t(), drop())
    refused("residual", ops.dropout, z(T, d), drop(), residual=z(T + 1, d))
    refused("yexp", ops.unpermute_combine_dropout, z(n + 1, d), gate, dest, drop())
    refused("topk_gate", ops.unpermute_combine_dropout, z(n, d), z(T, k + 1, dt=f32), dest, drop())
    refused("residual", ops.unpermute_combine_dropout, z(n, d), gate, dest, drop(), residual=z(T, d + 64))
    refused("dy", ops.unpermute_combine_dropout_bwd, z(T + 1, d), z(n, d), gate, dest, drop())
    refused("yexp", ops.unpermute_combine_dropout_bwd, z(T, d), z(n, d + 64), gate, dest, drop())


def test_plan():
    consistent(ops.adapter_plan, z(T, dt=i32), z(E + 1, dt=i32), L, row_token=z(n, dt=i32))
    consistent(ops.adapter_plan, z(T, dt=i32), z(E + 1, dt=i32), L, backward=True)
    refused("ids", ops.adapter_plan, z(T, dt=i64), z(E + 1, dt=i32), L)
    refused("offsets", ops.adapter_plan, z(T, dt=i32), z(E + 1), L)
    refused("row_token", ops.adapter_plan, z(T, dt=i32), z(E + 1, dt=i32), L, row_token=z(n, 1, dt=i32))
    for count in (0, 257):
        refused("adapters", ops.adapter_plan, z(T, dt=i32), z(E + 1, dt=i32), count)
    refused("experts", ops.adapter_plan, z(T, dt=i32), z(1, dt=i32), L)
    refused("experts", ops.adapter_plan, z(T, dt=i32), z(258, dt=i32), L)
    refused("rows", ops.adapter_plan, z(T, dt=i32), z(E + 1, dt=i32), L, row_token=z(0, dt=i32))
    refused("tokens", ops.adapter_plan, z(0, dt=i32), z(E + 1, dt=i32), L)


def plan(backward=True):
    p = ops.AdapterPlan()
    p.ids, p.offsets, p.row_token = z(T, dt=i32), z(E + 1, dt=i32), z(n, dt=i32)
    p.buf = z(64, dt=torch.uint8) if backward else None
    p.T, p.n, p.E, p.L, p.dev = T, n, E, L, -1
    p._rows = (0, 0, 0, 0, T, n, E, L)
    return p


def matrices(**kw):
    m = dict(a_gu=z(L, E, 2 * r, d), b_gate=z(L, E, r, f), b_up=z(L, E, r, f), a_down=z(L, E, r, f), b_down=z(L, E, r, d),
             scale=z(L, dt=f32))
    m.update(kw)
    up = [m[name] for name in ("a_gu", "b_gate", "b_up", "scale")]
    return up, [m[name] for name in ("a_down", "b_down", "scale")]


def test_adapter_calls():
    up, down = matrices()
    x, nf, nd = z(T, d), z(n, f), z(n, d)
    consistent(ops.adapter_gate_up, x, nf, nf, nf, plan(), *up)
    consistent(ops.adapter_gate_up, x, nf, nf, nf, plan(False), *up, drop=drop(), want_gu=False)
    consistent(ops.adapter_down, nf, nd, plan(), *down)
    consistent(ops.adapter_down_bwd, nd, nf, z(n, r), nf, nf, nf, nf, plan(), *down)
    consistent(ops.adapter_gate_up_bwd, nf, nf, x, z(n, 2 * r), nd, plan(), *up)
    refused("backward=True", ops.adapter_down_bwd, nd, nf, z(n, r), nf, nf, nf, nf, plan(False), *down)
    refused("backward=True", ops.adapter_gate_up_bwd, nf, nf, x, z(n, 2 * r), nd, plan(False), *up)
    refused("AdapterPlan", ops.adapter_gate_up, x, nf, nf, nf, None, *up)
    refused("AdapterPlan", ops.adapter_down, nf, nd, {}, *down)
    refused("x", ops.adapter_gate_up, z(n, d), nf, nf, nf, plan(), *up)
    refused("g", ops.adapter_gate_up, x, z(n - 1, f), nf, nf, plan(), *up)
    refused("u", ops.adapter_gate_up, x, nf, z(n, f, dt=f32), nf, plan(), *up)
    refused("a", ops.adapter_gate_up, x, nf, nf, z(f, n).t(), plan(), *up)
    refused("yexp", ops.adapter_down, nf, z(n, d + 64), plan(), *down)
    refused("v", ops.adapter_down_bwd, nd, nf, z(n, 2 * r), nf, nf, nf, nf, plan(), *down)
    refused("dg", ops.adapter_down_bwd, nd, nf, z(n, r), nf, nf, z(n, f + 64), nf, plan(), *down)
    refused("dxp", ops.adapter_gate_up_bwd, nf, nf, x, z(n, 2 * r), z(n, f), plan(), *up)
    for name, bad in (("a_gu", z(L, E, r, d)), ("a_gu", z(L + 1, E, 2 * r, d)), ("b_up", z(L, E, r, f + 64)),
                      ("scale", z(L)), ("b_gate", z(L, E, r, f, dt=f32))):
        refused(name, ops.adapter_gate_up, x, nf, nf, nf, plan(), *matrices(**{name: bad})[0])
    for name, bad in (("b_down", z(L, E, r + 8, d)), ("a_down", z(L, 1, r, f))):
        refused("b_down|a_down", ops.adapter_down, nf, nd, plan(), *matrices(**{name: bad})[1])
    for rank in (4, 12, 72):
        m = matrices(a_down=z(L, E, rank, f), b_down=z(L, E, rank, d))[1]
        refused("rank", ops.adapter_down, nf, nd, plan(), *m)
    m = matrices(a_down=z(L, E, r, 96), b_down=z(L, E, r, d))[1]
    refused("multiples of 64", ops.adapter_down, z(n, 96), nd, plan(), *m)


def args():
    w = layer.Weights(*(z(2, 64, 64) for _ in range(3)))
    ad = layer.Adapters(z(L, 2, 32, 64), *(z(L, 2, 16, 64) for _ in range(4)), z(L, dt=f32))
    return z(4, 64), w, ad


@pytest.mark.parametrize("kw,what", [
    (dict(adapters=True), "go together"),
    (dict(adapter_ids=True), "go together"),
    (dict(adapter_dropout=drop()), "needs adapters"),
    (dict(serving=True, fp8b=True, dropout=drop()), "serving"),
    (dict(serving=True, fp8b=True, frozen=True), "serving"),
    (dict(adapters=True, adapter_ids=True, adapter_dropout=drop(site=15)), "site"),
    (dict(adapters=True, adapter_ids=True, adapter_dropout=drop(site=3), dropout=drop(site=3)), "sites"),
    (dict(adapters=True, adapter_ids=True, adapter_dropout=drop(site=3), dropout=drop(site=4)), "sites"),
], ids=str)
def test_layer_options(kw, what):
    x, w, ad = args()
    if kw.get("adapters"):
        kw = kw | dict(adapters=ad)
    if kw.get("adapter_ids"):
        kw = kw | dict(adapter_ids=z(4, dt=i32))
    with pytest.raises(ValueError, match=what):
        layer.forward(x, w, 1, logits=torch.zeros(4, 2), **kw)


def test_layer_options_of_a_wrong_type():
    x, w, ad = args()
    for kw in (dict(dropout=0.1), dict(adapters=ad, adapter_ids=z(4, dt=i32), adapter_dropout=0.1)):
        with pytest.raises(TypeError, match="Dropout"):
            layer.forward(x, w, 1, logits=torch.zeros(4, 2), **kw)


def test_c_entry_points():
    lib = _lib.lib
    fake, odd = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1008)
    INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
    drops = lambda p=0.5, site=0, rng=fake, T=4, d=64: lib.moe_dropout(fake, None, rng, p, site, T, d, fake, None)    # noqa: E731
    assert drops(p=1.0) == INVALID and drops(p=-0.5) == INVALID and drops(p=float("nan")) == INVALID
    assert drops(site=16) == INVALID and drops(site=-1) == INVALID and drops(rng=None) == INVALID
    assert drops(rng=ctypes.c_void_p(0x1004)) == INVALID
    assert drops(T=0) == UNSUPPORTED and drops(d=96) == UNSUPPORTED
    assert lib.moe_dropout(odd, None, fake, 0.5, 0, 4, 64, fake, None) == INVALID
    assert lib.moe_dropout(fake, odd, fake, 0.5, 0, 4, 64, fake, None) == INVALID
    assert lib.moe_unpermute_combine_dropout(fake, fake, fake, None, fake, 0.5, 0, 4, 64, 17, fake, None) == UNSUPPORTED
    assert lib.moe_unpermute_combine_dropout(fake, None, fake, None, fake, 0.5, 0, 4, 64, 2, fake, None) == INVALID
    assert lib.moe_unpermute_combine_dropout_bwd(fake, fake, fake, fake, None, 0.5, 0, 4, 64, 2, fake, fake, None) == INVALID
    assert lib.moe_unpermute_combine_dropout_bwd(fake, fake, fake, fake, fake, 0.5, 0, 1 << 26, 64, 2, fake, fake, None) == UNSUPPORTED
    assert lib.moe_adapter_plan_bytes(16, 4, 3) > 0
    for bad in ((0, 4, 3), (16, 0, 3), (16, 257, 3), (16, 4, 0), (16, 4, 257), ((1 << 26) + 1, 4, 3)):
        assert lib.moe_adapter_plan_bytes(*bad) == 0
    need = lib.moe_adapter_plan_bytes(16, 4, 3)
    planned = lambda *a: lib.moe_adapter_plan(*a, None)                                                               # noqa: E731
    assert planned(fake, fake, fake, 8, 16, 4, 3, fake, need - 1) == WORKSPACE
    assert planned(fake, fake, fake, 8, 16, 4, 3, None, need) == WORKSPACE
    assert planned(None, fake, fake, 8, 16, 4, 3, fake, need) == INVALID
    assert planned(fake, None, fake, 8, 16, 4, 3, fake, need) == INVALID           # rows are tokens, but 16 is not 8
    assert planned(fake, fake, fake, 8, 16, 4, 3, odd, need) == INVALID
    assert planned(fake, fake, fake, 8, 16, 300, 3, fake, need) == UNSUPPORTED
    for bad in ((16, 96, 64, 8), (16, 64, 64, 12), (16, 64, 64, 72), (0, 64, 64, 8)):
        assert lib.moe_adapter_workspace_bytes(bad[0], 4, 3, *bad[1:], 1, 0) == 0
    ws = lib.moe_adapter_workspace_bytes(16, 4, 3, 192, 128, 16, 1, 0)
    rows = (fake, fake, fake, fake, 8, 16, 4, 3)

    def gate_up(rows=rows, dims=(192, 128, 16), gu=(fake, fake), p=0.0, rng=None, ws_bytes=ws, x=fake, scale=fake):
        return lib.moe_adapter_gate_up(x, *rows, *dims, fake, fake, fake, scale, rng, p, 0, fake, fake, fake, None, *gu, fake,
                                       fake, ws_bytes, None)
    assert gate_up(dims=(192, 128, 12)) == UNSUPPORTED and gate_up(dims=(100, 128, 16)) == UNSUPPORTED
    assert gate_up(gu=(fake, None)) == INVALID and gate_up(p=0.5) == INVALID and gate_up(x=odd) == INVALID
    assert gate_up(dims=((1 << 24) + 64, 128, 16)) == UNSUPPORTED
    assert gate_up(rows=(fake, fake, fake, None, 8, (1 << 22) + 1, 4, 3)) == UNSUPPORTED      # a workgroup a row
    assert gate_up(scale=None) == INVALID and gate_up(ws_bytes=ws - 1) == WORKSPACE
    assert gate_up(rows=(fake, fake, fake, odd, 8, 16, 4, 3)) == INVALID
    bwd = lib.moe_adapter_workspace_bytes(16, 4, 3, 192, 128, 16, 1, 1)

    def down_bwd(plan=fake, ws_bytes=bwd):
        return lib.moe_adapter_down_bwd(fake, fake, fake, fake, fake, fake, plan, 8, 16, 4, 3, 192, 128, 16, fake, fake, fake, None,
                                        0.0, 0, *[fake] * 9, ws_bytes, None)
    assert down_bwd(plan=None) == INVALID and down_bwd(ws_bytes=8) == WORKSPACE

    def gate_up_bwd(plan=fake, ws_bytes=bwd):
        return lib.moe_adapter_gate_up_bwd(fake, fake, fake, fake, fake, fake, fake, plan, 8, 16, 4, 3, 192, 128, 16, fake, fake,
                                           fake, fake, None, 0.0, 0, *[fake] * 6, ws_bytes, None)
    assert gate_up_bwd(plan=None) == INVALID and gate_up_bwd(ws_bytes=8) == WORKSPACE

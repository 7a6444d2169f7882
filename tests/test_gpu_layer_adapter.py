"""The layer with adapters, dropout and the residual: forward, backward, serving, in every format of the products.

In bf16 the whole layer is compared with 64-bit automatic differentiation of its definition, token by token, at the
layer's own bar (2e-2 of the largest).  In the 8-bit formats, whose operands are quantised between the steps, the layer has to equal the
library's calls written out one after the other, bit for bit: each of them has tests of its own.
"""

import numpy as np
import pytest
import torch

from gpu_util import BF16_TOL, assert_close, bf16_to_dev, bits, dev, f32_to_dev, host, i32_to_dev, note
from oracle import codecs, dropout

pytestmark = pytest.mark.gpu

SEED, OFFSET = 31, 17


def mods():
    from expert_ffn_layer_top_amd import layer, ops
    return layer, ops


class Case:
    def __init__(self, T=96, d=128, f=128, E=5, k=2, L=3, r=16, ids="mixed", seed=0):
        layer, ops = mods()
        g = np.random.default_rng([seed, T, d, f, E, k, L, r])
        self.T, self.d, self.f, self.E, self.k, self.L, self.r = T, d, f, E, k, L, r
        self.v = {}

        def t(name, *shape, std=1.0):
            b = codecs.f64_to_bf16(std * g.standard_normal(shape))
            self.v[name] = codecs.bf16_to_f64(b)
            return bf16_to_dev(b)
        self.x, self.dy, self.res = t("x", T, d), t("dy", T, d), t("res", T, d)
        self.w = layer.Weights(t("wg", E, f, d, std=d ** -0.5), t("wu", E, f, d, std=d ** -0.5), t("wd", E, d, f, std=f ** -0.5))
        self.v["logits"] = g.standard_normal((T, E)).astype(np.float32)
        self.logits = f32_to_dev(self.v["logits"])
        self.v["scale"] = (0.5 + g.random(L)).astype(np.float32)
        self.ad = layer.Adapters(t("a_gu", L, E, 2 * r, d, std=d ** -0.5), t("b_gate", L, E, r, f, std=0.5 * r ** -0.5),
                                 t("b_up", L, E, r, f, std=0.5 * r ** -0.5), t("a_down", L, E, r, f, std=f ** -0.5),
                                 t("b_down", L, E, r, d, std=0.5 * r ** -0.5), f32_to_dev(self.v["scale"]))
        self.v["ids"] = np.full(T, -1) if ids == "none" else g.integers(-1, L, T)
        self.ids = i32_to_dev(self.v["ids"])
        self.rng = torch.tensor([SEED, OFFSET], device=dev())
        self.adrop, self.drop = ops.Dropout(0.125, self.rng, 1), ops.Dropout(0.25, self.rng, 0)

    def run(self, backward=True, drops=True, **kw):
        layer, _ = mods()
        if drops:
            kw = dict(adapter_dropout=self.adrop, dropout=self.drop, residual=self.res) | kw
        ctx = layer.forward(self.x, self.w, self.k, logits=self.logits, adapters=self.ad, adapter_ids=self.ids, **kw)
        return (ctx, layer.backward(ctx, self.w, self.dy)) if backward else ctx


GRADS = ("dx", "d_logits", "dw_gate", "dw_up", "dw_down", "d_a_gu", "d_b_gate", "d_b_up", "d_a_down", "d_b_down")


@pytest.mark.parametrize("drops", [False, True], ids=["plain", "dropout"])
@pytest.mark.parametrize("T,d,f,E,k,L,r", [(96, 128, 128, 5, 2, 3, 16), (1, 64, 64, 2, 1, 1, 8), (70, 192, 64, 3, 3, 2, 40)])
def test_bf16_layer_against_automatic_differentiation(T, d, f, E, k, L, r, drops):
    note(f"layer adapters bf16 T={T} d={d} drops={drops}")
    c = Case(T, d, f, E, k, L, r)
    ctx, out = c.run(drops=drops)
    dest, idx = host(ctx["dest"]), host(ctx["topk_idx"])
    n = T * k
    one = lambda rows, cols: np.ones((rows, cols))                                   # noqa: E731
    m1 = dropout.factors(SEED, OFFSET, 1, n, d, 0.125) if drops else one(n, d)
    m2 = dropout.factors(SEED, OFFSET, 2, n, f, 0.125) if drops else one(n, f)
    m0 = dropout.factors(SEED, OFFSET, 0, T, d, 0.25) if drops else one(T, d)
    t = {name: torch.tensor(v, dtype=torch.float64, requires_grad=v.dtype.kind == "f") for name, v in c.v.items() if name != "ids"}
    rows = []
    for s in range(T):
        gate = torch.softmax(t["logits"][s][torch.from_numpy(idx[s]).long()], 0)
        total = 0.0
        for j in range(k):
            e, row, l = int(idx[s, j]), int(dest[s, j]), int(c.v["ids"][s])
            x = t["x"][s]
            g, u = t["wg"][e] @ x, t["wu"][e] @ x
            if l >= 0:
                v = t["a_gu"][l, e] @ (x * torch.from_numpy(m1[row]))
                g = g + t["scale"][l] * (v[:r] @ t["b_gate"][l, e])
                u = u + t["scale"][l] * (v[r:] @ t["b_up"][l, e])
            a = torch.nn.functional.silu(g) * u
            y = t["wd"][e] @ a
            if l >= 0:
                y = y + t["scale"][l] * ((t["a_down"][l, e] @ (a * torch.from_numpy(m2[row]))) @ t["b_down"][l, e])
            total = total + gate[j] * y
        rows.append(total * torch.from_numpy(m0[s]) + (t["res"][s] if drops else 0.0))
    y = torch.stack(rows)
    y.backward(t["dy"].detach())
    assert_close(codecs.bf16_to_f64(bits(ctx["y"])), y.detach().numpy(), BF16_TOL, "y")
    names = dict(dx="x", d_logits="logits", dw_gate="wg", dw_up="wu", dw_down="wd")
    for name in GRADS:
        grad = t[names.get(name, name[2:])].grad
        got = out[name].float().cpu().numpy()
        if grad is None:
            assert np.all(got == 0), name
        else:
            assert_close(got, grad.numpy(), BF16_TOL, name)


def written_out(c, fmt, drops):
    """The layer's step from the library's calls, by hand."""
    _, ops = mods()
    w, ad = c.w, c.ad
    up, down = (ad.a_gu, ad.b_gate, ad.b_up, ad.scale), (ad.a_down, ad.b_down, ad.scale)
    d0, d1, d2 = ((c.drop, c.adrop, ops.Dropout(0.125, c.rng, 2)) if drops else (None,) * 3)
    r = ops.route_topk(c.logits, c.k, pad=128)
    off, pad, n = r["offsets"], r["offsets_pad"], c.T * c.k
    plan = ops.adapter_plan(c.ids, off, c.L, row_token=r["row_token"], backward=True)
    mx = fmt == "mxfp8"
    q = w.quantize_mx() if mx else w.quantize_fp8b()
    if mx:
        xq = ops.permute_quant_mx(c.x, r["dest"])
        g, u, a = ops.grouped_gemm_gate_up(xq[0], off, q["wg"], q["wu"], scales=(xq[1], q["wg_s"], q["wu_s"]))
    else:
        g, u, a = ops.grouped_gemm_gate_up_fp8b(*ops.fp8b_quantize_rows(c.x, dest=r["dest"]), off, *q["wg"], *q["wu"])
    g, u, a, v1 = ops.adapter_gate_up(c.x, g, u, a, plan, *up, drop=d1, want_v=True)
    both = (lambda t: ops.mxfp8_quantize_rows_grouped(t, off, pad)) if mx else (lambda t: ops.fp8b_quantize_rows_grouped(t, off, pad))
    aq, as_, aT, aTs = both(a)
    yexp = ops.grouped_gemm_down_mx(aq, as_, off, q["wd"], q["wd_s"]) if mx else ops.grouped_gemm_down_fp8b(aq, as_, off, *q["wd"])
    yexp, v2 = ops.adapter_down(a, yexp, plan, *down, drop=d2, want_v=True)
    res = c.res if drops else None
    out = dict(y=ops.unpermute_combine_dropout(yexp, r["topk_gate"], r["dest"], d0, residual=res))
    dyexp, d_gate = ops.unpermute_combine_dropout_bwd(c.dy, yexp, r["topk_gate"], r["dest"], d0)
    out["d_logits"] = ops.route_topk_bwd(r["topk_gate"], r["topk_idx"], d_gate, c.E)
    dyq, dys, dyT, dyTs = both(dyexp)
    if mx:
        dg, du = ops.grouped_gemm_dgrad_down(dyq, off, q["wd_t"], g, u, scales=(dys, q["wd_t_s"]))
    else:
        dg, du = ops.grouped_gemm_dgrad_down_fp8b(dyq, dys, off, *q["wd_t"], g, u)
    dg, du, out["d_a_down"], out["d_b_down"] = ops.adapter_down_bwd(dyexp, a, v2, g, u, dg, du, plan, *down, drop=d2)
    (dgq, dgs, dgT, dgTs), (duq, dus, duT, duTs) = both(dg), both(du)
    if mx:
        dxp = ops.grouped_gemm_dgrad_gate_up(dgq, duq, off, q["wg_t"], q["wu_t"], scales=(dgs, dus, q["wg_t_s"], q["wu_t_s"]))
        xT, xTs = ops.mxfp8_quantize_grouped(c.x, off, pad, n, row_token=r["row_token"])
        out["dw_down"] = ops.grouped_gemm_wgrad_down(dyT, aT, off, n, offsets_pad=pad, scales=(dyTs, aTs))
        out["dw_gate"], out["dw_up"] = ops.grouped_gemm_wgrad_gate_up(dgT, duT, xT, off, n, offsets_pad=pad, scales=(dgTs, duTs, xTs))
    else:
        dxp = ops.grouped_gemm_dgrad_gate_up_fp8b(dgq, dgs, duq, dus, off, *q["wg_t"], *q["wu_t"])
        _, _, xT, xTs = ops.fp8b_quantize_rows_grouped(c.x, off, pad, row_token=r["row_token"], want_rows=False)
        out["dw_down"] = ops.grouped_gemm_wgrad_down_fp8b(dyT, dyTs, aT, aTs, off, pad, n)
        out["dw_gate"], out["dw_up"] = ops.grouped_gemm_wgrad_gate_up_fp8b(dgT, dgTs, duT, duTs, xT, xTs, off, pad, n)
    dxp, out["d_a_gu"], out["d_b_gate"], out["d_b_up"] = ops.adapter_gate_up_bwd(dg, du, c.x, v1, dxp, plan, *up, drop=d1)
    out["dx"] = ops.permute_bwd(dxp, r["dest"])
    return out


@pytest.mark.parametrize("drops", [False, True], ids=["plain", "dropout"])
@pytest.mark.parametrize("fmt", ["mxfp8", "fp8b"])
def test_8_bit_layer_is_its_calls_one_after_the_other(fmt, drops):
    note(f"layer adapters {fmt} drops={drops}")
    c = Case(T=150, d=256, f=128)
    ctx, out = c.run(drops=drops, **{fmt: True})
    for name, want in written_out(c, fmt, drops).items():
        assert torch.equal(ctx["y"] if name == "y" else out[name], want), name


@pytest.mark.parametrize("fmt", [{}, dict(mxfp8=True), dict(fp8b=True)], ids=["bf16", "mxfp8", "fp8b"])
def test_recompute_and_frozen_give_the_same_bits(fmt):
    note(f"layer adapters recompute, frozen {fmt}")
    c = Case(T=150, d=256, f=128)
    ctx, out = c.run(**fmt)
    for kw in (dict(recompute=True), dict(frozen=True), dict(recompute=True, frozen=True)):
        ctx2, out2 = c.run(**fmt, **kw)
        assert torch.equal(ctx["y"], ctx2["y"])
        for name in GRADS:
            if kw.get("frozen") and name.startswith("dw_"):
                assert name not in out2
            else:
                assert torch.equal(out[name], out2[name]), (kw, name)


@pytest.mark.parametrize("fmt", [{}, dict(mxfp8=True), dict(fp8b=True)], ids=["bf16", "mxfp8", "fp8b"])
def test_tokens_without_an_adapter_are_the_layer_itself(fmt):
    layer, _ = mods()
    note(f"layer without adapters {fmt}")
    c = Case(T=150, d=256, f=128, ids="none")
    ctx, out = c.run(drops=False, **fmt)
    ctx2 = layer.forward(c.x, c.w, c.k, logits=c.logits, **fmt)
    out2 = layer.backward(ctx2, c.w, c.dy)
    assert torch.equal(ctx["y"], ctx2["y"])
    for name in GRADS:
        if name in out2:
            assert torch.equal(out[name], out2[name]), name
        else:
            assert torch.count_nonzero(out[name]) == 0, name


def test_serving_matches_the_training_forward():
    """Few rows are not sorted and their sums are cut into slices, so the last bits may differ: y within two roundings of a, v and
    yexp (each 2^-8 of values no larger than the largest of yexp)."""
    note("layer adapters serving")
    for T in (1, 5, 96):
        c = Case(T=T, d=256, f=128)
        q = c.w.quantize_fp8b()
        y = c.run(backward=False, drops=False, fp8b=q)["y"]
        s = c.run(backward=False, drops=False, fp8b=q, serving=True)
        assert s["g"] is s["u"] is None and s["adapter_v2"] is None
        assert_close(s["y"].float().cpu().numpy(), y.float().cpu().numpy(), 6 * 2.0 ** -8, "y")


@pytest.mark.parametrize("fmt", [{}, dict(mxfp8=True), dict(fp8b=True)], ids=["bf16", "mxfp8", "fp8b"])
def test_dropout_and_residual_without_adapters(fmt):
    """y of the calls written out; the backward equals that of dy times the factors (rounded to bf16 under mxfp8)."""
    layer, ops = mods()
    note(f"layer dropout {fmt}")
    c = Case(T=130, d=256, f=128)
    ctx = layer.forward(c.x, c.w, c.k, logits=c.logits, dropout=c.drop, residual=c.res, **fmt)
    plain = layer.forward(c.x, c.w, c.k, logits=c.logits, **fmt)
    assert torch.equal(ctx["y"], ops.unpermute_combine_dropout(plain["yexp"], plain["topk_gate"], plain["dest"], c.drop, residual=c.res))
    c.rng[1] += 1                        # the program moves on: the backward keeps what the forward had
    out = layer.backward(ctx, c.w, c.dy)
    c.rng[1] -= 1
    dy = ops.dropout(c.dy, c.drop)
    if "mxfp8" in fmt:
        want = layer.backward(plain, c.w, dy)
        for name in ("dx", "d_logits", "dw_gate", "dw_up", "dw_down"):
            assert torch.equal(out[name], want[name]), name
    else:
        dyexp, d_gate = ops.unpermute_combine_dropout_bwd(c.dy, plain["yexp"], plain["topk_gate"], plain["dest"], c.drop)
        assert torch.equal(out["dyexp"], dyexp) and torch.equal(out["d_gate"], d_gate)
    only = layer.forward(c.x, c.w, c.k, logits=c.logits, residual=c.res, **fmt)
    assert torch.equal(only["y"], ops.unpermute_combine_dropout(plain["yexp"], plain["topk_gate"], plain["dest"], None, residual=c.res))


def test_a_training_step_captured_and_replayed():
    """Forward and backward with adapters and dropout in one graph; the ids and the generator's offset change between
    the replays, and eager steps run there too."""
    note("layer adapters captured")
    c = Case(T=96)

    def step():
        ctx, out = c.run(frozen=True)
        return [ctx["y"]] + [out[name] for name in GRADS if not name.startswith("dw_")]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    g = np.random.default_rng(1)
    seen = []
    for i in range(3):
        c.ids.copy_(torch.from_numpy(g.integers(-1, 3, 96).astype(np.int32)))
        c.rng[1] = i
        graph.replay()
        torch.cuda.synchronize()
        for s, t in zip(got, step()):
            assert torch.equal(s, t), i
        seen.append(got[0].clone())
    assert not torch.equal(seen[0], seen[1])

"""The layer on block-128 E4M3 products and with the scored router: forward, backward and serving together.

Every step of the layer is compared with the oracle's on the GPU's own inputs to that step.  The quantised
operands are a bit-exact function of bf16 tensors that the layer hands out, so each product is held to the
bounds of the products' own tests (half a step of bf16 and the matrix core's sums), and a step that read the
wrong tensor, layout or copy of a weight would miss them by far.  The sums outside the products have the bounds
of their own: `rows_tol`.
"""

import numpy as np
import pytest
import torch

from gpu_util import assert_close, bf16_to_dev, bits, f32_to_dev, host, note
from oracle import codecs, fp8b, moe, scored
from test_gpu_fp8b import assert_bf16, silu_slack, sum_tol

pytestmark = pytest.mark.gpu

SCORED = dict(score="sigmoid", n_group=4, topk_group=2, group_top=2, renormalize=True, scale=2.5)
SOFTMAX_ALL = dict(score="softmax", renormalize=False)


class Case:
    def __init__(self, T, d, f, E, k, seed=0):
        rng = np.random.default_rng(seed)
        self.T, self.d, self.f, self.E, self.k = T, d, f, E, k

        def bf16(*shape, std):
            b = codecs.f64_to_bf16(std * rng.standard_normal(shape))
            return b, codecs.bf16_to_f64(b)
        self.x, self.dy = bf16(T, d, std=1.0), bf16(T, d, std=1.0)
        self.wg, self.wu = bf16(E, f, d, std=d ** -0.5), bf16(E, f, d, std=d ** -0.5)
        self.wd = bf16(E, d, f, std=f ** -0.5)
        self.w_r = (rng.standard_normal((d, E)) * d ** -0.5).astype(np.float32)
        self.bias = (0.05 * rng.standard_normal(E)).astype(np.float32)

    def weights(self):
        from expert_ffn_layer_top_amd import layer
        return layer.Weights(bf16_to_dev(self.wg[0]), bf16_to_dev(self.wu[0]), bf16_to_dev(self.wd[0]),
                             w_r=f32_to_dev(self.w_r))

    def router(self, kind):
        from expert_ffn_layer_top_amd import layer
        if kind == "softmax":
            return None, None
        o = dict(SCORED, bias=self.bias) if kind == "scored" else dict(SOFTMAX_ALL)
        return layer.ScoredRouter(**{**o, "bias": f32_to_dev(self.bias)} if kind == "scored" else o), o

    def tensors(self):
        return bf16_to_dev(self.x[0]), bf16_to_dev(self.dy[0])


def value(t):
    return codecs.bf16_to_f64(bits(t))


def rows_tol(terms, size):
    """A fp32 sum of `terms` products, in any order: each product and each addition rounds once."""
    return 2 * terms * 2.0 ** -24 * size


def check_forward(c, ctx, route):
    logits = host(ctx["logits"])
    size = np.abs(c.x[1]) @ np.abs(c.w_r).astype(np.float64)
    assert (np.abs(logits - moe.router_project(c.x[0], c.w_r)) <= rows_tol(c.d, size)).all(), "logits"
    idx, gate, _ = moe.route_topk(logits, c.k) if route is None else scored.route(logits, c.k, **route)
    _, off, dest, row_token, pad = moe.route_metadata(idx, c.E, pad=128)
    for key, ref in dict(topk_idx=idx, dest=dest, offsets=off, row_token=row_token, offsets_pad=pad).items():
        assert np.array_equal(host(ctx[key]), ref), key
    assert_close(host(ctx["topk_gate"]), gate, 1e-5, "gates")
    xp = moe.permute(c.x[1], dest)
    x = fp8b.row_values(*fp8b.quantize_rows(xp))
    gr, gs, gl = fp8b.grouped_nt(x, fp8b.weight_values(*fp8b.quantize_weights(c.wg[1])), off)
    ur, us, ul = fp8b.grouped_nt(x, fp8b.weight_values(*fp8b.quantize_weights(c.wu[1])), off)
    dg, du = sum_tol(gs, gl, c.d), sum_tol(us, ul, c.d)
    assert_bf16(ctx["g"], gr, dg, "g")
    assert_bf16(ctx["u"], ur, du, "u")
    assert_bf16(ctx["a"], moe.silu(gr) * ur, silu_slack(gr, ur, dg, du), "a")
    a = fp8b.row_values(*fp8b.quantize_rows(value(ctx["a"])))
    yr, ys, yl = fp8b.grouped_nt(a, fp8b.weight_values(*fp8b.quantize_weights(c.wd[1])), off)
    assert_bf16(ctx["yexp"], yr, sum_tol(ys, yl, c.f), "yexp")
    yexp, gates = value(ctx["yexp"]), host(ctx["topk_gate"])
    assert_bf16(ctx["y"], moe.combine(yexp, gates, dest), rows_tol(c.k, moe.combine(np.abs(yexp), np.abs(gates), dest)), "y")
    return logits, idx, off, dest, pad


def check_backward(c, ctx, out, route, meta):
    logits, idx, off, dest, pad = meta
    gates, yexp = host(ctx["topk_gate"]), value(ctx["yexp"])
    dyexp, d_gate = moe.combine_bwd(c.dy[0], yexp, gates, dest)
    _, size = moe.combine_bwd(np.abs(c.dy[1]), np.abs(yexp), gates, dest)
    assert_bf16(out["dyexp"], dyexp, rows_tol(1, np.abs(dyexp)), "dyexp")
    assert (np.abs(host(out["d_gate"]) - d_gate) <= rows_tol(c.d, size)).all(), "d_gate"
    dg32 = host(out["d_gate"])
    if route is None:
        dl = moe.route_topk_bwd(gates, idx, dg32, c.E)
    else:
        dl = scored.route_bwd(logits, idx, dg32, route["score"], route["renormalize"], route.get("scale", 1.0))
    assert_close(host(out["d_logits"]), dl, 1e-5, "d_logits")
    dl = host(out["d_logits"])
    addend, dw_r = moe.router_project_bwd(c.x[0], c.w_r, dl)
    size = np.abs(c.x[1]).T @ np.abs(dl).astype(np.float64)
    assert (np.abs(host(out["dw_r"]) - dw_r) <= rows_tol(c.T, size)).all(), "dw_r"
    wg, wu, wd = (fp8b.weight_values(*fp8b.quantize_weights(w[1])).transpose(0, 2, 1) for w in (c.wg, c.wu, c.wd))
    dyexp, g, u = value(out["dyexp"]), value(ctx["g"]), value(ctx["u"])
    da, size, largest = fp8b.grouped_nt(fp8b.row_values(*fp8b.quantize_rows(dyexp)), wd, off)
    slack, s = sum_tol(size, largest, c.d), 1 / (1 + np.exp(-g))
    kg, ku = u * s * (1 + g * (1 - s)), g * s
    assert_bf16(out["dg"], da * kg, slack * np.abs(kg) + 16 * 2.0 ** -24 * np.abs(da * u) * (1 + np.abs(g)), "dg")
    assert_bf16(out["du"], da * ku, slack * np.abs(ku) + 16 * 2.0 ** -24 * np.abs(da * g), "du")
    dg, du = value(out["dg"]), value(out["du"])
    r0, s0, l0 = fp8b.grouped_nt(fp8b.row_values(*fp8b.quantize_rows(dg)), wg, off)
    r1, s1, l1 = fp8b.grouped_nt(fp8b.row_values(*fp8b.quantize_rows(du)), wu, off)
    assert_bf16(out["dxp"], r0 + r1, sum_tol(s0 + s1, l0 + l1, 2 * c.f + 128), "dxp")
    dxp = value(out["dxp"])
    size = moe.permute_bwd(np.abs(dxp), dest, addend=np.abs(dl).astype(np.float64) @ np.abs(c.w_r).T.astype(np.float64))
    assert_bf16(out["dx"], moe.permute_bwd(dxp, dest, addend=addend), rows_tol(c.k + c.E, size), "dx")

    def tokens(v):
        q, s = fp8b.quantize_tokens(v, off, pad, (c.T * c.k + 128 * c.E + 127) // 128 * 128)
        return fp8b.token_values(q, s, off, pad)
    x, K = tokens(moe.permute(c.x[1], dest)), int(np.diff(off).max())
    for key, left, right in (("dw_gate", dg, x), ("dw_up", du, x), ("dw_down", dyexp, tokens(value(ctx["a"])))):
        ref, size, largest = fp8b.grouped_tn(tokens(left), right, off)
        assert_bf16(out[key], ref, sum_tol(size, largest, K), key)


CASES = [((300, 256, 384, 8, 2), "scored"), ((129, 192, 320, 16, 3), "softmax_all"), ((640, 512, 512, 4, 2), "softmax"),
         ((1, 128, 64, 8, 4), "scored"), ((70, 64, 128, 1, 1), "softmax")]


@pytest.mark.parametrize("shape,kind", CASES, ids=lambda v: v if isinstance(v, str) else "x".join(map(str, v)))
def test_layer_step_by_step(shape, kind):
    from expert_ffn_layer_top_amd import layer
    c = Case(*shape)
    x, dy = c.tensors()
    w = c.weights()
    router, route = c.router(kind)
    note(f"layer block-128 {shape} {kind}")
    ctx = layer.forward(x, w, c.k, fp8b=True, router=router)
    out = layer.backward(ctx, w, dy)
    torch.cuda.synchronize()
    check_backward(c, ctx, out, route, check_forward(c, ctx, route))


@pytest.mark.parametrize("shape", [(300, 256, 384, 8, 2), (1, 128, 64, 8, 4), (5, 256, 192, 16, 2)],
                         ids=lambda v: "x".join(map(str, v)))
def test_serving_and_kept_copies_give_the_same(shape):
    """Serving, the recomputing forward and copies that the caller keeps change no bit."""
    from expert_ffn_layer_top_amd import layer
    c = Case(*shape)
    x, dy = c.tensors()
    w = c.weights()
    router, _ = c.router("scored")
    note(f"layer block-128 forms {shape}")
    ctx = layer.forward(x, w, c.k, fp8b=True, router=router)
    out = layer.backward(ctx, w, dy)
    served = layer.forward(x, w, c.k, fp8b=w.quantize_fp8b(transposed=False), router=router, serving=True)
    again = layer.forward(x, w, c.k, fp8b=w.quantize_fp8b(), router=router, recompute=True)
    assert again["g"] is None and again["a"] is None and served["g"] is None
    out2 = layer.backward(again, w, dy)
    torch.cuda.synchronize()
    assert torch.equal(served["y"], ctx["y"]) and torch.equal(again["y"], ctx["y"])
    for key in ("dx", "d_logits", "dw_r", "dw_gate", "dw_up", "dw_down"):
        assert torch.equal(out[key], out2[key]), key
    with pytest.raises(ValueError, match="serving"):
        layer.backward(served, w, dy)


def test_weight_update_is_seen():
    """fp8b=True quantises in every forward: a weight changed through `.data`, which bumps no version, is seen."""
    from expert_ffn_layer_top_amd import layer
    c = Case(200, 128, 192, 4, 2)
    x, _ = c.tensors()
    w = c.weights()
    router, _ = c.router("scored")
    note("layer block-128 weight update")
    y0 = layer.forward(x, w, c.k, fp8b=True, router=router)["y"]
    w.w_up.data.mul_(0.5)
    y1 = layer.forward(x, w, c.k, fp8b=True, router=router)["y"]
    torch.cuda.synchronize()
    assert torch.equal(y1, 0.5 * y0)       # a power of two goes through scales and roundings unchanged


@pytest.mark.parametrize("fmt", ["bf16", "mxfp8"])
def test_scored_router_with_the_other_formats(fmt):
    from expert_ffn_layer_top_amd import layer
    c = Case(300, 256, 256, 8, 2)
    x, dy = c.tensors()
    w = c.weights()
    router, route = c.router("scored")
    note(f"layer scored router {fmt}")
    ctx = layer.forward(x, w, c.k, mxfp8=fmt == "mxfp8", router=router)
    out = layer.backward(ctx, w, dy)
    torch.cuda.synchronize()
    logits = host(ctx["logits"])
    idx, gate, _ = scored.route(logits, c.k, **route)
    _, off, dest, _, _ = moe.route_metadata(idx, c.E)
    assert np.array_equal(host(ctx["topk_idx"]), idx) and np.array_equal(host(ctx["dest"]), dest)
    d_logits = scored.route_bwd(logits, idx, host(out["d_gate"]), "sigmoid", True, SCORED["scale"])
    assert_close(host(out["d_logits"]), d_logits, 1e-5, "d_logits")
    yexp, gates = value(ctx["yexp"]), host(ctx["topk_gate"])
    assert_bf16(ctx["y"], moe.combine(yexp, gates, dest), rows_tol(c.k, moe.combine(np.abs(yexp), np.abs(gates), dest)), "y")


def test_step_captured_and_replayed():
    """Forward and backward in one graph, eager steps and a second graph of a serving forward in between."""
    from expert_ffn_layer_top_amd import layer
    c = Case(200, 256, 192, 8, 2)
    x, dy = c.tensors()
    w = c.weights()
    router, _ = c.router("scored")
    keep = w.quantize_fp8b()
    keys = ("dx", "d_logits", "dw_r", "dw_gate", "dw_up", "dw_down")

    def step():
        ctx = layer.forward(x, w, c.k, fp8b=True, router=router)
        return ctx["y"], layer.backward(ctx, w, dy)

    def serve():
        return layer.forward(x[:3], w, c.k, fp8b=keep, router=router, serving=True)["y"]
    note("layer block-128 graph")
    y, out = step()
    ref = {key: out[key].clone() for key in keys}
    ys = serve()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(), serve()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        gy, gout = step()
    with torch.cuda.graph(g2):
        gys = serve()
    for i in range(3):
        g1.replay()
        g2.replay()
        torch.cuda.synchronize()
        assert torch.equal(gy, y) and torch.equal(gys, ys), f"replay {i}"
        for key in keys:
            assert torch.equal(gout[key], ref[key]), f"replay {i}: {key}"
        gy.zero_(), gys.zero_()
        step()
        torch.cuda.synchronize()

"""What is timed of the scored router and of the experts' products in block-scaled E4M3.

Three operators that a mixture-of-experts layer runs one after the other:

  route     scores of every expert (sigmoid or softmax of its logit), a bias for balance added for the
            choice alone, the best groups of experts, the k best experts of those, gates from the
            unbiased scores, and the row metadata of the expert buffers; its gradient
  quantise  E4M3 codes with one fp32 scale per block of 128: of activation rows (128 along the row) on
            their way into the expert buffers, of those rows and of blocks of 128 tokens of one expert
            together, and of weights (blocks of 128 x 128, both layouts)
  experts   the SwiGLU expert products on those codes, forward and backward

A case is a dict of plain values; `run` computes it in elementary torch operations (own = False) or
through the package's calls (own = True); `exact` in 64 bits from the definitions.
"""

import math

import torch

own = False

TINY = 2.0 ** -100          # a block's largest magnitude counts as at least this


def listed():
    return [
        # one token of a served sequence: the router's latency
        _route("route one token", T=1, E=256, k=8, n_group=8, topk_group=4, group_top=2),
        # a training batch of a wide layer with groups and the balance bias
        _route("route batch", T=32768, E=256, k=8, n_group=8, topk_group=4, group_top=2),
        # its gradient where no renormalisation keeps it sparse: softmax over all experts
        _route("route gradient", T=16384, E=128, k=8, score="softmax", renormalize=False, bias=False, grad=True),
        # a prompt's activations on their way into the expert buffers
        _quant("quantise rows", what="rows", T=8192, k=4, d=2048, E=64),
        # a training step's activations in both layouts (128 along the row, 128 tokens of an expert)
        _quant("quantise rows and tokens", what="both", T=16384, k=4, d=1536, E=32),
        # the expert weights after an optimizer step, for the forward and the backward products
        _quant("quantise weights", what="weights", T=1, k=1, E=64, d=7168, f=2048),
        # one token, k experts: the weights of k experts are read once
        _experts("experts one token", T=1, k=8, E=128, d=4096, f=768),
        # a batch of served sequences, a few rows for each expert
        _experts("experts decode batch", T=64, k=4, E=64, d=2048, f=1024),
        # a ragged prompt under uneven routing, sizes that are no multiple of 128
        _experts("experts ragged prompt", T=1003, k=4, E=16, d=2112, f=1344, zipf=0.2),
        # the largest training forward
        _experts("experts forward large", T=32768, k=4, E=64, d=7168, f=2048, train=True),
        # backward passes: even routing, and 128 experts under uneven routing
        _experts("experts backward", T=8192, k=4, E=64, d=2048, f=1024, grad=True),
        _experts("experts backward uneven", T=16384, k=8, E=128, d=4096, f=768, zipf=0.1, grad=True),
    ]


def _route(name, T, E, k, n_group=1, topk_group=1, group_top=1, score="sigmoid", renormalize=True, bias=True,
           grad=False, masked=0):
    return dict(name=name, op="route", T=T, E=E, k=k, n_group=n_group, topk_group=topk_group, group_top=group_top,
                score=score, renormalize=renormalize, bias=bias, scale=2.5, grad=grad, masked=masked)


def _quant(name, what, T, k, E, d, f=0):
    return dict(name=name, op="quantise", what=what, T=T, k=k, E=E, d=d, f=f)


def _experts(name, T, k, E, d, f, zipf=0.0, train=False, grad=False):
    return dict(name=name, op="experts", T=T, k=k, E=E, d=d, f=f, zipf=zipf, train=train, grad=grad)


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("route", "quantise", "experts", "experts"))
    if op == "route":
        n_group, per = rng.choice(((1, rng.randint(4, 256)), (2, 32), (4, 40), (8, 8), (8, 20), (8, 32), (16, 16)))
        E = n_group * per
        topk_group = rng.randint(1, n_group)
        k = rng.randint(1, min(16, topk_group * per))
        case = _route("", T=_log(rng, 1, 32768), E=E, k=k, n_group=n_group, topk_group=topk_group,
                      group_top=rng.choice((1, 2)), score=rng.choice(("sigmoid", "softmax")),
                      renormalize=rng.random() < 0.7, bias=rng.random() < 0.7, grad=rng.random() < 0.4,
                      masked=rng.choice((0, 0, 1, min(3, E - 1))))
    elif op == "quantise":
        what = rng.choice(("rows", "both", "weights"))
        if what == "weights":
            case = _quant("", what, T=1, k=1, E=_log(rng, 1, 64), d=64 * _log(rng, 2, 112), f=64 * _log(rng, 2, 32))
        else:
            case = _quant("", what, T=_log(rng, 1, 16384), k=rng.randint(1, 8), E=_log(rng, 8, 128),
                          d=64 * _log(rng, 2, 64))
    else:
        grad = rng.random() < 0.4
        d, f, E = 64 * _log(rng, 2, 112), 64 * _log(rng, 2, 32), _log(rng, 8, 128)
        k = rng.randint(1, 8)
        most = 32768 * 4 * 7168 * 2048 // (4 if grad else 1)
        T = _log(rng, 1, min(32768, most // (k * d * f)))
        case = _experts("", T=T, k=k, E=E, d=d, f=f, zipf=rng.choice((0.0, 0.1, 0.2)) if T * d * E < 1 << 32 else 0.0,
                        grad=grad, train=not grad and rng.random() < 0.4)
    del case["name"]
    return case


# ------------------------------------------------------------------------------------------ inputs

def _normal(gen, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)


def _codes(v, dims):
    """E4M3 codes and fp32 scales of v (fp32) with one block along `dims` (kept as size 1)."""
    amax = v.abs().amax(dim=dims, keepdim=True).clamp_min(TINY)
    inv = torch.full_like(amax, 448.0) / amax
    q = (v * inv).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q, amax * torch.full_like(amax, 1.0 / 448.0)


def _pad128(v, dim):
    short = -v.shape[dim] % 128
    if not short:
        return v
    shape = list(v.shape)
    shape[dim] = short
    return torch.cat([v, v.new_zeros(shape)], dim)


def _weight_codes(w):
    """w [E, R, C] -> codes [E, R, C], scales [E, ceil(R/128), ceil(C/128)]."""
    E, R, C = w.shape
    p = _pad128(_pad128(w.float(), 1), 2)
    q, s = _codes(p.view(E, p.shape[1] // 128, 128, p.shape[2] // 128, 128), (2, 4))
    return q.view(p.shape)[:, :R, :C].contiguous(), s[:, :, 0, :, 0].contiguous()


def _row_codes(x):
    """x [n, C] -> codes [n, C], scales [ceil(C/128), n]."""
    n, C = x.shape
    p = _pad128(x.float(), 1)
    q, s = _codes(p.view(n, -1, 128), 2)
    return q.view(p.shape)[:, :C].contiguous(), s[:, :, 0].t().contiguous()


def _routing(case, gen):
    """Row metadata of a random routing: chosen experts, rows by expert then token."""
    T, k, E = case["T"], case["k"], case["E"]
    logits = torch.randn((T, E), generator=gen, device="cuda")
    if case.get("zipf"):
        logits -= 3.0 * case["zipf"] * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
    idx = logits.topk(min(k, E), dim=1).indices.reshape(-1)
    order = torch.sort(idx, stable=True).indices
    dest = torch.empty_like(order)
    dest[order] = torch.arange(order.numel(), device="cuda")
    counts = torch.bincount(idx, minlength=E)
    zero = counts.new_zeros(1)
    offsets = torch.cat([zero, counts.cumsum(0)])
    pad = torch.cat([zero, ((counts + 127) // 128 * 128).cumsum(0)])
    row_e = idx[order]
    active = counts.nonzero().reshape(-1)
    slot = torch.full((E,), -1, device="cuda", dtype=torch.int64)
    slot[active] = torch.arange(active.numel(), device="cuda")
    return dict(dest=dest.view(T, -1).int(), offsets=offsets.int(), offsets_pad=pad.int(),
                row_token=(order // min(k, E)).int(), counts=counts.tolist(), active=active,
                cap=int(counts.max()), at=(slot[row_e], torch.arange(order.numel(), device="cuda") - offsets[row_e]),
                at_pad=pad[row_e] + torch.arange(order.numel(), device="cuda") - offsets[row_e])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 1000003 + 17)
    T, E = case["T"], case["E"]
    s = dict(case=case)
    if case["op"] == "route":
        s["logits"] = _normal(gen, T, E, std=1.5)
        if case["masked"]:
            s["logits"][:, E - case["masked"]:] = -math.inf         # experts that are not there
        s["bias"] = _normal(gen, E, std=0.05) if case["bias"] else None
        if case["grad"]:
            s["topk_idx"] = torch.rand((T, E), generator=gen, device="cuda").topk(case["k"], dim=1).indices.int()
            s["d_gate"] = _normal(gen, T, case["k"])
        return s
    d, f = case["d"], case["f"]
    if case["op"] == "quantise" and case["what"] == "weights":
        s["w"] = torch.stack([_normal(gen, f, d, std=0.02, dtype=torch.bfloat16) for _ in range(E)])
        return s
    s["route"] = _routing(case, gen)
    s["x"] = _normal(gen, T, d, dtype=torch.bfloat16)
    if case["op"] == "quantise":
        return s
    n = s["x"].shape[0] * min(case["k"], E)
    s["w"] = {}
    for name, R, C in (("gate", f, d), ("up", f, d), ("down", d, f)):
        parts = [_weight_codes(_normal(gen, 1, R, C, std=0.02, dtype=torch.bfloat16)) for _ in range(E)]
        q, sc = torch.cat([p[0].view(torch.uint8) for p in parts]), torch.cat([p[1] for p in parts])
        del parts
        if case["grad"]:                                            # the backward reads them transposed
            q, sc = q.transpose(1, 2).contiguous(), sc.transpose(1, 2).contiguous()
        s["w"][name] = (q, sc)
    if case["grad"]:
        s["g"], s["u"] = (_normal(gen, n, f, dtype=torch.bfloat16) for _ in range(2))
        s["a"] = (s["g"].float() * torch.sigmoid(s["g"].float()) * s["u"].float()).to(torch.bfloat16)
        s["dyexp"] = _normal(gen, n, d, std=0.3, dtype=torch.bfloat16)
    return s


# ------------------------------------------------------------------------------------- plain forms

def run(s):
    case = s["case"]
    if own:
        return _own(s)
    if case["op"] == "route":
        return _plain_route_bwd(s) if case["grad"] else _plain_route(s)
    if case["op"] == "quantise":
        return _plain_quantise(s)
    return _plain_backward(s) if case["grad"] else _plain_forward(s)


def _scores(logits, score):
    """Scores in 64 bits (choices sit next to each other); a NaN counts as -inf, +inf as the largest float."""
    top = torch.finfo(torch.float32).max
    l = torch.nan_to_num(logits.double(), nan=-math.inf, posinf=top, neginf=-math.inf)
    if score == "sigmoid":
        return l, torch.sigmoid(l)
    m = l.amax(dim=1, keepdim=True)
    e = torch.exp(l - torch.where(m == -math.inf, torch.zeros_like(m), m))
    return l, e / e.sum(dim=1, keepdim=True).clamp_min(1e-300)


def _plain_route(s):
    case = s["case"]
    T, E, k, G = case["T"], case["E"], case["k"], case["n_group"]
    l, p = _scores(s["logits"], case["score"])
    choice = p if s["bias"] is None else p + s["bias"].double()
    choice = torch.where(l == -math.inf, torch.full_like(choice, -math.inf), choice)
    rank = l if s["bias"] is None else choice       # without a bias the logits rank as the scores do
    if case["topk_group"] < G:
        best = choice.view(T, G, -1).sort(dim=2, descending=True).values[:, :, :case["group_top"]]
        total = torch.where(best == -math.inf, torch.zeros_like(best), best).sum(dim=2)
        total = torch.where(best[:, :, 0] == -math.inf, torch.full_like(total, -math.inf), total)
        order = total.sort(dim=1, descending=True, stable=True).indices[:, :case["topk_group"]]
        inside = torch.zeros((T, G), dtype=torch.bool, device=l.device).scatter_(1, order, True)
        inside = inside.repeat_interleave(E // G, dim=1)
    else:
        inside = torch.ones_like(choice, dtype=torch.bool)
    # chosen groups' experts before all others, the absent ones of them last
    first = rank.sort(dim=1, descending=True, stable=True).indices
    order = first.gather(1, inside.gather(1, first).to(torch.int8).sort(dim=1, descending=True, stable=True).indices)
    idx = order[:, :k]
    gate = p.gather(1, idx)
    if case["renormalize"]:
        total = gate.sum(dim=1, keepdim=True)
        gate = torch.where(total > 0, gate / total, torch.zeros_like(gate))
    gate = (gate * case["scale"]).float()
    e = idx.reshape(-1)
    rows = torch.sort(e, stable=True).indices
    dest = torch.empty_like(rows).scatter_(0, rows, torch.arange(T * k, device=l.device))
    counts = torch.zeros(E, dtype=torch.int64, device=l.device).scatter_add_(0, e, torch.ones_like(e))
    zero = counts.new_zeros(1)
    return dict(topk_idx=idx.int(), topk_gate=gate, counts=counts.int(), dest=dest.view(T, k).int(),
                row_token=(rows // k).int(), offsets=torch.cat([zero, counts.cumsum(0)]).int(),
                offsets_pad=torch.cat([zero, ((counts + 127) // 128 * 128).cumsum(0)]).int())


def _plain_route_bwd(s):
    case = s["case"]
    l, p = _scores(s["logits"], case["score"])
    idx = s["topk_idx"].long()
    pk, dg = p.gather(1, idx), s["d_gate"].double() * case["scale"]
    if case["renormalize"]:
        total = pk.sum(dim=1, keepdim=True)
        gate = torch.where(total > 0, pk / total, torch.zeros_like(pk))
        dg = torch.where(total > 0, (dg - (gate * dg).sum(dim=1, keepdim=True)) / total, torch.zeros_like(dg))
    ds = torch.zeros_like(p).scatter_(1, idx, dg)
    if case["score"] == "sigmoid":
        return (ds * p * (1.0 - p)).float()
    return (p * (ds - (p * ds).sum(dim=1, keepdim=True))).float()


def _token_codes(v, case, r, n):
    """v [n, C] fp32 -> codes [C, P], scales [P/128, C]: blocks of 128 tokens of one expert, zeros between."""
    C, P = v.shape[1], (n + 128 * case["E"] + 127) // 128 * 128
    p = torch.zeros((P, C), device=v.device)
    p[r["at_pad"]] = v
    q, sc = _codes(p.view(P // 128, 128, C), 1)
    return q.view(P, C).t().contiguous(), sc[:, 0, :].contiguous()


def _plain_quantise(s):
    case = s["case"]
    if case["what"] == "weights":
        q, sc = _weight_codes(s["w"])
        return dict(q=q, s=sc, qT=q.transpose(1, 2).contiguous(), sT=sc.transpose(1, 2).contiguous())
    r = s["route"]
    rows = s["x"][r["row_token"].long()]
    q, sc = _row_codes(rows)
    if case["what"] == "rows":
        return dict(q=q, s=sc)
    qT, sT = _token_codes(rows.float(), case, r, rows.shape[0])
    return dict(q=q, s=sc, qT=qT, sT=sT)


def _weight_values(w, active):
    q, sc = w                                                       # the codes as bytes
    q, sc = q[active].view(torch.float8_e4m3fn).float(), sc[active]
    sc = sc.repeat_interleave(128, dim=1)[:, :q.shape[1]].repeat_interleave(128, dim=2)[:, :, :q.shape[2]]
    return q * sc


def _row_values(x):
    q, sc = _row_codes(x)
    return q.float() * sc.t().repeat_interleave(128, dim=1)[:, :q.shape[1]]


def _product(v, w, r):
    """v [n, K] fp32 times its expert's w [K', N]^T: [n, N] fp32, all experts with rows in one product."""
    p = torch.zeros((w.shape[0], r["cap"], v.shape[1]), device=v.device)
    p[r["at"]] = v
    return torch.bmm(p, w.transpose(1, 2))[r["at"]]


def _plain_forward(s):
    case, r = s["case"], s["route"]
    v = _row_values(s["x"][r["row_token"].long()])
    g = _product(v, _weight_values(s["w"]["gate"], r["active"]), r)
    u = _product(v, _weight_values(s["w"]["up"], r["active"]), r)
    a = (g * torch.sigmoid(g) * u).to(torch.bfloat16)
    y = _product(_row_values(a), _weight_values(s["w"]["down"], r["active"]), r).to(torch.bfloat16)
    return dict(g=g.to(torch.bfloat16), u=u.to(torch.bfloat16), a=a, y=y) if case["train"] else dict(y=y)


def _weight_gradient(left, right, case, r):
    """dW [E, R, C] = left^T right over each expert's rows, both in codes of 128 tokens."""
    cap = (r["cap"] + 127) // 128 * 128
    A = r["active"].numel()

    def blocks(x):
        p = torch.zeros((A, cap, x.shape[1]), device=x.device)
        p[r["at"]] = x.float()
        q, sc = _codes(p.view(A, cap // 128, 128, -1), 2)
        return (q.float() * sc).view(A, cap, -1)

    out = torch.zeros((case["E"], left.shape[1], right.shape[1]), device=left.device, dtype=torch.bfloat16)
    out[r["active"]] = torch.bmm(blocks(left).transpose(1, 2).contiguous(), blocks(right)).to(torch.bfloat16)
    return out


def _plain_backward(s):
    case, r = s["case"], s["route"]
    da = _product(_row_values(s["dyexp"]), _weight_values(s["w"]["down"], r["active"]), r)
    g, u = s["g"].float(), s["u"].float()
    sg = torch.sigmoid(g)
    dg = (da * u * sg * (1.0 + g * (1.0 - sg))).to(torch.bfloat16)
    du = (da * g * sg).to(torch.bfloat16)
    dxp = _product(_row_values(dg), _weight_values(s["w"]["gate"], r["active"]), r)
    dxp += _product(_row_values(du), _weight_values(s["w"]["up"], r["active"]), r)
    rows = s["x"][r["row_token"].long()]
    return dict(dg=dg, du=du, dxp=dxp.to(torch.bfloat16), dw_down=_weight_gradient(s["dyexp"], s["a"], case, r),
                dw_gate=_weight_gradient(dg, rows, case, r), dw_up=_weight_gradient(du, rows, case, r))


# ------------------------------------------------------------------------------- the package's calls

def _own(s):
    from expert_ffn_layer_top_amd import ops
    case = s["case"]
    if case["op"] == "route":
        if case["grad"]:
            return ops.route_scored_bwd(s["logits"], s["topk_idx"], s["d_gate"], score=case["score"],
                                        renormalize=case["renormalize"], scale=case["scale"])
        out = ops.route_scored(s["logits"], case["k"], score=case["score"], bias=s["bias"], n_group=case["n_group"],
                               topk_group=case["topk_group"], group_top=case["group_top"],
                               renormalize=case["renormalize"], scale=case["scale"], pad=128)
        return {name: out[name] for name in ("topk_idx", "topk_gate", "counts", "dest", "row_token", "offsets",
                                             "offsets_pad")}
    e4m3 = torch.float8_e4m3fn
    if case["op"] == "quantise":
        if case["what"] == "weights":
            q, sc, qT, sT = ops.fp8b_quantize_weights(s["w"])
        elif case["what"] == "rows":
            q, sc = ops.fp8b_quantize_rows(s["x"], dest=s["route"]["dest"])
            return dict(q=q.view(e4m3), s=sc)
        else:
            r = s["route"]
            q, sc, qT, sT = ops.fp8b_quantize_rows_grouped(s["x"], r["offsets"], r["offsets_pad"],
                                                           row_token=r["row_token"])
        return dict(q=q.view(e4m3), s=sc, qT=qT.view(e4m3), sT=sT)
    r, w = s["route"], s["w"]
    off, pad = r["offsets"], r["offsets_pad"]
    if not case["grad"]:
        xq, xs = ops.fp8b_quantize_rows(s["x"], dest=r["dest"])
        g, u, a = ops.grouped_gemm_gate_up_fp8b(xq, xs, off, *w["gate"], *w["up"], want_gu=case["train"])
        aq, sa = ops.fp8b_quantize_rows(a)
        y = ops.grouped_gemm_down_fp8b(aq, sa, off, *w["down"])
        return dict(g=g, u=u, a=a, y=y) if case["train"] else dict(y=y)
    n = s["g"].shape[0]
    dyq, dys, dyT, dyTs = ops.fp8b_quantize_rows_grouped(s["dyexp"], off, pad)
    dg, du = ops.grouped_gemm_dgrad_down_fp8b(dyq, dys, off, *w["down"], s["g"], s["u"])
    _, _, aT, aTs = ops.fp8b_quantize_rows_grouped(s["a"], off, pad, want_rows=False)
    dw_down = ops.grouped_gemm_wgrad_down_fp8b(dyT, dyTs, aT, aTs, off, pad, n)
    dgq, dgs, dgT, dgTs = ops.fp8b_quantize_rows_grouped(dg, off, pad)
    duq, dus, duT, duTs = ops.fp8b_quantize_rows_grouped(du, off, pad)
    dxp = ops.grouped_gemm_dgrad_gate_up_fp8b(dgq, dgs, duq, dus, off, *w["gate"], *w["up"])
    _, _, xT, xTs = ops.fp8b_quantize_rows_grouped(s["x"], off, pad, row_token=r["row_token"], want_rows=False)
    dw_gate, dw_up = ops.grouped_gemm_wgrad_gate_up_fp8b(dgT, dgTs, duT, duTs, xT, xTs, off, pad, n)
    return dict(dg=dg, du=du, dxp=dxp, dw_down=dw_down, dw_gate=dw_gate, dw_up=dw_up)


# ------------------------------------------------------------------------------ what it has to move

def _busy(case):
    """Experts that have rows, on average, under even routing."""
    k = min(case["k"], case["E"])
    return case["E"] * (1.0 - (1.0 - k / case["E"]) ** case["T"])


def work(case):
    T, E, k = case["T"], case["E"], min(case["k"], case["E"])
    n = T * k
    if case["op"] == "route":
        if case["grad"]:
            sparse = case["renormalize"] or case["score"] == "sigmoid"
            return dict(bytes=T * E * 4 + (0 if sparse else T * E * 4) + n * 12, flops=T * E * 4)
        return dict(bytes=T * E * 4 + E * 4 + n * 16 + 12 * E, flops=T * E * 8)
    d, f = case["d"], case["f"]
    blocks = lambda rows, cols: rows * (cols + 4 * -(-cols // 128))     # noqa: E731  codes and their scales
    tokens = lambda cols: blocks(cols, n + 128 * E)                     # noqa: E731
    if case["op"] == "quantise":
        if case["what"] == "weights":
            return dict(bytes=E * d * f * 4 + 8 * E * -(-d // 128) * -(-f // 128), flops=E * d * f * 4)
        both = tokens(d) if case["what"] == "both" else 0
        return dict(bytes=T * d * 2 + n * 4 + blocks(n, d) + both, flops=n * d * 4)
    weights = _busy(case) * 3 * d * f
    if not case["grad"]:
        return dict(bytes=T * d * 2 + weights + n * d * 2 + (3 * n * f * 2 if case["train"] else 0), flops=6 * n * d * f)
    return dict(bytes=T * d * 2 + n * d * 2 + 3 * n * f * 2 + weights + 2 * n * f * 2 + n * d * 2 + E * 3 * d * f * 2,
                flops=12 * n * d * f)


# -------------------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        l = s["logits"].double().clamp(max=torch.finfo(torch.float32).max)
        if case["grad"]:
            idx, dg = s["topk_idx"].long(), s["d_gate"].double() * case["scale"]
            if case["score"] == "softmax" and not case["renormalize"]:
                p = torch.softmax(l, dim=1)
                pk = p.gather(1, idx)
                out = -p * (pk * dg).sum(1, keepdim=True)
                return out.scatter_add_(1, idx, pk * dg)
            lk = l.gather(1, idx)
            if case["score"] == "softmax":
                gate = torch.nan_to_num(torch.softmax(lk, dim=1))
                v = gate * (dg - (gate * dg).sum(1, keepdim=True))
            else:
                slope = torch.sigmoid(lk) * torch.sigmoid(-lk)
                v = dg * slope
                if case["renormalize"]:
                    gate = torch.nan_to_num(torch.softmax(torch.nn.functional.logsigmoid(lk), dim=1))
                    v = gate * torch.sigmoid(-lk) * (dg - (gate * dg).sum(1, keepdim=True))
            return torch.zeros_like(l).scatter_(1, idx, v)
        idx = _plain_route(s)["topk_idx"].long()
        lk = l.gather(1, idx)
        if case["renormalize"]:
            gate = torch.softmax(torch.nn.functional.logsigmoid(lk) if case["score"] == "sigmoid" else lk, dim=1)
        else:
            gate = torch.sigmoid(lk) if case["score"] == "sigmoid" else torch.softmax(l, dim=1).gather(1, idx)
        return dict(topk_idx=None, topk_gate=torch.nan_to_num(gate) * case["scale"], counts=None, dest=None,
                    row_token=None, offsets=None, offsets_pad=None)

    def blocks64(v, dim):
        """Values that the codes of v (blocks of 128 along dim of a matrix) stand for, and the scales.  A code is
        E4M3 of v times 448 / amax, which the definition rounds to fp32: quotients of short mantissas often
        lie on a border of two codes, and this rounding is what decides them."""
        v = v.double() if dim else v.double().t()
        m = torch.nn.functional.pad(v, (0, -v.shape[1] % 128)).view(v.shape[0], -1, 128)
        top = m.abs().amax(dim=2, keepdim=True).clamp_min(TINY)
        code = (m * (448.0 / top).float().double()).clamp(-448, 448).float().to(torch.float8_e4m3fn).double()
        val = (code * (top / 448.0)).view(v.shape[0], -1)[:, :v.shape[1]]
        code = code.view(v.shape[0], -1)[:, :v.shape[1]]
        return (val, code, top[:, :, 0] / 448.0) if dim else (val.t(), code.t(), top[:, :, 0] / 448.0)

    if case["op"] == "quantise" and case["what"] == "weights":
        q, sc = [], []
        for w in s["w"]:
            w = torch.nn.functional.pad(w.double(), (0, -w.shape[1] % 128, 0, -w.shape[0] % 128))
            top = torch.nn.functional.max_pool2d(w.abs()[None], 128)[0].clamp_min(TINY)
            big = top.repeat_interleave(128, 0).repeat_interleave(128, 1)
            q.append((w * (448.0 / big).float().double()).clamp(-448, 448).float().to(torch.float8_e4m3fn)[:case["f"], :case["d"]])
            sc.append(top / 448.0)
        q, sc = torch.stack([c.float() for c in q]), torch.stack(sc)
        return dict(q=q, s=sc, qT=q.transpose(1, 2), sT=sc.transpose(1, 2))
    r = s["route"]
    starts, E = [0], case["E"]
    for c in r["counts"]:
        starts.append(starts[-1] + c)
    rows = s["x"][r["row_token"].long()]
    n = rows.shape[0]
    if case["op"] == "quantise":
        _, code, sc = blocks64(rows, 1)
        if case["what"] == "rows":
            return dict(q=code.float(), s=sc.t())
        P = (n + 128 * E + 127) // 128 * 128
        qT = torch.zeros((P, case["d"]), device="cuda")
        sT = torch.full((P // 128, case["d"]), TINY / 448.0, device="cuda", dtype=torch.float64)
        at = 0
        for e in range(E):
            if r["counts"][e]:
                _, c, m = blocks64(rows[starts[e]:starts[e + 1]], 0)
                qT[at:at + c.shape[0]] = c.float()
                sT[at // 128:at // 128 + m.shape[1]] = m.t()
                at += 128 * m.shape[1]
        return dict(q=code.float(), s=sc.t(), qT=qT.t(), sT=sT)

    def weight64(name, e):
        q, sc = s["w"][name]
        sc = sc[e].double().repeat_interleave(128, 0)[:q.shape[1]].repeat_interleave(128, 1)[:, :q.shape[2]]
        return q[e].view(torch.float8_e4m3fn).double() * sc

    out = {}
    d, f = case["d"], case["f"]
    if not case["grad"]:
        for name, width in (("g", f), ("u", f), ("a", f), ("y", d)):
            out[name] = torch.empty((n, width), device="cuda", dtype=torch.float32 if n * width > 1 << 28 else torch.float64)
        for e in range(E):
            lo, hi = starts[e], starts[e + 1]
            if lo == hi:
                continue
            v = blocks64(rows[lo:hi], 1)[0]
            g, u = v @ weight64("gate", e).t(), v @ weight64("up", e).t()
            a = g / (1.0 + torch.exp(-g)) * u
            out["g"][lo:hi], out["u"][lo:hi], out["a"][lo:hi] = g, u, a
            out["y"][lo:hi] = blocks64(a.to(torch.bfloat16), 1)[0] @ weight64("down", e).t()
        return out if case["train"] else dict(y=out["y"])
    for name, shape in (("dg", (n, f)), ("du", (n, f)), ("dxp", (n, d)), ("dw_down", (E, d, f)), ("dw_gate", (E, f, d)),
                        ("dw_up", (E, f, d))):
        out[name] = torch.zeros(shape, device="cuda")
    for e in range(E):
        lo, hi = starts[e], starts[e + 1]
        if lo == hi:
            continue
        dy, g, u = s["dyexp"][lo:hi], s["g"][lo:hi].double(), s["u"][lo:hi].double()
        da = blocks64(dy, 1)[0] @ weight64("down", e).t()
        sg = 1.0 / (1.0 + torch.exp(-g))
        dg, du = da * u * (sg + g * sg * (1.0 - sg)), da * g * sg
        out["dg"][lo:hi], out["du"][lo:hi] = dg, du
        dg, du = dg.to(torch.bfloat16), du.to(torch.bfloat16)
        out["dxp"][lo:hi] = blocks64(dg, 1)[0] @ weight64("gate", e).t() + blocks64(du, 1)[0] @ weight64("up", e).t()
        x = blocks64(rows[lo:hi], 0)[0]
        out["dw_down"][e] = blocks64(dy, 0)[0].t() @ blocks64(s["a"][lo:hi], 0)[0]
        out["dw_gate"][e], out["dw_up"][e] = blocks64(dg, 0)[0].t() @ x, blocks64(du, 0)[0].t() @ x
    return out

"""What is timed of the experts' low-rank adapters and of the dropout whose mask is never stored.

  adapters  a served or fine-tuned layer adds to every expert product a product of low rank, chosen by the
            token's request: gate and up (with SwiGLU after them) and down, for rows that lie by expert in
            the expert buffers and of which any may have another adapter, or none; and the backward: the
            gradients of the adapters and of what passes through them
  dropout   random zeros from a counter-based generator: on the layer's combined output with the residual
            added, its gradient, and on plain rows; the adapters' inputs have it too while they are trained

A case is a dict of plain values; `run` computes it in elementary torch operations (own = False) or
through the package's calls (own = True); `exact` in 64 bits from the definitions.
"""

import math

import torch

own = False


def listed():
    return [
        # one token of a served sequence: its 8 experts' rows, one adapter of 16 loaded
        _adapt("adapters one token", T=1, k=8, E=128, d=4096, f=768, L=16, r=16, seqs=1, base=0.0),
        # a batch of served sequences, each with its own adapter, a quarter of them without one
        _adapt("adapters decode batch", T=64, k=4, E=64, d=2048, f=1024, L=8, r=16, seqs=64, base=0.25),
        # a few ragged prompts together, sizes that are no multiple of 128
        _adapt("adapters ragged prompts", T=1003, k=4, E=16, d=2112, f=1344, L=5, r=8, seqs=7, base=0.2, zipf=0.2),
        # many prompts of many requests together under uneven routing
        _adapt("adapters many prompts", T=8192, k=4, E=64, d=2048, f=1024, L=32, r=32, seqs=48, base=0.1, zipf=0.1),
        # the forward of a training step with one adapter and dropout on its input
        _adapt("adapters training forward", T=32768, k=4, E=64, d=7168, f=2048, L=1, r=16, seqs=1, base=0.0, p=0.05,
               train=True),
        # backward of a training step: one adapter with dropout, and four of rank 32 under uneven routing
        _adapt("adapters backward", T=8192, k=4, E=64, d=2048, f=1024, L=1, r=16, seqs=1, base=0.0, p=0.1, grad=True),
        _adapt("adapters backward uneven", T=16384, k=8, E=128, d=4096, f=768, L=4, r=32, seqs=16, base=0.0, zipf=0.1,
               grad=True),
        # the combined output of the smallest layer, of a usual and of the largest training batch
        _drop("dropout combine small", what="combine", T=256, k=2, E=8, d=128, p=0.1),
        _drop("dropout combine", what="combine", T=8192, k=4, E=64, d=2048, p=0.1),
        _drop("dropout combine large", what="combine", T=32768, k=4, E=64, d=7168, p=0.05),
        # its gradient
        _drop("dropout combine gradient", what="gradient", T=16384, k=8, E=128, d=4096, p=0.1),
        # rows alone: the gradient that reaches a layer whose combine backward quantises
        _drop("dropout rows", what="rows", T=16384, k=1, E=1, d=7168, p=0.1, residual=False),
    ]


def _adapt(name, T, k, E, d, f, L, r, seqs, base, zipf=0.0, p=0.0, train=False, grad=False):
    return dict(name=name, op="adapters", T=T, k=k, E=E, d=d, f=f, L=L, r=r, seqs=seqs, base=base, zipf=zipf, p=p,
                train=train, grad=grad)


def _drop(name, what, T, k, E, d, p, residual=True):
    return dict(name=name, op="dropout", what=what, T=T, k=k, E=E, d=d, p=p, residual=residual)


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.3:
        what = rng.choice(("combine", "gradient", "rows"))
        E = 1 if what == "rows" else _log(rng, 4, 128)
        case = _drop("", what, T=_log(rng, 1, 32768), k=1 if what == "rows" else rng.randint(1, min(8, E)), E=E,
                     d=64 * _log(rng, 1, 64), p=rng.choice((0.0, 0.05, 0.1, 0.3, 0.5)), residual=rng.random() < 0.5)
    else:
        grad = rng.random() < 0.4
        E, r = _log(rng, 1, 128), 8 * rng.randint(1, 8)
        d, f, k = 64 * _log(rng, 2, 112), 64 * _log(rng, 2, 32), rng.randint(1, min(8, E))
        L = _log(rng, 1, max(1, min(64, (1 << 28) // (E * r * (d + f)))))
        T = _log(rng, 1, min(16384, max(1, (1 << 28) // (k * d * (2 if grad else 1)))))
        case = _adapt("", T=T, k=k, E=E, d=d, f=f, L=L, r=r, seqs=_log(rng, 1, min(T, 64)), grad=grad,
                      base=rng.choice((0.0, 0.0, 0.3)), zipf=rng.choice((0.0, 0.1, 0.2)),
                      p=rng.choice((0.0, 0.0, 0.1)), train=not grad and rng.random() < 0.5)
    del case["name"]
    return case


# ------------------------------------------------------------------------------------------ inputs

def _normal(gen, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)


def _routing(case, gen):
    """Row metadata of a random routing: chosen experts, rows by expert then token."""
    T, k, E = case["T"], case["k"], case["E"]
    logits = torch.randn((T, E), generator=gen, device="cuda")
    if case.get("zipf"):
        logits -= 3.0 * case["zipf"] * torch.log(torch.arange(1, E + 1, device="cuda", dtype=torch.float32))
    top = logits.topk(k, dim=1)
    idx = top.indices.reshape(-1)
    order = torch.sort(idx, stable=True).indices
    dest = torch.empty_like(order)
    dest[order] = torch.arange(order.numel(), device="cuda")
    counts = torch.bincount(idx, minlength=E)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    return dict(dest=dest.view(T, k).int(), offsets=offsets.int(), row_token=(order // k).int(),
                gate=torch.softmax(top.values, dim=1))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed * 1000003 + 29)
    T, k, E, d = case["T"], case["k"], case["E"], case["d"]
    n = T * k
    s = dict(case=case)
    # the generator's seed and offset, which a program keeps on the GPU and advances from step to step
    s["rng"] = torch.randint(-(1 << 62), 1 << 62, (2,), generator=gen, device="cuda")
    if case["op"] == "dropout":
        s["res"] = _normal(gen, T, d) if case["residual"] else None
        if case["what"] == "rows":
            s["x"] = _normal(gen, T, d)
            return s
        s["route"] = _routing(case, gen)
        s["yexp"] = _normal(gen, n, d)
        s["dy"] = _normal(gen, T, d) if case["what"] == "gradient" else None
        return s
    f, L, r = case["f"], case["L"], case["r"]
    s["route"] = _routing(case, gen)
    # runs of tokens (sequences), each of one adapter or of none
    cuts = torch.randint(0, T, (case["seqs"] - 1,), generator=gen, device="cuda")
    at = torch.zeros(T, dtype=torch.int64, device="cuda").index_add_(0, cuts, torch.ones_like(cuts)).cumsum(0)
    which = torch.randint(0, L, (case["seqs"],), generator=gen, device="cuda")
    without = torch.rand(case["seqs"], generator=gen, device="cuda") < case["base"]
    s["ids"] = torch.where(without, torch.full_like(which, -1), which)[at].int()
    for name, R, C in (("a_gu", 2 * r, d), ("b_gate", r, f), ("b_up", r, f), ("a_down", r, f), ("b_down", r, d)):
        s[name] = _normal(gen, L, E, R, C, std=C ** -0.5 if name[0] == "a" else 0.5 * R ** -0.5)
    s["scale"] = torch.rand(L, generator=gen, device="cuda") + 0.5
    s["x"] = _normal(gen, T, d)
    s["g"], s["u"], s["y"] = _normal(gen, n, f), _normal(gen, n, f), _normal(gen, n, d)
    s["a"] = (s["g"].float() * torch.sigmoid(s["g"].float()) * s["u"].float()).to(torch.bfloat16)
    if case["grad"]:                                                # y: the gradient that reaches the experts
        s["dg"], s["du"], s["dxp"] = _normal(gen, n, f), _normal(gen, n, f), _normal(gen, n, d)
        s["v1"], s["v2"] = _normal(gen, n, 2 * r), _normal(gen, n, r)
    return s


# ------------------------------------------------------------------------------------- plain forms

def run(s):
    case = s["case"]
    if own:
        return _own(s)
    if case["op"] == "dropout":
        return _plain_dropout(s)
    return _plain_backward(s) if case["grad"] else _plain_forward(s)


def _factors(rng, p, site, rows, cols):
    """[rows, cols] fp32: 0 for a dropped element, 1 / (1 - p) for one that is kept, p in steps of 2^-16.

    The 16 bits of element (r, c) are piece c % 8 of Philox4x32 (7 rounds) of the counter
    (c / 8 + site 2^28, r, the offset's low and high half) under the key that the seed is."""
    low, drop = 0xffffffff, int(round(p * 65536))
    k0, k1, o0, o1 = rng[0] & low, (rng[0] >> 32) & low, rng[1] & low, (rng[1] >> 32) & low
    c0 = torch.arange(-(-cols // 8), device=rng.device).view(1, -1) + (site << 28)
    c1 = torch.arange(rows, device=rng.device).view(-1, 1)
    c0, c1 = torch.broadcast_tensors(c0, c1)
    c2, c3 = o0.expand_as(c0), o1.expand_as(c0)
    for i in range(7):
        m0, m1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        a, b = (k0 + i * 0x9E3779B9) & low, (k1 + i * 0xBB67AE85) & low
        c0, c1, c2, c3 = ((m1 >> 32) & low) ^ c1 ^ a, m1 & low, ((m0 >> 32) & low) ^ c3 ^ b, m0 & low
    w = torch.stack([c0, c1, c2, c3], dim=2)
    u = torch.stack([w & 0xffff, w >> 16], dim=3).view(rows, -1)[:, :cols]
    return torch.where(u >= drop, 65536.0 / (65536 - drop), 0.0).float()


def _dropped(v, s, site):
    p = s["case"]["p"]
    return v if p == 0.0 else v * _factors(s["rng"], p, site, *v.shape)


def _plain_dropout(s):
    case = s["case"]
    if case["what"] == "rows":
        out = _dropped(s["x"].float(), s, 0)
        return dict(y=(out if s["res"] is None else out + s["res"].float()).to(torch.bfloat16))
    gate, dest, yexp = s["route"]["gate"], s["route"]["dest"].long(), s["yexp"]
    if case["what"] == "combine":
        out = _dropped((yexp[dest].float() * gate[:, :, None]).sum(dim=1), s, 0)
        return dict(y=(out if s["res"] is None else out + s["res"].float()).to(torch.bfloat16))
    dy = _dropped(s["dy"].float(), s, 0)
    dyexp = torch.empty_like(yexp)
    dyexp[dest] = (dy[:, None, :] * gate[:, :, None]).to(torch.bfloat16)
    return dict(dyexp=dyexp, d_gate=(dy[:, None, :] * yexp[dest].float()).sum(dim=2))


def _groups(s):
    """Rows sorted by expert and adapter, in tiles of up to 64 rows of one expert and adapter."""
    E, L = s["case"]["E"], s["case"]["L"]
    token, off = s["route"]["row_token"].long(), s["route"]["offsets"].long()
    n = token.numel()
    l = s["ids"].long()[token]
    has = (l >= 0) & (l < L)
    key = torch.searchsorted(off[1:], torch.arange(n, device=l.device), right=True) * (L + 1) + torch.where(has, l, L)
    order = torch.sort(key, stable=True).indices
    key = key[order]
    counts = torch.zeros(E * (L + 1), dtype=torch.int64, device=l.device).scatter_add_(0, key, torch.ones_like(key))
    rank = torch.arange(n, device=l.device) - (counts.cumsum(0) - counts)[key]
    tiles = (counts + 63) // 64
    tile = (tiles.cumsum(0) - tiles)[key] + rank // 64
    of = torch.zeros(n // 64 + min(n, E * (L + 1)), dtype=torch.int64, device=l.device)
    of[tile] = key
    return dict(order=order, tile=tile, at=rank % 64, n_tiles=of.numel(), e=of // (L + 1), of=of,
                l=(of % (L + 1)).clamp(max=L - 1), has=has[:, None], token=token,
                scale=s["scale"][l.clamp(0, L - 1)][:, None])


def _padded(v, q):
    p = torch.zeros((q["n_tiles"], 64, v.shape[1]), device=v.device)
    p[q["tile"], q["at"]] = v[q["order"]].float()
    return p


def _low(v, w, q):
    """v [n, K] times the rows' adapters w [L, E, R, K], over K: [n, R] fp32, 0 for rows without one."""
    return _rows(torch.bmm(_padded(v, q), w[q["l"], q["e"]].float().transpose(1, 2)), q)


def _back(v, w, q):
    """v [n, R] times the rows' adapters w [L, E, R, K], over R: [n, K] fp32, 0 for rows without one."""
    return _rows(torch.bmm(_padded(v, q), w[q["l"], q["e"]].float()), q)


def _rows(p, q):
    out = torch.empty((q["order"].numel(), p.shape[2]), device=p.device)
    out[q["order"]] = p[q["tile"], q["at"]]
    return torch.where(q["has"], out, 0.0)


def _adapter_gradient(left, right, s, q):
    """[L, E, R, C] bf16: left^T right over the rows of each expert and adapter."""
    E, L = s["case"]["E"], s["case"]["L"]
    part = torch.bmm(_padded(left, q).transpose(1, 2), _padded(right, q))
    out = torch.zeros((E * (L + 1), *part.shape[1:]), device=part.device).index_add_(0, q["of"], part)
    return out.view(E, L + 1, *part.shape[1:])[:, :L].transpose(0, 1).to(torch.bfloat16)


def _plain_forward(s):
    q, r = _groups(s), s["case"]["r"]
    v1 = _low(_dropped(s["x"][q["token"]].float(), s, 1), s["a_gu"], q)
    g = s["g"].float() + q["scale"] * _back(v1[:, :r], s["b_gate"], q)
    u = s["u"].float() + q["scale"] * _back(v1[:, r:], s["b_up"], q)
    a = torch.where(q["has"], g * torch.sigmoid(g) * u, s["a"].float()).to(torch.bfloat16)
    v2 = _low(_dropped(a.float(), s, 2), s["a_down"], q)
    y = s["y"].float() + q["scale"] * _back(v2, s["b_down"], q)
    out = dict(a=a, y=y.to(torch.bfloat16))
    if s["case"]["train"]:
        out.update(g=g.to(torch.bfloat16), u=u.to(torch.bfloat16), v1=v1.to(torch.bfloat16), v2=v2.to(torch.bfloat16))
    return out


def _plain_backward(s):
    q, r = _groups(s), s["case"]["r"]
    dy, g, u = s["y"].float(), s["g"].float(), s["u"].float()
    dv2 = q["scale"] * _low(dy, s["b_down"], q)
    out = dict(d_b_down=_adapter_gradient(q["scale"] * s["v2"].float(), dy, s, q),
               d_a_down=_adapter_gradient(dv2, _dropped(s["a"].float(), s, 2), s, q))
    da = _dropped(_back(dv2, s["a_down"], q), s, 2)
    sg = torch.sigmoid(g)
    dg = (s["dg"].float() + da * u * sg * (1.0 + g * (1.0 - sg))).to(torch.bfloat16)
    du = (s["du"].float() + da * g * sg).to(torch.bfloat16)
    dv1 = q["scale"] * torch.cat([_low(dg, s["b_gate"], q), _low(du, s["b_up"], q)], dim=1)
    v1 = q["scale"] * s["v1"].float()
    out.update(dg=dg, du=du, d_b_gate=_adapter_gradient(v1[:, :r], dg, s, q), d_b_up=_adapter_gradient(v1[:, r:], du, s, q),
               d_a_gu=_adapter_gradient(dv1, _dropped(s["x"][q["token"]].float(), s, 1), s, q))
    out["dxp"] = (s["dxp"].float() + _dropped(_back(dv1, s["a_gu"], q), s, 1)).to(torch.bfloat16)
    return out


# ------------------------------------------------------------------------------- the package's calls

def _own(s):
    from expert_ffn_layer_top_amd import ops
    case = s["case"]
    drop = lambda site: ops.Dropout(case["p"], s["rng"], site) if case["p"] else None     # noqa: E731
    if case["op"] == "dropout":
        if case["what"] == "rows":
            return dict(y=ops.dropout(s["x"], ops.Dropout(case["p"], s["rng"], 0), residual=s["res"]))
        args = (s["route"]["gate"], s["route"]["dest"], ops.Dropout(case["p"], s["rng"], 0))
        if case["what"] == "combine":
            return dict(y=ops.unpermute_combine_dropout(s["yexp"], *args, residual=s["res"]))
        dyexp, d_gate = ops.unpermute_combine_dropout_bwd(s["dy"], s["yexp"], *args)
        return dict(dyexp=dyexp, d_gate=d_gate)
    plan = ops.adapter_plan(s["ids"], s["route"]["offsets"], case["L"], row_token=s["route"]["row_token"],
                            backward=case["grad"] or case["train"])
    up, down = (s["a_gu"], s["b_gate"], s["b_up"], s["scale"]), (s["a_down"], s["b_down"], s["scale"])
    if case["grad"]:
        out = {}
        out["dg"], out["du"], out["d_a_down"], out["d_b_down"] = ops.adapter_down_bwd(
            s["y"], s["a"], s["v2"], s["g"], s["u"], s["dg"], s["du"], plan, *down, drop=drop(2))
        out["dxp"], out["d_a_gu"], out["d_b_gate"], out["d_b_up"] = ops.adapter_gate_up_bwd(
            out["dg"], out["du"], s["x"], s["v1"], s["dxp"], plan, *up, drop=drop(1))
        return out
    train = case["train"]
    g, u, a, v1 = ops.adapter_gate_up(s["x"], s["g"], s["u"], s["a"], plan, *up, drop=drop(1), want_gu=train, want_v=train)
    y, v2 = ops.adapter_down(a, s["y"], plan, *down, drop=drop(2), want_v=train)
    return dict(a=a, y=y, g=g, u=u, v1=v1, v2=v2) if train else dict(a=a, y=y)


# ------------------------------------------------------------------------------ what it has to move

def work(case):
    T, k, d = case["T"], case["k"], case["d"]
    n = T * k
    if case["op"] == "dropout":
        res = 2 * T * d if case["residual"] else 0
        if case["what"] == "rows":
            return dict(bytes=4 * T * d + res, flops=2 * T * d)
        if case["what"] == "combine":
            return dict(bytes=2 * n * d + 8 * n + res + 2 * T * d, flops=2 * n * d + 2 * T * d)
        return dict(bytes=2 * T * d + 4 * n * d + 12 * n, flops=4 * n * d)
    f, E, L, r = case["f"], case["E"], case["L"], case["r"]
    rows = n * (1.0 - case["base"])                                 # rows with an adapter
    busy = min(E * L, E * min(L, case["seqs"]) * (1.0 - (1.0 - 1.0 / (E * min(L, case["seqs"]))) ** rows))
    weights = busy * (2 * r * d + 2 * r * f + r * f + r * d) * 2
    flops = 2 * rows * (2 * r * d + 2 * r * f + r * f + r * d)
    meta = 8 * n + 4 * T
    if not case["grad"]:
        kept = 4 * n * f + 6 * n * r if case["train"] else 0
        none = 2 * (n - rows) * f
        return dict(bytes=2 * T * d + 4 * n * f + none + 2 * n * f + kept + 4 * n * d + weights + meta, flops=flops)
    grads = E * L * (3 * r * d + 3 * r * f) * 2
    return dict(bytes=2 * n * d + 10 * n * f + 4 * n * f + 6 * n * r + 2 * T * d + 4 * n * d + weights + grads + meta,
                flops=3 * flops)


# -------------------------------------------------------------------------------------- in 64 bits

def _kept(s, site, rows, cols):
    """The factors in 64 bits.  The generator's products are formed from halves of 16 bits."""
    p = s["case"]["p"]
    if p == 0.0:
        return torch.ones((), dtype=torch.float64, device="cuda")
    seed, offset = (int(v) % (1 << 64) for v in s["rng"].tolist())
    key, mask = [seed % (1 << 32), seed >> 32], (1 << 32) - 1
    n8 = (cols + 7) // 8
    ctr = [torch.arange(n8, device="cuda").repeat(rows) | site << 28, torch.arange(rows, device="cuda").repeat_interleave(n8),
           torch.full((rows * n8,), offset % (1 << 32), device="cuda"), torch.full((rows * n8,), offset >> 32, device="cuda")]

    def halves(x, m):
        """(high, low) 32 bits of x m."""
        x0, x1, m0, m1 = x & 0xffff, x >> 16, m & 0xffff, m >> 16
        mid = x1 * m0 + ((x0 * m0) >> 16)
        mid2 = x0 * m1 + (mid & 0xffff)
        return x1 * m1 + (mid >> 16) + (mid2 >> 16), ((mid2 & 0xffff) << 16) | (x0 * m0 & 0xffff)

    for _ in range(7):
        (h0, l0), (h1, l1) = halves(ctr[0], 0xD2511F53), halves(ctr[2], 0xCD9E8D57)
        ctr = [h1 ^ ctr[1] ^ key[0], l1, h0 ^ ctr[3] ^ key[1], l0]
        key = [(key[0] + 0x9E3779B9) & mask, (key[1] + 0xBB67AE85) & mask]
    out = torch.empty((rows, n8, 8), dtype=torch.float64, device="cuda")
    cut = int(round(p * 65536))
    for j, w in enumerate(ctr):
        out[:, :, 2 * j] = ((w % 65536) >= cut).view(rows, n8)
        out[:, :, 2 * j + 1] = ((w // 65536) >= cut).view(rows, n8)
    return out.view(rows, 8 * n8)[:, :cols] / (1.0 - cut / 65536)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "dropout":
        T, d = case["T"], case["d"]
        m = _kept(s, 0, T, d)
        add = 0.0 if s["res"] is None else s["res"].double()
        if case["what"] == "rows":
            return dict(y=s["x"].double() * m + add)
        gate, dest = s["route"]["gate"].double(), s["route"]["dest"].long()
        if case["what"] == "combine":
            y = torch.zeros((T, d), dtype=torch.float64, device="cuda")
            for j in range(case["k"]):
                y += gate[:, j:j + 1] * s["yexp"][dest[:, j]].double()
            return dict(y=y * m + add)
        dy = s["dy"].double() * m
        dyexp = torch.empty(s["yexp"].shape, dtype=torch.float64, device="cuda")
        d_gate = torch.empty_like(gate)
        for j in range(case["k"]):
            dyexp[dest[:, j]] = gate[:, j:j + 1] * dy
            d_gate[:, j] = (dy * s["yexp"][dest[:, j]].double()).sum(1)
        return dict(dyexp=dyexp, d_gate=d_gate)

    E, L, r = case["E"], case["L"], case["r"]
    off, token, ids = s["route"]["offsets"].tolist(), s["route"]["row_token"].cpu(), s["ids"].cpu()
    n = token.numel()
    row_l = ids[token.long()]
    groups = []                                                     # (adapter, expert, its rows)
    for e in range(E):
        mine = row_l[off[e]:off[e + 1]]
        for l in mine.unique().tolist():
            if l >= 0:
                groups.append((l, e, (off[e] + (mine == l).nonzero().view(-1)).cuda()))
    token = token.cuda().long()
    scale = s["scale"].double()
    new = lambda *shape: torch.zeros(shape, dtype=torch.float64, device="cuda")     # noqa: E731
    f, d = case["f"], case["d"]
    mx, ma = _kept(s, 1, n, d), _kept(s, 2, n, f)
    at = lambda m, i: m if m.dim() == 0 else m[i]                   # noqa: E731
    W = lambda name, l, e: s[name][l, e].double()                   # noqa: E731
    if not case["grad"]:
        g, u, a, y = (s[name].double() for name in ("g", "u", "a", "y"))
        v1, v2 = new(n, 2 * r), new(n, r)
        for l, e, i in groups:
            v1[i] = (s["x"][token[i]].double() * at(mx, i)) @ W("a_gu", l, e).t()
            g[i] += scale[l] * (v1[i, :r] @ W("b_gate", l, e))
            u[i] += scale[l] * (v1[i, r:] @ W("b_up", l, e))
            a[i] = g[i] / (1.0 + torch.exp(-g[i])) * u[i]
            v2[i] = (a[i].to(torch.bfloat16).double() * at(ma, i)) @ W("a_down", l, e).t()
            y[i] += scale[l] * (v2[i] @ W("b_down", l, e))
        return dict(a=a, y=y, g=g, u=u, v1=v1, v2=v2) if case["train"] else dict(a=a, y=y)
    dg, du, dxp = (s[name].double() for name in ("dg", "du", "dxp"))
    out = dict(dg=dg, du=du, dxp=dxp)
    for name in ("a_gu", "b_gate", "b_up", "a_down", "b_down"):
        out["d_" + name] = torch.zeros(s[name].shape, dtype=torch.float64, device="cuda")
    for l, e, i in groups:
        dy, g, u = s["y"][i].double(), s["g"][i].double(), s["u"][i].double()
        dv2 = scale[l] * (dy @ W("b_down", l, e).t())
        out["d_b_down"][l, e] = scale[l] * (s["v2"][i].double().t() @ dy)
        out["d_a_down"][l, e] = dv2.t() @ (s["a"][i].double() * at(ma, i))
        da = (dv2 @ W("a_down", l, e)) * at(ma, i)
        sg = 1.0 / (1.0 + torch.exp(-g))
        dg[i] += da * u * (sg + g * sg * (1.0 - sg))
        du[i] += da * g * sg
        hg, hu = dg[i].to(torch.bfloat16).double(), du[i].to(torch.bfloat16).double()
        dv1 = scale[l] * torch.cat([hg @ W("b_gate", l, e).t(), hu @ W("b_up", l, e).t()], dim=1)
        v1 = scale[l] * s["v1"][i].double()
        out["d_b_gate"][l, e], out["d_b_up"][l, e] = v1[:, :r].t() @ hg, v1[:, r:].t() @ hu
        out["d_a_gu"][l, e] = dv1.t() @ (s["x"][token[i]].double() * at(mx, i))
        dxp[i] += (dv1 @ W("a_gu", l, e)) * at(mx, i)
    return out

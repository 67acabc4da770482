"""The W8A8 operators and the scored router, each in its plain form and through the library.

A case names one pass a user's program makes: a router's selection, an RMS norm with
the residual's addition, a linear layer on int8 operands, one grouped product of the
expert layer, or the whole of what stands between two residual additions.
"""
import math

import torch

own = False

DEV = "cuda"
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
EPS = 1e-6
SWIGLU, DOWN = "swiglu", "down"


def _router(score, groups, kept, top, renorm=True, scale=1.0):
    return {"score": score, "groups": groups, "kept": kept, "group_top": top, "renorm": renorm, "scale": scale}


def listed():
    return [
        # one sequence's next token: 256 experts in 8 groups, sigmoid scores and a balance bias
        {"name": "router 1 token", "op": "route", "T": 1, "E": 256, "k": 8, "masked": False, "bias": True,
         **_router("sigmoid", 8, 4, 2, scale=2.5)},
        # a prefill chunk through the same router
        {"name": "router 8192 tokens", "op": "route", "T": 8192, "E": 256, "k": 8, "masked": False, "bias": True,
         **_router("sigmoid", 8, 4, 2, scale=2.5)},
        # the norm before the expert layer, one token (hidden 2048)
        {"name": "norm 1 token", "op": "norm", "T": 1, "H": 2048, "residual": True},
        # the same norm over a long prefill (hidden 7168)
        {"name": "norm 8192 tokens", "op": "norm", "T": 8192, "H": 7168, "residual": True},
        # decode of 16 sequences: norm, int8 rows, a dense projection
        {"name": "norm linear 16 rows", "op": "linear", "first": "norm", "T": 16, "K": 4096, "N": 14336, "f32": False},
        # prefill of the same kind
        {"name": "norm linear 4096 rows", "op": "linear", "first": "norm", "T": 4096, "K": 7168, "N": 4096, "f32": False},
        # an odd number of rows and columns, fp32 results (a head whose result is not rounded)
        {"name": "linear 333 rows", "op": "linear", "first": "quantize", "T": 333, "K": 768, "N": 2064, "f32": True},
        # the largest product: a long prefill through a wide projection
        {"name": "linear 8192 rows", "op": "linear", "first": "quantize", "T": 8192, "K": 4096, "N": 14336, "f32": False},
        # gate/up of a decode batch: about 4 rows for each of 128 experts
        {"name": "gate up 64 tokens", "op": "grouped", "kind": SWIGLU, "T": 64, "E": 128, "k": 8, "H": 2048, "I": 768,
         "zipf": False},
        # down projection of a prefill whose experts' popularity follows Zipf's law
        {"name": "down 2048 tokens", "op": "grouped", "kind": DOWN, "T": 2048, "E": 128, "k": 8, "H": 2048, "I": 768,
         "zipf": True},
        # decode: norm, router and the whole expert layer for 16 tokens
        {"name": "experts 16 tokens", "op": "layer", "T": 16, "E": 128, "begin": 0, "local": 128, "k": 8, "H": 2048,
         "I": 768, "zipf": False, **_router("softmax", 1, 1, 1)},
        # prefill on one rank of eight: 32 of 256 experts
        {"name": "experts 2048 tokens", "op": "layer", "T": 2048, "E": 256, "begin": 32, "local": 32, "k": 8, "H": 7168,
         "I": 2048, "zipf": False, **_router("sigmoid", 8, 4, 2, scale=2.5)},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _draw_router(rng, E, k):
    groups = rng.choice([1, 1] + [n for n in (2, 4, 8) if E % (2 * n) == 0])
    kept = rng.randint(1, groups)
    while kept * (E // groups) < k:
        kept += 1
    return _router(rng.choice(["sigmoid", "softmax"]), groups, kept, rng.choice([1, 2]), rng.random() < 0.8,
                   round(rng.uniform(0.5, 3.0), 3))


def draw(rng):
    op = rng.choice(["route", "norm", "linear", "linear", "grouped", "grouped", "layer"])
    if op == "route":
        E, k = 8 * rng.randint(2, 64), rng.randint(1, 12)
        return {"op": op, "T": _log(rng, 1, 4096), "E": E, "k": k, "masked": rng.random() < 0.5, "bias": rng.random() < 0.7,
                **_draw_router(rng, E, k)}
    if op == "norm":
        return {"op": op, "T": _log(rng, 1, 8192), "H": 8 * _log(rng, 16, 896), "residual": rng.random() < 0.7}
    if op == "linear":
        first = rng.choice(["norm", "quantize"])
        return {"op": op, "first": first, "T": _log(rng, 1, 4096), "K": 128 * _log(rng, 2, 56),
                "N": 16 * _log(rng, 8, 512), "f32": first == "quantize" and rng.random() < 0.5}
    E = rng.choice([8, 16, 32, 60, 128])
    case = {"op": op, "T": _log(rng, 1, 1024), "E": E, "k": rng.randint(1, min(8, E)), "H": 128 * rng.randint(2, 16),
            "I": 128 * rng.randint(1, 8), "zipf": rng.random() < 0.5}
    if op == "grouped":
        return {**case, "kind": rng.choice([SWIGLU, DOWN])}
    begin = rng.choice([0, 0, E // 4])
    return {**case, "begin": begin, "local": E // 2 if begin else E, **_draw_router(rng, E, case["k"])}


# ---- inputs ---------------------------------------------------------------------------------

def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _scales(g, *shape):
    return torch.rand(*shape, generator=g, device=DEV) * 0.015 + 0.005


def _codes(g, *shape):
    return torch.randint(-127, 128, shape, generator=g, device=DEV, dtype=torch.int8)


def _bias(g, case):
    """A balance bias of a tenth of what the scores spread over."""
    return _normal(g, case["E"]) * (0.1 if case["score"] == "sigmoid" else 0.1 / case["E"])


def _logits(g, T, E, zipf):
    """Router logits: normal, or drawn so that the experts' popularity follows Zipf's law (s = 1.1)."""
    if not zipf:
        return _normal(g, T, E)
    p = torch.arange(1, E + 1, device=DEV, dtype=F32).pow(-1.1)[torch.randperm(E, generator=g, device=DEV)]
    u = torch.rand(T, E, generator=g, device=DEV).clamp_(1e-7, 1 - 1e-7)
    return torch.log(p) - torch.log(-torch.log(u))


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(case)
    op = case["op"]
    if op == "route":
        s["logits"] = _normal(g, case["T"], case["E"]) * 1.5
        if case["masked"]:       # experts that are switched off for some tokens
            s["logits"][torch.rand(case["T"], case["E"], generator=g, device=DEV) < 0.2] = -math.inf
        s["bias"] = _bias(g, case) if case["bias"] else None
    elif op == "norm":
        s["x"] = _normal(g, case["T"], case["H"]).to(BF16)
        s["res"] = (_normal(g, case["T"], case["H"]) * 2).to(BF16) if case["residual"] else None
        s["gain"] = (1 + 0.2 * _normal(g, case["H"])).to(BF16)
    elif op == "linear":
        s["x"] = _normal(g, case["T"], case["K"]).to(BF16)
        if case["first"] == "norm":
            s["res"] = (_normal(g, case["T"], case["K"]) * 2).to(BF16)
            s["gain"] = (1 + 0.2 * _normal(g, case["K"])).to(BF16)
        s["w"], s["ws"] = _codes(g, case["N"], case["K"]), _scales(g, case["N"]) / math.sqrt(case["K"])
    elif op == "grouped":
        T, E, k, H, I = (case[n] for n in ("T", "E", "k", "H", "I"))
        ids = _logits(g, T, E, case["zipf"]).argsort(dim=-1, descending=True)[:, :k].to(torch.int32).contiguous()
        # what the permutation gives: rows sorted by expert, each expert's in token order
        order = ids.flatten().long().argsort(stable=True)
        s["perm"] = order.to(torch.int32)
        s["offsets"] = torch.searchsorted(ids.flatten().long()[order], torch.arange(E + 1, device=DEV)).to(torch.int32)
        rows, K, N = (T, H, 2 * I) if case["kind"] == SWIGLU else (T * k, I, H)
        s["a"], s["as"] = _codes(g, rows, K), _scales(g, rows)
        s["w"], s["ws"] = _codes(g, E, N, K), _scales(g, E, N) / math.sqrt(K)
    else:
        T, E, L, H, I = (case[n] for n in ("T", "E", "local", "H", "I"))
        s["x"], s["res"] = _normal(g, T, H).to(BF16), (_normal(g, T, H) * 2).to(BF16)
        s["gain"] = (1 + 0.2 * _normal(g, H)).to(BF16)
        s["logits"], s["bias"] = _logits(g, T, E, case["zipf"]), _bias(g, case)
        s["w13"], s["s13"] = _codes(g, L, 2 * I, H), _scales(g, L, 2 * I) / math.sqrt(H)
        s["w2"], s["s2"] = _codes(g, L, H, I), _scales(g, L, H) / math.sqrt(I)
    return s


# ---- the plain form ---------------------------------------------------------------------------

def _plain_route(s):
    """Scores are binary32 values of the exact function (computed in 64 bits: a selection next to a border), and
    everything after them is binary32 arithmetic; larger selection score first, then the lower index."""
    T, E = s["logits"].shape
    l = s["logits"].double()
    if s["score"] == "sigmoid":
        score = (1 / (1 + torch.exp(-l))).float()
    else:
        p = torch.exp(l - l.amax(-1, keepdim=True))
        score = (p / p.sum(-1, keepdim=True)).float()
    score = torch.where(torch.isneginf(s["logits"]), torch.zeros_like(score), score)
    choice = torch.where(torch.isneginf(s["logits"]), s["logits"], score if s["bias"] is None else score + s["bias"])
    key = choice.double()
    if s["groups"] > 1:
        in_group = choice.view(T, s["groups"], -1).sort(dim=-1, descending=True, stable=True).values
        of_group = in_group[..., 0] if s["group_top"] == 1 else in_group[..., 0] + in_group[..., 1]
        rank = of_group.argsort(dim=-1, descending=True, stable=True).argsort(-1)
        out = (rank >= s["kept"]).repeat_interleave(E // s["groups"], -1)
        key = torch.where(torch.isneginf(key), key.new_tensor(-1e300), key).masked_fill(out, -math.inf)
    ids = key.argsort(dim=-1, descending=True, stable=True)[:, :s["k"]]
    w = score.gather(-1, ids)
    if s["renorm"]:
        total = w.sum(-1, keepdim=True)
        w = torch.where(total > 0, w / total, torch.zeros_like(w))
    return ids.to(torch.int32), w * s["scale"]


def _plain_norm(s):
    h = s["x"].float()
    if s["res"] is not None:
        h = (h + s["res"].float()).to(BF16).float()
    r = torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS)
    return h, h * r * s["gain"].float()


def _plain_quantize(y):
    """The codes as float values, and the scale of each row. The product first, then the division: of bfloat16 values
    many lie exactly between two codes, and a factor 127 / top rounded before it would push them off."""
    top = y.abs().amax(-1, keepdim=True)
    q = torch.round(y * 127 / torch.where(top > 0, top, torch.ones_like(top)))
    return q, top / 127


def _plain_grouped(a, scale, offsets, w, ws, kind, block):
    """Rows a[r] (codes), sorted by expert: blocks of `block` rows of one expert, one batched product over them.
    Returns one row more than it was given, to take what blocks hold past their expert's last row."""
    R, E = a.shape[0], w.shape[0]
    offsets = offsets.long()
    blocks = (offsets[1:] - offsets[:-1] + block - 1) // block
    last = blocks.cumsum(0)
    at = torch.arange(min(E, R) + R // block, device=DEV)        # at least as many blocks as there can be
    e = torch.searchsorted(last, at, right=True).clamp(max=E - 1)
    row = (offsets[e] + (at - last[e] + blocks[e]) * block)[:, None] + torch.arange(block, device=DEV)
    row = torch.where(row < offsets[e + 1][:, None], row, R)
    there = row.clamp(max=R - 1)
    c = torch.bmm(a[there], w[e].float().transpose(1, 2)) * scale[there] * ws[e][:, None, :]
    if kind == SWIGLU:
        gate, up = c.chunk(2, -1)
        c = gate / (1 + torch.exp(-gate)) * up
    out = c.new_zeros(R + 1, c.shape[-1])
    out[row.flatten()] = c.flatten(0, 1)
    return out


def _block(rows, experts):
    return max(4, min(64, 1 << max(0, rows // experts).bit_length()))


def _plain_layer(s):
    T, k, L = s["T"], s["k"], s["local"]
    h, y = _plain_norm(s)
    q, scale = _plain_quantize(y)
    ids, w = _plain_route(s)
    e = ids.flatten().long() - s["begin"]
    e = torch.where((e >= 0) & (e < L), e, L)                    # slots of other ranks' experts come last
    order = e.argsort(stable=True)
    offsets = torch.searchsorted(e[order], torch.arange(L + 1, device=DEV))
    token, block = order // k, _block(T * k, s["E"])
    mid = _plain_grouped(q[token], scale[token], offsets, s["w13"], s["s13"], SWIGLU, block)[:-1].to(BF16).float()
    q, scale = _plain_quantize(mid)
    out = _plain_grouped(q, scale, offsets, s["w2"], s["s2"], DOWN, block)[:-1].to(BF16).float()
    out = torch.where((e < L)[order][:, None], out, torch.zeros_like(out)) * w.flatten()[order][:, None]
    slots = torch.empty_like(out)
    slots[order] = out
    return ids, slots.view(T, k, -1).sum(1).to(BF16), h.to(BF16)


def run(state):
    s, op = state, state["op"]
    if own:
        return _own(s)
    if op == "route":
        return _plain_route(s)
    if op == "norm":
        h, y = _plain_norm(s)
        return (y.to(BF16), h.to(BF16)) if s["residual"] else y.to(BF16)
    if op == "linear":
        h, y = _plain_norm(s) if s["first"] == "norm" else (None, s["x"].float())
        q, scale = _plain_quantize(y)
        c = (q @ s["w"].float().t()) * scale * s["ws"]
        c = c if s["f32"] else c.to(BF16)
        return (c, h.to(BF16)) if s["first"] == "norm" else c
    if op == "grouped":
        perm = s["perm"].long()
        at = perm // s["k"] if s["kind"] == SWIGLU else torch.arange(perm.numel(), device=DEV)
        return _plain_grouped(s["a"].float()[at], s["as"][at][:, None], s["offsets"], s["w"], s["ws"], s["kind"],
                              _block(s["T"] * s["k"], s["E"]))[:-1].to(BF16)
    return _plain_layer(s)


# ---- the library's operators --------------------------------------------------------------------

def _own(s):
    from w4a16_grouped_gemm_amd import ops

    op = s["op"]
    if op == "route":
        return ops.route_scored(s["logits"], s["k"], bias=s["bias"], score=s["score"], num_groups=s["groups"],
                                topk_groups=s["kept"], group_top=s["group_top"], renormalize=s["renorm"],
                                scale=s["scale"])
    if op == "norm":
        if not s["residual"]:
            return ops.rms_norm(s["x"], s["gain"], eps=EPS)
        return ops.add_rms_norm(s["x"], s["res"], s["gain"], eps=EPS)
    if op == "linear":
        if s["first"] == "norm":
            q, scale, h = ops.add_rms_norm_int8(s["x"], s["res"], s["gain"], eps=EPS)
        else:
            q, scale = ops.int8_quantize(s["x"])
        c = ops.dense_gemm_w8a8(q, scale, s["w"], s["ws"], out_dtype=F32 if s["f32"] else BF16)
        return (c, h) if s["first"] == "norm" else c
    if op == "grouped":
        swiglu = s["kind"] == SWIGLU
        return ops.grouped_gemm_w8a8(ops.W13_SWIGLU if swiglu else ops.W2, s["a"], s["as"], s["offsets"], s["w"],
                                     s["ws"], num_tokens=s["T"], top_k=s["k"],
                                     a_row_index=s["perm"] if swiglu else None)
    q, scale, h = ops.add_rms_norm_int8(s["x"], s["res"], s["gain"], eps=EPS)
    ids, w = ops.route_scored(s["logits"], s["k"], bias=s["bias"], score=s["score"], num_groups=s["groups"],
                              topk_groups=s["kept"], group_top=s["group_top"], renormalize=s["renorm"],
                              scale=s["scale"])
    out = ops.moe_w8a8_forward(q, scale, ids, w, s["w13"], s["s13"], s["w2"], s["s2"], num_experts=s["E"],
                               expert_begin=s["begin"])
    return ids, out, h


# ---- what a pass cannot do without -----------------------------------------------------------------

def work(case):
    op, T = case["op"], case["T"]
    if op == "route":
        E, k = case["E"], case["k"]
        return {"bytes": 4 * T * E + 4 * E + 8 * T * k, "flops": T * E * 20}
    if op == "norm":
        n = T * case["H"]
        return {"bytes": (8 if case["residual"] else 4) * n + 2 * case["H"], "flops": 6 * n}
    if op == "linear":
        K, N = case["K"], case["N"]
        first = 6 if case["first"] == "norm" else 2          # x, residual and its sum; or x alone
        return {"bytes": first * T * K + N * K + 4 * N + T * N * (4 if case["f32"] else 2), "flops": 2 * T * N * K}
    E, k, H, I = (case[n] for n in ("E", "k", "H", "I"))
    L = case.get("local", E)
    slots = T * k * L / E
    # experts that at least one slot reaches, for slots spread evenly (popular ones draw more, so fewer are reached)
    reached = L * (1 - (1 - k / E) ** T)
    if op == "grouped":
        rows, K, N, cols = (T, H, 2 * I, I) if case["kind"] == SWIGLU else (T * k, I, H, H)
        return {"bytes": rows * (K + 4) + reached * N * (K + 4) + 2 * slots * cols + 4 * (T * k + E + 1),
                "flops": 2 * slots * N * K}
    return {"bytes": 8 * T * H + 4 * T * E + 4 * T * k + reached * (3 * H * I + 4 * (2 * I + H)),
            "flops": 6 * slots * H * I}


# ---- the definition in 64 bits ------------------------------------------------------------------------

def _exact_route(s):
    T, E = s["logits"].shape
    l, off = s["logits"].double(), s["logits"] == -math.inf
    prob = torch.sigmoid(l) if s["score"] == "sigmoid" else torch.softmax(l, -1)
    prob = prob.masked_fill(off, 0.0).nan_to_num(0.0)
    # the selection goes by binary32 scores plus the bias; an expert that is switched off comes after all others
    pick = prob.float() if s["bias"] is None else prob.float() + s["bias"]
    pick = pick.double().masked_fill(off, -math.inf)
    G, size = s["groups"], E // s["groups"]
    ids = torch.empty(T, s["k"], dtype=torch.int64, device=DEV)
    allowed = torch.ones(T, E, dtype=torch.bool, device=DEV)
    if G > 1:
        best = pick.view(T, G, size).clone()
        total = best.amax(-1)
        if s["group_top"] == 2:
            best.scatter_(-1, best.argmax(-1, keepdim=True), -math.inf)
            total = (total.float() + best.amax(-1).float()).double()
        total[total == -math.inf] = -1e30
        allowed.zero_()
        for _ in range(s["kept"]):
            m = total.amax(-1, keepdim=True)
            at = (total == m).to(torch.int32).argmax(-1)            # the first group that has the maximum
            total[torch.arange(T, device=DEV), at] = -1e38
            allowed.view(T, G, size)[torch.arange(T, device=DEV), at] = True
    pick[pick == -math.inf] = -1e30
    pick[~allowed] = -1e37
    for j in range(s["k"]):
        m = pick.amax(-1, keepdim=True)
        ids[:, j] = (pick == m).to(torch.int32).argmax(-1)
        pick[torch.arange(T, device=DEV), ids[:, j]] = -math.inf
    w = prob.gather(-1, ids)
    if s["renorm"]:
        w = w / w.sum(-1, keepdim=True).clamp(min=1e-300)
    return ids.to(torch.int32), w * s["scale"]


def _exact_norm(s):
    h = s["x"].double()
    if s["res"] is not None:
        h = h + s["res"].double()
    kept = h.float().to(BF16).double()
    return h, kept / (kept.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * s["gain"].double()


def _exact_quantize(y):
    top = y.abs().max(-1, keepdim=True).values
    return (127.0 * y / top.clamp(min=1e-300)).round(), top / 127.0


def _exact_experts(rows, scale, ids, w, ws, kind):
    """ids[r]: the expert of row r, or one past the last for a row of none (its result is zero)."""
    out = torch.zeros(rows.shape[0], w.shape[1] // 2 if kind == SWIGLU else w.shape[1], dtype=F64, device=DEV)
    for e in range(w.shape[0]):
        at = (ids == e).nonzero().flatten()
        if at.numel():
            c = (rows[at] @ w[e].double().T) * scale[at] * ws[e].double()
            if kind == SWIGLU:
                n = w.shape[1] // 2
                c = c[:, :n] * torch.sigmoid(c[:, :n]) * c[:, n:]
            out[at] = c
    return out


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "route":
        return _exact_route(s)
    if op == "norm":
        h, y = _exact_norm(s)
        return (y, h) if case["residual"] else y
    if op == "linear":
        h, y = _exact_norm(s) if case["first"] == "norm" else (None, s["x"].double())
        q, scale = _exact_quantize(y)
        c = torch.cat([q @ w.double().T for w in s["w"].split(2048)], 1) * scale * s["ws"].double()
        return (c, h) if case["first"] == "norm" else c
    if op == "grouped":
        at = torch.arange(s["perm"].numel(), device=DEV)
        e = torch.bucketize(at, s["offsets"][1:].long(), right=True)
        if case["kind"] == SWIGLU:
            at = s["perm"].long().div(case["k"], rounding_mode="floor")
        return _exact_experts(s["a"].double()[at], s["as"].double()[at][:, None], e, s["w"], s["ws"], case["kind"])
    h, y = _exact_norm(s)
    q, scale = _exact_quantize(y)
    ids, w = _exact_route(s)
    e = ids.flatten().long() - case["begin"]
    e[(e < 0) | (e >= case["local"])] = case["local"]
    token = torch.arange(e.numel(), device=DEV).div(case["k"], rounding_mode="floor")
    mid = _exact_experts(q[token], scale[token], e, s["w13"], s["s13"], SWIGLU).to(BF16).double()
    q, scale = _exact_quantize(mid)
    out = _exact_experts(q, scale, e, s["w2"], s["s2"], DOWN).to(BF16).double()
    return ids, (out.view(case["T"], case["k"], -1) * w[:, :, None]).sum(1), h

"""The FP8 operators (e4m3 codes, a scale for each block of 128), each in its plain form and through the library.

A case names one pass a user's program makes: the norm that turns a model's rows into FP8 rows, weights turned
into FP8 blocks when a model is loaded, a linear layer on FP8 operands, one grouped product of the expert layer,
or the norm and the whole expert layer behind it.
"""
import math

import torch

own = False

DEV = "cuda"
BF16, F32, F64, FP8 = torch.bfloat16, torch.float32, torch.float64, torch.float8_e4m3fn
EPS = 1e-6
TOP = 448.0                     # the largest e4m3 value
NOTHING = 2.0 ** -100           # a block whose largest magnitude is below this counts as zero
SWIGLU, DOWN = "swiglu", "down"


def listed():
    return [
        # the norm before a linear or expert layer, one sequence's next token (hidden 2048)
        {"name": "norm 1 token", "op": "norm", "T": 1, "K": 2048, "residual": True, "pow2": False},
        # the same norm over a long prefill (hidden 7168)
        {"name": "norm 8192 tokens", "op": "norm", "T": 8192, "K": 7168, "residual": True, "pow2": False},
        # a projection's weights when the model is loaded; the last block of rows is half one
        {"name": "weights 2112 x 7168", "op": "weights", "E": 1, "N": 2112, "K": 7168, "pow2": False},
        # the gate and up weights of one rank's 32 experts, scales that are powers of two
        {"name": "weights of 32 experts", "op": "weights", "E": 32, "N": 4096, "K": 7168, "pow2": True},
        # decode of one sequence: norm, then a wide projection
        {"name": "norm linear 1 row", "op": "linear", "first": "norm", "T": 1, "K": 4096, "N": 14336, "f32": False,
         "pow2": False},
        # an odd number of rows, a ragged block of columns, results that are not rounded
        {"name": "linear 333 rows", "op": "linear", "first": "quantize", "T": 333, "K": 7168, "N": 2112, "f32": True,
         "pow2": False},
        # prefill: norm, then a projection
        {"name": "norm linear 4096 rows", "op": "linear", "first": "norm", "T": 4096, "K": 7168, "N": 4096, "f32": False,
         "pow2": True},
        # the largest product: a long prefill through a wide projection
        {"name": "linear 8192 rows", "op": "linear", "first": "quantize", "T": 8192, "K": 4096, "N": 14336, "f32": False,
         "pow2": False},
        # gate/up of a decode batch: about 4 rows for each of 128 experts
        {"name": "gate up 64 tokens", "op": "grouped", "kind": SWIGLU, "T": 64, "E": 128, "k": 8, "H": 2048, "I": 768,
         "zipf": False},
        # down projection of a prefill whose experts' popularity follows Zipf's law
        {"name": "down 2048 tokens", "op": "grouped", "kind": DOWN, "T": 2048, "E": 128, "k": 8, "H": 2048, "I": 768,
         "zipf": True},
        # decode of 16 sequences: norm and the expert layer
        {"name": "experts 16 tokens", "op": "layer", "T": 16, "E": 128, "begin": 0, "local": 128, "k": 8, "H": 2048,
         "I": 768, "zipf": False, "pow2": False},
        # prefill on one rank of eight: 32 of 256 experts
        {"name": "experts 2048 tokens", "op": "layer", "T": 2048, "E": 256, "begin": 32, "local": 32, "k": 8, "H": 7168,
         "I": 2048, "zipf": False, "pow2": False},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["norm", "weights", "linear", "linear", "linear", "grouped", "grouped", "layer", "layer"])
    pow2 = rng.random() < 0.4
    if op == "norm":
        return {"op": op, "T": _log(rng, 1, 8192), "K": 128 * _log(rng, 1, 56), "residual": rng.random() < 0.7, "pow2": pow2}
    if op == "weights":
        return {"op": op, "E": _log(rng, 1, 32), "N": 16 * _log(rng, 1, 256), "K": 128 * _log(rng, 1, 56), "pow2": pow2}
    if op == "linear":
        first = rng.choice(["norm", "quantize"])
        return {"op": op, "first": first, "T": _log(rng, 1, 4096), "K": 128 * _log(rng, 1, 56),
                "N": 16 * _log(rng, 1, 512), "f32": first == "quantize" and rng.random() < 0.4, "pow2": pow2}
    E = rng.choice([8, 16, 32, 60, 128])
    case = {"op": op, "T": _log(rng, 1, 1024), "E": E, "k": rng.randint(1, min(8, E)), "H": 128 * rng.randint(1, 16),
            "I": 128 * rng.randint(1, 8), "zipf": rng.random() < 0.5}
    if op == "grouped":
        return {**case, "kind": rng.choice([SWIGLU, DOWN])}
    begin = rng.choice([0, 0, E // 4])
    return {**case, "begin": begin, "local": E // 2 if begin else E, "pow2": pow2}


# ---- inputs ---------------------------------------------------------------------------------

def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _codes(g, *shape):
    """Codes of normal values, each block's largest near the largest code."""
    out = torch.empty(shape, dtype=FP8, device=DEV)
    for part in out.view(-1, shape[-1]).split(1 << 16):
        part.copy_((_normal(g, *part.shape) * 110).clamp_(-TOP, TOP))
    return out


def _scales(g, *shape):
    return torch.rand(*shape, generator=g, device=DEV) * 0.006 + 0.007


def _logits(g, T, E, zipf):
    """Router logits: normal, or drawn so that the experts' popularity follows Zipf's law (s = 1.1)."""
    if not zipf:
        return _normal(g, T, E)
    p = torch.arange(1, E + 1, device=DEV, dtype=F32).pow(-1.1)[torch.randperm(E, generator=g, device=DEV)]
    u = torch.rand(T, E, generator=g, device=DEV).clamp_(1e-7, 1 - 1e-7)
    return torch.log(p) - torch.log(-torch.log(u))


def _blocks(n):
    return -(-n // 128)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(case)
    op = case["op"]
    if op in ("norm", "linear"):
        T, K = case["T"], case["K"]
        s["x"] = _normal(g, T, K).to(BF16)
        if op == "norm" or case["first"] == "norm":
            s["res"] = (_normal(g, T, K) * 2).to(BF16) if op == "linear" or case["residual"] else None
            s["gain"] = (1 + 0.2 * _normal(g, K)).to(BF16)
    if op == "linear":
        s["w"] = _codes(g, case["N"], K)
        s["ws"] = _scales(g, _blocks(case["N"]), K // 128) / math.sqrt(K)
    elif op == "weights":
        s["w"] = torch.empty(case["E"], case["N"], case["K"], dtype=BF16, device=DEV)
        for w in s["w"]:
            w.copy_(_normal(g, case["N"], case["K"]) / math.sqrt(case["K"]))
    elif op == "grouped":
        T, E, k, H, I = (case[n] for n in ("T", "E", "k", "H", "I"))
        ids = _logits(g, T, E, case["zipf"]).argsort(dim=-1, descending=True)[:, :k].to(torch.int32).contiguous()
        # what the permutation gives: rows sorted by expert, each expert's in token order
        order = ids.flatten().long().argsort(stable=True)
        s["perm"] = order.to(torch.int32)
        s["offsets"] = torch.searchsorted(ids.flatten().long()[order], torch.arange(E + 1, device=DEV)).to(torch.int32)
        rows, K, N = (T, H, 2 * I) if case["kind"] == SWIGLU else (T * k, I, H)
        s["a"], s["as"] = _codes(g, rows, K), _scales(g, rows, K // 128)
        s["w"], s["ws"] = _codes(g, E, N, K), _scales(g, E, N // 128, K // 128) / math.sqrt(K)
    elif op == "layer":
        T, E, L, k, H, I = (case[n] for n in ("T", "E", "local", "k", "H", "I"))
        s["x"], s["res"] = _normal(g, T, H).to(BF16), (_normal(g, T, H) * 2).to(BF16)
        s["gain"] = (1 + 0.2 * _normal(g, H)).to(BF16)
        top = _logits(g, T, E, case["zipf"]).softmax(-1).sort(dim=-1, descending=True)
        s["ids"] = top.indices[:, :k].to(torch.int32).contiguous()
        s["w"] = (top.values[:, :k] / top.values[:, :k].sum(-1, keepdim=True)).contiguous()
        s["w13"], s["s13"] = _codes(g, L, 2 * I, H), _scales(g, L, 2 * I // 128, H // 128) / math.sqrt(H)
        s["w2"], s["s2"] = _codes(g, L, H, I), _scales(g, L, H // 128, I // 128) / math.sqrt(I)
    return s


# ---- the plain form ---------------------------------------------------------------------------

def _plain_norm(s):
    """The sum h, the rows h times the gain (exact: products of bfloat16 values), and what the norm multiplies them by."""
    h = s["x"].float()
    if s["res"] is not None:
        h = (h + s["res"].float()).to(BF16).float()
    return h, h * s["gain"].float(), torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS)


def _plain_scale(top, pow2):
    """The scale of blocks whose largest magnitude is `top`: top / 448, or the least power of two that is not less."""
    if pow2:
        m, e = torch.frexp(top)
        s = torch.ldexp(torch.ones_like(top), e - 9 + (m > 0.875).int())
    else:
        s = top / TOP
    return torch.where(top >= NOTHING, s, torch.zeros_like(s))


def _plain_codes(y, top, pow2):
    """The product first, then the division: of bfloat16 values many lie exactly between two codes, and a factor
    448 / top rounded before it would push them off."""
    scale = _plain_scale(top, pow2)
    over = scale if pow2 else top
    q = y * (1.0 if pow2 else TOP) / torch.where(over > 0, over, torch.ones_like(over))
    return torch.where(top >= NOTHING, q, torch.zeros_like(q)).to(FP8), scale


def _plain_quantize(y, pow2, factor=None):
    """Codes, and a scale for each row's blocks of 128, of y, or of y with a factor for each row. The factor is the
    same in a value and its block's largest, so codes go without it, except where a power of two stands between."""
    b = y.view(y.shape[0], -1, 128)
    if factor is None:
        q, scale = _plain_codes(b, b.abs().amax(-1, keepdim=True), pow2)
    elif pow2:
        b = b * factor[..., None]
        q, scale = _plain_codes(b, b.abs().amax(-1, keepdim=True), True)
    else:
        top = b.abs().amax(-1, keepdim=True)
        q, _ = _plain_codes(b, top, False)
        scale = _plain_scale(top * factor[..., None], False)
    return q.view(y.shape), scale[..., 0]


def _plain_weights(w, pow2):
    E, N, K = w.shape
    full = torch.zeros(E, _blocks(N) * 128, K, device=DEV)
    full[:, :N] = w
    b = full.view(E, -1, 128, K // 128, 128)
    top = b.abs().amax((2, 4), keepdim=True)
    q, scale = _plain_codes(b, top, pow2)
    return q.view(E, -1, K)[:, :N], scale[:, :, 0, :, 0]


def _values(q, scale):
    """Rows of codes with a scale for each 128: the values they stand for."""
    return (q.float().view(*scale.shape, 128) * scale[..., None]).view(q.shape)


def _weight_values(w, ws):
    """[..., N, K] codes with a scale for each block of 128 x 128."""
    N = w.shape[-2]
    return _values(w, ws.repeat_interleave(128, -2)[..., :N, :])


def _plain_grouped(a, offsets, w, ws, kind, block):
    """Rows of values a[r], sorted by expert: blocks of `block` rows of one expert, one batched product over them.
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
    values = _weight_values(w.view(torch.uint8)[e].view(FP8), ws[e])
    c = torch.bmm(a[there], values.transpose(1, 2))
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
    h, u, r = _plain_norm(s)
    a = _values(*_plain_quantize(u, s["pow2"], r))
    e = s["ids"].flatten().long() - s["begin"]
    e = torch.where((e >= 0) & (e < L), e, L)                    # slots of other ranks' experts come last
    order = e.argsort(stable=True)
    offsets = torch.searchsorted(e[order], torch.arange(L + 1, device=DEV))
    token, block = order // k, _block(T * k, s["E"])
    mid = _plain_grouped(a[token], offsets, s["w13"], s["s13"], SWIGLU, block)[:-1].to(BF16).float()
    a = _values(*_plain_quantize(mid, s["pow2"]))
    out = _plain_grouped(a, offsets, s["w2"], s["s2"], DOWN, block)[:-1].to(BF16).float()
    out = torch.where((e < L)[order][:, None], out, torch.zeros_like(out)) * s["w"].flatten()[order][:, None]
    slots = torch.empty_like(out)
    slots[order] = out
    return slots.view(T, k, -1).sum(1).to(BF16), h.to(BF16)


def run(state):
    s, op = state, state["op"]
    if own:
        return _own(s)
    if op == "norm":
        h, u, r = _plain_norm(s)
        q, scale = _plain_quantize(u, s["pow2"], r)
        return (q, scale, h.to(BF16)) if s["residual"] else (q, scale)
    if op == "weights":
        return _plain_weights(s["w"], s["pow2"])
    if op == "linear":
        h, u, r = _plain_norm(s) if s["first"] == "norm" else (None, s["x"].float(), None)
        c = _values(*_plain_quantize(u, s["pow2"], r)) @ _weight_values(s["w"], s["ws"]).t()
        c = c if s["f32"] else c.to(BF16)
        return (c, h.to(BF16)) if s["first"] == "norm" else c
    if op == "grouped":
        a = _values(s["a"], s["as"])
        a = a[s["perm"].long() // s["k"]] if s["kind"] == SWIGLU else a
        return _plain_grouped(a, s["offsets"], s["w"], s["ws"], s["kind"], _block(s["T"] * s["k"], s["E"]))[:-1].to(BF16)
    return _plain_layer(s)


# ---- the library's operators --------------------------------------------------------------------

def _own(s):
    from w4a16_grouped_gemm_amd import ops

    op = s["op"]
    if op == "norm":
        if not s["residual"]:
            return ops.rms_norm_fp8(s["x"], s["gain"], eps=EPS, pow2=s["pow2"])
        return ops.add_rms_norm_fp8(s["x"], s["res"], s["gain"], eps=EPS, pow2=s["pow2"])
    if op == "weights":
        return ops.fp8_quantize_weights(s["w"], pow2=s["pow2"])
    if op == "linear":
        if s["first"] == "norm":
            q, scale, h = ops.add_rms_norm_fp8(s["x"], s["res"], s["gain"], eps=EPS, pow2=s["pow2"])
        else:
            q, scale = ops.fp8_quantize(s["x"], pow2=s["pow2"])
        c = ops.dense_gemm_fp8(q, scale, s["w"], s["ws"], out_dtype=F32 if s["f32"] else BF16)
        return (c, h) if s["first"] == "norm" else c
    if op == "grouped":
        swiglu = s["kind"] == SWIGLU
        return ops.grouped_gemm_fp8(ops.W13_SWIGLU if swiglu else ops.W2, s["a"], s["as"], s["offsets"], s["w"], s["ws"],
                                    num_tokens=s["T"], top_k=s["k"], a_row_index=s["perm"] if swiglu else None)
    q, scale, h = ops.add_rms_norm_fp8(s["x"], s["res"], s["gain"], eps=EPS, pow2=s["pow2"])
    out = ops.moe_fp8_forward(q, scale, s["ids"], s["w"], s["w13"], s["s13"], s["w2"], s["s2"], num_experts=s["E"],
                              expert_begin=s["begin"], pow2=s["pow2"])
    return out, h


# ---- what a pass cannot do without -----------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "norm":
        T, K = case["T"], case["K"]
        return {"bytes": T * K * (7 if case["residual"] else 3) + T * K // 32 + 2 * K, "flops": 8 * T * K}
    if op == "weights":
        n = case["E"] * case["N"] * case["K"]
        return {"bytes": 3 * n + 4 * case["E"] * _blocks(case["N"]) * case["K"] // 128, "flops": 4 * n}
    T = case["T"]
    if op == "linear":
        K, N = case["K"], case["N"]
        first = 6 if case["first"] == "norm" else 2          # x, residual and its sum; or x alone
        return {"bytes": first * T * K + N * K + 4 * _blocks(N) * K // 128 + T * N * (4 if case["f32"] else 2),
                "flops": 2 * T * N * K}
    E, k, H, I = (case[n] for n in ("E", "k", "H", "I"))
    L = case.get("local", E)
    slots = T * k * L / E
    # experts that at least one slot reaches, for slots spread evenly (popular ones draw more, so fewer are reached)
    reached = L * (1 - (1 - k / E) ** T)
    if op == "grouped":
        rows, K, N, cols = (T, H, 2 * I, I) if case["kind"] == SWIGLU else (T * k, I, H, H)
        return {"bytes": rows * (K + K // 32) + reached * N * K + 2 * slots * cols + 4 * (T * k + E + 1),
                "flops": 2 * slots * N * K}
    return {"bytes": 8 * T * H + 8 * T * k + reached * 3 * H * I, "flops": 6 * slots * H * I}


# ---- the definition in 64 bits ------------------------------------------------------------------------

def _exact_norm(s):
    h = s["x"].double()
    if s["res"] is not None:
        h = h + s["res"].double()
    kept = h.float().to(BF16).double()
    return h, kept * s["gain"].double(), (kept.pow(2).mean(-1, keepdim=True) + EPS).pow(-0.5)


def _exact_e4m3(v):
    """The nearest e4m3 value, ties to the even one: three bits behind the leading one, steps of 2^-9 at least."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return ((v / step).round() * step).clamp(-TOP, TOP)


def _exact_blocks(y, rows, pow2, factor=None):
    """Values y [R, K], each row times its factor, in blocks of rows x 128: codes and scales. The quotient of a value
    and its block's largest as it is, without the factor and not through a rounded scale: ties have to be ties."""
    R, K = y.shape
    padded = torch.zeros(-(-R // rows) * rows, K, dtype=F64, device=DEV)
    padded[:R] = y
    b = padded.view(-1, rows, K // 128, 128)
    by = torch.ones(R, 1, dtype=F64, device=DEV) if factor is None else factor
    if pow2 and factor is not None:
        b, by = b * factor[:, :, None, None], torch.ones_like(by)
    top = b.abs().amax((1, 3))
    scale = top / TOP if factor is None else top * by / TOP
    if pow2:
        scale = torch.exp2(torch.ceil(torch.log2(scale)))
    dead = top * by.max() < NOTHING
    scale[dead] = 0.0
    over = scale if pow2 else top
    q = _exact_e4m3(b * (1.0 if pow2 else TOP) / over.masked_fill(dead, 1.0)[:, None, :, None])
    q = q.masked_fill(dead[:, None, :, None], 0.0)
    return q.view(-1, K)[:R], scale


def _exact_weights(w, ws):
    """[N, K] codes and their blocks' scales as values in 64 bits."""
    full = torch.kron(ws.double(), torch.ones(128, 128, dtype=F64, device=DEV))
    return w.double() * full[:w.shape[0]]


def _exact_rows(q, scale):
    return q.double() * torch.kron(scale.double(), torch.ones(1, 128, dtype=F64, device=DEV))


def _exact_experts(rows, ids, w, ws, kind):
    """ids[r]: the expert of row r, or one past the last for a row of none (its result is zero)."""
    out = torch.zeros(rows.shape[0], w.shape[1] // 2 if kind == SWIGLU else w.shape[1], dtype=F64, device=DEV)
    for e in range(w.shape[0]):
        at = (ids == e).nonzero().flatten()
        if at.numel():
            c = rows[at] @ _exact_weights(w[e], ws[e]).T
            if kind == SWIGLU:
                n = w.shape[1] // 2
                c = c[:, :n] * torch.sigmoid(c[:, :n]) * c[:, n:]
            out[at] = c
    return out


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "norm":
        h, u, r = _exact_norm(s)
        q, scale = _exact_blocks(u, 1, case["pow2"], r)
        return (q, scale, h) if case["residual"] else (q, scale)
    if op == "weights":
        if case["E"] * case["N"] * case["K"] > 1 << 29:
            return None
        each = [_exact_blocks(w.double(), 128, case["pow2"]) for w in s["w"]]
        return torch.stack([q for q, _ in each]), torch.stack([t for _, t in each])
    if op == "linear":
        h, u, r = _exact_norm(s) if case["first"] == "norm" else (None, s["x"].double(), None)
        rows = _exact_rows(*_exact_blocks(u, 1, case["pow2"], r))
        c = torch.cat([rows @ _exact_weights(s["w"][n:n + 2048], s["ws"][n // 128:n // 128 + 16]).T
                       for n in range(0, case["N"], 2048)], 1)
        return (c, h) if case["first"] == "norm" else c
    if op == "grouped":
        rows = _exact_rows(s["a"], s["as"])
        at = torch.arange(s["perm"].numel(), device=DEV)
        e = torch.bucketize(at, s["offsets"][1:].long(), right=True)
        if case["kind"] == SWIGLU:
            at = s["perm"].long().div(case["k"], rounding_mode="floor")
        return _exact_experts(rows[at], e, s["w"], s["ws"], case["kind"])
    h, u, r = _exact_norm(s)
    rows = _exact_rows(*_exact_blocks(u, 1, case["pow2"], r))
    e = s["ids"].flatten().long() - case["begin"]
    e[(e < 0) | (e >= case["local"])] = case["local"]
    token = torch.arange(e.numel(), device=DEV).div(case["k"], rounding_mode="floor")
    mid = _exact_experts(rows[token], e, s["w13"], s["s13"], SWIGLU).to(BF16).double()
    mid = _exact_rows(*_exact_blocks(mid, 1, case["pow2"]))
    out = _exact_experts(mid, e, s["w2"], s["s2"], DOWN).to(BF16).double()
    return (out.view(case["T"], case["k"], -1) * s["w"].double()[:, :, None]).sum(1), h

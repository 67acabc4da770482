"""Routing on scores against its definition: binary32 scores of the exact (64-bit) function, then loops.

Ids must be equal. A weight is a score (rounded once), a sum of at most 16 by four levels, a quotient and a product:
seven half steps, and one more for a score whose 64-bit value lies next to a rounding border: 8 * 2^-24 relative.
"""
import numpy as np
import pytest
import torch

from helpers import say

pytestmark = pytest.mark.gpu


def reference(l, b, k, score, G, kept, top, renorm, scale):
    T, E = l.shape
    ids, ws = np.zeros((T, k), np.int32), np.zeros((T, k))
    d = l.astype(np.float64)
    for t in range(T):
        with np.errstate(all="ignore"):
            if score == "sigmoid":
                s = 1 / (1 + np.exp(-d[t]))
            else:
                p = np.exp(d[t] - np.nanmax(d[t]))
                s = p / np.nansum(p)
            s = s.astype(np.float32)
            c = s + b if b is not None else s
        masked = np.isneginf(l[t]) | np.isnan(c)
        s = np.where(masked, np.float32(0), s)
        c = np.where(masked, np.float32(-np.inf), c)
        allowed = list(range(E))
        if G > 1:
            size = E // G
            g = []
            for i in range(G):
                best = np.sort(c[i * size:(i + 1) * size])[::-1]
                g.append(best[0] if top == 1 else np.float32(best[0] + best[1]))
            groups = sorted(range(G), key=lambda i: (-g[i], i))[:kept]
            allowed = [e for e in allowed if e // size in groups]
        chosen = sorted(allowed, key=lambda e: (-c[e], e))[:k]
        w = s[chosen].astype(np.float64)
        if renorm:
            w = w / w.sum() if w.sum() > 0 else w * 0
        ids[t], ws[t] = chosen, w * np.float64(np.float32(scale))
    return ids, ws


def run(l, b, k, **kw):
    from w4a16_grouped_gemm_amd import ops
    ids, w = ops.route_scored(torch.from_numpy(l).cuda(), k, bias=None if b is None else torch.from_numpy(b).cuda(), **kw)
    return ids.cpu().numpy(), w.cpu().numpy()


def check(l, b, k, score="sigmoid", G=1, kept=1, top=1, renorm=True, scale=1.0):
    ids, w = run(l, b, k, score=score, num_groups=G, topk_groups=kept, group_top=top, renormalize=renorm, scale=scale)
    rid, rw = reference(l, b, k, score, G, kept, top, renorm, scale)
    assert np.array_equal(ids, rid)
    assert (np.abs(w - rw) <= 8 * 2.0 ** -24 * np.abs(rw) + 2.0 ** -148).all()


CASES = [  # T, E, k, G, kept, top
    (1, 8, 2, 1, 1, 1), (1, 256, 8, 8, 4, 2), (5, 1, 1, 1, 1, 1), (3, 16, 16, 1, 1, 1), (17, 60, 4, 4, 2, 1),
    (33, 64, 6, 8, 3, 2), (7, 65, 5, 5, 2, 2), (64, 128, 8, 1, 1, 1), (9, 160, 6, 8, 3, 1), (21, 256, 8, 8, 4, 2),
    (4, 257, 7, 1, 1, 1), (6, 512, 12, 16, 5, 2), (3, 1000, 16, 8, 2, 1), (2, 1024, 16, 64, 4, 2), (5, 128, 8, 64, 4, 1),
    (4097, 128, 8, 4, 2, 2)]


@pytest.mark.parametrize("T,E,k,G,kept,top", CASES)
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route(T, E, k, G, kept, top, score):
    say(f"route_scored T={T} E={E} k={k} G={G} kept={kept} top={top} {score}")
    rng = np.random.default_rng(T * 1000 + E + k)
    l = (rng.standard_normal((T, E)) * 1.5).astype(np.float32)
    b = (rng.standard_normal(E) * (0.1 if score == "sigmoid" else 0.1 / E)).astype(np.float32)
    check(l, b, k, score, G, kept, top, True, 2.5)
    check(l, None, k, score, G, kept, top, False)


@pytest.mark.parametrize("G,kept,top", [(1, 1, 1), (4, 2, 1), (4, 2, 2)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_ties_masks_and_nan(G, kept, top, score):
    rng = np.random.default_rng(5)
    l = rng.integers(-2, 3, (12, 32)).astype(np.float32)      # many equal scores
    l[1] = 0.0                                                # all equal
    l[2] = -np.inf                                            # nothing left
    l[3] = -np.inf
    l[3, 29] = 1.0                                            # one expert left
    l[4, ::2] = -np.inf
    l[5, :16] = -np.inf                                       # whole groups switched off
    l[6, 3] = np.nan
    l[7] = 40.0                                               # sigmoid saturates: equal scores
    l[7, 9] = 41.0
    l[8] = -200.0                                             # scores below binary32
    l[8, 4] = 0.0
    check(l, None, 6, score, G, kept, top)
    b = np.zeros(32, np.float32)
    b[7] = -np.inf                                            # an expert that is never wanted
    b[20] = 3.0
    check(l, b, 6, score, G, kept, top, False, 0.5)


MANY = [  # E, k, G, kept, top
    (256, 8, 8, 4, 2), (256, 16, 1, 1, 1), (250, 7, 1, 1, 1), (129, 5, 1, 1, 1), (128, 8, 4, 2, 1), (120, 6, 3, 2, 2),
    (96, 16, 4, 2, 2), (64, 6, 8, 3, 2), (60, 4, 5, 3, 2), (33, 3, 1, 1, 1), (8, 8, 1, 1, 1), (1, 1, 1, 1, 1), (160, 6, 8, 3, 1)]


@pytest.mark.parametrize("E,k,G,kept,top", MANY)
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("offset", [0, 1])
def test_many_tokens(E, k, G, kept, top, score, offset):
    """Each of 23 rows (ordinary, tied, masked, NaN) many times over, at every place of a workgroup; odd addresses."""
    say(f"route_scored many E={E} k={k} G={G} kept={kept} top={top} {score} offset={offset}")
    from w4a16_grouped_gemm_amd import ops
    rng = np.random.default_rng(E * 7 + k)
    l = (rng.standard_normal((23, E)) * 1.5).astype(np.float32)
    l[1] = 0.0
    l[2] = -np.inf
    l[3] = rng.integers(-2, 3, E)
    l[4, ::2] = -np.inf
    l[5, E // 2:] = -np.inf
    l[6, E // 3] = np.nan
    l[7] = 40.0
    l[8] = -200.0
    l[8, E // 2] = 0.0
    l[9] = rng.integers(0, 2, E)
    b = (rng.standard_normal(E) * (0.1 if score == "sigmoid" else 0.1 / E)).astype(np.float32)
    T = 4096 + 23
    rows = torch.arange(T) * 5 % 23
    for bias in (b, None):
        x = torch.empty(T * E + offset, device="cuda")[offset:].view(T, E)
        x.copy_(torch.from_numpy(l)[rows])
        y = None
        if bias is not None:
            y = torch.empty(E + offset, device="cuda")[offset:]
            y.copy_(torch.from_numpy(bias))
        ids, w = ops.route_scored(x, k, bias=y, score=score, num_groups=G, topk_groups=kept, group_top=top, scale=2.5)
        rid, rw = reference(l, bias, k, score, G, kept, top, True, 2.5)
        assert np.array_equal(ids.cpu().numpy(), rid[rows])
        assert (np.abs(w.cpu().numpy() - rw[rows]) <= 8 * 2.0 ** -24 * np.abs(rw[rows]) + 2.0 ** -148).all()


def test_infinite_logit_and_no_tokens():
    from w4a16_grouped_gemm_amd import ops
    l = np.zeros((2, 16), np.float32)
    l[0, 3] = np.inf
    ids, w = run(l, None, 4, score="softmax")
    assert ((ids >= 0) & (ids < 16)).all() and np.isfinite(w).all()
    ids, w = run(l, None, 4)
    assert ids[0, 0] == 3 and np.isfinite(w).all()
    ids, w = ops.route_scored(torch.empty(0, 16, device="cuda"), 4)
    assert ids.shape == (0, 4) and w.shape == (0, 4)


def test_softmax_without_bias_chooses_as_route():
    from w4a16_grouped_gemm_amd import ops
    g = torch.Generator().manual_seed(3)
    l = torch.randn(500, 128, generator=g).cuda()
    i0, w0 = ops.route(l, 8)
    i1, w1 = ops.route_scored(l, 8, score="softmax")
    assert torch.equal(i0, i1)
    torch.testing.assert_close(w0, w1, rtol=2e-6, atol=0)


def test_refusals():
    from w4a16_grouped_gemm_amd import ops
    l = torch.zeros(4, 32, device="cuda")
    for kw in [dict(num_groups=5), dict(num_groups=4, topk_groups=5), dict(group_top=3), dict(bias=l[0, :8]),
               dict(bias=l[0].double()), dict(score="max"), dict(num_groups=16, topk_groups=1)]:
        with pytest.raises(ValueError):
            ops.route_scored(l, 4, **kw)
    with pytest.raises(ValueError):
        ops.route_scored(l, 17)
    with pytest.raises(ValueError):
        ops.route_scored(l.t(), 2)


@pytest.mark.parametrize("k", [0, -1])
def test_refuses_no_slots(k):
    from w4a16_grouped_gemm_amd import ops
    with pytest.raises(ValueError):
        ops.route_scored(torch.zeros(4, 32, device="cuda"), k)


@pytest.mark.parametrize("E,k,G,kept,top", [(16, 16, 1, 1, 1), (32, 12, 4, 2, 1), (32, 12, 4, 2, 2), (128, 16, 1, 1, 1),
                                            (256, 16, 8, 2, 2), (160, 16, 8, 2, 1), (512, 16, 1, 1, 1), (1000, 16, 8, 2, 2)])
@pytest.mark.parametrize("T", [5, 4100])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_a_bias_of_minus_infinity_comes_before_what_is_switched_off(E, k, G, kept, top, T, score):
    """Experts that are left: first by c, then those whose bias alone is -inf, then the masked ones (logit -inf, or c
    NaN); lower index first in each. In its group's score a masked expert counts as -inf."""
    from w4a16_grouped_gemm_amd import ops
    say(f"route_scored -inf bias E={E} k={k} G={G} kept={kept} top={top} T={T} {score}")
    rng = np.random.default_rng(E + k)
    l = (rng.standard_normal((7, E)) * 1.5).astype(np.float32)
    l[:, rng.permutation(E)[:E // 3]] = -np.inf
    l[3, ::2] = np.nan
    l[4] = -np.inf
    b = np.full(E, -np.inf, np.float32)
    b[rng.permutation(E)[:max(2, k // 4)]] = 0.25
    b[1] = np.nan
    rows = np.arange(T) % 7
    ids, w = run(np.ascontiguousarray(l[rows]), b, k, score=score, num_groups=G, topk_groups=kept, group_top=top,
                 renormalize=False, scale=1.5)
    d = l.astype(np.float64)
    for t in range(7):
        with np.errstate(all="ignore"):
            p = 1 / (1 + np.exp(-d[t])) if score == "sigmoid" else np.exp(d[t] - np.nanmax(d[t]))
            s = (p if score == "sigmoid" else p / np.nansum(p)).astype(np.float32)
            c = s + b
        off = np.isneginf(l[t]) | np.isnan(c)
        c[off] = -np.inf
        allowed = range(E)
        if G > 1:
            best = -np.sort(-c.reshape(G, -1), axis=1)
            g = best[:, 0] if top == 1 else best[:, 0] + best[:, 1]
            groups = sorted(range(G), key=lambda i: (-g[i], i))[:kept]
            allowed = [e for e in range(E) if e // (E // G) in groups]
        want = sorted(allowed, key=lambda e: (off[e], -c[e], e))[:k]
        share = np.where(off, 0, s.astype(np.float64) * 1.5)[want]
        for i in np.flatnonzero(rows == t):
            assert np.array_equal(ids[i], want), t
            assert (np.abs(w[i] - share) <= 4 * 2.0 ** -24 * share + 2.0 ** -148).all()


@pytest.mark.parametrize("T,E,k,G,kept,top", [(9, 200, 8, 1, 1, 1), (7, 256, 16, 1, 1, 1), (4, 1000, 16, 1, 1, 1),
                                              (5, 360, 6, 8, 3, 2), (3, 512, 9, 2, 1, 1)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_of_more_sizes(T, E, k, G, kept, top, score):
    """The forms of the kernel that no size above reaches: many experts without groups, or in groups of any size."""
    test_route(T, E, k, G, kept, top, score)

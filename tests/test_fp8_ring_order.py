"""The order of the FP8 ring kernel's memory instructions and its counted waits, in the built code (CPU only).

A wave waits for a group's copies by the number of copies and loads that went out behind them, so each wait is right only
while the compiler emits exactly those, in the source's order. Read from the library's own code, for every instance: before
the loop the weights' copies of group 0, the scales of a quad (of two quads with two groups under way), the tokens' copies of
group 0, with four groups under way the next quad's scales, the other groups' copies; in the loop a wait, C copies and, behind
the first group of a quad, one set of scales' loads, each wait with its own count; and no other copy to LDS. An instance
whose experts may have several chunks of rows has two loops, one of them without non-temporal copies.
"""
import re

import pytest

from test_fp8_waits import KINDS, RINGS, checked, code_objects, pytestmark   # noqa: F401


def events(ins):
    """Copies to LDS ("N": non-temporal), 16-byte loads to registers and counted waits, in the code's order."""
    out = []
    for op, rest in ins:
        if op == "buffer_load_dwordx4":
            out.append(("N" if re.search(r"\bnt\b", rest) else "C") if " lds" in rest else "S")
        elif op == "s_waitcnt" and "vmcnt" in rest:
            out.append(int(re.search(r"vmcnt\((\d+)\)", rest).group(1)))
    return out


def starts(seq, part):
    return [i for i in range(len(seq) - len(part) + 1) if seq[i:i + len(part)] == part]


def instances():
    for nsub, tpw, wk, depth in RINGS:
        for kind, f32 in KINDS:
            if (kind == 0 and tpw == 1) or (f32 and nsub == 5):
                continue
            for once in (0, 1):
                if once if nsub > 1 or (kind == 0 and wk > 1) else wk == 1 and not once:
                    continue
                yield kind, f32, nsub, tpw, wk, depth, once


@pytest.fixture(scope="module")
def cos(tmp_path_factory):
    return code_objects(tmp_path_factory.mktemp("ring"))


@pytest.mark.parametrize("kind,f32,nsub,tpw,wk,depth,once", list(instances()))
def test_order(cos, kind, f32, nsub, tpw, wk, depth, once):
    sym = (f"_ZN3moe12_GLOBAL__N_115fp8_ring_kernelILi{kind}ELb{f32}ELi{nsub}ELi{tpw}ELi{wk}ELi{depth}ELb{once}EEEv"
           "NS0_7Fp8ArgsEi")
    ins, copies = checked(cos, sym)
    seq = events(ins)
    scales, weights, tokens = ["S"] * (nsub + (2 if kind == 0 else 1)), 2 * tpw, ["C"] * (2 * nsub)
    group = weights + len(tokens)

    def wait(j):
        return (depth - 1) * group + (len(scales) if depth == 4 or j in (1, 2) else 0)

    def loop(w):
        out = []
        for j in range(4):
            out += [wait(j)] + [w] * weights + tokens + (scales if j == 0 else [])
        return out

    w = "N" if once else "C"
    loops = [w] + (["C"] if once and wk == 1 else [])
    assert copies == group * (depth + 4 * len(loops)), sym        # all of them are in what follows
    for v in loops:
        assert len(starts(seq, loop(v))) == 1, (sym, v)
    before = [e for e in seq[:min(starts(seq, loop(v))[0] for v in loops)] if not isinstance(e, int)]
    assert before == ([w] * weights + scales * (2 if depth == 2 else 1) + tokens + scales * (depth == 4)
                      + ([w] * weights + tokens) * (depth - 1)), sym

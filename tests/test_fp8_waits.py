"""Guard of the FP8 tile and ring kernels' counted memory waits (CPU only).

Both copy to LDS with the buffer unit and wait for the copies by count: the tile kernel's copying waves have L = TM / 2
copies of tokens and LW = 2 TN of weights to a stage, of which those of one stage's weights may still be on their way at a
meeting (a stage and the weights of another at the first); a wave of the ring kernel has C = 2 (TPW + NSUB) copies to a
group and NSUB + 1 (two where it computes gate and up) loads of scales to four groups. Further loads in between would only
make a wait stricter, but a spill inside the loop would stall it, and a copy that the compiler split or gave an
instruction offset (which moves the LDS side too) would break it. Read from the built library's own code:
  * no scratch instruction;
  * every copy to LDS is one 16-byte instruction without an instruction offset;
  * the waits are there, in the tile kernel right before a barrier (but for the last stages', for everything).
"""
import os
import re
import shutil

import pytest

from test_tile_kernel_waits import BUNDLER, LIB, OBJDUMP, code_objects, disassemble, instructions

pytestmark = pytest.mark.skipif(not (os.path.exists(LIB) and os.path.exists(BUNDLER) and os.path.exists(OBJDUMP)
                                     and shutil.which("objcopy")), reason="needs the built library and the ROCm LLVM tools")

KINDS = [(0, 0), (1, 0), (1, 1)]               # SwiGLU, bf16 and fp32 results


def checked(cos, sym):
    """The kernel's instructions, the number of its copies to LDS."""
    ins = instructions(disassemble(cos, sym))
    assert len(ins) > 300
    copies = 0
    for op, rest in ins:
        assert not op.startswith("scratch_"), f"spill: {op}{rest}"
        if " lds" in rest and op.startswith("buffer_"):
            assert op == "buffer_load_dwordx4" and "offset:" not in rest, f"{op}{rest}"
            copies += 1
    return ins, copies


def waits(ins, before):
    """The counts waited for by s_waitcnt; only those right before an instruction `before`, where given."""
    found = set()
    for i, (op, rest) in enumerate(ins):
        if op == "s_waitcnt" and "vmcnt" in rest:
            nxt = next((o for o, _ in ins[i + 1:] if o != "s_nop"), "")
            if before is None or nxt == before:
                found.add(int(re.search(r"vmcnt\((\d+)\)", rest).group(1)))
    return found


@pytest.mark.parametrize("tn,tm", [(4, 8), (4, 4), (2, 4)])
def test_tile_kernel(tn, tm, tmp_path):
    cos = code_objects(tmp_path)
    lx, lw = tm // 2, 2 * tn
    for kind, f32 in KINDS:
        if f32 and tm == 8:
            continue
        sym = f"_ZN3moe12_GLOBAL__N_115fp8_tile_kernelILi{kind}ELb{f32}ELi{tn}ELi{tm}EEEvNS0_7Fp8ArgsEi"
        ins, copies = checked(cos, sym)
        assert copies >= 2 * (lx + lw)
        assert {lx + 2 * lw, lw} <= waits(ins, "s_barrier") and 0 in waits(ins, None), sym


RINGS = [(4, 4, 2, 2), (3, 4, 2, 2), (5, 4, 4, 2), (4, 4, 4, 2), (3, 4, 4, 2), (2, 4, 2, 2), (2, 4, 4, 2), (2, 2, 4, 2),
         (1, 4, 2, 2), (1, 2, 2, 2), (1, 2, 4, 2), (1, 1, 4, 4), (1, 2, 1, 2)]


@pytest.mark.parametrize("nsub,tpw,wk,depth", RINGS)
def test_ring_kernel(nsub, tpw, wk, depth, tmp_path):
    cos = code_objects(tmp_path)
    copy = 2 * (tpw + nsub)
    for kind, f32 in KINDS:
        if (kind == 0 and tpw == 1) or (f32 and nsub == 5):
            continue
        scales = nsub + (2 if kind == 0 else 1)
        for once in (0, 1):
            if once if nsub > 1 or (kind == 0 and wk > 1) else wk == 1 and not once:
                continue
            sym = (f"_ZN3moe12_GLOBAL__N_115fp8_ring_kernelILi{kind}ELb{f32}ELi{nsub}ELi{tpw}ELi{wk}ELi{depth}ELb{once}EEEv"
                   "NS0_7Fp8ArgsEi")
            ins, copies = checked(cos, sym)
            assert copies >= depth * copy
            ahead = (depth - 1) * copy
            assert ({ahead + scales} if depth == 4 else {ahead, ahead + scales}) <= waits(ins, None), sym

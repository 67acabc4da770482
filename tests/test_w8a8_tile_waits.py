"""Guard of the W8A8 tile kernel's counted memory waits (CPU only).

w8_tile_kernel copies its stages to LDS with the buffer unit and waits for them by count: a stage has L copies per
wave, and at a step's meeting those of NS - 3 stages may still be on their way. Further loads in between would only
make a wait stricter, but a spill inside the loop would stall it, and a copy that the compiler split or gave an
instruction offset (which moves the LDS side too) would break it. Read from the built library's own code:
  * no scratch instruction and no vector-memory instruction besides 16-byte copies, loads and 16-byte stores;
  * every copy to LDS is one 16-byte instruction without an instruction offset;
  * the loop's wait, (NS - 3) L, and the first one, (NS - 2) copies of tokens, precede a barrier.
"""
import os
import re
import shutil

import pytest

from test_tile_kernel_waits import BUNDLER, LIB, OBJDUMP, code_objects, disassemble, instructions

# (TN, TM, waves along the weights, waves along the tokens, stages) of the instantiated tiles
TILES = [(4, 4, 2, 2, 5), (4, 2, 2, 2, 3), (2, 2, 2, 2, 5), (2, 2, 4, 1, 4), (2, 1, 2, 2, 5)]
KINDS = [(0, 0), (1, 0), (1, 1)]               # SwiGLU, bf16 and fp32 results


@pytest.mark.skipif(not (os.path.exists(LIB) and os.path.exists(BUNDLER) and os.path.exists(OBJDUMP)
                         and shutil.which("objcopy")), reason="needs the built library and the ROCm LLVM tools")
@pytest.mark.parametrize("tn,tm,nwn,nwm,ns", TILES)
def test_waits_and_copies(tn, tm, nwn, nwm, ns, tmp_path):
    cos = code_objects(tmp_path)
    lm, per_stage = tm * nwm // 2, (tn * nwn + tm * nwm) // 2          # copies of a wave: 16 rows each, four waves
    for kind, f32 in KINDS:
        sym = (f"_ZN3moe12_GLOBAL__N_114w8_tile_kernelILi{kind}ELb{f32}ELi{tn}ELi{tm}ELi{nwn}ELi{nwm}ELi{ns}EEEvNS0_"
               "6W8ArgsEi")
        ins = instructions(disassemble(cos, sym))
        assert len(ins) > 300
        copies = 0
        for op, rest in ins:
            assert not op.startswith("scratch_"), f"spill: {op}{rest}"
            if " lds" in rest and op.startswith("buffer_"):
                assert op == "buffer_load_dwordx4" and "offset:" not in rest, f"{op}{rest}"
                copies += 1
            elif re.match(r"(buffer|global|flat)_store", op):
                assert op == "global_store_dwordx4", f"{op}{rest}"
        assert copies >= (ns - 1) * per_stage
        waits = set()
        for i, (op, rest) in enumerate(ins):
            if op == "s_waitcnt" and "vmcnt" in rest:
                nxt = next((o for o, _ in ins[i + 1:] if o != "s_nop"), "")
                if nxt == "s_barrier":
                    waits.add(int(re.search(r"vmcnt\((\d+)\)", rest).group(1)))
        assert {(ns - 2) * lm, (ns - 3) * per_stage} <= waits, (sorted(waits), sym)

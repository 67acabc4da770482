"""Where the waves of the W8A8 streaming kernel meet (CPU only).

With the rows quantized by the product (QV > 0) a workgroup's waves meet twice: when the rows are in LDS, and when the
partial sums are. How many groups of K a wave has differs between the waves (three groups for two waves: one and two),
so no meeting may stand in the branches that go by it: every wave has to come to the same one. Read from the built
library's own code: the two meetings are there once each.
"""
import os
import shutil

import pytest

from test_tile_kernel_waits import BUNDLER, LIB, OBJDUMP, code_objects, disassemble, instructions


@pytest.mark.skipif(not (os.path.exists(LIB) and os.path.exists(BUNDLER) and os.path.exists(OBJDUMP)
                         and shutil.which("objcopy")), reason="needs the built library and the ROCm LLVM tools")
@pytest.mark.parametrize("qv", [2, 4])
def test_each_meeting_is_there_once(qv, tmp_path):
    sym = f"_ZN3moe12_GLOBAL__N_116w8_stream_kernelILi1ELb0ELi1ELi2ELi2ELi2ELi{qv}EEEvNS0_6W8ArgsEi"
    ins = instructions(disassemble(code_objects(tmp_path), sym))
    assert len(ins) > 300
    assert sum(op == "s_barrier" for op, _ in ins) == 2

"""Direct loads to LDS in the kernels' sources: a load needs a wait state behind the write of M0, and M0 is reserved, so
that a clobber list that names it says nothing the compiler honours."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "post_bit_weight_awq_amd", "csrc")
ASM = re.compile(r"asm volatile\((.*?)\);", re.S)


def loads():
    for path in sorted(glob.glob(os.path.join(CSRC, "*"))):
        with open(path) as f:
            for m in ASM.finditer(f.read()):
                if "global_load_lds" in m.group(1):
                    yield os.path.basename(path), " ".join(m.group(1).split())


@pytest.mark.parametrize("source,asm", loads())
def test_m0_is_an_operand_and_waited_for(source, asm):
    text, rest = asm.split(" : ", 1)
    assert re.match(r'"s_nop 0\\n\\tglobal_load_lds_dword(x4)? ', text), "no wait state between M0's write and the load"
    assert "s_mov_b32 m0" not in text and '"{m0}"' in rest, "M0 is not an operand"
    assert '"memory"' in rest and '"m0"' not in rest

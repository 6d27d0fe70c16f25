"""What the kernels' inline assembly writes without naming it as an output: the address
register of loads to LDS has to be in the clobbers, or the compiler may keep a value of its
own there."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_activation_compression_amd", "csrc")


def test_assembly_that_writes_m0_names_it():
    seen = 0
    for path in sorted(glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.hip"))):
        for stmt in re.findall(r"\basm\b[^;]*;", open(path).read()):
            if re.search(r"\bs_mov_b32 m0\b", stmt):
                seen += 1
                assert '"m0"' in stmt.rsplit(":", 1)[1], f"{os.path.basename(path)}: {stmt}"
    assert seen >= 2

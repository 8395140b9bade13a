"""Inline assembly that writes m0 says so (the compiler may hold an m0 of its
own across a statement that does not)."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_scaled_fp4_permute_amd", "csrc")


def test_assembly_that_writes_m0_names_it():
    found = 0
    for path in sorted(glob.glob(os.path.join(CSRC, "*"))):
        for stmt in re.findall(r"\basm\b[^;]*;", open(path).read()):
            if re.search(r"s_mov_b32 m0\b", stmt):
                found += 1
                assert stmt.split(":")[-1].count('"m0"') == 1, f"{os.path.basename(path)}: {stmt}"
    assert found >= 2

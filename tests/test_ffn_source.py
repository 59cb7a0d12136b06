"""What the products' inline assembly tells the compiler, read from the source (CPU)."""
from __future__ import annotations

import glob
import os
import re

from hyper_connection_rank_amd import build


def _asm_statements():
    for path in sorted(glob.glob(os.path.join(build.CSRC, "*.h*"))):
        text = open(path).read()
        for m in re.finditer(r"\basm\s+volatile\s*\((.*?)\);", text, re.S):
            yield os.path.basename(path), text.count("\n", 0, m.start()) + 1, m.group(1)


def test_assembly_that_writes_m0_says_so():
    found = 0
    for name, line, text in _asm_statements():
        if re.search(r"s_mov_b32 m0\b", text):
            found += 1
            assert '"m0"' in text.rsplit(":", 1)[-1], f"{name}:{line} writes m0 without naming it as clobbered"
    assert found >= 4

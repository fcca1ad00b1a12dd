"""Loads straight into LDS take their LDS base from m0, and the hardware wants
a wait state between a scalar write of m0 and such a load.  The compiler adds
it to its own code but does not look into inline asm, so every such block has
it written out.  CPU only: reads the sources."""
import glob
import os
import re

import orthogonal_reparameterized_02_amd as pkg

CSRC = os.path.join(os.path.dirname(pkg.__file__), "csrc")


def blocks():
    for path in sorted(glob.glob(os.path.join(CSRC, "*.h*"))):
        text = open(path).read().replace("\\\n", "\n")
        for m in re.finditer(r'asm\s+volatile\s*\(((?:\s*"[^"]*")+)', text):
            yield os.path.basename(path), "".join(re.findall(r'"([^"]*)"', m[1])).replace("\\t", "").split("\\n")


def test_every_lds_load_waits_for_its_base():
    loads = 0
    for name, lines in blocks():
        for i, line in enumerate(lines):
            if line.startswith("buffer_load") and re.search(r"\blds\b", line):
                loads += 1
                assert i >= 2 and lines[i - 1].startswith("s_nop") and lines[i - 2].startswith("s_mov_b32 m0"), (name, lines)
            else:
                assert not re.search(r"\blds\b", line), (name, lines)
    assert loads >= 9

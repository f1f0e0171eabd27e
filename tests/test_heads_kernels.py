"""The built library holds kernels of query and key heads that some call reaches,
and no others (CPU: the names in its own symbol table)."""
from __future__ import annotations

import os
import re

import pytest

from newton_schulz_05_amd.binding import LIB_PATH

NAME = re.compile(rb"heads_(fwd|bwd)_kernelI([tf])Li(\d+)ELb([01])ELi(\d)E")


@pytest.mark.skipif(not os.path.exists(LIB_PATH), reason="not built")
def test_kernels_of_heads():
    with open(LIB_PATH, "rb") as f:
        kernels = set(NAME.findall(f.read()))
    # interleaved pairs fill their lanes, whole pieces of 8 bf16 do: at most 32 lanes for a head of 512
    want = set()
    for way in (b"fwd", b"bwd"):
        for t in (b"t", b"f"):
            for lanes in (4, 8, 16, 32, 64):
                for inter, kinds in ((0, (0, 2, 3)), (1, (0, 1, 2, 3))):
                    for kind in kinds:
                        if lanes == 64 and (inter or (t == b"t" and kind == 0)):
                            continue
                        want.add((way, t, b"%d" % lanes, b"%d" % inter, b"%d" % kind))
    assert kernels == want

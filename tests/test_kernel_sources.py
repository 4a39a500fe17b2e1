"""Rules that the kernel sources keep (no GPU)."""

from __future__ import annotations

import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "dense_gemm_epilogue_gb300", "csrc")


def code():
    """(file, line number, line without comments) of every kernel source."""
    for name in sorted(os.listdir(CSRC)):
        if name.endswith((".cu", ".cuh", ".h")):
            with open(os.path.join(CSRC, name)) as f:
                text = re.sub(r"/\*.*?\*/", lambda m: "\n" * m.group().count("\n"), f.read(), flags=re.S)
            for i, line in enumerate(text.split("\n"), 1):
                yield name, i, line.split("//")[0]


def test_no_non_coherent_loads():
    """Every kernel may start while the one before it still writes its inputs;
    a non-coherent load may be moved above the wait for that kernel."""
    bad = [(f, i, s) for f, i, s in code() if re.search(r"__ldg\b|ld\.global\.nc|__restrict__", s)]
    assert not bad, bad

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


def test_attention_rescales_o_behind_the_block_before():
    """With one tile a CTA the scores of a block are there before P V of the block
    before is issued.  Every rescaling of O waits for that product (PVD) first: the
    barrier of this block's own (PVA0) may be a phase behind, whose parity is the
    same."""
    with open(os.path.join(CSRC, "tg_kernel_attn.cuh")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    raises = [m.start() for m in re.finditer(r"\n\s*raise\(", text)]
    assert len(raises) == 2
    for at in raises:
        block = text[text.rindex("__any_sync", 0, at): at]
        assert re.search(r"NQ == 1 && !wait_warp\(bar\(C::PVD\), \(g \+ n - 1\) & 1", block), block
        if "PVA0" in block:
            assert block.index("C::PVD") < block.index("C::PVA0")

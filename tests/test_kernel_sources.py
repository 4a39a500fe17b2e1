"""Rules that the kernel sources keep (no GPU)."""

from __future__ import annotations

import os
import re
import shutil
import subprocess
import sys

import pytest

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


TAIL = r"""
#include <cstdio>
#include "tg_attn.h"
int main() {
    long long lq, i0, tiles, tokens, group;
    while (std::scanf("%lld %lld %lld %lld %lld", &lq, &i0, &tiles, &tokens, &group) == 5)
        std::printf("%d\n", tg::attn_tail_rows((int)lq, (int)i0, (int)tiles, (int)tokens, (int)group));
}
"""


def test_rows_of_a_parts_last_tile(tmp_path):
    """The kernel's own arithmetic on the host.  A part's last tile is full unless it is
    the sequence's last one, however much of the sequence is left behind it (2^31 rows,
    times 128 heads of a group)."""
    import dense_gemm_epilogue_gb300 as tg

    tg.build()
    build = sys.modules["dense_gemm_epilogue_gb300.build"]
    if shutil.which("g++") is None:
        pytest.skip("no C++ compiler")
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(build.nvcc()))), "include")
    src, exe = tmp_path / "tail.cpp", str(tmp_path / "tail")
    src.write_text(TAIL)
    subprocess.run(["g++", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover", "-I", CSRC, "-I", include,
                    str(src), "-o", exe], check=True)
    most = 2 ** 31 - 1 - 512
    cases = []
    for group in (1, 3, 7, 8, 100, 128):
        tokens = 128 // group
        for lq in (1, tokens, tokens + 1, 1000, 2 ** 24, 2 ** 24 + 1, 2 ** 30, most - 3, most):
            for i0 in (0, 1, lq // 2, lq - 1):
                every = -(-(lq - i0) // tokens)
                for tiles in (1, 2, every // 16, every // 2, every - 1, every):
                    if 1 <= tiles <= every:
                        cases.append((lq, i0, tiles, tokens, group))
    out = subprocess.run([exe], input="\n".join(" ".join(map(str, c)) for c in cases), text=True, check=True,
                         capture_output=True).stdout
    got = [int(v) for v in out.split()]
    want = [min(lq - i0 - (tiles - 1) * tokens, tokens) * group for lq, i0, tiles, tokens, group in cases]
    assert got == want
    # what a product of all that is left would wrap to
    assert any((lq - i0 - (tiles - 1) * tokens) * group >= 2 ** 31 for lq, i0, tiles, tokens, group in cases)


def test_dependents_start_behind_tensor_memory():
    """A kernel lets the next one start only behind the barrier that its allocation of
    tensor memory is before: one that allocated first would wait for this kernel to end,
    and this one for its columns."""
    for name in sorted(os.listdir(CSRC)):
        if not name.startswith("tg_kernel"):
            continue
        with open(os.path.join(CSRC, name)) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        at = [m.start() for m in re.finditer(r"\btmem_alloc(_pair)?\(", text)]
        for start, end in zip(at, at[1:] + [len(text)]):
            launch = text.find("griddep_launch()", start, end)
            if launch >= 0:
                assert re.search(r"__syncthreads\(\)|cluster_sync_all\(\)", text[start:launch]), (name, start)


def test_attention_helpers_are_reached():
    """Every device function of the attention sources is called by another."""
    every = " ".join(line for _, _, line in code())
    for name in ("tg_attn_ptx.cuh", "tg_attn_work.cuh", "tg_kernel_attn.cuh", "tg_kernel_attn_bwd.cuh"):
        text = "\n".join(line for f, _, line in code() if f == name)
        for f in re.findall(r"__forceinline__ \w+ (\w+)\(", text):
            assert len(re.findall(rf"\b{f}\b", every)) > 1, (name, f)

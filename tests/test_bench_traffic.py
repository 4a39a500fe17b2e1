"""The benchmark's DRAM traffic figure belongs to the dense GEMM's kernels: it is
dropped when their sources change and kept when another operator's do.  No GPU."""

from __future__ import annotations

import importlib
import json
import os
import re
import shutil

import pytest

import bench


@pytest.fixture
def b(monkeypatch, tmp_path):
    """build.py over a copy of the sources."""
    mod = importlib.import_module("dense_gemm_epilogue_gb300.build")
    copy = tmp_path / "csrc"
    shutil.copytree(mod.CSRC, copy)
    monkeypatch.setattr(mod, "CSRC", str(copy))
    return mod


def change(b, name):
    with open(os.path.join(b.CSRC, name), "a") as f:
        f.write("\n// changed\n")


@pytest.mark.parametrize("name", ["tg_mlp.cu", "tg_norm.cu", "tg_kernel_mlp.cuh", "tg_rows.cuh"])
def test_other_operators_do_not_touch_it(b, name):
    gemm, library = b.gemm_source_hash(), b.source_hash()
    change(b, name)
    assert b.gemm_source_hash() == gemm and b.source_hash() != library


@pytest.mark.parametrize("name", ["tg_kernel_pair.cuh", "tg_gemm.cu", "tg_ptx.cuh", "tg_inst_bf16.cu"])
def test_its_own_sources_do(b, name):
    gemm = b.gemm_source_hash()
    change(b, name)
    assert b.gemm_source_hash() != gemm


def test_every_file_that_the_pair_kernel_includes_counts(b):
    seen, todo = set(), ["tg_inst_bf16.cu", "tg_gemm.cu"]
    while todo:
        n = todo.pop()
        if n in seen or not os.path.exists(os.path.join(b.CSRC, n)):
            continue
        seen.add(n)
        with open(os.path.join(b.CSRC, n)) as f:
            todo += [os.path.basename(i) for i in re.findall(r'#include "([^"]+)"', f.read())]
    # tg_host.h only declares what tg_gemm.cu offers the other operators.
    assert seen - {"tg_host.h"} <= set(b.GEMM_SOURCES), seen


def test_the_benchmark_asks_by_that_hash(monkeypatch, tmp_path):
    (tmp_path / "profiles").mkdir()
    (tmp_path / "profiles" / "traffic.json").write_text(json.dumps(
        {bench.WORKLOAD: {"source_hash": "abc", "dram_bytes_per_launch": 7}}))
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    assert bench.load_traffic("abc") == 7 and bench.load_traffic("abd") is None
    with open(os.path.abspath(bench.__file__)) as f:
        assert "load_traffic(tg.gemm_source_hash())" in f.read()

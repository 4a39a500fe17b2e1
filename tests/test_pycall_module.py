"""The marshalling module (csrc/tg_pycall.c) is an optional speed-up: whatever
is wrong with it, the library builds, loads and answers through ctypes.  No
GPU."""

from __future__ import annotations

import warnings

import pytest


@pytest.fixture(scope="module")
def tg():
    import dense_gemm_epilogue_gb300 as tg

    tg.build()
    tg.load()
    return tg


@pytest.fixture
def unloaded(tg, monkeypatch):
    """The package as before its first load()."""
    monkeypatch.setattr(tg, "_lib", None)
    monkeypatch.setattr(tg, "_call", None)
    return tg


def answers(tg):
    assert tg.tg_version() == 100
    assert tg.tg_linear_workspace_bytes(64, 96, 128, 1 << 20, 128, 1 << 20, 128, "bf16") == 0
    assert tg.tg_layer_norm(0, 100, None, 100, None, None, 1e-5, None, 100, None, None, "f32") == tg.TG_OK


def test_a_module_that_does_not_load_is_left_out(unloaded, monkeypatch, tmp_path):
    bad = tmp_path / "_tgcall.so"
    bad.write_bytes(b"not a shared object")
    monkeypatch.setattr(unloaded, "_PYCALL_PATH", str(bad))
    with pytest.warns(RuntimeWarning, match="ctypes"):
        unloaded.load()
    assert unloaded._call is None
    answers(unloaded)


def test_a_module_of_other_entry_points_is_left_out(unloaded, monkeypatch):
    if not unloaded.os.path.exists(unloaded._PYCALL_PATH):
        pytest.skip("built without Python's headers")
    monkeypatch.setattr(unloaded, "_CALLS", ("tg_linear",))
    with pytest.warns(RuntimeWarning, match="ctypes"):
        unloaded.load()
    assert unloaded._call is None
    answers(unloaded)


def test_a_missing_module_is_no_error(unloaded, monkeypatch, tmp_path):
    monkeypatch.setattr(unloaded, "_PYCALL_PATH", str(tmp_path / "none.so"))
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        unloaded.load()
    assert unloaded._call is None
    answers(unloaded)


@pytest.fixture
def builder(tg, monkeypatch, tmp_path):
    """build.py with the module's file in an empty folder and the library done."""
    import importlib

    b = importlib.import_module("dense_gemm_epilogue_gb300.build")
    if not b.os.path.exists(b.os.path.join(b.sysconfig.get_paths()["include"], "Python.h")):
        pytest.skip("no Python headers")
    monkeypatch.setattr(b, "PYCALL", str(tmp_path / b.os.path.basename(b.PYCALL)))
    return b


def test_the_module_is_named_for_its_interpreter(builder):
    """Another Python's build neither loads this one's module nor takes it for
    its own."""
    suffix = builder.sysconfig.get_config_var("EXT_SUFFIX")
    assert len(suffix) > len(".so") and builder.PYCALL.endswith(suffix)


def test_a_missing_module_is_built_beside_a_finished_library(builder):
    """As after a first build without a compiler or Python's headers."""
    assert not builder.os.path.exists(builder.PYCALL)
    builder.build()
    assert builder.os.path.exists(builder.PYCALL)
    first = builder.os.stat(builder.PYCALL).st_mtime_ns
    builder.build()
    assert builder.os.stat(builder.PYCALL).st_mtime_ns == first


def test_a_changed_source_rebuilds_the_module_alone(builder, monkeypatch, tmp_path):
    builder.build()
    first = builder.os.stat(builder.PYCALL).st_mtime_ns
    library = builder.os.stat(builder.LIB).st_mtime_ns
    changed = tmp_path / "tg_pycall.c"
    changed.write_text(open(builder.PYCALL_SOURCE).read() + "/* changed */\n")
    monkeypatch.setattr(builder, "PYCALL_SOURCE", str(changed))
    builder.build()
    assert builder.os.stat(builder.PYCALL).st_mtime_ns != first
    assert builder.os.stat(builder.LIB).st_mtime_ns == library


def test_a_source_that_does_not_compile_leaves_the_library(builder, monkeypatch, tmp_path):
    bad = tmp_path / "tg_pycall.c"
    bad.write_text("#error not with these headers\n")
    monkeypatch.setattr(builder, "PYCALL_SOURCE", str(bad))
    with pytest.warns(RuntimeWarning, match="ctypes"):
        assert builder.build() == builder.LIB
    assert not builder.os.path.exists(builder.PYCALL)
    assert builder.os.path.exists(builder.LIB)


@pytest.mark.parametrize("through", ["module", "ctypes"])
def test_names_come_from_the_package_tables(tg, monkeypatch, through):
    """A name that the package's tables learn is known on either path."""
    if through == "ctypes":
        monkeypatch.setattr(tg, "_call", None)
    elif tg._call is None:
        pytest.skip("built without Python's headers")
    monkeypatch.setitem(tg.DTYPE_CODES, "brain", tg.TG_BF16)
    monkeypatch.setitem(tg.ACT_CODES, "swish", tg.TG_ACT_SILU)
    monkeypatch.setitem(tg.OUT_CODES, "single", tg.TG_OUT_F32)
    a = 1 << 20
    assert tg.tg_linear_workspace_bytes(64, 96, 128, a, 128, a, 128, "brain") == 0
    assert tg.tg_gated(0, 96, 128, None, 128, a, 128, a, 128, "swish", None, 96, None, 0, None, 0,
                       "brain") == tg.TG_OK
    assert tg.tg_layer_norm(0, 8, None, 8, None, None, 1e-5, None, 8, None, None, "single") == tg.TG_OK
    for bad in ("nothing", ""):
        with pytest.raises(KeyError):
            tg.tg_linear_workspace_bytes(64, 96, 128, a, 128, a, 128, bad)

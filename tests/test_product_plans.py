"""tg_product_plan_describe on the host (no GPU): its text, its refusals, and
what the planner may choose."""

from __future__ import annotations

import ctypes
import re

import pytest

from mlp_schedules import SCHEDULES, schedule

SMS = 152
PRODUCTS = ["linear", "gated", "linear_dx", "gated_dx", "linear_dw", "gated_dw"]


@pytest.fixture(scope="module")
def tg():
    import dense_gemm_epilogue_gb300 as tg

    tg.build()
    tg.load()
    return tg


def test_text(tg):
    d = tg.tg_product_plan_describe
    assert d("gated", 4, 14336, 4096, SMS) == "stream 128x16 tiles=112 k_blocks=64 grid=152"
    assert d("linear_dx", 50, 8, 300, SMS) == "stream 128x64 tiles=3 k_blocks=1 grid=1"
    assert d("linear", 4097, 8200, 1032, SMS) == (
        "pair 256x256 tiles=561 k_blocks=17 grid=152 raster=12 split=0x1 schedule=ticket beside=0")
    assert d("linear", 0, 8, 8, SMS) == d("linear_dx", 8, 8, 0, SMS) == "empty"
    assert d("linear", 8, 8, 0, SMS).startswith("single 128x128 tiles=1 k_blocks=0 ")
    assert d("gated_dx", 200, 1000, 136, SMS).split()[3] == "k_blocks=32"  # two pairs of 16


def test_refusals(tg):
    f = tg.load().tg_product_plan_describe
    buf = ctypes.create_string_buffer(200)
    assert f(0, 8, 8, 8, SMS, buf, 200) == tg.TG_OK
    for bad in ((-1, 8, 8, 8), (6, 8, 8, 8), (0, -1, 8, 8), (0, 8, -1, 8), (0, 8, 8, 1 << 31)):
        assert f(*bad, SMS, buf, 200) == tg.TG_ERR_INVALID_VALUE
    assert f(0, 8, 8, 8, SMS, None, 200) == tg.TG_ERR_INVALID_VALUE
    assert f(0, 8, 8, 8, SMS, buf, 0) == tg.TG_ERR_INVALID_VALUE
    assert f(0, 8, 8, 8, SMS, buf, 9) == tg.TG_ERR_INVALID_VALUE
    assert buf.value == b"stream 1"
    with pytest.raises(KeyError):
        tg.tg_product_plan_describe("product", 8, 8, 8, SMS)


def test_streaming_ends_at_32_or_64_tokens(tg):
    d = tg.tg_product_plan_describe
    for p, most in (("linear", 64), ("gated", 32), ("linear_dx", 64), ("gated_dx", 64)):
        assert d(p, most, 264, 520, SMS).startswith("stream ")
        assert not d(p, most + 1, 264, 520, SMS).startswith("stream ")
    for p in ("linear_dw", "gated_dw"):
        assert not d(p, 3, 264, 520, SMS).startswith("stream ")


def plans(tg, products=PRODUCTS):
    """Tile plans over a fixed sweep of sizes: the text's fields."""
    sizes = (1, 72, 129, 200, 333, 520, 777, 1001, 2056, 4096, 8200)
    for p in products:
        for m in sizes:
            for n in sizes:
                for k in (8, 136, 1000, 2100, 4096, 14336):
                    t = tg.tg_product_plan_describe(p, m, n, k, SMS)
                    r = re.fullmatch(r"(pair|single) (\d+)x(\d+) tiles=(\d+) k_blocks=(\d+) grid=(\d+) "
                                     r"raster=(\d+) split=(\d+)x(\d+) schedule=(ticket|static) beside=([01])", t)
                    if r:
                        yield p, (m, n, k), r[1], *[int(v) for v in r.groups()[1:9]], r[10], r[11] == "1"


def test_plans_keep_the_kernels_limits(tg):
    for p, size, kind, rows, cols, tiles, kb, grid, raster, tail, segs, sched, beside in plans(tg):
        cg = 2 if kind == "pair" else 1
        teams = SMS // cg
        assert rows == 128 * cg and cols in (128, 256), size
        assert 0 < grid <= SMS and grid % cg == 0 and 1 <= segs <= 4 and raster >= 1, size
        assert tail == (tiles % teams if segs > 1 else 0), size
        assert segs == 1 or (kb // segs >= 8 and tail * segs <= teams), size
        assert sched == "static" or (tiles >= 6 * teams and kb >= 16), size
        if beside and p.endswith("_dw"):
            assert segs == 1 and sched == "static", size


@pytest.mark.parametrize("m,n,k", [(777, 1001, 1365), (777, 1000, 1368), (600, 1100, 1300), (900, 1030, 1290)])
def test_gradients_planned_together_have_room(tg, m, n, k):
    """Both products at once: a CTA pair needs both SMs of a neighbouring two,
    and single CTAs in front of it take one SM of as many twos as there are."""
    def plan(p):
        r = re.match(r"(\w+) \S+ tiles=\d+ k_blocks=\d+ grid=(\d+) ", tg.tg_product_plan_describe(p, m, n, k, SMS))
        return r[1], int(r[2])

    (xkind, x), (wkind, w) = plan("linear_dx"), plan("linear_dw")
    assert x + w <= SMS
    if wkind == "pair":
        assert (x // 2 if xkind == "pair" else min(x, SMS // 2)) + w // 2 <= SMS // 2


def test_every_instantiated_tile_shape_is_chosen(tg):
    """Each product is compiled for exactly the tile shapes that its plans name."""
    shapes = {}
    for p, _, kind, rows, cols, *_ in plans(tg):
        shapes.setdefault(p, set()).add((kind, rows, cols))
    for p in PRODUCTS:
        forward = {("pair", 256, 256), ("single", 128, 256), ("single", 128, 128)}
        assert shapes[p] == (forward if p in ("linear", "gated") else forward | {("pair", 256, 128)}), p


@pytest.mark.parametrize("product,m,n,k,shape,order,split", SCHEDULES)
def test_schedules_are_planned_as_listed(tg, product, m, n, k, shape, order, split):
    """The GPU tests of these sizes run the schedules that they are listed for."""
    text = tg.tg_product_plan_describe(product, m, n, k, SMS)
    assert schedule(text, SMS) == (shape, order, split), text


def test_every_schedule_of_the_sweep_is_listed(tg):
    listed = {(s[0], s[4], s[5], s[6]) for s in SCHEDULES}
    for p, (m, n, k), *_ in plans(tg):
        found = schedule(tg.tg_product_plan_describe(p, m, n, k, SMS), SMS)
        assert (p, *found) in listed, (p, m, n, k, found)

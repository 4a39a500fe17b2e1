"""Rotary positions against FP64: layouts, partial heads, scalings, far
positions, strides, cache rows, in place, and the gradient.

Bound: the angle's sine and cosine are FP32 values within 2^-23 (the fraction of
a turn to 2^-27, the functions to an ulp, the amplitude's product a rounding);
with the two products and the sum, 2^-21 (|a| + |b|) amplitude; then the result's
rounding, half a step of the type."""

from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

from attn_harness import Tensor3, check, done, gen  # noqa: E402

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "f32": torch.float32}
U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "f32": 2.0 ** -24}
TINY = {"bf16": 0.0, "fp16": 2.0 ** -25, "f32": 0.0}


@pytest.fixture(scope="module")
def tg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import dense_gemm_epilogue_gb300 as tg

    tg.build()
    tg.load()
    return tg


def frequencies(rot, base=10000.0, scaling="none", factor=1.0, low=1.0, high=4.0, original=8192.0):
    if scaling == "base":
        base = base * factor ** (rot / (rot - 2))
    out = []
    for i in range(rot // 2):
        f = base ** (-2 * i / rot)
        if scaling == "linear":
            f /= factor
        if scaling == "bands":
            g = min(max((original * f / (2 * math.pi) - low) / (high - low), 0.0), 1.0)
            f = g * f + (1 - g) * f / factor
        out.append(f)
    return torch.tensor(out, dtype=torch.float64, device="cuda")


def turned(x, pos, freq, layout, amplitude, transpose):
    """FP64 (y, the bound before the result's rounding)."""
    r = 2 * len(freq)
    p = pos.double()[:, None, None] * freq
    c, s = torch.cos(p) * amplitude, torch.sin(p) * amplitude * (-1 if transpose else 1)
    y, e = x.clone(), torch.zeros_like(x)
    ia = torch.arange(0, r // 2, device="cuda") if layout == "halves" else torch.arange(0, r, 2, device="cuda")
    ib = ia + r // 2 if layout == "halves" else ia + 1
    a, b = x[..., ia], x[..., ib]
    y[..., ia] = a * c - b * s
    y[..., ib] = a * s + b * c
    err = 2.0 ** -21 * (a.abs() + b.abs()) * abs(amplitude)
    e[..., ia] = err
    e[..., ib] = err
    return y, e


def run(tg, tokens, heads, dim, rot, dtype="bf16", layout="halves", amplitude=1.0, positions=None, seed=3,
        transpose=False, inplace=False, rows=None, y_rows=0, shape={}, oshape=None, **scaling):
    x = Tensor3(tokens, heads, dim, dtype, fill=torch.randn(tokens, heads, dim, generator=gen(seed),
                                                            device="cuda"), **shape)
    freq = frequencies(rot, **scaling)
    steps = torch.tensor(tg.tg_rotary_steps(rot, **{"base": 10000.0, **scaling}),
                         dtype=torch.int64, device="cuda") if rot else None
    pos = torch.arange(tokens, device="cuda") if positions is None else positions
    want, e = turned(x.d(), pos, freq, layout, amplitude, transpose)
    u = U[dtype]
    bound = e + u * (want.abs() + e) + TINY[dtype]
    bound[..., rot:] = 0.0
    y = x if inplace else Tensor3(y_rows if rows is not None else tokens, heads, dim, dtype,
                                  **(shape if oshape is None else oshape))
    st = torch.cuda.current_stream()
    if transpose:
        status = tg.tg_rotary_backward(tokens, heads, dim, rot, *x.lay, *y.lay, positions, steps, layout,
                                       amplitude, dtype, st)
    else:
        status = tg.tg_rotary(tokens, heads, dim, rot, *x.lay, *y.lay, y_rows, positions, rows, steps,
                              layout, amplitude, dtype, st)
    done(tg, status, "tg_rotary")
    what = f"rotary {tokens}x{heads}x{dim} rot {rot} {dtype} {layout}"
    if rows is None:
        check(y.t, want, bound, what)
        assert y.kept_outside(torch.ones(tokens, dtype=torch.bool, device="cuda")), what
    else:
        go = (rows >= 0) & (rows < y_rows)
        check(y.t[rows[go]], want[go], bound[go], what)
        hit = torch.zeros(y_rows, dtype=torch.bool, device="cuda")
        hit[rows[go]] = True
        assert y.kept_outside(hit), what
    return y


@pytest.mark.parametrize("layout", ["halves", "pairs"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "f32"])
@pytest.mark.parametrize("tokens,heads,dim,rot", [(1, 1, 2, 2), (1, 40, 128, 128), (17, 3, 96, 32), (5, 2, 80, 20),
                                                  (300, 5, 72, 72), (1000, 1, 64, 0), (3, 7, 63, 62),
                                                  (2, 2, 4096, 4096), (9, 1, 256, 256), (700, 33, 128, 64)])
def test_sizes(tg, tokens, heads, dim, rot, dtype, layout):
    run(tg, tokens, heads, dim, rot, dtype, layout)


@pytest.mark.parametrize("scaling", [dict(base=10000.0, scaling="linear", factor=8.0),
                                     dict(base=10000.0, scaling="base", factor=4.0),
                                     dict(base=10000.0, scaling="bands", factor=8.0, low=1.0, high=4.0,
                                          original=8192.0),
                                     dict(base=10000.0, scaling="linear", factor=0.125)])
def test_scalings(tg, scaling):
    """(factor 1/8: the fastest pairs turn by more than a whole turn a position.)"""
    run(tg, 4096, 2, 128, 128, "f32", positions=torch.arange(4096, device="cuda") * 31, **scaling)


def test_far_and_negative_positions(tg):
    """At 2^24 positions 2^-53 of a position's angle is 2^-29 radians, far below the bound."""
    pos = torch.tensor([0, 1, -1, 131071, 1000000, -999999, 1 << 24, (1 << 24) - 1], device="cuda")
    for layout in ("halves", "pairs"):
        run(tg, 8, 3, 128, 128, "f32", layout, positions=pos)


@pytest.mark.parametrize("shape", [dict(pad=8), dict(pad=3), dict(gap=8), dict(gap=1), dict(heads_first=True),
                                   dict(heads_first=True, pad=5)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strides_and_in_place(tg, shape, dtype):
    for inplace in (False, True):
        run(tg, 61, 4, 72, 48, dtype, "halves", shape=shape, inplace=inplace)
    run(tg, 61, 4, 72, 48, dtype, "pairs", shape=shape, oshape=dict(pad=16))


def test_amplitude_and_gradient(tg):
    for layout in ("halves", "pairs"):
        run(tg, 50, 4, 128, 64, "fp16", layout, amplitude=1.25)
        run(tg, 50, 4, 128, 64, "bf16", layout, amplitude=1.25, transpose=True)
        run(tg, 50, 4, 128, 64, "f32", layout, amplitude=-0.5, transpose=True, inplace=True)


@pytest.mark.parametrize("rot", [0, 64])
def test_cache_rows(tg, rot):
    """Tokens to their rows of a cache; those outside are skipped, other rows kept."""
    rows = torch.tensor([5, 0, 99, -1, 100, 7, 1 << 40, 31], device="cuda")
    for dtype in ("bf16", "f32"):
        run(tg, 8, 6, 64, rot, dtype, "halves", rows=rows, y_rows=100, positions=rows.clone() % 1000,
            oshape=dict(pad=8))

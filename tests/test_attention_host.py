"""Argument checks and plans of the attention operators (no GPU): every refusal
comes back before CUDA is touched, empty problems launch nothing, frequencies
follow their formulas."""

from __future__ import annotations

import ctypes
import math

import pytest


@pytest.fixture(scope="module", params=["module", "ctypes"])
def tg(request):
    """Through the marshalling module, and through ctypes alone."""
    import dense_gemm_epilogue_gb300 as tg

    tg.build()
    tg.load()
    kept = tg._call
    if request.param == "ctypes":
        tg._call = None
    elif kept is None:
        pytest.skip("built without Python's headers")
    yield tg
    tg._call = kept


A = 1 << 20  # an aligned non-NULL address; never dereferenced here
INVALID, UNSUPPORTED, OK = 1, 2, 0
NAN, INF = float("nan"), float("inf")

SIZES = dict(seqs=2, q_rows=64, k_rows=96, heads=8, kv_heads=2, dim=64)


def attention(tg, **over):
    a = dict(SIZES, Q=A, ldq=512, hq=64, K=A, ldk=128, hk=64, V=A, ldv=128, hv=64, q_starts=A,
             q_lengths=None, k_starts=A, k_lengths=A, max_q=0, max_k=0, causal=1, scale=0.125, O=A, ldo=512,
             ho=64, LSE=A, dtype="bf16", workspace=None, stream=None)
    a.update(over)
    return tg.tg_attention(*a.values())


@pytest.mark.parametrize("over,status", [
    (dict(seqs=-1), INVALID), (dict(q_rows=-1), INVALID), (dict(k_rows=-1), INVALID),
    (dict(q_rows=1 << 31), INVALID), (dict(k_rows=1 << 40), INVALID), (dict(seqs=1 << 31), INVALID),
    (dict(heads=0), INVALID), (dict(kv_heads=0), INVALID), (dict(heads=7), INVALID), (dict(dim=0), INVALID),
    (dict(max_q=-1), INVALID), (dict(max_k=-5), INVALID), (dict(dtype="tf32"), INVALID), (dict(dtype=9), INVALID),
    (dict(dim=12), UNSUPPORTED), (dict(dim=136, hq=136, hk=136, hv=136, ho=136, ldq=1088, ldo=1088), UNSUPPORTED),
    (dict(heads=130, kv_heads=1), UNSUPPORTED),
    (dict(Q=None), INVALID), (dict(K=None), INVALID), (dict(V=None), INVALID), (dict(O=None), INVALID),
    (dict(Q=A + 2), INVALID), (dict(K=A + 8), INVALID), (dict(V=A + 4), INVALID), (dict(O=A + 2), INVALID),
    (dict(ldq=516), INVALID), (dict(hk=60), INVALID), (dict(hk=68), INVALID), (dict(ldv=56), INVALID),
    (dict(ldo=0), INVALID), (dict(ho=32), INVALID), (dict(LSE=A + 2), INVALID),
    (dict(q_starts=None), INVALID), (dict(k_starts=None), INVALID), (dict(q_starts=A + 4), INVALID),
    (dict(k_lengths=A + 2), INVALID), (dict(causal=2), INVALID), (dict(causal=-1), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=NAN), INVALID), (dict(scale=INF), INVALID),
    (dict(workspace=(None, -1)), INVALID), (dict(ldo=504), INVALID),  # rows within the row before
    (dict(seqs=0), OK), (dict(q_rows=0, Q=None, O=None), OK),
    (dict(seqs=0, Q=None, K=None, V=None, O=None, q_starts=None, k_starts=None), OK),
])
def test_attention_statuses(tg, over, status):
    assert attention(tg, **over) == status


def backward(tg, **over):
    a = dict(SIZES, Q=A, ldq=512, hq=64, K=A, ldk=128, hk=64, V=A, ldv=128, hv=64, O=A, ldo=512, ho=64, dO=A,
             lddo=512, hdo=64, LSE=A, q_starts=A, q_lengths=None, k_starts=A, k_lengths=None, max_q=0, max_k=0,
             causal=1, scale=0.125, dQ=A, lddq=512, hdq=64, dK=A, lddk=128, hdk=64, dV=A, lddv=128, hdv=64,
             dtype="fp16", workspace=(A, 1 << 20), stream=None)
    a.update(over)
    return tg.tg_attention_backward(*a.values())


@pytest.mark.parametrize("over,status", [
    (dict(seqs=-1), INVALID), (dict(heads=9), INVALID), (dict(dim=4), UNSUPPORTED), (dict(dtype="e4m3"), INVALID),
    (dict(Q=None), INVALID), (dict(K=None), INVALID), (dict(V=None), INVALID), (dict(O=None), INVALID),
    (dict(dO=None), INVALID), (dict(LSE=None), INVALID), (dict(LSE=A + 2), INVALID), (dict(dQ=A + 2), INVALID),
    (dict(dK=A + 8), INVALID), (dict(lddv=120), INVALID), (dict(hdq=56), INVALID), (dict(lddo=500), INVALID),
    (dict(q_starts=None), INVALID), (dict(k_starts=A + 1), INVALID), (dict(causal=3), INVALID),
    (dict(scale=0.0), INVALID), (dict(workspace=None), INVALID), (dict(workspace=(A, 4 * 8 * 64 - 1)), INVALID),
    (dict(workspace=(A + 8, 1 << 20)), INVALID), (dict(workspace=(A, -1)), INVALID),
    (dict(dQ=None, dK=None, dV=None), OK), (dict(seqs=0), OK),
    (dict(q_rows=0, k_rows=0, Q=None, K=None, V=None, O=None, dO=None, LSE=None), OK),
])
def test_backward_statuses(tg, over, status):
    assert backward(tg, **over) == status


def rotary(tg, **over):
    a = dict(tokens=4, heads=2, dim=64, rot=32, X=A, ldx=128, hx=64, Y=A, ldy=128, hy=64, y_rows=0, positions=A,
             rows=None, steps=A, layout="halves", amplitude=1.0, dtype="bf16", stream=None)
    a.update(over)
    return tg.tg_rotary(*a.values())


@pytest.mark.parametrize("over,status", [
    (dict(tokens=-1), INVALID), (dict(heads=-1), INVALID), (dict(dim=-2), INVALID), (dict(rot=-2), INVALID),
    (dict(rot=66), INVALID), (dict(rot=31), INVALID), (dict(tokens=1 << 31), INVALID),
    (dict(dim=4098, ldx=9000, ldy=9000, hx=4098, hy=4098), UNSUPPORTED),
    (dict(X=None), INVALID), (dict(Y=None), INVALID), (dict(X=A + 1), INVALID), (dict(Y=A + 2, dtype="f32"), INVALID),
    (dict(ldx=63), INVALID), (dict(hy=63), INVALID), (dict(ldy=100), INVALID), (dict(hy=140), INVALID), (dict(ldy=10), INVALID), (dict(steps=None), INVALID),
    (dict(steps=A + 4), INVALID), (dict(positions=A + 4), INVALID), (dict(rows=A + 1, y_rows=9), INVALID),
    (dict(rows=A, y_rows=-1), INVALID), (dict(layout=2), INVALID), (dict(layout=-1), INVALID),
    (dict(amplitude=NAN), INVALID), (dict(amplitude=INF), INVALID), (dict(dtype=3), INVALID),
    (dict(ldy=136), INVALID), (dict(ldx=160, hx=80), INVALID),  # in place, but for other strides
    (dict(tokens=0, X=None, Y=None), OK), (dict(heads=0, X=None, Y=None), OK), (dict(dim=0, rot=0), OK),
])
def test_rotary_statuses(tg, over, status):
    assert rotary(tg, **over) == status


@pytest.mark.parametrize("over,status", [
    (dict(rot=65), INVALID), (dict(dY=None), INVALID), (dict(dX=A + 1), INVALID), (dict(lddx=1), INVALID),
    (dict(steps=None), INVALID), (dict(layout=7), INVALID), (dict(tokens=0, dY=None, dX=None), OK),
])
def test_rotary_backward_statuses(tg, over, status):
    a = dict(tokens=4, heads=2, dim=64, rot=32, dY=A, lddy=128, hdy=64, dX=A, lddx=128, hdx=64, positions=None,
             steps=A, layout="pairs", amplitude=1.0, dtype="fp16", stream=None)
    a.update(over)
    assert tg.tg_rotary_backward(*a.values()) == status


def as_turns(steps):
    return [(v % (1 << 64)) / 2.0 ** 64 for v in steps]


@pytest.mark.parametrize("rot", [2, 4, 64, 128, 4096])
@pytest.mark.parametrize("scaling", ["none", "linear", "base", "bands"])
def test_frequencies(tg, rot, scaling):
    if scaling == "base" and rot == 2:
        with pytest.raises(tg.TgError):
            tg.tg_rotary_steps(rot, 10000.0, scaling, 8.0)
        return
    got = as_turns(tg.tg_rotary_steps(rot, 10000.0, scaling, 8.0, 1.0, 4.0, 8192.0))
    for i, t in enumerate(got):
        base = 10000.0 * 8.0 ** (rot / (rot - 2)) if scaling == "base" else 10000.0
        f = base ** (-2 * i / rot)
        if scaling == "linear":
            f /= 8
        if scaling == "bands":
            g = min(max((8192 * f / (2 * math.pi) - 1) / 3, 0), 1)
            f = g * f + (1 - g) * f / 8
        # pow's last place, at most a few of FP64's
        assert abs(t - f / (2 * math.pi)) <= 2 ** -49 * f + 2.0 ** -64


@pytest.mark.parametrize("over", [
    dict(rot=0), dict(rot=3), dict(rot=-2), dict(rot=4098), dict(base=0.0), dict(base=-1.0), dict(base=NAN),
    dict(base=INF), dict(factor=0.0), dict(factor=NAN), dict(scaling=4), dict(scaling=-1),
    dict(scaling="bands", low=4.0, high=1.0), dict(scaling="bands", original=0.0),
    dict(scaling="bands", high=INF),
])
def test_frequency_refusals(tg, over):
    a = dict(rot=64, base=10000.0, scaling="none", factor=1.0, low=1.0, high=4.0, original=8192.0)
    a.update(over)
    with pytest.raises(tg.TgError):
        tg.tg_rotary_steps(**a)


def plan(tg, *args, sms=152):
    text = tg.tg_attention_plan_describe(*args, sms)
    return dict((k, int(v)) for k, v in (x.split("=") for x in text.split()))


def test_plans(tg):
    """Pieces of work cover every tile of every sequence, key ranges every block."""
    # a long prompt: two row tiles a CTA, whole key ranges
    p = plan(tg, 1, 8192, 8192, 32, 8, 128, 8192, 8192, "bf16")
    assert p == {"tiles": 2, "ctas": 128 * 8, "ranges": 1, "blocks": 64}
    # one token over a long cache: single tiles, a whole round of CTAs
    p = plan(tg, 1, 1, 131072, 32, 8, 128, 1, 131072, "bf16")
    assert p["tiles"] == 1 and p["ctas"] >= 152 and p["ranges"] * p["blocks"] >= 1024
    # single tokens of several sequences: ranges of at most 16 blocks
    p = plan(tg, 32, 32, 32 * 8192, 32, 8, 128, 1, 8192, "bf16")
    assert p["tiles"] == 1 and p["blocks"] <= 16 and p["ranges"] * p["blocks"] >= 64
    # a chunk behind a long prefix: two tiles, key ranges
    p = plan(tg, 1, 500, 16500, 32, 8, 128, 500, 16500, "bf16")
    assert p["tiles"] == 2 and p["ranges"] > 1 and p["ranges"] * p["blocks"] >= 129
    # short texts: a tile a sequence
    p = plan(tg, 16, 333, 333, 12, 12, 80, 49, 49, "fp16")
    assert p == {"tiles": 1, "ctas": 16 * 12, "ranges": 1, "blocks": 1}
    assert tg.tg_attention_plan_describe(0, 5, 5, 1, 1, 64, 0, 0, "bf16", 152) == "empty"
    with pytest.raises(tg.TgError):
        tg.tg_attention_plan_describe(1, 5, 5, 3, 2, 64, 0, 0, "bf16", 152)


def test_argument_kinds(tg):
    with pytest.raises(KeyError):
        rotary(tg, layout="quarters")
    with pytest.raises(TypeError):
        attention(tg, Q="not a pointer")
    with pytest.raises((TypeError, ctypes.ArgumentError)):
        attention(tg, heads=1.5)
    with pytest.raises((TypeError, ctypes.ArgumentError)):
        backward(tg, scale="x")
    with pytest.raises(TypeError):
        backward(tg, stream="not a stream")


@pytest.mark.parametrize("rot,base", [(128, 500000.0), (64, 10000.0), (4096, 1e6), (2, 10000.0)])
@pytest.mark.parametrize("scaling", ["none", "linear", "base", "bands"])
def test_frequencies_to_the_nearest_step(tg, rot, base, scaling):
    """Against 60 digits.  A step is off by half of 2^-64 turns and by FP64's roundings: the
    exponent's, times ln base, and those of pow, 2 pi, base and the scaling, fewer than 32."""
    from decimal import Decimal as D
    from decimal import localcontext

    if scaling == "base" and rot == 2:
        pytest.skip("refused")
    got = tg.tg_rotary_steps(rot, base, scaling, 8.0, 1.0, 4.0, 8192.0)
    with localcontext() as c:
        c.prec = 60
        two_pi = 2 * D("3.14159265358979323846264338327950288419716939937510582097494459")
        b = D(base) * (D(8) ** (D(rot) / D(rot - 2)) if scaling == "base" else 1)
        for i, step in enumerate(got):
            f = b ** (-D(2 * i) / D(rot))
            if scaling == "linear":
                f /= 8
            if scaling == "bands":
                g = min(max((8192 * f / two_pi - 1) / 3, D(0)), D(1))
                f = g * f + (1 - g) * f / 8
            want = f / two_pi * 2 ** 64
            rel = (math.log(base * 8) + 32) * 2.0 ** -53
            assert abs(step % (1 << 64) - want) <= D(0.5) + want * D(rel), i


@pytest.mark.parametrize("over", [dict(base=1e300, factor=1e10), dict(base=10000.0, factor=1e200, rot=4),
                                  dict(base=1e-200, factor=1e-200, rot=4)])
def test_scaled_base_out_of_range(tg, over):
    """base factor^(rot/(rot-2)) beyond FP64: no frequencies that never turn."""
    with pytest.raises(tg.TgError):
        tg.tg_rotary_steps(**dict(dict(rot=64, scaling="base"), **over))


def test_frequencies_of_a_huge_rotary(tg):
    """Refused by the library, not by the memory for its answer."""
    for rot in (1 << 40, 1 << 62):
        with pytest.raises(tg.TgError):
            tg.tg_rotary_steps(rot, 10000.0)


def test_argument_counts_name_their_call(tg):
    """A wrong number of arguments is reported under the name of the call that was made."""
    if tg._call is None:
        pytest.skip("ctypes counts them")
    for name in ("tg_rotary", "tg_rotary_backward", "tg_attention_workspace_bytes", "tg_attention",
                 "tg_attention_backward_workspace_bytes", "tg_attention_backward"):
        with pytest.raises(TypeError, match=f"^{name}: 1 arguments"):
            getattr(tg._call, name)(1)


@pytest.mark.parametrize("sizes", [(1 << 29, (1 << 31) - 600, (1 << 31) - 600, 65536, 65536, 128, 1, 0),
                                   (1 << 29, 1 << 30, (1 << 31) - 600, 128, 128, 8, 2, 0)])
def test_more_pieces_than_a_grid(tg, sizes):
    """More row tiles than a grid has CTAs: TG_ERR_UNSUPPORTED, in the description as in the
    call."""
    with pytest.raises(tg.TgError, match="TG_ERR_UNSUPPORTED"):
        tg.tg_attention_plan_describe(*sizes, "bf16", 152)


@pytest.mark.parametrize("sizes", [(1 << 16, 1 << 16, (1 << 31) - 600, 64, 64, 64, 1, 0),
                                   (1 << 26, 1 << 26, (1 << 31) - 600, 8, 8, 8, 1, 0),
                                   (2, 3, (1 << 31) - 600, 8, 8, 8, 1, 0)])
def test_key_ranges_stay_within_a_grid(tg, sizes):
    p = plan(tg, *sizes, "bf16")
    assert p["ctas"] == sizes[0] * sizes[4] * p["ranges"] < 1 << 31
    assert p["ranges"] * p["blocks"] >= -(-sizes[2] // 128)

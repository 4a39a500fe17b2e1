"""The activations' far negative tails: y sigmoid(y) is a normal BF16 and FP32
number down to y = -91.8, and GELU's tail down to y = -10.15, where the logistic
function itself is subnormal or 1 + exp(-y) past FP32's largest number.

With K = 1 and X = 1 the pre-activations are W's values, without rounding.  The
references are FP64, y / (1 + exp(-t)); for GELU t = 2 sqrt(2/pi) (y + 0.044715
y^3), the logistic form of the tanh, which has no cancellation in 1 + tanh.

Bounds, relative to the value: u = -t log2 e, |u| < 192, is off by at most four
roundings of FP32 constants and products (2^-24 each) and one of its own, 5 |u|
2^-24 < 2^-14, so 2^u by less than ln 2 times that; exponential, reciprocal and
products add under 2^-20.  In all less than 2^-14.  Where the logistic function
is subnormal, 2^-150 of absolute error in it, times the factors it meets.
"""

from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import mlp_harness as h

REL = 2.0 ** -14
TINY = 2.0 ** -150  # half of FP32's smallest subnormal
BF16_TINY = 2.0 ** -134


@pytest.fixture(scope="module")
def tg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import dense_gemm_epilogue_gb300 as tg

    tg.build()
    tg.load()
    return tg


def tail(act):
    """BF16 values of the tail, from where it is ordinary to where it ends."""
    if act == "silu":
        v = torch.arange(-130.0, -60.0, 0.5)  # BF16's spacing is 1 from 128 on
        v = torch.cat([v, torch.tensor([-500.0, -1e4, -1e30, 0.0, 1.0, 90.0, 1e30])])
    else:
        v = torch.arange(-11.0, -7.0, 2.0 ** -4)
        v = torch.cat([v, torch.tensor([-15.5, -16.0, -500.0, -1e30, 0.0, 1.0, 16.0, 1e30])])
    return v.to(torch.bfloat16).cuda()


def logistic(act, y):
    t = y if act == "silu" else 2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3)
    return 1 / (1 + torch.exp(-t))


def slope(act, y):
    """d/dy of y logistic(t(y))."""
    s = logistic(act, y)
    dt = torch.ones_like(y) if act == "silu" else 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * y * y)
    d = s + torch.where(s == 1, torch.zeros_like(y), y * dt * s * (1 - s))
    size = s + torch.where(s == 1, torch.zeros_like(y), y.abs() * dt * s * (1 - s))
    factor = torch.where((s == 0) | (y > 0), torch.zeros_like(y), 1 + y.abs() * dt)
    return d, size, factor


def check(got, want, bound, what):
    bad = ~((got.double() - want).abs() <= bound)
    assert not bad.any(), (what, got[bad][:4], want[bad][:4], bound[bad][:4])


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("m", [3, 200])  # the streaming and the tile kernel
def test_linear_tail(tg, m, act):
    w = tail(act)
    n = w.numel()
    x = torch.ones(m, 8, dtype=torch.bfloat16, device="cuda")
    wm = torch.zeros(n, 8, dtype=torch.bfloat16, device="cuda")
    wm[:, 0] = w
    y = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    h.done(tg, tg.tg_linear(m, n, 1, x, 8, wm, 8, None, act, None, 0, y, n, None, 0, "bf16", None,
                            torch.cuda.current_stream()), "tg_linear")
    v = w.double()
    want = v * logistic(act, v)
    bound = (REL + h.U["bf16"]) * want.abs() + TINY * (1 + v.abs().clamp(max=1e4)) + BF16_TINY
    check(y, want.expand(m, n), bound.expand(m, n), f"linear {act}")


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("m", [3, 200])
def test_gated_tail(tg, m, act):
    """Times an up value of 2^30, so that the tail's end is no subnormal."""
    w = tail(act)
    w = w[w.abs() < 1e4]
    n, up = w.numel(), 2.0 ** 30
    x = torch.ones(m, 8, dtype=torch.bfloat16, device="cuda")
    wg = torch.zeros(n, 8, dtype=torch.bfloat16, device="cuda")
    wg[:, 0] = w
    wu = torch.zeros(n, 8, dtype=torch.bfloat16, device="cuda")
    wu[:, 0] = up
    y = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    h.done(tg, tg.tg_gated(m, n, 1, x, 8, wg, 8, wu, 8, act, y, n, None, 0, None, 0, "bf16", None,
                           torch.cuda.current_stream()), "tg_gated")
    v = w.double()
    want = v * logistic(act, v) * up
    bound = (REL + h.U["bf16"]) * want.abs() + up * TINY * (1 + v.abs()) + BF16_TINY
    check(y, want.expand(m, n), bound.expand(m, n), f"gated {act}")


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_backward_tail(tg, act):
    """db of one row is dY act'(Z) in FP32."""
    z = tail(act)[None].contiguous()
    n = z.numel()
    dy = torch.full((1, n), -2.0, dtype=torch.bfloat16, device="cuda")
    db = torch.empty(n, device="cuda")
    ws = h.space(tg.tg_linear_backward_workspace_bytes(1, n, 8, dy, n, None, 8, None, 8, act, "bf16"))
    h.done(tg, tg.tg_linear_backward(1, n, 8, dy, n, None, 8, None, 8, z, n, act, None, 8, None, 8,
                                     "bf16", db, "bf16", ws, torch.cuda.current_stream()), "backward")
    d, size, factor = slope(act, z[0].double())
    check(db, -2 * d, 2 * (REL * size + TINY * (2 + factor)), f"backward {act}")

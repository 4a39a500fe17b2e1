"""Seeded random feed-forward problems through the planner's own choices: sizes,
strides, bases, types and optional parts together, against the FP64 definitions
(tests/mlp_harness.py)."""

from __future__ import annotations

import math
import os
import random

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import mlp_harness as h

COUNT = int(os.environ.get("TG_MLP_FUZZ", "120"))


@pytest.fixture(scope="module")
def tg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import dense_gemm_epilogue_gb300 as tg

    tg.build()
    tg.load()
    return tg


def size(rng, hi):
    n = max(1, int(round(math.exp(rng.uniform(0.0, math.log(hi))))))
    unit = rng.choice([1, 1, 8, 64])
    return max(1, n // unit * unit)


@pytest.mark.parametrize("seed", range(COUNT))
def test_random_problem(tg, seed):
    rng = random.Random(7000 + seed)
    m, n, k = size(rng, 1500), size(rng, 2500), size(rng, 2500)
    dtype = rng.choice(["bf16", "fp16"])
    act = rng.choice(["none", "relu", "silu", "gelu_tanh"])
    pad, skew = rng.choice([(0, 0), (0, 0), (8, 0), (1, 0), (5, 3), (0, 1), (16, 8), (3, 7)])
    dw = rng.choice(["same", "f32"])
    op = rng.choice(["linear", "linear", "linear_backward", "gated", "gated_backward", "norm"])
    if op == "linear":
        opad, oskew = (pad, skew) if rng.random() < 0.5 else (rng.choice([0, 8, 1]), rng.choice([0, 8, 1]))
        residual = rng.random() < 0.5
        h.check_linear(tg, m, n, k, dtype, act, bias=rng.random() < 0.6, residual=residual,
                       save=rng.random() < 0.4, pad=pad, skew=skew, opad=opad, oskew=oskew, seed=seed,
                       inplace=residual and rng.random() < 0.3)
    elif op == "linear_backward":
        h.check_linear_backward(tg, m, n, k, dtype, act, bias=rng.random() < 0.7, pad=pad, skew=skew, dw=dw,
                                seed=seed, want_dx=rng.random() < 0.85, want_dw=rng.random() < 0.85)
    elif op == "gated":
        h.check_gated(tg, m, n, k, dtype, act, save=rng.random() < 0.4, pad=pad, skew=skew, seed=seed)
    elif op == "gated_backward":
        want = tuple(rng.random() < 0.85 for _ in range(3))
        h.check_gated_backward(tg, m, n, k, dtype, act, pad=pad, skew=skew, dw=dw, seed=seed, want=want)
    else:
        t = rng.choice(["bf16", "fp16", "f32"])
        cols = size(rng, 20000)
        rows = max(1, min(m, 20_000_000 // cols))
        h.check_norm(tg, rows, cols, t, affine=rng.random() < 0.7, save=rng.random() < 0.5, pad=pad,
                     skew=skew, seed=seed)
        h.check_norm_backward(tg, rows, cols, t, affine=rng.random() < 0.7, pad=pad, skew=skew, seed=seed)

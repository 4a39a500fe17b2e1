"""Attention over packed sequences against FP64 within derived bounds
(attn_harness.py): lengths, head layouts, masks, strides, paths."""

from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import attn_harness as ah  # noqa: E402


@pytest.fixture(scope="module")
def tg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import dense_gemm_epilogue_gb300 as tg

    tg.build()
    tg.load()
    return tg


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 127, 128, 129, 300])
def test_one_sequence(tg, n, dim, dtype):
    ah.check_forward(tg, ah.Problem([n], heads=2, kv=1, dim=dim, dtype=dtype, causal=n % 2 == 1))


@pytest.mark.parametrize("dim", [8, 16, 40, 72, 80, 96, 120])
def test_head_sizes_between_tiles(tg, dim):
    ah.check_forward(tg, ah.Problem([130, 7], heads=4, kv=2, dim=dim, dtype="fp16"))


@pytest.mark.parametrize("heads,kv", [(1, 1), (3, 1), (5, 1), (7, 7), (12, 4), (40, 2), (128, 1), (96, 2)])
def test_groups_of_heads(tg, heads, kv):
    ah.check_forward(tg, ah.Problem([70, 3], heads=heads, kv=kv, dim=64))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("q_len,k_len", [
    ([5, 0, 300, 1, 64], None),
    ([5, 0, 300, 1, 64], [9, 17, 411, 0, 64]),
    ([200, 130], [100, 3]),            # causal: rows without keys
    ([0, 0], [5, 0]),
    ([1, 1, 1], [700, 1, 129]),
    ([4, 4], [1000, 30]),
])
def test_packed_lengths(tg, q_len, k_len, causal):
    ah.check_forward(tg, ah.Problem(q_len, k_len, heads=4, kv=2, dim=64, causal=causal))


def test_many_tiles_two_a_cta(tg):
    """More row tiles than SMs: two a CTA, with odd counts and ragged ends."""
    ah.check_forward(tg, ah.Problem([700, 129, 385, 1, 0, 1000], heads=16, kv=16, dim=64, dtype="fp16"))
    ah.check_forward(tg, ah.Problem([1111, 260], heads=16, kv=8, dim=128))
    ah.check_forward(tg, ah.Problem([900, 513], [300, 1200], heads=16, kv=16, dim=128))
    ah.check_forward(tg, ah.Problem([640, 300], [257, 64], heads=24, kv=12, dim=96, causal=False))


@pytest.mark.parametrize("dim,dtype", [(128, "bf16"), (64, "fp16")])
def test_single_tokens_over_a_cache(tg, dim, dtype):
    """Slabs of 5000 rows, filled unevenly; long ones are cut into key ranges."""
    k = [5000, 1, 0, 4097, 640, 129]
    at = [5000 * i for i in range(6)]
    p = ah.Problem([1] * 6, k, heads=8, kv=2, dim=dim, dtype=dtype, k_at=at, k_rows=30000,
                   q_at=list(range(6)))
    assert tg.tg_attention_workspace_bytes(*p.sizes(), p.max_q, p.max_k, dtype) > 0
    ah.check_forward(tg, p)


@pytest.mark.parametrize("shape", [dict(pad=8), dict(gap=8), dict(pad=24, gap=16), dict(heads_first=True),
                                   dict(heads_first=True, pad=8, gap=64)])
def test_strides(tg, shape):
    ah.check_forward(tg, ah.Problem([150, 33], [170, 33], heads=4, kv=2, dim=72, **shape))


def test_rows_of_no_sequence(tg):
    """Gaps before, between and behind the sequences hold NaN and stay so."""
    p = ah.Problem([100, 37], [130, 1], heads=2, kv=2, dim=64, q_at=[7, 200], k_at=[3, 300], q_rows=260,
                   k_rows=320)
    ah.check_forward(tg, p)


@pytest.mark.parametrize("sigma,scale", [(4.0, 1.0), (0.01, 1.0), (1.0, 30.0), (1.0, 1e-6)])
def test_score_magnitudes(tg, sigma, scale):
    ah.check_forward(tg, ah.Problem([300], heads=2, kv=1, dim=64, sigma=sigma, scale=scale))


def test_growing_maxima(tg):
    """Later keys outgrow the reference again and again: every block rescales."""
    p = ah.Problem([400], heads=2, kv=2, dim=64, causal=False, scale=1.0)
    p.Q.t.fill_(0.25)
    ramp = torch.arange(400, device="cuda").float()[:, None, None] / 16
    p.K.t.copy_(ramp.expand(400, 2, 64).to(torch.bfloat16))
    ah.check_forward(tg, p)

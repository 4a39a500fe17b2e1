"""The attention's gradients against FP64 within derived bounds
(attn_harness.py), and against differences of the forward definition."""

from __future__ import annotations

import math

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
    ah.check_backward(tg, ah.Problem([n], heads=2, kv=1, dim=dim, dtype=dtype, causal=n % 2 == 1))


@pytest.mark.parametrize("dim", [8, 16, 40, 72, 80, 96, 120])
def test_head_sizes_between_tiles(tg, dim):
    ah.check_backward(tg, ah.Problem([130, 7], heads=4, kv=2, dim=dim, dtype="fp16"))


@pytest.mark.parametrize("heads,kv", [(1, 1), (3, 1), (5, 1), (7, 7), (12, 4), (40, 2), (128, 1), (96, 2)])
def test_groups_of_heads(tg, heads, kv):
    """The gradients of shared keys sum over their heads."""
    ah.check_backward(tg, ah.Problem([70, 3], heads=heads, kv=kv, dim=64))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("q_len,k_len", [
    ([5, 0, 300, 1, 64], None),
    ([5, 0, 300, 1, 64], [9, 17, 411, 0, 64]),
    ([200, 130], [100, 3]),            # causal: rows without keys
    ([0, 0], [5, 0]),                  # keys without rows: zeros
    ([1, 1, 1], [700, 1, 129]),
    ([4, 4], [1000, 30]),
])
def test_packed_lengths(tg, q_len, k_len, causal):
    ah.check_backward(tg, ah.Problem(q_len, k_len, heads=4, kv=2, dim=64, causal=causal))
    ah.check_backward(tg, ah.Problem(q_len, k_len, heads=3, kv=1, dim=128, causal=causal, dtype="fp16"))


@pytest.mark.parametrize("dim,dtype", [(64, "bf16"), (128, "fp16")])
@pytest.mark.parametrize("causal", [True, False])
def test_work_in_parts(tg, dim, dtype, causal):
    """One key head for many rows, and few rows over many keys: a key block's row tiles,
    and a row tile's key blocks, shared by several CTAs (the workspace holds their sums)."""
    for p in (ah.Problem([1500, 40, 0, 130], [300, 129, 5, 130], heads=8, kv=1, dim=dim, dtype=dtype, causal=causal),
              ah.Problem([60, 9], [4000, 700], heads=2, kv=2, dim=dim, dtype=dtype, causal=causal),
              ah.Problem([1300], heads=4, kv=1, dim=dim, dtype=dtype, causal=causal, scale=0.05)):
        delta = -(-4 * p.heads * p.q_rows // 16) * 16
        assert tg.tg_attention_backward_workspace_bytes(*p.sizes(), p.max_q, p.max_k, dtype) > delta
        out = ah.check_backward(tg, p)
        o, lse = ah.given(p)
        for n in ("dQ", "dK", "dV"):  # each wanted alone
            some = ah.run_backward(tg, p, o, lse, (n,))
            assert torch.equal(some[n].t, out[n].t), n


def test_many_tiles(tg):
    ah.check_backward(tg, ah.Problem([700, 129, 385, 1, 0, 1000], heads=16, kv=16, dim=64, dtype="fp16"))
    ah.check_backward(tg, ah.Problem([1111, 260], heads=16, kv=4, dim=128))
    ah.check_backward(tg, ah.Problem([640, 300], [257, 964], heads=24, kv=12, dim=96, causal=False))


@pytest.mark.parametrize("shape", [dict(pad=8), dict(gap=8), dict(pad=24, gap=16), dict(heads_first=True),
                                   dict(heads_first=True, pad=8, gap=64)])
def test_strides(tg, shape):
    ah.check_backward(tg, ah.Problem([150, 33], [170, 33], heads=4, kv=2, dim=72, **shape))


def test_rows_of_no_sequence(tg):
    """Gaps before, between and behind the sequences hold NaN and stay so."""
    for dim, heads in ((64, 2), (128, 6)):
        p = ah.Problem([100, 37], [130, 1], heads=heads, kv=2, dim=dim, q_at=[7, 200], k_at=[3, 300],
                       q_rows=260, k_rows=320)
        ah.check_backward(tg, p)


@pytest.mark.parametrize("sigma,scale", [(3.0, 1.0), (0.01, 1.0), (1.0, 30.0)])
def test_score_magnitudes(tg, sigma, scale):
    ah.check_backward(tg, ah.Problem([300], heads=2, kv=1, dim=64, sigma=sigma, scale=scale))


def test_wanted_gradients_only(tg):
    p = ah.Problem([200, 90], heads=4, kv=2, dim=64)
    o, lse = ah.given(p)
    every = ah.run_backward(tg, p, o, lse)
    for want in (("dQ",), ("dK",), ("dV",), ("dQ", "dV"), ("dK", "dV")):
        some = ah.run_backward(tg, p, o, lse, want)
        for n in ("dQ", "dK", "dV"):
            if n in want:
                assert torch.equal(some[n].t, every[n].t), (want, n)
            else:
                assert bool(torch.isnan(some[n].t).all()), (want, n)


def test_against_differences(tg):
    """sum(dO O) along a direction in Q, K and V: central differences of the FP64
    definition, against the kernels' gradients within their summed bounds."""
    p = ah.Problem([40, 9], [50, 9], heads=4, kv=2, dim=64, dtype="fp16")
    o, lse = ah.given(p)
    out = ah.run_backward(tg, p, o, lse)
    bound = ah.reference_backward(p, o, lse)
    x = {n: getattr(p, n).d() for n in "QKV"}

    def loss(v):
        total = 0.0
        for n in range(p.seqs):
            q0, q1, k0, k1 = p.q_at[n], p.q_at[n] + p.q_len[n], p.k_at[n], p.k_at[n] + p.k_len[n]
            for h in range(p.heads):
                s = p.scale * v["Q"][q0:q1, h] @ v["K"][k0:k1, h // p.g].t()
                see = torch.ones_like(s, dtype=torch.bool).tril(k1 - k0 - (q1 - q0))
                w = torch.softmax(s.masked_fill(~see, -math.inf), 1)
                total += float((p.dO.d()[q0:q1, h] * (w @ v["V"][k0:k1, h // p.g])).sum())
        return total

    g = ah.gen(11)
    for n in "QKV":
        d = torch.randn(x[n].shape, generator=g, dtype=torch.float64, device="cuda")
        h = 1e-4
        slope = (loss({**x, n: x[n] + h * d}) - loss({**x, n: x[n] - h * d})) / (2 * h)
        got = float((out["d" + n].d() * d).sum())
        # The differences are good to about 1e-6 of the loss's curvature; O's own rounding
        # (2^-11 of delta) reaches dQ and dK beside the bound.
        slack = float((bound["d" + n][1] * d.abs()).sum()) + 2.0 ** -11 * float(
            (bound["d" + n][0].abs() * d.abs()).sum()) + 1e-5 * abs(slope)
        assert abs(got - slope) <= slack, (n, got, slope, slack)


def test_infinities_behind_a_sequence(tg):
    """Rows, keys and values of other sequences in the same tile or block never matter."""
    for bad in (float("inf"), float("nan")):
        for heads, dim in ((2, 128), (6, 64)):
            p = ah.Problem([40, 30], [70, 90], heads=heads, kv=2, dim=dim, q_at=[0, 100], k_at=[0, 200], q_rows=200,
                           k_rows=400)
            o, lse = ah.given(p)
            want = ah.run_backward(tg, p, o, lse)
            for x in (p.K, p.V):
                x.t[70:200] = bad
                x.t[290:] = bad
            for x in (p.Q, p.dO, o):
                x.t[40:100] = bad
                x.t[130:] = bad
            lse[:, 40:100] = bad
            got = ah.run_backward(tg, p, o, lse)
            for n in want:
                rows = p.rows(keys=n != "dQ")
                assert torch.equal(got[n].t[rows], want[n].t[rows]), (n, bad, dim)


def test_repeats_streams_and_graphs(tg):
    """No sum depends on an order: bitwise the same again, on two streams at once, and
    replayed."""
    cases = [ah.Problem([500, 129, 1, 300], heads=8, kv=2, dim=128, seed=5),
             ah.Problem([700, 300], heads=16, kv=16, dim=64, dtype="fp16", seed=6)]
    given = [ah.given(p) for p in cases]
    want = [ah.run_backward(tg, p, *g) for p, g in zip(cases, given)]
    side = [torch.cuda.Stream() for _ in cases]

    def launch(p, o, lse, out, ws, s):
        lay = [x for n in ("dQ", "dK", "dV") for x in out[n].lay]
        tg.check(tg.tg_attention_backward(*p.sizes(), *p.Q.lay, *p.K.lay, *p.V.lay, *o.lay, *p.dO.lay, lse,
                                          *p.arrays(), p.max_q, p.max_k, p.causal, p.scale, *lay, p.dtype, ws, s))

    def fresh(p):
        return {"dQ": ah.Tensor3(p.q_rows, p.heads, p.dim, p.dtype), "dK": ah.Tensor3(p.k_rows, p.kv, p.dim, p.dtype),
                "dV": ah.Tensor3(p.k_rows, p.kv, p.dim, p.dtype)}

    spaces = [ah.space(tg.tg_attention_backward_workspace_bytes(*p.sizes(), p.max_q, p.max_k, p.dtype)) for p in cases]
    for _ in range(3):
        got = [fresh(p) for p in cases]
        torch.cuda.synchronize()
        for p, g, out, ws, s in zip(cases, given, got, spaces, side):
            launch(p, *g, out, ws, s)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(a[n].t, b[n].t) for n in b)
    for p, (o, lse), ws, b in zip(cases, given, spaces, want):
        out = fresh(p)
        graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=s):
            launch(p, o, lse, out, ws, s)
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out[n].t, b[n].t) for n in b)


def test_workspace_is_not_overrun(tg):
    p = ah.Problem([77, 1], heads=3, kv=1, dim=64)
    o, lse = ah.given(p)
    n = tg.tg_attention_backward_workspace_bytes(*p.sizes(), p.max_q, p.max_k, p.dtype)
    guard = torch.full((n + 256,), 0x5A, dtype=torch.uint8, device="cuda")
    out = ah.run_backward(tg, p, o, lse)
    lay = [x for k in ("dQ", "dK", "dV") for x in out[k].lay]
    ah.done(tg, tg.tg_attention_backward(*p.sizes(), *p.Q.lay, *p.K.lay, *p.V.lay, *o.lay, *p.dO.lay, lse,
                                         *p.arrays(), p.max_q, p.max_k, p.causal, p.scale, *lay, p.dtype,
                                         (guard, n), torch.cuda.current_stream()), "tg_attention_backward")
    assert bool((guard[n:] == 0x5A).all())

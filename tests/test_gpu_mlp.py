"""The feed-forward operators on the GPU against FP64 definitions
(tests/mlp_harness.py has the references and the derived bounds)."""

from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import mlp_harness as h


@pytest.fixture(scope="module")
def tg():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import dense_gemm_epilogue_gb300 as tg

    tg.build()
    tg.load()
    return tg


ACTS = ["none", "relu", "silu", "gelu_tanh"]

# Token counts around the streaming kernel's column counts and the tile edges.
TOKENS = [1, 2, 15, 16, 17, 32, 33, 64, 65, 127, 128, 129, 256, 257, 300]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("m", TOKENS)
def test_linear_token_counts(tg, m, dtype):
    h.check_linear(tg, m, 264, 200, dtype, "silu", bias=True, residual=True, save=True)


@pytest.mark.parametrize("m", [3, 130])
@pytest.mark.parametrize("n", [1, 7, 8, 63, 64, 65, 127, 128, 129, 256, 257, 520])
def test_linear_feature_counts(tg, m, n):
    h.check_linear(tg, m, n, 72, "bf16", "gelu_tanh", bias=True, residual=True)


@pytest.mark.parametrize("m", [5, 140])
@pytest.mark.parametrize("k", [1, 2, 7, 8, 15, 16, 63, 64, 65, 128, 1000, 4104])
def test_linear_reduction_lengths(tg, m, k):
    h.check_linear(tg, m, 136, k, "fp16", "none", bias=True)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("m", [4, 200])
def test_linear_epilogues(tg, m, act, bias, residual):
    h.check_linear(tg, m, 328, 192, "bf16", act, bias=bias, residual=residual, save=bias)


# pad 8: aligned rows; 1, 3: rows at odd addresses; skew: an unaligned base.
@pytest.mark.parametrize("pad,skew", [(8, 0), (1, 0), (3, 1), (0, 8), (0, 1), (8, 4)])
@pytest.mark.parametrize("m,n,k", [(9, 72, 88), (300, 152, 264), (1, 33, 65), (131, 65, 33)])
def test_linear_strides(tg, m, n, k, pad, skew):
    h.check_linear(tg, m, n, k, "fp16", "relu", bias=True, residual=True, save=True, pad=pad, skew=skew)


def test_linear_output_strides_alone(tg):
    """Aligned operands with unaligned outputs and residual, and the reverse."""
    h.check_linear(tg, 300, 200, 128, "bf16", "silu", residual=True, save=True, pad=0, opad=1, oskew=1)
    h.check_linear(tg, 300, 200, 128, "bf16", "silu", residual=True, save=True, pad=1, skew=1, opad=0, oskew=0)


@pytest.mark.parametrize("m", [6, 260])
def test_linear_residual_in_place(tg, m):
    h.check_linear(tg, m, 520, 136, "bf16", "gelu_tanh", bias=True, residual=True, inplace=True)


# K long for the tile count: split reductions (streaming shares and K segments).
@pytest.mark.parametrize("m,n,k", [(1, 128, 8192), (20, 300, 6000), (200, 200, 8200), (257, 513, 4096),
                                   (512, 1024, 4096), (1500, 1000, 2048)])
def test_linear_split_reductions(tg, m, n, k):
    h.check_linear(tg, m, n, k, "bf16", "none", bias=True, residual=True)


def test_linear_many_tiles(tg):
    """Enough tiles for the ticket schedule."""
    h.check_linear(tg, 4097, 8200, 136, "fp16", "gelu_tanh", bias=True, residual=True, save=True)


@pytest.mark.parametrize("m", [2, 150])
def test_linear_empty_reduction(tg, m):
    h.check_linear(tg, m, 100, 0, "bf16", "gelu_tanh", bias=True, residual=True)


@pytest.mark.parametrize("m", [7, 300])
def test_linear_nan_and_infinity_stay_in_their_rows(tg, m):
    g = h.gen(8)
    x, w = h.rows(g, m, 96, "bf16"), h.rows(g, 80, 96, "bf16", scale=0.1)
    x.t[2, 5] = float("nan")
    x.t[4, 9] = float("inf")
    y, _ = h.run_linear(tg, x, w, None, "relu", None, "bf16")
    want = h.act64("none", x.d() @ w.d().t())
    assert torch.isnan(y.t[2]).all()
    clean = [r for r in range(m) if r not in (2, 4)]
    assert torch.isfinite(y.t[clean]).all()
    inf = want[4]
    assert torch.equal(y.t[4][inf == math.inf].double(), inf[inf == math.inf])
    assert (y.t[4][inf == -math.inf] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("m,n,k", [(1, 64, 64), (1, 1, 1), (2, 8, 16), (65, 200, 72), (129, 257, 65),
                                   (300, 520, 264), (1000, 136, 2056), (40, 4096, 512)])
@pytest.mark.parametrize("act", ["none", "gelu_tanh"])
def test_linear_backward_sizes(tg, m, n, k, act, dtype):
    h.check_linear_backward(tg, m, n, k, dtype, act)


@pytest.mark.parametrize("act", ACTS)
def test_linear_backward_activations(tg, act):
    h.check_linear_backward(tg, 333, 264, 136, "bf16", act, dw="f32")


@pytest.mark.parametrize("pad,skew", [(8, 0), (1, 0), (3, 1), (0, 1), (16, 8)])
@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("dw", ["same", "f32"])
def test_linear_backward_strides(tg, pad, skew, act, dw):
    h.check_linear_backward(tg, 150, 93, 201, "fp16", act, pad=pad, skew=skew, dw=dw)


@pytest.mark.parametrize("dx,dw,db", [(True, False, False), (False, True, False), (False, False, True)])
@pytest.mark.parametrize("act", ["none", "relu"])
def test_linear_backward_parts(tg, dx, dw, db, act):
    h.check_linear_backward(tg, 70, 90, 110, "bf16", act, bias=db, want_dx=dx, want_dw=dw, pad=1)


def test_linear_backward_many_tiles(tg):
    h.check_linear_backward(tg, 520, 8200, 4104, "bf16", "relu")


@pytest.mark.parametrize("m,n,k", [(0, 40, 24), (24, 0, 40)])
def test_linear_backward_empty_reductions(tg, m, n, k):
    h.check_linear_backward(tg, m, n, k, "bf16", "none", bias=True)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("m", TOKENS)
def test_gated_token_counts(tg, m, dtype):
    h.check_gated(tg, m, 200, 136, dtype, "silu", save=True)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m", [3, 300])
def test_gated_activations(tg, m, act):
    h.check_gated(tg, m, 264, 192, "bf16", act, save=(act == "silu"))


@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (5, 127, 65), (140, 129, 7), (257, 64, 300), (20, 1000, 2000),
                                   (600, 1500, 4096), (1100, 2056, 72)])
def test_gated_sizes(tg, m, n, k):
    h.check_gated(tg, m, n, k, "fp16", "gelu_tanh", save=True)


@pytest.mark.parametrize("pad,skew", [(8, 0), (1, 0), (3, 1), (0, 1)])
@pytest.mark.parametrize("m", [10, 150])
def test_gated_strides(tg, m, pad, skew):
    h.check_gated(tg, m, 93, 201, "bf16", "silu", save=True, pad=pad, skew=skew)


def test_gated_empty_reduction(tg):
    h.check_gated(tg, 9, 70, 0, "bf16", "silu", save=True)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("m,n,k", [(1, 64, 64), (1, 1, 1), (65, 200, 72), (300, 520, 264), (513, 1032, 136),
                                   (40, 2048, 512)])
def test_gated_backward_sizes(tg, m, n, k, dtype):
    h.check_gated_backward(tg, m, n, k, dtype)


@pytest.mark.parametrize("act", ACTS)
def test_gated_backward_activations(tg, act):
    h.check_gated_backward(tg, 260, 136, 200, "bf16", act, dw="f32")


@pytest.mark.parametrize("pad,skew", [(8, 0), (1, 0), (3, 1), (0, 1)])
def test_gated_backward_strides(tg, pad, skew):
    h.check_gated_backward(tg, 150, 93, 201, "fp16", "gelu_tanh", pad=pad, skew=skew)


@pytest.mark.parametrize("want", [(True, False, False), (False, True, False), (False, False, True),
                                  (False, True, True)])
def test_gated_backward_parts(tg, want):
    h.check_gated_backward(tg, 140, 72, 88, "bf16", want=want)


@pytest.mark.parametrize("m,n,k", [(0, 40, 24), (24, 0, 40)])
def test_gated_backward_empty_reductions(tg, m, n, k):
    h.check_gated_backward(tg, m, n, k, "bf16")


NORM_COLS = [1, 2, 7, 31, 32, 64, 500, 512, 513, 1001, 2048, 2056, 4096, 4100, 8192, 8200, 16384,
             20000, 40000, 65536]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "f32"])
@pytest.mark.parametrize("n", NORM_COLS)
def test_norm_columns(tg, n, dtype):
    h.check_norm(tg, 5, n, dtype)
    h.check_norm_backward(tg, 5, n, dtype)


@pytest.mark.parametrize("m", [1, 2, 3, 127, 1000, 3001])
@pytest.mark.parametrize("n", [96, 1024, 5000])
def test_norm_rows(tg, m, n):
    h.check_norm(tg, m, n, "bf16")
    h.check_norm_backward(tg, m, n, "f32")


@pytest.mark.parametrize("pad,skew", [(8, 0), (1, 0), (3, 1), (0, 1)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_strides(tg, pad, skew, dtype):
    for n in (33, 1001, 9000):
        h.check_norm(tg, 40, n, dtype, pad=pad, skew=skew)
        h.check_norm_backward(tg, 40, n, dtype, pad=pad, skew=skew)


def test_norm_optional_parts(tg):
    h.check_norm(tg, 20, 300, "fp16", affine=False, save=False)
    for want in ((True, False, False), (False, True, False), (False, False, True), (True, False, True)):
        h.check_norm_backward(tg, 200, 300, "fp16", affine=False, want=want)


def test_norm_large_mean_and_constant_rows(tg):
    h.check_norm(tg, 30, 2000, "f32", scale=1.0, shift=300.0)
    x = h.Rows(4, 100, "f32", fill=torch.full((4, 100), 3.0, device="cuda"))
    y = h.Rows(4, 100, "f32")
    h.done(tg, tg.tg_layer_norm(4, 100, x, x.ld, None, None, 1e-5, y, y.ld, None, None, "f32",
                                torch.cuda.current_stream()), "constant rows")
    assert (y.t == 0).all()


def test_norm_backward_without_rows_gives_zero_sums(tg):
    dga = torch.full((50,), 7.0, device="cuda")
    dbe = torch.full((50,), 7.0, device="cuda")
    h.done(tg, tg.tg_layer_norm_backward(0, 50, None, 50, None, 50, None, None, None, None, 50, dga,
                                         dbe, "f32", None, torch.cuda.current_stream()), "no rows")
    assert (dga == 0).all() and (dbe == 0).all()


def test_norm_nan_stays_in_its_row(tg):
    g = h.gen(9)
    x = h.rows(g, 6, 700, "bf16")
    x.t[3, 11] = float("nan")
    y = h.Rows(6, 700, "bf16")
    h.done(tg, tg.tg_layer_norm(6, 700, x, x.ld, None, None, 1e-5, y, y.ld, None, None, "bf16",
                                torch.cuda.current_stream()), "NaN row")
    assert torch.isnan(y.t[3]).all()
    assert torch.isfinite(y.t[[0, 1, 2, 4, 5]]).all()


def test_norm_in_place(tg):
    g = h.gen(10)
    for n in (100, 1001, 5000, 12000):
        x = h.rows(g, 37, n, "bf16")
        wm, wr = h.norm_stats(x.d(), 1e-5)
        want = (x.d() - wm) * wr
        h.done(tg, tg.tg_layer_norm(37, n, x, x.ld, None, None, 1e-5, x, x.ld, None, None, "bf16",
                                    torch.cuda.current_stream()), "in place")
        h.check(x.t, want, h.rounded("bf16", want, 1e-5 * (1 + want.abs())), f"in place {n}")


def test_repeated_calls_agree_bit_for_bit(tg):
    """No atomics and fixed orders of summation, split reductions included."""
    a = [h.check_linear(tg, 30, 700, 4096, "bf16", "silu", bias=True).t.clone() for _ in range(3)]
    b = [h.check_linear(tg, 300, 300, 4096, "bf16").t.clone() for _ in range(3)]
    c = [[t.t.clone() if hasattr(t, "t") and not torch.is_tensor(t) else t.clone()
          for t in h.check_linear_backward(tg, 2000, 300, 200, "bf16", "gelu_tanh")] for _ in range(3)]
    for run in (a, b):
        assert all(torch.equal(run[0], r) for r in run[1:])
    for r in c[1:]:
        assert all(torch.equal(p, q) for p, q in zip(c[0], r))


def test_another_stream(tg):
    """Work queued on a stream of its own, with the inputs made there."""
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        for m in (4, 300):
            h.check_linear(tg, m, 520, 2048, "bf16", "silu", bias=True, residual=True)
            h.check_gated(tg, m, 520, 256, "bf16")
            h.check_linear_backward(tg, m, 264, 136, "bf16", "silu")
            h.check_norm_backward(tg, m, 777, "bf16")
    torch.cuda.current_stream().wait_stream(s)


def test_graph_capture(tg):
    """After one call on the stream, a whole forward and backward chain can be
    captured and replayed on new inputs."""
    g = h.gen(11)
    m, n, k = 200, 264, 136
    x, w = h.rows(g, m, k, "bf16"), h.rows(g, n, k, "bf16", scale=0.1)
    y, dx, dw = h.Rows(m, n, "bf16"), h.Rows(m, k, "bf16"), h.Rows(n, k, "bf16")
    ws = h.space(tg.tg_linear_backward_workspace_bytes(m, n, k, y, y.ld, x, x.ld, w, w.ld, "none", "bf16"))
    s = torch.cuda.Stream()

    def chain():
        tg.check(tg.tg_linear(m, n, k, x, x.ld, w, w.ld, None, "relu", None, 0, y, y.ld, None, 0,
                              "bf16", None, s))
        tg.check(tg.tg_linear_backward(m, n, k, y, y.ld, x, x.ld, w, w.ld, None, 0, "none", dx, dx.ld,
                                       dw, dw.ld, "bf16", None, "bf16", ws, s))

    with torch.cuda.stream(s):
        chain()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        chain()
    x.t.copy_(h.rows(g, m, k, "bf16").t)
    graph.replay()
    torch.cuda.synchronize()
    want, ye, _, _ = h.ref_linear(x, w, None, "relu", None, "bf16")
    h.check(y.t, want, ye, "replayed Y")
    v = y.d() @ w.d()
    h.check(dx.t, v, h.rounded("bf16", v, h.product_error(n, y.d().abs() @ w.d().abs())), "replayed dX")


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_gradients_against_differences(tg, act):
    """The formulas' gradients against central differences of the FP64
    forward: directional derivatives of sum(dY * Y) along random directions
    agree to the operators' 16-bit rounding."""
    g = h.gen(12)
    m, n, k, t = 24, 40, 32, 1e-4
    x, w = h.rows(g, m, k, "fp16"), h.rows(g, n, k, "fp16", scale=0.2)
    dy = h.rows(g, m, n, "fp16")
    _, z = h.run_linear(tg, x, w, None, act, None, "fp16", save=True)
    dx, dw = h.Rows(m, k, "fp16"), h.Rows(n, k, "fp16")
    ws = h.space(tg.tg_linear_backward_workspace_bytes(m, n, k, dy, dy.ld, x, x.ld, w, w.ld, act, "fp16"))
    h.done(tg, tg.tg_linear_backward(m, n, k, dy, dy.ld, x, x.ld, w, w.ld, z, z.ld, act, dx, dx.ld, dw,
                                     dw.ld, "fp16", None, "fp16", ws, torch.cuda.current_stream()), "backward")
    vx = torch.randn(m, k, generator=g, device="cuda").double()
    vw = torch.randn(n, k, generator=g, device="cuda").double()

    def loss(a, b):
        return float((dy.d() * h.act64(act, a @ b.t())).sum())

    for got, along, f in ((dx, vx, lambda e: loss(x.d() + e * vx, w.d())),
                          (dw, vw, lambda e: loss(x.d(), w.d() + e * vw))):
        want = (f(t) - f(-t)) / (2 * t)
        size = float((got.d() * along).abs().sum())
        # Three roundings to FP16 (Z, dZ, the gradient), each 2^-11 of a term.
        assert abs(float((got.d() * along).sum()) - want) <= 4 * 2.0 ** -11 * size + 1e-6


def test_norm_gradient_against_differences(tg):
    g = h.gen(13)
    m, n, t = 6, 50, 1e-5
    x, dy = h.rows(g, m, n, "f32"), h.rows(g, m, n, "f32")
    ga = 1 + 0.3 * torch.randn(n, generator=g, device="cuda")
    y = h.Rows(m, n, "f32")
    mean, rstd = torch.empty(m, device="cuda"), torch.empty(m, device="cuda")
    st = torch.cuda.current_stream()
    h.done(tg, tg.tg_layer_norm(m, n, x, x.ld, ga, None, 1e-5, y, y.ld, mean, rstd, "f32", st), "forward")
    dx, dga = h.Rows(m, n, "f32"), torch.empty(n, device="cuda")
    ws = h.space(tg.tg_layer_norm_backward_workspace_bytes(m, n))
    h.done(tg, tg.tg_layer_norm_backward(m, n, dy, dy.ld, x, x.ld, ga, mean, rstd, dx, dx.ld, dga, None,
                                         "f32", ws, st), "backward")
    vx = torch.randn(m, n, generator=g, device="cuda").double()
    vg = torch.randn(n, generator=g, device="cuda").double()

    def loss(a, b):
        mu, r = h.norm_stats(a, 1e-5)
        return float((dy.d() * (a - mu) * r * b).sum())

    for got, along, f in ((dx.d(), vx, lambda e: loss(x.d() + e * vx, ga.double())),
                          (dga.double(), vg, lambda e: loss(x.d(), ga.double() + e * vg))):
        want = (f(t) - f(-t)) / (2 * t)
        assert abs(float((got * along).sum()) - want) <= 1e-5 * float((got * along).abs().sum()) + 1e-7


# Aligned rows (ld a multiple of 8) whose last box ends inside 16 bytes.
@pytest.mark.parametrize("n", [1, 3, 65, 71, 193, 1001])
def test_ragged_columns_on_aligned_rows(tg, n):
    pad = -n % 8
    h.check_linear(tg, 200, n, 64, "bf16", "silu", bias=True, residual=True, save=True, pad=0,
                   opad=pad + 8, oskew=0)
    h.check_linear(tg, 200, n, 64, "bf16", "silu", opad=pad, oskew=0)
    h.check_linear_backward(tg, 64, 72, n, "fp16", pad=pad)
    h.check_linear_backward(tg, 64, 72, n, "fp16", pad=-n % 4, dw="f32")
    h.check_gated(tg, 150, n, 64, "bf16", save=True, pad=0)


def test_offsets_beyond_32_bits(tg):
    """Outputs, residuals and inputs whose element offsets pass 2^31."""
    m, n, k, ld = 70000, 72, 64, 33000
    g = h.gen(14)
    st = torch.cuda.current_stream()
    wide = torch.empty(m, ld, dtype=torch.bfloat16, device="cuda")  # 4.6 GB
    x = torch.randn(m, k, generator=g, device="cuda").to(torch.bfloat16)
    w = h.rows(g, n, k, "bf16", scale=0.1)
    y = wide[:, 100:100 + n]
    y.copy_(torch.randn(m, n, generator=g, device="cuda"))
    r = y[-300:].double()
    h.done(tg, tg.tg_linear(m, n, k, x, k, w, w.ld, None, "none", y, ld, y, ld, None, 0, "bf16", None,
                            st), "wide rows")
    want = x[-300:].double() @ w.d().t() + r
    e = h.product_error(k, x[-300:].double().abs() @ w.d().abs().t()) + 2.0 ** -23 * want.abs()
    h.check(y[-300:], want, h.rounded("bf16", want, e), "rows beyond 2^31 elements")
    x = wide[:, :512]
    x.copy_(torch.randn(m, 512, generator=g, device="cuda"))
    out = torch.empty(m, 512, dtype=torch.bfloat16, device="cuda")
    h.done(tg, tg.tg_layer_norm(m, 512, x, ld, None, None, 1e-5, out, 512, None, None, "bf16", st), "norm")
    mean, rstd = h.norm_stats(x[-300:].double(), 1e-5)
    want = (x[-300:].double() - mean) * rstd
    h.check(out[-300:], want, h.rounded("bf16", want, 1e-5 * (1 + want.abs())), "norm beyond 2^31 elements")
    # The backward pass reads dY there too (and repacks X's odd rows).
    dx = torch.empty(m, k, dtype=torch.bfloat16, device="cuda")
    db = torch.empty(n, device="cuda")
    ws = h.space(tg.tg_linear_backward_workspace_bytes(m, n, k, y, ld, wide[:, 1:], ld, w, w.ld, "none", "bf16"))
    h.done(tg, tg.tg_linear_backward(m, n, k, y, ld, None, k, w, w.ld, None, 0, "none", dx, k, None, k,
                                     "bf16", db, "bf16", ws, st), "backward")
    want = y[-300:].double() @ w.d()
    e = h.product_error(n, y[-300:].double().abs() @ w.d().abs())
    h.check(dx[-300:], want, h.rounded("bf16", want, e), "dX beyond 2^31 elements")
    s = y.double()
    h.check(db, s.sum(0), m * 2.0 ** -24 * s.abs().sum(0), "db over all rows")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("m", [1, 5, 16, 33, 64, 100, 128])
def test_input_gradients_of_few_tokens(tg, m, dtype):
    """Transposed weights through the streaming kernel, long reductions cut
    into shares, one and two operand pairs."""
    h.check_linear_backward(tg, m, 2000, 300, dtype, "silu", want_dw=False, bias=False)
    h.check_gated_backward(tg, m, 1000, 520, dtype, want=(True, False, False))


@pytest.mark.parametrize("ld_pad", range(8))
def test_every_row_alignment(tg, ld_pad):
    """Row strides and bases of every residue modulo 16 bytes."""
    for skew in range(8):
        h.check_linear(tg, 40, 70, 150, "bf16", bias=True, residual=True, save=True, pad=ld_pad, skew=skew)
        h.check_linear_backward(tg, 33, 70, 150, "fp16", "relu", pad=ld_pad, skew=skew)
        h.check_linear(tg, 140, 70, 24, "bf16", residual=True, pad=ld_pad, skew=skew)

"""Calls of the attention operators that their header allows and that no workload makes:
no keys at all, bounds left out, generous or too small, many sequences, one head with any
head stride, rows past 32-bit offsets, one workspace for calls in turn."""

from __future__ import annotations

import copy

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


def forward(tg, p, o, z, ws, st, max_q=None, max_k=None, q=None, k=None, v=None):
    tg.check(tg.tg_attention(*p.sizes(), *(q or p.Q.lay), *(k or p.K.lay), *(v or p.V.lay), *p.arrays(),
                             p.max_q if max_q is None else max_q, p.max_k if max_k is None else max_k, p.causal,
                             p.scale, *o, z, p.dtype, ws, st), "tg_attention")


def forward_space(tg, p):
    return ah.space(tg.tg_attention_workspace_bytes(*p.sizes(), p.max_q, p.max_k, p.dtype))


def backward_space(tg, p):
    return ah.space(tg.tg_attention_backward_workspace_bytes(*p.sizes(), p.max_q, p.max_k, p.dtype))


def device_ok(tg, st):
    status, where = tg.tg_check_device_status(st)
    tg.check(status, f"device status (wait site {where})")


@pytest.mark.parametrize("causal", [True, False])
def test_no_keys_at_all(tg, causal):
    """k_rows = 0, K and V NULL: zeros, LSE of -infinity, and zeros for dQ."""
    p = ah.Problem([200, 0, 3], [0, 0, 0], heads=4, kv=2, dim=72, causal=causal)
    st = torch.cuda.current_stream()
    o, z = ah.Tensor3(203, 4, 72, "bf16"), torch.full((4, 203), float("nan"), device="cuda")
    forward(tg, p, o.lay, z, forward_space(tg, p), st, k=(None, 0, 0), v=(None, 0, 0))
    device_ok(tg, st)
    assert bool((o.t == 0).all()) and bool((z == -float("inf")).all())
    dq = ah.Tensor3(203, 4, 72, "bf16")
    nothing = (None, 0, 0)
    tg.check(tg.tg_attention_backward(*p.sizes(), *p.Q.lay, *nothing, *nothing, *o.lay, *p.dO.lay, z, *p.arrays(),
                                      p.max_q, p.max_k, causal, p.scale, *dq.lay, *nothing, *nothing, "bf16",
                                      backward_space(tg, p), st), "tg_attention_backward")
    device_ok(tg, st)
    assert bool((dq.t == 0).all())


@pytest.mark.parametrize("max_q,max_k", [(0, 0), (700, 1500), (1 << 40, 1 << 40)])
def test_bounds_left_out_or_generous(tg, max_q, max_k):
    """(The plans differ from those by the lengths; the results stay within the bounds.)"""
    for q_len, k_len in (([1] * 5, [900, 1, 0, 130, 400]), ([300, 7, 129], [300, 64, 700])):
        p = ah.Problem(q_len, k_len, heads=4, kv=2, dim=64)
        p.max_q, p.max_k = max_q, max_k
        ah.check_forward(tg, p)
        ah.check_backward(tg, p)


def test_sequences_longer_than_the_bounds_are_cut(tg):
    p = ah.Problem([300, 40, 129], [260, 40, 300], heads=4, kv=2, dim=64, lengths=True)
    p.max_q, p.max_k = 130, 100
    cut = copy.copy(p)
    cut.q_len, cut.k_len = [130, 40, 129], [100, 40, 100]
    o, z = ah.run_forward(tg, p)
    want, eo, lse, el = ah.reference(cut)
    rows = cut.rows()
    ah.check(o.t[rows], want[rows], eo[rows], "O")
    ah.check(z[:, rows], lse[:, rows], el[:, rows], "LSE")
    assert o.kept_outside(rows) and bool(torch.isnan(z[:, ~rows]).all())
    given, lse = ah.given(cut)
    want = ah.reference_backward(cut, given, lse)
    for name, got in ah.run_backward(tg, p, given, lse).items():
        rows = cut.rows(keys=name != "dQ")
        ah.check(got.t[rows], want[name][0][rows], want[name][1][rows], name)
        assert got.kept_outside(rows), name


@pytest.mark.parametrize("causal", [True, False])
def test_many_sequences(tg, causal):
    """More than a warp looks at at once, empty ones among them."""
    g = torch.Generator().manual_seed(3)
    q_len = [int(n) for n in torch.randint(0, 200, (75,), generator=g)]
    k_len = [int(n) for n in torch.randint(0, 300, (75,), generator=g)]
    for i in (0, 31, 32, 33, 63, 64, 74):
        q_len[i] = 0
    p = ah.Problem(q_len, k_len, heads=4, kv=2, dim=64, causal=causal)
    ah.check_forward(tg, p)
    ah.check_backward(tg, p)


def test_one_head_with_any_head_stride(tg):
    """(hd is not looked at.)"""
    p = ah.Problem([150, 33], heads=1, kv=1, dim=64)
    want, z = ah.run_forward(tg, p)
    st = torch.cuda.current_stream()
    for hd in (0, -8, 3, 1 << 62):
        o, y = ah.Tensor3(183, 1, 64, "bf16"), torch.empty(1, 183, device="cuda")
        lay = [(x, x.ld, hd) for x in (p.Q, p.K, p.V, o)]
        forward(tg, p, lay[3], y, forward_space(tg, p), st, q=lay[0], k=lay[1], v=lay[2])
        assert torch.equal(o.t, want.t) and torch.equal(y, z), hd


def test_without_lse(tg):
    for p in (ah.Problem([150, 33], heads=4, kv=2, dim=64), ah.Problem([1] * 4, [900, 3000, 1, 2000], heads=8, kv=2)):
        want, _ = ah.run_forward(tg, p)
        got, _ = ah.run_forward(tg, p, lse=False)
        assert torch.equal(got.t, want.t)


class Wide:
    """Heads of 64 whose rows are 2^21 elements apart, at element `at` of each row."""

    LD = 1 << 21

    def __init__(self, buf, at, rows, heads, fill=None):
        self.t = torch.as_strided(buf, (rows, heads, 64), (self.LD, 64, 1), at)
        self.lay = (self.t, self.LD, 64)
        if fill is not None:
            self.t.copy_(fill)


@pytest.fixture
def wide_rows():
    buf = torch.zeros(1100 * Wide.LD // 4 + 4096, 4, dtype=torch.bfloat16, device="cuda").view(-1)
    yield buf
    del buf
    torch.cuda.empty_cache()


def test_gradients_past_32_bit_offsets(tg, wide_rows):
    """The bits that narrow rows give."""
    p = ah.Problem([450, 600], [500, 600], heads=4, kv=2, dim=64)
    given, lse = ah.given(p)
    want = ah.run_backward(tg, p, given, lse)
    q, o, dy = (Wide(wide_rows, 1024 * i, 1050, 4, x.t) for i, x in enumerate((p.Q, given, p.dO)))
    k, v = (Wide(wide_rows, 4096 + 1024 * i, 1100, 2, x.t) for i, x in enumerate((p.K, p.V)))
    out = {"dQ": Wide(wide_rows, 8192, 1050, 4), "dK": Wide(wide_rows, 9216, 1100, 2),
           "dV": Wide(wide_rows, 10240, 1100, 2)}
    st = torch.cuda.current_stream()
    tg.check(tg.tg_attention_backward(*p.sizes(), *q.lay, *k.lay, *v.lay, *o.lay, *dy.lay, lse, *p.arrays(), p.max_q,
                                      p.max_k, p.causal, p.scale, *out["dQ"].lay, *out["dK"].lay, *out["dV"].lay,
                                      p.dtype, backward_space(tg, p), st), "tg_attention_backward")
    device_ok(tg, st)
    for n in out:
        assert torch.equal(out[n].t, want[n].t), n


def test_rotary_past_32_bit_offsets(tg, wide_rows):
    st = torch.cuda.current_stream()
    steps = torch.tensor(tg.tg_rotary_steps(64, 10000.0), dtype=torch.int64, device="cuda")
    x = torch.randn(1100, 3, 64, generator=ah.gen(4), device="cuda").to(torch.bfloat16)
    want, a, b = torch.empty_like(x), Wide(wide_rows, 0, 1100, 3, x), Wide(wide_rows, 512, 1100, 3)
    to = torch.arange(1099, -1, -1, device="cuda")
    tg.check(tg.tg_rotary(1100, 3, 64, 64, x, 192, 64, want, 192, 64, 0, None, None, steps, "halves", 1.0, "bf16",
                          st), "tg_rotary")
    tg.check(tg.tg_rotary(1100, 3, 64, 64, *a.lay, *b.lay, 0, None, None, steps, "halves", 1.0, "bf16", st),
             "tg_rotary")
    assert torch.equal(b.t, want)
    tg.check(tg.tg_rotary(1100, 3, 64, 64, *a.lay, *b.lay, 1100, None, to, steps, "halves", 1.0, "bf16", st),
             "tg_rotary")
    assert torch.equal(b.t, want.flip(0))


def test_one_workspace_in_turn(tg):
    """Calls behind one another on a stream, and two captured graphs replayed in turn, share
    a workspace."""
    a = ah.Problem([1] * 4, [900, 3000, 1, 2000], heads=8, kv=2, dim=128, seed=5)
    b = ah.Problem([1300], heads=4, kv=1, dim=64, dtype="fp16", scale=0.05, seed=6)
    want_a, want_z = ah.run_forward(tg, a)
    given, lse = ah.given(b)
    want_b = ah.run_backward(tg, b, given, lse)
    n = max(tg.tg_attention_workspace_bytes(*a.sizes(), a.max_q, a.max_k, a.dtype),
            tg.tg_attention_backward_workspace_bytes(*b.sizes(), b.max_q, b.max_k, b.dtype))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    o, z = ah.Tensor3(4, 8, 128, "bf16"), torch.empty(8, 4, device="cuda")
    out = {"dQ": ah.Tensor3(1300, 4, 64, "fp16"), "dK": ah.Tensor3(1300, 1, 64, "fp16"),
           "dV": ah.Tensor3(1300, 1, 64, "fp16")}

    def run_a(st):
        forward(tg, a, o.lay, z, ws, st)

    def run_b(st):
        lay = [x for k in ("dQ", "dK", "dV") for x in out[k].lay]
        tg.check(tg.tg_attention_backward(*b.sizes(), *b.Q.lay, *b.K.lay, *b.V.lay, *given.lay, *b.dO.lay, lse,
                                          *b.arrays(), b.max_q, b.max_k, b.causal, b.scale, *lay, b.dtype, ws, st),
                 "tg_attention_backward")

    def same():
        torch.cuda.synchronize()
        assert torch.equal(o.t, want_a.t) and torch.equal(z, want_z)
        assert all(torch.equal(out[k].t, want_b[k].t) for k in out)
        for x in (o.t, z, *(v.t for v in out.values())):
            x.fill_(float("nan"))

    st = torch.cuda.current_stream()
    for _ in range(5):
        run_a(st)
        run_b(st)
    same()
    graphs, side = [], torch.cuda.Stream()
    for f in (run_a, run_b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            f(side)
        graphs.append(g)
    for _ in range(5):
        for g in graphs:
            g.replay()
    same()

"""The feed-forward operators where kernels overlap: the weight gradient beside
the input gradient, after row-wise work that both read.

(References and bounds as in mlp_harness.py.)"""

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


class Backward:
    """A linear layer's backward pass on rows that need repacking (pad odd) or
    not, its workspace and outputs."""

    def __init__(self, tg, m, n, k, dtype, pad=0, dw="same", seed=21):
        self.tg, self.m, self.n, self.k, self.dtype = tg, m, n, k, dtype
        self.dwt = dtype if dw == "same" else dw
        g = h.gen(seed + m + n + k)
        self.x, self.dy = h.rows(g, m, k, dtype, pad), h.rows(g, m, n, dtype, pad)
        self.w = h.rows(g, n, k, dtype, pad, 0, 1 / math.sqrt(k))
        self.z = h.rows(g, m, n, dtype, pad, 0, 1.5)
        self.ws = h.space(tg.tg_linear_backward_workspace_bytes(
            m, n, k, self.dy, self.dy.ld, self.x, self.x.ld, self.w, self.w.ld, "silu", dtype))
        self.new_outputs()

    def new_outputs(self):
        self.dx = h.Rows(self.m, self.k, self.dtype)
        self.dw = h.Rows(self.n, self.k, self.dwt)
        self.db = torch.full((self.n,), float("nan"), device="cuda")

    def outputs(self):
        return [self.dx.t, self.dw.t, self.db]

    def poison(self):
        """All bits set: NaN wherever a product reads too early."""
        self.ws.fill_(255)
        for t in self.outputs():
            t.fill_(float("nan"))

    def run(self, stream=None):
        o = self
        o.tg.check(o.tg.tg_linear_backward(
            o.m, o.n, o.k, o.dy, o.dy.ld, o.x, o.x.ld, o.w, o.w.ld, o.z, o.z.ld, "silu", o.dx, o.dx.ld,
            o.dw, o.dw.ld, o.dwt, o.db, o.dtype, o.ws, stream or torch.cuda.current_stream()))

    def check(self, what):
        dz = self.dy.d() * h.act_grad64("silu", self.z.d())
        e32 = h.FN * h.SLOPE * self.dy.d().abs()
        e = h.rounded(self.dtype, dz, e32)
        v, s = dz @ self.w.d(), dz.abs() @ self.w.d().abs()
        h.check(self.dx.t, v, h.rounded(self.dtype, v, h.product_error(self.n, s) + e @ self.w.d().abs()),
                what + " dX")
        v, s = dz.t() @ self.x.d(), dz.abs().t() @ self.x.d().abs()
        h.check(self.dw.t, v, h.rounded(self.dwt, v, h.product_error(self.m, s) + e.t() @ self.x.d().abs()),
                what + " dW")
        h.check(self.db, dz.sum(0), (self.m * 2.0 ** -24) * dz.abs().sum(0) + e32.sum(0) + 1e-30, what + " db")


# (400, 16384, 24): the row-wise launch moves 40 MB and more, each product a few
# hundred KB beside it; (9, 20000, 40), (100, 5000, 136): the streaming input
# gradient; (777, 1001, 1365): tiles of both products on the SMs at once.
@pytest.mark.parametrize("m,n,k,pad", [(400, 16384, 24, 0), (400, 16384, 24, 1), (9, 20000, 40, 0),
                                       (100, 5000, 136, 1), (777, 1001, 1365, 0), (300, 264, 136, 3)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_gradients_after_long_row_work(tg, m, n, k, pad, dtype):
    """Calls back to back, workspace and outputs set to NaN before each: what a
    product read before the row-wise kernel had written it would show."""
    b = Backward(tg, m, n, k, dtype, pad)
    kept = []
    for _ in range(8):
        b.poison()
        b.run()
        kept.append([t.clone() for t in b.outputs()])
    st, where = tg.tg_check_device_status(torch.cuda.current_stream())
    tg.check(st, f"wait site {where}")
    b.check(f"backward {m}x{n}x{k}")
    for other in kept[:-1]:
        assert all(torch.equal(p, q) for p, q in zip(kept[-1], other))


def test_graph_replays_the_whole_backward(tg):
    """Every output of a captured forward and backward chain, from NaN-filled
    outputs and workspace, on new inputs, twice; the second weight gradient is
    one that runs beside its input gradient."""
    b = Backward(tg, 200, 264, 136, "bf16", pad=1)
    assert tg.tg_product_plan_describe("linear_dw", 200, 264, 136).endswith("beside=1")
    y = h.Rows(200, 264, "bf16")
    ws = h.space(tg.tg_linear_workspace_bytes(200, 264, 136, b.x, b.x.ld, b.w, b.w.ld, "bf16"))
    s = torch.cuda.Stream()

    def chain():
        tg.check(tg.tg_linear(200, 264, 136, b.x, b.x.ld, b.w, b.w.ld, None, "silu", None, 0, y, y.ld,
                              b.z, b.z.ld, "bf16", ws, s))
        b.run(s)

    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        chain()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        chain()
    for seed in (31, 32):
        g = h.gen(seed)
        for m in (b.x, b.dy, b.w):
            m.t.copy_(torch.randn(m.rows, m.cols, generator=g, device="cuda") * (0.1 if m is b.w else 1.0))
        b.poison()
        for t in (y.t, b.z.t, ws):
            t.fill_(float("nan") if t.is_floating_point() else 255)
        graph.replay()
        torch.cuda.synchronize()
        want, ye, wz, ze = h.ref_linear(b.x, b.w, None, "silu", None, "bf16")
        h.check(y.t, want, ye, "replayed Y")
        h.check(b.z.t, wz, ze, "replayed Z")
        b.check("replayed")
        assert all(m.padding_kept() for m in (y, b.z, b.dx, b.dw))


def test_capture_on_a_stream_without_a_workspace(tg):
    """A backward call that splits no tile needs no library workspace: it can be
    captured on a stream that has made no call before (its kernels have run
    elsewhere), as graph helpers with a stream of their own do."""
    b = Backward(tg, 200, 264, 136, "bf16")
    for p in ("linear_dx", "linear_dw"):
        assert " split=0x1 schedule=static " in tg.tg_product_plan_describe(p, 200, 264, 136)
    b.run()
    torch.cuda.synchronize()
    s = torch.cuda.Stream(priority=-1)  # (of a pool that no other test takes from)
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        b.run(s)
    for _ in range(2):
        b.poison()
        graph.replay()
        torch.cuda.synchronize()
        b.check("captured on a fresh stream")


class StreamWork:
    """Calls of one host thread on a stream of its own (torch's current stream is
    the thread's, so each method enters it)."""

    def __init__(self, tg, seed):
        self.tg, self.stream, self.out = tg, torch.cuda.Stream(), []
        with torch.cuda.stream(self.stream):
            self.back = [Backward(tg, *size, seed=seed) for size in
                         ((200, 264, 136, "bf16"), (90, 1000, 520, "fp16", 1), (777, 1001, 1365, "fp16"))]
            g = h.gen(seed)
            self.forward = []
            for m, n, k in ((20, 300, 6000), (300, 300, 4096), (1500, 1000, 2048)):
                self.forward.append((h.rows(g, m, k, "bf16"), h.rows(g, n, k, "bf16", scale=0.02),
                                     h.Rows(m, n, "bf16")))
        self.stream.synchronize()

    def run(self):
        tg, st = self.tg, self.stream
        with torch.cuda.stream(st):
            for _ in range(20):
                for x, w, y in self.forward:
                    y.t.fill_(float("nan"))
                    tg.check(tg.tg_linear(x.rows, w.rows, x.cols, x, x.ld, w, w.ld, None, "none", None, 0,
                                          y, y.ld, None, 0, "bf16", None, st))
                    self.out.append(y.t.clone())
                for b in self.back:
                    b.poison()
                    b.run(st)
                    self.out += [t.clone() for t in b.outputs()]
        st.synchronize()


def test_two_streams_at_once(tg):
    """Two host threads, each with a stream, enqueue split, streaming and
    backward calls; results equal those of the same calls alone, bit for bit
    (flags, tickets, partial sums and the gate belong to a stream)."""
    import threading

    alone = [StreamWork(tg, seed) for seed in (41, 42)]
    for w in alone:
        w.run()
    both = [StreamWork(tg, seed) for seed in (41, 42)]
    threads = [threading.Thread(target=w.run) for w in both]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    st, where = tg.tg_check_device_status(torch.cuda.current_stream())
    tg.check(st, f"wait site {where}")
    for a, b in zip(alone, both):
        assert len(a.out) == len(b.out) == 240 and all(torch.equal(p, q) for p, q in zip(a.out, b.out))


GUARD = 8192


class Guarded:
    """A workspace of exactly the queried size, with sentinel bytes after it."""

    def __init__(self, nbytes):
        assert nbytes >= 0
        self.n = nbytes
        self.buf = torch.full((nbytes + GUARD,), 0x5A, dtype=torch.uint8, device="cuda")

    def arg(self):
        return self.buf.data_ptr(), self.n

    def check(self, what):
        assert (self.buf[self.n:] == 0x5A).all(), what


@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (3, 65, 33), (40, 70, 150), (129, 257, 65), (300, 93, 201),
                                   (777, 1001, 1365)])
@pytest.mark.parametrize("pad", [0, 1])
def test_workspaces_are_not_overrun(tg, m, n, k, pad):
    g = h.gen(51 + m)
    st = torch.cuda.current_stream()
    x, w, w2 = h.rows(g, m, k, "bf16", pad), h.rows(g, n, k, "bf16", pad), h.rows(g, n, k, "bf16", pad)
    a, b, c = (h.rows(g, m, n, "bf16", pad) for _ in range(3))
    y, dx, dw, dw2 = h.Rows(m, n, "bf16"), h.Rows(m, k, "bf16"), h.Rows(n, k, "f32"), h.Rows(n, k, "f32")
    db = torch.empty(n, device="cuda")
    s = Guarded(tg.tg_linear_workspace_bytes(m, n, k, x, x.ld, w, w.ld, "bf16"))
    h.done(tg, tg.tg_linear(m, n, k, x, x.ld, w, w.ld, None, "silu", None, 0, y, y.ld, None, 0, "bf16",
                            s.arg(), st), "linear")
    s.check("tg_linear")
    s = Guarded(tg.tg_gated_workspace_bytes(m, n, k, x, x.ld, w, w.ld, w2, w2.ld, "bf16"))
    h.done(tg, tg.tg_gated(m, n, k, x, x.ld, w, w.ld, w2, w2.ld, "silu", y, y.ld, None, 0, None, 0, "bf16",
                           s.arg(), st), "gated")
    s.check("tg_gated")
    for act in ("none", "silu"):
        s = Guarded(tg.tg_linear_backward_workspace_bytes(m, n, k, a, a.ld, x, x.ld, w, w.ld, act, "bf16"))
        h.done(tg, tg.tg_linear_backward(m, n, k, a, a.ld, x, x.ld, w, w.ld, b, b.ld, act, dx, dx.ld, dw,
                                         dw.ld, "f32", db, "bf16", s.arg(), st), "linear_backward")
        s.check("tg_linear_backward")
    s = Guarded(tg.tg_gated_backward_workspace_bytes(m, n, k, x, x.ld, w, w.ld, w2, w2.ld, "bf16"))
    h.done(tg, tg.tg_gated_backward(m, n, k, a, a.ld, x, x.ld, w, w.ld, w2, w2.ld, b, b.ld, c, c.ld, "silu",
                                    dx, dx.ld, dw, dw.ld, dw2, dw2.ld, "f32", "bf16", s.arg(), st),
           "gated_backward")
    s.check("tg_gated_backward")
    xn = x.t.float().contiguous()
    mean, rstd = (t.float().contiguous() for t in h.norm_stats(xn.double(), 1e-5))
    dn, dga, dbe = torch.empty_like(xn), torch.empty(k, device="cuda"), torch.empty(k, device="cuda")
    s = Guarded(tg.tg_layer_norm_backward_workspace_bytes(m, k))
    h.done(tg, tg.tg_layer_norm_backward(m, k, xn, k, xn, k, None, mean, rstd, dn, k, dga, dbe, "f32",
                                         s.arg(), st), "norm_backward")
    s.check("tg_layer_norm_backward")

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

"""A transformer block's feed-forward half on the library's operators, forward
and backward:

    y = x + W2 (silu(Wg n) * (Wu n)) + b2,   n = layer_norm(x; gamma, beta)

as the calls tg_layer_norm, tg_gated and tg_linear (with the residual added in
its epilogue), and their backward calls in reverse.  Weights are BF16 with FP32
vectors; `FeedForward.step` is one training step (plain SGD on FP32 copies of
the weights), `FeedForward.forward` alone serves, one token or many.

    python examples/feed_forward.py [tokens] [features] [hidden] [steps]

trains the block to reproduce a random teacher block of the same shape and
prints the loss, then the time of one decoded token.
"""

from __future__ import annotations

import math
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import dense_gemm_epilogue_gb300 as tg  # noqa: E402

EPS = 1e-5
BF16 = torch.bfloat16


def _space(nbytes: int):
    if nbytes < 0:
        raise RuntimeError("workspace query failed")
    return torch.empty(nbytes, dtype=torch.uint8, device="cuda") if nbytes else None


class FeedForward:
    """Parameters, the forward pass's saved tensors and the gradients."""

    def __init__(self, features: int, hidden: int, seed: int = 0, scale: float = 1.0):
        self.d, self.f = features, hidden
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def weight(rows, cols):
            w = torch.randn(rows, cols, generator=g, device="cuda") * (scale / math.sqrt(cols))
            return w  # FP32 master copy

        self.master = {
            "Wg": weight(hidden, features), "Wu": weight(hidden, features),
            "W2": weight(features, hidden), "b2": torch.zeros(features, device="cuda"),
            "gamma": torch.ones(features, device="cuda"), "beta": torch.zeros(features, device="cuda"),
        }
        self.grads = {}
        self.refresh()

    def refresh(self):
        """The BF16 weights that the products read, from the master copies."""
        self.w = {k: (v.to(BF16) if v.dim() == 2 else v) for k, v in self.master.items()}

    def forward(self, x: torch.Tensor, train: bool = False) -> torch.Tensor:
        m, d, f, w = x.shape[0], self.d, self.f, self.w
        st = torch.cuda.current_stream()

        def new(rows, cols):
            return torch.empty(rows, cols, dtype=BF16, device="cuda")

        n, h, y = new(m, d), new(m, f), new(m, d)
        mean = torch.empty(m, device="cuda") if train else None
        rstd = torch.empty(m, device="cuda") if train else None
        g, u = (new(m, f), new(m, f)) if train else (None, None)
        tg.check(tg.tg_layer_norm(m, d, x, x.stride(0), w["gamma"], w["beta"], EPS, n, d, mean, rstd,
                                  "bf16", st), "tg_layer_norm")
        ws = _space(tg.tg_gated_workspace_bytes(m, f, d, n, d, w["Wg"], d, w["Wu"], d, "bf16"))
        tg.check(tg.tg_gated(m, f, d, n, d, w["Wg"], d, w["Wu"], d, "silu", h, f, g, f, u, f, "bf16",
                             ws, st), "tg_gated")
        ws = _space(tg.tg_linear_workspace_bytes(m, d, f, h, f, w["W2"], f, "bf16"))
        tg.check(tg.tg_linear(m, d, f, h, f, w["W2"], f, w["b2"], "none", x, x.stride(0), y, d, None, 0,
                              "bf16", ws, st), "tg_linear")
        if train:
            self.saved = (x, n, mean, rstd, g, u, h)
        return y

    def backward(self, dy: torch.Tensor) -> torch.Tensor:
        """Gradients of the parameters into ``grads``; returns dx."""
        x, n, mean, rstd, g, u, h = self.saved
        m, d, f, w = x.shape[0], self.d, self.f, self.w
        st = torch.cuda.current_stream()
        f32 = torch.float32

        def new(rows, cols, dtype=BF16):
            return torch.empty(rows, cols, dtype=dtype, device="cuda")

        gr = {"Wg": new(f, d, f32), "Wu": new(f, d, f32), "W2": new(d, f, f32),
              "b2": torch.empty(d, device="cuda"), "gamma": torch.empty(d, device="cuda"),
              "beta": torch.empty(d, device="cuda")}
        dh, dn, dx = new(m, f), new(m, d), new(m, d)
        ld = dy.stride(0)
        ws = _space(tg.tg_linear_backward_workspace_bytes(m, d, f, dy, ld, h, f, w["W2"], f, "none", "bf16"))
        tg.check(tg.tg_linear_backward(m, d, f, dy, ld, h, f, w["W2"], f, None, 0, "none", dh, f,
                                       gr["W2"], f, "f32", gr["b2"], "bf16", ws, st), "tg_linear_backward")
        ws = _space(tg.tg_gated_backward_workspace_bytes(m, f, d, n, d, w["Wg"], d, w["Wu"], d, "bf16"))
        tg.check(tg.tg_gated_backward(m, f, d, dh, f, n, d, w["Wg"], d, w["Wu"], d, g, f, u, f, "silu",
                                      dn, d, gr["Wg"], d, gr["Wu"], d, "f32", "bf16", ws, st),
                 "tg_gated_backward")
        ws = _space(tg.tg_layer_norm_backward_workspace_bytes(m, d))
        tg.check(tg.tg_layer_norm_backward(m, d, dn, d, x, x.stride(0), w["gamma"], mean, rstd, dx, d,
                                           gr["gamma"], gr["beta"], "bf16", ws, st),
                 "tg_layer_norm_backward")
        self.grads = gr
        return dx + dy  # the residual's share

    def step(self, x: torch.Tensor, target: torch.Tensor, rate: float) -> torch.Tensor:
        """One SGD step on the mean squared error; returns the loss (a device scalar)."""
        y = self.forward(x, train=True)
        diff = y.float() - target.float()
        self.backward((diff * (2.0 / diff.numel())).to(BF16))
        for k, v in self.grads.items():
            self.master[k].sub_(v, alpha=rate)
        self.refresh()
        return diff.square().mean()


def main(argv) -> None:
    m, d, f, steps = [int(v) for v in (argv + [0] * 4)[:4]]
    m, d, f, steps = m or 4096, d or 1024, f or 4096, steps or 20
    tg.build()
    tg.load()
    teacher = FeedForward(d, f, seed=1)
    student = FeedForward(d, f, seed=2, scale=0.5)
    x = torch.randn(m, d, device="cuda").to(BF16)
    target = teacher.forward(x)
    for i in range(steps):
        loss = student.step(x, target, rate=0.2 * d)
        print(f"step {i}: loss {float(loss):.5f}")
    st, where = tg.tg_check_device_status(torch.cuda.current_stream())
    tg.check(st, f"device status (wait site {where})")
    token = x[:1]
    for _ in range(3):
        student.forward(token)
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(100):
        student.forward(token)
    b.record()
    torch.cuda.synchronize()
    print(f"one token: {a.elapsed_time(b) * 10:.1f} us")


if __name__ == "__main__":
    main(sys.argv[1:])

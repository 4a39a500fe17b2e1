"""A transformer block's attention half on the library's operators, forward,
backward and for single tokens over a cache:

    y = x + Wo attention(rotary(Wq n), rotary(Wk n), Wv n) + bo,
    n = layer_norm(x; gamma, beta)

as the calls tg_layer_norm, tg_linear (one product for Q, K and V), tg_rotary,
tg_attention and tg_linear (with the residual added in its epilogue), and their
backward calls in reverse.  Sequences of different lengths are packed one behind
the other; `Attention.decode` takes one new token of each over a cache that
`Attention.prefill` has filled: rotary writes the keys to their rows of the
cache, and, with nothing to turn, the values.

    python examples/attention.py [tokens] [heads] [kv_heads] [dim]

prints the time of a training step's forward and backward pass and of one decoded
token of each sequence.
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
BASE = 10000.0
BF16 = torch.bfloat16


def _space(nbytes: int):
    if nbytes < 0:
        raise RuntimeError("workspace query failed")
    return torch.empty(nbytes, dtype=torch.uint8, device="cuda") if nbytes else None


def starts_of(lengths) -> torch.Tensor:
    at = [0]
    for n in lengths:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int64, device="cuda")


class Attention:
    """Parameters, the forward pass's saved tensors, the gradients and the cache."""

    def __init__(self, heads: int, kv_heads: int, dim: int, seed: int = 0):
        self.h, self.kv, self.dim, self.d = heads, kv_heads, dim, heads * dim
        self.qkv = (heads + 2 * kv_heads) * dim
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def weight(rows, cols):
            return (torch.randn(rows, cols, generator=g, device="cuda") / math.sqrt(cols)).to(BF16)

        self.w = {"Wqkv": weight(self.qkv, self.d), "Wo": weight(self.d, self.d),
                  "bo": torch.zeros(self.d, device="cuda"), "gamma": torch.ones(self.d, device="cuda"),
                  "beta": torch.zeros(self.d, device="cuda")}
        self.steps = torch.tensor(tg.tg_rotary_steps(dim, BASE), dtype=torch.int64, device="cuda")
        self.scale = 1.0 / math.sqrt(dim)
        self.grads = {}

    # ------------------------------------------------------------------ pieces

    def _project(self, x, train):
        """n = layer_norm(x) and the packed Q, K, V rows."""
        m, d, w, st = x.shape[0], self.d, self.w, torch.cuda.current_stream()
        n, qkv = torch.empty(m, d, dtype=BF16, device="cuda"), torch.empty(m, self.qkv, dtype=BF16, device="cuda")
        mean, rstd = (torch.empty(m, device="cuda") if train else None for _ in range(2))
        tg.check(tg.tg_layer_norm(m, d, x, x.stride(0), w["gamma"], w["beta"], EPS, n, d, mean, rstd, "bf16",
                                  st), "tg_layer_norm")
        ws = _space(tg.tg_linear_workspace_bytes(m, self.qkv, d, n, d, w["Wqkv"], d, "bf16"))
        tg.check(tg.tg_linear(m, self.qkv, d, n, d, w["Wqkv"], d, None, "none", None, 0, qkv, self.qkv, None,
                              0, "bf16", ws, st), "tg_linear")
        return n, mean, rstd, qkv

    def _turn(self, qkv, heads, positions):
        """Rotary positions, in place, on the rows' first `heads` heads."""
        tg.check(tg.tg_rotary(qkv.shape[0], heads, self.dim, self.dim, qkv, self.qkv, self.dim, qkv, self.qkv,
                              self.dim, 0, positions, None, self.steps, "halves", 1.0, "bf16",
                              torch.cuda.current_stream()), "tg_rotary")

    def _parts(self, qkv):
        """Q, K and V inside the packed rows, as (first element's address, strides)."""
        e, a = self.dim * qkv.element_size(), qkv.data_ptr()
        lay = (self.qkv, self.dim)
        return (a, *lay), (a + self.h * e, *lay), (a + (self.h + self.kv) * e, *lay)

    def _output(self, o, x):
        m, d, w, st = x.shape[0], self.d, self.w, torch.cuda.current_stream()
        y = torch.empty(m, d, dtype=BF16, device="cuda")
        ws = _space(tg.tg_linear_workspace_bytes(m, d, d, o, d, w["Wo"], d, "bf16"))
        tg.check(tg.tg_linear(m, d, d, o, d, w["Wo"], d, w["bo"], "none", x, x.stride(0), y, d, None, 0, "bf16",
                              ws, st), "tg_linear")
        return y

    # ------------------------------------------------------------------ training

    def forward(self, x: torch.Tensor, starts: torch.Tensor, positions: torch.Tensor, longest: int = 0,
                train: bool = False) -> torch.Tensor:
        """x: the packed tokens; starts: where each sequence begins, and their end."""
        m, st = x.shape[0], torch.cuda.current_stream()
        n, mean, rstd, qkv = self._project(x, train)
        self._turn(qkv, self.h + self.kv, positions)
        o = torch.empty(m, self.d, dtype=BF16, device="cuda")
        lse = torch.empty(self.h, m, device="cuda") if train else None
        size = (starts.numel() - 1, m, m, self.h, self.kv, self.dim)
        q, k, v = self._parts(qkv)
        ws = _space(tg.tg_attention_workspace_bytes(*size, longest, longest, "bf16"))
        tg.check(tg.tg_attention(*size, *q, *k, *v, starts, None, starts, None, longest, longest, True,
                                 self.scale, o, self.d, self.dim, lse, "bf16", ws, st), "tg_attention")
        if train:
            self.saved = (x, n, mean, rstd, qkv, o, lse, starts, positions, longest)
        else:
            self.rows = qkv
        return self._output(o, x)

    def backward(self, dy: torch.Tensor) -> torch.Tensor:
        """Gradients of the parameters into ``grads``; returns dx."""
        x, n, mean, rstd, qkv, o, lse, starts, positions, longest = self.saved
        m, d, w, st, f32 = x.shape[0], self.d, self.w, torch.cuda.current_stream(), torch.float32

        def new(rows, cols, dtype=BF16):
            return torch.empty(rows, cols, dtype=dtype, device="cuda")

        gr = {"Wqkv": new(self.qkv, d, f32), "Wo": new(d, d, f32), "bo": torch.empty(d, device="cuda"),
              "gamma": torch.empty(d, device="cuda"), "beta": torch.empty(d, device="cuda")}
        do, dqkv, dn, dx = new(m, d), new(m, self.qkv), new(m, d), new(m, d)
        ld = dy.stride(0)
        ws = _space(tg.tg_linear_backward_workspace_bytes(m, d, d, dy, ld, o, d, w["Wo"], d, "none", "bf16"))
        tg.check(tg.tg_linear_backward(m, d, d, dy, ld, o, d, w["Wo"], d, None, 0, "none", do, d, gr["Wo"], d,
                                       "f32", gr["bo"], "bf16", ws, st), "tg_linear_backward")
        size = (starts.numel() - 1, m, m, self.h, self.kv, self.dim)
        ins, outs = self._parts(qkv), self._parts(dqkv)
        ws = _space(tg.tg_attention_backward_workspace_bytes(*size, longest, longest, "bf16"))
        tg.check(tg.tg_attention_backward(*size, *ins[0], *ins[1], *ins[2], o, d, self.dim, do, d, self.dim, lse,
                                          starts, None, starts, None, longest, longest, True, self.scale,
                                          *outs[0], *outs[1], *outs[2], "bf16", ws, st), "tg_attention_backward")
        tg.check(tg.tg_rotary_backward(m, self.h + self.kv, self.dim, self.dim, dqkv, self.qkv, self.dim, dqkv,
                                       self.qkv, self.dim, positions, self.steps, "halves", 1.0, "bf16", st),
                 "tg_rotary_backward")
        ws = _space(tg.tg_linear_backward_workspace_bytes(m, self.qkv, d, dqkv, self.qkv, n, d, w["Wqkv"], d,
                                                          "none", "bf16"))
        tg.check(tg.tg_linear_backward(m, self.qkv, d, dqkv, self.qkv, n, d, w["Wqkv"], d, None, 0, "none", dn, d,
                                       gr["Wqkv"], d, "f32", None, "bf16", ws, st), "tg_linear_backward")
        ws = _space(tg.tg_layer_norm_backward_workspace_bytes(m, d))
        tg.check(tg.tg_layer_norm_backward(m, d, dn, d, x, x.stride(0), w["gamma"], mean, rstd, dx, d,
                                           gr["gamma"], gr["beta"], "bf16", ws, st), "tg_layer_norm_backward")
        self.grads = gr
        return dx + dy  # the residual's share

    # ------------------------------------------------------------------ serving

    def prefill(self, x: torch.Tensor, lengths, capacity: int) -> torch.Tensor:
        """The prompts' outputs; their keys and values go to a cache of `capacity` rows
        for each sequence, as many as its prompt and the tokens to come may have."""
        if max(lengths) > capacity:
            raise ValueError(f"a prompt of {max(lengths)} tokens for {capacity} rows of a cache")
        starts = starts_of(lengths)
        positions = torch.cat([torch.arange(n, device="cuda") for n in lengths])
        y = self.forward(x, starts, positions, max(lengths))
        self.capacity, self.seqs, self.longest = capacity, len(lengths), max(lengths)
        self.cache = torch.empty(2, self.seqs * capacity, self.kv * self.dim, dtype=BF16, device="cuda")
        self.slabs = torch.arange(self.seqs, device="cuda") * capacity
        self.lengths = torch.tensor(lengths, dtype=torch.int64, device="cuda")
        rows = positions + torch.repeat_interleave(self.slabs, self.lengths)
        # (the keys have been turned already: rot = 0 copies)
        self._keep(self.rows, rows, None, 0)
        return y

    def _keep(self, qkv, rows, positions, rot):
        """Keys (turned) and values to their rows of the cache."""
        _, k, v = self._parts(qkv)
        for part, cache, r in ((k, self.cache[0], rot), (v, self.cache[1], 0)):
            tg.check(tg.tg_rotary(qkv.shape[0], self.kv, self.dim, r, *part, cache, self.kv * self.dim, self.dim,
                                  cache.shape[0], positions, rows, self.steps if r else None, "halves", 1.0,
                                  "bf16", torch.cuda.current_stream()), "tg_rotary")

    def decode(self, x: torch.Tensor) -> torch.Tensor:
        """One new token of each sequence (its row of x)."""
        if self.longest == self.capacity:  # (its next row is another sequence's first)
            raise ValueError(f"a sequence has filled the cache's {self.capacity} rows of its own")
        self.longest += 1
        m, st = self.seqs, torch.cuda.current_stream()
        _, _, _, qkv = self._project(x, False)
        positions = self.lengths  # the new token's
        rows = self.slabs + positions
        self._turn(qkv, self.h, positions)
        self._keep(qkv, rows, positions, self.dim)
        self.lengths = positions + 1
        o = torch.empty(m, self.d, dtype=BF16, device="cuda")
        size = (m, m, self.cache.shape[1], self.h, self.kv, self.dim)
        q = self._parts(qkv)[0]
        kv = (self.kv * self.dim, self.dim)
        each = torch.arange(m + 1, device="cuda")
        ws = _space(tg.tg_attention_workspace_bytes(*size, 1, self.capacity, "bf16"))
        tg.check(tg.tg_attention(*size, *q, self.cache[0], *kv, self.cache[1], *kv, each, None, self.slabs,
                                 self.lengths, 1, self.capacity, True, self.scale, o, self.d, self.dim, None,
                                 "bf16", ws, st), "tg_attention")
        return self._output(o, x)


def main(argv) -> None:
    m, heads, kv, dim = [int(v) for v in (argv + [0] * 4)[:4]]
    m, heads, kv, dim = m or 4096, heads or 16, kv or 4, dim or 128
    tg.build()
    tg.load()
    block = Attention(heads, kv, dim)
    lengths = [m // 2, m // 4, m - m // 2 - m // 4]
    starts = starts_of(lengths)
    positions = torch.cat([torch.arange(n, device="cuda") for n in lengths])
    x = torch.randn(m, heads * dim, device="cuda").to(BF16)
    dy = torch.randn(m, heads * dim, device="cuda").to(BF16)

    def timed(f, n=20):
        for _ in range(3):
            f()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(n):
            f()
        b.record()
        torch.cuda.synchronize()
        return a.elapsed_time(b) / n * 1e3

    print(f"forward: {timed(lambda: block.forward(x, starts, positions, max(lengths), True)):.1f} us")
    print(f"backward: {timed(lambda: block.backward(dy)):.1f} us")
    block.prefill(x, lengths, max(lengths) + 64)
    token = x[: len(lengths)]
    print(f"one token of {len(lengths)} sequences: {timed(lambda: block.decode(token)):.1f} us")
    st, where = tg.tg_check_device_status(torch.cuda.current_stream())
    tg.check(st, f"device status (wait site {where})")


if __name__ == "__main__":
    main(sys.argv[1:])

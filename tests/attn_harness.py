"""Inputs, FP64 references and error bounds for the attention operators.

The references are plain FP64 torch expressions of the definitions.  The
bounds are worst-case ones, from the kernels' arithmetic; U is half a step of
the 16-bit type (relative 2^-8 BF16, 2^-11 FP16):

* a score: products of 16-bit values are exact, every tensor-core step rounds
  or truncates the FP32 sum: (dim/8 + 32) 2^-23 times the sum of magnitudes,
  then the scale and the reference in one FP32 operation and their own
  roundings, 2^-22 (|s| + |m|) in natural units (m the row's maximum);
* a probability: that error as a factor, 2^-21 for the hardware exponential,
  U for the rounding to 16 bits, and half FP16's smallest subnormal (2^-25),
  probabilities being at least as large as those relative to the maximum;
* a sum of n probabilities: n FP32 roundings at most, but no more than the
  kernels' 32 a block and one for each block and range: (64 + n/32) 2^-23;
* a product with V (or dO, K, Q) over n terms: (n/8 + 32) 2^-23 of the sum of
  magnitudes, and n/128 rescalings of the accumulator at 2^-22 each;
* the result's rounding: U of the value, 2^-25 for FP16.
"""

from __future__ import annotations

import math

import torch

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
TINY = {"bf16": 0.0, "fp16": 2.0 ** -25}


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


class Tensor3:
    """rows x heads x dim values inside a wider buffer whose padding holds a
    sentinel (NaN): `pad` elements behind each row, `gap` between heads."""

    def __init__(self, rows, heads, dim, dtype, pad=0, gap=0, heads_first=False, fill=None):
        t = TYPES.get(dtype, torch.float32)
        if heads_first:
            self.ld, self.hd = dim + pad, max(rows, 1) * (dim + pad) + gap
            size = heads * self.hd
        else:
            self.hd = dim + gap
            self.ld = heads * self.hd + pad
            size = max(rows, 1) * self.ld
        self.buf = torch.full((size + 16,), float("nan"), dtype=t, device="cuda")
        self.t = torch.as_strided(self.buf, (rows, heads, dim), (self.ld, self.hd, 1))
        if fill is not None:
            self.t.copy_(fill)
        self.before = self.buf.clone()

    def data_ptr(self):
        return self.buf.data_ptr()

    @property
    def lay(self):
        return self, self.ld, self.hd

    def kept_outside(self, rows):
        """Everything but the given rows (a boolean mask) still holds what it held."""
        now, was = self.buf.clone(), self.before.clone()
        for b in (now, was):
            torch.as_strided(b, tuple(self.t.shape), (self.ld, self.hd, 1))[rows] = 0
        i = torch.int32 if self.buf.dtype == torch.float32 else torch.int16
        return torch.equal(now.view(i), was.view(i))

    def d(self):
        return self.t.double()


class Problem:
    """A packed batch: `q_len` and `k_len` rows a sequence, at `q_at` and `k_at`
    (one behind the other unless given), of tensors with `q_rows`, `k_rows` rows."""

    def __init__(self, q_len, k_len=None, heads=2, kv=1, dim=64, dtype="bf16", causal=True, seed=1,
                 q_at=None, k_at=None, q_rows=None, k_rows=None, scale=None, pad=0, gap=0,
                 heads_first=False, sigma=1.0, lengths=False, max_q=None, max_k=None):
        k_len = list(q_len) if k_len is None else k_len
        self.q_len, self.k_len, self.heads, self.kv, self.dim = q_len, k_len, heads, kv, dim
        self.dtype, self.causal, self.seqs, self.g = dtype, causal, len(q_len), heads // kv

        def starts(n, at):
            if at is not None:
                return list(at) + [0]
            s = [0]
            for v in n:
                s.append(s[-1] + v)
            return s

        self.q_at, self.k_at = starts(q_len, q_at), starts(k_len, k_at)
        self.q_rows = q_rows if q_rows is not None else sum(q_len)
        self.k_rows = k_rows if k_rows is not None else sum(k_len)
        self.scale = 1.0 / math.sqrt(dim) if scale is None else scale
        self.max_q = max(q_len + [1]) if max_q is None else max_q
        self.max_k = max(k_len + [1]) if max_k is None else max_k
        self.lengths = lengths or q_at is not None or k_at is not None
        g = gen(seed)
        self.shape = dict(pad=pad, gap=gap, heads_first=heads_first)

        def make(rows, at, n, h):
            x = Tensor3(rows, h, dim, dtype, **self.shape)
            for a, m in zip(at, n):
                if m:
                    x.t[a: a + m] = (torch.randn(m, h, dim, generator=g, device="cuda") * sigma).to(TYPES[dtype])
            x.before = x.buf.clone()
            return x

        self.Q = make(self.q_rows, self.q_at, q_len, heads)
        self.K = make(self.k_rows, self.k_at, k_len, kv)
        self.V = make(self.k_rows, self.k_at, k_len, kv)
        self.dO = make(self.q_rows, self.q_at, q_len, heads)
        self.dev = [torch.tensor(x, dtype=torch.int64, device="cuda")
                    for x in (self.q_at, q_len, self.k_at, k_len)]

    def rows(self, keys=False):
        m = torch.zeros(self.k_rows if keys else self.q_rows, dtype=torch.bool, device="cuda")
        for a, n in zip(*((self.k_at, self.k_len) if keys else (self.q_at, self.q_len))):
            m[a: a + n] = True
        return m

    def sizes(self):
        return self.seqs, self.q_rows, self.k_rows, self.heads, self.kv, self.dim

    def arrays(self):
        qa, ql, ka, kl = self.dev
        return (qa, ql, ka, kl) if self.lengths else (qa, None, ka, None)

    def pieces(self):
        """(rows, keys, head, key head, S in natural units, its error, mask) in FP64."""
        for n in range(self.seqs):
            a, b = self.q_len[n], self.k_len[n]
            if not a or not b:
                continue
            rows = slice(self.q_at[n], self.q_at[n] + a)
            keys = slice(self.k_at[n], self.k_at[n] + b)
            see = torch.ones(a, b, dtype=torch.bool, device="cuda")
            if self.causal:
                see = see.tril(b - a)
            for h in range(self.heads):
                k = self.K.d()[keys, h // self.g]
                q = self.Q.d()[rows, h]
                s = self.scale * (q @ k.t())
                e = abs(self.scale) * (self.dim / 8 + 32) * 2.0 ** -23 * (q.abs() @ k.abs().t())
                yield rows, keys, h, h // self.g, s.masked_fill(~see, -math.inf), e, see


def reference(p):
    """O, its bound, LSE, its bound."""
    o = torch.zeros(p.q_rows, p.heads, p.dim, dtype=torch.float64, device="cuda")
    eo = torch.zeros_like(o)
    lse = torch.full((p.heads, p.q_rows), -math.inf, dtype=torch.float64, device="cuda")
    el = torch.zeros_like(lse)
    for rows, keys, h, kh, s, e, see in p.pieces():
        z = torch.logsumexp(s, 1)
        seen = z != -math.inf
        w = torch.where(seen[:, None], torch.exp(s - z[:, None]), 0.0)
        v = p.V.d()[keys, kh]
        n = s.shape[1]
        top = torch.where(see, s, -math.inf).amax(1, keepdim=True).masked_fill(~seen[:, None], 0.0)
        es = torch.where(see, e + 2.0 ** -22 * (s.abs() + top.abs()), 0.0)
        rel = es + 2.0 ** -21
        sum_rel = (64 + n / 32) * 2.0 ** -23 + (w * rel).sum(1)
        o[rows, h] = w @ v
        lse[h, rows] = z
        el[h, rows] = torch.where(seen, sum_rel + 2.0 ** -21 * (z.abs() + top[:, 0].abs()) + 2.0 ** -22, 0.0)
        mag = w @ v.abs()
        err = (w * (rel + U[p.dtype])) @ v.abs() + mag * (sum_rel[:, None] + (n / 8 + 32) * 2.0 ** -23 +
                                                          n / 128 * 2.0 ** -22)
        # (a probability's smallest step, over the probabilities of a sum of at least 1)
        err = err + TINY[p.dtype] * (see.double() @ v.abs())
        eo[rows, h] = err + U[p.dtype] * ((w @ v).abs() + err) + TINY[p.dtype]
    return o, eo, lse, el


def check(got, want, bound, what):
    got = got.double()
    assert got.shape == want.shape, what
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan), f"{what}: NaN positions differ"
    bad = ((got - want).abs() > bound) & ~nan & (got != want)
    if bad.any():
        i = int(torch.nonzero(bad.reshape(-1))[0])
        raise AssertionError(
            f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound; first at {i}: "
            f"{float(got.reshape(-1)[i])} for {float(want.reshape(-1)[i])}, bound "
            f"{float(bound.reshape(-1)[i])}")


def space(nbytes):
    assert nbytes >= 0
    return torch.empty(nbytes, dtype=torch.uint8, device="cuda") if nbytes else None


def done(tg, status, what):
    tg.check(status, what)
    st, where = tg.tg_check_device_status(torch.cuda.current_stream())
    tg.check(st, f"{what}: device status (wait site {where})")


def run_forward(tg, p, lse=True):
    o = Tensor3(p.q_rows, p.heads, p.dim, p.dtype, **p.shape)
    z = torch.full((p.heads, p.q_rows), float("nan"), device="cuda") if lse else None
    ws = space(tg.tg_attention_workspace_bytes(*p.sizes(), p.max_q, p.max_k, p.dtype))
    done(tg, tg.tg_attention(*p.sizes(), *p.Q.lay, *p.K.lay, *p.V.lay, *p.arrays(), p.max_q, p.max_k,
                             p.causal, p.scale, *o.lay, z, p.dtype, ws, torch.cuda.current_stream()),
         "tg_attention")
    return o, z


def check_forward(tg, p, what="attention"):
    o, z = run_forward(tg, p)
    want, eo, lse, el = reference(p)
    rows = p.rows()
    check(o.t[rows], want[rows], eo[rows], what + " O")
    check(z[:, rows], lse[:, rows], el[:, rows], what + " LSE")
    assert o.kept_outside(rows), what + ": rows of no sequence were written"
    assert bool(torch.isnan(z[:, ~rows]).all()), what + ": LSE of no sequence was written"
    return o, z

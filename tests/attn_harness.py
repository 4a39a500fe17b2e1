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
* the result's rounding: U of the value, 2^-25 for FP16;
* the hardware exponential gives 0 for a result below FP32's smallest normal
  number, so a probability below 2^-126 is off by all of itself, less than 2^-126
  (in FP16 2^-25 covers it).  In the gradients, which start from LSE, such
  probabilities meet no larger one in a key's sum: 2^-126 stands in for 2^-25.
"""

from __future__ import annotations

import math

import torch

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
TINY = {"bf16": 2.0 ** -126, "fp16": 2.0 ** -25}


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


# ------------------------------------------------------------------ backward


def given(p):
    """The forward's O, rounded to the type, and LSE, as the backward pass reads them."""
    o, _, lse, _ = reference(p)
    rows = p.rows()
    x = Tensor3(p.q_rows, p.heads, p.dim, p.dtype, **p.shape)
    x.t[rows] = o[rows].to(TYPES[p.dtype])
    z = lse.float()
    z[:, ~rows] = float("nan")
    return x, z


def reference_backward(p, o, lse):
    """{name: (gradient, its bound)}."""
    f64 = dict(dtype=torch.float64, device="cuda")
    u, tiny = U[p.dtype], TINY[p.dtype]
    dq, dk, dv = (torch.zeros(r, h, p.dim, **f64) for r, h in ((p.q_rows, p.heads), (p.k_rows, p.kv), (p.k_rows, p.kv)))
    eq, ek, ev, mq, mk, mv = (torch.zeros_like(x) for x in (dq, dk, dv, dq, dk, dv))
    od, dod = o.d(), p.dO.d()
    for rows, keys, h, kh, s, e, see in p.pieces():
        z = lse[h, rows].double()[:, None]
        q, k, v, do = p.Q.d()[rows, h], p.K.d()[keys, kh], p.V.d()[keys, kh], dod[rows, h]
        some = z != -math.inf
        w = torch.where(see & some, torch.exp(s - z), 0.0)
        rel = torch.where(see, e + 2.0 ** -22 * (s.abs() + z.abs()), 0.0) + 2.0 ** -21
        rel = torch.where(some, rel, 0.0)
        ep = torch.where(see, w * (rel + u) + tiny, 0.0)
        delta = (do * od[rows, h]).sum(1, keepdim=True)
        dp = do @ v.t() - delta
        short = (p.dim / 8 + 32) * 2.0 ** -23
        edp = short * (do.abs() @ v.abs().t() + (do * od[rows, h]).abs().sum(1, keepdim=True)) + 2.0 ** -23 * dp.abs()
        ds = w * dp
        eds = w * (1 + rel) * edp + ds.abs() * (rel + 2.0 ** -22 + u)
        eds = torch.where(see & some, eds + u * eds + tiny, 0.0)
        dv[keys, kh] += w.t() @ do
        ev[keys, kh] += ep.t() @ do.abs()
        mv[keys, kh] += w.t() @ do.abs()
        dk[keys, kh] += p.scale * (ds.t() @ q)
        ek[keys, kh] += p.scale * (eds.t() @ q.abs())
        mk[keys, kh] += p.scale * (ds.abs().t() @ q.abs())
        dq[rows, h] = p.scale * (ds @ k)
        eq[rows, h] = p.scale * (eds @ k.abs())
        mq[rows, h] = p.scale * (ds.abs() @ k.abs())
    out = {}
    for name, x, e, m, n in (("dQ", dq, eq, mq, max(p.k_len + [0])),
                             ("dK", dk, ek, mk, p.g * max(p.q_len + [0])),
                             ("dV", dv, ev, mv, p.g * max(p.q_len + [0]))):
        e = e + (n / 8 + 32) * 2.0 ** -23 * m + 2.0 ** -23 * x.abs()
        out[name] = (x, e + u * (x.abs() + e) + tiny)
    return out


def run_backward(tg, p, o, lse, want=("dQ", "dK", "dV")):
    out = {"dQ": Tensor3(p.q_rows, p.heads, p.dim, p.dtype, **p.shape),
           "dK": Tensor3(p.k_rows, p.kv, p.dim, p.dtype, **p.shape),
           "dV": Tensor3(p.k_rows, p.kv, p.dim, p.dtype, **p.shape)}
    lay = [x for n in ("dQ", "dK", "dV") for x in (out[n].lay if n in want else (None, 0, 0))]
    ws = space(tg.tg_attention_backward_workspace_bytes(*p.sizes(), p.max_q, p.max_k, p.dtype))
    done(tg, tg.tg_attention_backward(*p.sizes(), *p.Q.lay, *p.K.lay, *p.V.lay, *o.lay, *p.dO.lay, lse,
                                      *p.arrays(), p.max_q, p.max_k, p.causal, p.scale, *lay, p.dtype, ws,
                                      torch.cuda.current_stream()), "tg_attention_backward")
    return out


def check_backward(tg, p, what="attention_backward"):
    o, lse = given(p)
    out = run_backward(tg, p, o, lse)
    want = reference_backward(p, o, lse)
    for name, got in out.items():
        rows = p.rows(keys=name != "dQ")
        x, bound = want[name]
        check(got.t[rows], x[rows], bound[rows], f"{what} {name}")
        assert got.kept_outside(rows), f"{what} {name}: rows of no sequence were written"
    return out

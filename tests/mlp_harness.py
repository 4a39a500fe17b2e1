"""Inputs, FP64 references and error bounds for the feed-forward operators.

The references are plain FP64 torch expressions of the definitions.  The
bounds are worst-case ones, from the kernels' arithmetic:

* a product of K terms: every tensor-core step (16 terms) and every join of K
  segments rounds (or truncates) the FP32 accumulator once, so the error is at
  most (K/16 + 16) 2^-23 times the sum S of the terms' magnitudes; K/8 + 32
  is used, for steps of 8;
* an activation in FP32: relative 2^-18 of its value (a hardware exponential
  and reciprocal, a few FP32 operations), times its largest slope (1.13) for
  an error of its argument;
* a rounding to a 16-bit type: relative 2^-8 (BF16: 8 significand bits) or
  2^-11 (FP16) of the value, and half the smallest subnormal of FP16 (2^-25).
  (BF16's smallest subnormals do not matter here: they are FP32's.)
* a sum of n FP32 values: n 2^-24 times the sum of magnitudes.
"""

from __future__ import annotations

import math

import torch

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "f32": torch.float32}
U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "f32": 2.0 ** -24}
TINY = {"bf16": 0.0, "fp16": 2.0 ** -25, "f32": 0.0}
SLOPE = 1.13  # the largest |derivative| of the activations
FN = 2.0 ** -18  # relative error of an activation or its derivative in FP32
GELU_C = math.sqrt(2.0 / math.pi)


def act64(name, x):
    if name == "none":
        return x
    if name == "relu":
        return torch.where(x > 0, x, torch.zeros_like(x))
    if name == "silu":
        return x / (1 + torch.exp(-x))
    return 0.5 * x * (1 + torch.tanh(GELU_C * (x + 0.044715 * x ** 3)))


def act_grad64(name, x):
    if name == "none":
        return torch.ones_like(x)
    if name == "relu":
        return (x > 0).double()
    if name == "silu":
        s = 1 / (1 + torch.exp(-x))
        return s + x * s * (1 - s)
    t = torch.tanh(GELU_C * (x + 0.044715 * x ** 3))
    return 0.5 * (1 + t) + 0.5 * x * (1 - t * t) * GELU_C * (1 + 3 * 0.044715 * x * x)


class Rows:
    """A rows x cols matrix inside a wider buffer whose padding holds a
    sentinel; `skew` shifts its base by that many elements."""

    def __init__(self, rows, cols, dtype, pad=0, skew=0, fill=None):
        self.dtype = TYPES[dtype]
        self.ld = max(cols + pad, 1)
        self.rows, self.cols, self.skew = rows, cols, skew
        self.buf = torch.full((rows * self.ld + skew + 16,), float("nan"), dtype=self.dtype,
                              device="cuda")
        self.t = self.buf[skew: skew + rows * self.ld].view(rows, self.ld)[:, :cols]
        if fill is not None:
            self.t.copy_(fill)
        self.before = self.buf.clone()

    def data_ptr(self):
        return self.t.data_ptr() if self.t.numel() else self.buf.data_ptr()

    def padding_kept(self):
        """Every element outside the matrix still holds the sentinel."""
        now, was = self.buf.clone(), self.before.clone()
        for b in (now, was):
            b[self.skew: self.skew + self.rows * self.ld].view(self.rows, self.ld)[:, : self.cols] = 0
        i = torch.int32 if self.dtype == torch.float32 else torch.int16
        return torch.equal(now.view(i), was.view(i))

    def d(self):
        return self.t.double()


def rows(g, m, n, dtype, pad=0, skew=0, scale=1.0, shift=0.0):
    v = torch.randn(m, n, generator=g, device="cuda") * scale + shift
    return Rows(m, n, dtype, pad, skew, v.to(TYPES[dtype]))


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def product_error(k, s):
    return (k / 8 + 32) * 2.0 ** -23 * s


def rounded(dtype, value, err):
    """Bound on the error of `value` known to within `err`, rounded to dtype."""
    return err + U[dtype] * (value.abs() + err) + TINY[dtype]


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


# ------------------------------------------------------------------ operators on Rows


def run_linear(tg, x, w, bias, act, r, dtype, save=False, y=None, pad=0, skew=0, stream=None):
    m, k, n = x.rows, x.cols, w.rows
    y = y or Rows(m, n, dtype, pad, skew)
    z = Rows(m, n, dtype, pad, skew) if save else None
    st = stream or torch.cuda.current_stream()
    ws = space(tg.tg_linear_workspace_bytes(m, n, k, x, x.ld, w, w.ld, dtype))
    done(tg, tg.tg_linear(m, n, k, x, x.ld, w, w.ld, bias, act, r, r.ld if r else 0, y, y.ld, z,
                          z.ld if z else 0, dtype, ws, st), "tg_linear")
    return y, z


def ref_linear(x, w, bias, act, r, dtype):
    """(Y, its bound, Z, its bound)."""
    k = x.cols
    z = x.d() @ w.d().t()
    s = x.d().abs() @ w.d().abs().t()
    ze = product_error(k, s)
    if bias is not None:
        z = z + bias.double()
        ze = ze + 2.0 ** -23 * z.abs()
    y = act64(act, z)
    ye = SLOPE * ze + FN * y.abs()
    if r is not None:
        y = y + r.d()
        ye = ye + 2.0 ** -23 * y.abs()
    return y, rounded(dtype, y, ye), z, rounded(dtype, z, ze)


def check_linear(tg, m, n, k, dtype, act="none", bias=False, residual=False, save=False, pad=0,
                 skew=0, opad=None, oskew=None, seed=1, inplace=False):
    g = gen(seed + 31 * m + 17 * n + k)
    x = rows(g, m, k, dtype, pad, skew)
    w = rows(g, n, k, dtype, pad, skew, 1 / math.sqrt(max(k, 1)))
    b = torch.randn(n, generator=g, device="cuda") if bias else None
    opad = pad if opad is None else opad
    oskew = skew if oskew is None else oskew
    r = rows(g, m, n, dtype, opad, oskew) if residual else None
    want, ye, wz, ze = ref_linear(x, w, b, act, r, dtype)
    y, z = run_linear(tg, x, w, b, act, r, dtype, save, r if inplace else None, opad, oskew)
    what = f"linear {m}x{n}x{k} {dtype} {act}"
    check(y.t, want, ye, what + " Y")
    assert y.padding_kept(), what
    if save:
        check(z.t, wz, ze, what + " Z")
        assert z.padding_kept(), what
    return y


def check_linear_backward(tg, m, n, k, dtype, act="none", bias=True, pad=0, skew=0, dw="same",
                          seed=2, want_dx=True, want_dw=True):
    g = gen(seed + 31 * m + 17 * n + k)
    x = rows(g, m, k, dtype, pad, skew)
    w = rows(g, n, k, dtype, pad, skew, 1 / math.sqrt(max(k, 1)))
    dy = rows(g, m, n, dtype, pad, skew)
    z = rows(g, m, n, dtype, pad, skew, 1.5) if act != "none" else None
    dwt = dtype if dw == "same" else dw
    dx = Rows(m, k, dtype, pad, skew) if want_dx else None
    dwm = Rows(n, k, dwt, pad, skew) if want_dw else None
    db = torch.full((n,), float("nan"), device="cuda") if bias else None
    ws = space(tg.tg_linear_backward_workspace_bytes(m, n, k, dy, dy.ld, x, x.ld, w, w.ld, act, dtype))
    done(tg, tg.tg_linear_backward(m, n, k, dy, dy.ld, x, x.ld, w, w.ld, z, z.ld if z else 0, act,
                                   dx, dx.ld if dx else 0, dwm, dwm.ld if dwm else 0, dwt, db,
                                   dtype, ws, torch.cuda.current_stream()), "tg_linear_backward")
    what = f"linear_backward {m}x{n}x{k} {dtype} {act}"
    dz = dy.d()
    e = torch.zeros_like(dz)  # error of dZ as the products read it
    e32 = torch.zeros_like(dz)
    if act != "none":
        dz = dz * act_grad64(act, z.d())
        e32 = FN * SLOPE * dy.d().abs()
        e = rounded(dtype, dz, e32)
    if want_dx:
        v, s = dz @ w.d(), dz.abs() @ w.d().abs()
        check(dx.t, v, rounded(dtype, v, product_error(n, s) + e @ w.d().abs()), what + " dX")
        assert dx.padding_kept(), what
    if want_dw:
        v, s = dz.t() @ x.d(), dz.abs().t() @ x.d().abs()
        check(dwm.t, v, rounded(dwt, v, product_error(m, s) + e.t() @ x.d().abs()), what + " dW")
        assert dwm.padding_kept(), what
    if bias:
        check(db, dz.sum(0), (m * 2.0 ** -24) * dz.abs().sum(0) + e32.sum(0) + 1e-30, what + " db")
    return dx, dwm, db


def check_gated(tg, m, n, k, dtype, act="silu", save=False, pad=0, skew=0, seed=3):
    g = gen(seed + 31 * m + 17 * n + k)
    x = rows(g, m, k, dtype, pad, skew)
    s = 1 / math.sqrt(max(k, 1))
    wg, wu = rows(g, n, k, dtype, pad, skew, s), rows(g, n, k, dtype, pad, skew, s)
    h = Rows(m, n, dtype, pad, skew)
    gg, uu = (Rows(m, n, dtype, pad, skew), Rows(m, n, dtype, pad, skew)) if save else (None, None)
    ws = space(tg.tg_gated_workspace_bytes(m, n, k, x, x.ld, wg, wg.ld, wu, wu.ld, dtype))
    done(tg, tg.tg_gated(m, n, k, x, x.ld, wg, wg.ld, wu, wu.ld, act, h, h.ld, gg,
                         gg.ld if save else 0, uu, uu.ld if save else 0, dtype, ws,
                         torch.cuda.current_stream()), "tg_gated")
    what = f"gated {m}x{n}x{k} {dtype} {act}"
    vg, vu = x.d() @ wg.d().t(), x.d() @ wu.d().t()
    eg = product_error(k, x.d().abs() @ wg.d().abs().t())
    eu = product_error(k, x.d().abs() @ wu.d().abs().t())
    a = act64(act, vg)
    ea = SLOPE * eg + FN * a.abs()
    e = a.abs() * eu + vu.abs() * ea + ea * eu + 2.0 ** -23 * (a * vu).abs()
    check(h.t, a * vu, rounded(dtype, a * vu, e), what + " H")
    assert h.padding_kept(), what
    if save:
        check(gg.t, vg, rounded(dtype, vg, eg), what + " G")
        check(uu.t, vu, rounded(dtype, vu, eu), what + " U")
        assert gg.padding_kept() and uu.padding_kept(), what
    return h


def check_gated_backward(tg, m, n, k, dtype, act="silu", pad=0, skew=0, dw="same", seed=4,
                         want=(True, True, True)):
    g = gen(seed + 31 * m + 17 * n + k)
    x = rows(g, m, k, dtype, pad, skew)
    s = 1 / math.sqrt(max(k, 1))
    wg, wu = rows(g, n, k, dtype, pad, skew, s), rows(g, n, k, dtype, pad, skew, s)
    dh, gg, uu = (rows(g, m, n, dtype, pad, skew) for _ in range(3))
    dwt = dtype if dw == "same" else dw
    dx = Rows(m, k, dtype, pad, skew) if want[0] else None
    dwg = Rows(n, k, dwt, pad, skew) if want[1] else None
    dwu = Rows(n, k, dwt, pad, skew) if want[2] else None
    ld = lambda r: r.ld if r else 0  # noqa: E731
    ws = space(tg.tg_gated_backward_workspace_bytes(m, n, k, x, x.ld, wg, wg.ld, wu, wu.ld, dtype))
    done(tg, tg.tg_gated_backward(m, n, k, dh, dh.ld, x, x.ld, wg, wg.ld, wu, wu.ld, gg, gg.ld, uu,
                                  uu.ld, act, dx, ld(dx), dwg, ld(dwg), dwu, ld(dwu), dwt, dtype,
                                  ws, torch.cuda.current_stream()), "tg_gated_backward")
    what = f"gated_backward {m}x{n}x{k} {dtype} {act}"
    a = act64(act, gg.d())
    dg, du = dh.d() * uu.d() * act_grad64(act, gg.d()), dh.d() * a
    eg = rounded(dtype, dg, (FN * SLOPE + 2.0 ** -22) * (dh.d() * uu.d()).abs())
    eu = rounded(dtype, du, (FN + 2.0 ** -22) * du.abs())
    if want[0]:
        v = dg @ wg.d() + du @ wu.d()
        t = dg.abs() @ wg.d().abs() + du.abs() @ wu.d().abs()
        e = product_error(2 * n, t) + eg @ wg.d().abs() + eu @ wu.d().abs()
        check(dx.t, v, rounded(dtype, v, e), what + " dX")
        assert dx.padding_kept(), what
    for out, d, ed, name in ((dwg, dg, eg, "dWg"), (dwu, du, eu, "dWu")):
        if out is None:
            continue
        v = d.t() @ x.d()
        e = product_error(m, d.abs().t() @ x.d().abs()) + ed.t() @ x.d().abs()
        check(out.t, v, rounded(dwt, v, e), f"{what} {name}")
        assert out.padding_kept(), what


def norm_stats(x, eps):
    mean = x.mean(1, keepdim=True)
    var = ((x - mean) ** 2).mean(1, keepdim=True)
    return mean, (var + eps) ** -0.5


def check_norm(tg, m, n, dtype, affine=True, save=True, pad=0, skew=0, scale=1.5, shift=0.25,
               eps=1e-5, seed=5):
    """FP32 error of the normalised value: 64 roundings' worth (16 terms a
    thread, 5 + 4 + 3 levels of the tree, both statistics, the product), of the
    row's largest magnitude in units of its deviation and of xh itself."""
    g = gen(seed + 31 * m + n)
    x = rows(g, m, n, dtype, pad, skew, scale, shift)
    ga = 1 + 0.3 * torch.randn(n, generator=g, device="cuda") if affine else None
    be = torch.randn(n, generator=g, device="cuda") if affine else None
    y = Rows(m, n, dtype, pad, skew)
    mean = torch.full((m,), float("nan"), device="cuda") if save else None
    rstd = torch.full((m,), float("nan"), device="cuda") if save else None
    done(tg, tg.tg_layer_norm(m, n, x, x.ld, ga, be, eps, y, y.ld, mean, rstd, dtype,
                              torch.cuda.current_stream()), "tg_layer_norm")
    what = f"layer_norm {m}x{n} {dtype}"
    # eps reaches the kernel as FP32.
    wm, wr = norm_stats(x.d(), float(torch.tensor(eps, dtype=torch.float32)))
    xh = (x.d() - wm) * wr
    top = x.d().abs().amax(1, keepdim=True) * wr
    e = 64 * 2.0 ** -24 * (top + xh.abs() * (1 + top * top * 2.0 ** -20) + 1)
    v = xh
    if affine:
        v = xh * ga.double() + be.double()
        e = e * ga.double().abs() + 2.0 ** -23 * (v.abs() + be.double().abs())
    check(y.t, v, rounded(dtype, v, e), what + " Y")
    assert y.padding_kept(), what
    if save:
        check(mean, wm[:, 0], 64 * 2.0 ** -24 * x.d().abs().mean(1) + 1e-30, what + " mean")
        check(rstd, wr[:, 0], 64 * 2.0 ** -24 * (1 + top[:, 0]) * wr[:, 0], what + " rstd")


def check_norm_backward(tg, m, n, dtype, affine=True, pad=0, skew=0, seed=6, want=(True, True, True)):
    g = gen(seed + 31 * m + n)
    x = rows(g, m, n, dtype, pad, skew, 1.5, 0.25)
    dy = rows(g, m, n, dtype, pad, skew)
    ga = 1 + 0.3 * torch.randn(n, generator=g, device="cuda") if affine else None
    wm, wr = norm_stats(x.d(), 1e-5)
    mean, rstd = wm[:, 0].float().contiguous(), wr[:, 0].float().contiguous()
    wm, wr = mean.double()[:, None], rstd.double()[:, None]
    dx = Rows(m, n, dtype, pad, skew) if want[0] else None
    dga = torch.full((n,), float("nan"), device="cuda") if want[1] else None
    dbe = torch.full((n,), float("nan"), device="cuda") if want[2] else None
    ws = space(tg.tg_layer_norm_backward_workspace_bytes(m, n))
    done(tg, tg.tg_layer_norm_backward(m, n, dy, dy.ld, x, x.ld, ga, mean, rstd, dx,
                                       dx.ld if dx else 0, dga, dbe, dtype, ws,
                                       torch.cuda.current_stream()), "tg_layer_norm_backward")
    what = f"layer_norm_backward {m}x{n} {dtype}"
    xh = (x.d() - wm) * wr
    a = dy.d() * ga.double() if affine else dy.d()
    if want[0]:
        s1, s2 = a.mean(1, keepdim=True), (a * xh).mean(1, keepdim=True)
        v = wr * (a - s1 - xh * s2)
        e = 64 * 2.0 ** -24 * wr * (a.abs() + a.abs().mean(1, keepdim=True) +
                                    xh.abs() * (a * xh).abs().mean(1, keepdim=True))
        check(dx.t, v, rounded(dtype, v, e), what + " dX")
        assert dx.padding_kept(), what
    if want[1]:
        t = dy.d() * xh
        check(dga, t.sum(0), (m + 8) * 2.0 ** -24 * t.abs().sum(0) + 1e-30, what + " dgamma")
    if want[2]:
        check(dbe, dy.d().sum(0), m * 2.0 ** -24 * dy.d().abs().sum(0) + 1e-30, what + " dbeta")

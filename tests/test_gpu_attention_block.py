"""The example attention block: its forward pass and all gradients against FP64
autograd on the same BF16 weights, and tokens decoded over its cache against the
whole sequence at once."""

from __future__ import annotations

import math
import os
import sys

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def at():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import attention

    attention.tg.build()
    attention.tg.load()
    return attention


def reference(at, block, x, lengths, dy=None):
    """(y, dx, gradients) in FP64."""
    p = {k: v.double().requires_grad_() for k, v in block.w.items()}
    a = x.double().requires_grad_()
    h, kv, d = block.h, block.kv, block.dim
    mean = a.mean(1, keepdim=True)
    var = ((a - mean) ** 2).mean(1, keepdim=True)
    n = (a - mean) / torch.sqrt(var + 1e-5) * p["gamma"] + p["beta"]
    qkv = (n @ p["Wqkv"].t()).view(-1, h + 2 * kv, d)
    pos = torch.cat([torch.arange(m, device="cuda") for m in lengths]).double()
    f = at.BASE ** (-torch.arange(0, d, 2, dtype=torch.float64, device="cuda") / d)
    c, s = torch.cos(pos[:, None] * f)[:, None], torch.sin(pos[:, None] * f)[:, None]
    lo, hi = qkv[:, : h + kv, : d // 2], qkv[:, : h + kv, d // 2:]
    turned = torch.cat([lo * c - hi * s, lo * s + hi * c], -1)
    out, at0 = [], 0
    for m in lengths:
        q, k = turned[at0: at0 + m, :h], turned[at0: at0 + m, h:].repeat_interleave(h // kv, 1)
        v = qkv[at0: at0 + m, h + kv:].repeat_interleave(h // kv, 1)
        sc = torch.einsum("ihd,jhd->hij", q, k) / math.sqrt(d)
        sc = sc.masked_fill(torch.ones(m, m, dtype=torch.bool, device="cuda").triu(1), -math.inf)
        out.append(torch.einsum("hij,jhd->ihd", torch.softmax(sc, -1), v).reshape(m, h * d))
        at0 += m
    y = a + torch.cat(out) @ p["Wo"].t() + p["bo"]
    if dy is None:
        return y.detach()
    (y * dy.double()).sum().backward()
    return y.detach(), a.grad, {k: v.grad for k, v in p.items()}


# Norm-wise: each quantity passes at most ten roundings to BF16 on its way (n, QKV,
# its turn, P, O; dO, dS, dQ, dK, dV, their turn, dn, the result), 2^-8 each at worst.
LIMIT = 10 * 2.0 ** -8


def close(got, ref, what):
    err = float((got.double() - ref).norm() / ref.norm())
    assert err <= LIMIT, f"{what}: {err}"


@pytest.mark.parametrize("lengths,h,kv,d", [([1], 2, 1, 64), ([5, 130, 0, 64], 4, 2, 64), ([300, 77], 6, 2, 128),
                                            ([33, 200], 5, 5, 80)])
def test_block_against_autograd(at, lengths, h, kv, d):
    torch.manual_seed(5)
    block = at.Attention(h, kv, d, seed=3)
    block.w["gamma"] += 0.2 * torch.randn(h * d, device="cuda")
    block.w["beta"] += 0.2 * torch.randn(h * d, device="cuda")
    block.w["bo"] += 0.2 * torch.randn(h * d, device="cuda")
    m = sum(lengths)
    x, dy = (torch.randn(m, h * d, device="cuda").to(torch.bfloat16) for _ in range(2))
    starts = at.starts_of(lengths)
    pos = torch.cat([torch.arange(n, device="cuda") for n in lengths])
    y = block.forward(x, starts, pos, max(lengths), train=True)
    dx = block.backward(dy)
    want_y, want_dx, want = reference(at, block, x, lengths, dy)
    close(y, want_y, "y")
    close(dx, want_dx, "dx")
    for k, v in want.items():
        close(block.grads[k], v, "d" + k)
    assert torch.equal(block.forward(x, starts, pos, max(lengths)), y)  # serving gives what training computed


def test_decoding_continues_the_prompt(at):
    """Token by token over the cache: the rows of the whole sequences at once."""
    torch.manual_seed(6)
    block = at.Attention(8, 2, 64, seed=4)
    full, prompt = [40, 300, 9], [33, 290, 1]
    xs = [torch.randn(n, 512, device="cuda").to(torch.bfloat16) for n in full]
    want = reference(at, block, torch.cat(xs), full).split(full)
    y = block.prefill(torch.cat([x[:n] for x, n in zip(xs, prompt)]), prompt, 320)
    for got, ref, n in zip(y.split(prompt), want, prompt):
        close(got, ref[:n], "prompt")
    for i in range(7):
        got = block.decode(torch.stack([x[n + i] for x, n in zip(xs, prompt)]))
        close(got, torch.stack([ref[n + i] for ref, n in zip(want, prompt)]), f"token {i}")


def test_full_cache_is_refused(at):
    """A sequence that has filled its rows of the cache: an error before anything is
    written, and no other sequence's keys and values change.  Nor is a prompt taken that
    is longer than its rows."""
    torch.manual_seed(7)
    block = at.Attention(4, 2, 64, seed=5)
    x = torch.randn(9, 256, device="cuda").to(torch.bfloat16)
    with pytest.raises(ValueError):
        block.prefill(x, [7, 2], 6)
    block.prefill(x, [7, 2], 8)
    block.decode(x[:2])
    kept, lengths = block.cache.clone(), block.lengths.clone()
    for _ in range(2):
        with pytest.raises(ValueError):
            block.decode(x[:2])
    torch.cuda.synchronize()
    # (rows that nothing was written to hold anything)
    assert torch.equal(block.cache.view(torch.int16), kept.view(torch.int16))
    assert torch.equal(block.lengths, lengths)

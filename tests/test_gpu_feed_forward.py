"""The example feed-forward block: its forward pass and all gradients against
FP64 autograd on the same BF16 weights, and a short training run."""

from __future__ import annotations

import os
import sys

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ff():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import feed_forward

    feed_forward.tg.build()
    feed_forward.tg.load()
    return feed_forward


def reference(block, x, dy):
    """(y, dx, gradients) in FP64."""
    p = {k: v.double().requires_grad_() for k, v in block.w.items()}
    a = x.double().requires_grad_()
    mean = a.mean(1, keepdim=True)
    var = ((a - mean) ** 2).mean(1, keepdim=True)
    n = (a - mean) / torch.sqrt(var + 1e-5) * p["gamma"] + p["beta"]
    g, u = n @ p["Wg"].t(), n @ p["Wu"].t()
    y = a + (g / (1 + torch.exp(-g)) * u) @ p["W2"].t() + p["b2"]
    (y * dy.double()).sum().backward()
    return y.detach(), a.grad, {k: v.grad for k, v in p.items()}


@pytest.mark.parametrize("m,d,f", [(1, 64, 128), (37, 200, 333), (300, 264, 520), (1000, 512, 1536)])
def test_block_against_autograd(ff, m, d, f):
    """Norm-wise: each quantity passes at most six roundings to BF16 on its
    way (n, G or U, H, dH, dG, the result), 2^-8 each at worst."""
    torch.manual_seed(5)
    block = ff.FeedForward(d, f, seed=3)
    block.master["gamma"] += 0.2 * torch.randn(d, device="cuda")
    block.master["beta"] += 0.2 * torch.randn(d, device="cuda")
    block.master["b2"] += 0.2 * torch.randn(d, device="cuda")
    block.refresh()
    x = torch.randn(m, d, device="cuda").to(torch.bfloat16)
    dy = torch.randn(m, d, device="cuda").to(torch.bfloat16)
    y = block.forward(x, train=True)
    dx = block.backward(dy)
    want_y, want_dx, want = reference(block, x, dy)
    limit = 6 * 2.0 ** -8

    def close(got, ref, what):
        err = float((got.double() - ref).norm() / ref.norm())
        assert err <= limit, f"{what}: {err}"

    close(y, want_y, "y")
    close(dx, want_dx, "dx")
    for k, v in want.items():
        close(block.grads[k], v, "d" + k)
    assert torch.equal(block.forward(x), y)  # serving gives what training computed


def test_training_reduces_the_loss(ff):
    torch.manual_seed(6)
    teacher, student = ff.FeedForward(128, 256, seed=1), ff.FeedForward(128, 256, seed=2, scale=0.5)
    x = torch.randn(512, 128, device="cuda").to(torch.bfloat16)
    target = teacher.forward(x)
    losses = [float(student.step(x, target, rate=0.2 * 128)) for _ in range(30)]
    assert losses[-1] < 0.5 * losses[0], losses

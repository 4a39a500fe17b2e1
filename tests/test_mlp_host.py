"""Argument checks of the feed-forward operators (no GPU): every refusal comes
back before CUDA is touched, empty problems launch nothing, and the workspace
queries follow the documented rules."""

from __future__ import annotations

import ctypes

import pytest


@pytest.fixture(scope="module", params=["module", "ctypes"])
def tg(request):
    """Through the marshalling module, and through ctypes alone."""
    import dense_gemm_epilogue_gb300 as tg

    tg.build()
    tg.load()
    kept = tg._call
    if request.param == "ctypes":
        tg._call = None
    elif kept is None:
        pytest.skip("built without Python's headers")
    yield tg
    tg._call = kept


A = 1 << 20  # an aligned non-NULL address; never dereferenced here
INVALID, UNSUPPORTED, OK = 1, 2, 0


def linear(tg, **over):
    a = dict(M=64, N=96, K=128, X=A, ldx=128, W=A, ldw=128, bias=A, act="silu", R=A, ldr=96, Y=A,
             ldy=96, Z=A, ldz=96, dtype="bf16", workspace=None, stream=None)
    a.update(over)
    return tg.tg_linear(*a.values())


@pytest.mark.parametrize("over", [
    dict(M=-1), dict(N=-1), dict(K=-1), dict(M=1 << 31), dict(N=1 << 40), dict(K=1 << 31),
    dict(ldx=127), dict(ldw=127), dict(ldy=95), dict(ldr=95), dict(ldz=95),
    dict(X=None), dict(W=None), dict(Y=None), dict(X=A + 1), dict(W=A + 1), dict(Y=A + 1),
    dict(R=A + 1), dict(Z=A + 1), dict(bias=A + 2), dict(act=4), dict(act=-1), dict(dtype="tf32"),
    dict(dtype="e4m3"), dict(dtype=9), dict(workspace=(None, -1)),
    dict(ldx=129),                             # rows that need a repack, without a workspace
    dict(ldx=129, workspace=(A, 128)),         # one too small
    dict(ldx=129, workspace=(A + 8, 1 << 20)),  # one not aligned
    dict(X=A + 2, ldx=128),
])
def test_linear_refuses(tg, over):
    assert linear(tg, **over) == INVALID


def test_linear_empty_outputs(tg):
    assert linear(tg, M=0, X=None, Y=None, R=None, Z=None) == OK
    assert linear(tg, N=0, W=None, Y=None, R=None, Z=None, bias=None) == OK


def linear_backward(tg, **over):
    a = dict(M=64, N=96, K=128, dY=A, lddy=96, X=A, ldx=128, W=A, ldw=128, Z=A, ldz=96, act="relu",
             dX=A, lddx=128, dW=A, lddw=128, dw_dtype="bf16", db=A, dtype="bf16", workspace=None,
             stream=None)
    a.update(over)
    return tg.tg_linear_backward(*a.values())


@pytest.mark.parametrize("over", [
    dict(M=-1), dict(K=-5), dict(N=1 << 31), dict(lddy=95), dict(ldx=127), dict(ldw=127),
    dict(ldz=95), dict(lddx=127), dict(lddw=127), dict(dY=None), dict(X=None), dict(W=None),
    dict(Z=None), dict(dw_dtype="fp16"), dict(dw_dtype=7), dict(dtype="f32x"), dict(db=A + 1),
    dict(dW=A + 2, dw_dtype="f32"), dict(dX=A + 1), dict(act=9), dict(workspace=(None, -1)),
] )
def test_linear_backward_refuses(tg, over):
    if over.get("dtype") == "f32x":
        over = dict(dtype=2)
    assert linear_backward(tg, **over) == INVALID


def test_linear_backward_wants_nothing(tg):
    assert linear_backward(tg, dX=None, dW=None, db=None) == OK
    assert linear_backward(tg, dX=None, dW=None, db=None, X=None, W=None) == OK
    assert linear_backward(tg, M=0, dY=None, X=None, Z=None, dX=None, dW=None, db=None) == OK


def gated(tg, **over):
    a = dict(M=64, N=96, K=128, X=A, ldx=128, Wg=A, ldwg=128, Wu=A, ldwu=128, act="silu", H=A,
             ldh=96, G=A, ldg=96, U=A, ldu=96, dtype="fp16", workspace=None, stream=None)
    a.update(over)
    return tg.tg_gated(*a.values())


@pytest.mark.parametrize("over", [
    dict(M=-1), dict(ldx=127), dict(ldwg=127), dict(ldwu=127), dict(ldh=95), dict(ldg=95),
    dict(ldu=95), dict(X=None), dict(Wg=None), dict(Wu=None), dict(H=None), dict(Wg=A + 1),
    dict(G=A + 1), dict(act=4), dict(dtype="e5m2"), dict(ldwg=129), dict(Wu=A + 2),
])
def test_gated_refuses(tg, over):
    assert gated(tg, **over) == INVALID


def test_gated_empty_outputs(tg):
    assert gated(tg, M=0, X=None, H=None, G=None, U=None) == OK
    assert gated(tg, N=0, Wg=None, Wu=None, H=None, G=None, U=None) == OK


def gated_backward(tg, **over):
    a = dict(M=64, N=96, K=128, dH=A, lddh=96, X=A, ldx=128, Wg=A, ldwg=128, Wu=A, ldwu=128, G=A,
             ldg=96, U=A, ldu=96, act="silu", dX=A, lddx=128, dWg=A, lddwg=128, dWu=A, lddwu=128,
             dw_dtype="bf16", dtype="bf16", workspace=None, stream=None)
    a.update(over)
    return tg.tg_gated_backward(*a.values())


@pytest.mark.parametrize("over", [
    dict(N=-1), dict(lddh=95), dict(ldg=95), dict(ldu=95), dict(ldwg=127), dict(lddx=127),
    dict(lddwg=127), dict(lddwu=127), dict(dH=None), dict(G=None), dict(U=None), dict(X=None),
    dict(Wg=None), dict(Wu=None), dict(dw_dtype="fp16"), dict(dtype="tf32"), dict(dWu=A + 1),
    dict(act=-2),
])
def test_gated_backward_refuses(tg, over):
    assert gated_backward(tg, **over) == INVALID


def test_gated_backward_wants_nothing(tg):
    assert gated_backward(tg, dX=None, dWg=None, dWu=None) == OK


def norm(tg, **over):
    a = dict(M=8, N=100, X=A, ldx=100, gamma=A, beta=A, eps=1e-5, Y=A, ldy=100, mean=A, rstd=A,
             dtype="f32", stream=None)
    a.update(over)
    return tg.tg_layer_norm(*a.values())


@pytest.mark.parametrize("over,status", [
    (dict(M=-1), INVALID), (dict(N=-1), INVALID), (dict(N=0), INVALID), (dict(ldx=99), INVALID),
    (dict(ldy=99), INVALID), (dict(X=None), INVALID), (dict(Y=None), INVALID),
    (dict(X=A + 2), INVALID), (dict(gamma=A + 1), INVALID), (dict(beta=A + 2), INVALID),
    (dict(mean=A + 2), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(dtype=3), INVALID), (dict(N=65537, ldx=65537, ldy=65537), UNSUPPORTED),
    (dict(M=0, X=None, Y=None), OK),
])
def test_norm_statuses(tg, over, status):
    assert norm(tg, **over) == status


def norm_backward(tg, **over):
    a = dict(M=8, N=100, dY=A, lddy=100, X=A, ldx=100, gamma=A, mean=A, rstd=A, dX=A, lddx=100,
             dgamma=A, dbeta=A, dtype="bf16", workspace=None, stream=None)
    a.update(over)
    return tg.tg_layer_norm_backward(*a.values())


@pytest.mark.parametrize("over,status", [
    (dict(M=-1), INVALID), (dict(N=0), INVALID), (dict(lddy=99), INVALID), (dict(ldx=99), INVALID),
    (dict(lddx=99), INVALID), (dict(dY=None), INVALID), (dict(X=None), INVALID),
    (dict(mean=None), INVALID), (dict(rstd=None), INVALID), (dict(dX=A + 1), INVALID),
    (dict(dgamma=A + 2), INVALID), (dict(dtype=5), INVALID), (dict(workspace=(None, -4)), INVALID),
    (dict(N=70000, lddy=70000, ldx=70000, lddx=70000), UNSUPPORTED),
    (dict(dX=None, dgamma=None, dbeta=None), OK),
    (dict(M=0, N=0, dY=None, X=None, mean=None, rstd=None, dX=None), OK),
])
def test_norm_backward_statuses(tg, over, status):
    assert norm_backward(tg, **over) == status


def test_forward_workspace_rules(tg):
    """Nothing for rows that TMA can address; a padded copy of each operand
    that it cannot; a single row's stride does not matter."""
    size = tg.tg_linear_workspace_bytes
    assert size(64, 96, 128, A, 128, A, 128, "bf16") == 0
    assert size(64, 96, 120, A, 128, A, 120, "bf16") == 0
    x_only = size(64, 96, 121, A, 121, A, 128, "bf16")
    assert x_only >= 64 * 128 * 2 and x_only % 16 == 0
    both = size(64, 96, 121, A, 121, A, 121, "bf16")
    assert both >= x_only + 96 * 128 * 2
    assert size(1, 96, 121, A, 121, A, 128, "bf16") == 0
    assert size(1, 96, 121, A + 2, 121, A, 128, "bf16") > 0
    assert size(64, 96, 0, None, 0, None, 0, "bf16") == 0
    assert size(-1, 96, 128, A, 128, A, 128, "bf16") == -1
    assert size(64, 96, 128, A, 127, A, 128, "bf16") == -1
    assert size(64, 96, 128, A, 128, A, 128, "tf32") == -1
    g = tg.tg_gated_workspace_bytes
    assert g(64, 96, 128, A, 128, A, 128, A, 128, "fp16") == 0
    assert g(64, 96, 128, A, 128, A, 129, A, 129, "fp16") >= 2 * 96 * 128 * 2
    assert g(64, 96, 128, A, 128, A, 128, A, 127, "fp16") == -1


def test_gated_backward_workspace_holds_both_gradients(tg):
    size = tg.tg_gated_backward_workspace_bytes
    assert size(64, 96, 128, A, 128, A, 128, A, 128, "bf16") >= 2 * 64 * 96 * 2
    assert size(0, 96, 128, A, 128, A, 128, A, 128, "bf16") == 0
    assert size(64, 96, 128, A, 127, A, 128, A, 128, "bf16") == -1


def test_act_names(tg):
    assert tg.ACT_CODES == {"none": 0, "relu": 1, "silu": 2, "gelu_tanh": 3}
    with pytest.raises(KeyError):
        linear(tg, act="swish")


def test_argument_kinds(tg):
    """Integers, index-like objects, tensors and None; everything else is a
    TypeError naming the type."""
    class Seven:
        def __index__(self):
            return 7

    assert norm(tg, M=0, N=Seven(), ldx=Seven(), ldy=Seven(), X=None, Y=None) == OK
    with pytest.raises(TypeError):
        linear(tg, X="not a pointer")
    with pytest.raises(TypeError):
        linear(tg, stream="not a stream")
    with pytest.raises((TypeError, ctypes.ArgumentError)):
        linear(tg, K=1.5)

    class Stream:
        cuda_stream = 0

    assert linear(tg, M=0, X=None, Y=None, R=None, Z=None, stream=Stream()) == OK


def test_tensors_as_pointers_and_workspaces(tg):
    torch = pytest.importorskip("torch")
    x = torch.zeros(64, 129, dtype=torch.bfloat16)
    ws = torch.empty(64, dtype=torch.uint8)
    assert linear(tg, M=0, X=x, ldx=129, workspace=ws) == OK
    assert linear(tg, X=x, ldx=129, workspace=ws) == INVALID  # a workspace too small

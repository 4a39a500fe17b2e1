"""Every schedule of the feed-forward products on the GPU (tests/mlp_schedules.py
lists a size for each), against the FP64 definitions."""

from __future__ import annotations

import pytest

from mlp_schedules import SCHEDULES, schedule

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


def run(tg, product, m, n, k, dtype, f32):
    if product == "linear":
        h.check_linear(tg, m, n, k, dtype, "gelu_tanh", bias=True, residual=True, save=f32)
    elif product == "gated":
        h.check_gated(tg, m, n, k, dtype, "silu", save=f32)
    elif product.startswith("linear"):
        h.check_linear_backward(tg, m, n, k, dtype, "silu", dw="f32" if f32 else "same")
    else:
        h.check_gated_backward(tg, m, n, k, dtype, "gelu_tanh", dw="f32" if f32 else "same")


@pytest.mark.parametrize("product,m,n,k,shape,order,split", SCHEDULES)
def test_schedule(tg, product, m, n, k, shape, order, split):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    text = tg.tg_product_plan_describe(product, m, n, k)
    if sms == 152:
        assert schedule(text, sms) == (shape, order, split), text
    i = SCHEDULES.index((product, m, n, k, shape, order, split))
    run(tg, product, m, n, k, ("bf16", "fp16")[i % 2], i // 2 % 2 == 1)
    if order == "ticket":  # the counter must be back at zero
        run(tg, product, m, n, k, ("fp16", "bf16")[i % 2], i // 2 % 2 == 0)
    torch.cuda.empty_cache()

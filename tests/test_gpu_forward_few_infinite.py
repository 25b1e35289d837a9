"""moe_forward_few with an infinity beside finite values that fp16 does not hold: the sums are the
infinity that the layer's definition gives, not NaN of infinities of both signs."""
import pytest
import torch

from tests.gpu_helpers import require_gpu
from tests.test_gpu_forward_few import Layer, call
from tests.train_helpers import gen

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module")
def moe():
    require_gpu()
    from grouped_gemm_serving_gb300 import moe as m
    assert m.moe_get_device_error() == 0
    yield m
    assert m.moe_get_device_error() == 0


def positive(dtype, E, H, I):
    """Every weight positive."""
    layer = Layer(gen(H + I), dtype, E, H, I)
    for w in (layer.W1, layer.W2):
        w.view(torch.uint8 if dtype == "fp8" else torch.int16).bitwise_and_(0x7F if dtype == "fp8" else 0x7FFF)
        small = w.float() < 0.001
        w[:] = torch.where(small, torch.tensor(0.5), w.float()).to(w.dtype)
    return layer


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("T", [2, 12, 40])
@pytest.mark.parametrize("other", [-1.0, -70000.0, -1e30])
def test_in_x(moe, dtype, T, other):
    """x: infinity once, negative elsewhere.  Gate and up are infinite, h and every sum too."""
    E, H, I = 2, 384, 256
    layer = positive(dtype, E, H, I)
    x = torch.full((T, H), other, dtype=torch.bfloat16, device="cuda")
    x[0] = 1.0
    x[1:, 200] = INF
    ids = (torch.arange(T, device="cuda", dtype=torch.int32) % E)[:, None].contiguous()
    out, _, _ = call(moe, layer, x, ids=ids, w=torch.ones(T, 1, device="cuda"))
    assert bool(out[0].isfinite().all()) and bool((out[0] != 0).all())
    assert bool((out[1:] == INF).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("T", [2, 12, 40])
@pytest.mark.parametrize("sign", [1, -1])
def test_in_h(moe, dtype, T, sign):
    """x finite.  Even features overflow to an infinite h, odd ones are large and of the other sign."""
    E, H, I = 1, 256, 256
    layer = positive(dtype, E, H, I)
    large, small = (448.0, 2.0 ** -9) if dtype == "fp8" else (1e18, 1e3)   # h: past fp32; past fp16 (with FP8's scale 1e31)
    layer.W1[:, 0:I:2] = large
    layer.W1[:, 1:I:2] = small
    layer.W1[:, I::2] = sign * large
    layer.W1[:, I + 1::2] = -sign * small
    if dtype == "fp8":
        layer.s1[:] = 1e16
    x = torch.ones(T, H, dtype=torch.bfloat16, device="cuda")
    out, _, _ = call(moe, layer, x, ids=torch.zeros(T, 1, dtype=torch.int32, device="cuda"), w=torch.ones(T, 1, device="cuda"))
    assert bool((out == sign * INF).all())

"""moe_forward_few where rows of x are so long that a chunk holds five to seven of an expert's,
with several chunks an expert."""
import pytest
import torch

from tests.gpu_helpers import require_gpu
from tests.test_gpu_forward_few import Layer, call, check
from tests.train_helpers import gen, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    require_gpu()
    from grouped_gemm_serving_gb300 import moe as m
    assert m.moe_get_device_error() == 0
    yield m
    assert m.moe_get_device_error() == 0


@pytest.mark.parametrize("dtype,T,E,k,H,I", [
    ("bf16", 64, 4, 2, 7168, 72), ("bf16", 16, 2, 2, 5760, 136), ("bf16", 8, 2, 2, 7168, 264), ("bf16", 33, 3, 1, 72, 7168),
    ("fp8", 64, 4, 2, 7168, 128), ("fp8", 16, 2, 2, 5120, 256), ("fp8", 7, 2, 2, 7168, 384), ("fp8", 50, 3, 2, 128, 7168),
])
def test_several_chunks_an_expert(moe, dtype, T, E, k, H, I):
    g = gen(T + H)
    layer = Layer(g, dtype, E, H, I)
    x, logits = randn(g, T, H), torch.randn(T, E, generator=g, device="cuda")
    out, ids, w = call(moe, layer, x, logits=logits, k=k, guard=2)
    check(layer, x, ids, w, out)
    for _ in range(5):
        assert torch.equal(call(moe, layer, x, logits=logits, k=k)[0], out)

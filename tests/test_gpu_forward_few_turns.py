"""moe_forward_few where experts have several chunks of rows, which take turns over the features, and many
units a block: every unit once, the same bits from every pass and replay."""
import pytest
import torch

from tests.gpu_helpers import require_gpu
from tests.test_gpu_forward_few import Layer, call, check, gen, randn, workspace

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    require_gpu()
    from grouped_gemm_serving_gb300 import moe as m
    yield m
    assert m.moe_get_device_error() == 0


# Rows of the most picked experts fill two to four chunks.
CASES = [
    ("bf16", 17, 64, 8, 1024, 1024),
    ("bf16", 64, 40, 4, 1000, 1368),   # columns that fill no tile, features that fill no unit
    ("bf16", 33, 24, 6, 2880, 2088),
    ("fp8", 64, 96, 8, 1152, 640),     # a block of scales that several blocks' runs share
    ("fp8", 40, 48, 2, 2048, 1408),
]


def skewed(g, T, E):
    """The first eight experts are picked most: several chunks of rows each."""
    logits = torch.randn(T, E, generator=g, device="cuda")
    logits[:, :8] += 1.5
    return logits


@pytest.mark.parametrize("dtype,T,E,k,H,I", CASES)
def test_layer(moe, dtype, T, E, k, H, I):
    g = gen(T + E + H)
    layer = Layer(g, dtype, E, H, I)
    x, logits = randn(g, T, H), skewed(g, T, E)
    out, ids, w = call(moe, layer, x, logits=logits, k=k, guard=2)
    check(layer, x, ids, w, out)
    for _ in range(10):
        assert torch.equal(call(moe, layer, x, logits=logits, k=k)[0], out)


def test_replays(moe):
    """Two calls of a graph behind one another, over one workspace, replayed with other inputs."""
    T, E, k, H, I = 20, 64, 8, 1024, 1024
    g = gen(1)
    layer = Layer(g, "bf16", E, H, I)
    x, logits, out = randn(g, T, H), skewed(g, T, E), torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    args = moe.forward_args(dtype=moe.MOE_BF16, T=T, E=E, k=k, H=H, I=I, x=x, W1=layer.W1, W2=layer.W2, out=out, logits=logits)
    n = moe.moe_forward_few_workspace_size(args)
    ws = workspace(n)
    moe.moe_forward_few(args, ws, n)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(2):
            moe.moe_forward_few(args, ws, n)
    for seed in (2, 3, 4):
        logits.copy_(skewed(gen(seed), T, E))
        x.copy_(randn(gen(seed + 10), T, H))
        out.fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        want, _, _ = call(moe, layer, x, logits=logits, k=k)
        assert torch.equal(got, want)

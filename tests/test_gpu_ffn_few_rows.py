"""moe_ffn_forward around the row count where it changes kernels, and rows of one
expert that hold infinities and NaN next to another expert's."""
import pytest
import torch

from tests.gpu_helpers import require_gpu
from tests.train_helpers import HALF, NOISE, gen, randn, rounded, within, workspace

pytestmark = pytest.mark.gpu
ACC = 2.0 ** -12


@pytest.fixture(scope="module")
def moe():
    require_gpu()
    from grouped_gemm_serving_gb300 import moe as m
    return m


@pytest.mark.parametrize("H,I", [(8, 8), (2880, 136), (264, 1000), (1000, 24)])
@pytest.mark.parametrize("counts,spare", [([1], 0), ([8], 0), ([9, 0, 1], 2), ([0, 17, 3, 5], 0), ([32], 0), ([1] * 31, 1),
                                          ([16, 0, 16], 0), ([33], 0), ([25, 0, 8], 0)])
def test_forward(moe, counts, spare, H, I):
    g = gen(sum(counts) + H)
    E, P = len(counts), sum(counts)
    M = P + spare
    ends = torch.tensor([0] + counts).cumsum(0)
    x = randn(g, M, H)
    x[P:] = float("nan")
    W1, W2 = randn(g, E, 2 * I, H, std=H ** -0.5), randn(g, E, H, I, std=I ** -0.5)
    Y1, h, y = (torch.full((M, n), 7, dtype=torch.bfloat16, device="cuda") for n in (2 * I, I, H))
    moe.moe_ffn_forward(x, W1, W2, ends.to(torch.int32).cuda(), E, M, H, I, Y1, h, y)
    assert moe.moe_get_device_error() == 0
    for e in range(E):
        a, b = int(ends[e]), int(ends[e + 1])
        z = x[a:b].double() @ W1[e].double().t()
        zs = (x[a:b].double().square() @ W1[e].double().t().square()).sqrt()
        within(Y1[a:b], z, rounded(z, torch.bfloat16) + ACC * zs)
        hh = torch.nn.functional.silu(z[:, :I]) * z[:, I:]
        ref = hh @ W2[e].double().t()
        spread = (hh.square() @ W2[e].double().t().square()).sqrt()
        within(y[a:b], ref, rounded(ref, torch.bfloat16) + (NOISE + ACC) * spread)
    assert bool((y[P:] == 0).all()) and bool((h[P:] == 0).all()) and bool((Y1[P:] == 0).all())
    # without the kept pre-activations, and again: the same bits
    for _ in range(2):
        y2 = torch.empty_like(y)
        moe.moe_ffn_forward(x, W1, W2, ends.to(torch.int32).cuda(), E, M, H, I, None, h, y2)
        assert torch.equal(y2, y)


def test_invalid_offsets_are_reported(moe):
    x, W1, W2 = (torch.zeros(*s, dtype=torch.bfloat16, device="cuda") for s in ((8, 64), (2, 64, 64), (2, 64, 32)))
    y, h = torch.full_like(x, 7), torch.empty(8, 32, dtype=torch.bfloat16, device="cuda")
    for bad in ([0, 5, 9], [0, 5, 4], [1, 5, 8]):
        moe.moe_ffn_forward(x, W1, W2, torch.tensor(bad, dtype=torch.int32, device="cuda"), 2, 8, 64, 32, None, h, y)
        assert moe.moe_get_device_error() == moe.MOE_DEVERR_OFFSETS
        assert bool((y == 7).all())


@pytest.mark.parametrize("rows", [3, 70])
def test_another_experts_nan_stays_there(moe, rows):
    """Expert 1's rows hold NaN and infinities: expert 0's outputs and gradients are what they are without them."""
    H, I, E = 136, 72, 2
    g = gen(rows)
    off = torch.tensor([0, rows, 2 * rows], dtype=torch.int32, device="cuda")
    M = 2 * rows
    x, W1, W2, dy = randn(g, M, H), randn(g, E, 2 * I, H), randn(g, E, H, I), randn(g, M, H)
    outs = []
    for fill in (None, float("nan"), float("inf")):
        x1, dy1 = x.clone(), dy.clone()
        if fill is not None:
            x1[rows:] = fill
            dy1[rows:] = fill
        Y1, h, y = torch.empty(M, 2 * I, dtype=x.dtype, device="cuda"), torch.empty(M, I, dtype=x.dtype, device="cuda"), torch.empty_like(x)
        moe.moe_ffn_forward(x1, W1, W2, off, E, M, H, I, Y1, h, y)
        dx, dW1, dW2 = torch.empty_like(x), torch.empty_like(W1), torch.empty_like(W2)
        n = moe.moe_ffn_backward_workspace_size(E, M, H, I)
        moe.moe_ffn_backward(x1, W1, W2, Y1, dy1, off, E, M, H, I, dx, dW1, dW2, workspace(n), n)
        outs.append((y[:rows], Y1[:rows], dx[:rows], dW1[0], dW2[0]))
    for other in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(outs[0], other))

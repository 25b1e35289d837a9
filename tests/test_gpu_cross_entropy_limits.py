"""moe_cross_entropy_forward / _backward where labels are no labels and where
sizes come near what 32 bits count."""
import pytest
import torch

from tests.gpu_helpers import require_gpu
from tests.train_helpers import gen, randn, workspace

pytestmark = pytest.mark.gpu
IGNORE = -100


@pytest.fixture(scope="module")
def moe():
    require_gpu()
    from grouped_gemm_serving_gb300 import moe as m
    yield m
    torch.cuda.empty_cache()


def _run(moe, x, W, labels, dloss):
    (T, H), V = x.shape, W.shape[0]
    loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    n = moe.moe_cross_entropy_forward_workspace_size(T, H, V)
    moe.moe_cross_entropy_forward(x, W, labels, T, H, V, IGNORE, loss, lse, workspace(n), n)
    first = moe.moe_get_device_error()
    dx, dW = torch.full_like(x, 7), torch.full_like(W, 7)
    n = moe.moe_cross_entropy_backward_workspace_size(T, H, V)
    moe.moe_cross_entropy_backward(x, W, labels, lse, dloss, T, H, V, IGNORE, dx, dW, workspace(n), n)
    return (loss, lse, dx, dW), (first, moe.moe_get_device_error())


@pytest.mark.parametrize("T", [100, 140, 700])
@pytest.mark.parametrize("at", ["V", "last", "negative"])
def test_invalid_labels_count_as_ignored_whatever_their_rows_hold(moe, T, at):
    """Rows with a label outside [0, V) that hold NaN or infinities: reported, zero loss and gradients, and
    every other value as if the label were the ignored one."""
    g = gen(T)
    H, V = 72, 700
    bad = {"V": V, "last": 2 ** 31 - 1, "negative": -1}[at]
    x, W = randn(g, T, H), randn(g, V, H, std=0.1)
    labels = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    out = torch.zeros(T, dtype=torch.bool, device="cuda")
    out[::3] = True
    dloss = torch.rand(T, generator=g, device="cuda")
    want, err = _run(moe, x, W, torch.where(out, IGNORE, labels), dloss)
    assert err == (0, 0)
    for fill in (0.0, float("nan"), float("inf")):
        x1, d1 = x.clone(), dloss.clone()
        x1[out] = fill
        d1[out] = fill
        got, err = _run(moe, x1, W, torch.where(out, bad, labels), d1)
        assert err == (moe.MOE_DEVERR_LABEL, moe.MOE_DEVERR_LABEL)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1][~out], want[1][~out])
        assert torch.equal(got[2], want[2]) and torch.equal(got[3], want[3])
        assert bool((got[2][out] == 0).all())

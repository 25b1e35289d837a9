"""moe_ffn_forward / moe_ffn_backward against the block's formulas in 64 bits:
one row, one expert, idle experts, ragged rows across every tile edge, feature
counts that leave half tiles, NaN in the rows of no expert."""
import pytest
import torch

from tests.gpu_helpers import require_gpu
from tests.train_helpers import HALF, NOISE, gen, randn, rounded, within, workspace

pytestmark = pytest.mark.gpu
ACC = 2.0 ** -12   # fp32 sums of up to a few thousand terms, of which each addition may lose a unit in 2^23


@pytest.fixture(scope="module")
def moe():
    require_gpu()
    from grouped_gemm_serving_gb300 import moe as m
    return m


CASES = [
    # rows of each expert, spare rows, H, I
    ([1], 0, 8, 8),
    ([4], 3, 2880, 136),
    ([0, 1, 0, 2], 0, 264, 72),
    ([0, 0], 5, 64, 64),
    ([300], 0, 512, 1368),
    ([257, 0, 15, 64, 1, 511, 16], 19, 1000, 328),
    ([33, 31, 130], 1, 136, 2880),
    ([7] * 40 + [0] * 20 + [90], 0, 192, 128),
]


def _make(counts, spare, H, I, seed):
    g = gen(seed)
    E, P = len(counts), sum(counts)
    M = max(1, P + spare)
    ends = torch.tensor([0] + counts).cumsum(0)
    x = randn(g, M, H)
    x[P:] = float("nan")
    W1, W2 = randn(g, E, 2 * I, H, std=H ** -0.5), randn(g, E, H, I, std=I ** -0.5)
    return g, E, P, M, ends.tolist(), ends.to(torch.int32).cuda(), x, W1, W2


def _pieces(counts, ends):
    return [(e, ends[e], ends[e + 1]) for e in range(len(counts)) if counts[e]]


@pytest.mark.parametrize("keep", [True, False])
@pytest.mark.parametrize("counts,spare,H,I", CASES)
def test_forward(moe, counts, spare, H, I, keep):
    g, E, P, M, ends, off, x, W1, W2 = _make(counts, spare, H, I, seed=H + I)
    Y1 = torch.full((M, 2 * I), 7, dtype=torch.bfloat16, device="cuda") if keep else None
    h = torch.full((M, I), 7, dtype=torch.bfloat16, device="cuda")
    y = torch.full((M, H), 7, dtype=torch.bfloat16, device="cuda")
    moe.moe_ffn_forward(x, W1, W2, off, E, M, H, I, Y1, h, y)
    assert moe.moe_get_device_error() == 0
    for e, a, b in _pieces(counts, ends):
        z = x[a:b].double() @ W1[e].double().t()
        zs = (x[a:b].double().square() @ W1[e].double().t().square()).sqrt()
        if keep:
            within(Y1[a:b], z, rounded(z, torch.bfloat16) + ACC * zs)
        hh = torch.nn.functional.silu(z[:, :I]) * z[:, I:]
        ref = hh @ W2[e].double().t()
        spread = (hh.square() @ W2[e].double().t().square()).sqrt()
        within(y[a:b], ref, rounded(ref, torch.bfloat16) + (NOISE + ACC) * spread)
    assert bool((y[P:] == 0).all()) and bool((h[P:] == 0).all()) and (not keep or bool((Y1[P:] == 0).all()))


@pytest.mark.parametrize("counts,spare,H,I", CASES)
def test_backward(moe, counts, spare, H, I):
    g, E, P, M, ends, off, x, W1, W2 = _make(counts, spare, H, I, seed=2 * H + I)
    Y1, dy = randn(g, M, 2 * I), randn(g, M, H)
    Y1[P:] = float("nan")
    dy[P:] = float("nan")
    dx, dW1, dW2 = torch.full_like(x, 7), torch.full_like(W1, 7), torch.full_like(W2, 7)
    n = moe.moe_ffn_backward_workspace_size(E, M, H, I)
    moe.moe_ffn_backward(x, W1, W2, Y1, dy, off, E, M, H, I, dx, dW1, dW2, workspace(n), n)
    assert moe.moe_get_device_error() == 0
    # dh and dY1 may each be rounded to bf16 before the products they enter: at
    # most two independent roundings
    two = 2 ** 0.5 * NOISE + ACC
    for e in range(E):
        a, b = ends[e], ends[e + 1]
        if a == b:
            assert bool((dW1[e] == 0).all()) and bool((dW2[e] == 0).all())
            continue
        z = Y1[a:b].double().requires_grad_()
        h = torch.nn.functional.silu(z[:, :I]) * z[:, I:]
        y = h @ W2[e].double().t()
        dz, = torch.autograd.grad(y, z, dy[a:b].double())
        h = h.detach()
        # dh's own noise reaches dz through the activation's slopes: of dh's size times theirs
        ref = dz @ W1[e].double()
        within(dx[a:b], ref, rounded(ref, torch.bfloat16) + two * (dz.square() @ W1[e].double().square()).sqrt())
        ref = dz.t() @ x[a:b].double()
        within(dW1[e], ref, rounded(ref, torch.bfloat16) + two * (dz.t().square() @ x[a:b].double().square()).sqrt())
        ref = dy[a:b].double().t() @ h
        within(dW2[e], ref, rounded(ref, torch.bfloat16) + (NOISE + ACC) * (dy[a:b].double().t().square() @ h.square()).sqrt())
    assert bool((dx[P:] == 0).all())


def test_forward_equals_the_grouped_gemms(moe):
    g, E, P, M, ends, off, x, W1, W2 = _make([40, 0, 300, 5], 9, 264, 200, seed=1)
    H, I = 264, 200
    y, h = torch.empty_like(x), torch.empty(M, I, dtype=torch.bfloat16, device="cuda")
    Y1 = torch.empty(M, 2 * I, dtype=torch.bfloat16, device="cuda")
    h2, y2 = torch.empty_like(h), torch.empty_like(y)
    moe.moe_grouped_gemm(moe.MOE_BF16, x, None, W1, None, off, E, M, 2 * I, H, moe.MOE_EPI_SWIGLU, h2, None)
    moe.moe_grouped_gemm(moe.MOE_BF16, h2, None, W2, None, off, E, M, H, I, moe.MOE_EPI_STORE, y2, None)
    moe.moe_ffn_forward(x, W1, W2, off, E, M, H, I, Y1, h, y)
    assert torch.equal(h, h2) and torch.equal(y, y2)


def test_some_gradients_only(moe):
    g, E, P, M, ends, off, x, W1, W2 = _make([20, 70], 0, 128, 96, seed=4)
    H, I = 128, 96
    Y1, dy = randn(g, M, 2 * I), randn(g, M, H)
    n = moe.moe_ffn_backward_workspace_size(E, M, H, I)
    ws = workspace(n)
    full = torch.empty_like(x), torch.empty_like(W1), torch.empty_like(W2)
    moe.moe_ffn_backward(x, W1, W2, Y1, dy, off, E, M, H, I, *full, ws, n)
    for i in range(3):
        only = [None, None, None]
        only[i] = torch.empty_like(full[i])
        moe.moe_ffn_backward(x if i == 1 else None, W1, W2, Y1, dy, off, E, M, H, I, *only, ws, n)
        assert torch.equal(only[i], full[i])
    again = [torch.empty_like(t) for t in full]
    moe.moe_ffn_backward(x, W1, W2, Y1, dy, off, E, M, H, I, *again, ws, n)
    assert all(torch.equal(a, b) for a, b in zip(again, full))


def test_saturated_gates(moe):
    """Gates far from zero on both sides: silu is 0 or the gate itself, and nothing is NaN."""
    H, I, M = 64, 64, 16
    g = gen(6)
    Y1 = torch.cat([torch.full((M, I), -3e4, device="cuda"), torch.full((M, I), 2.0, device="cuda")], 1).to(torch.bfloat16)
    Y1[::2, :I] = 3e4
    off = torch.tensor([0, M], dtype=torch.int32, device="cuda")
    x, W1, W2, dy = randn(g, M, H), randn(g, 1, 2 * I, H), randn(g, 1, H, I), randn(g, M, H)
    dx, dW1, dW2 = torch.empty_like(x), torch.empty_like(W1), torch.empty_like(W2)
    n = moe.moe_ffn_backward_workspace_size(1, M, H, I)
    moe.moe_ffn_backward(x, W1, W2, Y1, dy, off, 1, M, H, I, dx, dW1, dW2, workspace(n), n)
    assert all(bool(torch.isfinite(t).all()) for t in (dx, dW1, dW2))
    assert bool((dx[1::2] == 0).all())                                  # closed gates pass nothing back
    ref = dy[::2].double().t() @ torch.full((M // 2, I), 6e4, dtype=torch.float64, device="cuda")
    within(dW2[0], ref, 4 * HALF * dy[::2].double().abs().sum(0)[:, None] * 6e4)


def test_gradient_against_differences(moe):
    """<dW2, D> and <dx, d> are derivatives of <dy, y>: central differences of the whole block in 64 bits."""
    g, E, P, M, ends, off, x, W1, W2 = _make([24], 0, 64, 40, seed=8)
    H, I = 64, 40
    dy = randn(g, M, H)
    Y1, h, y = torch.empty(M, 2 * I, dtype=torch.bfloat16, device="cuda"), torch.empty(M, I, dtype=torch.bfloat16, device="cuda"), torch.empty_like(x)
    moe.moe_ffn_forward(x, W1, W2, off, E, M, H, I, Y1, h, y)
    dx, dW1, dW2 = torch.empty_like(x), torch.empty_like(W1), torch.empty_like(W2)
    n = moe.moe_ffn_backward_workspace_size(1, M, H, I)
    moe.moe_ffn_backward(x, W1, W2, Y1, dy, off, 1, M, H, I, dx, dW1, dW2, workspace(n), n)

    def f(x64, w1, w2):
        z = x64 @ w1.t()
        return ((torch.nn.functional.silu(z[:, :I]) * z[:, I:]) @ w2.t() * dy.double()).sum()

    base = [x.double(), W1[0].double(), W2[0].double()]
    for i, grad in enumerate((dx, dW1[0], dW2[0])):
        d = torch.randn(grad.shape, generator=g, device="cuda").double()
        step = 1e-4
        lo, hi = list(base), list(base)
        lo[i], hi[i] = base[i] - step * d, base[i] + step * d
        want = (f(*hi) - f(*lo)) / (2 * step)
        got = (grad.double() * d).sum()
        # the kept pre-activations, dY1, h and the gradient are each rounded to bf16 (independent errors)
        spread = (grad.double() * d).square().sum().sqrt()
        assert abs(got - want) <= 6 * 4 * HALF * spread


def test_invalid_offsets_are_reported(moe):
    g, E, P, M, ends, off, x, W1, W2 = _make([20, 70], 0, 128, 96, seed=4)
    bad = torch.tensor([0, 60, 50], dtype=torch.int32, device="cuda")
    y, h = torch.full_like(x, 7), torch.empty(M, 96, dtype=torch.bfloat16, device="cuda")
    moe.moe_ffn_forward(x, W1, W2, bad, E, M, 128, 96, None, h, y)
    assert moe.moe_get_device_error() == moe.MOE_DEVERR_OFFSETS
    assert bool((y == 7).all())

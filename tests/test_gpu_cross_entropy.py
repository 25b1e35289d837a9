"""moe_cross_entropy_forward / _backward against the formulas in 64 bits: one
token and one vocabulary row, odd sizes on both sides of every tile edge,
several vocabulary pieces, ignored and invalid labels, logits that overflow
an exponential, more logits than 32 bits count."""
import pytest
import torch

from tests.gpu_helpers import require_gpu
from tests.train_helpers import EPS, HALF, NOISE, gen, randn, rounded, within, workspace

pytestmark = pytest.mark.gpu
IGNORE = -100
UNDER = 2.0 ** -125   # probabilities and gradients below the normal numbers of fp32 and bf16 may be flushed to zero


@pytest.fixture(scope="module")
def moe():
    require_gpu()
    from grouped_gemm_serving_gb300 import moe as m
    return m


def _acc(H):
    """Relative error of a tensor-core sum over H: one addition per 16 terms, each losing at most a unit in 2^23
    of a partial sum, which stays within a few times the root of the summed squares."""
    return 4 * (H / 16 + 16) * 2.0 ** -23


def _make(T, H, V, seed, ignored=0.0, scale=1.0):
    g = gen(seed)
    x, W = randn(g, T, H, std=scale), randn(g, V, H, std=H ** -0.5)
    labels = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    labels[torch.rand(T, generator=g, device="cuda") < ignored] = IGNORE
    return g, x, W, labels


def _forward(moe, x, W, labels, ignore=IGNORE):
    (T, H), V = x.shape, W.shape[0]
    loss, lse = torch.full((T,), 7.0, device="cuda"), torch.full((T,), 7.0, device="cuda")
    n = moe.moe_cross_entropy_forward_workspace_size(T, H, V)
    moe.moe_cross_entropy_forward(x, W, labels, T, H, V, ignore, loss, lse, workspace(n), n)
    return loss, lse


def _backward(moe, x, W, labels, lse, dloss, ignore=IGNORE, want=(True, True)):
    (T, H), V = x.shape, W.shape[0]
    dx = torch.full_like(x, 7) if want[0] else None
    dW = torch.full_like(W, 7) if want[1] else None
    n = moe.moe_cross_entropy_backward_workspace_size(T, H, V)
    moe.moe_cross_entropy_backward(x, W, labels, lse, dloss, T, H, V, ignore, dx, dW, workspace(n), n)
    return dx, dW


CASES = [
    # T, H, V, ignored, scale of x
    (1, 8, 1, 0.0, 1), (1, 2880, 1000, 0.0, 1), (7, 64, 5, 0.0, 1), (16, 264, 257, 0.2, 1), (127, 72, 33, 0.0, 1),
    (128, 128, 4096, 0.1, 1), (129, 1000, 999, 0.5, 1), (256, 200, 2560, 0.0, 30), (257, 512, 5003, 0.3, 1),
    (300, 2880, 32000, 0.0, 4), (1021, 520, 50257, 0.3, 1), (513, 64, 19457, 0.0, 60),
]


def _check_forward(loss, lse, x, W, labels):
    z = x.double() @ W.double().t()
    # the largest spread of a logit's terms in the row bounds every logit's error
    zs = (x.double().square() @ W.double().square().t()).sqrt().amax(1)
    want = torch.logsumexp(z, 1)
    # exp2 is off by 2 units, its argument by a rounding of the largest logit's size
    tol = _acc(x.shape[1]) * zs + 8 * EPS * (1 + want.abs() + z.abs().amax(1))
    within(lse, want, tol)
    at = z.gather(1, labels.clamp(min=0).long()[:, None])[:, 0]
    counts = labels != IGNORE
    within(loss, torch.where(counts, want - at, 0.0), 2 * tol)
    assert bool((loss[~counts] == 0).all())


def _check_backward(dx, dW, x, W, labels, lse, dloss):
    X, M = x.double(), W.double()
    counts = (labels != IGNORE).double()[:, None]
    G = torch.exp(X @ M.t() - lse.double()[:, None])
    G.scatter_add_(1, labels.clamp(min=0).long()[:, None], -torch.ones_like(counts))
    G *= counts
    d = torch.where(labels != IGNORE, dloss.double(), 0.0)[:, None]
    zs = (X.square() @ M.square().t()).sqrt().amax()
    # a probability is off by its logit's error and by that of lse times log2 e
    dp = _acc(x.shape[1]) * zs + 8 * EPS * (1 + lse.double().abs().amax())
    P = (G + (G < 0).double()).abs()           # the probabilities, whose relative error dp is
    if dx is not None:
        ref = d * (G @ M)
        spread = d.abs() * (G.square() @ M.square()).sqrt()
        within(dx, ref, rounded(ref, torch.bfloat16) + (NOISE + _acc(W.shape[0])) * spread + dp * d.abs() * (P @ M.abs())
               + UNDER * M.abs().sum(0))
    if dW is not None:
        ref = (G * d).t() @ X
        spread = ((G * d).square().t() @ X.square()).sqrt()
        within(dW, ref, rounded(ref, torch.bfloat16) + (2 ** 0.5 * NOISE + _acc(x.shape[0])) * spread
               + dp * ((P * d.abs()).t() @ X.abs()) + UNDER * (1 + (d * X).abs().sum(0)))


@pytest.mark.parametrize("T,H,V,ignored,scale", CASES)
def test_forward(moe, T, H, V, ignored, scale):
    _, x, W, labels = _make(T, H, V, T + H + V, ignored, scale)
    loss, lse = _forward(moe, x, W, labels)
    assert moe.moe_get_device_error() == 0
    _check_forward(loss, lse, x, W, labels)


@pytest.mark.parametrize("T,H,V,ignored,scale", CASES)
def test_backward(moe, T, H, V, ignored, scale):
    g, x, W, labels = _make(T, H, V, T + H + V + 1, ignored, scale)
    lse = torch.logsumexp(x.double() @ W.double().t(), 1).float()
    dloss = torch.rand(T, generator=g, device="cuda") * 2 / T
    dloss[labels == IGNORE] = float("nan")     # what does not count is not read into any product
    dx, dW = _backward(moe, x, W, labels, lse, dloss)
    assert moe.moe_get_device_error() == 0
    _check_backward(dx, dW, x, W, labels, lse, dloss)


def test_several_pieces(moe):
    """More vocabulary rows than one piece's gradient holds: dx is summed over the pieces."""
    T, H, V = 4099, 72, 70001
    assert moe.moe_cross_entropy_backward_workspace_size(T, H, V) < T * V * 2
    g, x, W, labels = _make(T, H, V, 5, 0.1)
    loss, lse = _forward(moe, x, W, labels)
    dloss = torch.full((T,), 1.0 / T, device="cuda")
    dx, dW = _backward(moe, x, W, labels, lse, dloss)
    assert moe.moe_get_device_error() == 0
    _check_forward(loss, lse, x, W, labels)
    _check_backward(dx, dW, x, W, labels, lse, dloss)
    for want in ((True, False), (False, True)):
        a, b = _backward(moe, x, W, labels, lse, dloss, want=want)
        assert torch.equal(a, dx) if want[0] else torch.equal(b, dW)


def test_more_logits_than_32_bits(moe):
    T, H, V = 66001, 8, 33001
    g, x, W, labels = _make(T, H, V, 6)
    loss, lse = _forward(moe, x, W, labels)
    dloss = torch.ones(T, device="cuda")
    dx, _ = _backward(moe, x, W, labels, lse, dloss, want=(True, False))
    assert moe.moe_get_device_error() == 0
    rows = torch.cat([torch.arange(0, T, 997), torch.tensor([T - 1])]).cuda()
    _check_forward(loss[rows], lse[rows], x[rows], W, labels[rows])
    _check_backward(dx[rows], None, x[rows], W, labels[rows], lse[rows], dloss[rows])


# The vocabulary goes in pieces and the contraction of each piece in two ranges of
# 64 rows' blocks; the last piece is a single row, so that one range has nothing.
@pytest.mark.parametrize("T,H,V", [(26941, 8, 92417), (19815, 64, 173057)])
def test_a_last_piece_of_one_row(moe, T, H, V):
    g, x, W, labels = _make(T, H, V, 7)
    loss, lse = _forward(moe, x, W, labels)
    dloss = torch.ones(T, device="cuda")
    dx, _ = _backward(moe, x, W, labels, lse, dloss, want=(True, False))
    assert moe.moe_get_device_error() == 0
    rows = torch.cat([torch.arange(0, T, 997), torch.tensor([T - 1])]).cuda()
    _check_backward(dx[rows], None, x[rows], W, labels[rows], lse[rows], dloss[rows])


@pytest.mark.parametrize("T,H,V,c", [(200, 2880, 5000, 18), (64, 4096, 3001, 20), (5, 1000, 1, 20), (300, 512, 2, 8)])
def test_nearly_certain_labels(moe, T, H, V, c):
    """The label's entry of the gradient is minus the little that the other words have."""
    g, x, W, labels = _make(T, H, V, 11)
    x = (W[labels.long()].double() * c).to(torch.bfloat16)
    _, lse = _forward(moe, x, W, labels)
    dloss = torch.ones(T, device="cuda")
    dx, dW = _backward(moe, x, W, labels, lse, dloss)
    assert moe.moe_get_device_error() == 0
    X, M = x.double(), W.double()
    z = X @ M.t()
    G = torch.softmax(z, 1)
    one = torch.nn.functional.one_hot(labels.long(), V).double()
    P = G * (1 - one)
    G = P - one * P.sum(1, keepdim=True)
    # z_l: 2 H / 64 + 6 roundings of a warp's partial sums, independent, each at most EPS of a sum that stays below
    # z_l (six standard deviations stay below 6 EPS of it); lse: its own rounding and a few of the logarithm's
    dg = (6 * z.amax(1, keepdim=True) + 8 * lse.double().abs()[:, None] + 8) * EPS
    # the other words' logits come from the tensor cores
    zs = (X.square() @ M.square().t()).sqrt().amax()
    dp = _acc(H) * zs + 8 * EPS * (1 + z.abs().amax())
    noise = ((NOISE + 2.0 ** -12) * G).square()
    ref = G @ M
    within(dx, ref, rounded(ref, torch.bfloat16) + (noise @ M.square()).sqrt() + dg * M[labels.long()].abs() + dp * (P @ M.abs()))
    ref = G.t() @ X
    within(dW, ref, rounded(ref, torch.bfloat16) + (2 * noise.t() @ X.square()).sqrt() + (one * dg).t() @ X.abs()
           + dp * (P.t() @ X.abs()))


def test_nothing_counts(moe):
    _, x, W, labels = _make(33, 64, 500, 7)
    labels[:] = IGNORE
    loss, lse = _forward(moe, x, W, labels)
    assert bool((loss == 0).all()) and bool(torch.isfinite(lse).all())
    dx, dW = _backward(moe, x, W, labels, lse, torch.full((33,), float("inf"), device="cuda"))
    assert bool((dx == 0).all()) and bool((dW == 0).all())


def test_invalid_labels_are_reported(moe):
    _, x, W, labels = _make(40, 64, 500, 8)
    labels[3], labels[20], labels[30] = 500, -1, 2 ** 31 - 1
    good = torch.ones(40, dtype=torch.bool, device="cuda")
    good[[3, 20, 30]] = False
    loss, lse = _forward(moe, x, W, labels)
    assert moe.moe_get_device_error() == moe.MOE_DEVERR_LABEL
    assert bool((loss[~good] == 0).all())
    dloss = torch.ones(40, device="cuda")
    dx, dW = _backward(moe, x, W, labels, lse, dloss)
    assert moe.moe_get_device_error() == moe.MOE_DEVERR_LABEL
    clean = torch.where(good, labels, IGNORE)
    _check_forward(loss, lse, x, W, clean)
    _check_backward(dx, dW, x, W, clean, lse, dloss)


def test_any_label_can_be_the_ignored_one(moe):
    _, x, W, labels = _make(50, 64, 10, 9)
    loss, lse = _forward(moe, x, W, labels, ignore=3)
    assert moe.moe_get_device_error() == 0
    _check_forward(loss, lse, x, W, torch.where(labels == 3, IGNORE, labels))


def test_bits_repeat(moe):
    _, x, W, labels = _make(700, 520, 9001, 10, 0.2)
    dloss = torch.full((700,), 1.0 / 700, device="cuda")
    outs = []
    for _ in range(2):
        loss, lse = _forward(moe, x, W, labels)
        outs.append((loss, lse, *_backward(moe, x, W, labels, lse, dloss)))
    assert all(torch.equal(a, b) for a, b in zip(*outs))


def test_gradient_against_differences(moe):
    """<dx, d> and <dW, D> are derivatives of the weighted loss: central differences in 64 bits."""
    g, x, W, labels = _make(20, 64, 300, 11, 0.2)
    _, lse = _forward(moe, x, W, labels)
    dloss = torch.rand(20, generator=g, device="cuda")
    grads = _backward(moe, x, W, labels, lse, dloss)
    base = [x.double(), W.double()]

    def f(x64, w64):
        l = torch.nn.functional.cross_entropy(x64 @ w64.t(), labels.long(), ignore_index=IGNORE, reduction="none")
        return (l * dloss.double()).sum()

    for i, grad in enumerate(grads):
        d = torch.randn(grad.shape, generator=g, device="cuda").double()
        lo, hi = list(base), list(base)
        lo[i], hi[i] = base[i] - 1e-4 * d, base[i] + 1e-4 * d
        want = (f(*hi) - f(*lo)) / 2e-4
        # G, dloss * x and the gradient itself are each rounded to bf16
        assert abs((grad.double() * d).sum() - want) <= 6 * 3 * HALF * (grad.double() * d).square().sum().sqrt()

"""moe_cross_entropy_forward / _backward where labels are no labels and where
sizes come near what 32 bits count."""
import math

import pytest
import torch

from tests import test_gpu_cross_entropy as base
from tests.gpu_helpers import require_gpu
from tests.train_helpers import EPS, HALF, gen, randn, workspace

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


@pytest.mark.parametrize("T,V", [(1, 2_100_000_000), (3, 2 ** 31 - 257)])
def test_vocabularies_up_to_the_limit(moe, T, V):
    """All logits are 0 but those of a few rows; the gradients at the label, those rows and the last one."""
    H, g = 8, gen(V % 1000)
    x = torch.ones(T, H, dtype=torch.bfloat16, device="cuda")
    W = torch.zeros(V, H, dtype=torch.bfloat16, device="cuda")
    rows = torch.tensor([0, 5, 2 ** 27 - 1, 2 ** 27, 2_013_265_919, V - 1], device="cuda")
    W[rows] = randn(g, len(rows), H, std=3.0)
    labels = rows[[1, 4, 5][:T]].int()
    (loss, lse, dx, dW), err = _run(moe, x, W, labels, torch.ones(T, device="cuda"))
    assert err == (0, 0)
    z = W[rows].double().sum(1)
    total = V - len(rows) + z.exp().sum()
    # a thread of the join adds up to 2^17 parts one after the other, each of at most 128 terms
    tol = 2.0 ** 18 * EPS
    at = W[labels.long()].double().sum(1)
    assert bool(((lse.double() - total.log()).abs() <= tol).all())
    assert bool(((loss.double() - (total.log() - at)).abs() <= tol).all())
    some = torch.cat([rows, torch.tensor([1, V // 2, V - 2], device="cuda")])
    p = W[some].double().sum(1).exp() / total
    G = p[None] - (labels[:, None] == some[None]).double()
    assert bool(((dW[some].double() - G.sum(0)[:, None]).abs() <= 2 * T * (tol * p + HALF * G.abs().sum(0))[:, None]).all())
    assert not bool((dW == 7).any())
    q = z.exp() / total
    want = (q[:, None] * W[rows].double()).sum(0) - W[labels.long()].double()
    spread = (q[:, None] * W[rows].double().abs()).sum(0) + W[labels.long()].double().abs()
    assert bool(((dx.double() - want).abs() <= 2 * (HALF + tol) * spread).all())


def test_tokens_up_to_the_limit(moe):
    """2^31 - 257 tokens, nearly all of them zeros without a label (a hundred GB of rows and partial sums)."""
    T, H, V, g = 2 ** 31 - 257, 8, 2, gen(8)
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    W = randn(g, V, H)
    labels = torch.full((T,), IGNORE, dtype=torch.int32, device="cuda")
    at = torch.tensor([0, 1, 2 ** 30 + 3, T - 304, T - 303, T - 1], device="cuda")
    x[at], labels[at] = randn(g, len(at), H), torch.tensor([0, 1, 1, 0, 1, 0], dtype=torch.int32, device="cuda")
    loss, lse = torch.full((T,), 7.0, device="cuda"), torch.full((T,), 7.0, device="cuda")
    n = moe.moe_cross_entropy_forward_workspace_size(T, H, V)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    moe.moe_cross_entropy_forward(x, W, labels, T, H, V, IGNORE, loss, lse, ws, n)
    assert moe.moe_get_device_error() == 0
    z = x[at].double() @ W.double().t()
    zs = (x[at].double().square() @ W.double().square().t()).sqrt().amax(1)
    want = torch.logsumexp(z, 1)
    tol = 4 * (H / 16 + 16) * 2.0 ** -23 * zs + 8 * EPS * (1 + want.abs() + z.abs().amax(1))
    assert bool(((lse[at].double() - want).abs() <= tol).all())
    assert bool(((loss[at].double() - (want - z.gather(1, labels[at].long()[:, None])[:, 0])).abs() <= 2 * tol).all())
    loss[at], lse[at] = 0.0, torch.tensor(2.0).log().cuda()
    assert not bool(loss.any())
    low, high = torch.aminmax(lse)
    assert max(abs(low.item() - math.log(2)), abs(high.item() - math.log(2))) <= 16 * EPS


def _plan(moe, T, H, V):
    """(pieces, vocabulary rows of the last one, ranges of dx's contraction) of a backward call, the ranges from
    what its workspace holds: G of a piece, x in one or two copies, three values a token, a sum for each range."""
    def up(n, m):
        return -(-n // m) * m

    piece = min(V, max(2048, 2 ** 27 // T // 256 * 256))
    n = -(-V // piece)
    if n > 1:
        piece = up(-(-V // n), 256)
    n = -(-V // piece)
    rest, ld = moe.moe_cross_entropy_backward_workspace_size(T, H, V), up(H, 64)
    for b in (T * up(piece, 64) * 2, T * ld * 2, 0 if ld == H else T * ld * 2, 4 * T, 4 * (T + 1), 8):
        rest -= up(b, 256)
    ranges = rest // (4 * T * H)
    assert rest == up(4 * ranges * T * H, 256), "the workspace is not laid out as this test reads it"
    return n, V - (n - 1) * piece, ranges


def test_a_last_piece_with_fewer_blocks_than_ranges(moe):
    """Sizes, looked for on this device, whose dx is cut into several ranges of 64-row blocks while the last
    piece has one such block: the ranges past it must add nothing."""
    found = []
    for piece in range(2048, 9000, 256):
        V = piece * (piece // 256) + 1
        for H in (8, 64):
            for T in range(2 ** 27 // (piece + 256) + 1, 2 ** 27 // piece + 1, 61):
                n, last, ranges = _plan(moe, T, H, V)
                if n > 1 and last <= 64 and ranges > 1:
                    found.append((T * V * H, T, H, V))
    assert found, "no size reaches the case on this device"
    for _, T, H, V in sorted(found)[:1] + sorted(found)[-1:]:
        _, x, W, labels = base._make(T, H, V, 7)
        _, lse = base._forward(moe, x, W, labels)
        dloss = torch.ones(T, device="cuda")
        dx, _ = base._backward(moe, x, W, labels, lse, dloss, want=(True, False))
        assert moe.moe_get_device_error() == 0
        rows = torch.cat([torch.arange(0, T, 997), torch.tensor([T - 1])]).cuda()
        base._check_backward(dx[rows], None, x[rows], W, labels[rows], lse[rows], dloss[rows])

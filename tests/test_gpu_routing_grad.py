"""The routing gradients (moe_combine_backward, moe_permute_backward,
moe_route_backward) against automatic differentiation of the formulas in 64
bits, with sentinel slots, tokens without any live slot, and NaN in the rows
that must not be read."""
import pytest
import torch

from tests.gpu_helpers import require_gpu
from tests.train_helpers import EPS, gen, randn, rounded, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    require_gpu()
    from grouped_gemm_serving_gb300 import moe as m
    return m


def _route(moe, T, k, E, sentinel, seed, renorm=True):
    g = gen(seed)
    logits, bias = torch.randn(T, E, generator=g, device="cuda"), 0.5 * torch.randn(E, generator=g, device="cuda")
    mask = torch.zeros(T * k, dtype=torch.uint8, device="cuda")
    mask[torch.randperm(T * k, generator=g, device="cuda")[:sentinel]] = 1
    if sentinel:
        mask[:k] = 1   # a token without any live slot
    r = moe.route_sort_t(E, k, logits=logits, expert_bias=bias, sentinel_mask=mask, renormalize=renorm)
    assert moe.moe_get_device_error() == 0
    return g, logits, bias, r


CASES = [(1, 1, 1, 8, 0), (3, 2, 8, 264, 2), (64, 4, 32, 2880, 9), (300, 8, 128, 1000, 500), (1300, 4, 32, 72, 0),
         (1217, 8, 256, 2048, 100), (1500, 5, 64, 520, 3), (1250, 32, 32, 64, 77)]


@pytest.mark.parametrize("T,k,E,H,sentinel", CASES)
def test_combine_and_permute(moe, T, k, E, H, sentinel):
    g, _, _, r = _route(moe, T, k, E, sentinel, seed=T + H)
    ids, w, at = r["ids"], r["w"], r["row_pos"].long()
    live = ids.flatten() != E
    L = int(live.sum())
    dout, Y2, dxp = randn(g, T, H), randn(g, T * k, H), randn(g, T * k, H)
    Y2[L:] = float("nan")
    dxp[L:] = float("nan")
    dY2, dw = torch.full_like(Y2, 7), torch.full((T, k), 7.0, device="cuda")
    dx = torch.full((T, H), 7, dtype=torch.bfloat16, device="cuda")
    moe.moe_combine_backward(dout, Y2, ids, w, r["row_pos"], T, k, H, E, dY2, dw)
    moe.moe_permute_backward(dxp, ids, r["row_pos"], T, k, H, E, dx)
    assert moe.moe_get_device_error() == 0
    y = torch.where(live[:, None], Y2[at].double(), 0.0).view(T, k, H)
    d = dout.double()[:, None, :]
    ref = torch.where(live.view(T, k, 1), w.double()[:, :, None] * d, 0.0)
    within(dY2[at].view(T, k, H), ref, rounded(ref, torch.bfloat16))
    within(dw, (y * d).sum(2), (H + 4) * EPS * (y * d).abs().sum(2))
    assert bool((dw.flatten()[~live] == 0).all())
    rows = torch.where(live[:, None], dxp[at].double(), 0.0).view(T, k, H)
    ref = rows.sum(1)
    within(dx, ref, rounded(ref, torch.bfloat16) + (k + 1) * EPS * rows.abs().sum(1))


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (5, 1, 7), (64, 4, 32), (37, 8, 33), (300, 3, 64), (129, 8, 128), (77, 32, 256)])
def test_route(moe, T, k, E, renorm):
    g = gen(T + E)
    logits, bias = torch.randn(T, E, generator=g, device="cuda"), 0.5 * torch.randn(E, generator=g, device="cuda")
    dw = torch.randn(T, k, generator=g, device="cuda")
    out = torch.full((T, E), 7.0, device="cuda")
    for b in (bias, None):
        moe.moe_route_backward(logits, b, dw, T, E, k, renorm, out)
        l = (logits if b is None else logits + b).double().requires_grad_()
        ids = torch.topk(l, k, dim=1)[1]
        p = torch.softmax(l.gather(1, ids), 1) if renorm else torch.softmax(l, 1).gather(1, ids)
        ref, = torch.autograd.grad((p * dw.double()).sum(), l)
        # a probability is off by a few roundings (exp: 2 units) and the sum's E + 4; it multiplies a
        # difference of dw and their mean
        top = dw.double().abs().amax(1, keepdim=True)
        full = torch.softmax(l.gather(1, ids), 1) if renorm else torch.softmax(l, 1)
        scale = torch.zeros_like(ref).scatter_(1, ids, full.detach()) if renorm else full.detach()
        within(out, ref, scale * 2 * top * (E + 24) * EPS + 1e-30)


def test_route_ties_and_nan(moe):
    """Equal logits go to the lower expert; a NaN logit is never picked and gets no gradient."""
    logits = torch.tensor([[1.0, 2.0, 2.0, 2.0], [float("nan"), 0.0, -0.0, -5.0]], device="cuda")
    dw = torch.tensor([[1.0, -1.0], [0.5, 0.0]], device="cuda")
    out = torch.empty(2, 4, device="cuda")
    moe.moe_route_backward(logits, None, dw, 2, 4, 2, True, out)
    want = torch.tensor([[0, 0.5, -0.5, 0], [0, 0.125, -0.125, 0]], dtype=torch.float64, device="cuda")
    within(out, want, 1e-6)


def test_out_of_range_row_is_reported(moe):
    T, k, E, H = 4, 2, 4, 64
    ids = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    w = torch.ones(T, k, device="cuda")
    pos = torch.arange(T * k, dtype=torch.int32, device="cuda")
    pos[3] = T * k     # one past the last row: skipped and reported, never followed
    x = torch.ones(T * k, H, dtype=torch.bfloat16, device="cuda")
    dY2, dw = torch.full_like(x, 7), torch.empty(T, k, device="cuda")
    moe.moe_combine_backward(x[:T].contiguous(), x, ids, w, pos, T, k, H, E, dY2, dw)
    assert moe.moe_get_device_error() == moe.MOE_DEVERR_ROUTE
    assert bool((dY2[3] == 7).all()) and bool((dY2[4] == 1).all())


def test_bits_repeat_and_match_the_layer(moe):
    """The permute's gradient with unit weights is moe_combine's sum, bit for bit."""
    T, k, E, H = 500, 4, 16, 520
    g, _, _, r = _route(moe, T, k, E, 40, seed=3)
    dxp = randn(g, T * k, H)
    a, b = torch.empty(T, H, dtype=torch.bfloat16, device="cuda"), torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    moe.moe_permute_backward(dxp, r["ids"], r["row_pos"], T, k, H, E, a)
    moe.moe_combine(dxp, r["ids"], torch.ones(T, k, device="cuda"), r["row_pos"], T, k, H, E, b)
    assert torch.equal(a, b)

"""moe_route_backward_ids against automatic differentiation in 64 bits through
the ids in hand: equal logits in either order, picks in any order or of another
router, masked slots behind the combine's gradient, and ids that are refused."""
import pytest
import torch

from tests.gpu_helpers import require_gpu
from tests.train_helpers import EPS, gen, randn, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    require_gpu()
    from grouped_gemm_serving_gb300 import moe as m
    return m


def _check(out, l, picks, dw, renorm):
    """picks, dw: every pick that the softmax saw and its gradient (0 for a masked one)."""
    l = l.double().requires_grad_()
    E = l.shape[1]
    full = torch.softmax(l.gather(1, picks), 1) if renorm else torch.softmax(l, 1)
    p = full if renorm else full.gather(1, picks)
    ref, = torch.autograd.grad((p * dw.double()).sum(), l)
    # a probability is off by a few roundings (exp: 2 units) and the sum's E + 4; it multiplies a
    # difference of dw and their mean
    top = dw.double().abs().amax(1, keepdim=True)
    scale = torch.zeros_like(ref).scatter_(1, picks, full.detach()) if renorm else full.detach()
    within(out, ref, scale * 2 * top * (E + 24) * EPS + 1e-30)


def _topk(l, k, upper):
    """The k largest of every row; of equal ones the lower ids first, or the upper."""
    if not upper:
        return torch.sort(l, dim=1, descending=True, stable=True)[1][:, :k]
    return l.shape[1] - 1 - torch.sort(l.flip(1), dim=1, descending=True, stable=True)[1][:, :k]


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("upper", [False, True])
@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (5, 2, 7), (64, 4, 32), (37, 8, 33), (300, 8, 128), (77, 32, 256)])
def test_equal_logits_in_either_order(moe, T, k, E, upper, renorm):
    g = gen(T + E)
    logits = (torch.randn(T, E, generator=g, device="cuda") * 8).round() / 8   # as a router in few bits: many ties
    ids = _topk(logits, k, upper)
    if T > 10:
        assert bool((logits.gather(1, ids).diff(dim=1) == 0).any())
    dw, out = torch.randn(T, k, generator=g, device="cuda"), torch.full((T, E), 7.0, device="cuda")
    moe.moe_route_backward_ids(logits, None, ids.to(torch.int32), dw, T, E, k, renorm, out)
    assert moe.moe_get_device_error() == 0
    _check(out, logits, ids, dw, renorm)


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,k,E", [(3, 3, 8), (65, 4, 40), (200, 6, 100), (50, 32, 256)])
def test_any_picks_in_any_order(moe, T, k, E, renorm):
    """A router that does not take the largest logits, such as one limited to some groups of experts."""
    g = gen(T + k)
    logits, bias = torch.randn(T, E, generator=g, device="cuda"), torch.randn(E, generator=g, device="cuda")
    ids = torch.rand(T, E, generator=g, device="cuda").argsort(1)[:, :k].contiguous()
    dw, out = torch.randn(T, k, generator=g, device="cuda"), torch.full((T, E), 7.0, device="cuda")
    moe.moe_route_backward_ids(logits, bias, ids.to(torch.int32), dw, T, E, k, renorm, out)
    assert moe.moe_get_device_error() == 0
    _check(out, logits + bias, ids, dw, renorm)


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,k,E,masked", [(1, 2, 4, 1), (64, 4, 32, 60), (300, 8, 128, 700), (40, 32, 256, 400)])
def test_masked_slots_behind_the_combine(moe, T, k, E, masked, renorm):
    """Masked slots still count in the softmax: the gradients of the combine and of the top-k softmax in turn."""
    H, g = 72, gen(T + masked)
    logits, bias = torch.randn(T, E, generator=g, device="cuda"), 0.5 * torch.randn(E, generator=g, device="cuda")
    mask = torch.zeros(T * k, dtype=torch.uint8, device="cuda")
    mask[torch.randperm(T * k, generator=g, device="cuda")[:masked]] = 1
    mask[:k] = 1   # a token without any live slot
    r = moe.route_sort_t(E, k, logits=logits, expert_bias=bias, sentinel_mask=mask, renormalize=renorm)
    dout, Y2 = randn(g, T, H), randn(g, T * k, H)
    dY2, dw, out = torch.empty_like(Y2), torch.empty(T, k, device="cuda"), torch.full((T, E), 7.0, device="cuda")
    moe.moe_combine_backward(dout, Y2, r["ids"], r["w"], r["row_pos"], T, k, H, E, dY2, dw)
    moe.moe_route_backward_ids(logits, bias, r["ids"], dw, T, E, k, renorm, out)
    assert moe.moe_get_device_error() == 0
    live = (mask == 0).view(T, k)
    picks = _topk(logits + bias, k, False)
    assert torch.equal(torch.where(live, picks, E).int(), r["ids"])
    _check(out, logits + bias, picks, torch.where(live, dw, 0.0), renorm)
    # what a masked slot's gradient holds is not read
    again = torch.full_like(out, 7)
    moe.moe_route_backward_ids(logits, bias, r["ids"], torch.where(live, dw, float("nan")), T, E, k, renorm, again)
    assert torch.equal(out, again)


def test_bits_of_the_call_without_ids(moe):
    """For moe_route_sort's own picks both calls give the same bits."""
    T, k, E, g = 500, 8, 128, gen(9)
    logits = torch.randn(T, E, generator=g, device="cuda").bfloat16().float()
    r = moe.route_sort_t(E, k, logits=logits)
    dw = torch.randn(T, k, generator=g, device="cuda")
    a, b = torch.empty(T, E, device="cuda"), torch.empty(T, E, device="cuda")
    for renorm in (True, False):
        moe.moe_route_backward(logits, None, dw, T, E, k, renorm, a)
        moe.moe_route_backward_ids(logits, None, r["ids"], dw, T, E, k, renorm, b)
        assert torch.equal(a, b)


def test_nan_logits_that_are_not_picked(moe):
    logits = torch.tensor([[float("nan"), 0.0, -1.0, -5.0]], device="cuda")
    out = torch.empty(1, 4, device="cuda")
    ids = torch.tensor([[4, 1]], dtype=torch.int32, device="cuda")   # one slot masked: expert 2 had it
    dw = torch.tensor([[3.0, 0.5]], device="cuda")
    moe.moe_route_backward_ids(logits, None, ids, dw, 1, 4, 2, True, out)
    p = torch.softmax(torch.tensor([0.0, -1.0], dtype=torch.float64, device="cuda"), 0)
    want = torch.stack([0 * p[0], p[0] * (0.5 - 0.5 * p[0]), -p[1] * 0.5 * p[0], 0 * p[0]])[None]
    within(out, want, 40 * EPS)


def test_bad_ids_are_reported(moe):
    """An id outside [0, E] and a repeated one: reported, their slots as sentinels."""
    g = gen(2)
    E, k = 6, 3
    logits, dw = torch.randn(1, E, generator=g, device="cuda"), torch.randn(1, k, generator=g, device="cuda")
    a, b = torch.empty(1, E, device="cuda"), torch.empty(1, E, device="cuda")
    for bad in ((2, 7, 4), (2, -1, 4), (2, 2, 4), (2, 2 ** 31 - 1, 4)):
        moe.moe_route_backward_ids(logits, None, torch.tensor([bad], dtype=torch.int32, device="cuda"), dw, 1, E, k, True, a)
        assert moe.moe_get_device_error() == moe.MOE_DEVERR_ROUTE
        moe.moe_route_backward_ids(logits, None, torch.tensor([[2, E, 4]], dtype=torch.int32, device="cuda"), dw, 1, E, k, True, b)
        assert moe.moe_get_device_error() == 0
        assert torch.equal(a, b)

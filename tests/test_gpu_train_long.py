"""The training-step operators on tensors whose offsets pass 32 bits, checked
at rows on both sides of element 2^31 and at the last one."""
import pytest
import torch

from tests.gpu_helpers import require_gpu
from tests.train_helpers import EPS, NOISE, gen, randn, rounded, within, workspace

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
ACC = 2.0 ** -12   # fp32 sums of up to a few thousand terms, of which each addition may lose a unit in 2^23
OVER = 2 ** 31


@pytest.fixture(scope="module")
def moe():
    require_gpu()
    from grouped_gemm_serving_gb300 import moe as m
    yield m
    torch.cuda.empty_cache()


def _around(rows, width):
    """A few rows: the first, those around element 2^31, the last."""
    mid = OVER // width
    return torch.tensor(sorted({0, mid - 1, mid, mid + 1, rows - 1})).cuda()


@pytest.mark.parametrize("rows,H", [(300001, 7168), (2 ** 31 // 40 + 77, 40), (2 ** 31 // 1003 + 50, 1003)])
def test_layer_norm(moe, rows, H):
    g = gen(rows)
    x, dy, w = randn(g, rows, H), randn(g, rows, H), randn(g, H)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    dw, db = torch.empty(H, dtype=BF16, device="cuda"), torch.empty(H, dtype=BF16, device="cuda")
    moe.moe_layer_norm_forward(moe.MOE_BF16, x, H, rows, H, moe.MOE_BF16, w, None, 1e-5, y, H, mean, rstd)
    n = moe.moe_layer_norm_backward_workspace_size(rows, H)
    moe.moe_layer_norm_backward(moe.MOE_BF16, dy, H, x, H, rows, H, moe.MOE_BF16, w, mean, rstd, dx, H, dw, db, workspace(n), n)
    assert moe.moe_get_device_error() == 0
    at = _around(rows, H)
    xs, ds, wd = x[at].double(), dy[at].double(), w.double()
    m = xs.mean(1, keepdim=True)
    r = (xs.var(1, unbiased=False, keepdim=True) + 1e-5).rsqrt()
    xh = (xs - m) * r
    # mean and rstd are off by some (H + 16) roundings of fp32, relative to rows of size 1
    slack = (3 * H + 64) * EPS
    ref = xh * wd
    within(y[at], ref, rounded(ref, BF16) + slack * (1 + xh.abs()) * wd.abs())
    gw = ds * wd
    ref = r * (gw - gw.mean(1, keepdim=True) - xh * (gw * xh).mean(1, keepdim=True))
    size = r * (gw.abs() + (1 + xh.abs()) * (gw.abs() * (1 + xh.abs())).mean(1, keepdim=True))
    within(dx[at], ref, rounded(ref, BF16) + 2 * slack * size)


def test_as_many_rows_as_fit_32_bits(moe):
    """Rows of one element: y is the bias, dx zero, dbias the sum of dy."""
    rows = 2 ** 31 - 1
    x = torch.zeros(rows, 1, dtype=BF16, device="cuda")
    dy = torch.zeros(rows, 1, dtype=BF16, device="cuda")
    dy[0] = dy[rows // 2] = dy[-1] = 1
    mean, rstd = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
    dx = torch.full((rows, 1), 7, dtype=BF16, device="cuda")
    dw, db = torch.empty(1, device="cuda"), torch.empty(1, device="cuda")
    n = moe.moe_layer_norm_backward_workspace_size(rows, 1)
    moe.moe_layer_norm_backward(moe.MOE_BF16, dy, 1, x, 1, rows, 1, moe.MOE_F32, None, mean, rstd, dx, 1, dw, db, workspace(n), n)
    assert moe.moe_get_device_error() == 0
    assert db.item() == 3 and dw.item() == 0
    assert bool((dx[:5] == 0).all()) and bool((dx[-5:] == 0).all()) and int((dx != 0).sum()) == 0


def test_routing(moe):
    T, k, E, H = 2 ** 31 // (8 * 1024) + 100, 8, 32, 1024
    g = gen(5)
    r = moe.route_sort_t(E, k, logits=torch.randn(T, E, generator=g, device="cuda"))
    at = r["row_pos"].long()
    dout, Y2 = randn(g, T, H), randn(g, T * k, H)
    dY2, dw, dx = torch.empty_like(Y2), torch.empty(T, k, device="cuda"), torch.empty_like(dout)
    moe.moe_combine_backward(dout, Y2, r["ids"], r["w"], r["row_pos"], T, k, H, E, dY2, dw)
    moe.moe_permute_backward(Y2, r["ids"], r["row_pos"], T, k, H, E, dx)
    assert moe.moe_get_device_error() == 0
    # tokens of the first rows, of those around element 2^31 and of the last
    rows = _around(T * k, H)
    token = torch.empty(T * k, dtype=torch.int64, device="cuda")
    token[at] = torch.arange(T * k, device="cuda") // k
    t = torch.cat([token[rows], torch.tensor([0, T - 1]).cuda()])
    p = at.view(T, k)[t]
    d, y, w = dout[t].double()[:, None, :], Y2[p].double(), r["w"][t].double()[:, :, None]
    within(dY2[p], w * d, rounded(w * d, BF16))
    within(dw[t], (y * d).sum(2), (H + 4) * EPS * (y * d).abs().sum(2))
    within(dx[t], y.sum(1), rounded(y.sum(1), BF16) + (k + 1) * EPS * y.abs().sum(1))


def test_ffn(moe):
    H, I, E = 64, 1024, 3
    M = OVER // (2 * I) + 1000
    g = gen(9)
    x, dy = randn(g, M, H), randn(g, M, H)
    W1, W2 = randn(g, E, 2 * I, H, std=H ** -0.5), randn(g, E, H, I, std=I ** -0.5)
    ends = [0, M // 3, M - 700, M]
    off = torch.tensor(ends, dtype=torch.int32, device="cuda")
    Y1, h, y = (torch.empty(M, n, dtype=BF16, device="cuda") for n in (2 * I, I, H))
    moe.moe_ffn_forward(x, W1, W2, off, E, M, H, I, Y1, h, y)
    dx, dW1, dW2 = torch.empty_like(x), torch.empty_like(W1), torch.empty_like(W2)
    n = moe.moe_ffn_backward_workspace_size(E, M, H, I)
    moe.moe_ffn_backward(x, W1, W2, Y1, dy, off, E, M, H, I, dx, dW1, dW2, workspace(n), n)
    assert moe.moe_get_device_error() == 0
    for p in _around(M, 2 * I).tolist():
        e = sum(p >= b for b in ends[1:3])
        w1, w2 = W1[e].double(), W2[e].double()
        z = x[p].double() @ w1.t()
        within(Y1[p], z, rounded(z, BF16) + ACC * (x[p].double().square() @ w1.t().square()).sqrt())
        hh = torch.nn.functional.silu(z[:I]) * z[I:]
        ref = hh @ w2.t()
        within(y[p], ref, rounded(ref, BF16) + (NOISE + ACC) * (hh.square() @ w2.t().square()).sqrt())
        z = Y1[p].double().requires_grad_()
        hh = torch.nn.functional.silu(z[:I]) * z[I:]
        dz, = torch.autograd.grad(hh @ w2.t(), z, dy[p].double())
        ref = dz @ w1
        within(dx[p], ref, rounded(ref, BF16) + (2 ** 0.5 * NOISE + ACC) * (dz.square() @ w1.square()).sqrt())
    # the last expert's weight gradients: all of its rows lie past element 2^31
    a = ends[2]
    assert a * 2 * I > OVER
    z = Y1[a:].double().requires_grad_()
    hh = torch.nn.functional.silu(z[:, :I]) * z[:, I:]
    dz, = torch.autograd.grad(hh @ W2[2].double().t(), z, dy[a:].double())
    ref = dz.t() @ x[a:].double()
    within(dW1[2], ref, rounded(ref, BF16) + (2 ** 0.5 * NOISE + ACC) * (dz.t().square() @ x[a:].double().square()).sqrt())

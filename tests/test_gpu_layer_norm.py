"""moe_layer_norm_forward / _backward against the formulas in 64 bits: both
types, rows of every width class (one warp, one block, wider than any block
holds), odd widths, rows that lie apart, absent weight and bias, one row."""
import pytest
import torch

from tests.gpu_helpers import require_gpu
from tests.train_helpers import EPS, gen, randn, rounded, within, workspace

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def moe():
    require_gpu()
    from grouped_gemm_serving_gb300 import moe as m
    return m


def _dt(moe, t):
    return moe.MOE_BF16 if t == BF16 else moe.MOE_F32


def _rows(g, rows, H, pad, dtype, shift=0.5):
    x = torch.randn(rows, H + pad, generator=g, device="cuda")
    return (x * torch.exp(torch.randn(rows, 1, generator=g, device="cuda") * 0.5) + shift).to(dtype)[:, :H]


CASES = [
    # rows, H, dtype, wdtype, weight, bias, pad
    (1, 2880, BF16, BF16, True, True, 0),
    (1, 1, F32, F32, True, True, 0),
    (5, 8, BF16, F32, True, False, 0),
    (37, 255, BF16, BF16, True, True, 0),
    (300, 256, F32, F32, True, True, 4),
    (129, 1000, BF16, F32, False, False, 8),
    (200, 1024, F32, F32, True, True, 0),
    (33, 1003, F32, F32, True, True, 5),
    (700, 2048, BF16, BF16, True, True, 0),
    (50, 2049, BF16, F32, True, True, 0),
    (401, 4096, F32, F32, False, True, 0),
    (900, 7168, BF16, F32, True, True, 0),
    (20, 8200, BF16, BF16, True, True, 3),
    (17, 16384, F32, F32, True, True, 0),
    (700, 16400, BF16, F32, True, True, 0),
    (3, 40001, F32, F32, True, True, 0),
]


def _inputs(rows, H, dtype, wdtype, weight, bias, pad, seed):
    g = gen(seed)
    x = _rows(g, rows, H, pad, dtype)
    w = (1 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(wdtype) if weight else None
    b = randn(g, H, std=0.3, dtype=wdtype) if bias else None
    return g, x, w, b


def _forward64(x, w, b, eps):
    x = x.double()
    mean = x.mean(1, keepdim=True)
    rstd = ((x - mean).square().mean(1, keepdim=True) + eps) ** -0.5
    n = (x - mean) * rstd
    y = n * (w.double() if w is not None else 1) + (b.double() if b is not None else 0)
    return y, mean, rstd, n


@pytest.mark.parametrize("rows,H,dtype,wdtype,weight,bias,pad", CASES)
def test_forward(moe, rows, H, dtype, wdtype, weight, bias, pad):
    _, x, w, b = _inputs(rows, H, dtype, wdtype, weight, bias, pad, seed=rows + H)
    y = torch.full((rows, H + pad), 7, dtype=dtype, device="cuda")
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    moe.moe_layer_norm_forward(_dt(moe, dtype), x, x.stride(0), rows, H, _dt(moe, wdtype), w, b, 1e-5, y, H + pad, mean, rstd)
    ref, m, r, n = _forward64(x, w, b, 1e-5)
    size = x.double().abs().mean(1, keepdim=True)
    # a mean is a sum of H terms; a difference inherits its error, and n scales it by rstd
    dm = (H + 4) * EPS * size
    within(mean[:, None], m, dm + 1e-30)
    dr = r * ((H + 16) * EPS + 2 * dm * r)    # relative error of a sum of squares, halved by the root
    within(rstd[:, None], r, dr)
    wa = w.double().abs() if w is not None else 1.0
    tol = wa * (dm * r + n.abs() * dr / r + 4 * EPS * (n.abs() + (x.double().abs() + m.abs()) * r))
    within(y[:, :H], ref, tol + rounded(ref, dtype) + 4 * EPS * ref.abs())
    assert bool((y[:, H:] == 7).all())        # nothing between the rows is written


@pytest.mark.parametrize("rows,H,dtype,wdtype,weight,bias,pad", CASES)
def test_backward(moe, rows, H, dtype, wdtype, weight, bias, pad):
    g, x, w, b = _inputs(rows, H, dtype, wdtype, weight, bias, pad, seed=2 * rows + H)
    dy = _rows(g, rows, H, pad, dtype, shift=0.1)
    _, m, r, _ = _forward64(x, w, b, 1e-5)
    mean, rstd = m.float().flatten(), r.float().flatten()
    dx = torch.full((rows, H + pad), 7, dtype=dtype, device="cuda")
    dw, db = torch.empty(H, dtype=wdtype, device="cuda"), torch.empty(H, dtype=wdtype, device="cuda")
    n = moe.moe_layer_norm_backward_workspace_size(rows, H)
    moe.moe_layer_norm_backward(_dt(moe, dtype), dy, dy.stride(0), x, x.stride(0), rows, H, _dt(moe, wdtype), w,
                                mean, rstd, dx, H + pad, dw, db, workspace(n), n)
    d, m, r = dy.double(), mean.double()[:, None], rstd.double()[:, None]
    xh = (x.double() - m) * r
    gw = d * (w.double() if w is not None else 1)
    ref = r * (gw - gw.mean(1, keepdim=True) - xh * (gw * xh).mean(1, keepdim=True))
    # xh carries the rounding of a difference; the two means are sums of H terms
    exh = 4 * EPS * (x.double().abs() + m.abs()) * r
    e0 = (H + 4) * EPS * gw.abs().mean(1, keepdim=True)
    e1 = (H + 8) * EPS * (gw * xh).abs().mean(1, keepdim=True) + (gw.abs() * exh).mean(1, keepdim=True)
    tol = r * (4 * EPS * gw.abs() + e0 + xh.abs() * e1 + exh * (gw * xh).mean(1, keepdim=True).abs()) + 8 * EPS * ref.abs()
    within(dx[:, :H], ref, tol + rounded(ref, dtype))
    assert bool((dx[:, H:] == 7).all())
    rw, rb = (d * xh).sum(0), d.sum(0)
    within(dw, rw, (rows + 16) * EPS * (d * xh).abs().sum(0) + (d.abs() * exh).sum(0) + rounded(rw, wdtype))
    within(db, rb, (rows + 16) * EPS * d.abs().sum(0) + rounded(rb, wdtype))


def test_large_offset_keeps_the_spread(moe):
    """Rows far from zero: the squares are summed of x - mean, so the spread survives."""
    g = gen(5)
    x = torch.randn(64, 2048, generator=g, device="cuda") + 4096.0
    y = torch.empty_like(x)
    moe.moe_layer_norm_forward(moe.MOE_F32, x, 2048, 64, 2048, moe.MOE_F32, None, None, 0.0, y, 2048, None, None)
    ref, m, r, _ = _forward64(x, None, None, 0.0)
    # the mean of 2048 values near 4096 is off by a few units in its last place (2^-11)
    within(y, ref, r * 16 * 2.0 ** -11 + 1e-4 * ref.abs())


def test_gradient_against_differences(moe):
    """<dx, d> is the derivative of <dy, y> along d, by central differences of the formula in 64 bits."""
    g = gen(9)
    rows, H = 7, 193
    x, w, b = randn(g, rows, H, dtype=F32), randn(g, H, dtype=F32), randn(g, H, dtype=F32)
    dy, d = randn(g, rows, H, dtype=F32), randn(g, rows, H, dtype=F32)
    dw_dir = randn(g, H, dtype=F32)
    mean, rstd, y = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda"), torch.empty_like(x)
    moe.moe_layer_norm_forward(moe.MOE_F32, x, H, rows, H, moe.MOE_F32, w, b, 1e-5, y, H, mean, rstd)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    n = moe.moe_layer_norm_backward_workspace_size(rows, H)
    moe.moe_layer_norm_backward(moe.MOE_F32, dy, H, x, H, rows, H, moe.MOE_F32, w, mean, rstd, dx, H, dw, db, workspace(n), n)

    def f(sx, sw):
        return (_forward64(x.double() + sx * d.double(), w.double() + sw * dw_dir.double(), b, 1e-5)[0] * dy.double()).sum()

    h = 1e-4   # the third derivative's term is of size h^2, the gradients' own errors of size 1e-6
    for got, want in ((dx.double() * d.double()).sum(), (f(h, 0) - f(-h, 0)) / (2 * h)), \
                     ((dw.double() * dw_dir.double()).sum(), (f(0, h) - f(0, -h)) / (2 * h)):
        assert abs(got - want) <= 1e-4 * (dx.double() * d.double()).abs().sum()


def test_in_place_and_without_some_gradients(moe):
    g = gen(11)
    rows, H = 77, 520
    x, w, dy = randn(g, rows, H), randn(g, H), randn(g, rows, H)
    ref, mean, rstd = torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    moe.moe_layer_norm_forward(moe.MOE_BF16, x, H, rows, H, moe.MOE_BF16, w, None, 1e-5, ref, H, mean, rstd)
    same = x.clone()
    moe.moe_layer_norm_forward(moe.MOE_BF16, same, H, rows, H, moe.MOE_BF16, w, None, 1e-5, same, H, None, None)
    assert torch.equal(same, ref)
    n = moe.moe_layer_norm_backward_workspace_size(rows, H)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    back = (moe.MOE_BF16, dy, H, x, H, rows, H, moe.MOE_BF16, w, mean, rstd)
    moe.moe_layer_norm_backward(*back, dx, H, dw, None, workspace(n), n)
    only = torch.empty_like(x)
    moe.moe_layer_norm_backward(*back, only, H, None, None, None, 0)      # no sums: no workspace
    assert torch.equal(only, dx)
    only = torch.empty_like(w)
    moe.moe_layer_norm_backward(*back, None, 0, only, None, workspace(n), n)
    assert torch.equal(only, dw)
    moe.moe_layer_norm_backward(moe.MOE_BF16, dy, H, x, H, rows, H, moe.MOE_BF16, w, mean, rstd, dy, H, None, None, None, 0)
    assert torch.equal(dy, dx)


def test_bits_repeat(moe):
    g = gen(13)
    rows, H = 5000, 1024
    x, dy, w = randn(g, rows, H), randn(g, rows, H), randn(g, H)
    mean, rstd = x.float().mean(1), torch.rsqrt(x.float().var(1, unbiased=False) + 1e-5)
    n = moe.moe_layer_norm_backward_workspace_size(rows, H)
    outs = []
    for _ in range(2):
        dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)
        moe.moe_layer_norm_backward(moe.MOE_BF16, dy, H, x, H, rows, H, moe.MOE_BF16, w, mean, rstd, dx, H, dw, db, workspace(n), n)
        outs.append((dx, dw, db))
    assert all(torch.equal(a, b) for a, b in zip(*outs))


def test_another_stream(moe):
    g = gen(15)
    x = randn(g, 300, 2880)
    y, other = torch.empty_like(x), torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    moe.moe_layer_norm_forward(moe.MOE_BF16, x, 2880, 300, 2880, moe.MOE_BF16, None, None, 1e-5, y, 2880, None, None, stream=other)
    other.synchronize()
    within(y, _forward64(x, None, None, 1e-5)[0], 0.02)

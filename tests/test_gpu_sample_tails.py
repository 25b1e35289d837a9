"""moe_sample over long tails of light tokens, whose weights' roundings add up.

A weight is a whole number of 2^-45 of the largest one, to the nearest, off by at most
half of that and 2^-35 of itself; sums of them are exact, and a draw takes the first
token at which they exceed floor(u * total).  So the boundary behind the first j tokens,
F_j of the sum S (the largest weight is 1), is off by at most
    (half_j + F_j half_all + 2^-45) / S + 2^-34 F_j,
half_j the roundings of the first j tokens' weights: 2^-46 a token, or what their values
make it."""
import numpy as np
import pytest
import torch

from tests.gpu_helpers import require_gpu
from tests.test_gpu_sample import draw

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    require_gpu()
    from grouped_gemm_serving_gb300 import moe as m
    yield m
    assert m.moe_get_device_error() == 0


def boundaries(l, T=1.0):
    """Running sums of the weights in 80 or 128 bits, as shares of their sum, and the sum in units of the largest."""
    w = np.exp((l.astype(np.float64) - float(l.max())) / T).astype(np.longdouble)
    sums = np.cumsum(w)
    return (sums / sums[-1]).astype(np.float64), float(sums[-1])


def draws(moe, l, u, rows=64, T=None):
    """The tokens that one row of logits gives for all these u."""
    logits = torch.from_numpy(l).cuda().expand(rows, len(l)).contiguous()
    out = []
    for at in range(0, len(u), rows):
        some = u[at:at + rows].tolist()
        some += [0.5] * (rows - len(some))
        out += draw(moe, logits, u=some, temperature=None if T is None else [T] * rows)[0]
    return np.array(out[:len(u)])


def test_weights_are_rounded_to_the_nearest(moe):
    """Tail tokens whose weights are 0.85 to 0.95 above a multiple of 2^-44: cut to it they would
    lose nine tenths of a unit each, to the nearest they gain 0.15 at most, a boundary near the
    tail's end 2^-29.5 of the sum against 2^-27.  u lies between those."""
    rng = np.random.default_rng(1)
    V = 131072
    tail = rng.uniform(-16, -14, 20 * V).astype(np.float32)
    units = np.exp(tail.astype(np.float64)) * 2.0 ** 44
    tail = tail[(units % 1 > 0.85) & (units % 1 < 0.95)][:V - 1]
    assert len(tail) == V - 1
    l = np.append(tail, np.float32(0))
    F, S = boundaries(l)
    j = np.arange(V // 2, V - 1)
    half = 0.15 * 2.0 ** -44
    bound = (half * (j + 1) + F[j] * half * V + 2.0 ** -45) / S + 2.0 ** -34 * F[j]
    cut = (0.85 * (j + 1) - 0.95 * F[j] * V) * 2.0 ** -44 / S - 2.0 ** -34 * F[j]   # how far cut weights move it, at least
    u = (F[j] - bound).astype(np.float32)
    u = np.where(u.astype(np.float64) < F[j] - bound, u, np.nextafter(u, np.float32(0)))
    between = u.astype(np.float64) > F[j] - cut
    assert between.sum() > V // 8
    j, u = j[between], u[between]
    some = rng.choice(len(j), 512, replace=False)
    assert np.array_equal(draws(moe, l, u[some]), j[some])


@pytest.mark.parametrize("V,lo,hi,T", [(131072, -16, -14, 1.0), (262144, -34, -32, 1.0), (327680, -14, -9, 0.7), (100000, -0.5, 0, 1.0)])
def test_boundaries_are_where_the_header_says(moe, V, lo, hi, T):
    """Any u: the token is one whose share, widened by the bound, has u."""
    rng = np.random.default_rng(V)
    l = rng.uniform(lo, hi, V).astype(np.float32)
    l[V // 3] = 0
    F, S = boundaries(l, float(np.float32(T)))
    u = np.concatenate([rng.random(512), 2.0 ** rng.uniform(-30, -1, 128), F[rng.integers(0, V - 1, 384)]]).astype(np.float32)
    token = draws(moe, l, u, T=T)
    before = np.where(token > 0, F[token - 1], 0.0)
    off = lambda f, j: (2.0 ** -46 * (j + f * V) + 2.0 ** -45) / S + 2.0 ** -34 * f  # noqa: E731
    assert (u >= before - off(before, token)).all() and (u <= F[token] + off(F[token], token + 1)).all()


@pytest.mark.parametrize("settings", [dict(), dict(top_p=0.999)])
def test_the_largest_sum(moe, settings):
    """All logits of the largest vocabulary alike: 327680 of the largest weight, whose sum nearly fills 64 bits."""
    V, rows = 327680, 12
    u = np.concatenate([np.random.default_rng(2).random(rows - 3), [0.0, 0.5, 1 - 2.0 ** -24]]).astype(np.float32)
    kept = int(np.ceil(float(np.float32(settings["top_p"])) * V)) if settings else V
    logits = torch.full((rows, V), -2.0, device="cuda")
    token, logprob = draw(moe, logits, u=u.tolist(), **{n: [v] * rows for n, v in settings.items()})
    assert token == [int(x) for x in np.floor(u.astype(np.float64) * kept)]
    assert np.allclose(logprob, -np.log(kept), rtol=1e-6, atol=0)

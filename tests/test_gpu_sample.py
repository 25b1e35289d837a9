"""moe_sample against the definition in 64 bits, row by row: tokens have to be equal.

A token may differ only where u falls within the kernel's error of a boundary between
two tokens, some 2^-37 of the sum: with the at most 2^17 boundaries of a row here,
once in 2^20 rows.  The inputs are fixed; the tests draw some thousand rows."""
import math

import numpy as np
import pytest
import torch

from tests.gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    require_gpu()
    from grouped_gemm_serving_gb300 import moe as m
    yield m
    assert m.moe_get_device_error() == 0


def reference(l, T=1.0, k=0, p=1.0, min_p=0.0, u=0.5):
    """The definition, for one row of float64 logits (values of bf16 or fp32): token, logprob."""
    V = len(l)
    l = np.where(np.isnan(l), -np.inf, l)
    top = l.max()
    if top == -np.inf:
        return -1, -math.inf
    order = np.lexsort((np.arange(V), -l))   # logit descending, index ascending
    if not T >= 2.0 ** -126:
        return int(order[0]), 0.0
    if top == np.inf:
        w = (l == np.inf).astype(np.float64)
    else:
        with np.errstate(under="ignore", invalid="ignore"):
            w = np.where(l == top, 1.0, np.where(l == -np.inf, 0.0, np.exp((l - top) / T)))
    n = k if 0 < k < V else V
    kept = order[:n]
    if p < 1:
        sums = np.cumsum(w[kept])
        kept = kept[:max(1, int(np.searchsorted(sums, p * w[kept].sum(), side="left")) + 1)]
    if min_p > 0:
        kept = kept[w[kept] >= min(min_p, 1.0)]
    kept = np.sort(kept)
    sums = np.cumsum(w[kept])
    u = 0.0 if not u > 0 else min(u, 1 - 2.0 ** -24)
    at = int(np.searchsorted(sums, u * sums[-1], side="right"))
    return int(kept[at]), math.log(w[kept[at]] / sums[-1])


def draw(moe, logits, *, stream=None, want_logprob=True, **settings):
    rows, V = logits.shape
    kinds = dict(temperature=torch.float32, top_k=torch.int32, top_p=torch.float32, min_p=torch.float32, u=torch.float32)
    on = {n: torch.tensor(v, dtype=kinds[n], device="cuda") if v is not None else None for n, v in settings.items()}
    token = torch.full((rows + 3,), -7, dtype=torch.int32, device="cuda")
    logprob = torch.full((rows + 3,), 7.0, device="cuda")
    moe.moe_sample(moe.MOE_BF16 if logits.dtype == torch.bfloat16 else moe.MOE_F32, logits, logits.stride(0) if rows > 1 else max(V, logits.stride(0)), rows, V,
                   on.get("temperature"), on.get("top_k"), on.get("top_p"), on.get("min_p"), on["u"], token,
                   logprob if want_logprob else None, stream)
    torch.cuda.synchronize()
    assert token[rows:].tolist() == [-7] * 3 and logprob[rows:].tolist() == [7.0] * 3
    return token[:rows].tolist(), logprob[:rows].tolist()


def check(moe, logits, **settings):
    token, logprob = draw(moe, logits, **settings)
    l = logits.double().cpu().numpy()
    for r in range(logits.shape[0]):
        at = lambda n, none: float(np.float32(settings[n][r])) if settings.get(n) is not None else none  # noqa: E731
        k = settings["top_k"][r] if settings.get("top_k") is not None else 0
        want = reference(l[r], at("temperature", 1.0), k, at("top_p", 1.0), at("min_p", 0.0), at("u", 0.0))
        assert token[r] == want[0], (r, token[r], want, {n: v[r] for n, v in settings.items() if v is not None})
        # fp32: (l - L) / T and log1p of the other weights, a few roundings each, of one sign
        assert logprob[r] == want[1] or abs(logprob[r] - want[1]) <= 1e-6 * abs(want[1]) + 1e-12, (r, logprob[r], want)


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def logits_of(g, rows, V, dtype, std=3.0, pad=0, shift=0):
    """Rows of a wider buffer, `shift` elements behind a 16-byte boundary."""
    ld = V + pad
    flat = torch.randn(rows * ld + shift, generator=g, device="cuda") * std
    return flat.to(dtype)[shift:].view(rows, ld)[:, :V]


SIZES = [(1, 0, 0), (2, 0, 0), (3, 5, 1), (7, 1, 0), (8, 0, 0), (31, 2, 1), (64, 0, 3), (65, 0, 0), (100, 3, 0), (513, 0, 1), (1000, 0, 0),
         (4096, 0, 0), (4097, 7, 0), (32000, 0, 0), (50257, 0, 1), (131072, 0, 0), (151936, 64, 0)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V,pad,shift", SIZES)
def test_settings_by_row(moe, dtype, V, pad, shift):
    g = gen(V + pad)
    rng = np.random.default_rng(V + 1)
    rows = 40
    logits = logits_of(g, rows, V, dtype, pad=pad, shift=shift)
    pick = lambda *values: [values[i] for i in rng.integers(0, len(values), rows)]  # noqa: E731
    check(moe, logits, temperature=pick(0.0, 0.3, 0.7, 1.0, 1.0, 2.5), top_k=pick(0, 0, 1, 2, 5, 50, 200, 256, 257, 1000, V, V + 1, -3),
          top_p=pick(1.0, 1.0, 0.0, 1e-6, 0.3, 0.9, 0.999, 1.5), min_p=pick(0.0, 0.0, 0.05, 0.5, 1.0, 2.0, -1.0), u=rng.random(rows).tolist())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [1000, 50257, 262144])
@pytest.mark.parametrize("kind", ["k", "p", "min_p", "nothing", "k and p"])
def test_each_filter_alone(moe, dtype, V, kind):
    """Flat and steep rows: none, some and many tokens within a bin of the cut."""
    rng = np.random.default_rng(V)
    rows = 16
    std = torch.tensor([0.0, 0.01, 0.3, 1.0, 3.0, 10.0, 30.0, 2.0] * 2, device="cuda")
    logits = (logits_of(gen(V), rows, V, torch.float32, std=1.0) * std[:, None]).to(dtype)
    u = rng.random(rows).tolist()
    k = rng.integers(1, V, rows).tolist() if kind == "k" else [3, 40, 250, 256, 257, 900, 1024, 1025, 2000, V - 1, 1, 7, 64, 65, 128, 129]
    check(moe, logits, top_k=[min(x, V - 1) for x in k] if kind in ("k", "k and p") else None,
          top_p=rng.random(rows).tolist() if "p" in kind.split() else None,
          min_p=(0.3 * rng.random(rows)).tolist() if kind == "min_p" else None, u=u)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_ties(moe, dtype):
    """Equal logits: the lower index comes first in the order, and weights are exactly equal."""
    for V in (8, 1000, 5000, 70000):
        logits = torch.full((9, V), 2.5, dtype=dtype, device="cuda")
        logits[8, V // 2:] = 3.0
        check(moe, logits, u=[0.0, 0.25, 0.5, 0.999, 0.5, 0.5, 0.9, 0.1, 0.3], top_k=[0, 4, 0, 7, 0, 3, 0, V - 1, V // 2 + 2],
              top_p=[1.0, 1.0, 0.5, 1.0, 0.25, 0.5, 0.99, 0.1, 1.0])
    few = torch.tensor([[1.0, 0.0, -0.0, 1.0, -float("inf"), 1.0, 0.0, 1.0]], dtype=dtype, device="cuda")   # -0 and +0 tie
    for k in range(1, 8):
        for u in (0.0, 0.3, 0.6, 0.99):
            check(moe, few, top_k=[k], u=[u])


def test_values_that_are_not_finite(moe):
    inf, nan = float("inf"), float("nan")
    for V in (16, 3000):
        logits = torch.randn(8, V, generator=gen(V), device="cuda")
        logits[0] = -inf
        logits[1] = nan
        logits[2, ::2] = nan
        logits[3, 5], logits[3, 9] = inf, inf
        logits[4, 1:] = -inf
        logits[5, :] = -3.4028234663852886e38
        logits[6, :-3] = -3.4028234663852886e38
        logits[7] *= 1e38
        for dtype in (torch.float32, torch.bfloat16):
            for u in (0.1, 0.5, 0.9):
                for settings in (dict(), dict(top_k=[3] * 8), dict(top_p=[0.7] * 8), dict(min_p=[0.1] * 8), dict(top_k=[10] * 8, top_p=[0.5] * 8),
                                 dict(temperature=[0.0] * 8)):
                    check(moe, logits.to(dtype), u=[u] * 8, **settings)


def test_extreme_settings(moe):
    V = 5000
    logits = torch.randn(1, V, generator=gen(3), device="cuda").expand(12, V).contiguous()
    tiny = 2.0 ** -126
    check(moe, logits, temperature=[float("inf"), 1e30, 1e-30, tiny, tiny / 2, -1.0, float("nan"), 1e-3, 100.0, 1.0, 1.0, 1.0],
          u=[0.5, 0.3, 0.9, 0.9, 0.9, 0.9, 0.9, 0.7, 0.2, -0.5, 1.0, 7.0])
    check(moe, logits, top_p=[float("nan"), float("inf"), -1.0, 1 - 2.0 ** -24, 2.0 ** -149, 2.0 ** -30, 0.5, 0.5, 0.5, 0.5, 0.5, 0.5],
          u=[0.5, 0.5, 0.5, 0.5, 0.5, 0.5, float("nan"), 0.0, 2.0 ** -149, 2.0 ** -40, 1 - 2.0 ** -24, float("inf")])


def test_where_u_falls_among_few(moe):
    """Every boundary between tokens, from both sides."""
    logits = torch.tensor([[math.log(2.0 ** -i) if i else 0.0 for i in range(6)]], device="cuda")
    l = logits.double().cpu().numpy()[0]
    w = np.exp(l - l.max())
    edges = np.cumsum(w) / w.sum()
    for e in edges[:-1]:
        for off in (-1e-5, 1e-5):
            check(moe, logits, u=[float(e + off)])
    uniform = torch.zeros(1, 8, device="cuda")
    for i in range(8):
        assert draw(moe, uniform, u=[i / 8])[0] == [i]   # at a boundary exactly: the token behind it


def test_the_draw_follows_the_distribution(moe):
    """u over a fine grid gives every token its share."""
    logits = torch.randn(1, 20, generator=gen(4), device="cuda")
    n = 4000
    token, _ = draw(moe, logits.expand(n, 20).contiguous(), u=[(i + 0.5) / n for i in range(n)], top_k=[12] * n)
    w = torch.softmax(torch.topk(logits[0].double(), 12).values, 0)
    ids = torch.topk(logits[0], 12).indices.tolist()
    counts = np.bincount(token, minlength=20)
    for i, share in zip(ids, w.tolist()):
        assert abs(counts[i] - n * share) <= 1.01
    assert counts.sum() == sum(counts[i] for i in ids)


def test_largest_vocabulary_and_many_rows(moe):
    g = gen(5)
    rng = np.random.default_rng(6)
    for dtype in (torch.bfloat16, torch.float32):
        logits = logits_of(g, 3, 327680, dtype)
        check(moe, logits, top_k=[0, 100, 0], top_p=[0.9, 0.9, 1.0], u=[0.4, 0.6, 0.8])
    rows = 700
    logits = logits_of(g, rows, 3000, torch.bfloat16)
    check(moe, logits, top_k=rng.integers(0, 300, rows).tolist(), top_p=(0.5 + 0.6 * rng.random(rows)).tolist(), u=rng.random(rows).tolist())


def test_no_settings_no_logprob(moe):
    logits = logits_of(gen(7), 5, 777, torch.float32)
    u = [0.1, 0.3, 0.5, 0.7, 0.9]
    token, logprob = draw(moe, logits, u=u, want_logprob=False)
    assert token == draw(moe, logits, u=u, temperature=[1.0] * 5, top_k=[0] * 5, top_p=[1.0] * 5, min_p=[0.0] * 5)[0]
    assert logprob == [7.0] * 5


def test_graph_and_streams(moe):
    g = gen(8)
    logits = logits_of(g, 9, 40000, torch.bfloat16)
    u = torch.rand(9, generator=g, device="cuda")
    p = torch.full((9,), 0.9, device="cuda")
    token = torch.empty(9, dtype=torch.int32, device="cuda")

    def run(t, stream=None):
        moe.moe_sample(moe.MOE_BF16, logits, 40000, 9, 40000, None, None, p, None, u, t, None, stream)

    run(token)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(token)
    for seed in (9, 10):
        u.copy_(torch.rand(9, generator=gen(seed), device="cuda"))
        token.fill_(-1)
        graph.replay()
        eager = torch.empty_like(token)
        run(eager)
        torch.cuda.synchronize()
        assert torch.equal(token, eager)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    both = []
    for _ in range(20):
        for stream in (None, side):
            both.append(torch.empty_like(token))
            run(both[-1], stream)
    torch.cuda.synchronize()
    assert all(torch.equal(t, token) for t in both)


def test_rows_past_32_bit_offsets(moe):
    g = gen(11)
    ld = 1 << 30
    big = torch.empty(4 * ld + 1000, dtype=torch.bfloat16, device="cuda")
    rows = big[:4 * ld].view(4, ld)[:, :1000]
    rows.copy_(logits_of(g, 4, 1000, torch.bfloat16))
    check(moe, rows, top_k=[50, 0, 0, 5], top_p=[0.9, 0.8, 1.0, 1.0], u=[0.3, 0.6, 0.9, 0.2])

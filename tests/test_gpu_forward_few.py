"""The whole expert layer for a few tokens (moe_forward_few) against the same layer
in 64 bits, token by token, from the weights' values.

The tolerance: one rounding of the result to bf16; the rounding of h to the second
product's operand, independent from element to element, of standard deviation HALF /
sqrt(3) (bf16; fp16's 2^-11 for FP8) of its terms w[t, j] W2[e, n, i] h[i]; and fp32
sums, at most n EPS of the sum of the terms' magnitudes, where the first product's
error passes through silu(g) u, whose derivatives by g and u are at most 1.1 |u| and
|g|."""
import pytest
import torch

from tests.gpu_helpers import require_gpu
from tests.train_helpers import EPS, HALF, NOISE, gen, randn, within, workspace

pytestmark = pytest.mark.gpu
F64 = torch.float64


@pytest.fixture(scope="module")
def moe():
    require_gpu()
    from grouped_gemm_serving_gb300 import moe as m
    assert m.moe_get_device_error() == 0
    yield m
    assert m.moe_get_device_error() == 0


class Layer:
    """Weights of a layer, in fp8 with a scale per 128 x 128 block, and their values."""

    def __init__(self, g, dtype, E, H, I):
        self.dtype, self.E, self.H, self.I = dtype, E, H, I
        if dtype == "bf16":
            self.W1, self.W2 = randn(g, E, 2 * I, H, std=H ** -0.5), randn(g, E, H, I, std=I ** -0.5)
            self.s1 = self.s2 = None
            self.v1, self.v2 = self.W1.double(), self.W2.double()
        else:
            def make(N, K):
                q = (torch.randn(E, N, K, generator=g, device="cuda") * 100).clamp_(-448, 448).to(torch.float8_e4m3fn)
                s = (0.01 * K ** -0.5 * torch.exp(0.5 * torch.randn(E, -(-N // 128), K // 128, generator=g, device="cuda"))).float()
                wide = s.double().repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)
                return q, s, q.double() * wide
            self.W1, self.s1, self.v1 = make(2 * I, H)
            self.W2, self.s2, self.v2 = make(H, I)


def call(moe, layer, x, *, logits=None, bias=None, mask=None, ids=None, w=None, renorm=True, k=None, stream=None, guard=0, ws=None):
    """One call into fresh outputs: out, ids, w.  guard: rows behind out that must stay as they are."""
    T = x.shape[0]
    k = k or ids.shape[1]
    whole = torch.full((T + guard, layer.H), 7.0, dtype=torch.bfloat16, device="cuda")
    out = whole[:T]
    if ids is None:
        ids = torch.full((T, k), -5, dtype=torch.int32, device="cuda")
        w = torch.full((T, k), -5.0, device="cuda")
    a = moe.forward_args(dtype=moe.MOE_BF16 if layer.dtype == "bf16" else moe.MOE_FP8_E4M3_B128, T=T, E=layer.E, k=k, H=layer.H, I=layer.I, x=x,
                         W1=layer.W1, W2=layer.W2, W1_scales=layer.s1, W2_scales=layer.s2, out=out, logits=logits, expert_bias=bias,
                         sentinel_mask=mask, topk_ids=ids, topk_w=w, renormalize=renorm)
    n = moe.moe_forward_few_workspace_size(a)
    assert n > 0
    ws = workspace(n) if ws is None else ws
    moe.moe_forward_few(a, ws, n, stream)
    if guard:
        assert bool((whole[T:] == 7.0).all())
    return out, ids, w


def check(layer, x, ids, w, out):
    """out against the layer in 64 bits for these picks and weights."""
    T, k = ids.shape
    E, H, I = layer.E, layer.H, layer.I
    half_h = HALF if layer.dtype == "bf16" else 2.0 ** -11
    ref = torch.zeros(T, H, dtype=F64, device="cuda")
    var, tol = torch.zeros_like(ref), torch.zeros_like(ref)
    for t in range(T):
        xt = x[t].double()
        for j in range(k):
            e = int(ids[t, j])
            if e == E:
                continue
            z, az = layer.v1[e] @ xt, layer.v1[e].abs() @ xt.abs()
            g, u, dz = z[:I], z[I:], H * EPS * az
            h = torch.nn.functional.silu(g) * u
            dh = 1.1 * u.abs() * dz[:I] + g.abs() * dz[I:] + 8 * EPS * h.abs()
            wt = abs(float(w[t, j]))
            terms = layer.v2[e] * h
            ref[t] += float(w[t, j]) * terms.sum(1)
            var[t] += (wt * half_h / 3 ** 0.5) ** 2 * terms.square().sum(1)
            tol[t] += wt * (layer.v2[e].abs() @ dh + (I + k + 2) * EPS * terms.abs().sum(1))
    within(out, ref, 1.01 * HALF * ref.abs() + 6 * var.sqrt() * 1.01 + 2 * tol)


def picks(moe, logits, bias, mask, k, E, renorm):
    r = moe.route_sort_t(E, k, logits=logits, expert_bias=bias, sentinel_mask=mask, renormalize=renorm)
    return r["ids"], r["w"]


CASES = [
    # dtype, T, E, k, H, I, bias, renorm, sentinels
    ("bf16", 1, 32, 4, 256, 192, True, True, 0),
    ("bf16", 1, 1, 1, 8, 8, False, True, 0),
    ("bf16", 2, 3, 2, 72, 40, False, False, 1),
    ("bf16", 5, 8, 3, 1000, 1368, True, True, 4),       # columns that fill no tile, features that fill no unit
    ("bf16", 8, 256, 8, 512, 64, True, False, 3),
    ("bf16", 9, 40, 2, 520, 136, False, True, 0),
    ("bf16", 17, 64, 6, 640, 72, True, True, 20),
    ("bf16", 33, 5, 1, 264, 520, False, False, 0),
    ("bf16", 64, 2, 2, 192, 264, False, True, 0),       # 64 rows of each expert: four chunks
    ("bf16", 64, 128, 8, 256, 128, True, True, 100),
    ("bf16", 40, 3, 2, 2880, 96, True, True, 0),        # fewer rows at a time than a chunk could have
    ("bf16", 12, 4, 2, 16392, 40, False, True, 0),      # rows of x so long that few fit
    ("bf16", 3, 2, 1, 32768, 16, False, True, 0),
    ("bf16", 6, 2, 2, 24, 32768, False, True, 0),
    ("bf16", 32, 64, 32, 128, 64, True, False, 0),      # 1024 slots
    ("fp8", 1, 32, 4, 256, 384, True, True, 0),
    ("fp8", 1, 1, 1, 128, 128, False, True, 0),
    ("fp8", 6, 7, 3, 1152, 640, True, False, 5),        # nine tiles: a second stage with one
    ("fp8", 8, 256, 8, 256, 128, True, True, 0),
    ("fp8", 16, 4, 2, 384, 256, False, True, 0),
    ("fp8", 64, 3, 2, 2048, 128, True, True, 9),
    ("fp8", 20, 2, 1, 16384, 128, False, True, 0),
    ("fp8", 10, 2, 2, 128, 4224, False, True, 0),
]


@pytest.mark.parametrize("dtype,T,E,k,H,I,bias,renorm,sentinels", CASES)
def test_layer(moe, dtype, T, E, k, H, I, bias, renorm, sentinels):
    g = gen(T * 1000 + E + H)
    layer = Layer(g, dtype, E, H, I)
    x = randn(g, T, H)
    logits = torch.randn(T, E, generator=g, device="cuda")
    b = 0.5 * torch.randn(E, generator=g, device="cuda") if bias else None
    mask = None
    if sentinels:
        mask = torch.zeros(T * k, dtype=torch.uint8, device="cuda")
        mask[torch.randperm(T * k, generator=g, device="cuda")[:sentinels]] = 1
    out, ids, w = call(moe, layer, x, logits=logits, bias=b, mask=mask, k=k, renorm=renorm, guard=3)
    want_ids, want_w = picks(moe, logits, b, mask, k, E, renorm)
    assert torch.equal(ids, want_ids)
    assert torch.equal(w, want_w)   # moe_route_sort's, bit for bit
    check(layer, x, ids, w, out)
    again, _, _ = call(moe, layer, x, logits=logits, bias=b, mask=mask, k=k, renorm=renorm)
    assert torch.equal(again, out)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("T", [1, 7, 30, 64])
def test_given_picks(moe, dtype, T):
    """Ids and weights given: any weights, an expert twice for a token, sentinels, a token without experts."""
    g = gen(T)
    E, k, H, I = 6, 4, 384, 256
    layer = Layer(g, dtype, E, H, I)
    x = randn(g, T, H)
    ids = torch.randint(0, E + 1, (T, k), generator=g, device="cuda", dtype=torch.int32)
    ids[:, 1] = ids[:, 0]
    ids[T // 2] = E
    w = torch.randn(T, k, generator=g, device="cuda")
    kept = ids.clone(), w.clone()
    out, _, _ = call(moe, layer, x, ids=ids, w=w, guard=1)
    assert torch.equal(ids, kept[0]) and torch.equal(w, kept[1])
    check(layer, x, ids, w, out)
    assert bool((out[T // 2] == 0).all())


def test_no_expert_at_all(moe):
    layer = Layer(gen(1), "bf16", 4, 136, 72)
    ids = torch.full((9, 2), 4, dtype=torch.int32, device="cuda")
    out, _, _ = call(moe, layer, randn(gen(2), 9, 136), ids=ids, w=torch.full((9, 2), float("nan"), device="cuda"))
    assert bool((out == 0).all())


def test_invalid_ids_are_sentinels(moe):
    g = gen(3)
    layer = Layer(g, "bf16", 5, 128, 64)
    x, w = randn(g, 4, 128), torch.rand(4, 2, generator=g, device="cuda")
    ids = torch.tensor([[0, 1], [-1, 2], [6, 3], [2 ** 31 - 1, -2 ** 31]], dtype=torch.int32, device="cuda")
    out, _, _ = call(moe, layer, x, ids=ids, w=w)
    assert moe.moe_get_device_error() == moe.MOE_DEVERR_ROUTE
    assert ids.tolist() == [[0, 1], [5, 2], [5, 3], [5, 5]]
    check(layer, x, ids, w, out)


def test_nan_logits(moe):
    g = gen(4)
    layer = Layer(g, "bf16", 40, 128, 64)
    x, logits = randn(g, 3, 128), torch.randn(3, 40, generator=g, device="cuda")
    logits[1, 2:] = float("nan")
    logits[2, ::2] = -float("inf")
    out, ids, w = call(moe, layer, x, logits=logits, k=4)
    assert moe.moe_get_device_error() == moe.MOE_DEVERR_ROUTE
    want_ids, want_w = picks(moe, logits, None, None, 4, 40, True)
    assert moe.moe_get_device_error() == moe.MOE_DEVERR_ROUTE
    assert torch.equal(ids, want_ids) and torch.equal(w[[0, 2]], want_w[[0, 2]])
    check(layer, x[[0, 2]], ids[[0, 2]], w[[0, 2]], out[[0, 2]])


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_what_is_not_finite_stays_with_its_token(moe, dtype):
    g = gen(5)
    T, E, H, I = 20, 3, 256, 128
    layer = Layer(g, dtype, E, H, I)
    x, logits = randn(g, T, H), torch.randn(T, E, generator=g, device="cuda")
    clean, _, _ = call(moe, layer, x, logits=logits, k=2)
    x[3, 7], x[11, 200] = float("nan"), float("inf")
    out, _, _ = call(moe, layer, x, logits=logits, k=2)
    rest = [t for t in range(T) if t not in (3, 11)]
    assert torch.equal(out[rest], clean[rest])
    assert bool(out[3].isnan().all()) and not bool(out[11].isfinite().any())


def test_large_and_small_values(moe):
    """FP8 holds x in fp16, scaled: rows far outside of fp16's range, and with a wide range within."""
    g = gen(6)
    layer = Layer(g, "fp8", 2, 256, 128)
    for scale in (2.0 ** 40, 2.0 ** -40):
        x = randn(g, 4, 256, std=scale)
        x[1, ::2] *= 2.0 ** -12
        x[2] = 0
        layer.s1 = torch.full_like(layer.s1, 0.01 / scale)   # h of ordinary size
        layer.v1 = layer.W1.double() * (0.01 / scale if scale > 1 else float(torch.tensor(0.01 / scale, dtype=torch.float32)))
        layer.v1 = layer.W1.double() * layer.s1.double()[0, 0, 0]
        logits = torch.randn(4, 2, generator=g, device="cuda")
        out, ids, w = call(moe, layer, x, logits=logits, k=2)
        check(layer, x, ids, w, out)
        assert bool((out[2] == 0).all())


def test_a_weight_that_is_nan(moe):
    layer = Layer(gen(7), "fp8", 2, 128, 128)
    layer.W2.view(torch.uint8)[1, 5, 9] = 0x7F
    ids = torch.tensor([[0], [1]], dtype=torch.int32, device="cuda")
    out, _, _ = call(moe, layer, randn(gen(8), 2, 128), ids=ids, w=torch.ones(2, 1, device="cuda"))
    assert bool(out[0].isfinite().all()) and bool(out[1, 5].isnan()) and int(out[1].isnan().sum()) == 1


def test_out_over_x_and_picks_not_wanted(moe):
    g = gen(9)
    layer = Layer(g, "bf16", 8, 256, 128)
    x, logits = randn(g, 6, 256), torch.randn(6, 8, generator=g, device="cuda")
    want, _, _ = call(moe, layer, x, logits=logits, k=2)
    a = moe.forward_args(dtype=moe.MOE_BF16, T=6, E=8, k=2, H=256, I=128, x=x, W1=layer.W1, W2=layer.W2, out=x, logits=logits)
    n = moe.moe_forward_few_workspace_size(a)
    moe.moe_forward_few(a, workspace(n), n)
    assert torch.equal(x, want)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_graphs_and_streams(moe, dtype):
    """Captured, replayed with other inputs, two graphs over one workspace in turn, on another stream beside an eager call."""
    g = gen(10)
    T, E, k, H, I = 5, 16, 3, 512, 256
    layer = Layer(g, dtype, E, H, I)
    x, logits = randn(g, T, H), torch.randn(T, E, generator=g, device="cuda")
    x2, logits2 = randn(g, 23, H), torch.randn(23, E, generator=g, device="cuda")
    kw = dict(dtype=moe.MOE_BF16 if dtype == "bf16" else moe.MOE_FP8_E4M3_B128, E=E, k=k, H=H, I=I, W1=layer.W1, W2=layer.W2, W1_scales=layer.s1,
              W2_scales=layer.s2)
    out, out2 = torch.empty_like(x), torch.empty_like(x2)
    a = moe.forward_args(T=T, x=x, logits=logits, out=out, **kw)
    b = moe.forward_args(T=23, x=x2, logits=logits2, out=out2, **kw)
    n = moe.moe_forward_few_workspace_size(b)
    ws = workspace(n)
    moe.moe_forward_few(a, ws, n)
    torch.cuda.synchronize()
    graphs = []
    for args in (a, b):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            moe.moe_forward_few(args, ws, n)
        graphs.append(graph)
    for seed in (11, 12):
        h = gen(seed)
        x.copy_(randn(h, T, H))
        logits.copy_(torch.randn(T, E, generator=h, device="cuda"))
        x2.copy_(randn(h, 23, H))
        out.fill_(9), out2.fill_(9)
        for graph in graphs + graphs[:1]:
            graph.replay()
        torch.cuda.synchronize()
        for xs, ls, got in ((x, logits, out), (x2, logits2, out2)):
            want, _, _ = call(moe, layer, xs, logits=ls, k=k)
            assert torch.equal(got, want)
    # calls on two streams at once: each with a workspace and an output that are there before and after
    want, _, _ = call(moe, layer, x, logits=logits, k=k)
    side = torch.cuda.Stream()
    calls = []
    for i in range(40):
        got = torch.full_like(x, 9)
        calls.append((moe.forward_args(T=T, x=x, logits=logits, out=got, **kw), workspace(n), side if i % 2 else None, got))
    torch.cuda.synchronize()
    for args, space, stream, _ in calls:
        moe.moe_forward_few(args, space, n, stream)
    torch.cuda.synchronize()
    assert all(torch.equal(got, want) for *_, got in calls)


def test_many_passes_agree(moe):
    """The same bits from every pass, over sizes that leave blocks without units and rings of several depths."""
    g = gen(13)
    for dtype, T, E, k, H, I in [("bf16", 64, 8, 2, 1536, 512), ("fp8", 64, 8, 2, 1536, 512), ("bf16", 3, 4, 2, 64, 8), ("fp8", 12, 64, 8, 7168, 256)]:
        layer = Layer(g, dtype, E, H, I)
        x, logits = randn(g, T, H), torch.randn(T, E, generator=g, device="cuda")
        first, ids, w = call(moe, layer, x, logits=logits, k=k)
        check(layer, x, ids, w, first)
        for _ in range(30):
            assert torch.equal(call(moe, layer, x, logits=logits, k=k)[0], first)
        del layer


def test_weights_past_32_bit_offsets(moe):
    """Experts that start behind 2^32 elements."""
    g = gen(14)
    E, H, I = 256, 4096, 2432
    W1 = torch.empty(E, 2 * I, H, dtype=torch.bfloat16, device="cuda")
    W2 = torch.empty(E, H, I, dtype=torch.bfloat16, device="cuda")
    assert W1.numel() > 1 << 32
    layer = Layer(g, "bf16", 2, H, I)
    for at, e in ((0, 0), (1, E - 1)):
        W1[e], W2[e] = layer.W1[at], layer.W2[at]
    x = randn(g, 3, H)
    w = torch.rand(3, 2, generator=g, device="cuda")
    far = torch.tensor([[E - 1, 0], [E - 1, E], [0, E - 1]], dtype=torch.int32, device="cuda")
    near = torch.tensor([[1, 0], [1, 2], [0, 1]], dtype=torch.int32, device="cuda")
    v1, v2 = layer.v1, layer.v2
    layer.W1, layer.W2, layer.E = W1, W2, E
    out, _, _ = call(moe, layer, x, ids=far, w=w)
    layer.E = 2
    check(layer, x, near, w, out)

"""The training-step operators inside a CUDA graph, on another stream than the
current one, and with garbage where nothing may be read."""
import pytest
import torch

from tests.gpu_helpers import require_gpu
from tests.train_helpers import gen, randn, workspace

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def moe():
    require_gpu()
    from grouped_gemm_serving_gb300 import moe as m
    return m


def _steps(moe):
    """(name, call(stream), outputs) of every operator on inputs of its own."""
    g = gen(3)
    T, k, E, H, I, V = 300, 2, 6, 264, 136, 1003

    def empty(*s, dtype=BF16):
        return torch.full(s, 7, dtype=dtype, device="cuda")

    F32 = torch.float32
    x, dy, w = randn(g, T, H), randn(g, T, H), randn(g, H)
    mean, rstd, y = empty(T, dtype=F32), empty(T, dtype=F32), empty(T, H)
    yield ("norm forward", lambda s: moe.moe_layer_norm_forward(moe.MOE_BF16, x, H, T, H, moe.MOE_BF16, w, w, 1e-5, y, H, mean, rstd, stream=s),
           (y, mean, rstd))
    m, r = x.float().mean(1), torch.rsqrt(x.float().var(1, unbiased=False) + 1e-5)
    dx, dw, db = empty(T, H), empty(H), empty(H)
    n1 = moe.moe_layer_norm_backward_workspace_size(T, H)
    ws1 = workspace(n1)
    yield ("norm backward", lambda s: moe.moe_layer_norm_backward(moe.MOE_BF16, dy, H, x, H, T, H, moe.MOE_BF16, w, m, r, dx, H, dw, db, ws1, n1, stream=s),
           (dx, dw, db))
    logits = torch.randn(T, E, generator=g, device="cuda")
    route = moe.route_sort_t(E, k, logits=logits)
    R = T * k
    xp, W1, W2, dY = randn(g, R, H), randn(g, E, 2 * I, H), randn(g, E, H, I), randn(g, R, H)
    for rows, off in ((R, route["offsets"]), (20, torch.tensor([0, 3, 3, 9, 20, 20, 20], dtype=torch.int32, device="cuda"))):
        Y1, h, Y2 = empty(rows, 2 * I), empty(rows, I), empty(rows, H)
        yield (f"ffn forward {rows}", lambda s, a=(xp, W1, W2, off, E, rows, H, I, Y1, h, Y2): moe.moe_ffn_forward(*a, stream=s), (Y1, h, Y2))
    kept = randn(g, R, 2 * I)
    dxp, dW1, dW2 = empty(R, H), empty(E, 2 * I, H), empty(E, H, I)
    n2 = moe.moe_ffn_backward_workspace_size(E, R, H, I)
    ws2 = workspace(n2)
    yield ("ffn backward", lambda s: moe.moe_ffn_backward(xp, W1, W2, kept, dY, route["offsets"], E, R, H, I, dxp, dW1, dW2, ws2, n2, stream=s),
           (dxp, dW1, dW2))
    dY2, dtw, dxt, dl = empty(R, H), empty(T, k, dtype=F32), empty(T, H), empty(T, E, dtype=F32)

    def routing(s):
        moe.moe_combine_backward(dy, xp, route["ids"], route["w"], route["row_pos"], T, k, H, E, dY2, dtw, stream=s)
        moe.moe_permute_backward(dY, route["ids"], route["row_pos"], T, k, H, E, dxt, stream=s)
        moe.moe_route_backward(logits, None, dtw, T, E, k, True, dl, stream=s)

    yield "routing backward", routing, (dY2, dtw, dxt, dl)
    W = randn(g, V, H, std=0.06)
    labels = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    loss, lse = empty(T, dtype=F32), empty(T, dtype=F32)
    n3 = moe.moe_cross_entropy_forward_workspace_size(T, H, V)
    ws3 = workspace(n3)
    yield ("cross entropy forward", lambda s: moe.moe_cross_entropy_forward(x, W, labels, T, H, V, -100, loss, lse, ws3, n3, stream=s), (loss, lse))
    given = torch.logsumexp(x.float() @ W.float().t(), 1)
    dloss = torch.full((T,), 1.0 / T, device="cuda")
    dxe, dWe = empty(T, H), empty(V, H)
    n4 = moe.moe_cross_entropy_backward_workspace_size(T, H, V)
    ws4 = workspace(n4)
    yield ("cross entropy backward", lambda s: moe.moe_cross_entropy_backward(x, W, labels, given, dloss, T, H, V, -100, dxe, dWe, ws4, n4, stream=s),
           (dxe, dWe))


def test_graphs_and_streams(moe):
    for name, call, outs in _steps(moe):
        call(None)
        torch.cuda.synchronize()
        want = [t.clone() for t in outs]
        for t in outs:
            t.zero_()
        other = torch.cuda.Stream()
        other.wait_stream(torch.cuda.current_stream())
        call(other)
        other.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), name
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(None)
        for _ in range(2):
            for t in outs:
                t.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs, want)), name
        assert moe.moe_get_device_error() == 0, name


def test_ignored_tokens_may_hold_anything(moe):
    """Rows of x (and their lse) whose label is ignored: NaN and infinities stay out of the loss and of every gradient."""
    g = gen(4)
    T, H, V = 140, 72, 700
    x, W = randn(g, T, H), randn(g, V, H, std=0.1)
    labels = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    out = torch.zeros(T, dtype=torch.bool, device="cuda")
    out[::3] = True
    labels[out] = -100
    dloss = torch.rand(T, generator=g, device="cuda")
    results = []
    for fill in (0.0, float("nan"), float("inf")):
        x1, d1 = x.clone(), dloss.clone()
        x1[out] = fill
        d1[out] = fill
        loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
        n = moe.moe_cross_entropy_forward_workspace_size(T, H, V)
        moe.moe_cross_entropy_forward(x1, W, labels, T, H, V, -100, loss, lse, workspace(n), n)
        dx, dW = torch.empty_like(x), torch.empty_like(W)
        n = moe.moe_cross_entropy_backward_workspace_size(T, H, V)
        moe.moe_cross_entropy_backward(x1, W, labels, lse, d1, T, H, V, -100, dx, dW, workspace(n), n)
        assert moe.moe_get_device_error() == 0
        results.append((loss, lse[~out], dx, dW))
    for other in results[1:]:
        assert all(torch.equal(a, b) for a, b in zip(results[0], other))

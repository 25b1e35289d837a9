"""A generation step by the library's calls alone: the layer for a few tokens, the
norm behind it, the vocabulary's product and the draw, as one captured graph."""
import pytest
import torch

from tests.gpu_helpers import require_gpu
from tests.test_gpu_sample import reference
from tests.train_helpers import HALF, gen, randn, workspace

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("T", [1, 6, 64])
def test_step(dtype, T):
    require_gpu()
    from grouped_gemm_serving_gb300 import moe
    from tests.test_gpu_forward_few import Layer, check
    g = gen(T)
    E, k, H, I, V = 16, 4, 512, 384, 5003
    padded = 5008   # the product's columns
    layer = Layer(g, dtype, E, H, I)
    head = torch.zeros(padded, H, dtype=torch.bfloat16, device="cuda")
    head[:V] = randn(g, V, H, std=2 * H ** -0.5)
    norm_w, norm_b = 1 + 0.1 * torch.randn(H, generator=g, device="cuda"), 0.1 * torch.randn(H, generator=g, device="cuda")
    offsets = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    x, router = randn(g, T, H), torch.randn(T, E, generator=g, device="cuda")
    u = torch.rand(T, generator=g, device="cuda")
    temperature, top_p = torch.full((T,), 0.8, device="cuda"), torch.full((T,), 0.9, device="cuda")
    top_k = torch.full((T,), 40, dtype=torch.int32, device="cuda")
    ids, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    out, hidden = torch.empty_like(x), torch.empty_like(x)
    logits = torch.empty(T, padded, dtype=torch.bfloat16, device="cuda")
    token, logprob = torch.empty(T, dtype=torch.int32, device="cuda"), torch.empty(T, device="cuda")
    args = moe.forward_args(dtype=moe.MOE_BF16 if dtype == "bf16" else moe.MOE_FP8_E4M3_B128, T=T, E=E, k=k, H=H, I=I, x=x, W1=layer.W1, W2=layer.W2,
                            W1_scales=layer.s1, W2_scales=layer.s2, out=out, logits=router, topk_ids=ids, topk_w=w)
    n = moe.moe_forward_few_workspace_size(args)
    ws = workspace(n)

    def step():
        moe.moe_forward_few(args, ws, n)
        moe.moe_layer_norm_forward(moe.MOE_BF16, out, H, T, H, moe.MOE_F32, norm_w, norm_b, 1e-5, hidden, H, None, None)
        moe.moe_grouped_gemm(moe.MOE_BF16, hidden, None, head, None, offsets, 1, T, padded, H, moe.MOE_EPI_STORE, logits, None)
        moe.moe_sample(moe.MOE_BF16, logits, padded, T, V, temperature, top_k, top_p, None, u, token, logprob)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2):
        h = gen(seed)
        x.copy_(randn(h, T, H))
        router.copy_(torch.randn(T, E, generator=h, device="cuda"))
        u.copy_(torch.rand(T, generator=h, device="cuda"))
        token.fill_(-1)
        graph.replay()
        torch.cuda.synchronize()
        assert moe.moe_get_device_error() == 0
        check(layer, x, ids, w, out)
        normed = torch.nn.functional.layer_norm(out.double(), (H,), norm_w.double(), norm_b.double(), 1e-5)
        assert bool(((hidden.double() - normed).abs() <= 1.02 * HALF * normed.abs() + 1e-5).all())
        product = hidden.double() @ head.double().t()
        assert bool(((logits.double() - product).abs() <= 1.02 * HALF * product.abs() + 1e-4).all())
        rows = logits[:, :V].double().cpu().numpy()
        for t in range(T):
            want = reference(rows[t], float(temperature[t]), 40, float(top_p[t]), 0.0, float(u[t]))
            assert int(token[t]) == want[0] and abs(float(logprob[t]) - want[1]) <= 1e-6 * abs(want[1]) + 1e-12

"""moe_sample on both sides of where the number of blocks a row changes: eight a row, or fewer where
there are more rows than fit at once and half the blocks still hold the row."""
import numpy as np
import pytest
import torch

from tests.gpu_helpers import require_gpu
from tests.test_gpu_sample import draw, gen, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    require_gpu()
    from grouped_gemm_serving_gb300 import moe as m
    yield m
    assert m.moe_get_device_error() == 0


# Tokens of a block: around 40960, an eighth of the largest vocabulary, and around 42600 in bf16 and
# 21296 in fp32, the most that two blocks an SM hold beside their histograms.
SLICES = {torch.bfloat16: [40952, 40960, 40968, 42000, 42592, 42600, 42608], torch.float32: [20480, 20488, 21000, 21288, 21296, 21304, 21312]}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("blocks,rows", [(4, 50), (2, 100), (1, 200)])   # on 152 SMs; on others another number of blocks
@pytest.mark.parametrize("at", range(7))
def test_largest_slices(moe, dtype, blocks, rows, at):
    """Ten rows with settings of their own, again and again."""
    n = 10
    V = SLICES[dtype][at] * blocks - 3 * (at % 2)   # the last block's slice is full, or is not
    rng = np.random.default_rng(V)
    logits = (3 * torch.randn(n, V, generator=gen(V), device="cuda")).to(dtype).repeat(rows // n, 1)
    settings = dict(top_k=[0, 0, 1, 50, 1000, 0, 50, 1000, 300, 0], top_p=[1.0, 0.9, 1.0, 1.0, 1.0, 0.5, 0.9, 0.9, 0.99, 0.999], u=rng.random(n).tolist())
    token, logprob = draw(moe, logits, **{name: v * (rows // n) for name, v in settings.items()})
    assert token == token[:n] * (rows // n) and logprob == logprob[:n] * (rows // n)
    l = logits[:n].double().cpu().numpy()
    for r in range(n):
        want = reference(l[r], 1.0, settings["top_k"][r], float(np.float32(settings["top_p"][r])), 0.0, float(np.float32(settings["u"][r])))
        assert token[r] == want[0] and abs(logprob[r] - want[1]) <= 1e-6 * abs(want[1]) + 1e-12, (r, token[r], logprob[r], want)

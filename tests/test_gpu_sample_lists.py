"""moe_sample where a cut falls among many tokens that are close to each other: lists that are
divided by their keys before they are ordered, lists of few values, bins that hold more than a list."""
import numpy as np
import pytest
import torch

from tests.gpu_helpers import require_gpu
from tests.test_gpu_sample import check, gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    require_gpu()
    from grouped_gemm_serving_gb300 import moe as m
    yield m
    assert m.moe_get_device_error() == 0


# Logits spread evenly over `width` below `top`.  A bin of the first histogram is 0.00677
# temperatures wide: these leave about 50 to 7000 tokens in one.
SPREADS = [(131072, 16.0, 3.0), (32000, 1.0, 7.5), (32000, 0.4, 0.2), (32000, 0.2, -5.0), (50257, 0.8, 0.4), (131072, 0.7, 100.0),
           (131072, 0.125, 0.0625), (5000, 0.0625, 1.0)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V,width,top", SPREADS)
@pytest.mark.parametrize("kind", ["p", "k", "k and p"])
def test_tokens_close_to_each_other(moe, dtype, V, width, top, kind):
    rows = 12
    rng = np.random.default_rng(V + int(1000 * width))
    logits = (top - width * torch.rand(rows, V, generator=gen(V), device="cuda")).to(dtype)
    pick = lambda *values: [values[i] for i in rng.integers(0, len(values), rows)]  # noqa: E731
    check(moe, logits, temperature=pick(0.5, 1.0, 1.0, 2.0), top_k=pick(300, 700, 1500, 4000) if "k" in kind else None,
          top_p=pick(0.01, 0.3, 0.6, 0.9, 0.999) if "p" in kind else None, u=rng.random(rows).tolist())


@pytest.mark.parametrize("values", [1, 2, 3, 40])
@pytest.mark.parametrize("kind", ["p", "k", "few k"])
def test_lists_of_few_values(moe, values, kind):
    """Neighbouring fp32 values, many tokens each: the order within them is the index."""
    rows, V = 10, 3000
    rng = np.random.default_rng(values)
    steps = torch.randint(0, values, (rows, V), generator=gen(values), device="cuda", dtype=torch.int32)
    logits = (torch.ones(rows, V, device="cuda").view(torch.int32) + steps).view(torch.float32)
    logits[:, ::3] = -4.0   # leaves 2000, and below 1024 with the next ones out too
    logits[::2, 1::3] = -30.0
    logits[1::4, 600:] = -30.0
    check(moe, logits, top_k=(rng.integers(257, 900, rows) if kind == "k" else rng.integers(1, 256, rows)).tolist() if "k" in kind else None,
          top_p=rng.random(rows).tolist() if kind == "p" else None, u=rng.random(rows).tolist())


def test_first_histogram_s_last_bin(moe):
    """Rows whose cut lies more than 20 octaves below the largest weight: most tokens in one bin."""
    rows, V = 8, 100000
    logits = -14.0 - 3.0 * torch.rand(rows, V, generator=gen(8), device="cuda")
    logits[:, 4711] = 0.0
    p = [1 - 2.0 ** -i for i in (7, 9, 10, 11, 12, 14, 20, 24)]
    check(moe, logits, top_p=p, u=[0.1, 0.95, 0.9999, 0.99999, 0.3, 0.99999, 0.999999, 0.9999999])
    check(moe, logits, top_k=[2, 257, 1000, 20000, 50000, 99998, 99999, 300], u=[0.999999] * rows)

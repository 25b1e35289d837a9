"""moe_sample with clusters whose blocks reach their first exchange at different times: rows so
short that most blocks of a cluster have no token and no load to wait for, in launches large enough
that clusters start all the time while others end."""
import numpy as np
import pytest
import torch

from tests.gpu_helpers import require_gpu
from tests.test_gpu_sample import check, draw, gen, logits_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    require_gpu()
    from grouped_gemm_serving_gb300 import moe as m
    yield m
    assert m.moe_get_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [1, 7, 9, 65, 100, 300])
@pytest.mark.parametrize("rows", [1, 37, 60, 150])   # eight blocks a row, eight, four, two or one
def test_blocks_without_tokens(moe, dtype, V, rows):
    rng = np.random.default_rng(V + rows)
    logits = logits_of(gen(V + rows), rows, V, dtype)
    pick = lambda *values: [values[i] for i in rng.integers(0, len(values), rows)]  # noqa: E731
    check(moe, logits, temperature=pick(0.0, 0.7, 1.0), top_k=pick(0, 1, 5, 50), top_p=pick(1.0, 0.5, 0.9), min_p=pick(0.0, 0.1), u=rng.random(rows).tolist())


def test_the_same_tokens_every_time(moe):
    """Many launches behind one another, without and with filters."""
    rows, V = 38, 100
    logits = logits_of(gen(1), rows, V, torch.float32)
    u = np.random.default_rng(1).random(rows).tolist()
    for settings in (dict(), dict(top_k=[5] * rows), dict(top_p=[0.7] * rows)):
        first = draw(moe, logits, u=u, **settings)
        for _ in range(50):
            assert draw(moe, logits, u=u, **settings) == first

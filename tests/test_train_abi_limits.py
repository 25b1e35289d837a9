"""Refusals of the training-step entry points on the host (small integers stand
for device pointers, so they run only where no kernel can launch) and workspace
sizes at the limits."""
import pytest
import torch

from grouped_gemm_serving_gb300 import build as gbuild

host_only = pytest.mark.skipif(torch.cuda.is_available(), reason="fake-pointer rejection tests run only without a GPU")


@pytest.fixture(scope="module")
def moe():
    gbuild.build()
    from grouped_gemm_serving_gb300 import moe as m
    return m


ROUTE_IDS = (16, 16, 16, 16, 4, 8, 2, 1, 16, None)


@host_only
@pytest.mark.parametrize("at,value", [(0, None), (2, None), (3, None), (8, None), (2, 20), (4, 0), (5, 257), (6, 9), (6, 33)])
def test_route_backward_ids_refuses(moe, at, value):
    args = list(ROUTE_IDS)
    args[at] = value
    assert moe.lib().moe_route_backward_ids(*args) == moe.MOE_ERR_INVALID_ARG

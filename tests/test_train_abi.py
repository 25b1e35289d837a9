"""The training-step entry points refuse bad arguments on the host, before
anything is launched (small integers stand for device pointers, so these run
only where no kernel can launch)."""
import pytest
import torch

from grouped_gemm_serving_gb300 import build as gbuild

host_only = pytest.mark.skipif(torch.cuda.is_available(), reason="fake-pointer rejection tests run only without a GPU")


@pytest.fixture(scope="module")
def moe():
    gbuild.build()
    from grouped_gemm_serving_gb300 import moe as m
    return m


NORM = (0, 16, 64, 4, 64, 0, 16, 16, 1e-5, 16, 64, 16, 16, None)
NORM_BACK = (0, 16, 64, 16, 64, 4, 64, 0, 16, 16, 16, 16, 64, 16, 16, 16, 1 << 20, None)
FFN = (16, 16, 16, 16, 8, 64, 64, 64, 16, 16, 16, None)
FFN_BACK = (16, 16, 16, 16, 16, 16, 8, 64, 64, 64, 16, 16, 16, 16, 1 << 30, None)
COMBINE = (16, 16, 16, 16, 16, 4, 2, 64, 8, 16, 16, None)
PERMUTE = (16, 16, 16, 4, 2, 64, 8, 16, None)
ROUTE = (16, 16, 16, 4, 8, 2, 1, 16, None)
XENT = (16, 16, 16, 4, 64, 500, -100, 16, 16, 16, 1 << 30, None)
XENT_BACK = (16, 16, 16, 16, 16, 4, 64, 500, -100, 16, 16, 16, 1 << 30, None)


def _with(args, **at):
    out = list(args)
    for i, v in at.items():
        out[int(i[1:])] = v
    return tuple(out)


@host_only
@pytest.mark.parametrize("name,args", [
    ("moe_layer_norm_forward", _with(NORM, _0=1)),               # FP8 rows
    ("moe_layer_norm_forward", _with(NORM, _0=2, _5=0)),         # fp32 rows with bf16 weights
    ("moe_layer_norm_forward", _with(NORM, _1=None)),
    ("moe_layer_norm_forward", _with(NORM, _1=17)),              # half an element off
    ("moe_layer_norm_forward", _with(NORM, _2=63)),              # rows that overlap
    ("moe_layer_norm_forward", _with(NORM, _3=0)),
    ("moe_layer_norm_forward", _with(NORM, _8=-1.0)),
    ("moe_layer_norm_forward", _with(NORM, _8=float("nan"))),
    ("moe_layer_norm_forward", _with(NORM, _6=8)),               # weight misaligned
    ("moe_layer_norm_backward", _with(NORM_BACK, _0=7)),
    ("moe_layer_norm_backward", _with(NORM_BACK, _9=None)),      # no mean
    ("moe_layer_norm_backward", _with(NORM_BACK, _12=63)),
    ("moe_layer_norm_backward", _with(NORM_BACK, _11=None, _13=None, _14=None)),   # nothing wanted
    ("moe_ffn_forward", _with(FFN, _3=None)),
    ("moe_ffn_forward", _with(FFN, _4=257)),
    ("moe_ffn_forward", _with(FFN, _5=0)),
    ("moe_ffn_forward", _with(FFN, _6=60)),
    ("moe_ffn_forward", _with(FFN, _7=4)),
    ("moe_ffn_forward", _with(FFN, _8=18)),
    ("moe_ffn_backward", _with(FFN_BACK, _3=None)),
    ("moe_ffn_backward", _with(FFN_BACK, _10=None, _11=None, _12=None)),
    ("moe_ffn_backward", _with(FFN_BACK, _0=None)),              # dW1 needs x
    ("moe_ffn_backward", _with(FFN_BACK, _13=24)),
    ("moe_combine_backward", _with(COMBINE, _0=None)),
    ("moe_combine_backward", _with(COMBINE, _6=33)),
    ("moe_combine_backward", _with(COMBINE, _7=60)),
    ("moe_combine_backward", _with(COMBINE, _9=8)),
    ("moe_permute_backward", _with(PERMUTE, _3=0)),
    ("moe_permute_backward", _with(PERMUTE, _5=12)),
    ("moe_permute_backward", _with(PERMUTE, _7=None)),
    ("moe_route_backward", _with(ROUTE, _4=257)),
    ("moe_route_backward", _with(ROUTE, _5=9)),
    ("moe_route_backward", _with(ROUTE, _7=None)),
    ("moe_cross_entropy_forward", _with(XENT, _1=None)),
    ("moe_cross_entropy_forward", _with(XENT, _3=0)),
    ("moe_cross_entropy_forward", _with(XENT, _4=60)),
    ("moe_cross_entropy_forward", _with(XENT, _5=0)),
    ("moe_cross_entropy_forward", _with(XENT, _5=2 ** 31 - 1)),
    ("moe_cross_entropy_forward", _with(XENT, _8=24)),
    ("moe_cross_entropy_forward", _with(XENT, _9=24)),
    ("moe_cross_entropy_backward", _with(XENT_BACK, _3=None)),
    ("moe_cross_entropy_backward", _with(XENT_BACK, _5=-1)),
    ("moe_cross_entropy_backward", _with(XENT_BACK, _9=None, _10=None)),   # nothing wanted
    ("moe_cross_entropy_backward", _with(XENT_BACK, _0=18)),
])
def test_refused(moe, name, args):
    assert getattr(moe.lib(), name)(*args) == moe.MOE_ERR_INVALID_ARG


@host_only
@pytest.mark.parametrize("name,args", [
    ("moe_layer_norm_backward", _with(NORM_BACK, _15=None)),
    ("moe_layer_norm_backward", _with(NORM_BACK, _16=64)),
    ("moe_ffn_backward", _with(FFN_BACK, _13=None)),
    ("moe_ffn_backward", _with(FFN_BACK, _14=1024)),
    ("moe_cross_entropy_forward", _with(XENT, _9=None)),
    ("moe_cross_entropy_forward", _with(XENT, _10=8)),
    ("moe_cross_entropy_backward", _with(XENT_BACK, _11=None)),
    ("moe_cross_entropy_backward", _with(XENT_BACK, _12=8)),
])
def test_workspace_missing(moe, name, args):
    assert getattr(moe.lib(), name)(*args) == moe.MOE_ERR_WORKSPACE


def test_workspace_sizes(moe):
    assert moe.moe_layer_norm_backward_workspace_size(0, 64) == 0
    assert moe.moe_layer_norm_backward_workspace_size(1, 64) >= 2 * 64 * 4
    assert moe.moe_ffn_backward_workspace_size(0, 64, 64, 64) == 0
    assert moe.moe_ffn_backward_workspace_size(8, 64, 64, 60) == 0
    assert moe.moe_ffn_backward_workspace_size(8, 64, 64, 64) >= 64 * 64 * 2 * 3   # dY1 and h
    assert moe.moe_cross_entropy_forward_workspace_size(0, 64, 500) == 0
    assert moe.moe_cross_entropy_backward_workspace_size(4, 60, 500) == 0
    # one piece: the gradient of all logits in bf16; many tokens: pieces of at least 2048 vocabulary rows
    assert moe.moe_cross_entropy_backward_workspace_size(64, 64, 512) >= 64 * 512 * 2 + 64 * 64 * 2
    assert moe.moe_cross_entropy_backward_workspace_size(1 << 17, 64, 131072) < 1 << 30

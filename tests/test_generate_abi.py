"""The generation step's entry points refuse bad arguments on the host, before
anything is launched (small integers stand for device pointers, so these run only
where no kernel can launch)."""
import ctypes as C

import pytest
import torch

from grouped_gemm_serving_gb300 import build as gbuild

host_only = pytest.mark.skipif(torch.cuda.is_available(), reason="fake-pointer rejection tests run only without a GPU")


@pytest.fixture(scope="module")
def moe():
    gbuild.build()
    from grouped_gemm_serving_gb300 import moe as m
    return m


# dtype, logits, ld, rows, V, temperature, top_k, top_p, min_p, u, token, logprob, stream
SAMPLE = (0, 16, 500, 4, 500, 16, 16, 16, 16, 16, 16, 16, None)


def _with(args, **at):
    out = list(args)
    for i, v in at.items():
        out[int(i[1:])] = v
    return tuple(out)


@host_only
@pytest.mark.parametrize("args", [
    _with(SAMPLE, _0=1),                # FP8 logits
    _with(SAMPLE, _0=7),
    _with(SAMPLE, _1=None),
    _with(SAMPLE, _1=17),               # half an element off
    _with(SAMPLE, _0=2, _1=18),
    _with(SAMPLE, _2=499),              # rows that overlap
    _with(SAMPLE, _3=0),
    _with(SAMPLE, _4=0),
    _with(SAMPLE, _4=-1, _2=0),
    _with(SAMPLE, _5=8),
    _with(SAMPLE, _6=20),
    _with(SAMPLE, _7=24),
    _with(SAMPLE, _8=4),
    _with(SAMPLE, _9=None),
    _with(SAMPLE, _9=24),
    _with(SAMPLE, _10=None),
    _with(SAMPLE, _10=20),
    _with(SAMPLE, _11=24),
])
def test_sample_refused(moe, args):
    assert moe.lib().moe_sample(*args) == moe.MOE_ERR_INVALID_ARG


@host_only
@pytest.mark.parametrize("args", [_with(SAMPLE, _2=400000, _4=327681), _with(SAMPLE, _3=(1 << 27) + 1)])
def test_sample_unsupported(moe, args):
    assert moe.lib().moe_sample(*args) == moe.MOE_ERR_UNSUPPORTED


def _args(moe, **kw):
    base = dict(dtype=moe.MOE_BF16, T=4, E=8, k=2, H=128, I=256, x=16, W1=16, W2=16, out=16, logits=16, topk_ids=16, topk_w=16)
    base.update(kw)
    return moe.forward_args(**base)


BAD = [dict(T=0), dict(T=-1), dict(E=0), dict(E=257), dict(k=0), dict(k=9), dict(E=64, k=33), dict(H=0), dict(H=12), dict(I=4), dict(I=20),
       dict(dtype=2), dict(dtype=1), dict(dtype=1, W1_scales=16, W2_scales=16, H=192), dict(dtype=1, W1_scales=16, W2_scales=16, I=64),
       dict(dtype=1, W1_scales=18, W2_scales=16), dict(dtype=1, W1_scales=16, W2_scales=2), dict(x=None), dict(W1=None), dict(W2=None),
       dict(out=None), dict(logits=None, topk_ids=None), dict(logits=None, topk_w=None), dict(x=8), dict(W1=24), dict(W2=20),
       dict(out=18), dict(logits=4), dict(topk_ids=4), dict(topk_w=8), dict(expert_bias=4)]


@host_only
@pytest.mark.parametrize("bad", BAD, ids=str)
def test_few_refused(moe, bad):
    assert moe.lib().moe_forward_few(C.byref(_args(moe, **bad)), 16, 1 << 30, None) == moe.MOE_ERR_INVALID_ARG


@host_only
def test_few_null(moe):
    assert moe.lib().moe_forward_few(None, 16, 1 << 30, None) == moe.MOE_ERR_INVALID_ARG
    assert moe.lib().moe_forward_few_workspace_size(None) == 0


UNSUPPORTED = [dict(T=65), dict(T=64, E=64, k=17), dict(T=33, E=64, k=32), dict(H=32776), dict(I=40000), dict(host_io=True), dict(gather=True),
               dict(fused_combine=True), dict(T=1 << 30)]


@host_only
@pytest.mark.parametrize("kw", UNSUPPORTED, ids=str)
def test_few_unsupported(moe, kw):
    a = _args(moe, **kw)
    assert moe.lib().moe_forward_few(C.byref(a), 16, 1 << 30, None) == moe.MOE_ERR_UNSUPPORTED
    assert moe.moe_forward_few_workspace_size(a) == 0


@host_only
def test_few_workspace(moe):
    a = _args(moe)
    n = moe.moe_forward_few_workspace_size(a)
    assert moe.lib().moe_forward_few(C.byref(a), None, n, None) == moe.MOE_ERR_WORKSPACE
    assert moe.lib().moe_forward_few(C.byref(a), 16, n - 1, None) == moe.MOE_ERR_WORKSPACE
    assert moe.lib().moe_forward_few(C.byref(a), 24, n, None) == moe.MOE_ERR_INVALID_ARG


def test_few_workspace_size(moe):
    rows = 4 * 2
    n = moe.moe_forward_few_workspace_size(_args(moe))
    assert n >= rows * 256 * 2 + rows * 128 * 4                      # h in bf16, y in fp32
    q = moe.moe_forward_few_workspace_size(_args(moe, dtype=moe.MOE_FP8_E4M3_B128, W1_scales=16, W2_scales=16))
    assert q >= n + rows * 256 * 2                                   # h in fp32
    assert moe.moe_forward_few_workspace_size(_args(moe, T=64, E=256, k=16, H=32768, I=32768)) > 1024 * 32768 * 6

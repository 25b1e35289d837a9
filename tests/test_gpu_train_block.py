"""The training step of examples/train_block.py: its gradients against automatic
differentiation of the same model in 64 bits, and a loss that falls."""
import importlib.util
import os

import pytest
import torch

from tests.gpu_helpers import require_gpu
from tests.train_helpers import HALF

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_block.py")


@pytest.fixture(scope="module")
def example():
    require_gpu()
    spec = importlib.util.spec_from_file_location("train_block", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _reference(block, tokens, labels, dloss, ids):
    """The same model in 64 bits with the picks given, differentiated automatically."""
    w = {n: t.double().requires_grad_() for n, t in block.w.items()}
    x = w["embed"][tokens].detach().requires_grad_()
    norm = torch.nn.functional.layer_norm
    n1 = norm(x, (block.H,), w["norm1"], w["bias1"], 1e-5)
    p = torch.softmax((n1 @ w["router"].t()).gather(1, ids), 1)
    out = torch.zeros_like(x)
    for e in range(block.E):
        for j in range(block.k):
            rows = (ids[:, j] == e).nonzero()[:, 0]
            z = n1[rows] @ w["W1"][e].t()
            y = (torch.nn.functional.silu(z[:, :block.I]) * z[:, block.I:]) @ w["W2"][e].t()
            out = out.index_add(0, rows, p[rows, j, None] * y)
    n2 = norm(x + out, (block.H,), w["norm2"], w["bias2"], 1e-5)
    loss = torch.nn.functional.cross_entropy(n2 @ w["head"].t(), labels.long(), ignore_index=-100, reduction="none")
    (loss * dloss.double()).sum().backward()
    return loss.detach(), dict({n: t.grad for n, t in w.items()}, embed=x.grad)


def test_gradients(example):
    block = example.Block(T=200, E=8, k=2, H=136, I=104, V=1003, seed=3)
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    tokens = torch.randint(0, block.V, (block.T,), generator=g, device="cuda")
    labels = torch.randint(0, block.V, (block.T,), generator=g, device="cuda", dtype=torch.int32)
    labels[::7] = -100
    dloss = torch.full((block.T,), 1.0 / int((labels != -100).sum()), device="cuda")
    loss = block.forward(tokens, labels)
    grads = block.backward(labels, dloss)
    assert example.moe.moe_get_device_error() == 0
    ref_loss, ref = _reference(block, tokens, labels, dloss, block.route["ids"].long())
    # Every activation on the way is rounded to bf16, some twenty times from the embedding to a gradient: errors of
    # at most HALF each, independent, so the whole is within 2 sqrt(20) HALF of the gradient's size
    assert ((loss.double() - ref_loss).abs() <= 20 ** 0.5 * HALF * (1 + ref_loss)).all()
    for name, got in grads.items():
        off = (got.double() - ref[name]).norm() / ref[name].norm()
        assert off <= 2 * 20 ** 0.5 * HALF, (name, float(off))


def test_loss_falls(example):
    losses = example.main(["--steps", "12", "--tokens", "512", "--experts", "8", "--topk", "2", "--hidden", "128",
                           "--intermediate", "128", "--vocab", "1000"])
    assert losses[-1] < losses[0] - 0.5

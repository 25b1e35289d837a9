"""One training step of a small model around the expert layer, with every
gradient computed by the library: layer norm -> router -> experts -> combine ->
residual -> layer norm -> softmax cross entropy, then the way back and a plain
gradient step on all weights.

    python examples/train_block.py [--steps 20] [--tokens 2048] [--vocab 32000]

Random weights and a synthetic task (every token has to name its successor in
a fixed permutation of the vocabulary); the loss falls from about log(vocab).
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from grouped_gemm_serving_gb300 import moe  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
IGNORE = -100


def empty(*shape, dtype=BF16):
    return torch.empty(*shape, dtype=dtype, device="cuda")


def scratch(nbytes):
    return empty(max(nbytes, 16), dtype=torch.uint8), nbytes


class Block:
    """The weights of the model, the buffers of a step of T tokens, and the step itself."""

    def __init__(self, T, E, k, H, I, V, seed=0):
        self.T, self.E, self.k, self.H, self.I, self.V = T, E, k, H, I, V
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def randn(*shape, std, dtype=BF16):
            return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

        self.w = dict(
            embed=randn(V, H, std=1.0), head=randn(V, H, std=H ** -0.5), router=randn(E, H, std=H ** -0.5, dtype=F32),
            norm1=torch.ones(H, device="cuda"), bias1=torch.zeros(H, device="cuda"),
            norm2=torch.ones(H, device="cuda"), bias2=torch.zeros(H, device="cuda"),
            W1=randn(E, 2 * I, H, std=H ** -0.5), W2=randn(E, H, I, std=I ** -0.5))
        R = T * k
        self.n1, self.mean1, self.rstd1 = empty(T, H), empty(T, dtype=F32), empty(T, dtype=F32)
        self.n2, self.mean2, self.rstd2 = empty(T, H), empty(T, dtype=F32), empty(T, dtype=F32)
        self.xp, self.Y1, self.h, self.Y2, self.out = empty(R, H), empty(R, 2 * I), empty(R, I), empty(R, H), empty(T, H)
        self.loss, self.lse = empty(T, dtype=F32), empty(T, dtype=F32)
        self.dn2, self.dhead = empty(T, H), empty(V, H)
        self.dr, self.dY2, self.dw = empty(T, H), empty(R, H), empty(T, k, dtype=F32)
        self.dxp, self.dn1, self.dx = empty(R, H), empty(T, H), empty(T, H)
        self.dW1, self.dW2 = empty(E, 2 * I, H), empty(E, H, I)
        self.dlogits = empty(T, E, dtype=F32)
        self.dnorm1, self.dbias1, self.dnorm2, self.dbias2 = (empty(H, dtype=F32) for _ in range(4))
        self.ws_norm = scratch(moe.moe_layer_norm_backward_workspace_size(T, H))
        self.ws_ffn = scratch(moe.moe_ffn_backward_workspace_size(E, R, H, I))
        self.ws_loss = scratch(moe.moe_cross_entropy_forward_workspace_size(T, H, V))
        self.ws_back = scratch(moe.moe_cross_entropy_backward_workspace_size(T, H, V))

    def norm(self, x, weight, bias, y, mean, rstd):
        moe.moe_layer_norm_forward(moe.MOE_BF16, x, self.H, self.T, self.H, moe.MOE_F32, weight, bias, 1e-5, y, self.H,
                                   mean, rstd)

    def norm_backward(self, dy, x, weight, mean, rstd, dx, dweight, dbias):
        moe.moe_layer_norm_backward(moe.MOE_BF16, dy, self.H, x, self.H, self.T, self.H, moe.MOE_F32, weight, mean, rstd,
                                    dx, self.H, dweight, dbias, *self.ws_norm)

    def forward(self, tokens, labels):
        T, E, k, H, I, w = self.T, self.E, self.k, self.H, self.I, self.w
        self.x = w["embed"][tokens]
        self.norm(self.x, w["norm1"], w["bias1"], self.n1, self.mean1, self.rstd1)
        self.logits = self.n1.float() @ w["router"].t()
        self.route = r = moe.route_sort_t(E, k, logits=self.logits)
        moe.moe_permute(moe.MOE_BF16, self.n1, None, T, H, k, r["sorted_rows"], r["offsets"], E, T * k, self.xp, None)
        moe.moe_ffn_forward(self.xp, w["W1"], w["W2"], r["offsets"], E, T * k, H, I, self.Y1, self.h, self.Y2)
        moe.moe_combine(self.Y2, r["ids"], r["w"], r["row_pos"], T, k, H, E, self.out)
        self.r = self.x + self.out
        self.norm(self.r, w["norm2"], w["bias2"], self.n2, self.mean2, self.rstd2)
        moe.moe_cross_entropy_forward(self.n2, w["head"], labels, T, H, self.V, IGNORE, self.loss, self.lse, *self.ws_loss)
        return self.loss

    def backward(self, labels, dloss):
        """Gradients of sum(dloss * loss) for every weight, by name (the embedding's by row of the batch)."""
        T, E, k, H, I, w, r = self.T, self.E, self.k, self.H, self.I, self.w, self.route
        moe.moe_cross_entropy_backward(self.n2, w["head"], labels, self.lse, dloss, T, H, self.V, IGNORE, self.dn2,
                                       self.dhead, *self.ws_back)
        self.norm_backward(self.dn2, self.r, w["norm2"], self.mean2, self.rstd2, self.dr, self.dnorm2, self.dbias2)
        moe.moe_combine_backward(self.dr, self.Y2, r["ids"], r["w"], r["row_pos"], T, k, H, E, self.dY2, self.dw)
        moe.moe_ffn_backward(self.xp, w["W1"], w["W2"], self.Y1, self.dY2, r["offsets"], E, T * k, H, I, self.dxp, self.dW1,
                             self.dW2, *self.ws_ffn)
        moe.moe_permute_backward(self.dxp, r["ids"], r["row_pos"], T, k, H, E, self.dn1)
        moe.moe_route_backward_ids(self.logits, None, r["ids"], self.dw, T, E, k, True, self.dlogits)
        drouter = self.dlogits.t() @ self.n1.float()
        self.dn1 += (self.dlogits @ w["router"]).to(BF16)
        self.norm_backward(self.dn1, self.x, w["norm1"], self.mean1, self.rstd1, self.dx, self.dnorm1, self.dbias1)
        self.dx += self.dr   # the residual
        return dict(embed=self.dx, head=self.dhead, router=drouter, norm1=self.dnorm1, bias1=self.dbias1,
                    norm2=self.dnorm2, bias2=self.dbias2, W1=self.dW1, W2=self.dW2)

    def step(self, tokens, labels, lr):
        loss = self.forward(tokens, labels)
        counts = (labels != IGNORE).sum()
        dloss = (1.0 / counts).to(F32).expand(self.T).contiguous()
        for name, grad in self.backward(labels, dloss).items():
            if name == "embed":
                self.w[name].index_add_(0, tokens, grad, alpha=-lr)
            else:
                self.w[name] -= (lr * grad).to(self.w[name].dtype)
        return loss.sum() / counts


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--experts", type=int, default=32)
    ap.add_argument("--topk", type=int, default=4)
    ap.add_argument("--hidden", type=int, default=512)
    ap.add_argument("--intermediate", type=int, default=512)
    ap.add_argument("--vocab", type=int, default=32000)
    ap.add_argument("--lr", type=float, default=2.0)
    a = ap.parse_args(argv)
    block = Block(a.tokens, a.experts, a.topk, a.hidden, a.intermediate, a.vocab)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    successor = torch.randperm(a.vocab, generator=g, device="cuda")
    used = torch.randperm(a.vocab, generator=g, device="cuda")[:max(1, a.tokens // 4)]
    losses = []
    for step in range(a.steps):
        tokens = used[torch.randint(0, used.numel(), (a.tokens,), generator=g, device="cuda")]
        labels = successor[tokens].to(torch.int32)
        labels[::16] = IGNORE   # as a prompt's tokens
        losses.append(block.step(tokens, labels, a.lr).item())
        print(f"step {step}: loss {losses[-1]:.4f}")
    if moe.moe_get_device_error() != 0:
        raise RuntimeError("a kernel reported an error")
    return losses


if __name__ == "__main__":
    main()

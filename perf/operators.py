"""The training-step operators next to the expert layer, as they are measured.

Each case is one pass through one of them, in its plain form (elementary torch
operations in 32 bits, rounded once at the end) or, with ``own`` set, through
the entry points of ``grouped_gemm_serving_gb300.moe``:

  ffn           the gated feed-forward block of the experts (one expert: a
                dense block); forward, or the gradients of x, W1 and W2
  xent          softmax cross entropy of tokens against a vocabulary matrix,
                without the logits being kept; forward, or the gradients of
                the tokens and of the matrix
  layer_norm    forward, or the gradients of x, the weight and the bias
  routing       the gradients of the combine, of the permute and of the top-k
                softmax, which a backward pass through the layer runs in turn

The sizes are those of this repository's synthetic layers (H = I = 2880 with
32 experts top-4, H = 2048 and I = 768 with 128 experts top-8, H = 7168) and
generic ones: vocabularies of 32000, 50257 and 131072, odd and ragged rows.
"""
import math

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
IGNORE = -100


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one generated token through its four experts of the 32-expert layer: latency, weights from memory
        dict(name="ffn fwd 1 token 32e", op="ffn", way="forward", E=32, busy=4, rows=4, spare=0, H=2880, I=2880, keep=False),
        # a small ragged batch: idle experts, rows of no expert, sizes that fill no tile
        dict(name="ffn fwd ragged", op="ffn", way="forward", E=8, busy=6, rows=1037, spare=19, H=1000, I=1368, keep=True),
        # the backward pass of a training step of the 32-expert layer: 4096 tokens, top-4
        dict(name="ffn bwd 32e", op="ffn", way="backward", E=32, busy=32, rows=16384, spare=0, H=2880, I=2880, keep=True),
        # scoring a few tokens (a short prompt's likelihood): the vocabulary matrix from memory
        dict(name="xent fwd 16 tokens", op="xent", way="forward", T=16, H=2048, V=32000, ignored=0.0),
        # the loss of a training step of 4096 tokens over a large vocabulary
        dict(name="xent fwd 4096", op="xent", way="forward", T=4096, H=2880, V=131072, ignored=0.0),
        # a fine-tuning batch: odd token count and vocabulary, the prompt's tokens carry no loss
        dict(name="xent bwd ragged", op="xent", way="backward", T=1021, H=1000, V=50257, ignored=0.3),
        # the gradient of that training step's loss
        dict(name="xent bwd 4096", op="xent", way="backward", T=4096, H=2880, V=131072, ignored=0.02),
        # the norm in front of the layer for one generated token: latency
        dict(name="norm fwd 1 row", op="layer_norm", way="forward", rows=1, H=2880, dtype="bf16", wdtype="bf16", bias=True, pad=0),
        # fp32 rows of an odd width in a wider buffer
        dict(name="norm bwd odd fp32", op="layer_norm", way="backward", rows=3001, H=1003, dtype="f32", wdtype="f32", bias=True, pad=5),
        # the backward pass of the norm in front of a wide layer, fp32 master weights
        dict(name="norm bwd 16384", op="layer_norm", way="backward", rows=16384, H=7168, dtype="bf16", wdtype="f32", bias=True, pad=0),
        # routing gradients of a small batch with sentinel slots
        dict(name="routing bwd 64", op="routing", way="backward", T=64, k=4, E=32, H=2880, sentinel=8, renorm=True),
        # routing gradients of the 128-expert layer's training step
        dict(name="routing bwd 8192", op="routing", way="backward", T=8192, k=8, E=128, H=2048, sentinel=0, renorm=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _eights(rng, lo, hi):
    return 8 * _log(rng, lo // 8, hi // 8)


def draw(rng):
    kind = rng.choice(["ffn forward", "ffn backward", "xent forward", "xent backward", "layer_norm forward",
                       "layer_norm backward", "routing backward"])
    op, way = kind.split()
    top = {c["op"] + " " + c["way"]: work(c) for c in listed()}  # the largest of each kind comes last
    while True:
        if op == "ffn":
            E = _log(rng, 1, 128)
            rows = _log(rng, 1, 16384)
            case = dict(op=op, way=way, E=E, busy=rng.randint(1, min(E, rows)), rows=rows,
                        spare=rng.choice([0, 0, rng.randint(1, 200)]), H=_eights(rng, 64, 7168), I=_eights(rng, 64, 5760),
                        keep=way == "backward" or rng.random() < 0.6)
            fits = 6 * E * case["H"] * case["I"] <= 2e9
            cap = top["ffn backward"]
        elif op == "xent":
            case = dict(op=op, way=way, T=_log(rng, 1, 8192), H=_eights(rng, 64, 7168), V=_log(rng, 100, 131072),
                        ignored=rng.choice([0.0, 0.1, 0.5]))
            fits = case["T"] * case["V"] <= 1 << 29
            cap = top["xent backward"]
        elif op == "layer_norm":
            dtype = rng.choice(["bf16", "bf16", "f32"])
            case = dict(op=op, way=way, rows=_log(rng, 1, 65536), H=_log(rng, 16, 16384), dtype=dtype,
                        wdtype=rng.choice([dtype, "f32"]), bias=rng.random() < 0.7, pad=rng.choice([0, 0, rng.randint(1, 64)]))
            fits, cap = True, top["layer_norm backward"]
        else:
            E = _log(rng, 2, 256)
            T, k = _log(rng, 1, 16384), rng.randint(1, min(E, 8))
            case = dict(op=op, way=way, T=T, k=k, E=E, H=_eights(rng, 64, 7168),
                        sentinel=rng.choice([0, rng.randint(0, T * k)]), renorm=rng.random() < 0.7)
            fits, cap = True, top["routing backward"]
        w = work(case)
        if fits and w["flops"] <= cap["flops"] and w["bytes"] <= max(cap["bytes"], 2e9 if op in ("ffn", "xent") else 0):
            return case


def work(case):
    c = case
    if c["op"] == "ffn":
        P, M, H, I = c["rows"], c["rows"] + c["spare"], c["H"], c["I"]
        weights = 3 * H * I * 2
        if c["way"] == "forward":
            return {"bytes": P * H * 2 + c["busy"] * weights + M * H * 2 + (M * 2 * I * 2 if c["keep"] else 0),
                    "flops": 6 * P * H * I}
        return {"bytes": P * (2 * H + 2 * I) * 2 + M * H * 2 + (c["busy"] + c["E"]) * weights, "flops": 12 * P * H * I}
    if c["op"] == "xent":
        T, H, V = c["T"], c["H"], c["V"]
        if c["way"] == "forward":
            return {"bytes": (T + V) * H * 2 + 12 * T, "flops": 2 * T * H * V}
        return {"bytes": 2 * (T + V) * H * 2 + 12 * T, "flops": 6 * T * H * V}
    if c["op"] == "layer_norm":
        n, e, w = c["rows"] * c["H"], 2 if c["dtype"] == "bf16" else 4, 2 if c["wdtype"] == "bf16" else 4
        if c["way"] == "forward":
            return {"bytes": 2 * n * e + (2 if c["bias"] else 1) * c["H"] * w + 8 * c["rows"], "flops": 7 * n}
        return {"bytes": 3 * n * e + (3 if c["bias"] else 2) * c["H"] * w + 8 * c["rows"], "flops": 14 * n}
    T, R, H, E = c["T"], c["T"] * c["k"], c["H"], c["E"]
    # dout and Y2 read, dY2 written; dxp read, dx written; the logits read, their gradient written
    return {"bytes": (2 * T + 3 * R) * H * 2 + 2 * T * E * 4 + R * 16, "flops": 5 * R * H + 6 * T * E}


# ---------------------------------------------------------------- inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape, std=1.0, dtype=BF16):
    return (torch.randn(*shape, generator=g, device="cuda", dtype=F32) * std).to(dtype)


def _weights(g, E, N, K, std):
    w = torch.empty(E, N, K, dtype=BF16, device="cuda")
    for e in range(E):
        w[e] = torch.randn(N, K, generator=g, device="cuda", dtype=F32) * std
    return w


def _counts(case, seed):
    """Rows of each expert: `busy` of them have at least one, skewed as a router's picks are."""
    g = torch.Generator()
    g.manual_seed(seed)
    E, busy, rows = case["E"], case["busy"], case["rows"]
    who = torch.randperm(E, generator=g)[:busy]
    share = torch.exp(0.5 * torch.randn(busy, generator=g))
    part = torch.multinomial(share, rows - busy, replacement=True, generator=g) if rows > busy else torch.zeros(0, dtype=torch.long)
    counts = torch.zeros(E, dtype=torch.long)
    counts[who] = 1 + torch.bincount(part, minlength=busy)
    return counts.tolist()


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case=case, buffers={})
    if case["op"] == "ffn":
        E, H, I, P = case["E"], case["H"], case["I"], case["rows"]
        M = P + case["spare"]
        counts = _counts(case, seed)
        ends = [sum(counts[:e]) for e in range(E + 1)]
        s["rows_of"] = [(e, ends[e], ends[e + 1]) for e in range(E) if counts[e]]
        s["offsets"] = torch.tensor(ends, dtype=torch.int32, device="cuda")
        s["x"] = _randn(g, M, H)
        s["x"][P:] = float("nan")  # rows of no expert are never read
        s["W1"], s["W2"] = _weights(g, E, 2 * I, H, 0.02), _weights(g, E, H, I, 0.02)
        if case["way"] == "backward":
            # what the forward pass kept: pre-activations of the spread that x and W1 give
            s["Y1"] = _randn(g, M, 2 * I, std=0.02 * math.sqrt(H))
            s["dy"] = _randn(g, M, H, std=1e-3)
            s["Y1"][P:] = float("nan")
            s["dy"][P:] = float("nan")
    elif case["op"] == "xent":
        T, H, V = case["T"], case["H"], case["V"]
        s["W"] = _weights(g, 1, V, H, 0.02)[0]
        s["labels"] = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
        # half of the tokens have learned their label, the others have not
        learned = (torch.rand(T, 1, generator=g, device="cuda") < 0.5).float() * (9.0 / (0.02 * 0.02 * H))
        s["x"] = (torch.randn(T, H, generator=g, device="cuda") + learned * s["W"][s["labels"].long()].float()).to(BF16)
        out = torch.rand(T, generator=g, device="cuda") < case["ignored"]
        s["labels"][out] = IGNORE
        if case["way"] == "backward":
            # the forward pass's log-sum-exp, and the gradient of a mean over the tokens that count
            s["lse"] = torch.cat([torch.logsumexp(x.float() @ s["W"].float().t(), 1) for x in s["x"].split(2048)])
            s["dloss"] = torch.full((T,), 1.0 / max(1, T - int(out.sum())), dtype=F32, device="cuda")
    elif case["op"] == "layer_norm":
        rows, H = case["rows"], case["H"]
        dt, wt = (BF16 if case["dtype"] == "bf16" else F32), (BF16 if case["wdtype"] == "bf16" else F32)
        ld = H + case["pad"]
        # hidden states: a spread per row, an offset common to it
        scale = torch.exp(torch.randn(rows, 1, generator=g, device="cuda") * 0.5)
        shift = torch.randn(rows, 1, generator=g, device="cuda") * 0.5
        s["x"] = (torch.randn(rows, ld, generator=g, device="cuda") * scale + shift).to(dt)[:, :H]
        s["weight"] = (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(wt)
        s["bias"] = _randn(g, H, std=0.1, dtype=wt) if case["bias"] else None
        if case["way"] == "backward":
            s["dy"] = _randn(g, rows, ld, std=1e-2, dtype=dt)[:, :H]
            x = s["x"].float()
            s["mean"] = x.mean(1)
            s["rstd"] = torch.rsqrt((x - s["mean"][:, None]).square().mean(1) + 1e-5)
    else:
        T, k, E, H = case["T"], case["k"], case["E"], case["H"]
        s["logits"] = torch.randn(T, E, generator=g, device="cuda")
        s["bias"] = 0.5 * torch.randn(E, generator=g, device="cuda")
        l = s["logits"] + s["bias"]
        top, ids = torch.topk(l, k, dim=1)
        s["w"] = (torch.softmax(top, 1) if case["renorm"] else torch.softmax(l, 1).gather(1, ids)).contiguous()
        ids = ids.to(torch.int32)
        ids.view(-1)[torch.randperm(T * k, generator=g, device="cuda")[:case["sentinel"]]] = E
        s["ids"] = ids
        order = torch.argsort(ids.view(-1), stable=True)
        s["row_pos"] = torch.empty(T * k, dtype=torch.int32, device="cuda")
        s["row_pos"][order] = torch.arange(T * k, dtype=torch.int32, device="cuda")
        s["dout"] = _randn(g, T, H, std=1e-3)
        s["Y2"] = _randn(g, T * k, H, std=0.3)
        s["dxp"] = _randn(g, T * k, H, std=1e-3)
        live = int((ids != E).sum())
        s["Y2"][live:] = 0  # what the forward and backward GEMMs write for rows of no expert
        s["dxp"][live:] = 0
    return s


# ---------------------------------------------------------------- one pass
def run(state):
    c = state["case"]
    side = _OWN if own else _PLAIN
    return side[c["op"] + " " + c["way"]](state, c)


# The plain forms: 32 bits, rounded once at the end.
def _plain_ffn_forward(s, c):
    M, H, I = c["rows"] + c["spare"], c["H"], c["I"]
    y = torch.zeros(M, H, dtype=BF16, device="cuda")
    kept = torch.zeros(M, 2 * I, dtype=BF16, device="cuda") if c["keep"] else None
    for e, a, b in s["rows_of"]:  # one product per expert
        z = s["x"][a:b].float() @ s["W1"][e].float().t()
        gate, up = z[:, :I], z[:, I:]
        y[a:b] = ((gate / (1 + torch.exp(-gate)) * up) @ s["W2"][e].float().t()).to(BF16)
        if kept is not None:
            kept[a:b] = z.to(BF16)
    return {"y": y, "Y1": kept} if c["keep"] else {"y": y}


def _plain_ffn_backward(s, c):
    M, H, I = c["rows"] + c["spare"], c["H"], c["I"]
    dx = torch.zeros(M, H, dtype=BF16, device="cuda")
    dW1, dW2 = torch.zeros_like(s["W1"]), torch.zeros_like(s["W2"])
    for e, a, b in s["rows_of"]:  # one set of products per expert
        x, dy, z = s["x"][a:b].float(), s["dy"][a:b].float(), s["Y1"][a:b].float()
        gate, up = z[:, :I], z[:, I:]
        sig = 1 / (1 + torch.exp(-gate))
        dh = dy @ s["W2"][e].float()
        dW2[e] = (dy.t() @ (gate * sig * up)).to(BF16)
        dz = torch.cat([dh * up * sig * (1 + gate * (1 - sig)), dh * gate * sig], 1)
        dx[a:b] = (dz @ s["W1"][e].float()).to(BF16)
        dW1[e] = (dz.t() @ x).to(BF16)
    return {"dx": dx, "dW1": dW1, "dW2": dW2}


def _plain_xent_forward(s, c):
    z = s["x"].float() @ s["W"].float().t()
    top = z.amax(1)
    lse = top + torch.log(torch.exp(z - top[:, None]).sum(1))
    counts = s["labels"] != IGNORE
    at = z.gather(1, s["labels"].clamp(min=0).long()[:, None])[:, 0]
    return {"loss": torch.where(counts, lse - at, torch.zeros_like(lse)), "lse": lse}


def _plain_xent_backward(s, c):
    x, W = s["x"].float(), s["W"].float()
    counts = (s["labels"] != IGNORE).float()[:, None]
    G = torch.exp(x @ W.t() - s["lse"][:, None])
    G.scatter_add_(1, s["labels"].clamp(min=0).long()[:, None], -torch.ones_like(counts))
    G *= counts * s["dloss"][:, None]
    return {"dx": (G @ W).to(BF16), "dW": (G.t() @ x).to(BF16)}


def _plain_norm_forward(s, c):
    x = s["x"].float()
    mean = x.mean(1)
    rstd = torch.rsqrt((x - mean[:, None]).square().mean(1) + 1e-5)
    y = (x - mean[:, None]) * rstd[:, None] * s["weight"].float()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return {"y": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}


def _plain_norm_backward(s, c):
    x, dy, w = s["x"].float(), s["dy"].float(), s["weight"].float()
    xh = (x - s["mean"][:, None]) * s["rstd"][:, None]
    g = dy * w
    dx = s["rstd"][:, None] * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    out = {"dx": dx.to(s["x"].dtype), "dweight": (dy * xh).sum(0).to(s["weight"].dtype)}
    if s["bias"] is not None:
        out["dbias"] = dy.sum(0).to(s["bias"].dtype)
    return out


def _plain_routing_backward(s, c):
    T, k, H, E = c["T"], c["k"], c["H"], c["E"]
    live = s["ids"] != E
    at = s["row_pos"].long().view(T, k)
    dout = s["dout"].float()[:, None, :]
    dY2 = torch.empty(T * k, H, dtype=BF16, device="cuda")
    dY2[at.view(-1)] = ((s["w"] * live)[:, :, None] * dout).to(BF16).view(T * k, H)
    dw = (s["Y2"][at].float() * dout).sum(2) * live
    dx = (s["dxp"][at].float() * live[:, :, None]).sum(1).to(BF16)
    l = s["logits"] + s["bias"]
    top, ids = torch.topk(l, k, dim=1)
    dlogits = torch.zeros_like(l)
    if c["renorm"]:
        p = torch.softmax(top, 1)
        dlogits.scatter_(1, ids, p * (dw - (p * dw).sum(1, keepdim=True)))
    else:
        p = torch.softmax(l, 1)
        full = torch.zeros_like(l).scatter_(1, ids, dw)
        dlogits = p * (full - (p * full).sum(1, keepdim=True))
    return {"dY2": dY2, "dtopk_w": dw, "dx": dx, "dlogits": dlogits}


_PLAIN = {"ffn forward": _plain_ffn_forward, "ffn backward": _plain_ffn_backward, "xent forward": _plain_xent_forward,
          "xent backward": _plain_xent_backward, "layer_norm forward": _plain_norm_forward,
          "layer_norm backward": _plain_norm_backward, "routing backward": _plain_routing_backward}


# The framework's entry points.
def _moe():
    from grouped_gemm_serving_gb300 import moe
    return moe


def _kept(s, name, make):
    """Outputs and workspaces live as long as the state, as a training loop keeps them."""
    if name not in s["buffers"]:
        s["buffers"][name] = make()
    return s["buffers"][name]


def _empty(*shape, dtype=BF16):
    return lambda: torch.empty(*shape, dtype=dtype, device="cuda")


def _workspace(s, size):
    def make():
        n = size()
        return torch.empty(max(n, 16), dtype=torch.uint8, device="cuda"), n
    return _kept(s, "ws", make)


def _own_ffn_forward(s, c):
    moe, M, H, I = _moe(), c["rows"] + c["spare"], c["H"], c["I"]
    y, h = _kept(s, "y", _empty(M, H)), _kept(s, "h", _empty(M, I))
    Y1 = _kept(s, "Y1", _empty(M, 2 * I)) if c["keep"] else None
    moe.moe_ffn_forward(s["x"], s["W1"], s["W2"], s["offsets"], c["E"], M, H, I, Y1, h, y)
    return {"y": y, "Y1": Y1} if c["keep"] else {"y": y}


def _own_ffn_backward(s, c):
    moe, M, H, I = _moe(), c["rows"] + c["spare"], c["H"], c["I"]
    dx = _kept(s, "dx", _empty(M, H))
    dW1, dW2 = _kept(s, "dW1", _empty(c["E"], 2 * I, H)), _kept(s, "dW2", _empty(c["E"], H, I))
    ws, n = _workspace(s, lambda: moe.moe_ffn_backward_workspace_size(c["E"], M, H, I))
    moe.moe_ffn_backward(s["x"], s["W1"], s["W2"], s["Y1"], s["dy"], s["offsets"], c["E"], M, H, I, dx, dW1, dW2, ws, n)
    return {"dx": dx, "dW1": dW1, "dW2": dW2}


def _own_xent_forward(s, c):
    moe, T, H, V = _moe(), c["T"], c["H"], c["V"]
    loss, lse = _kept(s, "loss", _empty(T, dtype=F32)), _kept(s, "lse", _empty(T, dtype=F32))
    ws, n = _workspace(s, lambda: moe.moe_cross_entropy_forward_workspace_size(T, H, V))
    moe.moe_cross_entropy_forward(s["x"], s["W"], s["labels"], T, H, V, IGNORE, loss, lse, ws, n)
    return {"loss": loss, "lse": lse}


def _own_xent_backward(s, c):
    moe, T, H, V = _moe(), c["T"], c["H"], c["V"]
    dx, dW = _kept(s, "dx", _empty(T, H)), _kept(s, "dW", _empty(V, H))
    ws, n = _workspace(s, lambda: moe.moe_cross_entropy_backward_workspace_size(T, H, V))
    moe.moe_cross_entropy_backward(s["x"], s["W"], s["labels"], s["lse"], s["dloss"], T, H, V, IGNORE, dx, dW, ws, n)
    return {"dx": dx, "dW": dW}


def _norm_types(moe, c):
    return [moe.MOE_BF16 if c[t] == "bf16" else moe.MOE_F32 for t in ("dtype", "wdtype")]


def _own_norm_forward(s, c):
    moe, rows, H, x = _moe(), c["rows"], c["H"], s["x"]
    y = _kept(s, "y", _empty(rows, H, dtype=x.dtype))
    mean, rstd = _kept(s, "mean", _empty(rows, dtype=F32)), _kept(s, "rstd", _empty(rows, dtype=F32))
    dt, wt = _norm_types(moe, c)
    moe.moe_layer_norm_forward(dt, x, x.stride(0), rows, H, wt, s["weight"], s["bias"], 1e-5, y, H, mean, rstd)
    return {"y": y, "mean": mean, "rstd": rstd}


def _own_norm_backward(s, c):
    moe, rows, H, x, dy = _moe(), c["rows"], c["H"], s["x"], s["dy"]
    dx = _kept(s, "dx", _empty(rows, H, dtype=x.dtype))
    dweight = _kept(s, "dweight", _empty(H, dtype=s["weight"].dtype))
    dbias = _kept(s, "dbias", _empty(H, dtype=s["weight"].dtype)) if s["bias"] is not None else None
    dt, wt = _norm_types(moe, c)
    ws, n = _workspace(s, lambda: moe.moe_layer_norm_backward_workspace_size(rows, H))
    moe.moe_layer_norm_backward(dt, dy, dy.stride(0), x, x.stride(0), rows, H, wt, s["weight"], s["mean"], s["rstd"],
                                dx, H, dweight, dbias, ws, n)
    out = {"dx": dx, "dweight": dweight}
    return dict(out, dbias=dbias) if dbias is not None else out


def _own_routing_backward(s, c):
    moe, T, k, H, E = _moe(), c["T"], c["k"], c["H"], c["E"]
    dY2, dw = _kept(s, "dY2", _empty(T * k, H)), _kept(s, "dw", _empty(T, k, dtype=F32))
    dx, dlogits = _kept(s, "dx", _empty(T, H)), _kept(s, "dlogits", _empty(T, E, dtype=F32))
    moe.moe_combine_backward(s["dout"], s["Y2"], s["ids"], s["w"], s["row_pos"], T, k, H, E, dY2, dw)
    moe.moe_permute_backward(s["dxp"], s["ids"], s["row_pos"], T, k, H, E, dx)
    moe.moe_route_backward(s["logits"], s["bias"], dw, T, E, k, c["renorm"], dlogits)
    return {"dY2": dY2, "dtopk_w": dw, "dx": dx, "dlogits": dlogits}


_OWN = {"ffn forward": _own_ffn_forward, "ffn backward": _own_ffn_backward, "xent forward": _own_xent_forward,
        "xent backward": _own_xent_backward, "layer_norm forward": _own_norm_forward,
        "layer_norm backward": _own_norm_backward, "routing backward": _own_routing_backward}


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    """What run() returns for these inputs, from the definitions in 64 bits: derivatives by automatic
    differentiation of the forward formula, row by row or piece by piece where that keeps it small."""
    s, c = prepare(case, seed), case
    if c["op"] == "ffn":
        return _exact_ffn(s, c)
    if c["op"] == "xent":
        return _exact_xent(s, c)
    if c["op"] == "layer_norm":
        return _exact_norm(s, c)
    return _exact_routing(s, c)


def _exact_ffn(s, c):
    M, H, I = c["rows"] + c["spare"], c["H"], c["I"]
    silu = torch.nn.functional.silu
    if c["way"] == "forward":
        y, Y1 = torch.zeros(M, H, dtype=F64, device="cuda"), torch.zeros(M, 2 * I, dtype=F64, device="cuda")
        for e, a, b in s["rows_of"]:
            Y1[a:b] = torch.einsum("ph,nh->pn", s["x"][a:b].double(), s["W1"][e].double())
            y[a:b] = torch.einsum("pi,hi->ph", silu(Y1[a:b, :I]) * Y1[a:b, I:], s["W2"][e].double())
        return {"y": y, "Y1": Y1} if c["keep"] else {"y": y}
    dx = torch.zeros(M, H, dtype=F64, device="cuda")
    dW1 = torch.zeros(s["W1"].shape, dtype=F64, device="cuda")
    dW2 = torch.zeros(s["W2"].shape, dtype=F64, device="cuda")
    for e, a, b in s["rows_of"]:
        Y1 = s["Y1"][a:b].double().requires_grad_()
        W2 = s["W2"][e].double().requires_grad_()
        y = torch.einsum("pi,hi->ph", silu(Y1[:, :I]) * Y1[:, I:], W2)
        dY1, dW2[e] = torch.autograd.grad(y, (Y1, W2), s["dy"][a:b].double())
        dx[a:b] = torch.einsum("pn,nh->ph", dY1, s["W1"][e].double())
        dW1[e] = torch.einsum("pn,ph->nh", dY1, s["x"][a:b].double())
    return {"dx": dx, "dW1": dW1, "dW2": dW2}


def _exact_xent(s, c):
    T = c["T"]
    W, labels = s["W"].double(), s["labels"].long()
    if c["way"] == "forward":
        loss, lse = torch.zeros(T, dtype=F64, device="cuda"), torch.zeros(T, dtype=F64, device="cuda")
        for a in range(0, T, 1024):
            logp = s["x"][a:a + 1024].double() @ W.t()
            lse[a:a + 1024] = torch.logsumexp(logp, 1)
            loss[a:a + 1024] = torch.nn.functional.cross_entropy(logp, labels[a:a + 1024], ignore_index=IGNORE, reduction="none")
        return {"loss": loss, "lse": lse}
    dx, dW = torch.zeros(s["x"].shape, dtype=F64, device="cuda"), torch.zeros_like(W)
    for a in range(0, T, 1024):
        x, label = s["x"][a:a + 1024].double(), labels[a:a + 1024]
        z = (x @ W.t()).requires_grad_()
        loss = torch.nn.functional.cross_entropy(z, label, ignore_index=IGNORE, reduction="none")
        G, = torch.autograd.grad(loss, z, s["dloss"][a:a + 1024].double())
        dx[a:a + 1024] = G @ W
        dW += G.t() @ x
        del z, loss, G
    return {"dx": dx, "dW": dW}


def _exact_norm(s, c):
    if c["rows"] * c["H"] > 1 << 28:
        return None
    x = s["x"].double().requires_grad_(c["way"] == "backward")
    w, b = s["weight"].double(), s["bias"].double() if s["bias"] is not None else None
    if c["way"] == "forward":
        var, mean = torch.var_mean(x, 1, unbiased=False)
        return {"y": torch.nn.functional.layer_norm(x, (c["H"],), w, b, 1e-5), "mean": mean, "rstd": (var + 1e-5) ** -0.5}
    w.requires_grad_()
    y = torch.nn.functional.layer_norm(x, (c["H"],), w, None, 1e-5)
    dx, dw = torch.autograd.grad(y, (x, w), s["dy"].double())
    out = {"dx": dx, "dweight": dw}
    return dict(out, dbias=s["dy"].double().sum(0)) if b is not None else out


def _exact_routing(s, c):
    T, k, E, H = c["T"], c["k"], c["E"], c["H"]
    at, live = s["row_pos"].long(), (s["ids"] != E).view(-1)
    w = s["w"].double().view(-1)
    dout = s["dout"].double()
    dY2 = torch.zeros(T * k, H, dtype=F64, device="cuda")
    dw = torch.zeros(T * k, dtype=F64, device="cuda")
    dx = torch.zeros(T, H, dtype=F64, device="cuda")
    for j in range(k):  # slot j of every token
        r, on = at[j::k], live[j::k].double()
        dY2[r] = (w[j::k] * on)[:, None] * dout
        dw[j::k] = torch.einsum("th,th->t", s["Y2"][r].double(), dout) * on
        dx += s["dxp"][r].double() * on[:, None]
    l = (s["logits"] + s["bias"]).double().requires_grad_()  # the router's sum is one 32-bit addition
    ids = torch.argsort(l.detach(), dim=1, descending=True, stable=True)[:, :k]
    p = torch.softmax(l.gather(1, ids), 1) if c["renorm"] else torch.softmax(l, 1).gather(1, ids)
    dlogits, = torch.autograd.grad(p, l, dw.view(T, k))
    return {"dY2": dY2, "dtopk_w": dw.view(T, k), "dx": dx, "dlogits": dlogits}

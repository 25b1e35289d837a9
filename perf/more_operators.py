"""The operators of a generation step around the expert layer, as they are measured.

Each case is one pass through one of them, in its plain form (elementary torch
operations in 32 bits, rounded once at the end; in 64 bits for the cumulative
sums that a draw is taken from) or, with ``own`` set, through the entry points
of ``grouped_gemm_serving_gb300.moe``:

  layer     the whole expert layer for a few tokens: top-k routing (or given
            ids and weights), gate_up, SwiGLU, down and the weighted sum, with
            bf16 weights or e4m3 weights scaled per 128 x 128 block
  sample    one token per row of logits: temperature, top-k, top-p and min-p
            by row, drawn with given uniform numbers

The sizes are those of this repository's synthetic layers (H = I = 2880 with
32 experts top-4, H = 2048 and I = 768 with 128 experts top-8, H = 7168 and
I = 2048 with 256 experts top-8 in FP8) and generic ones: vocabularies of
32000, 50257 and 131072, odd and ragged rows.
"""
import math

import torch

own = False

BF16, F32, F64, FP8 = torch.bfloat16, torch.float32, torch.float64, torch.float8_e4m3fn


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # one generated token in the 32-expert layer: latency, the weights of its four experts from memory
        dict(name="layer 1 token 32e", op="layer", dtype="bf16", T=1, E=32, k=4, H=2880, I=2880, routed=True, bias=True, renorm=True, sentinel=0),
        # five sequences on a rank that holds some of the experts: ids and weights given, slots of other ranks' experts, odd sizes
        dict(name="layer 5 tokens shard", op="layer", dtype="bf16", T=5, E=8, k=3, H=1000, I=1368, routed=False, bias=False, renorm=True, sentinel=4),
        # a small batch of sequences in the 128-expert layer, weights not renormalised
        dict(name="layer 11 tokens 128e", op="layer", dtype="bf16", T=11, E=128, k=8, H=2048, I=768, routed=True, bias=True, renorm=False, sentinel=0),
        # a full generation batch of the 32-expert layer: nearly all weights
        dict(name="layer 64 tokens 32e", op="layer", dtype="bf16", T=64, E=32, k=4, H=2880, I=2880, routed=True, bias=True, renorm=True, sentinel=0),
        # one generated token in the FP8 layer
        dict(name="layer 1 token fp8 256e", op="layer", dtype="fp8", T=1, E=256, k=8, H=7168, I=2048, routed=True, bias=True, renorm=True, sentinel=0),
        # a generation batch of the FP8 layer
        dict(name="layer 32 tokens fp8 256e", op="layer", dtype="fp8", T=32, E=256, k=8, H=7168, I=2048, routed=True, bias=True, renorm=True, sentinel=0),
        # one sequence with the usual filters: latency
        dict(name="sample 1 row", op="sample", dtype="bf16", rows=1, V=32000, pad=0, mode="k and p", banned=0.0),
        # a batch whose requests each bring their own settings, greedy ones among them; a grammar bans half the tokens
        dict(name="sample 33 rows mixed", op="sample", dtype="f32", rows=33, V=50257, pad=47, mode="mixed", banned=0.5),
        # a full batch over a large vocabulary, nucleus only: no top-k bounds the work
        dict(name="sample 64 rows top-p", op="sample", dtype="f32", rows=64, V=131072, pad=0, mode="p", banned=0.0),
        # a large batch with top-k
        dict(name="sample 256 rows top-k", op="sample", dtype="bf16", rows=256, V=131072, pad=0, mode="k", banned=0.0),
        # the whole distribution, only what is far below the best token cut off
        dict(name="sample 8 rows min-p", op="sample", dtype="bf16", rows=8, V=131072, pad=0, mode="min_p", banned=0.0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["layer", "layer", "sample"])
    most = {c["op"]: work(c)["bytes"] for c in listed() if c["name"] in ("layer 32 tokens fp8 256e", "sample 256 rows top-k")}
    while True:
        if op == "layer":
            dtype = rng.choice(["bf16", "fp8"])
            unit = 8 if dtype == "bf16" else 128
            E = _log(rng, 2, 256)
            T, k = _log(rng, 1, 64), rng.randint(1, min(E, 8))
            routed = rng.random() < 0.7
            case = dict(op=op, dtype=dtype, T=T, E=E, k=k, H=unit * _log(rng, -(-64 // unit), 7168 // unit),
                        I=unit * _log(rng, -(-64 // unit), 5760 // unit), routed=routed, bias=routed and rng.random() < 0.6,
                        renorm=rng.random() < 0.7, sentinel=rng.choice([0, 0, rng.randint(0, T * k)]))
            fits = 3 * E * case["H"] * case["I"] <= 4e9
        else:
            case = dict(op=op, dtype=rng.choice(["bf16", "f32"]), rows=_log(rng, 1, 256), V=_log(rng, 100, 262144),
                        pad=rng.choice([0, 0, rng.randint(1, 64)]), mode=rng.choice(["k and p", "mixed", "p", "k", "min_p"]),
                        banned=rng.choice([0.0, 0.0, 0.5]))
            fits = case["rows"] * case["V"] <= 256 * 131072
        if fits and work(case)["bytes"] <= most[op]:
            return case


def work(case):
    c = case
    if c["op"] == "layer":
        T, E, k, H, I = c["T"], c["E"], c["k"], c["H"], c["I"]
        slots = T * k - c["sentinel"]
        # experts with a row, taking the picks as even: those of the slots that no other slot shares
        busy = min(slots, E * (1 - (1 - 1 / E) ** slots))
        weights = 3 * H * I * 2 if c["dtype"] == "bf16" else 3 * H * I * (1 + 4 / 128 ** 2)
        routing = T * E * 4 + T * k * 8
        return {"bytes": busy * weights + 2 * T * H * 2 + routing, "flops": 6 * slots * H * I}
    n = c["rows"] * c["V"]
    return {"bytes": n * (2 if c["dtype"] == "bf16" else 4) + 28 * c["rows"], "flops": 5 * n}


# ---------------------------------------------------------------- inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape, std=1.0, dtype=BF16):
    return (torch.randn(*shape, generator=g, device="cuda", dtype=F32) * std).to(dtype)


def _weights(g, E, N, K, dtype):
    """Weights of standard deviation 0.02: bf16, or e4m3 with a scale per 128 x 128 block."""
    w = torch.empty(E, N, K, dtype=BF16 if dtype == "bf16" else FP8, device="cuda")
    std = 0.02 if dtype == "bf16" else 90.0   # blocks scaled so that their largest of 16384 is near 448
    for e in range(E):
        w[e] = (torch.randn(N, K, generator=g, device="cuda", dtype=F32) * std).clamp_(-448, 448).to(w.dtype)
    if dtype == "bf16":
        return w, None
    spread = torch.exp(0.3 * torch.randn(E, N // 128, K // 128, generator=g, device="cuda"))
    return w, 0.02 / std * spread


def prepare(case, seed):
    g, c = _generator(seed), case
    s = dict(case=case, buffers={})
    if c["op"] == "layer":
        T, E, k, H, I = c["T"], c["E"], c["k"], c["H"], c["I"]
        s["x"] = _randn(g, T, H)
        s["W1"], s["W1_scales"] = _weights(g, E, 2 * I, H, c["dtype"])
        s["W2"], s["W2_scales"] = _weights(g, E, H, I, c["dtype"])
        logits = torch.randn(T, E, generator=g, device="cuda")
        out = torch.zeros(T * k, dtype=torch.uint8, device="cuda")
        out[torch.randperm(T * k, generator=g, device="cuda")[:c["sentinel"]]] = 1
        if c["routed"]:
            s["logits"] = logits
            s["bias"] = 0.5 * torch.randn(E, generator=g, device="cuda") if c["bias"] else None
            s["mask"] = out if c["sentinel"] else None
        else:
            top, ids = torch.topk(logits, k, dim=1)
            s["ids"] = torch.where(out.view(T, k).bool(), E, ids).to(torch.int32)
            s["w"] = torch.softmax(top, 1).contiguous()
        return s
    rows, V = c["rows"], c["V"]
    dtype = BF16 if c["dtype"] == "bf16" else F32

    def rand(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    # logits as a language model's: they fall with the logarithm of the token's rank, steeper where it is sure
    steep = 1.0 + 1.5 * rand(rows, 1)
    rank = rand(rows, V + c["pad"]) * V + 1
    logits = 6.0 - steep * torch.log(rank) + 0.5 * torch.randn(rows, V + c["pad"], generator=g, device="cuda")
    if c["banned"]:
        logits.masked_fill_(rand(rows, V + c["pad"]) < c["banned"], -math.inf)
    s["logits"] = logits.to(dtype)[:, :V]
    s["u"] = rand(rows)
    pick = rand(rows, 4)
    mode = c["mode"]
    temperature = 0.6 + 0.6 * pick[:, 0]
    top_k = torch.tensor([20, 40, 50, 200], device="cuda")[(4 * pick[:, 1]).long()].to(torch.int32)
    top_p = torch.tensor([0.8, 0.9, 0.95, 0.99], device="cuda")[(4 * pick[:, 2]).long()]
    min_p = torch.tensor([0.02, 0.05, 0.1, 0.2], device="cuda")[(4 * pick[:, 3]).long()]
    if mode == "mixed":
        kind = torch.randint(0, 6, (rows,), generator=g, device="cuda")
        temperature = torch.where(kind == 0, 0.0, temperature)     # greedy
        top_k = torch.where((kind == 1) | (kind == 2), top_k, 0)   # 0: all tokens
        top_p = torch.where((kind == 2) | (kind == 3), top_p, 1.0)
        min_p = torch.where(kind == 4, min_p, 0.0)                 # kind 5: nothing but the temperature
    s["temperature"] = temperature
    s["top_k"] = top_k if mode in ("k", "k and p", "mixed") else None
    s["top_p"] = top_p if mode in ("p", "k and p", "mixed") else None
    s["min_p"] = min_p if mode in ("min_p", "mixed") else None
    return s


# ---------------------------------------------------------------- one pass
def run(state):
    c = state["case"]
    if own:
        return _own_layer(state, c) if c["op"] == "layer" else _own_sample(state, c)
    return _plain_layer(state, c) if c["op"] == "layer" else _plain_sample(state, c)


def _wide(w, scales, ids):
    """The weights of these experts in 32 bits."""
    v = w[ids].float()
    if scales is None:
        return v
    n, N, K = v.shape
    blocks = v.view(n, N // 128, 128, K // 128, 128) * scales[ids][:, :, None, :, None]
    return blocks.view(n, N, K)


def _plain_layer(s, c):
    T, E, k, I = c["T"], c["E"], c["k"], c["I"]
    if c["routed"]:
        l = s["logits"] + s["bias"] if s["bias"] is not None else s["logits"]
        top, ids = torch.sort(l, dim=1, descending=True, stable=True)   # ties to the lower id
        top, ids = top[:, :k], ids[:, :k]
        e = torch.exp(top - top[:, :1])
        w = e / (e if c["renorm"] else torch.exp(l - top[:, :1])).sum(1, keepdim=True)
        if s["mask"] is not None:
            ids = torch.where(s["mask"].view(T, k) != 0, E, ids)
    else:
        ids, w = s["ids"].long(), s["w"]
    live = (ids != E).float()
    at = ids.clamp(max=E - 1)
    x = s["x"].float()
    y = torch.empty(T, c["H"], dtype=F32, device="cuda")
    for t in range(T):  # one token's experts at a time: all of them at once would not fit
        z = _wide(s["W1"], s["W1_scales"], at[t]) @ x[t]
        gate, up = z[:, :I], z[:, I:]
        h = gate / (1 + torch.exp(-gate)) * up
        each = (_wide(s["W2"], s["W2_scales"], at[t]) @ h[:, :, None])[:, :, 0]
        y[t] = (each * (w[t] * live[t])[:, None]).sum(0)
    out = {"out": y.to(BF16)}
    return dict(out, ids=ids.to(torch.int32), w=w) if c["routed"] else out


def _plain_sample(s, c):
    """A draw is decided by where u falls among cumulative sums of all the weights, hence 64 bits."""
    z = s["logits"].double()
    rows, V = z.shape
    temperature = s["temperature"].double()[:, None]
    best = z.amax(1, keepdim=True)
    greedy = temperature <= 0
    w = torch.exp((z - best) / torch.where(greedy, torch.ones_like(temperature), temperature))
    order = torch.sort(s["logits"], dim=1, descending=True, stable=True).indices   # ties to the lowest index
    ranked = w.gather(1, order)
    place = torch.arange(V, device="cuda")[None, :]
    keep = torch.ones(rows, V, dtype=torch.bool, device="cuda")
    if s["top_k"] is not None:
        top_k = s["top_k"].long()[:, None]
        keep &= (place < top_k) | (top_k <= 0)
    if s["top_p"] is not None:
        top_p = s["top_p"].double()[:, None]
        ranked = ranked * keep
        before = torch.cumsum(ranked, 1) - ranked   # the weight of better tokens
        keep &= (before < top_p * ranked.sum(1, keepdim=True)) | (top_p >= 1) | (place == 0)
    if s["min_p"] is not None:
        keep &= ranked >= s["min_p"].double()[:, None]
    keep &= (place == 0) | ~greedy
    w = w * torch.zeros_like(keep).scatter_(1, order, keep)
    upto = torch.cumsum(w, 1)   # in the order of the vocabulary
    total = upto[:, -1:]
    token = (upto <= s["u"].double()[:, None] * total).sum(1, keepdim=True)
    logprob = torch.log(w.gather(1, token) / total)[:, 0]
    return {"token": token[:, 0].to(torch.int32), "logprob": logprob.float()}


def _moe():
    from grouped_gemm_serving_gb300 import moe
    return moe


def _kept(s, name, make):
    """Outputs, arguments and workspaces live as long as the state, as a serving loop keeps them."""
    if name not in s["buffers"]:
        s["buffers"][name] = make()
    return s["buffers"][name]


def _layer_call(s, c):
    moe, T, k, H = _moe(), c["T"], c["k"], c["H"]
    given = not c["routed"]
    ids = s["ids"] if given else torch.empty(T, k, dtype=torch.int32, device="cuda")
    w = s["w"] if given else torch.empty(T, k, dtype=F32, device="cuda")
    out = torch.empty(T, H, dtype=BF16, device="cuda")
    args = moe.forward_args(dtype=moe.MOE_BF16 if c["dtype"] == "bf16" else moe.MOE_FP8_E4M3_B128, T=T, E=c["E"], k=k, H=H,
                            I=c["I"], x=s["x"], W1=s["W1"], W2=s["W2"], W1_scales=s["W1_scales"], W2_scales=s["W2_scales"],
                            out=out, logits=None if given else s["logits"], expert_bias=None if given else s["bias"],
                            sentinel_mask=None if given else s["mask"], topk_ids=ids, topk_w=w, renormalize=c["renorm"])
    n = moe.moe_forward_few_workspace_size(args)
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    return args, ws, n, {"out": out} if given else {"out": out, "ids": ids, "w": w}


def _own_layer(s, c):
    args, ws, n, out = _kept(s, "call", lambda: _layer_call(s, c))
    _moe().moe_forward_few(args, ws, n)
    return out


def _own_sample(s, c):
    moe, rows = _moe(), c["rows"]
    token = _kept(s, "token", lambda: torch.empty(rows, dtype=torch.int32, device="cuda"))
    logprob = _kept(s, "logprob", lambda: torch.empty(rows, dtype=F32, device="cuda"))
    moe.moe_sample(moe.MOE_BF16 if c["dtype"] == "bf16" else moe.MOE_F32, s["logits"], s["logits"].stride(0), rows, c["V"],
                   s["temperature"], s["top_k"], s["top_p"], s["min_p"], s["u"], token, logprob)
    return {"token": token, "logprob": logprob}


# ---------------------------------------------------------------- 64 bits
def exact(case, seed):
    """What run() returns for these inputs, from the definitions in 64 bits: expert by expert, and row by row."""
    s, c = prepare(case, seed), case
    return _exact_layer(s, c) if c["op"] == "layer" else _exact_sample(s, c)


def _exact_layer(s, c):
    T, E, k, H, I = c["T"], c["E"], c["k"], c["H"], c["I"]
    if c["routed"]:
        l = s["logits"] if s["bias"] is None else s["logits"] + s["bias"]   # the router's sum is one 32-bit addition
        ids = torch.argsort(-l.double(), dim=1, stable=True)[:, :k]
        l = l.double()
        w = torch.softmax(l.gather(1, ids), 1) if c["renorm"] else torch.softmax(l, 1).gather(1, ids)
        if s["mask"] is not None:
            ids = ids.masked_fill(s["mask"].view(T, k).bool(), E)
    else:
        ids, w = s["ids"].long(), s["w"].double()
    y = torch.zeros(T, H, dtype=F64, device="cuda")

    def weight(name, e):
        v, scales = s[name][e].double(), s[name + "_scales"]
        if scales is not None:
            v = v * scales[e].double().repeat_interleave(128, 0).repeat_interleave(128, 1)
        return v

    for e in sorted(set(ids.flatten().tolist()) - {E}):
        tokens, slots = (ids == e).nonzero(as_tuple=True)
        z = torch.einsum("th,nh->tn", s["x"][tokens].double(), weight("W1", e))
        h = torch.nn.functional.silu(z[:, :I]) * z[:, I:]
        y.index_add_(0, tokens, torch.einsum("ti,hi->th", h, weight("W2", e)) * w[tokens, slots][:, None])
    return {"out": y, "ids": ids.to(torch.int32), "w": w} if c["routed"] else {"out": y}


def _exact_sample(s, c):
    token = torch.empty(c["rows"], dtype=torch.int32, device="cuda")
    logprob = torch.zeros(c["rows"], dtype=F64, device="cuda")
    for r in range(c["rows"]):
        z = s["logits"][r].double()
        if s["temperature"][r] <= 0:
            token[r] = int((z == z.max()).nonzero()[0])
            continue
        p = torch.softmax(z / s["temperature"][r].double(), 0)
        p, ids = torch.sort(p, descending=True, stable=True)   # the logits' order: the map is monotone
        n = c["V"]
        if s["top_k"] is not None and 0 < int(s["top_k"][r]) < n:
            n = int(s["top_k"][r])
        if s["top_p"] is not None and float(s["top_p"][r]) < 1:
            share = torch.cumsum(p[:n], 0) / p[:n].sum()
            n = min(n, 1 + int((share < s["top_p"][r].double()).sum()))
        if s["min_p"] is not None:
            n = min(n, max(1, int((p >= s["min_p"][r].double() * p[0]).sum())))
        kept, where = torch.sort(ids[:n])
        q = p[:n][where] / p[:n].sum()
        at = int(torch.searchsorted(torch.cumsum(q, 0), s["u"][r].double(), right=True).clamp(max=n - 1))
        token[r], logprob[r] = int(kept[at]), torch.log(q[at])
    return {"token": token, "logprob": logprob}

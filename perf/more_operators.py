"""Cases of the sequence operators: the token embedding with its weight's
gradient, and attention over packed documents, forward and backward.

A case's ``op`` names the pass:

  embed       embedding: the rows of the vocabulary's weight, scaled
  embed_grad  embedding_weight_grad: the gradient of all of the weight's rows
  attn        attention: causal or not, with capped scores (``cap``), a bias by
              distance (``slopes``), documents packed into the rows (``docs``,
              with ``pad`` tokens behind the last one), prefixes that all of
              their document sees (``prefix``, a share of its length)
  attn_grad   attention_backward of the same

With ``own`` false ``run`` computes the plain form (elementary torch
operations in 32 bits, rounded once); with ``own`` true it calls the
framework.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
PAD = 0              # the token that stands for none
MOST_SCORES = 32 * 8192 * 8192


# ---- cases -------------------------------------------------------------------

def listed():
    return [
        # one token of a decoder: latency
        {"name": "embed 1 token", "op": "embed", "T": 1, "D": 4096, "V": 32000, "weight": "bf16",
         "out": "bf16", "scale": 1.0, "padded": False},
        # a micro-batch over a large vocabulary into an fp32 residual stream,
        # scaled by the root of the width
        {"name": "embed 8k 131k", "op": "embed", "T": 8192, "D": 4096, "V": 131072,
         "weight": "bf16", "out": "f32", "scale": 64.0, "padded": True},
        # the gradient of a short ragged batch of fine-tuning examples in fp16
        {"name": "embed grad ragged f16", "op": "embed_grad", "T": 1037, "D": 1000, "V": 50021,
         "grad": "f16", "out": "f16", "scale": 1.0, "padded": True},
        # a micro-batch of pre-training, into the shard's fp32 gradient
        {"name": "embed grad 16k 131k", "op": "embed_grad", "T": 16384, "D": 4096, "V": 131072,
         "grad": "bf16", "out": "f32", "scale": 64.0, "padded": False},
        # one short example: latency
        {"name": "attn 1 x 60", "op": "attn", "B": 1, "S": 60, "Hq": 32, "Hk": 8, "D": 128,
         "dtype": "bf16", "causal": True, "cap": 0.0, "slopes": False, "docs": 0, "pad": 0,
         "prefix": 0.0},
        # a packed micro-batch with capped scores, a padded end
        {"name": "attn packed 4k capped", "op": "attn", "B": 1, "S": 4096, "Hq": 32, "Hk": 8,
         "D": 128, "dtype": "bf16", "causal": True, "cap": 50.0, "slopes": False, "docs": 9,
         "pad": 61, "prefix": 0.0},
        # five prompts with their answers: prefixes seen whole, a bias by
        # distance, odd lengths, fp16
        {"name": "attn prefix ragged f16", "op": "attn", "B": 5, "S": 777, "Hq": 12, "Hk": 12,
         "D": 80, "dtype": "f16", "causal": True, "cap": 0.0, "slopes": True, "docs": 0,
         "pad": 0, "prefix": 0.4},
        # a long context at the shard recipes' width
        {"name": "attn 8k causal", "op": "attn", "B": 1, "S": 8192, "Hq": 32, "Hk": 32, "D": 128,
         "dtype": "bf16", "causal": True, "cap": 0.0, "slopes": False, "docs": 0, "pad": 0,
         "prefix": 0.0},
        # the backward pass of the short example
        {"name": "attn grad 1 x 60", "op": "attn_grad", "B": 1, "S": 60, "Hq": 32, "Hk": 8,
         "D": 128, "dtype": "bf16", "causal": True, "cap": 0.0, "slopes": False, "docs": 0,
         "pad": 0, "prefix": 0.0},
        # of the packed micro-batch
        {"name": "attn grad packed 4k capped", "op": "attn_grad", "B": 1, "S": 4096, "Hq": 32,
         "Hk": 8, "D": 128, "dtype": "bf16", "causal": True, "cap": 50.0, "slopes": False,
         "docs": 9, "pad": 61, "prefix": 0.0},
        # of the prompts with their answers
        {"name": "attn grad prefix ragged f16", "op": "attn_grad", "B": 5, "S": 777, "Hq": 12,
         "Hk": 12, "D": 80, "dtype": "f16", "causal": True, "cap": 0.0, "slopes": True,
         "docs": 0, "pad": 0, "prefix": 0.4},
        # of the long context
        {"name": "attn grad 8k causal", "op": "attn_grad", "B": 1, "S": 8192, "Hq": 32, "Hk": 32,
         "D": 128, "dtype": "bf16", "causal": True, "cap": 0.0, "slopes": False, "docs": 0,
         "pad": 0, "prefix": 0.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "attn", "attn_grad"])
    half = rng.choice(["bf16", "f16"])
    if op in ("embed", "embed_grad"):
        d = _log(rng, 64, 4096)
        d = max(128, d // 128 * 128) if rng.random() < 0.6 else d
        c = {"op": op, "T": _log(rng, 1, 16384), "D": d, "V": _log(rng, 1000, 131072)}
        kind = rng.choice([half, "f32"])
        c |= {"weight" if op == "embed" else "grad": kind, "out": rng.choice([kind, "f32"])}
        return c | {"scale": rng.choice([1.0, 64.0]), "padded": rng.random() < 0.5}
    hk = rng.choice([1, 2, 3, 8])
    hq = hk * rng.choice([1, 1, 2, 4])
    most = int(math.sqrt(MOST_SCORES / hq))
    t = min(most, _log(rng, 1, 16384))
    b = rng.choice([1, 1, 2, 7])
    s = max(1, t // b)
    docs = rng.choice([0, 0, 1, _log(rng, 2, 40)])
    pad = min(b * s, rng.choice([0, rng.randint(1, 200)])) if docs else 0
    causal = rng.random() < 0.8
    return {"op": op, "B": b, "S": s, "Hq": hq, "Hk": hk,
            "D": rng.choice([64, 128, 128, 8 * rng.randint(2, 16)]), "dtype": half,
            "causal": causal, "cap": rng.choice([0.0, 0.0, 30.0, 50.0]),
            "slopes": rng.random() < 0.4, "docs": docs, "pad": pad,
            "prefix": rng.choice([0.0, 0.0, 0.3, 1.0]) if causal else 0.0}


# ---- inputs --------------------------------------------------------------------

def _lengths(case):
    """The lengths of a case's documents (or sequences): a few long ones, many
    short ones; they stand in another order with every seed."""
    if not case["docs"]:
        return [case["S"]] * case["B"]
    total, n = case["B"] * case["S"] - case["pad"], case["docs"]
    share = [(i + 1) ** -0.8 for i in range(n)]
    ends = [round(total * sum(share[:i + 1]) / sum(share)) for i in range(n)]
    return [b - a for a, b in zip([0] + ends, ends)]


def _prefixes(case, lengths):
    return [int(case["prefix"] * n) for n in lengths]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    s = {"case": dict(case)}
    if case["op"] in ("embed", "embed_grad"):
        T, D, V = case["T"], case["D"], case["V"]
        # tokens by rank: the n-th most frequent is 1 / n as frequent as the first
        rank = torch.exp(torch.rand(T, generator=gen, device="cuda") * math.log(V))
        s["tokens"] = (rank.long() - 1).clamp(0, V - 1)
        if case["op"] == "embed":
            s["w"] = (normal(V, D) / math.sqrt(D)).to(DTYPES[case["weight"]])
            return s
        s["grad"] = (normal(T, D) * 1e-2).to(DTYPES[case["grad"]])
        s["out"] = torch.empty(V, D, dtype=DTYPES[case["out"]], device="cuda")
        return s

    B, S, Hq, Hk, D = (case[k] for k in ("B", "S", "Hq", "Hk", "D"))
    T, dt = B * S, DTYPES[case["dtype"]]
    # what the projection of a layer's rows leaves: all heads of a token together
    qkv = normal(B, S, Hq + 2 * Hk, D)
    qkv[:, :, :Hq + Hk] *= 1.3
    qkv = qkv.to(dt)
    s["q"], s["k"], s["v"] = qkv.split([Hq, Hk, Hk], 2)
    lengths = _lengths(case)
    order = torch.randperm(len(lengths), generator=torch.Generator().manual_seed(seed)).tolist()
    lengths = [lengths[i] for i in order]
    s["offsets"], s["prefix"], s["slopes"] = None, None, None
    if case["docs"]:
        s["offsets"] = torch.tensor([0] + lengths, device="cuda").cumsum(0).to(torch.int32)
    if case["prefix"]:
        s["prefix"] = torch.tensor(_prefixes(case, lengths), dtype=torch.int32, device="cuda")
    if case["slopes"]:
        s["slopes"] = 2.0 ** (-8.0 * torch.arange(1, Hq + 1, device="cuda") / Hq)
    if case["op"] == "attn_grad":
        # what a forward pass left behind, and the gradient that comes back
        z, mask = _scores(s)[:2]
        p, lse = _softmax(z, mask)
        s["out"] = (p @ _heads(s["v"], Hq // Hk)).transpose(0, 1).reshape(B, S, Hq, D).to(dt)
        s["lse"] = lse.t().reshape(B, S, Hq).contiguous()
        s["grad"] = (normal(B, S, Hq, D) * 1e-2).to(dt)
    return s


# ---- plain forms ---------------------------------------------------------------

def _embed(s):
    c = s["case"]
    x = s["w"][s["tokens"]].float() * c["scale"]
    if c["padded"]:
        x = torch.where((s["tokens"] == PAD)[:, None], 0.0, x)
    return {"x": x.to(DTYPES[c["out"]])}


def _embed_grad(s):
    c = s["case"]
    g = s["grad"].float() * c["scale"]
    if c["padded"]:
        g = torch.where((s["tokens"] == PAD)[:, None], 0.0, g)
    out = torch.zeros(c["V"], c["D"], device="cuda").index_add_(0, s["tokens"], g)
    s["out"].copy_(out)
    return {"grad_w": s["out"]}


def _heads(x, group=1):
    """[B, S, H, D] -> fp32 [H * group, B S, D]."""
    x = x.flatten(0, 1).transpose(0, 1).float()
    return x.repeat_interleave(group, 0) if group > 1 else x


def _mask(s):
    """Which key (column) each query (row) sees, [T, T]."""
    c = s["case"]
    T = c["B"] * c["S"]
    at = torch.arange(T, device="cuda")
    if s["offsets"] is None:
        doc, first = at // c["S"], at // c["S"] * c["S"]
        inside = torch.ones_like(at, dtype=torch.bool)
    else:
        doc = torch.searchsorted(s["offsets"].long(), at, right=True) - 1
        first, inside = s["offsets"].long()[doc], at < s["offsets"][-1]
    mask = (doc[:, None] == doc) & inside[:, None] & inside
    if c["causal"]:
        seen = at[:, None] >= at
        if s["prefix"] is not None:
            most = s["prefix"].shape[0] - 1
            seen = seen | (at < first + s["prefix"].long()[doc.clamp(max=most)])
        mask = mask & seen
    return mask


def _scores(s):
    """(scores [Hq, T, T], mask, tanh of the capped ones)."""
    c = s["case"]
    z = _heads(s["q"]) @ _heads(s["k"], c["Hq"] // c["Hk"]).transpose(1, 2)
    z.mul_(1.0 / math.sqrt(c["D"]))
    t = None
    if c["cap"]:
        t = torch.tanh(z / c["cap"])
        z = t * c["cap"]
    if c["slopes"]:
        at = torch.arange(z.shape[1], device="cuda")
        z = z - s["slopes"][:, None, None] * (at[:, None] - at).abs().float()
    return z, _mask(s), t


def _softmax(z, mask):
    """(probabilities, lse [Hq, T]); a row that sees nothing has none."""
    z = z.masked_fill(~mask, -math.inf)
    top = z.amax(2, keepdim=True)
    p = torch.exp(z - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(2, keepdim=True)
    lse = (top + total.log())[:, :, 0]
    return p / torch.where(total == 0, 1.0, total), lse


def _attn(s):
    c = s["case"]
    z, mask, _ = _scores(s)
    p, lse = _softmax(z, mask)
    out = p @ _heads(s["v"], c["Hq"] // c["Hk"])
    shape = (c["B"], c["S"], c["Hq"])
    return {"out": out.transpose(0, 1).reshape(*shape, c["D"]).to(s["q"].dtype),
            "lse": lse.t().reshape(shape)}


def _attn_grad(s):
    c = s["case"]
    group, dt = c["Hq"] // c["Hk"], s["q"].dtype
    z, mask, t = _scores(s)
    lse = s["lse"].flatten(0, 1).t()[:, :, None]
    p = torch.exp((z - lse).masked_fill_(~mask, -math.inf))
    del z
    go, q = _heads(s["grad"]), _heads(s["q"])
    gv = p.transpose(1, 2) @ go
    dz = go @ _heads(s["v"], group).transpose(1, 2)
    dz.sub_((go * _heads(s["out"])).sum(2, keepdim=True)).mul_(p)
    del p
    if t is not None:
        dz.mul_(1.0 - t * t)
    dz.masked_fill_(~mask, 0.0).mul_(1.0 / math.sqrt(c["D"]))
    gq = dz @ _heads(s["k"], group)
    gk = dz.transpose(1, 2) @ q

    def tokens(x, heads):     # summed over the query heads that share one
        x = x.view(heads, -1, *x.shape[1:]).sum(1)
        return x.transpose(0, 1).reshape(c["B"], c["S"], heads, c["D"]).to(dt)

    return {"q": tokens(gq, c["Hq"]), "k": tokens(gk, c["Hk"]), "v": tokens(gv, c["Hk"])}


# ---- the framework's calls -------------------------------------------------------

def _own_embed(s):
    import adamw_optimizer_step_persistent_gb300 as fadam
    c = s["case"]
    return {"x": fadam.embedding(s["tokens"], s["w"], scale=c["scale"], dtype=DTYPES[c["out"]],
                                 padding_index=PAD if c["padded"] else None)}


def _own_embed_grad(s):
    import adamw_optimizer_step_persistent_gb300 as fadam
    c = s["case"]
    return {"grad_w": fadam.embedding_weight_grad(s["grad"], s["tokens"], out=s["out"],
                                                  scale=c["scale"],
                                                  padding_index=PAD if c["padded"] else None)}


def _own_attn(s):
    import adamw_optimizer_step_persistent_gb300 as fadam
    c = s["case"]
    r = fadam.attention(s["q"], s["k"], s["v"], causal=c["causal"], softcap=c["cap"],
                        slopes=s["slopes"], documents=s["offsets"], prefix=s["prefix"])
    return {"out": r.out, "lse": r.lse}


def _own_attn_grad(s):
    import adamw_optimizer_step_persistent_gb300 as fadam
    c = s["case"]
    r = fadam.attention_backward(s["grad"], s["q"], s["k"], s["v"], s["out"], s["lse"],
                                 causal=c["causal"], softcap=c["cap"], slopes=s["slopes"],
                                 documents=s["offsets"], prefix=s["prefix"])
    return {"q": r.q, "k": r.k, "v": r.v}


_PLAIN = {"embed": _embed, "embed_grad": _embed_grad, "attn": _attn, "attn_grad": _attn_grad}
_OWN = {"embed": _own_embed, "embed_grad": _own_embed_grad, "attn": _own_attn,
        "attn_grad": _own_attn_grad}


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ---- what a pass cannot do without -------------------------------------------------

def _pairs(case):
    """Pairs of a query and a key that it sees, of one head."""
    total = 0
    for n, p in zip(_lengths(case), _prefixes(case, _lengths(case))):
        total += n * (n + 1) // 2 + p * (p - 1) // 2 if case["causal"] else n * n
    return total


def work(case):
    size = {"bf16": 2, "f16": 2, "f32": 4}
    if case["op"] in ("embed", "embed_grad"):
        T, D, V = case["T"], case["D"], case["V"]
        # different tokens among T that are 1 / n frequent, n = 1 .. V
        log_v = math.log(V)
        seen = min(T, sum(1.0 - math.exp(-T * math.log1p(1.0 / n) / log_v) for n in range(1, V)))
        if case["op"] == "embed":
            return {"bytes": seen * D * size[case["weight"]] + T * D * size[case["out"]] + 8 * T,
                    "flops": T * D}
        return {"bytes": T * D * size[case["grad"]] + V * D * size[case["out"]] + 8 * T,
                "flops": T * D}
    T, Hq, Hk, D = case["B"] * case["S"], case["Hq"], case["Hk"], case["D"]
    rows_q, rows_k = 2 * T * Hq * D, 2 * T * Hk * D
    if case["op"] == "attn":
        return {"bytes": 2 * rows_q + 2 * rows_k + 4 * T * Hq, "flops": 4 * D * Hq * _pairs(case)}
    # q, k, v, out, its gradient and lse in; three gradients out
    return {"bytes": 4 * rows_q + 4 * rows_k + 4 * T * Hq, "flops": 10 * D * Hq * _pairs(case)}


# ---- the definition in 64 bits -------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "embed":
        w = s["w"].double() * c["scale"]
        x = w[s["tokens"]]
        if c["padded"]:
            x[s["tokens"] == PAD] = 0
        return {"x": x}
    if c["op"] == "embed_grad":
        counted = s["tokens"] != PAD if c["padded"] else torch.ones_like(s["tokens"], dtype=torch.bool)
        out = torch.zeros(c["V"], c["D"], dtype=torch.float64, device="cuda")
        out.index_put_((s["tokens"][counted],), s["grad"][counted].double() * c["scale"],
                       accumulate=True)
        return {"grad_w": out}
    if 10 * c["D"] * c["Hq"] * (c["B"] * c["S"]) ** 2 > 8e12:
        return None
    Hq, Hk, D, T = c["Hq"], c["Hk"], c["D"], c["B"] * c["S"]
    lengths = [c["S"]] * c["B"]
    if s["offsets"] is not None:
        ends = s["offsets"].tolist()
        lengths = [b - a for a, b in zip(ends, ends[1:])]
    prefixes = [0] * len(lengths) if s["prefix"] is None else s["prefix"].tolist()
    q, k, v = (s[n].reshape(T, -1, D).double() for n in "qkv")
    grads = c["op"] == "attn_grad"
    go = s["grad"].reshape(T, Hq, D).double() if grads else None
    out, lse = torch.zeros_like(q), torch.full((T, Hq), -math.inf, dtype=torch.float64, device="cuda")
    gq, gk, gv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    start = 0
    for n, p in zip(lengths, prefixes):       # document by document, head by head
        rows = slice(start, start + n)
        start += n
        if n == 0:
            continue
        apart = torch.arange(n, device="cuda")[:, None] - torch.arange(n, device="cuda")[None]
        hidden = apart < 0
        hidden[:, :p] = False
        for h in range(Hq):
            kh, vh = k[rows, h * Hk // Hq], v[rows, h * Hk // Hq]
            z = q[rows, h] @ kh.T / math.sqrt(D)
            slope = 1.0
            if c["cap"]:
                t = torch.tanh(z / c["cap"])
                z, slope = c["cap"] * t, 1 - t ** 2
            if s["slopes"] is not None:
                z = z - s["slopes"][h].double() * apart.abs()
            if c["causal"]:
                z[hidden] = -math.inf
            a = torch.softmax(z, 1)
            lse[rows, h] = torch.logsumexp(z, 1)
            out[rows, h] = a @ vh
            if grads:
                da = go[rows, h] @ vh.T
                dz = slope * a * (da - (a * da).sum(1, keepdim=True)) / math.sqrt(D)
                gq[rows, h] = dz @ kh
                gk[rows, h * Hk // Hq] += dz.T @ q[rows, h]
                gv[rows, h * Hk // Hq] += a.T @ go[rows, h]
    shape = (c["B"], c["S"])
    if grads:
        return {"q": gq.reshape(*shape, Hq, D), "k": gk.reshape(*shape, Hk, D),
                "v": gv.reshape(*shape, Hk, D)}
    return {"out": out.reshape(*shape, Hq, D), "lse": lse.reshape(*shape, Hq)}

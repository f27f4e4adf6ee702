"""What the serving operators are measured on.

Three operators over the quantizer's output: products with 4-bit codes and
group scales (one matrix), the same grouped by expert over rows sorted by
expert, and the log probabilities, entropy and top alternatives of logits.

``own`` false: the plain form, elementary torch operations in float32.
``own`` true: the calls a user makes of post_mixed_precision_amd.
"""
import math
import random

import torch

own = False

DEV = "cuda:0"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    def lin(name, t, n, m, g, x, y):
        return {"name": name, "op": "linear", "t": t, "n": n, "m": m, "g": g, "x": x, "y": y}

    def exp(name, e, tokens, top, n, m, g, x, y, gather, weighted):
        return {"name": name, "op": "experts", "e": e, "tokens": tokens, "top": top, "n": n, "m": m, "g": g,
                "x": x, "y": y, "gather": gather, "weighted": weighted}

    def lp(name, t, v, pad, x, top):
        return {"name": name, "op": "logprobs", "t": t, "v": v, "pad": pad, "x": x, "top": top}

    return [
        # one token through a 7B attention projection: launch and latency
        lin("linear-token-4096", 1, 4096, 4096, 128, "bf16", "bf16"),
        # one token through the 70B-shaped MLP projection: the weights' bytes
        lin("linear-token-28672x8192", 1, 28672, 8192, 128, "bf16", "f32"),
        # a decode batch through the 13B-shaped MLP projection
        lin("linear-batch16-13824x5120", 16, 13824, 5120, 64, "bf16", "bf16"),
        # a short float32 prompt, odd sizes, the smallest groups
        lin("linear-odd-f32", 77, 1003, 1056, 32, "f32", "f32"),
        # one calibration sequence through the 7B down projection
        lin("linear-prompt-4096x11008", 2048, 4096, 11008, 128, "bf16", "bf16"),
        # two tokens, two experts each: most experts idle
        exp("experts-step", 8, 2, 2, 4096, 4096, 128, "bf16", "bf16", True, False),
        # a decode batch over many small experts, weighted by the router's gates
        exp("experts-batch-64", 64, 128, 8, 1024, 2048, 64, "bf16", "f32", False, True),
        # a prompt over eight 7B-shaped MLPs, gathered from the token order
        exp("experts-prompt-11008", 8, 2048, 2, 11008, 4096, 128, "bf16", "bf16", True, False),
        # one sampled token with its alternatives
        lp("score-token", 1, 32000, 0, "f32", 5),
        # a decode batch over a large vocabulary, bfloat16 logits (ties)
        lp("score-step-131072", 16, 131072, 0, "bf16", 20),
        # a ragged piece of text, rows padded past the vocabulary
        lp("score-odd", 333, 100003, 13, "f32", 1),
        # perplexity of one calibration sequence
        lp("score-corpus", 2048, 32000, 0, "f32", 0),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng: random.Random):
    op = rng.choice(["linear", "linear", "experts", "logprobs"])
    if op == "linear":
        while True:
            g = rng.choice([32, 64, 128])
            c = {"op": op, "t": _logint(rng, 1, 2048), "n": _logint(rng, 64, 28672),
                 "m": g * _logint(rng, 2, 11008 // g), "g": g, "x": rng.choice(["bf16", "bf16", "f32"]),
                 "y": rng.choice(["bf16", "f32"])}
            if c["t"] * c["n"] * c["m"] * (3 if c["x"] == "f32" else 1) <= 2048 * 4096 * 11008:
                return c
    if op == "experts":
        while True:
            g = rng.choice([32, 64, 128])
            e = _logint(rng, 2, 64)
            c = {"op": op, "e": e, "tokens": _logint(rng, 1, 2048), "top": rng.randint(1, min(8, e)),
                 "n": _logint(rng, 64, 11008), "m": g * _logint(rng, 2, 8192 // g), "g": g,
                 "x": rng.choice(["bf16", "bf16", "f32"]), "y": rng.choice(["bf16", "f32"]),
                 "gather": rng.random() < 0.5, "weighted": rng.random() < 0.5}
            if (c["tokens"] * c["top"] * c["n"] * c["m"] * (3 if c["x"] == "f32" else 1) <= 4096 * 11008 * 4096
                    and e * c["n"] * c["m"] <= 8 * 11008 * 4096):
                return c
    while True:
        v = _logint(rng, 1000, 200000)
        c = {"op": op, "t": _logint(rng, 1, 2048), "v": v, "pad": rng.choice([0, 0, rng.randint(1, 64)]),
             "x": rng.choice(["bf16", "f32"]), "top": rng.choice([0, 1, 5, 20, 32])}
        if c["t"] * v <= 2048 * 32000:
            return c


def _rows(case):
    return case["tokens"] * case["top"]


def _assignment(case):
    """Rows per expert, uneven, with idle experts: the assignment a router with
    unequal favour makes, fixed by the case's sizes."""
    rng = random.Random(case["e"] * 1000003 + case["tokens"] * 101 + case["top"])
    favour = [rng.random() ** 2 + 1e-3 for _ in range(case["e"])]
    picks = []
    for tok in range(case["tokens"]):
        left = list(range(case["e"]))
        for _ in range(case["top"]):
            j = rng.choices(range(len(left)), weights=[favour[x] for x in left])[0]
            picks.append((left.pop(j), tok))
    picks.sort()
    counts = [0] * case["e"]
    for x, _ in picks:
        counts[x] += 1
    bounds = [0]
    for n in counts:
        bounds.append(bounds[-1] + n)
    return bounds, [tok for _, tok in picks]


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _activations(gen, t, m, dt):
    """Gaussian rows with a few strong channels, as hidden states have them."""
    x = torch.randn((t, m), generator=gen, device=DEV)
    strong = torch.rand((m,), generator=gen, device=DEV) < 0.01
    return (x * torch.where(strong, 8.0, 1.0)).to(dt)


def _codes(gen, shape, g):
    """Codes, scale and zero as a 4-bit min-max quantizer of N(0, 0.015^2) leaves them."""
    k = shape[-1] // g
    codes = (7.5 + 3.0 * torch.randn(shape, generator=gen, device=DEV)).round_().clamp_(0, 15).to(torch.uint8)
    scale = 0.005 * (0.8 + 0.4 * torch.rand((*shape[:-1], k), generator=gen, device=DEV))
    zero = 7.5 + 0.7 * torch.randn((*shape[:-1], k), generator=gen, device=DEV)
    return codes, scale, zero


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    st = {"case": case}
    if case["op"] == "logprobs":
        t, v = case["t"], case["v"]
        full = 3.0 * torch.randn((t, v + case["pad"]), generator=gen, device=DEV)
        st["logits"] = full.to(DT[case["x"]])[:, :v]
        st["ids"] = torch.randint(0, v, (t,), generator=gen, device=DEV)
        return st
    n, m, g = case["n"], case["m"], case["g"]
    if case["op"] == "linear":
        st["X"] = _activations(gen, case["t"], m, DT[case["x"]])
        st["codes"], st["scale"], st["zero"] = _codes(gen, (n, m), g)
    else:
        bounds, rows = _assignment(case)
        st["bounds"] = bounds
        st["offsets"] = torch.tensor(bounds, dtype=torch.int32, device=DEV)
        st["rows"] = torch.tensor(rows, dtype=torch.int32, device=DEV) if case["gather"] else None
        st["X"] = _activations(gen, case["tokens"] if case["gather"] else _rows(case), m, DT[case["x"]])
        st["gates"] = torch.rand((_rows(case),), generator=gen, device=DEV) if case["weighted"] else None
        st["codes"], st["scale"], st["zero"] = _codes(gen, (case["e"], n, m), g)
    if own:
        import post_mixed_precision_amd as slim
        st["packed"] = slim.pack4(st["codes"], st["scale"], st["zero"], g)   # laid out once, as a server does
        del st["codes"], st["scale"], st["zero"]
    return st


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def _plain_weight(codes, scale, zero, g):
    n, m = codes.shape
    return ((codes.float().view(n, m // g, g) - zero[:, :, None]) * scale[:, :, None]).view(n, m)


def _plain_linear(st):
    c = st["case"]
    W = _plain_weight(st["codes"], st["scale"], st["zero"], c["g"])
    return (st["X"].float() @ W.t()).to(DT[c["y"]])


def _plain_experts(st):
    c = st["case"]
    out = torch.empty((_rows(c), c["n"]), dtype=DT[c["y"]], device=DEV)
    for e in range(c["e"]):
        a, b = st["bounds"][e], st["bounds"][e + 1]
        if a == b:
            continue
        x = st["X"][st["rows"][a:b].long()] if c["gather"] else st["X"][a:b]
        y = x.float() @ _plain_weight(st["codes"][e], st["scale"][e], st["zero"][e], c["g"]).t()
        if c["weighted"]:
            y = y * st["gates"][a:b, None]
        out[a:b] = y.to(out.dtype)
    return out


def _plain_logprobs(st):
    c = st["case"]
    x = st["logits"].float()
    mx = x.amax(dim=1, keepdim=True)
    d = x - mx
    ex = d.exp()
    z = ex.sum(dim=1, keepdim=True)
    lse = z.log()
    out = {"logprob": (d.gather(1, st["ids"][:, None]) - lse)[:, 0],
           "entropy": (lse - (ex * d).sum(dim=1, keepdim=True) / z)[:, 0]}
    if c["top"]:
        left = x.clone()
        vals, ids = [], []
        for _ in range(c["top"]):
            i = left.argmax(dim=1, keepdim=True)          # the first of equals
            ids.append(i)
            vals.append(d.gather(1, i) - lse)
            left.scatter_(1, i, float("-inf"))
        out["top_logprob"] = torch.cat(vals, dim=1)
        out["top_id"] = torch.cat(ids, dim=1).to(torch.int32)
    return out


def run(state):
    c = state["case"]
    if not own:
        return {"linear": _plain_linear, "experts": _plain_experts, "logprobs": _plain_logprobs}[c["op"]](state)
    import post_mixed_precision_amd as slim
    if c["op"] == "linear":
        return slim.q4_linear(state["X"], state["packed"], c["n"], c["g"], out_dtype=DT[c["y"]])
    if c["op"] == "experts":
        return slim.q4_experts(state["X"], state["offsets"], state["packed"], c["n"], c["g"], rows=state["rows"],
                               row_scale=state["gates"], out_dtype=DT[c["y"]])
    return slim.token_logprobs(state["logits"], state["ids"], top=c["top"])


# --------------------------------------------------------------------------
# what a pass cannot do without, and the definition in float64
# --------------------------------------------------------------------------
def work(case):
    el = {"bf16": 2, "f32": 4}
    if case["op"] == "logprobs":
        t, v = case["t"], case["v"]
        return {"bytes": t * v * el[case["x"]] + t * 16 + t * case["top"] * 8, "flops": 6 * t * v}
    n, m, g = case["n"], case["m"], case["g"]
    weight = n * m // 2 + 8 * n * (m // g)
    if case["op"] == "linear":
        t = case["t"]
        return {"bytes": weight + t * m * el[case["x"]] + t * n * el[case["y"]], "flops": 2 * t * n * m}
    bounds, _ = _assignment(case)
    busy = sum(1 for a, b in zip(bounds, bounds[1:]) if b > a)
    r = _rows(case)
    xin = (case["tokens"] if case["gather"] else r) * m * el[case["x"]]
    side = 4 * (case["e"] + 1) + (4 * r if case["gather"] else 0) + (4 * r if case["weighted"] else 0)
    return {"bytes": busy * weight + xin + r * n * el[case["y"]] + side, "flops": 2 * r * n * m}


def _exact_product(x, codes, scale, zero, g):
    w = codes.double()
    w -= zero.double().repeat_interleave(g, dim=-1)
    w *= scale.double().repeat_interleave(g, dim=-1)
    return torch.mm(x.double(), w.transpose(0, 1).contiguous())


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = kept
    if case["op"] == "linear":
        return _exact_product(st["X"], st["codes"], st["scale"], st["zero"], case["g"])
    if case["op"] == "experts":
        x = st["X"] if st["rows"] is None else st["X"].index_select(0, st["rows"].long())
        pieces = []
        for e, (a, b) in enumerate(zip(st["bounds"], st["bounds"][1:])):
            if b > a:
                pieces.append(_exact_product(x[a:b], st["codes"][e], st["scale"][e], st["zero"][e], case["g"]))
        y = torch.cat(pieces)
        return y if st["gates"] is None else y * st["gates"].double().unsqueeze(1)
    lps, ents, tops, tids = [], [], [], []
    step = max(1, (1 << 25) // case["v"])
    for a in range(0, case["t"], step):
        x = st["logits"][a:a + step].double()
        p = torch.exp(x)                       # logits of a few units: no shift needed in float64
        total = p.sum(dim=1)
        logp = x - torch.log(total).unsqueeze(1)
        p /= total.unsqueeze(1)
        pick = torch.arange(x.shape[0], device=x.device)
        lps.append(logp[pick, st["ids"][a:a + step]])
        ents.append(-(p * logp).sum(dim=1))
        if case["top"]:
            order = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :case["top"]]
            tops.append(torch.gather(logp, 1, order))
            tids.append(order.to(torch.int32))
    out = {"logprob": torch.cat(lps), "entropy": torch.cat(ents)}
    if case["top"]:
        out["top_logprob"], out["top_id"] = torch.cat(tops), torch.cat(tids)
    return out

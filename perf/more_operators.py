"""What the decode step's operators are measured on.

Three operators of a decode step around the quantized layers: keys and values
appended to a paged 4-bit cache with the position rotation applied on the way
(and read back), attention over that cache, and the verification of drafted
tokens against the target's probabilities.

``own`` false: the plain form, elementary torch operations in float32 (float64
for rotations, and for probabilities whose running sum is compared).
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
    def app(name, t, hq, hkv, d, g, page, rot, inter, x, pad):
        return {"name": name, "op": "append", "t": t, "hq": hq, "hkv": hkv, "d": d, "g": g, "page": page,
                "rot": rot, "inter": inter, "x": x, "pad": pad}

    def att(name, b, ql, length, hq, hkv, d, g, page, x, y, ragged=False, idle=False):
        return {"name": name, "op": "attention", "b": b, "ql": ql, "len": length, "hq": hq, "hkv": hkv, "d": d,
                "g": g, "page": page, "x": x, "y": y, "ragged": ragged, "idle": idle}

    def ver(name, b, k, v, pad, x, draft, temp):
        return {"name": name, "op": "verify", "b": b, "k": k, "v": v, "pad": pad, "x": x, "draft": draft,
                "temp": temp}

    return [
        # one new token of one sequence, heads of a 4096-wide layer: launch and latency
        app("append-token", 1, 32, 32, 128, 128, 64, 128, False, "bf16", False),
        # one calibration-length prompt, 64 query heads over 8
        app("append-prompt", 2048, 64, 8, 128, 64, 64, 128, False, "bf16", False),
        # a ragged step in float32: odd heads, small groups, half the channels rotated in pairs, padded rows
        app("append-odd", 333, 15, 5, 64, 32, 16, 32, True, "f32", True),
        # one token of one sequence over a calibration-length context, every head its own
        att("attention-token", 1, 1, 2048, 32, 32, 128, 128, 64, "bf16", "bf16"),
        # a decode batch, contexts of mixed lengths, heads shared by eight
        att("attention-batch", 16, 1, 8192, 64, 8, 128, 128, 64, "bf16", "bf16"),
        # one token over a long context
        att("attention-long", 1, 1, 131072, 64, 8, 128, 64, 256, "bf16", "bf16"),
        # five drafted tokens in each of eight sequences, heads of a 5120-wide layer
        att("attention-draft", 8, 5, 3001, 40, 40, 128, 128, 32, "bf16", "bf16"),
        # a prompt and the next piece of a longer one, in one call
        att("attention-prompt", 2, 1024, 4096, 32, 8, 128, 128, 64, "bf16", "bf16", True),
        # float32, short heads, small groups, small pages, uneven queries, an idle sequence
        att("attention-odd", 7, 9, 777, 15, 5, 64, 32, 16, "f32", "f32", True, True),
        # one sequence with four drafted tokens
        ver("verify-one", 1, 4, 32000, 0, "f32", True, 1.0),
        # a batch over a large vocabulary, bfloat16 logits
        ver("verify-batch", 32, 5, 131072, 0, "bf16", True, 0.8),
        # drafts without probabilities (looked up), odd vocabulary, rows padded past it
        ver("verify-lookup", 9, 3, 100003, 13, "f32", False, 1.0),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng: random.Random):
    op = rng.choice(["append", "attention", "attention", "attention", "verify"])
    d = rng.choice([64, 128, 128, 256])
    g = rng.choice([x for x in (32, 64, 128) if x <= d])
    page = rng.choice([16, 32, 64, 128, 256])
    hkv = rng.choice([1, 2, 4, 5, 8, 16, 32, 40])
    hq = hkv * rng.choice([1, 1, 2, 3, 4, 5, 8, 16])
    if op == "append":
        while True:
            c = {"op": op, "t": _logint(rng, 1, 4096), "hq": hq, "hkv": hkv, "d": d, "g": g, "page": page,
                 "rot": rng.choice([0, d, d, d // 2]), "inter": rng.random() < 0.3,
                 "x": rng.choice(["bf16", "bf16", "f32"]), "pad": rng.random() < 0.3}
            if c["t"] * (hq + hkv) * d * (2 if c["x"] == "f32" else 1) <= 2048 * 72 * 128:
                return c
            hq = hkv
    if op == "attention":
        while True:
            ql = rng.choice([1, 1, rng.randint(2, 9), _logint(rng, 10, 1024)])
            x = rng.choice(["bf16", "bf16", "f32"])
            c = {"op": op, "b": _logint(rng, 1, 64), "ql": ql, "len": ql + _logint(rng, 1, 131072), "hq": hq,
                 "hkv": hkv, "d": d, "g": g, "page": page, "x": x, "y": rng.choice([x, x, "f32", "bf16"]),
                 "ragged": rng.random() < 0.5, "idle": rng.random() < 0.3}
            w = work(c)
            rows = c["b"] * c["len"] * hkv * d
            if rows <= 131072 * 8 * 128 and w["flops"] * (3 if x == "f32" else 1) <= 2 * 1024 * 4096 * 32 * 128 * 2 \
                    and c["b"] * hq * ql * c["len"] <= 1 << 28:
                return c
    while True:
        c = {"op": op, "b": _logint(rng, 1, 64), "k": rng.randint(1, 8), "v": _logint(rng, 1000, 200000),
             "pad": rng.choice([0, 0, rng.randint(1, 64)]), "x": rng.choice(["bf16", "f32"]),
             "draft": rng.random() < 0.7, "temp": rng.choice([1.0, 1.0, 0.5, 1.3])}
        if c["b"] * (2 * c["k"] + 1) * c["v"] * (2 if c["x"] == "f32" else 1) <= 32 * 11 * 131072:
            return c


def _lengths(case):
    """(query tokens, context length) of each sequence, the new tokens counted in the length: the
    first has the case's full sizes, the others less, fixed by the case's sizes."""
    rng = random.Random(case["b"] * 1000003 + case["ql"] * 101 + case["len"])
    out = []
    for i in range(case["b"]):
        ql = case["ql"] if i == 0 or not case["ragged"] else max(1, int(case["ql"] * rng.random()))
        length = case["len"] if i == 0 else max(ql, int(case["len"] * (0.2 + 0.8 * rng.random())))
        if case["ragged"] and i == 1:
            length = ql                              # a prompt from its first token
        if case["idle"] and i == 2:
            length = 0                               # a padded row of the batch
            if case["ragged"]:
                ql = 0
        out.append((ql, length))
    return out


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _heads(gen, t, h, d, strong=True):
    """Keys or queries: Gaussian with a few strong channels in every head, as keys have them."""
    x = torch.randn((t, h, d), generator=gen, device=DEV)
    if strong:
        x *= torch.where(torch.rand((h, d), generator=gen, device=DEV) < 0.03, 5.0, 1.0)
    return x


def _rotary(positions, rot):
    """cos and sin of every position, [positions, rot], angles in float64."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    a = torch.arange(positions, dtype=torch.float64, device=DEV)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], dim=1).float()


def _prepare_append(case, gen, st):
    t, hq, hkv, d, page = case["t"], case["hq"], case["hkv"], case["d"], case["page"]
    dt = DT[case["x"]]
    # the rows a fused projection leaves: queries, keys and values of a token side by side
    qkv = torch.cat([_heads(gen, t, hq + hkv, d).view(t, -1), _heads(gen, t, hkv, d, False).view(t, -1)], dim=1).to(dt)
    st["q"] = qkv[:, :hq * d].view(t, hq, d)
    st["k"] = qkv[:, hq * d:(hq + hkv) * d].view(t, hkv, d)
    st["v"] = qkv[:, (hq + hkv) * d:].view(t, hkv, d)
    st["pages"] = pages = t // page + 9
    first = int(torch.randint(0, 3000, (1,), generator=gen, device=DEV))
    st["positions"] = torch.arange(first, first + t, dtype=torch.int32, device=DEV)
    order = torch.randperm(pages, generator=gen, device=DEV)
    seat = torch.arange(t, device=DEV) + first % page
    st["slots"] = (order[seat // page] * page + seat % page).to(torch.int32)
    if case["pad"]:
        st["slots"][torch.rand((t,), generator=gen, device=DEV) < 0.1] = -1
    st["rotary"] = _rotary(8192, case["rot"]) if case["rot"] else None
    if own:
        import post_mixed_precision_amd as slim
        st["cache"] = slim.kv4_cache(pages, hkv, d, case["g"], page)
    else:
        st["cache"] = {}
        for name in ("k", "v"):
            st["cache"][name] = [torch.zeros((pages * page, hkv, d), dtype=torch.uint8, device=DEV),
                                 torch.zeros((pages * page, hkv, d // case["g"]), device=DEV),
                                 torch.zeros((pages * page, hkv, d // case["g"]), device=DEV)]


def _prepare_attention(case, gen, st):
    hq, hkv, d, g, page = case["hq"], case["hkv"], case["d"], case["g"], case["page"]
    st["seqs"] = seqs = _lengths(case)
    tq = sum(q for q, _ in seqs)
    st["q"] = _heads(gen, tq, hq, d, False).to(DT[case["x"]])
    bounds = [0]
    for q, _ in seqs:
        bounds.append(bounds[-1] + q)
    st["bounds"] = bounds
    st["lengths"] = torch.tensor([n for _, n in seqs], dtype=torch.int32, device=DEV)
    st["offsets"] = torch.tensor(bounds, dtype=torch.int32, device=DEV) if case["ragged"] else None
    per = -(-case["len"] // page)
    need = [-(-n // page) for _, n in seqs]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    table = torch.zeros((case["b"], per), dtype=torch.int32, device=DEV)
    if own:
        import post_mixed_precision_amd as slim
        st["cache"] = slim.kv4_cache(pages, hkv, d, g, page)
    else:
        st["kv"] = []
    used = 0
    for i, (_, n) in enumerate(seqs):
        table[i, :need[i]] = order[used:used + need[i]]
        used += need[i]
        k = _heads(gen, n, hkv, d).to(DT[case["x"]])
        v = _heads(gen, n, hkv, d, False).to(DT[case["x"]])
        if own:
            at = torch.arange(n, device=DEV)
            slim.kv4_append(k, v, (table[i].long()[at // page] * page + at % page).to(torch.int32), st["cache"], g)
        else:
            st["kv"].append((_quantize(k.float(), g), _quantize(v.float(), g)))
    st["table"] = table
    if not case["ragged"]:
        st["q"] = st["q"].view(case["b"], case["ql"], hq, d)


def _prepare_verify(case, gen, st):
    b, k, v = case["b"], case["k"], case["v"]
    full = 3.0 * torch.randn((b, k + 1, v + case["pad"]), generator=gen, device=DEV)
    guess = full[:, :k] + 0.7 * torch.randn((b, k, v + case["pad"]), generator=gen, device=DEV)
    st["target"] = full.to(DT[case["x"]])[:, :, :v]
    st["draft"] = guess.to(DT[case["x"]])[:, :, :v] if case["draft"] else None
    # drafted as the smaller model samples: the largest of its logits with Gumbel noise
    noise = -torch.log(-torch.log(torch.rand((b, k, v), generator=gen, device=DEV).clamp_(1e-20, 1 - 1e-7)))
    st["tokens"] = (guess[:, :, :v] / case["temp"] + noise).argmax(dim=2)
    if b > 2:
        st["tokens"][2, k - 1:] = -1                 # one sequence drafted less
    st["uniform"] = torch.rand((b, k + 1), generator=gen, device=DEV)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    st = {"case": case}
    {"append": _prepare_append, "attention": _prepare_attention, "verify": _prepare_verify}[case["op"]](case, gen, st)
    return st


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def _rounded(x, up):
    """float32 to the next bfloat16 value up (of positive x) or down, held in float32."""
    u = x.view(torch.int32)
    more = (u + 0xFFFF) & ~0xFFFF
    if up:
        return more.view(torch.float32)
    return torch.where(u < 0, more, u & ~0xFFFF).view(torch.float32)


def _quantize(x, g):
    """float32 [t, h, d] -> codes uint8 [t, h, d], step and low end of every group (bfloat16 values)."""
    t, h, d = x.shape
    xg = x.view(t, h, d // g, g)
    low = _rounded(xg.amin(dim=3).contiguous(), False)
    step = _rounded(((xg.amax(dim=3) - low).double() / 15.0).float(), True)
    step = torch.where(step > 0, step.clamp_min(2.0 ** -126), step)
    inv = torch.where(step > 0, (1.0 / step.double()).float(), torch.zeros_like(step))
    codes = ((xg - low[..., None]) * inv[..., None]).round().clamp(0, 15)
    return codes.to(torch.uint8).view(t, h, d), step, low


def _values(codes, step, low, g):
    t, h, d = codes.shape
    return (codes.float().view(t, h, d // g, g) * step[..., None] + low[..., None]).view(t, h, d)


def _rotate(x, st):
    """The first rot channels of every head turned, in float64; the rest as they are."""
    c = st["case"]
    if not c["rot"]:
        return x.float()
    row = st["rotary"][st["positions"].long()].double()
    cos, sin = row[:, None, :c["rot"] // 2], row[:, None, c["rot"] // 2:]
    y = x.double()
    if c["inter"]:
        a, b = y[..., 0:c["rot"]:2], y[..., 1:c["rot"]:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = y[..., :c["rot"] // 2], y[..., c["rot"] // 2:c["rot"]]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([turned, y[..., c["rot"]:]], dim=-1).float()


def _plain_append(st):
    c = st["case"]
    held = st["slots"] >= 0
    slot = st["slots"].long()
    out = {"q": _rotate(st["q"], st).to(st["q"].dtype)}
    for name, x in (("k", _rotate(st["k"], st)), ("v", st["v"].float())):
        store = st["cache"][name]
        for kept, new in zip(store, _quantize(x.contiguous(), c["g"])):
            kept[slot[held]] = new[held]
        values = _values(*[kept[slot.clamp(min=0)] for kept in store], c["g"])
        out[name] = torch.where(held[:, None, None], values, torch.zeros_like(values))
    return out


def _plain_attention(st):
    c = st["case"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    grp = hq // hkv
    q = st["q"].reshape(-1, hq, d)
    out = torch.zeros((q.shape[0], hq, d), dtype=DT[c["y"]], device=DEV)
    for (ql, n), a, kv in zip(st["seqs"], st["bounds"], st["kv"]):
        if ql == 0 or n == 0:
            continue
        k = _values(*kv[0], c["g"]).permute(1, 2, 0).contiguous()
        v = _values(*kv[1], c["g"]).permute(1, 0, 2).contiguous()
        x = q[a:a + ql].float().view(ql, hkv, grp, d).permute(1, 2, 0, 3).reshape(hkv, grp * ql, d)
        s = torch.bmm(x, k).view(hkv, grp, ql, n) * d ** -0.5
        if ql > 1:
            at = torch.arange(n, device=DEV)
            s.masked_fill_(at[None, :] > torch.arange(n - ql, n, device=DEV)[:, None], float("-inf"))
        s = (s - s.amax(dim=3, keepdim=True)).exp()
        s = s / s.sum(dim=3, keepdim=True)
        o = torch.bmm(s.view(hkv, grp * ql, n), v).view(hkv, grp, ql, d)
        out[a:a + ql] = o.permute(2, 0, 1, 3).reshape(ql, hq, d).to(out.dtype)
    return out if c["ragged"] else out.view(st["q"].shape)


def _probabilities(logits, temp):
    x = logits.double() / temp
    e = (x - x.amax(dim=-1, keepdim=True)).exp()
    return e / e.sum(dim=-1, keepdim=True)


def _plain_verify(st):
    c = st["case"]
    k, tokens = c["k"], st["tokens"]
    p = _probabilities(st["target"], c["temp"])
    at = tokens.clamp(min=0)[..., None]
    if c["draft"]:
        q = _probabilities(st["draft"], c["temp"])
    else:
        q = torch.zeros_like(p[:, :k]).scatter_(2, at, 1.0)
    u = st["uniform"].double()
    good = (u[:, :k] * q.gather(2, at)[..., 0] < p[:, :k].gather(2, at)[..., 0]) & (tokens >= 0)
    accepted = good.long().cumprod(dim=1).sum(dim=1)
    rows = torch.arange(c["b"], device=DEV)
    ended = torch.cat([tokens, torch.full_like(tokens[:, :1], -1)], dim=1)[rows, accepted] < 0
    mass = p[rows, accepted]
    left = (mass - q[rows, accepted.clamp(max=k - 1)]).clamp(min=0)
    mass = torch.where(ended[:, None], mass, left)
    run_sum = mass.cumsum(dim=1)
    pick = (run_sum <= u[:, k:] * run_sum[:, -1:]).sum(dim=1)
    places = torch.arange(k + 1, device=DEV)[None, :]
    ids = torch.cat([tokens, torch.full_like(tokens[:, :1], -1)], dim=1)
    ids = torch.where(places < accepted[:, None], ids, torch.full_like(ids, -1))
    ids[rows, accepted] = pick
    return {"accepted": accepted.to(torch.int32), "ids": ids}


def run(state):
    c = state["case"]
    if not own:
        return {"append": _plain_append, "attention": _plain_attention, "verify": _plain_verify}[c["op"]](state)
    import post_mixed_precision_amd as slim
    if c["op"] == "append":
        q = slim.kv4_append(state["k"], state["v"], state["slots"], state["cache"], c["g"], rotary=state["rotary"],
                            positions=state["positions"] if c["rot"] else None, interleaved=c["inter"], q=state["q"])
        k, v = slim.kv4_read(state["slots"], state["cache"], c["d"], c["g"])
        return {"q": q, "k": k, "v": v}
    if c["op"] == "attention":
        return slim.kv4_attention(state["q"], state["cache"], state["table"], state["lengths"], c["g"],
                                  offsets=state["offsets"], out_dtype=DT[c["y"]])
    return slim.verify_draft(state["target"], state["tokens"], state["uniform"], draft=state["draft"],
                             temperature=c["temp"])


# --------------------------------------------------------------------------
# what a pass cannot do without, and the definition in float64
# --------------------------------------------------------------------------
def work(case):
    el = {"bf16": 2, "f32": 4}
    if case["op"] == "verify":
        n = case["b"] * ((2 * case["k"] + 1) if case["draft"] else case["k"] + 1) * case["v"]
        return {"bytes": n * el[case["x"]] + case["b"] * (8 * case["k"] + 4 * (case["k"] + 1) + 8 * (case["k"] + 1) + 4),
                "flops": 4 * n}
    hkv, d = case["hkv"], case["d"]
    held = d // 2 + 4 * d // case["g"]                  # bytes of a token's key (or value) in a head
    if case["op"] == "append":
        t, hq = case["t"], case["hq"]
        moved = t * (hq + 2 * hkv) * d * el[case["x"]] + t * hq * d * el[case["x"]] + 2 * t * hkv * d * 4
        return {"bytes": moved + 4 * t * hkv * held + t * (case["rot"] * 4 + 8), "flops": t * (6 * hq + 12 * hkv) * d}
    nbytes = flops = 0
    for ql, n in _lengths(case):
        nbytes += 2 * n * hkv * held + ql * case["hq"] * d * (el[case["x"]] + el[case["y"]]) + 4 * -(-n // case["page"])
        pairs = ql * n - ql * (ql - 1) // 2 if n else 0
        flops += 4 * pairs * case["hq"] * d
    return {"bytes": nbytes, "flops": flops}


def _held(x, g):
    """The float32 values that float64 x is held as: the low end of a group is its least value at 8
    significant bits (downwards), the step 1/15 of the range at 8 bits (upwards), and differences,
    quotients and reciprocals are float32."""
    def at8(y, how):
        m, e = torch.frexp(y)
        return torch.ldexp(how(m * 256.0), e - 8)
    t, h, d = x.shape
    xg = x.reshape(t, h, d // g, g)
    low = at8(xg.min(dim=3, keepdim=True).values, torch.floor)
    spread = (xg.max(dim=3, keepdim=True).values - low).float().double()
    step = at8((spread / 15.0).float().double(), torch.ceil)
    n = (xg - low).float().double() * torch.where(step > 0, 1.0 / step, step).float().double()
    n = torch.floor(n.float().double() + 0.5) - ((n.float().double() - torch.floor(n.float().double()) == 0.5)
                                                  & (torch.floor(n.float().double()) % 2 == 0)).double()
    return (torch.clamp(n, 0.0, 15.0) * step + low).float().double().view(t, h, d)


def _exact_append(st, case):
    t, rot = case["t"], case["rot"]
    out = {}
    for name in ("q", "k"):
        x = st[name].double().clone()
        if rot:
            # a pair as a complex number, turned by the position's unit
            row = st["rotary"].double()[st["positions"].long()]
            turn = torch.complex(row[:, :rot // 2], row[:, rot // 2:]).unsqueeze(1)
            first = slice(0, rot, 2) if case["inter"] else slice(0, rot // 2)
            second = slice(1, rot, 2) if case["inter"] else slice(rot // 2, rot)
            z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * turn
            x[..., first], x[..., second] = z.real, z.imag
        out[name] = x
    gone = (st["slots"] < 0).view(t, 1, 1)
    out["k"] = _held(out["k"].float().double(), case["g"]).masked_fill(gone, 0.0)
    out["v"] = _held(st["v"].double(), case["g"]).masked_fill(gone, 0.0)
    return out


def _exact_attention(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    st = {"case": case}
    _prepare_attention(case, gen, st)
    hq, hkv, d, g = case["hq"], case["hkv"], case["d"], case["g"]
    q = st["q"].reshape(-1, hq, d).double()
    out = torch.zeros_like(q)
    for (ql, n), a, (kk, vv) in zip(st["seqs"], st["bounds"], st["kv"]):
        if ql == 0 or n == 0:
            continue
        behind = torch.ones((ql, n), dtype=torch.bool, device=DEV).tril(n - ql)
        for h in range(hkv):
            part = []
            for codes, step, low in (kk, vv):
                s = step[:, h].double().repeat_interleave(g, dim=1)
                part.append(torch.addcmul(low[:, h].double().repeat_interleave(g, dim=1), codes[:, h].double(), s))
            for j in range(h * (hq // hkv), (h + 1) * (hq // hkv)):
                w = torch.mm(q[a:a + ql, j], part[0].t().contiguous()) / math.sqrt(d)
                w = torch.softmax(w.masked_fill(~behind, -math.inf), dim=1)
                out[a:a + ql, j] = torch.mm(w, part[1])
    return out if case["ragged"] else out.view(st["q"].shape)


def _exact_verify(st, case):
    b, k, v = case["b"], case["k"], case["v"]
    ids = torch.full((b, k + 1), -1, dtype=torch.int64)
    accepted = torch.zeros((b,), dtype=torch.int32)
    tokens, u = st["tokens"].cpu(), st["uniform"].double().cpu()
    for i in range(b):
        j, mass = 0, None
        while True:
            logp = torch.log_softmax(st["target"][i, j].double() / case["temp"], dim=0)
            x = int(tokens[i, j]) if j < k else -1
            if x < 0:
                mass = logp.exp()
                break
            if case["draft"]:
                logq = torch.log_softmax(st["draft"][i, j].double() / case["temp"], dim=0)
            else:
                logq = torch.full((v,), -math.inf, dtype=torch.float64, device=DEV)
                logq[x] = 0.0
            if float(u[i, j]) < math.exp(float(logp[x] - logq[x])):
                ids[i, j] = x
                j += 1
                continue
            mass = torch.relu(logp.exp() - logq.exp())
            break
        total = torch.cumsum(mass, dim=0)
        ids[i, j] = int(torch.searchsorted(total, (u[i, k].to(DEV) * total[-1]).view(1), right=True))
        accepted[i] = j
    return {"accepted": accepted.to(DEV), "ids": ids.to(DEV)}


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        if case["op"] == "attention":
            return _exact_attention(case, seed)
        st = prepare(case, seed)
        return _exact_append(st, case) if case["op"] == "append" else _exact_verify(st, case)
    finally:
        own = kept

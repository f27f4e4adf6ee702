"""The decode step's operators - the 4-bit key/value cache, attention over it and the verification of
drafted tokens - against the oracle, through the binding.

The cache is compared word for word.  Attention's tolerance, from the arithmetic (see _attention): a
score's error is at most 2^-23 (dim + 16) of scale sum |q| (|code step| + |low|), plus what rounding
its power's argument adds, and it enters the weights as a factor; sums over the tokens add 2^-23 a term of
a lane's chain; a bfloat16 output adds 2^-8 of the value.  Weights times steps are rounded to three
bfloat16 terms (float32 q or output, nothing is lost) or two (bfloat16, few rows: 2^-8 of what the first
leaves, below 2^-15 as it is truncated).  Many rows of bfloat16 (outputs too) have both factors in float16, whose
rounding is at most 2^-11: a value is code step + low, each of step, low and value rounded once, and a
group is no smaller than 2^-9 of a unit in which float16's least halves are 2^-25, so 15 codes and two
roundings more of those are below 2^-12 of the group; a weight moves by 2^-11 of itself or by 2^-25
beside a greatest one of at least 2^8, and the sum it is divided by moves with it.
"""
import numpy as np
import pytest

import oracle

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def slim():
    import post_mixed_precision_amd as s
    s.load_library()
    return s


def _gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda:0")


def _i32(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda:0")


def _host(t):
    """What the oracle takes: float32, or bfloat16 bits."""
    t = t.detach().cpu()
    return t.contiguous().view(torch.int16).numpy().view(np.uint16) if t.dtype == torch.bfloat16 else t.numpy()


def _rows(rng, t, h, d, dt, channels=True):
    x = rng.standard_normal((t, h, d)).astype(np.float32)
    if channels:
        x *= np.where(rng.random((h, d)) < 0.05, 6.0, 1.0).astype(np.float32)
    return torch.from_numpy(x).to(DT[dt])


def _table(rng, npos, rot):
    a = rng.uniform(0, 2 * np.pi, (npos, rot // 2))
    return np.concatenate([np.cos(a), np.sin(a)], axis=1).astype(np.float32)


def _oracle_put(cache, slots, page, dim, group, k, v):
    """k, v float32 [t, heads, dim], as rotated."""
    qk, qv = oracle.kv4_quantize(k, group), oracle.kv4_quantize(v, group)
    for i, s in enumerate(slots):
        if 0 <= s < cache.shape[0] * page:
            oracle.kv4_put(cache, s, page, dim, group, [x[i] for x in qk], [x[i] for x in qv])
    return oracle.kv4_values(*qk, group), oracle.kv4_values(*qv, group)


def _slots(rng, t, pages, page):
    s = rng.permutation(pages * page)[:t].astype(np.int32)
    if t > 4:
        s[2], s[t - 1] = -1, pages * page + 5        # skipped
    return s


# t, query heads, heads, dim, group, page, rotated channels, interleaved, dtype
APPEND = [
    (1, 0, 1, 64, 32, 16, 0, False, "bf16"),
    (1, 8, 2, 128, 128, 64, 128, False, "bf16"),
    (5, 4, 4, 128, 64, 16, 128, True, "f32"),
    (37, 6, 3, 64, 64, 32, 32, False, "bf16"),
    (64, 2, 1, 256, 32, 256, 256, False, "bf16"),
    (33, 5, 5, 256, 128, 128, 20, False, "f32"),     # halves of 10 channels: partners are not aligned
    (21, 3, 1, 128, 32, 16, 6, True, "bf16"),
    (19, 1, 1, 64, 32, 16, 2, False, "f32"),
    (130, 15, 5, 64, 32, 16, 64, False, "f32"),
    (50, 2, 2, 256, 64, 64, 130, True, "bf16"),
]


@pytest.mark.parametrize("t,hq,heads,dim,group,page,rot,inter,dt", APPEND)
def test_append_words(slim, t, hq, heads, dim, group, page, rot, inter, dt):
    print(f"append t={t} hq={hq} heads={heads} dim={dim} g={group} page={page} rot={rot} {inter} {dt}", flush=True)
    rng = np.random.default_rng(t * 1000 + dim)
    pages = -(-t // page) + 2
    k, v = _rows(rng, t, heads, dim, dt), _rows(rng, t, heads, dim, dt, False)
    q = _rows(rng, t, hq, dim, dt, False) if hq else None
    slots = _slots(rng, t, pages, page)
    table = _table(rng, 40, rot) if rot else None
    pos = rng.integers(0, 40, t).astype(np.int32) if rot else None
    if rot and t > 8:
        pos[1], pos[5] = -1, 40                      # outside the table
    kr = oracle.rotate(_host(k), table, pos, inter)
    before = rng.integers(0, 1 << 32, (pages, heads, oracle.kv4_words(page, dim, group)), dtype=np.uint32)
    want = before.copy()
    wk, wv = _oracle_put(want, slots, page, dim, group, kr, oracle.as_f32(_host(v)))
    cache = _gpu(before.view(np.int32))
    assert slim.kv4_cache(pages, heads, dim, group, page).shape == cache.shape
    out = slim.kv4_append(k.cuda(), v.cuda(), _gpu(slots), cache, group, rotary=None if table is None else _gpu(table),
                          positions=None if pos is None else _gpu(pos), interleaved=inter,
                          q=None if q is None else q.cuda())
    np.testing.assert_array_equal(cache.cpu().numpy().view(np.uint32), want)
    if hq:
        qr = oracle.rotate(_host(q), table, pos, inter)
        got = out.float().cpu().numpy()
        ref = oracle.bf16_round(qr) if dt == "bf16" else qr
        np.testing.assert_array_equal(got, ref)
    else:
        assert out is None
    # and back: what the slots stand for
    rk, rv = slim.kv4_read(_gpu(slots), cache, dim, group)
    kept = (slots >= 0) & (slots < pages * page)
    for got, ref in ((rk.cpu().numpy(), wk), (rv.cpu().numpy(), wv)):
        np.testing.assert_array_equal(got[kept], ref[kept])
        assert np.all(got[slots < 0] == 0) and np.isnan(got[slots >= pages * page]).all()
    rk, rv = slim.kv4_read(_gpu(slots), cache, dim, group, out_dtype=torch.bfloat16)
    np.testing.assert_array_equal(rk.float().cpu().numpy()[kept], oracle.bf16_round(wk)[kept])
    np.testing.assert_array_equal(rv.float().cpu().numpy()[kept], oracle.bf16_round(wv)[kept])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("lead", [0, 1, 8])
def test_append_strided_rows(slim, dt, lead):
    """Views of a fused projection, aligned and not, a key head expanded, heads before tokens."""
    rng = np.random.default_rng(lead)
    t, hq, heads, dim, group, page = 9, 4, 2, 64, 32, 16
    width = lead + (hq + 2 * heads) * dim + 3 * (lead % 2)
    qkv = torch.from_numpy(rng.standard_normal((t, width)).astype(np.float32)).to(DT[dt]).cuda()
    q = qkv[:, lead:lead + hq * dim].view(t, hq, dim)
    k = qkv[:, lead + hq * dim:lead + (hq + heads) * dim].view(t, heads, dim)
    v = qkv[:, lead + (hq + heads) * dim:lead + (hq + 2 * heads) * dim].view(t, heads, dim)
    slots, pos, table = _i32(range(3, 12)), _i32(range(9)), _gpu(_table(rng, 9, 64))

    def run(q, k, v):
        cache = slim.kv4_cache(1, heads, dim, group, page)
        return slim.kv4_append(k, v, slots, cache, group, rotary=table, positions=pos, q=q), cache
    a, ca = run(q, k, v)
    b, cb = run(q.contiguous(), k.contiguous(), v.contiguous())
    assert torch.equal(a, b) and torch.equal(ca, cb)
    hk = k.permute(1, 0, 2).contiguous().permute(1, 0, 2)
    a, ca = run(q, hk, v[:, :1].expand(t, heads, dim))
    b, cb = run(q, k, v[:, :1].repeat(1, heads, 1))
    assert torch.equal(a, b) and torch.equal(ca, cb)


def test_append_extremes(slim):
    x = np.zeros((12, 1, 64), np.float32)
    x[0, 0, 3], x[1, 0, 40], x[2, 0, 0], x[3, 0, 0] = np.nan, np.inf, 3.3e38, 1e-42
    x[2, 0, 1], x[4, 0, 7], x[5] = -3.3e38, -np.inf, 0.1
    x[6, 0] = np.float32(2.0 ** -130) * np.arange(64)
    x[7, 0] = -0.0
    x[8, 0, ::2] = np.float32(-1e-38)
    x[9, 0] = 1000 + np.linspace(0, 1e-3, 64)
    x[10, 0, :] = np.array([0xffffffff, 0x7fffffff], np.uint32).view(np.float32)[np.arange(64) % 2]
    x[11, 0] = np.linspace(-1e38, 3e38, 64)
    want = np.zeros((1, 1, oracle.kv4_words(16, 64, 32)), np.uint32)
    wk, _ = _oracle_put(want, range(12), 16, 64, 32, x, x)
    cache = slim.kv4_cache(1, 1, 64, 32, 16)
    g = _gpu(x)
    slim.kv4_append(g, g, _i32(range(12)), cache, 32)
    k, v = slim.kv4_read(_i32(range(12)), cache, 64, 32)
    np.testing.assert_array_equal(k.cpu().numpy(), wk)
    np.testing.assert_array_equal(v.cpu().numpy(), wk)


def test_nothing_to_append_or_read(slim):
    cache = slim.kv4_cache(1, 2, 64, 32, 16)
    k = torch.zeros((0, 2, 64), device="cuda:0")
    q = slim.kv4_append(k, k, _i32([]), cache, 32, q=torch.zeros((0, 4, 64), device="cuda:0"))
    assert q.shape == (0, 4, 64) and not cache.any()
    k, v = slim.kv4_read(_i32([]), cache, 64, 32)
    assert k.shape == (0, 2, 64) and v.shape == (0, 2, 64)


# ---------------------------------------------------------------- attention
class Context:
    """A cache with sequences of given lengths on shuffled pages, and their values."""

    def __init__(self, slim, seed, lengths, heads, dim, group, page, dt="bf16", spare=2, values=None, keys=None):
        rng = np.random.default_rng(seed)
        need = [max(0, -(-n // page)) for n in lengths]
        per = max(1, max(need))
        pages = sum(need) + spare
        order = rng.permutation(pages).astype(np.int32)
        self.table = np.full((len(lengths), per), -1, np.int32)      # what no length reaches is not read
        self.k, self.v, used = [], [], 0
        self.cache = slim.kv4_cache(pages, heads, dim, group, page)
        self.cache.fill_(0x7fc07fc0)                                 # pairs never written are NaN
        for i, n in enumerate(lengths):
            self.table[i, :need[i]] = order[used:used + need[i]]
            used += need[i]
            k, v = _rows(rng, max(n, 0), heads, dim, dt), _rows(rng, max(n, 0), heads, dim, dt, False)
            if keys is not None:
                k = torch.from_numpy(keys(rng, k.float().numpy())).to(DT[dt])
            if values is not None:
                v = torch.from_numpy(values(rng, v.float().numpy())).to(DT[dt])
            at = np.arange(max(n, 0))
            slots = (self.table[i, at // page] * page + at % page).astype(np.int32)
            slim.kv4_append(k.cuda(), v.cuda(), _gpu(slots), self.cache, group)
            kq, vq = (oracle.kv4_quantize(oracle.as_f32(_host(x)), group) for x in (k, v))
            self.k.append((kq, oracle.kv4_values(*kq, group)))
            self.v.append((vq, oracle.kv4_values(*vq, group)))
        self.lengths, self.group, self.page, self.pages = list(lengths), group, page, pages


def _attention(ctx, i, q, scale, causal, odt, qdt, many=True):
    """float64 result of sequence i and its tolerance; many: bfloat16 rows may be taken by float16."""
    short = qdt == "bf16" and odt == "bf16"
    q = oracle.as_f64(_host(q)) if isinstance(q, torch.Tensor) else q
    k, v = ctx.k[i][1].astype(np.float64), ctx.v[i][1].astype(np.float64)
    want = oracle.attention(q, k, v, scale, causal)
    n, hq, dim = q.shape
    tol = np.zeros(q.shape)
    g = ctx.group

    def size(x):                                     # |code step| and |low| of every entry
        (codes, step, low), _ = x
        return codes * np.repeat(step, g, -1).astype(np.float64), np.abs(np.repeat(low, g, -1)).astype(np.float64)
    kc, kl = size(ctx.k[i])
    vc, vl = size(ctx.v[i])
    grp = hq // k.shape[1]
    for a in range(n):
        reach = len(k) - n + a + 1 if causal else len(k)
        if reach <= 0:
            continue
        for h in range(hq):
            hh = h // grp
            s = scale * (k[:reach, hh] @ q[a, h])
            p = np.exp(s - s.max())
            p /= p.sum()
            ds = 2.0 ** -23 * ((dim + 16) * abs(scale) * ((kc + kl)[:reach, hh] @ np.abs(q[a, h])) + 4 * np.abs(s).max() + 8)
            part, whole = p @ vc[:reach, hh], p @ (vc + vl)[:reach, hh]
            chain = 2.0 ** -23 * (reach / 16 + 64)
            tol[a, h] = (2.0 ** -15 if short else 0) * part + (2 * ds.max() + chain) * whole
            if short and many:
                x = np.abs(v[:reach, hh])
                top = np.repeat(x.reshape(reach, -1, g).max(-1), g, -1)
                lost = 2.0 ** -11 * (vc + vl)[:reach, hh] + 2.0 ** -11 * x + 2.0 ** -12 * top
                tol[a, h] += p @ lost + (2.0 ** -11 * p + 2.0 ** -33) @ (x + np.abs(want[a, h]))
    return want, tol + (2.0 ** -8 * np.abs(want) if odt == "bf16" else 0) + 2.0 ** -120


def _check(ctx, i, got, q, scale, causal, odt, qdt, what="", many=True):
    want, tol = _attention(ctx, i, q, scale, causal, odt, qdt, many)
    got = got.double().cpu().numpy()
    worst = np.max(np.abs(got - want) / tol) if got.size else 0.0
    assert worst <= 1, f"{what} sequence {i}: {worst} of the tolerance"


# lengths, query tokens, query heads, heads, dim, group, page, q dtype, out dtype, causal
ATTENTION = [
    ([1], 1, 1, 1, 64, 32, 16, "bf16", "bf16", True),
    ([2, 1, 17], 1, 4, 2, 128, 128, 64, "bf16", "f32", True),
    ([33], 1, 8, 1, 128, 64, 16, "bf16", "bf16", True),
    ([500, 31, 32, 0, 1000], 1, 16, 2, 128, 128, 32, "bf16", "bf16", True),
    ([257, 100], 5, 10, 2, 128, 32, 64, "bf16", "bf16", True),
    ([70, 700], 9, 6, 2, 64, 64, 256, "bf16", "f32", True),
    ([64, 3000], 1, 32, 1, 256, 128, 64, "bf16", "bf16", True),
    ([300], 40, 3, 1, 256, 32, 16, "bf16", "bf16", True),
    ([130, 129], 50, 4, 4, 128, 128, 128, "bf16", "bf16", True),
    ([450], 200, 4, 1, 64, 32, 16, "bf16", "f32", True),
    ([333], 70, 2, 2, 128, 64, 32, "bf16", "bf16", False),
    ([3, 40], 6, 2, 1, 64, 32, 16, "bf16", "bf16", True),       # more query tokens than tokens
    ([1, 90], 1, 2, 1, 64, 64, 16, "f32", "f32", True),
    ([777, 5], 3, 15, 5, 64, 32, 16, "f32", "f32", True),
    ([200], 30, 4, 2, 128, 128, 64, "f32", "f32", True),
    ([1025], 7, 12, 3, 128, 32, 16, "f32", "bf16", False),
    ([150, 0, 40], 2, 3, 3, 256, 64, 32, "f32", "f32", True),
    ([90], 33, 5, 1, 64, 64, 64, "f32", "f32", True),
    ([5000], 1, 24, 8, 128, 128, 256, "f32", "f32", True),
    ([20000], 2, 2, 1, 128, 64, 64, "bf16", "f32", True),
]


@pytest.mark.parametrize("lengths,n,hq,heads,dim,group,page,qdt,odt,causal", ATTENTION)
def test_attention(slim, lengths, n, hq, heads, dim, group, page, qdt, odt, causal):
    print(f"attention {lengths} n={n} hq={hq} heads={heads} dim={dim} g={group} page={page} {qdt} {odt} {causal}",
          flush=True)
    ctx = Context(slim, sum(lengths) + dim, lengths, heads, dim, group, page, qdt)
    rng = np.random.default_rng(n)
    q = _rows(rng, len(lengths) * n, hq, dim, qdt, False).view(len(lengths), n, hq, dim)
    out = slim.kv4_attention(q.cuda(), ctx.cache, _gpu(ctx.table), _i32(lengths), group, causal=causal,
                             out_dtype=DT[odt])
    assert out.shape == q.shape and out.dtype == DT[odt]
    for i, length in enumerate(lengths):
        if length == 0:
            assert not out[i].any()
        else:
            _check(ctx, i, out[i], q[i], dim ** -0.5, causal, odt, qdt, many=n * hq // heads > 32)
    again = slim.kv4_attention(q.cuda(), ctx.cache, _gpu(ctx.table), _i32(lengths), group, causal=causal,
                               out_dtype=DT[odt])
    assert torch.equal(out, again)


# every head size and group on every kernel: few rows, some, many
EVERY = [([97, 40 + n], n, 3, 1, dim, group, 32, qdt, odt, True)
         for dim in (64, 128, 256) for group in (32, 64, 128) if group <= dim
         for qdt, odt in (("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32")) for n in (2, 9, 25)]
# tiles for fewer rows where a head has four groups or more
EVERY += [([700, 90 + n], n, 3, 1, dim, dim // 4, 32, qdt, odt, True) for dim in (128, 256)
          for qdt, odt in (("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32")) for n in (11, 21)]
# and enough runs for the join by four waves
JOINED = [([3000 + n, 1700], n, 3, 1, 128, 64, 64, "bf16", "bf16", True) for n in (1, 9, 25)] + \
         [([2500 + n], n, 3, 1, dim, 64, 64, "f32", "f32", True) for dim in (64, 256) for n in (1, 25)]


@pytest.mark.parametrize("lengths,n,hq,heads,dim,group,page,qdt,odt,causal", EVERY + JOINED)
def test_attention_every_kernel(slim, lengths, n, hq, heads, dim, group, page, qdt, odt, causal):
    test_attention(slim, lengths, n, hq, heads, dim, group, page, qdt, odt, causal)


@pytest.mark.parametrize("qdt", ["bf16", "f32"])
@pytest.mark.parametrize("counts,lengths,heads,hq,dim,group,page", [
    ([3, 0, 1, 20], [40, 9, 1, 300], 2, 6, 64, 32, 16),
    ([1, 1, 1, 1, 1], [5, 700, 0, 33, 64], 1, 8, 128, 128, 64),
    ([100, 1, 37], [100, 2000, 90], 2, 2, 128, 64, 32),
    ([0, 0, 7], [0, 50, 7], 3, 3, 256, 128, 16),
])
def test_attention_uneven(slim, qdt, counts, lengths, heads, hq, dim, group, page):
    """Query tokens by offsets; rows before the first and behind the last sequence stay as they were."""
    ctx = Context(slim, 7, lengths, heads, dim, group, page, qdt)
    rng = np.random.default_rng(8)
    off = np.concatenate([[2], 2 + np.cumsum(counts)]).astype(np.int32)
    tq = int(off[-1]) + 3
    q = _rows(rng, tq, hq, dim, qdt, False)
    out = torch.full((tq, hq, dim), 7.0, dtype=DT[qdt], device="cuda:0")
    got = slim.kv4_attention(q.cuda(), ctx.cache, _gpu(ctx.table), _i32(lengths), group, offsets=_gpu(off), scale=0.2,
                             out=out)
    assert got is out
    assert torch.all(out[:2] == 7) and torch.all(out[-3:] == 7)
    for i, length in enumerate(lengths):
        a, b = int(off[i]), int(off[i + 1])
        if length == 0:
            assert not out[a:b].any()
        elif b > a:
            _check(ctx, i, out[a:b], q[a:b], 0.2, True, qdt, qdt)


def test_attention_many_sequences(slim):
    """More sequences than a wave has lanes, uneven, bounds scanned several a lane."""
    rng = np.random.default_rng(3)
    b = 150
    counts = rng.integers(0, 4, b)
    lengths = [int(c + rng.integers(0, 60)) if i % 7 else 0 for i, c in enumerate(counts)]
    counts = [c if n else 0 for c, n in zip(counts, lengths)]
    ctx = Context(slim, 9, lengths, 1, 64, 32, 16)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    q = _rows(rng, int(off[-1]), 3, 64, "bf16", False)
    out = slim.kv4_attention(q.cuda(), ctx.cache, _gpu(ctx.table), _i32(lengths), 32, offsets=_gpu(off))
    for i in range(b):
        if counts[i]:
            _check(ctx, i, out[off[i]:off[i + 1]], q[off[i]:off[i + 1]], 64 ** -0.5, True, "bf16", "bf16")


def _by_tiles(ctx, tq, grp, dim):
    """Whether a call's rows are taken as many rows are: by the average of all sequences, as the header states it."""
    cap = ctx.table.shape[1] * ctx.page
    return -(-tq // len(ctx.lengths)) * grp > (32 if dim // ctx.group >= 4 and cap > 512 else 64)


def _batch(slim, ctx, counts, hq, dim, qdt, seed):
    """A batch by offsets, every sequence judged by the rounding of its call and no more."""
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    tq, heads = int(off[-1]), ctx.cache.shape[1]
    many = _by_tiles(ctx, tq, hq // heads, dim)
    q = _rows(np.random.default_rng(seed), tq, hq, dim, qdt, False)
    out = slim.kv4_attention(q.cuda(), ctx.cache, _gpu(ctx.table), _i32(ctx.lengths), ctx.group, offsets=_gpu(off))
    for i, length in enumerate(ctx.lengths):
        a, b = int(off[i]), int(off[i + 1])
        if length == 0:
            assert not out[a:b].any()
        elif b > a:
            _check(ctx, i, out[a:b], q[a:b], dim ** -0.5, True, qdt, qdt, f"many rows {many}", many=many)
    return many


@pytest.mark.parametrize("qdt", ["bf16", "f32"])
@pytest.mark.parametrize("b,grp,prompt,group,many", [
    (64, 1, 300, 64, False),                 # the prompt's rows in the kernel of few rows
    (64, 1, 300, 32, False),
    (32, 4, 600, 64, True),                  # single tokens in the kernel of many rows
    (16, 8, 200, 128, True),
    (40, 8, 100, 32, False),
])
def test_attention_a_prompt_among_single_tokens(slim, qdt, b, grp, prompt, group, many):
    """One call for a prompt and many sequences of a token each, of all lengths: whichever kernel the average chooses."""
    rng = np.random.default_rng(b + grp)
    at = b // 3
    lengths = [int(x) for x in rng.integers(1, 900, b)]
    lengths[at], lengths[5] = prompt + 150, 1
    counts = [1] * b
    counts[at] = prompt
    ctx = Context(slim, 16, lengths, 1, 128, group, 32, qdt)
    assert _batch(slim, ctx, counts, grp, 128, qdt, 1) == many


@pytest.mark.parametrize("b,most,long", [(150, 3, 60), (1100, 2, 3000), (1100, 1, 5000), (4096, 1, 4)])
def test_attention_few_rows_of_many_sequences(slim, b, most, long):
    """Few rows a sequence in batches of fewer and more than 1024 sequences (those are not cut), one of them far longer
    than the others."""
    rng = np.random.default_rng(b + most)
    counts = [int(x) for x in rng.integers(0, most + 1, b)]
    lengths = [c + int(x) if c else 0 for c, x in zip(counts, rng.integers(0, 4, b))]
    counts[b // 2], lengths[b // 2] = most, long
    ctx = Context(slim, 17, lengths, 1, 64, 32, 16)
    assert not _batch(slim, ctx, counts, 2, 64, "bf16", 2)


@pytest.mark.parametrize("qdt", ["bf16", "f32"])
@pytest.mark.parametrize("counts,lengths,heads,hq,dim,group,page", [
    ([3, 0, 1, 20], [40, 9, 1, 300], 2, 6, 64, 32, 16),
    ([1, 1, 1, 1, 1], [5, 700, 0, 33, 64], 1, 8, 128, 128, 64),
    ([0, 0, 7], [0, 50, 7], 3, 3, 256, 128, 16),
])
def test_attention_uneven_few_rows(slim, qdt, counts, lengths, heads, hq, dim, group, page):
    """Uneven batches of few rows, without the allowance that many rows have."""
    ctx = Context(slim, 7, lengths, heads, dim, group, page, qdt)
    assert not _batch(slim, ctx, counts, hq, dim, qdt, 8)


@pytest.mark.parametrize("offsets", [[0, 5, 3, 12], [0, -1, 4, 12], [0, 4, 8, 13]])
@pytest.mark.parametrize("lengths", [[30, 30, 30], [3000, 30, 30]])
def test_attention_bad_offsets(slim, offsets, lengths):
    ctx = Context(slim, 1, lengths, 2, 64, 32, 16)
    q = _rows(np.random.default_rng(0), 12, 4, 64, "bf16", False).cuda()
    out = slim.kv4_attention(q, ctx.cache, _gpu(ctx.table), _i32(lengths), 32, offsets=_i32(offsets))
    assert torch.isnan(out).all()


@pytest.mark.parametrize("qdt", ["bf16", "f32"])
@pytest.mark.parametrize("length", [200, 4010])
def test_attention_bad_pages_and_lengths(slim, qdt, length):
    """A page outside the cache: NaN for the rows that reach it and no others; a length past the table: NaN."""
    page, n = 32, 60
    ctx = Context(slim, 2, [length, 50, 64], 1, 128, 64, page, qdt)
    q = _rows(np.random.default_rng(0), 3 * n, 2, 128, qdt, False).view(3, n, 2, 128)
    table = ctx.table.copy()
    at = length - 40
    table[0, at // page] = ctx.pages
    table[2, 1] = -5
    first = at // page * page                        # the first token of the lost page
    cap = table.shape[1] * page
    out = slim.kv4_attention(q.cuda(), ctx.cache, _gpu(table), _i32([length, cap + 1, 64]), 64)
    reach = np.arange(length - n + 1, length + 1)    # tokens each row attends to
    lost = reach > first
    assert torch.isnan(out[0][torch.from_numpy(lost)]).all()
    assert lost.any() and not lost.all()
    want, tol = _attention(ctx, 0, q[0], 128 ** -0.5, True, qdt, qdt)
    err = np.abs(out[0].double().cpu().numpy() - want)[~lost]
    assert np.all(err <= tol[~lost])
    assert torch.isnan(out[1]).all()
    reach = np.arange(64 - n + 1, 65)
    assert torch.isnan(out[2][torch.from_numpy(reach > 32)]).all()
    assert not torch.isnan(out[2][torch.from_numpy(reach <= 32)]).any()
    neg = slim.kv4_attention(q.cuda(), ctx.cache, _gpu(ctx.table), _i32([-3, 0, -2 ** 31]), 64)
    assert not neg.any()


@pytest.mark.parametrize("qdt", ["bf16", "f32"])
def test_attention_nan_behind_a_row(slim, qdt):
    """A token appended as NaN spoils the rows that attend to it and no row before it; infinities in one
    row of q stay in that row."""
    n, length = 30, 90
    ctx = Context(slim, 3, [length], 2, 64, 64, 16, qdt)
    bad = length - 10
    k = torch.zeros((1, 2, 64), dtype=DT[qdt], device="cuda:0")
    k[0, 1, 5] = float("nan")
    slot = int(ctx.table[0, bad // 16]) * 16 + bad % 16
    vk = torch.from_numpy(ctx.v[0][1][bad:bad + 1]).to(DT[qdt]).cuda()
    slim.kv4_append(k, vk, _i32([slot]), ctx.cache, 64)
    q = _rows(np.random.default_rng(0), n, 4, 64, qdt, False).view(1, n, 4, 64)
    q[0, 3, 2, 1] = float("inf")
    out = slim.kv4_attention(q.cuda(), ctx.cache, _gpu(ctx.table), _i32([length]), 64)[0]
    first = bad - (length - n)                       # the row whose own token is the bad one
    assert torch.isnan(out[first:, 2:]).all()
    rest = out[:first, 2:].clone()
    assert torch.isnan(rest[3, 0]).all()
    rest[3, 0] = 0
    assert torch.isfinite(rest).all()
    want, tol = _attention(ctx, 0, torch.nan_to_num(q[0], posinf=0.0), 64 ** -0.5, True, qdt, qdt)
    err = np.abs(out.double().cpu().numpy() - want)
    err[3, 2] = 0
    assert np.all(err[:first] <= tol[:first])


def test_attention_peaks(slim):
    """Scores of some hundreds: one token takes all the weight, maxima grow from tile to tile."""
    ctx = Context(slim, 5, [600], 1, 128, 128, 16, "f32")
    q = 30 * _rows(np.random.default_rng(0), 4, 2, 128, "f32", False).view(1, 4, 2, 128)
    out = slim.kv4_attention(q.cuda(), ctx.cache, _gpu(ctx.table), _i32([600]), 128)
    _check(ctx, 0, out[0], q[0], 128 ** -0.5, True, "f32", "f32")
    out = slim.kv4_attention(q.cuda(), ctx.cache, _gpu(ctx.table), _i32([600]), 128, scale=0.0, causal=False)
    np.testing.assert_allclose(out[0, 0, 0].cpu().numpy(), ctx.v[0][1].mean(0)[0], atol=1e-4)
    out = slim.kv4_attention(q.cuda(), ctx.cache, _gpu(ctx.table), _i32([600]), 128, scale=-0.3)
    _check(ctx, 0, out[0], q[0], -0.3, True, "f32", "f32")


def _scaled(f):
    """Values whose size goes by the token, as f(rng, n) has it."""
    return lambda rng, v: (v.astype(np.float64) * f(rng, len(v))[:, None, None]).astype(np.float32)


RANGES = {
    "grow": _scaled(lambda rng, n: 2.0 ** np.linspace(0, 40, n)),         # past the range many times
    "shrink": _scaled(lambda rng, n: 2.0 ** np.linspace(0, -40, n)),
    "first": _scaled(lambda rng, n: np.where(np.arange(n) < 3, 2.0 ** 20, 1.0)),
    "last": _scaled(lambda rng, n: np.where(np.arange(n) > n - 4, 2.0 ** 20, 1.0)),
    "mixed": _scaled(lambda rng, n: rng.choice([0.0, 1.0, 2.0 ** -6, 2.0 ** -14, 2.0 ** -30], n)),
    "near": _scaled(lambda rng, n: 2.0 ** rng.uniform(-8, 0, n)),          # small ones, but inside it
    "tiny": _scaled(lambda rng, n: np.full(n, 2.0 ** -95)),
    "tinier": _scaled(lambda rng, n: np.full(n, 2.0 ** -110)),             # past what the unit goes to
    "huge": _scaled(lambda rng, n: np.full(n, 2.0 ** 95)),
    "constant": lambda rng, v: np.broadcast_to(rng.standard_normal((len(v), 1, 1)), v.shape).astype(np.float32),
    "offset": lambda rng, v: (100 + 0.5 * v).astype(np.float32),
    "one group": lambda rng, v: v * np.where(np.arange(v.shape[2]) < 32, np.float32(2.0 ** 18), np.float32(1)),
}


@pytest.mark.parametrize("lengths,n,hq,heads,dim,group", [
    ([400, 90], 70, 2, 2, 128, 128),
    ([2500], 90, 2, 1, 64, 32),             # runs joined
    ([333, 150], 40, 2, 1, 256, 64),
])
@pytest.mark.parametrize("what", RANGES)
@pytest.mark.parametrize("odt", ["bf16", "f32"])
def test_attention_many_rows_ranges(slim, odt, what, lengths, n, hq, heads, dim, group):
    """Values inside and past what float16 holds beside the first ones, for many rows."""
    ctx = Context(slim, 11, lengths, heads, dim, group, 32, values=RANGES[what])
    q = 3 * _rows(np.random.default_rng(1), len(lengths) * n, hq, dim, "bf16", False).view(len(lengths), n, hq, dim)
    for causal in (True, False):
        out = slim.kv4_attention(q.cuda(), ctx.cache, _gpu(ctx.table), _i32(lengths), group, causal=causal,
                                 out_dtype=DT[odt])
        for i in range(len(lengths)):
            _check(ctx, i, out[i], q[i], dim ** -0.5, causal, odt, "bf16", f"{what} {causal}")


@pytest.mark.parametrize("n", [1, 100])
@pytest.mark.parametrize("far", [18, 24, 30])
def test_attention_small_weights_count(slim, n, far):
    """One token has nearly all the weight and a value of 0: what is left are the others, 2^-far each."""
    def keys(rng, k):
        return np.where(np.arange(len(k)) == 5, 1.0, 0.5)[:, None, None] * np.ones(k.shape, np.float32)

    def values(rng, v):
        v = 1 + 0.2 * v
        v[5] = 0
        return v
    ctx = Context(slim, 14, [900], 1, 128, 64, 16, values=values, keys=lambda rng, k: keys(rng, k).astype(np.float32))
    q = torch.full((1, n, 2, 128), far * np.log(2) / 64, dtype=torch.bfloat16)
    out = slim.kv4_attention(q.cuda(), ctx.cache, _gpu(ctx.table), _i32([900]), 64, causal=False, scale=1.0)
    _check(ctx, 0, out[0], q[0], 1.0, False, "bf16", "bf16", many=n > 32)
    assert (out > 0).all()


@pytest.mark.parametrize("zero", ["all channels", "one group"])
@pytest.mark.parametrize("length", [900, 2500])
@pytest.mark.parametrize("far", [22, 26, 30, 36])
def test_attention_many_rows_beside_a_value_of_zero(slim, far, length, zero):
    """Nearly all the weight on a token whose value is 0, in one group or in all: what is left are weights 2^-far below
    it, and those count as exactly as in a call of few rows (no float16 allowance)."""
    at = 41 if length == 900 else length - 3         # of the first tile, of the last one

    def keys(rng, k):
        return np.where(np.arange(len(k)) == at, 1.0, 0.5)[:, None, None].astype(np.float32) * np.ones_like(k)

    def values(rng, v):
        v = 1 + 0.2 * v
        v[at, :, 64 if zero[0] == "o" else 0:] = 0
        return v
    ctx = Context(slim, 15, [length], 1, 128, 64, 16, values=values, keys=keys)
    q = torch.full((1, 100, 2, 128), far * np.log(2) / 64, dtype=torch.bfloat16)
    out = slim.kv4_attention(q.cuda(), ctx.cache, _gpu(ctx.table), _i32([length]), 64, causal=False, scale=1.0)
    want, tol = _attention(ctx, 0, q[0], 1.0, False, "bf16", "bf16", many=False)
    err = np.abs(out[0].double().cpu().numpy() - want)
    assert np.all((err <= tol)[..., 64:])            # the other group's are one weight's, and within it as well
    if zero[0] == "a":
        assert np.all(err <= tol)


def test_attention_many_rows_of_nothing(slim):
    """Values of 0 are 0, and so are rows before the first token."""
    ctx = Context(slim, 12, [100, 20], 2, 64, 64, 16, values=lambda rng, v: 0 * v)
    q = _rows(np.random.default_rng(1), 180, 4, 64, "bf16", False).view(2, 90, 4, 64).cuda()
    out = slim.kv4_attention(q, ctx.cache, _gpu(ctx.table), _i32([100, 20]), 64)
    assert not out.any()
    ctx = Context(slim, 12, [100, 20], 2, 64, 64, 16)
    out = slim.kv4_attention(q, ctx.cache, _gpu(ctx.table), _i32([100, 20]), 64)
    assert not out[1, :70].any()
    _check(ctx, 1, out[1], q[1].cpu(), 64 ** -0.5, True, "bf16", "bf16")


@pytest.mark.parametrize("length,n", [(150, 100), (2000, 70), (70, 70)])
@pytest.mark.parametrize("where", ["key", "value", "infinite value"])
def test_attention_many_rows_nan_behind_a_row(slim, length, n, where):
    ctx = Context(slim, 13, [length], 2, 128, 64, 16)
    bad = length - n // 2
    k = torch.from_numpy(ctx.k[0][1][bad:bad + 1]).to(torch.bfloat16).cuda()
    v = torch.from_numpy(ctx.v[0][1][bad:bad + 1]).to(torch.bfloat16).cuda()
    (k if where == "key" else v)[0, 1, 70] = float("inf" if where[0] == "i" else "nan")
    slot = int(ctx.table[0, bad // 16]) * 16 + bad % 16
    slim.kv4_append(k, v, _i32([slot]), ctx.cache, 64)
    q = _rows(np.random.default_rng(0), n, 4, 128, "bf16", False).view(1, n, 4, 128)
    out = slim.kv4_attention(q.cuda(), ctx.cache, _gpu(ctx.table), _i32([length]), 64)[0]
    first = bad - (length - n)                       # the row whose own token is the bad one
    spoilt = out[first:, 2:] if where == "key" else out[first:, 2:, 64:]
    assert torch.isnan(spoilt).all()
    want, tol = _attention(ctx, 0, q[0], 128 ** -0.5, True, "bf16", "bf16")
    err = np.abs(out.double().cpu().numpy() - want)
    assert np.all(err[:first] <= tol[:first])        # no NaN either


def test_attention_pages_past_32_bits(slim):
    """Records more than 4 GiB into the cache: the last pages of a long one."""
    dim, group, page, heads = 128, 128, 256, 8
    words = oracle.kv4_words(page, dim, group)
    pages = (5 << 30) // (heads * words * 4)
    cache = torch.empty((pages, heads, words), dtype=torch.int32, device="cuda:0")
    rng = np.random.default_rng(1)
    length = 300
    k, v = _rows(rng, length, heads, dim, "bf16").cuda(), _rows(rng, length, heads, dim, "bf16", False).cuda()
    q = _rows(rng, 1, heads, dim, "bf16", False).view(1, 1, heads, dim).cuda()
    small = slim.kv4_cache(2, heads, dim, group, page)
    at = np.arange(length)
    slim.kv4_append(k, v, _i32(at), small, group)
    want = slim.kv4_attention(q, small, _i32([[0, 1]]), _i32([length]), group)
    slots = np.where(at < 256, (pages - 1) * page + at, (pages - 2) * page + at - 256).astype(np.int32)
    slim.kv4_append(k, v, _gpu(slots), cache, group)
    got = slim.kv4_attention(q, cache, _i32([[pages - 1, pages - 2]]), _i32([length]), group)
    assert torch.equal(got, want)
    for a, b in zip(slim.kv4_read(_gpu(slots), cache, dim, group), slim.kv4_read(_i32(at), small, dim, group)):
        assert torch.equal(a, b)


# ---------------------------------------------------------------- drafts
def _drafts(seed, b, k, v, dt, draft=True, pad=0, spread=3.0):
    rng = np.random.default_rng(seed)
    t = (spread * rng.standard_normal((b, k + 1, v + pad))).astype(np.float32)
    d = t[:, :k] + rng.standard_normal((b, k, v + pad)).astype(np.float32)
    target, dr = torch.from_numpy(t).to(DT[dt]), torch.from_numpy(d).to(DT[dt])
    tokens = (dr.float().numpy()[:, :, :v] + rng.gumbel(size=(b, k, v))).argmax(-1)
    return target[:, :, :v], dr[:, :, :v] if draft else None, tokens, rng.random((b, k + 1)).astype(np.float32)


def _verify(slim, target, tokens, uniform, draft, temperature=1.0):
    out = slim.verify_draft(target.cuda(), _gpu(tokens), _gpu(uniform), draft=None if draft is None else draft.cuda(),
                            temperature=temperature)
    b, k = tokens.shape
    assert out["accepted"].shape == (b,) and out["ids"].shape == (b, k + 1)
    acc, ids, margin = oracle.verify_draft([[_host(r) for r in s] for s in target], tokens, uniform,
                                           None if draft is None else [[_host(r) for r in s] for s in draft], temperature)
    # float64 on both sides: sums of v terms agree to v 2^-53, so nothing nearer than this may differ
    sure = margin > 1e-11
    assert sure.all()
    np.testing.assert_array_equal(out["accepted"].cpu().numpy(), acc)
    np.testing.assert_array_equal(out["ids"].cpu().numpy(), ids)
    return acc, ids


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("temperature", [1.0, 1e-300, 1e300, 1e36])
@pytest.mark.parametrize("v", [700, 9001])
def test_draft_extreme_logits(slim, dt, draft, temperature, v):
    """Masks of the type's lowest value, whole rows of it, logits of 10^30, temperatures near 0 and infinity."""
    rng = np.random.default_rng(v)
    low = float(torch.finfo(DT[dt]).min)
    b, k = 7, 2
    t = 3 * rng.standard_normal((b, k + 1, v))
    t[0] = low
    t[1][:, ::2] = low
    t[2] *= 1e30
    t[3][:, 7:] = -np.inf
    t[4] = np.where(rng.random(t[4].shape) < 0.5, 1e20, 0.99e20)
    t[5][:, :v // 2] = -np.inf
    t[5][:, v // 2:] = low
    t[6][:, v - 3:] = 50.0
    d = t[[6, 1, 2, 3, 0, 4, 5], :k] + 0.0
    target, dr = torch.from_numpy(t).to(DT[dt]), torch.from_numpy(d).to(DT[dt])
    tokens = rng.integers(0, v, (b, k))
    tokens[3], tokens[6, 0] = 3, v - 1
    u = rng.random((b, k + 1)).astype(np.float32)
    _verify(slim, target, tokens, u, dr if draft else None, temperature)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("temperature", [1e-5, 1e-8, 1e-9, 1e-10, 1e-12, 1e-40, 1e-305])
def test_draft_small_temperatures(slim, dt, temperature):
    """As far as the greatest logit alone has weight, whether it is 0, near 0 or large; the next float below it has
    none, and equal ones share."""
    rng = np.random.default_rng(4)
    b, k, v = 5, 2, 5000
    t = -np.abs(rng.standard_normal((b, k + 1, v))) - 0.01
    t[0][:, 17] = 0.0
    t[1] += 20
    t[2][:, 40:44] = 0.0
    t[3] *= 1e-30
    t[4] = 3e4 - np.abs(t[4])
    target = torch.from_numpy(t).to(DT[dt])
    tokens = target.float().argmax(-1)[:, :k].numpy().copy()
    tokens[1, 1] = (tokens[1, 1] + 1) % v
    u = (0.1 + 0.8 * rng.random((b, k + 1))).astype(np.float32)
    _verify(slim, target, tokens, u, None, temperature)


DRAFTS = [
    (1, 1, 1, "f32", True, 0, 1.0),
    (1, 4, 1000, "f32", True, 0, 1.0),
    (3, 2, 2049, "bf16", True, 3, 0.7),
    (7, 3, 10007, "f32", False, 13, 1.0),
    (20, 5, 333, "bf16", True, 0, 1.3),
    (40, 8, 2000, "bf16", False, 1, 1.0),
    (2, 32, 5000, "f32", True, 0, 1.0),
    (65, 1, 100, "f32", True, 0, 2.0),
    (4, 3, 70001, "bf16", True, 0, 1.0),
    (60, 5, 17000, "bf16", True, 7, 0.9),      # segments of 8192
]


@pytest.mark.parametrize("b,k,v,dt,draft,pad,temperature", DRAFTS)
def test_verify_draft(slim, b, k, v, dt, draft, pad, temperature):
    print(f"verify b={b} k={k} v={v} {dt} {draft} pad={pad} T={temperature}", flush=True)
    target, dr, tokens, uniform = _drafts(b * 31 + v, b, k, v, dt, draft, pad)
    if b > 2:
        tokens[1, k // 2:] = -1
        tokens[2, 0] = v + 5                         # outside the vocabulary: refused
    acc, _ = _verify(slim, target, tokens, uniform, dr, temperature)
    if b >= 20:
        assert acc.max() > 0 and acc.min() == 0


def test_verify_draft_ends(slim):
    """Uniforms at their ends, equal rows, point masses, masked entries, rows without a distribution."""
    inf = float("inf")
    v = 300
    target, dr, tokens, uniform = _drafts(1, 10, 2, v, "f32")
    target, dr = target.clone(), dr.clone()
    uniform[0] = 0.0
    uniform[1, 2] = np.nextafter(np.float32(1), np.float32(0))
    dr[2] = target[2, :2]                            # p = q: always taken
    target[3, 0, 10:] = -inf                         # masked: never drawn, never taken
    tokens[3, 0] = 20
    target[4, 0] = float("nan")
    target[5, 1, 7] = inf
    dr[6, 0] = -inf
    target[7, 0] = -inf
    target[7, 0, 5] = 0.0                            # a point mass
    tokens[7, 0], uniform[7, 0] = 6, 0.0
    dr[8, 0, :] = -inf
    dr[8, 0, 4] = 1.0
    tokens[8, 0], uniform[8, 0] = 4, 0.999
    target[9, 2] = float("nan")
    dr[9], uniform[9, :2] = target[9, :2], 0.5
    out = slim.verify_draft(target.cuda(), _gpu(tokens), _gpu(uniform), draft=dr.cuda())
    acc, ids, margin = oracle.verify_draft([[_host(r) for r in s] for s in target], tokens, uniform,
                                           [[_host(r) for r in s] for s in dr])
    np.testing.assert_array_equal(out["accepted"].cpu().numpy(), acc)
    np.testing.assert_array_equal(out["ids"].cpu().numpy(), ids)
    assert acc[2] == 2 and ids[4, 0] == -1 and ids[6, 0] == -1 and ids[7, 0] == 5 and acc[9] == 2 and ids[9, 2] == -1


@pytest.mark.parametrize("far,drawn", [(-30.0, 9), (-706.0, 9), (-708.0, -1), (-800.0, -1)])
def test_verify_draft_least_powers(slim, far, drawn):
    """What is left to draw from is one entry e^far of the greatest: 2^-1018.5 counts, 2^-1021.4 is 0, as the header has it."""
    target = torch.full((1, 2, 300), -float("inf"))
    target[0, :, 3] = 0.0
    dr = target[:, :1].clone()
    target[0, :, 9] = far
    out = slim.verify_draft(target.cuda(), _gpu(np.array([[5]])), _gpu(np.array([[0.5, 0.5]], np.float32)), draft=dr.cuda())
    assert int(out["accepted"][0]) == 0 and out["ids"][0].tolist() == [drawn, -1]


def test_verify_draft_shared_rows(slim):
    """One target row for every sequence (stride 0), and no sequences at all."""
    target, dr, tokens, uniform = _drafts(2, 6, 2, 500, "bf16")
    one = target[:1].expand(6, 3, 500)
    a = slim.verify_draft(one.cuda()[:1].expand(6, 3, 500), _gpu(tokens), _gpu(uniform), draft=dr.cuda())
    b = slim.verify_draft(one.contiguous().cuda(), _gpu(tokens), _gpu(uniform), draft=dr.cuda())
    assert torch.equal(a["ids"], b["ids"])
    out = slim.verify_draft(target[:0].cuda(), _gpu(tokens[:0]), _gpu(uniform[:0]))
    assert out["accepted"].shape == (0,) and out["ids"].shape == (0, 3)


# ---------------------------------------------------------------- as they are used
def _step(slim, st):
    """A decode step with drafted tokens: cache, attention, an output layer in 4 bits, the drafts judged."""
    q = slim.kv4_append(st["k"], st["v"], st["slots"], st["cache"], st["group"], rotary=st["rotary"],
                        positions=st["positions"], q=st["q"])
    b, n = st["tokens"].shape[0], st["tokens"].shape[1] + 1
    o = slim.kv4_attention(q.view(b, n, *q.shape[1:]), st["cache"], st["table"], st["lengths"], st["group"])
    h = o.reshape(b * n, -1)
    logits = slim.q4_linear(h, st["head"], st["vocabulary"], 128)
    out = slim.verify_draft(logits.view(b, n, -1), st["tokens"], st["uniform"], draft=st["draft"], temperature=0.9)
    return {"q": q, "o": o, "logits": logits, **out}


def _step_state(slim, seed, dt="bf16"):
    rng = np.random.default_rng(seed)
    b, n, hq, heads, dim, group, page, vocabulary = 3, 4, 4, 2, 64, 32, 16, 517
    lengths = [70, 33, 4]
    st = {"group": group, "vocabulary": vocabulary, "cache": slim.kv4_cache(20, heads, dim, group, page)}
    table = rng.permutation(20)[:15].reshape(3, 5).astype(np.int32)
    st["table"], st["lengths"] = _gpu(table), _i32(lengths)
    past_k, past_v = [], []
    rot = _table(rng, 100, dim)
    st["rotary"] = _gpu(rot)
    slot = lambda i, p: int(table[i, p // page]) * page + p % page  # noqa: E731
    for i, length in enumerate(lengths):
        m = length - n
        k, v = _rows(rng, m, heads, dim, dt), _rows(rng, m, heads, dim, dt, False)
        past_k.append(k), past_v.append(v)
        if m:
            slim.kv4_append(k.cuda(), v.cuda(), _i32([slot(i, p) for p in range(m)]), st["cache"], group,
                            rotary=st["rotary"], positions=_i32(range(m)))
    k, v, q = (_rows(rng, b * n, h, dim, dt, c) for h, c in ((heads, True), (heads, False), (hq, False)))
    pos = [length - n + j for length in lengths for j in range(n)]
    st["k"], st["v"], st["q"], st["positions"] = k.cuda(), v.cuda(), q.cuda(), _i32(pos)
    st["slots"] = _i32([slot(i // n, p) for i, p in enumerate(pos)])
    codes = rng.integers(0, 16, size=(vocabulary, hq * dim), dtype=np.uint8)
    scale = rng.uniform(0.02, 0.05, (vocabulary, hq * dim // 128)).astype(np.float32)
    zero = rng.uniform(6, 9, (vocabulary, hq * dim // 128)).astype(np.float32)
    st["head"] = slim.pack4(_gpu(codes), _gpu(scale), _gpu(zero), 128)
    st["draft"] = _gpu(rng.standard_normal((b, n - 1, vocabulary)).astype(np.float32) * 2)
    st["tokens"] = _gpu(rng.integers(0, vocabulary, (b, n - 1)))
    st["uniform"] = _gpu(rng.random((b, n)).astype(np.float32))
    host = dict(lengths=lengths, n=n, rot=rot, k=k, v=v, q=q, pos=pos, past_k=past_k, past_v=past_v, codes=codes,
                scale=scale, zero=zero, group=group, dim=dim)
    return st, host


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_a_decode_step(slim, dt):
    """The operators one after another, each against its definition on what the one before it gave."""
    st, h = _step_state(slim, 1, dt)
    out = _step(slim, st)
    qr = oracle.rotate(_host(h["q"]), h["rot"], h["pos"], False)
    np.testing.assert_array_equal(out["q"].float().cpu().numpy(), oracle.bf16_round(qr) if dt == "bf16" else qr)
    n = h["n"]
    ctx = Context.__new__(Context)
    ctx.group, ctx.k, ctx.v = h["group"], [], []
    for i, length in enumerate(h["lengths"]):
        new = slice(i * n, (i + 1) * n)
        k = np.concatenate([oracle.rotate(_host(h["past_k"][i]), h["rot"], range(length - n), False),
                            oracle.rotate(_host(h["k"][new]), h["rot"], h["pos"][new], False)])
        v = np.concatenate([oracle.as_f32(_host(x)) for x in (h["past_v"][i], h["v"][new])])
        for x, to in ((k, ctx.k), (v, ctx.v)):
            z = oracle.kv4_quantize(x, h["group"])
            to.append((z, oracle.kv4_values(*z, h["group"])))
        _check(ctx, i, out["o"][i], out["q"][new], h["dim"] ** -0.5, True, dt, dt)
    want = oracle.q4_linear(_host(out["o"].reshape(len(h["lengths"]) * n, -1)), h["codes"], h["scale"], h["zero"], 128)
    assert np.abs(out["logits"].cpu().numpy() - want).max() < 1e-4 * np.abs(want).max()
    acc, ids, margin = oracle.verify_draft(out["logits"].view(-1, n, st["vocabulary"]).cpu().numpy(), st["tokens"].cpu().numpy(),
                                           st["uniform"].cpu().numpy(), st["draft"].cpu().numpy(), 0.9)
    assert (margin > 1e-11).all()
    np.testing.assert_array_equal(out["accepted"].cpu().numpy(), acc)
    np.testing.assert_array_equal(out["ids"].cpu().numpy(), ids)


def _equal(a, b):
    return all(torch.equal(a[k], b[k]) for k in a)


def test_a_step_on_a_side_stream_and_from_graphs(slim):
    """On another stream than the inputs' own, and from two captured graphs replayed in turns with other inputs and
    eager work between."""
    st, _ = _step_state(slim, 2)
    eager = _step(slim, st)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = _step(slim, st)
    side.synchronize()
    assert _equal(eager, again)
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = _step(slim, st)
        graphs.append((gr, out))
    for turn in range(5):
        fresh, _ = _step_state(slim, 10 + turn)
        for name in ("k", "v", "q", "tokens", "uniform", "draft", "table", "lengths", "slots", "positions", "rotary", "head"):
            st[name].copy_(fresh[name])
        st["cache"].copy_(fresh["cache"])
        kept = st["cache"].clone()
        eager = _step(slim, st)
        after = st["cache"].clone()
        st["cache"].copy_(kept)
        gr, out = graphs[turn % 2]
        gr.replay()
        torch.cuda.synchronize()
        assert _equal(eager, out) and torch.equal(st["cache"], after)


def test_steps_from_two_threads(slim):
    """Steps from two host threads, each on a stream of its own, against what each gives alone."""
    import threading
    states = [_step_state(slim, 20 + i)[0] for i in range(2)]
    alone = [_step(slim, st) for st in states]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(30):
                out = _step(slim, states[i])
                stream.synchronize()
                if not _equal(out, alone[i]):
                    wrong.append(i)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not wrong


def test_long_rows_in_graphs(slim):
    """Calls with a workspace (runs that are joined; many rows), captured twice, replayed in turns."""
    ctx = Context(slim, 6, [3000, 900], 2, 128, 128, 64)
    rng = np.random.default_rng(7)
    q = _rows(rng, 2 * 40, 4, 128, "bf16", False).view(2, 40, 4, 128).cuda()
    one = _rows(rng, 2, 4, 128, "bf16", False).view(2, 1, 4, 128).cuda()
    table, lengths = _gpu(ctx.table), _i32([3000, 900])

    def run():
        return [slim.kv4_attention(x, ctx.cache, table, lengths, 128) for x in (q, one)]
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = run()
        graphs.append((gr, out))
    for turn in range(6):
        q.copy_(_rows(rng, 2 * 40, 4, 128, "bf16", False).view(2, 40, 4, 128))
        lengths.copy_(_i32([3000 - 100 * turn, 900 - turn]))
        eager = run()
        graphs[turn % 2][0].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, graphs[turn % 2][1]))


def test_many_sequences_of_uneven_lengths(slim):
    """More sequences than a wave has lanes with a long one among them: its runs, the others whole."""
    rng = np.random.default_rng(8)
    lengths = [int(x) for x in rng.integers(0, 50, 130)]
    lengths[77] = 5000
    ctx = Context(slim, 11, lengths, 1, 64, 64, 32)
    q = _rows(rng, 130, 2, 64, "bf16", False).view(130, 1, 2, 64)
    out = slim.kv4_attention(q.cuda(), ctx.cache, _gpu(ctx.table), _i32(lengths), 64)
    for i in range(130):
        if lengths[i]:
            _check(ctx, i, out[i], q[i], 64 ** -0.5, True, "bf16", "bf16")
        else:
            assert not out[i].any()


def test_the_most_sequences(slim):
    """4096 of them, uniform and by offsets."""
    rng = np.random.default_rng(9)
    lengths = [int(x) for x in rng.integers(0, 5, 4096)]
    ctx = Context(slim, 12, lengths, 1, 64, 32, 16)
    q = _rows(rng, 4096, 1, 64, "bf16", False)
    out = slim.kv4_attention(q.view(4096, 1, 1, 64).cuda(), ctx.cache, _gpu(ctx.table), _i32(lengths), 32)
    off = slim.kv4_attention(q.cuda(), ctx.cache, _gpu(ctx.table), _i32(lengths), 32, offsets=_i32(range(4097)))
    assert torch.equal(out.view(4096, 1, 64), off)
    for i in list(range(0, 4096, 97)) + [4095]:
        if lengths[i]:
            _check(ctx, i, out[i], q[i:i + 1], 64 ** -0.5, True, "bf16", "bf16")
        else:
            assert not out[i].any()


def test_append_in_several_launches(slim):
    """More items than a launch takes: tokens of 1024 heads (values checked at both ends and around the seam)."""
    heads, dim, page = 1024, 64, 16
    per = (1 << 31) // (2 * heads * (dim // 8))          # tokens a launch takes without queries
    t = per + 5
    one = torch.randn((1, heads, dim), device="cuda:0").to(torch.bfloat16)
    rows = one.expand(t, heads, dim)
    slots = torch.full((t,), -1, dtype=torch.int32, device="cuda:0")
    put = [0, 1, per - 1, per, per + 4]
    for i, x in enumerate(put):
        slots[x] = i
    cache = slim.kv4_cache(1, heads, dim, 32, page)
    slim.kv4_append(rows, rows, slots, cache, 32)
    want = slim.kv4_cache(1, heads, dim, 32, page)
    slim.kv4_append(one.expand(5, heads, dim).contiguous(), one.expand(5, heads, dim).contiguous(), _i32(range(5)), want, 32)
    assert torch.equal(cache, want)


def test_verify_draft_extremes(slim):
    """The most drafted tokens; rows of 2^24 logits; thousands of sequences of a small vocabulary."""
    target, dr, tokens, uniform = _drafts(40, 1, 32, 50, "f32")
    dr = target[:, :32].clone()                          # all accepted
    acc, _ = _verify(slim, target, tokens, uniform, dr)
    assert acc[0] == 32
    v = 1 << 24
    gen = torch.Generator(device="cuda:0")
    gen.manual_seed(3)
    target = torch.randn((1, 2, v), generator=gen, device="cuda:0").to(torch.bfloat16)
    u = torch.tensor([[0.5, 0.73]], device="cuda:0")
    out = slim.verify_draft(target, torch.tensor([[5]], device="cuda:0"), u)
    p = torch.softmax(target[0, 0].double(), 0)
    assert float(p[5]) < 0.4 and int(out["accepted"][0]) == 0
    p[5] = 0
    run = p.cumsum(0)
    assert int(out["ids"][0, 0]) == int((run <= u[0, 1].double() * run[-1]).sum())
    b = 5000
    target, dr, tokens, uniform = _drafts(41, b, 1, 7, "f32")
    acc, _ = _verify(slim, target, tokens, uniform, dr)
    assert 0 < acc.mean() < 1


def test_outputs_over_inputs_are_refused(slim):
    cache = slim.kv4_cache(3, 2, 64, 32, 16)
    q = torch.zeros((4, 1, 4, 64), device="cuda:0")
    with pytest.raises(slim.SlimError, match="out: overlaps q"):
        slim.kv4_attention(q, cache, _i32([[0, 1]] * 4), _i32([1] * 4), 32, out=q)
    words = cache.view(-1)
    with pytest.raises(slim.SlimError, match="overlaps"):
        slim.kv4_append(torch.zeros((5, 2, 64), device="cuda:0"), torch.zeros((5, 2, 64), device="cuda:0"), words[:5],
                        cache, 32)
    k = words[:640].view(torch.float32).view(5, 2, 64)
    with pytest.raises(slim.SlimError, match="overlaps"):
        slim.kv4_append(k, k, _i32(range(5)), cache, 32)
    host = torch.zeros((5, 2, 64))
    with pytest.raises(slim.SlimError, match="GPU"):
        slim.kv4_append(host, host, _i32(range(5)), cache, 32)

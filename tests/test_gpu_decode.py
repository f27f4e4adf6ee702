"""The decode step's operators - the 4-bit key/value cache, attention over it and the verification of
drafted tokens - against the oracle, through the binding.

The cache is compared word for word.  Attention's tolerance, from the arithmetic (see _attention): a
score's error is at most 2^-23 (dim + 16) of scale sum |q| (|code step| + |low|), plus what rounding
its power's argument adds, and it enters the weights as a factor; weights of the second product round
by 2^-8 (bfloat16 q) or not (three terms); sums over the tokens add 2^-23 a term of a lane's chain; a
bfloat16 output adds 2^-8 of the value.
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

    def __init__(self, slim, seed, lengths, heads, dim, group, page, dt="bf16", spare=2):
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
            at = np.arange(max(n, 0))
            slots = (self.table[i, at // page] * page + at % page).astype(np.int32)
            slim.kv4_append(k.cuda(), v.cuda(), _gpu(slots), self.cache, group)
            kq, vq = (oracle.kv4_quantize(oracle.as_f32(_host(x)), group) for x in (k, v))
            self.k.append((kq, oracle.kv4_values(*kq, group)))
            self.v.append((vq, oracle.kv4_values(*vq, group)))
        self.lengths, self.group, self.page, self.pages = list(lengths), group, page, pages


def _attention(ctx, i, q, scale, causal, odt, qdt):
    """float64 result of sequence i and its tolerance."""
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
            tol[a, h] = (2.0 ** -8 if qdt == "bf16" else 0) * part + (2 * ds.max() + chain) * whole
    return want, tol + (2.0 ** -8 * np.abs(want) if odt == "bf16" else 0) + 1e-30


def _check(ctx, i, got, q, scale, causal, odt, qdt, what=""):
    want, tol = _attention(ctx, i, q, scale, causal, odt, qdt)
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
            _check(ctx, i, out[i], q[i], dim ** -0.5, causal, odt, qdt)
    again = slim.kv4_attention(q.cuda(), ctx.cache, _gpu(ctx.table), _i32(lengths), group, causal=causal,
                               out_dtype=DT[odt])
    assert torch.equal(out, again)


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


def test_verify_draft_shared_rows(slim):
    """One target row for every sequence (stride 0), and no sequences at all."""
    target, dr, tokens, uniform = _drafts(2, 6, 2, 500, "bf16")
    one = target[:1].expand(6, 3, 500)
    a = slim.verify_draft(one.cuda()[:1].expand(6, 3, 500), _gpu(tokens), _gpu(uniform), draft=dr.cuda())
    b = slim.verify_draft(one.contiguous().cuda(), _gpu(tokens), _gpu(uniform), draft=dr.cuda())
    assert torch.equal(a["ids"], b["ids"])
    out = slim.verify_draft(target[:0].cuda(), _gpu(tokens[:0]), _gpu(uniform[:0]))
    assert out["accepted"].shape == (0,) and out["ids"].shape == (0, 3)

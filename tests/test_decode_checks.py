"""The decode step's calls reject bad arguments on the host: the C ABI by status code, the binding by an error naming
the argument (CPU only: nothing is enqueued, no pointer is dereferenced)."""
import ctypes
import os

import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.skipif(
    not os.path.exists(os.path.join(ROOT, "post_mixed_precision_amd", "libslim.so")),
    reason="libslim.so not built (run __graft_entry__.build())")

FAKE = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4100)
BYTE = ctypes.c_void_p(4097)


@pytest.fixture(scope="module")
def L():
    from post_mixed_precision_amd import _lib
    _lib.load_library()
    return _lib


@pytest.fixture(scope="module")
def lib(L):
    return L.load_library()


def raises(L, fn, *words):
    with pytest.raises(L.SlimError) as e:
        fn()
    for w in words:
        assert w in str(e.value), str(e.value)


def test_words(lib):
    assert lib.slim_kv4_words(64, 128, 128) == 4 * (512 + 32)
    assert lib.slim_kv4_words(16, 64, 32) == 256 + 64
    for bad in ((8, 64, 32), (48, 64, 32), (512, 64, 32), (16, 96, 32), (16, 64, 128), (16, 64, 48), (-16, 64, 32)):
        assert lib.slim_kv4_words(*bad) == -1


def test_append_abi(lib):
    def call(**kw):
        g = kw.get
        return lib.slim_kv4_append(g("k", FAKE), g("krow", 256), g("khead", 64), g("v", FAKE), g("vrow", 256), 64,
                                   g("xdt", 1), g("t", 4), g("heads", 4), g("dim", 64), g("group", 32), g("slots", FAKE),
                                   g("cache", FAKE), g("pages", 8), g("page", 16), g("rotary", FAKE), g("npos", 100),
                                   g("rot", 64), 0, g("pos", FAKE), g("q", FAKE), g("hq", 8), 512, 64,
                                   g("out", FAKE), None)
    assert call(k=None) == -1 and call(v=None) == -1 and call(slots=None) == -1 and call(cache=None) == -1
    assert call(pos=None) == -1 and call(q=None) == -1 and call(out=None) == -1
    assert call(xdt=2) == -3
    assert call(t=-1) == -2 and call(t=(1 << 20) + 1) == -2 and call(heads=0) == -2 and call(heads=1025) == -2
    assert call(dim=96) == -2 and call(group=128) == -2 and call(page=24) == -2 and call(pages=0) == -2
    assert call(pages=(1 << 26) + 1) == -2 and call(hq=-1) == -2 and call(hq=1025) == -2
    assert call(krow=-1) == -2 and call(khead=-64) == -2 and call(vrow=1 << 41) == -2
    assert call(rot=0) == -2 and call(rot=66) == -2 and call(rot=7) == -2 and call(npos=0) == -2
    assert call(cache=ODD) == -7 and call(out=ODD) == -7 and call(k=BYTE) == -7 and call(xdt=0, v=ctypes.c_void_p(4098)) == -7
    assert call(t=0, k=None, v=None, slots=None, cache=None) == 0


def test_read_abi(lib):
    def call(**kw):
        g = kw.get
        return lib.slim_kv4_read(g("slots", FAKE), g("t", 4), g("cache", FAKE), g("pages", 8), g("page", 16), g("heads", 4),
                                 g("dim", 64), g("group", 32), g("k", FAKE), g("v", FAKE), g("odt", 0), None)
    assert call(slots=None) == -1 and call(cache=None) == -1 and call(k=None) == -1 and call(v=None) == -1
    assert call(odt=3) == -3
    assert call(t=-1) == -2 and call(heads=0) == -2 and call(dim=32) == -2 and call(page=8) == -2 and call(pages=0) == -2
    assert call(cache=ODD) == -7 and call(k=ODD) == -7 and call(v=ODD) == -7
    assert call(t=0, slots=None) == 0


def test_attention_abi(lib):
    def call(**kw):
        g = kw.get
        return lib.slim_kv4_attention(g("q", FAKE), g("qdt", 1), g("tq", 4), g("hq", 8), g("cache", FAKE), g("pages", 8),
                                      g("page", 16), g("heads", 4), g("dim", 64), g("group", 32), g("table", FAKE),
                                      g("b", 4), g("per", 1000), g("lengths", FAKE), g("offsets", None), g("scale", 0.1), 1,
                                      g("out", FAKE), g("odt", 1), g("ws", FAKE), g("wsb", 1 << 40), None)
    assert call(q=None) == -1 and call(cache=None) == -1 and call(table=None) == -1 and call(lengths=None) == -1
    assert call(out=None) == -1
    assert call(qdt=2) == -3 and call(odt=-1) == -3
    assert call(hq=6) == -2 and call(hq=0) == -2 and call(hq=1028) == -2 and call(heads=0) == -2
    assert call(dim=80) == -2 and call(group=128) == -2 and call(page=20) == -2 and call(pages=0) == -2
    assert call(b=0) == -2 and call(b=4097, tq=4097) == -2 and call(tq=5) == -2 and call(tq=-1) == -2
    assert call(tq=(1 << 20) + 4) == -2 and call(per=0) == -2 and call(per=1 << 27) == -2
    assert call(tq=1 << 20, hq=128) == -2                    # 2^27 rows
    assert call(scale=float("nan")) == -4 and call(scale=float("inf")) == -4 and call(scale=1e300) == -4
    assert call(q=ODD) == -7 and call(cache=ODD) == -7 and call(out=ODD) == -7
    assert call(tq=0, q=None, out=None) == 0
    need = lib.slim_kv4_attention_workspace(4, 4, 0, 8, 4, 64, 32, 1000, 16, 1, 1)
    assert need > 0
    assert call(wsb=need - 1) == -5 and call(ws=None) == -5 and call(ws=ODD) == -7
    assert lib.slim_kv4_attention_workspace(4, 5, 0, 8, 4, 64, 32, 1000, 16, 1, 1) == 0
    assert lib.slim_kv4_attention_workspace(4, 4, 0, 8, 4, 64, 128, 1000, 16, 1, 1) == 0
    assert lib.slim_kv4_attention_workspace(4, 4, 0, 8, 4, 64, 32, 1, 16, 1, 1) == 0      # 16 tokens: nothing to join


def test_attention_workspace_of_extreme_shapes(lib):
    for qdt in (0, 1):
        for b, tq in ((1, 1), (4096, 4096), (1, 1 << 20), (1024, 1 << 20)):
            for hq, heads in ((1, 1), (1024, 1), (1024, 1024)):
                need = lib.slim_kv4_attention_workspace(b, tq, 1, hq, heads, 256, 32, 1 << 22, 256, qdt, qdt)
                assert need < 1 << 38


def test_verify_abi(lib):
    def call(**kw):
        g = kw.get
        return lib.slim_verify_draft(g("t", FAKE), g("tseq", 400), g("trow", 100), g("d", FAKE), g("dseq", 300),
                                     g("drow", 100), g("dt", 0), g("b", 4), g("k", 3), g("v", 100), g("tok", FAKE),
                                     g("u", FAKE), g("temp", 1.0), g("acc", FAKE), g("ids", FAKE), g("ws", FAKE),
                                     g("wsb", 1 << 40), None)
    assert call(t=None) == -1 and call(tok=None) == -1 and call(u=None) == -1 and call(acc=None) == -1
    assert call(ids=None) == -1
    assert call(dt=4) == -3
    assert call(b=-1) == -2 and call(b=65537) == -2 and call(k=0) == -2 and call(k=33) == -2 and call(v=0) == -2
    assert call(v=(1 << 24) + 1, trow=1 << 25, drow=1 << 25) == -2 and call(trow=99) == -2 and call(drow=99) == -2
    assert call(tseq=-1) == -2 and call(dseq=-1) == -2 and call(b=65536, v=1 << 24, trow=1 << 24, drow=1 << 24) == -2
    for temp in (0.0, -1.0, float("nan"), float("inf"), 1e-320):
        assert call(temp=temp) == -4
    assert call(t=BYTE) == -7 and call(d=ctypes.c_void_p(4098)) == -7
    assert call(b=0, t=None) == 0
    need = lib.slim_verify_draft_workspace(4, 3, 100)
    assert need > 0
    assert call(wsb=need - 1) == -5 and call(ws=None) == -5 and call(ws=ODD) == -7
    assert lib.slim_verify_draft_workspace(4, 0, 100) == 0 and lib.slim_verify_draft_workspace(0, 3, 100) == 0


def _bf(*s):
    return torch.zeros(s, dtype=torch.bfloat16)


def _f(*s):
    return torch.zeros(s)


def _i(*s):
    return torch.zeros(s, dtype=torch.int32)


def test_cache_binding(L):
    raises(L, lambda: L.kv4_cache(4, 2, 96, 32), "96")
    raises(L, lambda: L.kv4_cache(4, 2, 64, 128), "groups of 128")
    raises(L, lambda: L.kv4_cache(4, 2, 64, 32, page=24), "24")
    raises(L, lambda: L.kv4_cache(0, 2, 64, 32), "pages")
    raises(L, lambda: L.kv4_cache(4, 0, 64, 32), "heads")
    raises(L, lambda: L.kv4_cache(1 << 27, 1, 64, 32, page=16), "range")
    assert L.kv4_cache(3, 2, 64, 32, page=16, device="cpu").shape == (3, 2, 320)


def test_append_binding(L):
    cache = L.kv4_cache(3, 2, 64, 32, page=16, device="cpu")
    k, s, rot, pos = _bf(5, 2, 64), _i(5), _f(9, 64), _i(5)
    go = L.kv4_append
    raises(L, lambda: go([1], k, s, cache, 32), "k", "tensor")
    raises(L, lambda: go(k.half(), k.half(), s, cache, 32), "k", "dtype")
    raises(L, lambda: go(k, k.float(), s, cache, 32), "v", "dtype")
    raises(L, lambda: go(k, _bf(5, 3, 64), s, cache, 32), "v", "shape")
    raises(L, lambda: go(_bf(5, 64), k, s, cache, 32), "k", "shape")
    raises(L, lambda: go(k, k, s.long(), cache, 32), "slots", "dtype")
    raises(L, lambda: go(k, k, _i(4), cache, 32), "slots", "shape")
    raises(L, lambda: go(k, k, s, _i(3, 3, 320), 32), "cache", "shape")
    raises(L, lambda: go(k, k, s, cache, 64), "cache", "words")
    raises(L, lambda: go(k, k, s, cache.float(), 32), "cache", "dtype")
    raises(L, lambda: go(k, k, s, cache, 32, rotary=rot), "together")
    raises(L, lambda: go(k, k, s, cache, 32, positions=pos), "together")
    raises(L, lambda: go(k, k, s, cache, 32, rotary=_f(9, 66), positions=pos), "rotary")
    raises(L, lambda: go(k, k, s, cache, 32, rotary=_f(9, 7), positions=pos), "rotary")
    raises(L, lambda: go(k, k, s, cache, 32, rotary=rot, positions=_i(6)), "positions")
    raises(L, lambda: go(k, k, s, cache, 32, q=_bf(5, 4, 32)), "q", "shape")
    raises(L, lambda: go(k, k, s, cache, 32, q=_f(5, 4, 64)), "q", "dtype")
    raises(L, lambda: go(_bf(5, 64, 2).transpose(1, 2), k, s, cache, 32), "k", "contiguous")
    raises(L, lambda: go(k, k, s, cache, 32), "GPU")
    raises(L, lambda: L.kv4_read(s.long(), cache, 64, 32), "slots", "dtype")
    raises(L, lambda: L.kv4_read(s, cache, 128, 32), "cache")
    raises(L, lambda: L.kv4_read(s, cache, 64, 32, out_dtype=torch.float16), "out_dtype")
    raises(L, lambda: L.kv4_read(s, cache, 64, 32), "GPU")


def test_attention_binding(L):
    cache = L.kv4_cache(3, 2, 64, 32, page=16, device="cpu")
    q, table, lengths = _bf(4, 1, 4, 64), _i(4, 2), _i(4)
    go = L.kv4_attention
    raises(L, lambda: go(None, cache, table, lengths, 32), "q")
    raises(L, lambda: go(q.half(), cache, table, lengths, 32), "q", "dtype")
    raises(L, lambda: go(_bf(4, 4, 64), cache, table, lengths, 32), "q", "shape")
    raises(L, lambda: go(_bf(4, 1, 3, 64), cache, table, lengths, 32), "heads")
    raises(L, lambda: go(_bf(3, 1, 4, 64), cache, table, lengths, 32), "sequences")
    raises(L, lambda: go(q, cache, table.long(), lengths, 32), "table", "dtype")
    raises(L, lambda: go(q, cache, _i(4, 0), lengths, 32), "table")
    raises(L, lambda: go(q, cache, table, _i(3), 32), "lengths", "shape")
    raises(L, lambda: go(q, cache, table, lengths, 64), "cache", "words")
    raises(L, lambda: go(q.view(4, 4, 64), cache, table, lengths, 32, offsets=_i(4)), "offsets", "shape")
    raises(L, lambda: go(q, cache, table, lengths, 32, offsets=_i(5)), "q", "shape")
    raises(L, lambda: go(q, cache, table, lengths, 32, out_dtype=torch.float16), "out_dtype")
    raises(L, lambda: go(q, cache, table, lengths, 32, out=_bf(4, 1, 4, 32)), "out", "shape")
    raises(L, lambda: go(q, cache, table, lengths, 32, out=_f(4, 1, 4, 64)), "out", "dtype")
    raises(L, lambda: go(_bf(5000, 1, 4, 64), cache, _i(5000, 2), _i(5000), 32), "range")
    raises(L, lambda: go(_bf(4, 1, 64, 4).transpose(2, 3), cache, table, lengths, 32), "contiguous")
    raises(L, lambda: go(q, cache, table, lengths, 32), "GPU")


def test_verify_binding(L):
    t, d = _f(2, 4, 10), _f(2, 3, 10)
    tok, u = torch.zeros((2, 3), dtype=torch.int64), _f(2, 4)
    go = L.verify_draft
    raises(L, lambda: go(t.double(), tok, u), "target", "dtype")
    raises(L, lambda: go(t[0], tok, u), "target", "shape")
    raises(L, lambda: go(t[:, :1], tok[:, :0], u[:, :1]), "target", "rows")
    raises(L, lambda: go(_f(2, 34, 10), torch.zeros((2, 33), dtype=torch.int64), _f(2, 34)), "target", "rows")
    raises(L, lambda: go(_f(2, 4, 0), tok, u), "target")
    raises(L, lambda: go(t, tok.int(), u), "tokens", "dtype")
    raises(L, lambda: go(t, tok[:, :2], u), "tokens", "shape")
    raises(L, lambda: go(t, tok, u[:, :3]), "uniform", "shape")
    raises(L, lambda: go(t, tok, u.double()), "uniform", "dtype")
    raises(L, lambda: go(t, tok, u, draft=t), "draft", "shape")
    raises(L, lambda: go(t, tok, u, draft=d.bfloat16()), "draft", "dtype")
    raises(L, lambda: go(_f(2, 10, 4).transpose(1, 2), tok, u), "target", "contiguous")
    raises(L, lambda: go(t, tok, u, draft=_f(2, 1, 10).expand(2, 3, 10)), "draft", "overlap")
    for temp in (0, -1.0, float("nan"), float("inf")):
        raises(L, lambda: go(t, tok, u, temperature=temp), "temperature")
    raises(L, lambda: go(t, tok, u, draft=d), "GPU")


def test_outputs_over_inputs_are_refused_on_the_gpu_only_after_types(L):
    # an output given over an input: named once all are on a GPU (see the GPU tests); types come first
    cache = L.kv4_cache(3, 2, 64, 32, page=16, device="cpu")
    q = _bf(4, 1, 4, 64)
    raises(L, lambda: L.kv4_attention(q, cache, _i(4, 2), _i(4), 32, out=q), "GPU")

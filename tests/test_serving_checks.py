"""The serving calls reject bad arguments on the host: the C ABI by status
code, the binding by an error naming the argument (CPU only: nothing is
enqueued, no pointer is dereferenced)."""
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


def test_pack4_words(lib):
    assert lib.slim_pack4_words(1, 4096, 4096, 128) == 256 * 32 * 288
    assert lib.slim_pack4_words(3, 17, 96, 32) == 3 * 2 * 1 * 384
    assert lib.slim_pack4_words(0, 16, 128, 128) == 0
    for bad in ((1, 16, 100, 128), (1, 16, 128, 48), (-1, 16, 128, 128), (1025, 16, 128, 128), (1, -1, 128, 128),
                (1, (1 << 20) + 1, 128, 128), (1, 16, 0, 128), (1, 16, 65536 + 128, 128)):
        assert lib.slim_pack4_words(*bad) == -1


def test_pack4_abi(lib):
    def call(**kw):
        return lib.slim_pack4(kw.get("c", FAKE), kw.get("s", FAKE), kw.get("z", FAKE), kw.get("e", 1), kw.get("n", 16),
                              kw.get("m", 128), kw.get("g", 128), kw.get("p", FAKE), None, None)
    assert call(c=None) == -1 and call(s=None) == -1 and call(z=None) == -1 and call(p=None) == -1
    assert call(m=96) == -2 and call(g=16) == -2 and call(n=-1) == -2 and call(e=2000) == -2
    assert call(c=ODD) == -7 and call(p=ODD) == -7
    assert call(n=0, c=None) == 0 and call(e=0, c=None) == 0


def test_q4_linear_abi(lib):
    def call(**kw):
        return lib.slim_q4_linear(kw.get("X", FAKE), kw.get("xdt", 1), kw.get("t", 4), kw.get("m", 256),
                                  kw.get("W", FAKE), kw.get("n", 64), kw.get("g", 128), kw.get("Y", FAKE),
                                  kw.get("ydt", 1), kw.get("ws", FAKE), kw.get("wsb", 1 << 40), None)
    assert call(X=None) == -1 and call(W=None) == -1 and call(Y=None) == -1
    assert call(xdt=2) == -3 and call(ydt=-1) == -3
    assert call(t=-1) == -2 and call(t=65537) == -2 and call(m=200) == -2 and call(n=0) == -2 and call(g=256) == -2
    assert call(n=(1 << 20) + 1) == -2
    assert call(X=ODD) == -7 and call(W=ODD) == -7
    assert call(Y=ctypes.c_void_p(4097)) == -7 and call(ydt=0, Y=ctypes.c_void_p(4098)) == -7
    assert call(t=0, X=None, Y=None) == 0
    need = lib.slim_q4_linear_workspace(2048, 4096, 4096, 128, 1)
    assert need > 0
    if need:
        assert call(t=2048, n=4096, m=4096, wsb=need - 1) == -5
        assert call(t=2048, n=4096, m=4096, ws=None) == -5
    assert lib.slim_q4_linear_workspace(-1, 4096, 4096, 128, 1) == 0


def test_q4_experts_abi(lib):
    def call(**kw):
        return lib.slim_q4_experts(kw.get("X", FAKE), kw.get("xdt", 1), kw.get("tx", 8), kw.get("m", 256),
                                   kw.get("rows", FAKE), None, kw.get("r", 16), kw.get("off", FAKE), kw.get("e", 4),
                                   kw.get("W", FAKE), kw.get("n", 64), kw.get("g", 128), kw.get("Y", FAKE),
                                   kw.get("ydt", 0), FAKE, 1 << 40, None)
    assert call(X=None) == -1 and call(off=None) == -1 and call(W=None) == -1 and call(Y=None) == -1
    assert call(xdt=5) == -3 and call(ydt=5) == -3
    assert call(e=0) == -2 and call(e=1025) == -2 and call(r=-1) == -2 and call(r=(1 << 20) + 1) == -2
    assert call(tx=0) == -2 and call(rows=None) == -2        # no gather: as many rows of X as of Y
    assert call(m=250) == -2 and call(n=0) == -2
    assert call(X=ODD) == -7
    assert call(r=0, tx=0, X=None) == 0


def test_token_logprobs_abi(lib):
    def call(**kw):
        return lib.slim_token_logprobs(kw.get("L", FAKE), kw.get("ldt", 0), kw.get("t", 4), kw.get("v", 100),
                                       kw.get("ld", 100), kw.get("ids", FAKE), kw.get("top", 5), kw.get("lp", FAKE),
                                       None, kw.get("tl", FAKE), kw.get("ti", FAKE), kw.get("ws", FAKE),
                                       kw.get("wsb", 1 << 40), None)
    assert call(L=None) == -1 and call(ids=None) == -1 and call(tl=None) == -1 and call(ti=None) == -1
    assert call(ldt=9) == -3
    assert call(v=0) == -2 and call(ld=99) == -2 and call(t=-1) == -2 and call(v=(1 << 24) + 1, ld=1 << 25) == -2
    assert call(top=-1) == -4 and call(top=65) == -4 and call(v=3, ld=3, top=4) == -4
    assert call(L=ctypes.c_void_p(4098)) == -7
    assert call(t=0, L=None) == 0
    need = lib.slim_token_logprobs_workspace(1, 131072, 20)
    assert need > 0
    assert call(t=1, v=131072, ld=131072, top=20, wsb=need - 1) == -5
    assert call(t=1, v=131072, ld=131072, top=20, ws=None) == -5
    assert call(t=1, v=131072, ld=131072, top=20, ws=ODD) == -7
    assert lib.slim_token_logprobs_workspace(1, 3, 4) == 0


def _u8(*s):
    return torch.zeros(s, dtype=torch.uint8)


def _f(*s):
    return torch.zeros(s)


def _i(*s):
    return torch.zeros(s, dtype=torch.int32)


def _bf(*s):
    return torch.zeros(s, dtype=torch.bfloat16)


def test_pack4_binding(L):
    raises(L, lambda: L.pack4(_f(16, 128), _f(16, 1), _f(16, 1), 128), "codes", "dtype")
    raises(L, lambda: L.pack4(_u8(128), _f(1), _f(1), 128), "codes")
    raises(L, lambda: L.pack4(_u8(16, 100), _f(16, 1), _f(16, 1), 128), "group")
    raises(L, lambda: L.pack4(_u8(16, 128), _f(16, 2), _f(16, 1), 128), "scale", "shape")
    raises(L, lambda: L.pack4(_u8(2, 16, 128), _f(2, 16, 1), _f(16, 1), 128), "zero", "shape")
    raises(L, lambda: L.pack4(_u8(16, 128), _f(16, 1), _f(16, 1), 128, info=_f(1)), "info", "dtype")
    raises(L, lambda: L.pack4(_u8(16, 128), _f(16, 1), _f(16, 1), 128), "GPU")


def test_q4_binding(L):
    W = _i(288)
    raises(L, lambda: L.q4_linear(torch.zeros((2, 128), dtype=torch.float16), W, 16, 128), "X", "dtype")
    raises(L, lambda: L.q4_linear(_bf(2, 128), _i(287), 16, 128), "packed", "shape")
    raises(L, lambda: L.q4_linear(_bf(2, 128), W, 17, 128), "packed", "shape")
    raises(L, lambda: L.q4_linear(_bf(2, 128), W, 0, 128), "shape")
    raises(L, lambda: L.q4_linear(_bf(2, 128), W, 16, 128, out_dtype=torch.float16), "out_dtype")
    raises(L, lambda: L.q4_linear(_bf(2, 128), W, 16, 128, Y=_f(2, 17)), "Y", "shape")
    raises(L, lambda: L.q4_linear(_bf(2, 128), W, 16, 128, out_dtype=torch.bfloat16, Y=_f(2, 16)), "Y", "dtype")
    raises(L, lambda: L.q4_linear(_bf(2, 128), W, 16, 128), "GPU")
    raises(L, lambda: L.q4_experts(_bf(2, 128), torch.zeros(2, dtype=torch.int64), W, 16, 128), "offsets", "dtype")
    raises(L, lambda: L.q4_experts(_bf(2, 128), _i(1), W, 16, 128), "offsets")
    raises(L, lambda: L.q4_experts(_bf(2, 128), _i(3), W, 16, 128), "packed", "shape")
    raises(L, lambda: L.q4_experts(_bf(2, 128), _i(2), W, 16, 128, rows=_f(3)), "rows", "dtype")
    raises(L, lambda: L.q4_experts(_bf(2, 128), _i(2), W, 16, 128, rows=_i(3), row_scale=_f(2)), "row_scale", "shape")
    raises(L, lambda: L.q4_experts(_bf(0, 128), _i(2), W, 16, 128, rows=_i(3)), "X")
    raises(L, lambda: L.q4_experts(_bf(2, 128), _i(2), W, 16, 128), "GPU")


def test_token_logprobs_binding(L):
    ids = torch.zeros(3, dtype=torch.int64)
    raises(L, lambda: L.token_logprobs(torch.zeros((3, 8), dtype=torch.float64), ids), "logits", "dtype")
    raises(L, lambda: L.token_logprobs(_f(3, 8), ids[:2]), "ids", "shape")
    raises(L, lambda: L.token_logprobs(_f(3, 8), ids.int()), "ids", "dtype")
    raises(L, lambda: L.token_logprobs(_f(3, 8), ids, top=9), "top")
    raises(L, lambda: L.token_logprobs(_f(3, 100), ids, top=65), "top")
    raises(L, lambda: L.token_logprobs(_f(3, 0), ids), "entries")
    raises(L, lambda: L.token_logprobs(_f(8, 3).t(), ids), "contiguous")
    raises(L, lambda: L.token_logprobs(_f(1, 8).expand(3, 8), ids), "overlap")
    raises(L, lambda: L.token_logprobs(_f(3, 8), ids), "GPU")


def test_layer_paths(L):
    import post_mixed_precision_amd as slim
    raises(L, lambda: slim.quantize_layer(_bf(8, 256), _bf(8, 256), avg_bits=4, nibbles=True), "nibbles")
    ids = torch.zeros(4, dtype=torch.int64)
    raises(L, lambda: slim.score_tokens(_bf(3, 128), ids, _i(288), 16, 128), "ids")
    raises(L, lambda: slim.score_tokens(_bf(4, 128), ids, _i(288), 16, 128, block=0), "block")
    raises(L, lambda: slim.score_tokens(_bf(4, 128), ids, _i(287), 16, 128), "packed")


def test_workspace_sizes_of_extreme_shapes(lib):
    # no rows, one row, the most rows, experts and outputs: sizes that fit what they describe
    assert lib.slim_q4_linear_workspace(0, 4096, 4096, 128, 1) == 0
    assert lib.slim_q4_experts_workspace(0, 0, 8, 4096, 4096, 128, 1) == 0
    assert lib.slim_q4_experts_workspace(5, 0, 1024, 1 << 20, 65536, 32, 0) == 0
    for xdt in (0, 1):
        assert lib.slim_q4_linear_workspace(1, 1, 32, 32, xdt) == 0
        assert lib.slim_q4_experts_workspace(1, 1, 1024, 1, 32, 32, xdt) == 0
        for e in (1, 7, 1024):
            for tx, r in ((1, 1), (1 << 20, 1), (1, 1 << 20), (1 << 20, 1 << 20)):
                for n in (1, 1 << 20):
                    need = lib.slim_q4_experts_workspace(tx, r, e, n, 65536, 32, xdt)
                    rows = min(tx, r)
                    assert need == 0 or need >= rows * (65536 // 32) * 4
                    assert need < 1 << 48


# ------------------------------------------------------------------ how far X reaches
# The tile kernel reads gathered rows by 32-bit offsets from X's first row, or, where they would
# not reach the last row, from a copy of the gathered rows in their order (compact).  What it
# reads is a row of m bfloat16 values in place, of whole records where m does not end with one
# (then always a copy), or of three bfloat16 planes.
REACH = 0xfff00000


def _up(v, k):
    return -(-v // k)


def _row_bytes(m, xdt):
    return 768 * _up(m, 128) if xdt == 0 else 2 * m if m % 128 == 0 else 256 * _up(m, 128)


def _tile_bytes(nrow, m, g, xdt, copy):
    sums = _up(nrow * _up(m, 128) * (128 // g) * 4, 16) * 16
    return sums + (nrow * 256 * _up(m, 128) * (3 if xdt == 0 else 1) if copy else 0)


@pytest.mark.parametrize("m,g,xdt", [(4128, 32, 1), (2112, 64, 1), (65504, 32, 1), (4096, 128, 1), (8192, 32, 1),
                                     (4096, 128, 0), (2016, 32, 0), (65536, 64, 0)])
def test_gather_workspace_around_32_bit_reach(lib, m, g, xdt):
    # more rows of Y than X has, so that the size tells a compact workspace (r rows) from X's own tx rows
    r, e, n = 1 << 20, 8, 1024
    last = (REACH - 1) // _row_bytes(m, xdt)             # the most rows of X within reach
    assert last < r
    for tx in (last - 1, last, last + 1, last + 2, (1 << 32) // _row_bytes(m, xdt)):
        near = tx * _row_bytes(m, xdt) < REACH
        assert near == (tx <= last)
        need = lib.slim_q4_experts_workspace(tx, r, e, n, m, g, xdt)
        copy = xdt == 0 or m % 128 != 0 or not near
        assert need == _tile_bytes(tx if near else r, m, g, xdt, copy), (tx, need)


def test_workspace_of_far_rows_in_order(lib):
    # without a gather a tile's rows lie together, so that X of any size is read in place
    t, m = 65536, 32768
    assert t * _row_bytes(m, 1) >= REACH
    assert lib.slim_q4_linear_workspace(t, 4096, m, 128, 1) == _tile_bytes(t, m, 128, 1, False)
    for m in (32768 + 32, 65536 - 64):                   # but for rows that end inside a record
        assert lib.slim_q4_linear_workspace(t, 4096, m, 32, 1) == _tile_bytes(t, m, 32, 1, True)
    assert lib.slim_q4_linear_workspace(t, 4096, m, 32, 0) == _tile_bytes(t, m, 32, 0, True)


def test_outputs_over_inputs_are_refused(L):
    X, W = _f(16, 128), _i(288)
    raises(L, lambda: L.q4_linear(X[:, :].view(16, 128), _i(288 * 8), 128, 128, Y=X), "Y", "overlaps X")
    raises(L, lambda: L.q4_linear(X[:4], _i(288 * 8), 128, 128, Y=X[3:7]), "Y", "overlaps X")
    raises(L, lambda: L.q4_linear(X[:4], _i(288 * 8), 128, 128, Y=X[4:8]), "GPU")        # side by side
    raises(L, lambda: L.q4_linear(X[4:], _i(288 * 8), 128, 128, Y=X[:12]), "Y", "overlaps X")
    raises(L, lambda: L.q4_linear(_f(2, 128), W, 16, 128, Y=W[:32].view(torch.float32).view(2, 16)), "Y", "packed")
    off, gates = _i(2), _f(32)
    raises(L, lambda: L.q4_experts(X[:2], off, _i(288 * 8), 128, 128, Y=X[1:3]), "Y", "overlaps X")
    raises(L, lambda: L.q4_experts(X[:2], off, W, 16, 128, row_scale=gates[:2], Y=gates.view(2, 16)), "Y", "row_scale")
    raises(L, lambda: L.q4_experts(_f(0, 128), off, W, 16, 128, Y=_f(0, 16)), "GPU")     # nothing overlaps nothing


def test_score_tokens_refuses_before_it_allocates(L):
    import post_mixed_precision_amd as slim
    X, ids, W = _bf(4, 128), torch.zeros(4, dtype=torch.int64), _i(288)
    for n in (-1, 0, 1 << 50, (1 << 20) + 1):
        raises(L, lambda: slim.score_tokens(X, ids, W, n, 128, block=2), "layer shape")
        raises(L, lambda: slim.score_tokens(X, ids, W, n, 128), "layer shape")
    raises(L, lambda: slim.score_tokens(X, ids, W, 17, 128, block=2), "packed")
    raises(L, lambda: slim.score_tokens(X, ids, W, 16, 100, block=2), "group")
    raises(L, lambda: slim.score_tokens(X, ids, W, 16, 128, top=17, block=2), "top")
    raises(L, lambda: slim.score_tokens(X, ids, W, 16, 128, top=-1, block=2), "top")
    # a million outputs by 65536 rows: no buffer of that size is made for tensors that are not on a GPU
    words = L.load_library().slim_pack4_words(1, 1 << 20, 32, 32)
    big = torch.zeros(1, dtype=torch.int32).expand(words)
    raises(L, lambda: slim.score_tokens(_bf(70000, 32), torch.zeros(70000, dtype=torch.int64), big, 1 << 20, 32,
                                        block=65536), "GPU")

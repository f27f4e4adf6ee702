"""The rules by which the 4-bit products choose a kernel, its shape and its
workspace (csrc/q4_plan.hpp, plain C++), on the CPU: what they choose has a
GPU case, the GPU cases run on the kernel they are written for, and sizes hold
what the kernels read and write."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

pytest.importorskip("torch")
import test_gpu_serving as gpu  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "post_mixed_precision_amd", "csrc")
CXX = shutil.which("g++") or shutil.which("c++")
LIB = os.path.join(ROOT, "post_mixed_precision_amd", "libslim.so")
REACH = 0xfff00000          # bytes that 32-bit offsets may span

SOURCE = """
#include "q4_plan.hpp"
using namespace slim;
extern "C" void choose(int64_t r, int64_t e, int64_t n, int64_t m, int g, int xbf16, int *out) {
  out[0] = use_tiles(r, e, n, m, xbf16);
  if (out[0]) {
    out[1] = narrow_tiles(r, e, n), out[2] = column_parts(r, e, n, m);
  } else {
    const StreamShape s = stream_shape(r, e, n, m, g, xbf16);
    out[1] = s.blocks, out[2] = s.tiles, out[3] = s.waves, out[4] = s.records, out[5] = s.ahead;
  }
}
extern "C" void sizes(int64_t tx, int64_t r, int64_t e, int64_t n, int64_t m, int g, int xbf16, int gather,
                      int64_t *out) {
  const TileWs w = tile_ws(tx, r, e, n, m, g, xbf16, gather);
  out[0] = w.compact, out[1] = w.copy, out[2] = w.parts, out[3] = w.nrow;
  out[4] = w.planes, out[5] = w.partial, out[6] = w.bytes;
}
extern "C" int64_t most_tiles(int64_t r, int64_t e, int64_t tok) { return max_tiles(r, e, tok); }
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    if CXX is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("plan")
    src, so = d / "plan.cpp", d / "plan.so"
    src.write_text(SOURCE)
    r = subprocess.run([CXX, "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC, str(src), "-o",
                        str(so)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    lib = ctypes.CDLL(str(so))
    i64 = ctypes.c_int64
    lib.choose.argtypes = [i64] * 4 + [ctypes.c_int] * 2 + [ctypes.POINTER(ctypes.c_int)]
    lib.sizes.argtypes = [i64] * 5 + [ctypes.c_int] * 3 + [ctypes.POINTER(i64)]
    lib.most_tiles.argtypes, lib.most_tiles.restype = [i64] * 3, i64
    return lib


def choose(plan, r, e, n, m, g, xdt):
    """The kernel as GPU cases name it: "tile 128x256", with " split 3" where the columns are, or
    "stream 4x1x16x1": row blocks x row tiles x waves x records, with " ahead"."""
    out = (ctypes.c_int * 6)()
    plan.choose(r, e, n, m, g, xdt == "bf16", out)
    if out[0]:
        return ("tile 64x512" if out[1] else "tile 128x256") + (f" split {out[2]}" if out[2] > 1 else "")
    return "stream " + "x".join(map(str, out[1:5])) + (" ahead" if out[5] else "")


def sizes(plan, tx, r, e, n, m, g, xdt, gather):
    out = (ctypes.c_int64 * 7)()
    plan.sizes(tx, r, e, n, m, g, xdt == "bf16", gather, out)
    return dict(zip(("compact", "copy", "parts", "nrow", "planes", "partial", "bytes"), out))


def _shapes(count, seed=0):
    """Layers and rows over the whole documented range, what fits a card more often."""
    rng = random.Random(seed)

    def logint(lo, hi):
        return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))
    for _ in range(count):
        big = rng.random() < 0.2
        g = rng.choice((32, 64, 128))
        m = g * logint(1, (65536 if big else 14336) // g)
        n = logint(1, 1 << 20 if big else 32768)
        e = 1 if rng.random() < 0.5 else logint(1, 1024 if big else 64)
        r = logint(1, 1 << 20 if big else 8192)
        yield r, e, n, m, g, rng.choice(("bf16", "f32"))


def test_gpu_cases_run_on_the_kernel_they_name(plan):
    for kernel, t, n, m, g, xdt, ydt in gpu.LINEAR_KERNELS:
        assert choose(plan, t, 1, n, m, g, xdt) == kernel, (t, n, m, g, xdt)
    for kernel, counts, n, m, g, xdt, ydt, gather, weighted, before, behind in gpu.EXPERT_KERNELS:
        r = before + sum(counts) + behind
        assert choose(plan, r, len(counts), n, m, g, xdt) == kernel, (r, len(counts), n, m, g, xdt)


def test_every_kernel_that_can_be_chosen_has_a_gpu_case(plan):
    def keys(r, e, n, m, g, xdt):
        """What is compiled for it, and over how many workgroups its columns are split."""
        kernel, _, parts = choose(plan, r, e, n, m, g, xdt).partition(" split ")
        return {(kernel, g, xdt, bool(parts)), ("parts", parts, xdt)}
    have = set()
    for t, n, m, g, xdt, _ in [*gpu.LINEAR, *(c[1:] for c in gpu.LINEAR_KERNELS)]:
        have |= keys(t, 1, n, m, g, xdt)
    for counts, n, m, g, xdt, _, _, _, before, behind in [*gpu.EXPERTS, *(c[1:] for c in gpu.EXPERT_KERNELS)]:
        have |= keys(before + sum(counts) + behind, len(counts), n, m, g, xdt)
    for shape in _shapes(40000):
        assert keys(*shape) <= have, (keys(*shape) - have, shape)


def test_32_bit_offsets_reach_all_gathered_rows(plan):
    def row(m, xdt):                # bytes of a row of X as the tile kernel reads it
        return 768 * -(-m // 128) if xdt == "f32" else 2 * m if m % 128 == 0 else 256 * -(-m // 128)
    rng = random.Random(1)
    seen = set()
    for r, e, n, m, g, xdt in _shapes(4000, 2):
        last = min((REACH - 1) // row(m, xdt), 1 << 20)      # the most rows within reach
        for tx in {max(1, min(1 << 20, last + d)) for d in (-1, 0, 1, 1000)} | {rng.randint(1, 1 << 20), r}:
            w = sizes(plan, tx, r, e, n, m, g, xdt, 1)
            if not w["compact"]:
                assert tx * row(m, xdt) < REACH and w["nrow"] == tx
                assert tx * -(-m // 128) * (128 // g) * 4 < REACH      # nor do the group sums pass it
            else:
                assert w["nrow"] == r and (r < tx or tx * row(m, xdt) >= REACH)
            # rows gathered from too far are copied in their order; float32 X always is, as planes
            assert w["copy"] == (xdt == "bf16" and (m % 128 != 0 or tx * row(m, xdt) >= REACH))
            seen.add((xdt, m % 128 == 0, w["compact"], r == tx))
            if tx == r:                                       # without a gather: X is read where it is
                o = sizes(plan, tx, r, e, n, m, g, xdt, 0)
                assert not o["compact"] and o["nrow"] == r and o["copy"] == (xdt == "bf16" and m % 128 != 0)
                assert o["bytes"] <= w["bytes"] and o["parts"] == w["parts"]
    for xdt in ("bf16", "f32"):
        for whole in (False, True):
            for compact in (False, True):
                for same in (False, True):
                    # as many rows as X has pass 2^32 bytes only if wide and many
                    assert (xdt, whole, compact, same) in seen, (xdt, whole, compact, same)


def test_workspace_holds_what_the_tile_kernel_keeps(plan):
    for r, e, n, m, g, xdt in _shapes(4000, 3):
        for tx, gather in ((r, 0), (r, 1), (max(1, r // 2), 1), (min(1 << 20, 3 * r), 1)):
            w = sizes(plan, tx, r, e, n, m, g, xdt, gather)
            nch = -(-m // 128)
            assert w["planes"] % 16 == 0 and w["partial"] % 16 == 0
            assert w["planes"] >= w["nrow"] * nch * (128 // g) * 4                     # group sums
            planes = 3 if xdt == "f32" else 1 if w["copy"] else 0
            assert w["partial"] - w["planes"] == w["nrow"] * planes * nch * 256        # X's planes, or its copy
            partial = w["parts"] * r * n * 4 if w["parts"] > 1 else 0
            assert w["bytes"] - w["partial"] == partial
            assert 1 <= w["parts"] <= max(1, min(4, nch // 4))                         # four records at least to each


def test_tiles_of_ragged_ranges_fit_the_grid(plan):
    rng = random.Random(4)
    for _ in range(3000):
        e = rng.randint(1, 40)
        counts = [rng.choice((0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, rng.randint(0, 700))) for _ in range(e)]
        r = sum(counts) + rng.choice((0, 0, 5))
        if r:
            for tok in (16, 32, 64, 128):
                assert sum(-(-c // tok) for c in counts) <= plan.most_tiles(r, e, tok)
                assert -(-r // tok) <= plan.most_tiles(r, e, tok)       # bounds out of order: the plain row range


@pytest.mark.skipif(not os.path.exists(LIB), reason="libslim.so not built (run __graft_entry__.build())")
def test_library_asks_for_these_sizes(plan):
    import post_mixed_precision_amd as slim
    lib = slim.load_library()
    for r, e, n, m, g, xdt in _shapes(2000, 5):
        bf = xdt == "bf16"
        tile = choose(plan, r, e, n, m, g, xdt).startswith("tile")
        for tx in (r, max(1, r // 3), min(1 << 20, 2 * r)):
            want = sizes(plan, tx, r, e, n, m, g, xdt, 1)["bytes"] if tile else 0
            assert lib.slim_q4_experts_workspace(tx, r, e, n, m, g, bf) == want
        if e == 1 and r <= 65536:
            want = sizes(plan, r, r, 1, n, m, g, xdt, 0)["bytes"] if tile else 0
            assert lib.slim_q4_linear_workspace(r, n, m, g, bf) == want

"""The rules by which attention over the 4-bit cache is cut (csrc/kv4_plan.hpp, plain C++), on the CPU: the GPU cases
run on the kernel they are written for, the runs that a wave works out from the lengths stay within what the host
provided for, and workspaces hold them."""
import ctypes
import os
import random
import shutil
import subprocess

import numpy as np
import pytest

pytest.importorskip("torch")
import test_gpu_decode as gpu  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "post_mixed_precision_amd", "csrc")
CXX = shutil.which("g++") or shutil.which("c++")

SOURCE = """
#include "kv4_plan.hpp"
using namespace slim;
extern "C" void plan(int64_t b, int64_t tq, int uniform, int64_t hq, int64_t hkv, int dim, int group, int64_t cap,
                     int f32, int64_t *out) {
  const Kv4Plan p = kv4_plan(b, tq, uniform, hq, hkv, dim, group, cap, f32);
  out[0] = p.tile, out[1] = p.nq, out[2] = p.tm, out[3] = p.tiles, out[4] = p.slots, out[5] = p.extra;
  out[6] = p.least, out[7] = p.most, out[8] = p.ws_bytes;
}
extern "C" int64_t words(int page, int dim, int group) {
  return kv4_shape(page, dim, group) ? kv4_page_words(page, dim, group) : -1;
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    if CXX is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("plan")
    src, so = d / "plan.cpp", d / "plan.so"
    src.write_text(SOURCE)
    r = subprocess.run([CXX, "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC, str(src), "-o",
                        str(so)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    lib = ctypes.CDLL(str(so))
    i64, i = ctypes.c_int64, ctypes.c_int
    lib.plan.argtypes = [i64, i64, i, i64, i64, i, i, i64, i, ctypes.POINTER(i64)]
    lib.words.argtypes, lib.words.restype = [i, i, i], i64
    return lib


def plan(lib, b, tq, uniform, hq, hkv, dim, group, cap, f32):
    out = (ctypes.c_int64 * 9)()
    lib.plan(b, tq, uniform, hq, hkv, dim, group, cap, f32, out)
    return dict(zip(("tile", "nq", "tm", "tiles", "slots", "extra", "least", "most", "ws"), out))


def runs(p, rows, lengths):
    """What find_work makes of the lengths: (first run, runs) of every tile, in order."""
    f = np.float32
    tiles = [-(-r // p["tm"]) for r in rows]
    t32 = [-(-max(n, 0) // 32) for n in lengths]
    chunk = 1 << 26
    if p["extra"]:
        work = f(0)
        for n, t in zip(tiles, t32):
            work += f(n) * f(t)
        for more in (sum(tiles), sum(tiles) // 2, 0) if len(rows) <= 64 else (0,):
            share = work * f(1.01) / f(p["extra"] + more)
            chunk = p["least"] if share < p["least"] else int(min(share, f(1 << 26))) + 1
            if sum(n * max(1, -(-t // chunk)) for n, t in zip(tiles, t32)) <= p["slots"] + p["extra"]:
                break
    out, first = [], 0
    for n, t in zip(tiles, t32):
        r = 1 if t <= chunk else -(-t // chunk)
        for _ in range(n):
            out.append((first, r))
            first += r
    return out, first


def test_words(lib):
    assert lib.words(16, 64, 32) == 4 * 64 + 64
    assert lib.words(256, 256, 32) == 16 * (1024 + 256)
    for bad in ((8, 64, 32), (48, 64, 32), (512, 64, 32), (16, 96, 32), (16, 64, 128), (16, 64, 16), (0, 64, 32)):
        assert lib.words(*bad) == -1


def test_every_kernel_has_a_gpu_case(lib):
    seen = set()
    for lengths, n, hq, heads, dim, group, page, qdt, odt, _ in gpu.ATTENTION + gpu.EVERY + gpu.JOINED:
        cap = max(1, max(-(-x // page) for x in lengths)) * page
        p = plan(lib, len(lengths), len(lengths) * n, 1, hq, heads, dim, group, cap, "f32" in (qdt, odt))
        seen.add((dim, group, "mixed" if (qdt, odt) == ("bf16", "f32") else qdt, p["tile"], p["nq"]))
        seen.add(("joined", p["extra"] > 0, p["most"] > 8))
    assert ("joined", True, True) in seen and ("joined", True, False) in seen and ("joined", False, False) in seen
    for dim in (64, 128, 256):
        for group in (32, 64, 128):
            if group > dim:
                continue
            for qdt in ("bf16", "f32", "mixed"):
                kinds = {s[3:] for s in seen if s[:3] == (dim, group, qdt)}
                wide = qdt == "bf16" and dim < 256
                want = {(0, 1), (1, 2 if wide and dim // group < 4 else 1)} | ({(0, 2)} if wide else set())
                assert kinds >= want, (dim, group, qdt, kinds)


def test_runs_stay_within_what_there_is(lib):
    rng = random.Random(5)
    for _ in range(1500):
        b = rng.choice([1, 2, 7, 64, 65, 200, 1024, 1500])
        hkv = rng.choice([1, 2, 8, 32])
        hq = hkv * rng.choice([1, 3, 8, 16])
        dim = rng.choice([64, 128, 256])
        group = rng.choice([g for g in (32, 64, 128) if g <= dim])
        uniform = rng.random() < 0.5
        cap = 16 * rng.choice([1, 4, 100, 1000, 60000])
        if uniform:
            counts = [rng.choice([1, 1, 2, 9, 300])] * b
        else:
            counts = [rng.choice([0, 1, 1, 2, 500]) for _ in range(b)]
        tq = sum(counts)
        if tq == 0 or tq > 1 << 20:
            continue
        lengths = [rng.choice([0, 1, cap // 3, cap, cap, rng.randint(0, cap), -5]) for _ in range(b)]
        if rng.random() < 0.3:
            lengths = [min(100, cap)] * (b - 1) + [cap]          # one long among short ones
        p = plan(lib, b, tq + (0 if uniform else rng.randint(0, 5)), uniform, hq, hkv, dim, group, cap, rng.random() < 0.5)
        rows = [c * (hq // hkv) for c in counts]
        tiles = sum(-(-r // p["tm"]) for r in rows)
        assert tiles <= p["slots"]
        if uniform:
            assert tiles == p["slots"] and all(-(-r // p["tm"]) == p["tiles"] for r in rows)
        made, last = runs(p, rows, lengths)
        assert last <= p["slots"] + p["extra"]
        if p["extra"]:
            need = ((p["slots"] + p["extra"]) * hkv * p["tm"] * (dim + 2) * 4 + p["slots"] * 32)
            assert p["ws"] >= need
            assert last * hkv < 1 << 24
        else:
            assert p["ws"] == 0 and all(r == 1 for _, r in made)


def test_one_long_sequence_is_spread(lib):
    # 64 sequences of 100 tokens and one of 131072, 8 heads: its tokens over many workgroups
    p = plan(lib, 65, 65, 1, 64, 8, 128, 128, 131072, 0)
    made, _ = runs(p, [8] * 65, [100] * 64 + [131072])
    assert made[-1][1] >= 16 and all(r == 1 for _, r in made[:-1])

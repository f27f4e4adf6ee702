"""The 4-bit products (one matrix, or one per expert) and the token log
probabilities against the float64 oracle, through the binding.

Tolerances, from the arithmetic.  Products: X and the codes enter exactly, so
an output's error comes from the float32 sums: at most g (3 g for float32 X,
which enters as three terms) additions inside a group, k over the groups and a
handful in joining partial sums, each off by at most 2^-23 of a partial sum
that never exceeds sum_c |x_c| (q_c + |z|) s.  A bfloat16 output adds half a
step, 2^-8 of the value.  Log probabilities: see _lp_bounds.
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


def _layer(seed, e, n, m, g):
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 16, size=(e, n, m), dtype=np.uint8)
    scale = rng.uniform(1e-3, 1e-2, size=(e, n, m // g)).astype(np.float32)
    zero = rng.uniform(0, 15, size=(e, n, m // g)).astype(np.float32)
    return codes, scale, zero


def _x(seed, t, m, dt):
    x = torch.from_numpy(np.random.default_rng(seed).standard_normal((t, m)).astype(np.float32))
    return x.to(DT[dt])


def _gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda:0")


def _bound(x, codes, scale, zero, g, xdt, ydt, exact):
    k = codes.shape[-1] // g
    mag = np.abs(x) @ ((codes + np.repeat(np.abs(zero), g, -1)) * np.repeat(np.abs(scale), g, -1)).astype(np.float64).T
    terms = (g if xdt == "bf16" else 3 * g) + k + 24
    return 2.0 ** -23 * terms * mag + (2.0 ** -8 * np.abs(exact) if ydt == "bf16" else 0) + 1e-30


@pytest.mark.parametrize("e,n,m,g", [(1, 16, 128, 128), (1, 1, 32, 32), (3, 37, 96, 32), (2, 130, 320, 64),
                                     (1, 256, 1152, 128)])
def test_pack4_layout(slim, e, n, m, g):
    print(f"pack4 e={e} n={n} m={m} g={g}", flush=True)
    codes, scale, zero = _layer(n, e, n, m, g)
    want = oracle.pack4(codes, scale, zero, g)
    info = torch.zeros(1, dtype=torch.int32, device="cuda:0")
    got = slim.pack4(_gpu(codes), _gpu(scale), _gpu(zero), g, info=info)
    np.testing.assert_array_equal(got.cpu().numpy().view(np.uint32), want)
    assert info.item() == 0
    if e == 1:
        got = slim.pack4(_gpu(codes[0]), _gpu(scale[0]), _gpu(zero[0]), g)
        np.testing.assert_array_equal(got.cpu().numpy().view(np.uint32), want)
    codes[0, n - 1, m - 1] |= 0x40                          # above 15: flagged, low bits kept
    got = slim.pack4(_gpu(codes), _gpu(scale), _gpu(zero), g, info=info)
    np.testing.assert_array_equal(got.cpu().numpy().view(np.uint32), want)
    assert info.item() == 1


# Sizes of all kinds.  The headings say what the cases were written for; the choice of kernel has moved
# some of them since, and LINEAR_KERNELS and EXPERT_KERNELS below name the kernel that runs.
LINEAR = [
    (1, 16, 128, 128, "bf16", "f32"),
    (1, 1, 32, 32, "f32", "bf16"),           # one output, a quarter of a record
    (1, 1000, 2048, 128, "bf16", "bf16"),
    (2, 257, 320, 64, "bf16", "f32"),        # half a record at the end of the row
    (4, 130, 96, 32, "f32", "f32"),
    (5, 48, 1088, 64, "bf16", "bf16"),
    (8, 100, 4224, 128, "f32", "f32"),
    (9, 31, 160, 32, "bf16", "f32"),
    (16, 513, 384, 128, "bf16", "bf16"),
    (17, 64, 256, 64, "bf16", "f32"),
    (33, 200, 416, 32, "f32", "bf16"),
    (48, 1040, 640, 128, "bf16", "f32"),
    (64, 129, 192, 64, "bf16", "bf16"),
    (65, 300, 512, 128, "bf16", "f32"),
    (100, 520, 224, 32, "bf16", "bf16"),
    (128, 256, 256, 128, "f32", "f32"),
    (129, 272, 2112, 64, "bf16", "f32"),
    (300, 1003, 1056, 32, "bf16", "bf16"),
    (257, 385, 1152, 128, "f32", "bf16"),
    (700, 640, 640, 128, "bf16", "f32"),
    # enough rows and outputs for the tile kernel: 3, 4, 5, 6, 7 stages
    (1537, 2100, 384, 128, "bf16", "f32"),
    (1700, 1800, 512, 64, "bf16", "bf16"),
    (1600, 2048, 640, 32, "bf16", "f32"),
    (1300, 2570, 768, 128, "bf16", "bf16"),
    (1410, 2310, 576, 64, "bf16", "f32"),     # a row that ends inside a record: X is copied
    (3000, 1033, 800, 32, "bf16", "bf16"),
    (1290, 2320, 384, 128, "f32", "f32"),     # float32 X: three planes
    (1665, 1793, 288, 32, "f32", "bf16"),
    (2049, 1500, 320, 64, "f32", "f32"),
    # and its columns split over two, three and four workgroups
    (500, 2600, 1024, 128, "bf16", "bf16"),
    (700, 3000, 1536, 64, "bf16", "f32"),
    (400, 2500, 2080, 32, "bf16", "bf16"),
    (385, 2309, 1152, 128, "f32", "f32"),
    # tiles of 64 rows by 512 outputs: 255 of them for 261 of 128 by 256
    (1088, 7300, 384, 128, "bf16", "bf16"),
    (1085, 7200, 576, 64, "bf16", "f32"),
    (1088, 7300, 416, 32, "bf16", "f32"),
    (1030, 7425, 640, 128, "f32", "f32"),
    (1088, 7171, 288, 32, "f32", "bf16"),
    # one and two stages
    (2000, 2100, 128, 128, "bf16", "bf16"),
    (2000, 2100, 96, 32, "f32", "f32"),
    (1900, 2300, 256, 64, "bf16", "f32"),
    (1700, 2200, 192, 64, "bf16", "bf16"),
    (1600, 7000, 160, 32, "bf16", "bf16"),
    # columns split over two, three and four workgroups
    (1000, 4096, 2048, 128, "bf16", "bf16"),
    (600, 4000, 4128, 32, "bf16", "f32"),
    (640, 2400, 6080, 64, "bf16", "bf16"),
    (640, 2411, 6144, 128, "bf16", "f32"),
    (484, 4873, 1920, 128, "f32", "f32"),
    # few rows of a long and wide matrix, in tiles with the columns split, and streamed
    (64, 7000, 8192, 128, "bf16", "bf16"),
    (30, 6200, 384, 128, "bf16", "f32"),
    (33, 12300, 640, 64, "bf16", "bf16"),
    (5, 20500, 1408, 32, "bf16", "f32"),
    (40, 12400, 416, 32, "bf16", "f32"),
    (18, 10300, 1184, 32, "f32", "bf16"),
    (1, 20480, 2176, 128, "bf16", "f32"),
    (1, 13000, 2304, 64, "f32", "f32"),
    # streaming, 32 rows at a time
    (64, 25000, 128, 128, "bf16", "bf16"),
    (100, 13000, 96, 32, "f32", "f32"),
]


@pytest.mark.parametrize("t,n,m,g,xdt,ydt", LINEAR)
def test_q4_linear(slim, t, n, m, g, xdt, ydt):
    print(f"q4_linear t={t} n={n} m={m} g={g} {xdt} -> {ydt}", flush=True)
    codes, scale, zero = _layer(t + n + m, 1, n, m, g)
    X = _x(t * n, t, m, xdt)
    packed = slim.pack4(_gpu(codes), _gpu(scale), _gpu(zero), g)
    Y = torch.full((t + 1, n), 7.0, dtype=DT[ydt], device="cuda:0")
    out = slim.q4_linear(X.to("cuda:0"), packed, n, g, out_dtype=DT[ydt], Y=Y[:t])
    assert out.data_ptr() == Y.data_ptr()
    assert torch.all(Y[t] == 7.0)                           # the row behind the last is left alone
    again = slim.q4_linear(X.to("cuda:0"), packed, n, g, out_dtype=DT[ydt])
    assert torch.equal(again, out)                          # a fixed order of sums
    x = X.double().numpy()
    exact = x @ oracle.q4_weight(codes[0], scale[0], zero[0], g).T
    err = np.abs(out.double().cpu().numpy() - exact)
    bound = _bound(x, codes[0], scale[0], zero[0], g, xdt, ydt, exact)
    assert np.all(err <= bound), float(np.max(err / bound))


def test_q4_linear_scales_and_zeros_of_any_sign(slim):
    # negative, zero and huge scales, zeros far outside the code range
    n, m, g, t = 40, 256, 64, 3
    codes, scale, zero = _layer(5, 1, n, m, g)
    scale[0, ::3] *= -1
    scale[0, 1::3] = 0
    scale[0, 2] = 1e6
    zero[0, ::2] = -40.0
    X = _x(6, t, m, "f32")
    Y = slim.q4_linear(X.to("cuda:0"), slim.pack4(_gpu(codes), _gpu(scale), _gpu(zero), g), n, g)
    x = X.double().numpy()
    exact = x @ oracle.q4_weight(codes[0], scale[0], zero[0], g).T
    err = np.abs(Y.double().cpu().numpy() - exact)
    assert np.all(err <= _bound(x, codes[0], scale[0], zero[0], g, "f32", "f32", exact))


@pytest.mark.parametrize("t,n,m,g", [(3, 48, 256, 128), (40, 48, 96, 32), (200, 48, 256, 128), (1500, 2100, 384, 128),
                                     (1500, 2100, 320, 64), (500, 2600, 1024, 128), (1088, 7300, 384, 128),
                                     (640, 2400, 6144, 128)])
def test_q4_linear_nonfinite_row_stays_in_its_row(slim, t, n, m, g):
    codes, scale, zero = _layer(7, 1, n, m, g)
    X = _x(8, t, m, "bf16").to("cuda:0")
    packed = slim.pack4(_gpu(codes), _gpu(scale), _gpu(zero), g)
    clean = slim.q4_linear(X, packed, n, g)
    X[1, 5] = float("nan")
    X[2, 9] = float("inf")
    Y = slim.q4_linear(X, packed, n, g)
    assert not torch.isfinite(Y[1:3]).any()
    keep = [a for a in range(t) if a not in (1, 2)]
    assert torch.equal(Y[keep], clean[keep])


def test_q4_linear_no_tokens(slim):
    codes, scale, zero = _layer(9, 1, 16, 128, 128)
    packed = slim.pack4(_gpu(codes), _gpu(scale), _gpu(zero), 128)
    assert slim.q4_linear(torch.empty((0, 128), device="cuda:0"), packed, 16, 128).shape == (0, 16)


def test_q4_linear_agrees_with_the_planes(slim):
    # the same 3-bit-average layer through both layouts
    n, m, g, t = 96, 512, 128, 7
    rng = np.random.default_rng(10)
    bits = np.array([2, 3, 4, 3], dtype=np.int8)
    codes = np.concatenate([rng.integers(0, 2 ** b, size=(n, g), dtype=np.uint8) for b in bits], axis=1)
    scale = rng.uniform(1e-3, 1e-2, size=(n, 4)).astype(np.float32)
    zero = rng.uniform(0, 3, size=(n, 4)).astype(np.float32)
    X = _x(11, t, m, "bf16").to("cuda:0")
    planes, info = slim.pack(_gpu(codes), _gpu(bits), g, 3)
    a = slim.qlinear(X, planes, _gpu(bits), _gpu(scale), _gpu(zero), g, 3).double().cpu().numpy()
    b = slim.q4_linear(X, slim.pack4(_gpu(codes), _gpu(scale), _gpu(zero), g), n, g).double().cpu().numpy()
    x = X.double().cpu().numpy()
    bound = _bound(x, codes, scale, zero, g, "bf16", "f32", b)
    assert np.all(np.abs(a - b) <= 2 * bound)


# ------------------------------------------------------------------ experts
def _counts_to_offsets(counts, first=0):
    return np.concatenate([[first], first + np.cumsum(counts)]).astype(np.int32)


EXPERTS = [
    # counts, n, m, g, xdt, ydt, gather, weighted, rows before and behind
    ([1], 16, 128, 128, "bf16", "f32", False, False, 0, 0),
    ([2, 0, 1, 1], 100, 256, 64, "bf16", "bf16", True, True, 0, 0),
    ([0, 0, 5, 0], 33, 96, 32, "f32", "f32", False, True, 2, 3),
    ([17, 1, 0, 40, 16], 200, 384, 128, "bf16", "f32", True, False, 1, 1),
    ([300, 0, 7, 65], 130, 320, 64, "bf16", "bf16", True, True, 0, 5),
    ([129, 128, 127, 0, 260], 272, 640, 128, "bf16", "f32", False, False, 3, 0),
    ([200, 90], 96, 160, 32, "f32", "bf16", True, True, 0, 0),
    ([1] * 65, 16, 128, 128, "bf16", "f32", True, False, 0, 0),      # more experts than lanes
    ([3, 0] * 75, 24, 64, 64, "bf16", "bf16", False, True, 0, 1),
    ([0, 0, 0], 16, 128, 128, "bf16", "f32", False, False, 0, 4),    # no rows at all
    ([700, 500, 0, 900], 300, 256, 128, "bf16", "bf16", True, False, 0, 0),
    # the tile kernel
    ([700, 500, 0, 900], 1600, 384, 128, "bf16", "bf16", True, False, 0, 0),
    ([129, 0, 1, 1400, 128, 0, 300], 1700, 320, 64, "bf16", "f32", False, True, 5, 7),
    ([900, 333, 700], 1610, 640, 32, "bf16", "bf16", True, True, 0, 130),
    ([400, 0, 1100, 513], 1550, 288, 32, "f32", "f32", True, True, 1, 0),
    ([1000, 1000], 1540, 512, 128, "f32", "bf16", False, False, 0, 3),
    # with tiles of 64 rows by 512 outputs
    ([66] * 30 + [0, 132] * 17, 1000, 320, 64, "bf16", "bf16", True, True, 0, 0),
    ([1400, 1332, 1300], 2000, 640, 32, "bf16", "bf16", False, True, 0, 0),
    ([1, 2630, 1397], 1800, 384, 128, "bf16", "f32", True, False, 1, 3),
    ([64, 2567, 1400], 2048, 288, 32, "f32", "f32", True, True, 1, 0),
    ([1000, 0, 3032], 1793, 512, 128, "f32", "bf16", False, False, 0, 0),
    ([1600, 1500, 2200], 1450, 384, 128, "bf16", "f32", True, True, 0, 0),
    ([2100, 1, 3199], 1400, 352, 32, "bf16", "bf16", False, True, 0, 0),
    ([5000, 150, 147], 1500, 320, 64, "f32", "bf16", True, False, 1, 2),
    ([1750, 1850, 1700], 1290, 288, 32, "f32", "f32", False, False, 0, 0),
    # experts of some 50 rows, streamed 32 rows at a time, and of some 40, long enough for tiles
    ([50, 0, 90, 33, 64, 45, 61, 57], 1100, 256, 64, "bf16", "bf16", True, True, 0, 0),
    ([40, 64, 0, 65, 3, 30, 70, 48], 5700, 2048, 128, "bf16", "bf16", True, True, 0, 0),
    ([41, 0, 20, 77], 4200, 2112, 64, "bf16", "f32", False, False, 0, 1),
    # with its columns split
    ([300, 0, 7, 200], 2600, 1024, 128, "bf16", "bf16", True, True, 2, 9),
    ([0, 290, 410], 2100, 1216, 64, "f32", "f32", False, True, 3, 1),
    ([300, 0, 7, 200], 4100, 6144, 128, "bf16", "bf16", True, True, 2, 9),
    ([0, 380, 380], 4000, 4160, 64, "f32", "f32", False, True, 3, 1),
]


@pytest.mark.parametrize("counts,n,m,g,xdt,ydt,gather,weighted,before,behind", EXPERTS)
def test_q4_experts(slim, counts, n, m, g, xdt, ydt, gather, weighted, before, behind):
    e, r = len(counts), before + sum(counts) + behind
    print(f"q4_experts e={e} r={r} n={n} m={m} g={g} {xdt} -> {ydt} gather={gather} weighted={weighted}", flush=True)
    rng = np.random.default_rng(r + n)
    off = _counts_to_offsets(counts, before)
    codes, scale, zero = _layer(r + m, e, n, m, g)
    tx = max(1, r // 2) if gather else r
    rows = rng.integers(0, tx, size=r).astype(np.int32) if gather else None
    gates = rng.uniform(-1, 1, size=r).astype(np.float32) if weighted else None
    X = _x(r, tx, m, xdt)
    packed = slim.pack4(_gpu(codes), _gpu(scale), _gpu(zero), g)
    Y = torch.full((r, n), 7.0, dtype=DT[ydt], device="cuda:0")
    slim.q4_experts(X.to("cuda:0"), _gpu(off), packed, n, g, rows=None if rows is None else _gpu(rows),
                    row_scale=None if gates is None else _gpu(gates), out_dtype=DT[ydt], Y=Y)
    y = Y.double().cpu().numpy()
    assert np.all(y[:before] == 7.0) and np.all(y[off[-1]:] == 7.0)
    x = X.double().numpy()
    for j in range(e):
        a, b = off[j], off[j + 1]
        if a == b:
            continue
        xs = x[a:b] if rows is None else x[rows[a:b]]
        w = np.ones(b - a) if gates is None else gates[a:b].astype(np.float64)
        exact = (xs @ oracle.q4_weight(codes[j], scale[j], zero[j], g).T) * w[:, None]
        bound = _bound(xs * np.abs(w)[:, None], codes[j], scale[j], zero[j], g, xdt, ydt, exact)
        bound += 2.0 ** -24 * np.abs(exact)                 # the product with the row's factor
        err = np.abs(y[a:b] - exact)
        assert np.all(err <= bound), (j, float(np.max(err / bound)))


@pytest.mark.parametrize("per,n,m,xdt", [(3, 32, 128, "bf16"), (150, 32, 128, "f32"), (700, 1600, 384, "bf16"),
                                         (700, 1600, 384, "f32"), (200, 2600, 1024, "bf16"),
                                         (1344, 2000, 384, "bf16"), (1344, 2000, 384, "f32"),
                                         (1768, 1400, 384, "bf16"), (1768, 1400, 384, "f32"),
                                         (200, 4100, 6144, "bf16")])
def test_q4_experts_bad_rows_and_offsets(slim, per, n, m, xdt):
    # checked by the kernels before anything is read through them
    e, g = 3, 128
    r = e * per
    codes, scale, zero = _layer(12, e, n, m, g)
    packed = slim.pack4(_gpu(codes), _gpu(scale), _gpu(zero), g)
    X = _x(13, 4, m, xdt).to("cuda:0")
    rows = np.arange(r, dtype=np.int32) % 4
    off = _counts_to_offsets([per] * e)
    good = slim.q4_experts(X, _gpu(off), packed, n, g, rows=_gpu(rows))
    assert torch.isfinite(good).all()
    bad = rows.copy()
    bad[1], bad[r - 1] = -1, 4
    Y = slim.q4_experts(X, _gpu(off), packed, n, g, rows=_gpu(bad))
    assert torch.isnan(Y[1]).all() and torch.isnan(Y[r - 1]).all()
    keep = [a for a in range(r) if a not in (1, r - 1)]
    assert torch.equal(Y[keep], good[keep])
    for bounds in ([0, per, per - 1, r], [0, per, 2 * per, r + 1], [-1, per, 2 * per, r],
                   [0, 2 ** 31 - 1, -2 ** 31, r]):
        Y = slim.q4_experts(X, _gpu(np.array(bounds, dtype=np.int32)), packed, n, g, rows=_gpu(rows))
        assert torch.isnan(Y).all(), bounds


@pytest.mark.parametrize("tx,n,m,g,xdt", [(5000, 1600, 384, 128, "bf16"), (3000, 1700, 320, 64, "bf16"),
                                          (2500, 1600, 288, 32, "f32"), (3000, 2600, 1024, 128, "f32"),
                                          (900, 40, 96, 32, "bf16"), (5000, 9000, 384, 128, "bf16"),
                                          (3000, 9000, 320, 64, "bf16"), (2500, 9000, 288, 32, "f32"),
                                          (3000, 4000, 4096, 128, "f32")])
def test_q4_experts_gather_of_few_rows(slim, tx, n, m, g, xdt):
    # X has more rows than are asked for, some of them twice
    e, counts = 2, [400, 300]
    r = sum(counts)
    codes, scale, zero = _layer(70, e, n, m, g)
    rows = np.random.default_rng(71).integers(0, tx, size=r).astype(np.int32)
    rows[:3] = rows[5], 0, tx - 1
    X = _x(72, tx, m, xdt)
    Y = slim.q4_experts(X.to("cuda:0"), _gpu(_counts_to_offsets(counts)),
                        slim.pack4(_gpu(codes), _gpu(scale), _gpu(zero), g), n, g, rows=_gpu(rows))
    x = X.double().numpy()[rows]
    for j, (a, b) in enumerate(((0, counts[0]), (counts[0], r))):
        exact = x[a:b] @ oracle.q4_weight(codes[j], scale[j], zero[j], g).T
        err = np.abs(Y[a:b].double().cpu().numpy() - exact)
        bound = _bound(x[a:b], codes[j], scale[j], zero[j], g, xdt, "f32", exact)
        assert np.all(err <= bound), float(np.max(err / bound))


def test_q4_experts_gather_over_4_gib(slim):
    # rows of X further apart than a 32-bit offset, in the tile kernel; the same rows in order agree
    tx, n, m, g, r = 40000, 9216, 65536, 128, 128
    X = torch.zeros((tx, m), dtype=torch.bfloat16, device="cuda:0")
    rows = torch.cat([torch.arange(64), torch.arange(tx - 64, tx)]).to(torch.int32).to("cuda:0")
    gen = torch.Generator(device="cuda:0")
    gen.manual_seed(80)
    X[:64] = torch.randn((64, m), generator=gen, device="cuda:0")
    X[tx - 64:] = torch.randn((64, m), generator=gen, device="cuda:0")
    codes = torch.randint(0, 16, (1, n, m), generator=gen, device="cuda:0").to(torch.uint8)
    scale = torch.rand((1, n, m // g), generator=gen, device="cuda:0") * 0.01
    zero = 7.5 + torch.rand((1, n, m // g), generator=gen, device="cuda:0")
    packed = slim.pack4(codes, scale, zero, g)
    off = torch.tensor([0, r], dtype=torch.int32, device="cuda:0")
    lib = slim.load_library()
    assert lib.slim_q4_experts_workspace(tx, r, 1, n, m, g, 1) > 2 * r * m      # the copy of the gathered rows
    Y = slim.q4_experts(X, off, packed, n, g, rows=rows)
    one = slim.q4_linear(X[rows.long()].contiguous(), packed, n, g)
    torch.testing.assert_close(Y, one, rtol=1e-4, atol=1e-3)


@pytest.mark.parametrize("tx,n,m,g", [(32768, 256, 65504, 32), (520000, 200, 4128, 32)])
def test_q4_experts_gather_with_a_copy_over_4_gib(slim, tx, n, m, g):
    # X itself is within a 32-bit offset, its copy with rows padded to whole records is not
    print(f"q4_experts gather tx=r={tx} n={n} m={m} g={g}", flush=True)
    nch = -(-m // 128)
    assert 2 * m * tx < 0xfff00000 < 1 << 32 <= 256 * nch * tx
    lib = slim.load_library()
    assert lib.slim_q4_experts_workspace(tx, tx, 2, n, m, g, 1) >= 256 * nch * tx    # the tile kernel, with the copy
    gen = torch.Generator(device="cuda:0")
    gen.manual_seed(81)
    X = torch.randn((tx, m), generator=gen, device="cuda:0", dtype=torch.bfloat16)
    codes, scale, zero = _layer(82, 2, n, m, g)
    packed = slim.pack4(_gpu(codes), _gpu(scale), _gpu(zero), g)
    rows = torch.randperm(tx, generator=gen, device="cuda:0").to(torch.int32)
    wrap = min((1 << 32) // (256 * nch), tx - 1)             # rows on both sides of where an offset would wrap
    rows[:5] = torch.tensor([0, 1, tx - 1, wrap - 1, wrap], device="cuda:0")
    cut = tx // 2 + 3
    Y = slim.q4_experts(X, torch.tensor([0, cut, tx], dtype=torch.int32, device="cuda:0"), packed, n, g, rows=rows)
    at = torch.cat([torch.arange(24), torch.arange(cut - 4, cut + 4), torch.arange(tx - 24, tx)]).to("cuda:0")
    x = X[rows[at].long()].double().cpu().numpy()
    y, at = Y[at].double().cpu().numpy(), at.cpu().numpy()
    for j in range(2):
        mine = (at >= cut) == (j == 1)
        exact = x[mine] @ oracle.q4_weight(codes[j], scale[j], zero[j], g).T
        bound = _bound(x[mine], codes[j], scale[j], zero[j], g, "bf16", "f32", exact)
        err = np.abs(y[mine] - exact)
        assert np.all(err <= bound), float(np.max(err / bound))


@pytest.mark.parametrize("t,n,m,g", [(65536, 200, 32896, 128), (33400, 256, 64480, 32)])
def test_rows_in_order_over_4_gib(slim, t, n, m, g):
    # no gather: the tile kernel reads X where it is (or a copy with padded rows), past 32-bit offsets
    print(f"q4_linear t={t} n={n} m={m} g={g}", flush=True)
    assert 2 * m * t >= 1 << 32
    copy = 0 if m % 128 == 0 else t * -(-m // 128) * 256
    lib = slim.load_library()
    assert copy < lib.slim_q4_linear_workspace(t, n, m, g, 1) < copy + 2 * m * t
    gen = torch.Generator(device="cuda:0")
    gen.manual_seed(83)
    X = torch.randn((t, m), generator=gen, device="cuda:0", dtype=torch.bfloat16)
    codes, scale, zero = _layer(84, 1, n, m, g)
    packed = slim.pack4(_gpu(codes), _gpu(scale), _gpu(zero), g)
    wrap = min((1 << 32) // (2 * m), t - 2)
    at = torch.tensor([0, 1, 127, 128, wrap - 1, wrap, wrap + 1, t - 2, t - 1], device="cuda:0")
    Y = slim.q4_linear(X, packed, n, g)
    off = torch.tensor([5, t], dtype=torch.int32, device="cuda:0")
    E = slim.q4_experts(X, off, packed, n, g, Y=torch.full((t, n), 7.0, device="cuda:0"))
    assert torch.all(E[:5] == 7.0)
    x = X[at].double().cpu().numpy()
    exact = x @ oracle.q4_weight(codes[0], scale[0], zero[0], g).T
    bound = _bound(x, codes[0], scale[0], zero[0], g, "bf16", "f32", exact)
    assert np.all(np.abs(Y[at].double().cpu().numpy() - exact) <= bound)
    assert np.all(np.abs(E[at].double().cpu().numpy() - exact)[2:] <= bound[2:])


def test_q4_experts_matches_single_layers(slim):
    e, n, m, g = 4, 160, 512, 128
    codes, scale, zero = _layer(14, e, n, m, g)
    counts = [5, 0, 30, 1]
    off = _counts_to_offsets(counts)
    X = _x(15, sum(counts), m, "bf16").to("cuda:0")
    Y = slim.q4_experts(X, _gpu(off), slim.pack4(_gpu(codes), _gpu(scale), _gpu(zero), g), n, g)
    for j in range(e):
        a, b = int(off[j]), int(off[j + 1])
        if a < b:
            one = slim.q4_linear(X[a:b].contiguous(), slim.pack4(_gpu(codes[j]), _gpu(scale[j]), _gpu(zero[j]), g), n, g)
            torch.testing.assert_close(Y[a:b], one, rtol=1e-4, atol=1e-4)


# ------------------------------------------------------------------ every kernel that can be chosen
# What runs is chosen by estimates from the sizes; each case names the kernel it is for (row blocks x
# row tiles x waves x records; rows x outputs), which test_serving_plan.py holds against the rules.
LINEAR_KERNELS = [
    # 16 waves: a batch of 16 (and less) through a wide layer, and many rows through a small one
    ("stream 4x1x16x1", 16, 12400, 2240, 64, "bf16", "bf16"),
    ("stream 4x1x16x1", 3, 12900, 2144, 32, "bf16", "f32"),
    ("stream 4x1x16x1", 530, 337, 2176, 128, "bf16", "f32"),
    ("stream 4x1x16x1", 400, 475, 2208, 32, "f32", "bf16"),
    ("stream 4x1x16x1", 61, 3100, 2304, 128, "f32", "f32"),
    ("stream 4x1x16x1", 16, 12400, 2112, 64, "f32", "f32"),
    # two row blocks
    ("stream 2x1x8x2", 16, 5000, 2080, 32, "bf16", "f32"),
    ("stream 2x1x8x2", 40, 1650, 320, 64, "bf16", "bf16"),
    ("stream 2x1x8x2", 12, 5001, 1152, 128, "bf16", "f32"),
    ("stream 2x1x8x2", 7, 4700, 416, 32, "f32", "bf16"),
    ("stream 2x1x8x2", 33, 1700, 1088, 64, "f32", "f32"),
    # one
    ("stream 1x1x8x2", 5, 300, 1984, 64, "f32", "f32"),
    # four, a record ahead
    ("stream 4x1x4x1 ahead", 9, 12700, 1088, 64, "bf16", "bf16"),
    ("stream 4x1x4x1 ahead", 30, 7000, 960, 64, "f32", "bf16"),
    ("stream 4x1x4x1 ahead", 100, 4000, 1920, 128, "f32", "bf16"),
    # by 8 waves
    ("stream 4x1x8x1", 100, 4000, 2048, 128, "f32", "f32"),
    ("stream 4x1x8x1", 17, 10300, 2432, 128, "f32", "bf16"),
    # tiles that few rows leave part empty
    ("tile 128x256 split 4", 127, 13492, 3392, 64, "bf16", "f32"),
    ("tile 128x256 split 4", 100, 14716, 2016, 32, "f32", "bf16"),
    ("tile 128x256", 123, 15004, 32, 32, "bf16", "bf16"),
    # columns split over two, three and four workgroups
    ("tile 128x256 split 2", 2521, 1490, 1280, 128, "bf16", "f32"),
    ("tile 128x256 split 3", 1066, 2255, 2208, 32, "bf16", "bf16"),
    ("tile 128x256 split 2", 2243, 1310, 992, 32, "f32", "f32"),
    ("tile 128x256 split 3", 2185, 988, 1472, 32, "f32", "bf16"),
    ("tile 128x256 split 4", 1179, 1504, 1984, 64, "f32", "f32"),
    ("tile 64x512", 1034, 7235, 320, 64, "f32", "f32"),
]


@pytest.mark.parametrize("kernel,t,n,m,g,xdt,ydt", LINEAR_KERNELS)
def test_q4_linear_of_every_kernel(slim, kernel, t, n, m, g, xdt, ydt):
    need = slim.load_library().slim_q4_linear_workspace(t, n, m, g, xdt == "bf16")
    assert (need > 0) == kernel.startswith("tile")
    test_q4_linear(slim, t, n, m, g, xdt, ydt)


_FEW = [5, 0, 1, 3, 0, 2, 4, 1]
EXPERT_KERNELS = [
    ("stream 1x1x8x2", [2, 0, 3], 100, 224, 32, "bf16", "bf16", True, False, 1, 0),
    ("stream 1x1x8x2", [2, 0, 3], 100, 192, 64, "f32", "f32", False, True, 0, 2),
    ("stream 1x1x8x2", [18, 1, 30], 70, 2304, 128, "f32", "f32", True, True, 0, 0),
    ("stream 2x1x8x2", _FEW, 700, 2080, 32, "bf16", "f32", True, True, 0, 0),
    ("stream 2x1x8x2", _FEW, 690, 1152, 128, "bf16", "bf16", False, True, 0, 0),
    ("stream 2x1x8x2", _FEW, 705, 288, 32, "f32", "f32", True, False, 0, 0),
    ("stream 2x1x8x2", _FEW, 700, 960, 64, "f32", "bf16", False, False, 0, 0),
    ("stream 2x1x8x2", _FEW, 700, 2432, 128, "f32", "f32", True, True, 0, 0),
    ("stream 4x1x16x1", _FEW, 1700, 2144, 32, "bf16", "bf16", True, True, 0, 0),
    ("stream 4x1x16x1", _FEW, 1690, 2240, 64, "bf16", "f32", False, True, 0, 0),
    ("stream 4x1x16x1", _FEW, 1700, 2432, 128, "bf16", "bf16", True, False, 0, 0),
    ("stream 4x1x16x1", _FEW, 1710, 2336, 32, "f32", "f32", False, False, 0, 0),
    ("stream 4x1x16x1", _FEW, 1700, 2112, 64, "f32", "bf16", True, True, 0, 0),
    ("stream 4x1x16x1", _FEW, 1700, 2176, 128, "f32", "f32", True, True, 0, 0),
    ("stream 4x1x4x1 ahead", _FEW, 1700, 1952, 32, "bf16", "f32", True, True, 0, 0),
    ("stream 4x1x4x1 ahead", [20, 40, 0, 17, 33], 1900, 608, 32, "f32", "bf16", True, False, 1, 1),
    ("stream 4x1x4x1 ahead", _FEW, 1700, 1152, 128, "f32", "f32", False, True, 0, 0),
    ("stream 4x1x8x1", [40, 3, 0, 50, 20, 31], 1710, 2432, 128, "f32", "bf16", True, True, 1, 2),
    ("stream 4x2x4x1 ahead", [50, 0, 90, 33, 64, 45, 61, 57], 1100, 224, 32, "bf16", "f32", True, True, 0, 0),
    ("tile 128x256", [900, 0, 517, 1, 700, 599], 1700, 192, 64, "f32", "bf16", True, True, 1, 2),
    ("tile 128x256 split 2", [1000, 795], 1951, 1472, 32, "bf16", "f32", True, False, 0, 3),
    ("tile 128x256 split 3", [600, 743], 1571, 2688, 64, "bf16", "bf16", False, True, 2, 0),
    ("tile 128x256 split 2", [1000, 710], 1761, 992, 32, "f32", "f32", True, True, 0, 0),
    ("tile 128x256 split 4", [1700, 0, 2031], 412, 2560, 128, "f32", "bf16", False, False, 1, 1),
    ("tile 64x512", [30, 0, 1, 60, 3, 20, 64, 7, 8, 9, 10], 6027, 128, 128, "f32", "f32", True, True, 0, 0),
]


@pytest.mark.parametrize("kernel,counts,n,m,g,xdt,ydt,gather,weighted,before,behind", EXPERT_KERNELS)
def test_q4_experts_of_every_kernel(slim, kernel, counts, n, m, g, xdt, ydt, gather, weighted, before, behind):
    r = before + sum(counts) + behind
    need = slim.load_library().slim_q4_experts_workspace(r, r, len(counts), n, m, g, xdt == "bf16")
    assert (need > 0) == kernel.startswith("tile")
    test_q4_experts(slim, counts, n, m, g, xdt, ydt, gather, weighted, before, behind)


# tiles; with planes of float32 X; with a copy of X; columns split
TILED = [(1537, 2100, 384, 128, "bf16"), (1290, 2320, 384, 128, "f32"), (1410, 2310, 576, 64, "bf16"),
         (1066, 2255, 2208, 32, "bf16"), (2243, 1310, 992, 32, "f32")]


@pytest.mark.parametrize("ydt", ["bf16", "f32"])
@pytest.mark.parametrize("t,n,m,g,xdt", TILED)
def test_q4_tiles_to_outputs_that_start_anywhere(slim, t, n, m, g, xdt, ydt):
    print(f"q4_linear t={t} n={n} m={m} g={g} {xdt} -> {ydt}, one element off", flush=True)
    assert slim.load_library().slim_q4_linear_workspace(t, n, m, g, xdt == "bf16") > 0
    codes, scale, zero = _layer(90, 1, n, m, g)
    packed = slim.pack4(_gpu(codes), _gpu(scale), _gpu(zero), g)
    X = _x(91, t, m, xdt).to("cuda:0")
    flat = torch.full((t * n + 3,), 7.0, dtype=DT[ydt], device="cuda:0")
    out = slim.q4_linear(X, packed, n, g, out_dtype=DT[ydt], Y=flat[1:1 + t * n].view(t, n))
    assert torch.equal(out, slim.q4_linear(X, packed, n, g, out_dtype=DT[ydt]))
    assert flat[0] == 7 and torch.all(flat[1 + t * n:] == 7)


@pytest.mark.parametrize("t,n,m,g,xdt", TILED)
def test_tiles_in_two_graphs(slim, t, n, m, g, xdt):
    # each captured call has a workspace of its own (sums, planes or a copy of X, partial sums): replays in
    # any order agree with eager calls between them, also after X has changed
    print(f"graphs of q4_linear and q4_experts t={t} n={n} m={m} g={g} {xdt}", flush=True)
    assert slim.load_library().slim_q4_linear_workspace(t, n, m, g, xdt == "bf16") > 0
    codes, scale, zero = _layer(92, 2, n, m, g)
    packed = slim.pack4(_gpu(codes), _gpu(scale), _gpu(zero), g)
    first = slim.pack4(_gpu(codes[0]), _gpu(scale[0]), _gpu(zero[0]), g)
    X = _x(93, t, m, xdt).to("cuda:0")
    off = torch.tensor([0, t // 3, t], dtype=torch.int32, device="cuda:0")
    rows = torch.arange(t - 1, -1, -1, device="cuda:0").to(torch.int32)

    def calls():
        return slim.q4_linear(X, first, n, g), slim.q4_experts(X, off, packed, n, g, rows=rows)
    eager = calls()
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = calls()
        graphs.append((gr, out))
    for turn, i in enumerate((0, 1, 1, 0, 1)):
        if turn == 2:
            X.neg_()
            off[1] = t // 2
            eager = calls()
        graphs[i][0].replay()
        again = calls()
        torch.cuda.synchronize()
        for a, b, c in zip(graphs[i][1], again, eager):
            assert torch.equal(a, b) and torch.equal(b, c), turn


# ------------------------------------------------------------------ log probabilities
def _lp_bounds(x, out):
    """Float32 error bounds.  d = x - M is off by 2^-24 |d|; e^d by 3 2^-24 (1 +
    |d|) relative (the product with log2 e and the power); a lane adds at most
    V / 64 + 2 terms, the joins some 20 more, each step 2^-24, so ln S is off
    by rS below (entries with |d| > 104 underflow to 0 and S >= 1).  W's terms
    e^d d carry |d| / S <= D on top, and the last operations round once more."""
    eps = 2.0 ** -24
    v = x.shape[1]
    fin = np.where(np.isfinite(x), x, 0.0)
    d = np.minimum(fin.max(axis=1) - fin.min(axis=1), 104.0)
    rs = eps * (v / 64 + 40 + 4 * (1 + d))
    lp = rs + eps * 4 * (1 + np.abs(np.nan_to_num(out["logprob"], neginf=0.0)))
    ent = 2 * rs * (1 + out["entropy"]) + eps * 8 * (1 + np.abs(out["entropy"]) + d)
    return lp, ent, rs


def _check_lp(got, x, ids, top):
    want = oracle.token_logprobs(x, ids, top)
    lp_b, ent_b, rs = _lp_bounds(x, want)
    lp, ent = got["logprob"].double().cpu().numpy(), got["entropy"].double().cpu().numpy()
    for g, w, b in ((lp, want["logprob"], lp_b), (ent, want["entropy"], ent_b)):
        same = (g == w) | (np.isnan(g) & np.isnan(w))
        with np.errstate(invalid="ignore"):
            ok = same | (np.abs(g - w) <= b)
        assert ok.all(), (g[~ok], w[~ok], b[~ok])
    if top:
        np.testing.assert_array_equal(got["top_id"].cpu().numpy(), want["top_id"])
        tl, wl = got["top_logprob"].double().cpu().numpy(), want["top_logprob"]
        same = (tl == wl) | (np.isnan(tl) & np.isnan(wl))
        with np.errstate(invalid="ignore"):
            ok = same | (np.abs(tl - wl) <= rs[:, None] + 2.0 ** -22 * (1 + np.abs(wl)))
        assert ok.all()


def _logits(seed, t, v, pad, off, dt, scale=3.0):
    x = torch.from_numpy((scale * np.random.default_rng(seed).standard_normal((t, off + v + pad))).astype(np.float32))
    x = x.to(DT[dt])
    return x[:, off:off + v]


@pytest.mark.parametrize("t,v,pad,off,dt,top", [
    (1, 1, 0, 0, "f32", 1),
    (1, 7, 0, 0, "bf16", 7),
    (3, 64, 0, 0, "f32", 64),              # the longest list, the whole row
    (5, 100, 1, 0, "f32", 5),              # rows not aligned to 16 bytes
    (4, 255, 3, 1, "bf16", 20),            # the first row neither
    (2, 4097, 0, 0, "f32", 3),             # two segments
    (1, 32000, 0, 0, "bf16", 5),
    (3, 50001, 6, 3, "bf16", 20),          # segments of rows that start anywhere
    (2, 131072, 0, 0, "f32", 64),
    (1500, 501, 0, 0, "f32", 2),           # one segment a row
    (40, 5000, 2, 0, "bf16", 0),
])
def test_token_logprobs(slim, t, v, pad, off, dt, top):
    print(f"token_logprobs t={t} v={v} pad={pad} off={off} {dt} top={top}", flush=True)
    x = _logits(t + v, t, v, pad, off, dt)
    ids = np.random.default_rng(v).integers(0, v, size=t)
    ids[t // 2] = -100 if t > 1 else ids[t // 2]
    whole = _logits(t + v, t, v, pad, off, dt)._base if pad or off else None
    base = (x if whole is None else whole).to("cuda:0")
    g = base if whole is None else base[:, off:off + v]
    got = slim.token_logprobs(g, _gpu(ids), top=top)
    assert ("top_id" in got) == (top > 0)
    _check_lp(got, x.double().numpy(), ids, top)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("v", [300, 9000])
def test_token_logprobs_masked_and_bad_rows(slim, dt, v):
    low = torch.finfo(DT[dt]).min
    x = _logits(3, 12, v, 0, 0, dt).clone()
    inf = float("inf")
    x[0] = -inf                              # nothing left
    x[1] = low                               # everything at the type's lowest value: uniform
    x[2, 1:] = -inf                          # one entry left: certain
    x[3, : v // 2] = -inf
    x[4, ::2] = low
    x[5, v // 3] = float("nan")
    x[6, v - 1] = inf
    x[7] = 0.0                               # ties everywhere
    x[8, :5] = 50.0                          # ties at the top
    x[9] = torch.sort(x[9]).values           # rising: every entry is a new maximum
    x[10, 3:] = -inf                         # fewer entries than asked for
    x[11, 0], x[11, 1] = -0.0, 0.0           # equal, whatever their bits
    x[11, 2:] = -1.0
    ids = np.array([0, v - 1, 0, 0, 0, 0, 0, v, -1, v - 1, 7, 1])
    got = slim.token_logprobs(x.to("cuda:0"), _gpu(ids), top=8)
    _check_lp(got, x.double().numpy(), ids, 8)
    lp = got["logprob"].cpu()
    assert torch.isnan(lp[[0, 5, 6, 7]]).all() and lp[8] == 0 and lp[2] == 0 and lp[3] == -inf
    assert got["top_id"][11, 0].item() == 0


def test_token_logprobs_large_logits(slim):
    # differences that overflow float32, and values near its ends
    x = torch.zeros((3, 600))
    x[0, 0], x[0, 1] = 3.4e38, -3.4e38
    x[1] = -3.0e38
    x[2] = 1e4 + torch.arange(600) * 0.01
    ids = np.array([0, 3, 599])
    got = slim.token_logprobs(x.to("cuda:0"), _gpu(ids), top=2)
    assert got["logprob"][0].item() == 0 and got["entropy"][0].item() == 0
    _check_lp(got, x.double().numpy(), ids, 2)


@pytest.mark.parametrize("t,v,dt,top", [(7, 60000, "f32", 20), (5, 30000, "bf16", 64), (300, 26000, "f32", 5),
                                        (80, 70000, "bf16", 20)])
def test_token_logprobs_thresholds_that_keep_moving(slim, t, v, dt, top):
    # rows in which every wave finds better entries again and again, at its own time
    print(f"token_logprobs t={t} v={v} {dt} top={top}", flush=True)
    j = torch.arange(v, dtype=torch.float64)
    rng = np.random.default_rng(v)
    kinds = [j / v * 9,                                  # rising: the last entries win
             -j / v * 9,                                 # falling: the first do
             (j % 1024) / 100 + j / v,                   # a saw that rises
             torch.floor(j / v * 40),                    # steps of ties
             (j // 1024 % 4 * 7 + j % 1024 / 200) + j / v,   # one wave after another ahead
             torch.from_numpy(3 * rng.standard_normal(v))]
    x = torch.stack([kinds[a % len(kinds)] for a in range(t)]).to(DT[dt])
    ids = rng.integers(0, v, size=t)
    got = slim.token_logprobs(x.to("cuda:0"), _gpu(ids), top=top)
    n = min(t, 2 * len(kinds))                           # rows of a kind are alike: the oracle sorts some
    _check_lp({k: a[:n] for k, a in got.items()}, x[:n].double().numpy(), ids[:n], top)
    for a in range(len(kinds), t):
        assert torch.equal(got["top_id"][a], got["top_id"][a % len(kinds)]), a
        assert torch.equal(got["top_logprob"][a], got["top_logprob"][a % len(kinds)]), a


def test_token_logprobs_no_rows(slim):
    got = slim.token_logprobs(torch.empty((0, 10), device="cuda:0"), torch.empty(0, dtype=torch.int64, device="cuda:0"),
                              top=2)
    assert got["logprob"].shape == (0,) and got["top_id"].shape == (0, 2)


# ------------------------------------------------------------------ together
def test_run_of_the_operators_eager_side_stream_and_graph(slim):
    """A decode step as a server runs it: experts gathered by token and weighted
    by the router's gates, summed over the choices, the head, the scores; eager
    against the float64 chain, then on a side stream and from a replayed graph
    with new inputs in the same buffers."""
    t, d, h, v, e, g, top = 6, 256, 384, 1000, 4, 64, 2
    rng = np.random.default_rng(20)
    up, head = _layer(21, e, h, d, g), _layer(22, 1, v, h, g)
    pu = slim.pack4(*[_gpu(a) for a in up], g)
    ph = slim.pack4(*[_gpu(a) for a in head], g)
    zc = lambda lay: (lay[0].astype(np.float64) - np.repeat(lay[2], g, -1)) * np.repeat(lay[1], g, -1)  # noqa: E731
    wu, wh = zc(up), zc(head)[0]

    def inputs(seed):
        r = np.random.default_rng(seed)
        x = torch.from_numpy(r.standard_normal((t, d)).astype(np.float32)).to(torch.bfloat16)
        picks = sorted((int(j), a) for a in range(t) for j in r.choice(e, size=top, replace=False))
        counts = np.bincount([p[0] for p in picks], minlength=e)
        rows = np.array([p[1] for p in picks], dtype=np.int32)
        gates = r.uniform(0.2, 0.8, size=t * top).astype(np.float32)
        back = np.array([[i for i, p in enumerate(picks) if p[1] == a] for a in range(t)])
        return (x, torch.from_numpy(_counts_to_offsets(counts)), torch.from_numpy(rows), torch.from_numpy(gates),
                torch.from_numpy(back), torch.from_numpy(r.integers(0, v, size=t)))

    def step(x, off, rows, gates, back, ids):
        y = slim.q4_experts(x, off, pu, h, g, rows=rows, row_scale=gates)
        z = y[back].sum(dim=1).to(torch.bfloat16)
        logits = slim.q4_linear(z, ph, v, g)
        return z, logits, slim.token_logprobs(logits, ids, top=5)

    buf = [a.to("cuda:0") for a in inputs(0)]
    z, logits, s = step(*buf)
    x, off, rows, gates, back, ids = [a.double().numpy() if a.dtype == torch.bfloat16 else a.numpy() for a in inputs(0)]
    y = np.zeros((t * top, h))
    for j in range(e):
        for a in range(off[j], off[j + 1]):
            y[a] = wu[j] @ x[rows[a]] * gates[a]
    zr = y[back].sum(axis=1)
    np.testing.assert_allclose(z.double().cpu().numpy(), zr, rtol=2.0 ** -7, atol=1e-3)
    lr = z.double().cpu().numpy() @ wh.T
    np.testing.assert_allclose(logits.double().cpu().numpy(), lr, rtol=1e-4, atol=1e-4 * np.abs(lr).max())
    _check_lp(s, logits.double().cpu().numpy(), ids, 5)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        z2, logits2, s2 = step(*buf)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(logits, logits2) and all(torch.equal(s[k], s2[k]) for k in s)

    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        zg, lg, sg = step(*buf)
    for seed in (1, 2, 3):
        new = inputs(seed)
        for b, a in zip(buf, new):
            b.copy_(a)
        graph.replay()
        torch.cuda.synchronize()
        got = [lg.clone(), {k: sg[k].clone() for k in sg}]
        _, le, se = step(*buf)
        assert torch.equal(got[0], le) and all(torch.equal(got[1][k], se[k]) for k in se), seed


@pytest.mark.parametrize("avg", [2, 3])
def test_quantized_layer_served_and_scored(slim, avg):
    """quantize_layer's codes through both layouts, and the layer as an output
    layer: the scores of its logits, formed in blocks."""
    n, m, g, T = 300, 512, 128, 70
    W = (0.02 * _x(50, n, m, "f32")).to(torch.bfloat16).to("cuda:0")
    X = _x(51, 256, m, "bf16").to("cuda:0")
    q = slim.quantize_layer(X, W, g, avg, nibbles=True)
    assert int(q["info"]) == 0 and int(q["pack_info"]) == 0
    codes, scale, zero = (q[k].cpu().numpy() for k in ("codes", "scale", "zero"))
    Xt = X[:T].contiguous()
    a = slim.qlinear(Xt, q["packed"], q["bits"], q["scale"], q["zero"], g, avg).double().cpu().numpy()
    b = slim.q4_linear(Xt, q["packed4"], n, g)
    x = Xt.double().cpu().numpy()
    exact = x @ oracle.q4_weight(codes, scale, zero, g).T
    bound = _bound(x, codes, scale, zero, g, "bf16", "f32", exact)
    assert np.all(np.abs(b.double().cpu().numpy() - exact) <= bound) and np.all(np.abs(a - exact) <= 2 * bound)
    ids = torch.arange(T, device="cuda:0") * 4
    ids[3] = -1
    whole = slim.score_tokens(Xt, ids, q["packed4"], n, g, top=3)
    _check_lp(whole, b.double().cpu().numpy(), ids.cpu().numpy(), 3)
    cut = slim.score_tokens(Xt, ids, q["packed4"], n, g, top=3, block=32)
    for a0 in range(0, T, 32):                  # a block's product may take another order of sums
        lg = slim.q4_linear(Xt[a0:a0 + 32].contiguous(), q["packed4"], n, g)
        part = {k: v[a0:a0 + 32] for k, v in cut.items()}
        _check_lp(part, lg.double().cpu().numpy(), ids[a0:a0 + 32].cpu().numpy(), 3)


def test_two_graphs_share_inputs(slim):
    # each captured call has its own workspace: replays in any order agree
    n, m, g, t, v = 2600, 1024, 128, 500, 40000
    codes, scale, zero = _layer(30, 1, n, m, g)
    packed = slim.pack4(_gpu(codes), _gpu(scale), _gpu(zero), g)
    X = _x(31, t, m, "f32").to("cuda:0")
    L = _logits(32, 3, v, 0, 0, "f32").to("cuda:0")
    ids = torch.tensor([1, 2, 3], device="cuda:0")
    want = slim.q4_linear(X, packed, n, g), slim.token_logprobs(L, ids, top=4)
    graphs = []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = slim.q4_linear(X, packed, n, g), slim.token_logprobs(L, ids, top=4)
        graphs.append((gr, out))
    for i in (0, 1, 1, 0, 1):
        graphs[i][0].replay()
        torch.cuda.synchronize()
        y, s = graphs[i][1]
        assert torch.equal(y, want[0]) and all(torch.equal(s[k], want[1][k]) for k in s)


def test_most_rows_and_unaligned_outputs(slim):
    # 2^20 rows of 16: more tiles than one grid axis takes; then an output that starts anywhere
    e, n, m, g, r = 2, 16, 32, 32, 1 << 20
    codes, scale, zero = _layer(60, e, n, m, g)
    packed = slim.pack4(_gpu(codes), _gpu(scale), _gpu(zero), g)
    X = _x(61, 50, m, "bf16").to("cuda:0")
    rows = (torch.arange(r, device="cuda:0") % 50).to(torch.int32)
    off = torch.tensor([0, r // 2 + 3, r], dtype=torch.int32, device="cuda:0")
    Y = slim.q4_experts(X, off, packed, n, g, rows=rows)
    for j, (a, b) in enumerate(((0, r // 2 + 3), (r // 2 + 3, r))):
        exact = X.double().cpu().numpy() @ oracle.q4_weight(codes[j], scale[j], zero[j], g).T
        one = Y[a:a + 50][torch.argsort(rows[a:a + 50])]
        bound = _bound(X.double().cpu().numpy(), codes[j], scale[j], zero[j], g, "bf16", "f32", exact)
        assert np.all(np.abs(one.double().cpu().numpy() - exact) <= bound)
        whole = Y[a:a + (b - a) // 50 * 50].view(-1, 50, n)
        assert torch.equal(whole, whole[:1].expand_as(whole))
    p1 = slim.pack4(_gpu(codes[0]), _gpu(scale[0]), _gpu(zero[0]), g)
    flat = torch.full((50 * n + 3,), 7.0, dtype=torch.bfloat16, device="cuda:0")
    out = slim.q4_linear(X, p1, n, g, out_dtype=torch.bfloat16, Y=flat[1:1 + 50 * n].view(50, n))
    assert torch.equal(out, slim.q4_linear(X, p1, n, g, out_dtype=torch.bfloat16))
    assert flat[0] == 7 and torch.all(flat[1 + 50 * n:] == 7)


def test_long_offsets_past_32_bits(slim):
    # more than 2^31 bytes before the last expert's matrix and the last row's logits
    e, n, m, g = 40, 16384, 8192, 128           # 75 MB a matrix, 3 GB in all
    words = slim.load_library().slim_pack4_words(1, n, m, g)
    packed = torch.zeros(e * words, dtype=torch.int32, device="cuda:0")
    codes, scale, zero = _layer(40, 1, n, m, g)
    packed[(e - 1) * words:] = slim.pack4(_gpu(codes), _gpu(scale), _gpu(zero), g)
    X = _x(41, 3, m, "bf16").to("cuda:0")
    off = torch.tensor([0] * e + [3], dtype=torch.int32, device="cuda:0")
    Y = slim.q4_experts(X, off, packed, n, g)
    one = slim.q4_linear(X, packed[(e - 1) * words:].clone(), n, g)
    # the two calls may join their partial sums in different orders: each is
    # within the bound of the exact value, so they are within twice of each other
    x = X.double().cpu().numpy()
    part = slice(n - 256, n)
    exact = x @ oracle.q4_weight(codes[0][part], scale[0][part], zero[0][part], g).T
    bound = _bound(x, codes[0][part], scale[0][part], zero[0][part], g, "bf16", "f32", exact)
    assert np.all(np.abs(Y[:, part].double().cpu().numpy() - exact) <= bound)
    assert np.all(np.abs((Y - one)[:, part].double().cpu().numpy()) <= 2 * bound)
    torch.testing.assert_close(Y, one, rtol=1e-4, atol=1e-3)
    del packed, Y, one
    t, v = 20000, 60000                          # 2.4 GB of bfloat16
    L = torch.zeros((t, v), dtype=torch.bfloat16, device="cuda:0")
    L[t - 1] = _logits(42, 1, v, 0, 0, "bf16").to("cuda:0")[0]
    ids = torch.full((t,), v - 1, device="cuda:0")
    got = slim.token_logprobs(L, ids, top=3)
    last = {k: a[t - 1:] for k, a in got.items()}
    _check_lp(last, L[t - 1:].double().cpu().numpy(), np.array([v - 1]), 3)
    assert got["top_id"][:t - 1].eq(torch.arange(3, device="cuda:0")).all()


# ------------------------------------------------------------------ the largest sizes
def _check_rows(got, x, codes, scale, zero, g, xdt):
    """Rows of Y, float64 rows of X and one matrix's codes."""
    exact = x @ oracle.q4_weight(codes, scale, zero, g).T
    bound = _bound(x, codes, scale, zero, g, xdt, "f32", exact)
    err = np.abs(got.double().cpu().numpy() - exact)
    assert np.all(err <= bound), float(np.max(err / bound))


@pytest.mark.parametrize("t,m,tiles", [(3, 640, False), (200, 32, True)])
def test_q4_linear_of_the_most_outputs(slim, t, m, tiles):
    n, g = 1 << 20, 32
    print(f"q4_linear t={t} n={n} m={m}", flush=True)
    assert (slim.load_library().slim_q4_linear_workspace(t, n, m, g, 1) > 0) == tiles
    gen = torch.Generator(device="cuda:0")
    gen.manual_seed(100)
    codes = torch.randint(0, 16, (n, m), generator=gen, device="cuda:0", dtype=torch.uint8)
    scale = 1e-3 + 0.01 * torch.rand((n, m // g), generator=gen, device="cuda:0")
    zero = 15 * torch.rand((n, m // g), generator=gen, device="cuda:0")
    X = _x(101, t, m, "bf16")
    Y = slim.q4_linear(X.to("cuda:0"), slim.pack4(codes, scale, zero, g), n, g)
    x = X.double().numpy()
    at = [0, 1, 2] if t < 100 else [0, 63, 64, 127, 128, 199]
    for a, b in ((0, 700), (n // 2 - 300, n // 2 + 300), (n - 700, n)):
        _check_rows(Y[at, a:b], x[at], *(w[a:b].cpu().numpy() for w in (codes, scale, zero)), g, "bf16")


@pytest.mark.parametrize("r,n,m,tiles", [(3000, 48, 160, False), (100000, 256, 128, True)])
def test_q4_experts_of_the_most_experts(slim, r, n, m, tiles):
    e, g = 1024, 32
    print(f"q4_experts e={e} r={r} n={n} m={m}", flush=True)
    assert (slim.load_library().slim_q4_experts_workspace(r, r, e, n, m, g, 1) > 0) == tiles
    rng = np.random.default_rng(102)
    off = np.sort(rng.integers(0, r + 1, size=e + 1)).astype(np.int32)
    off[1:1 + e // 4] = off[1]                               # a quarter of them have no rows
    off[0], off[-1] = 2, r - 3
    off = np.clip(off, 2, r - 3)
    codes, scale, zero = _layer(103, e, n, m, g)
    X = _x(104, r, m, "bf16")
    Y = torch.full((r, n), 7.0, device="cuda:0")
    slim.q4_experts(X.to("cuda:0"), _gpu(off), slim.pack4(_gpu(codes), _gpu(scale), _gpu(zero), g), n, g, Y=Y)
    assert torch.all(Y[:2] == 7.0) and torch.all(Y[r - 3:] == 7.0)
    x = X.double().numpy()
    for j in (0, 1, e // 4, e // 4 + 1, *range(300, e, 37), e - 1):
        a, b = off[j], off[j + 1]
        if a < b:
            _check_rows(Y[a:b], x[a:b], codes[j], scale[j], zero[j], g, "bf16")


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_token_logprobs_of_the_longest_rows(slim, dt):
    v, top = 1 << 24, 64
    print(f"token_logprobs v={v} {dt} top={top}", flush=True)
    x = _logits(105, 2, v, 0, 0, dt)
    x[1, v - 1] = 30.0
    ids = np.array([v - 1, v - 1])
    got = slim.token_logprobs(x.to("cuda:0"), _gpu(ids), top=top)
    # _check_lp, with numpy's sort in place of Python's
    xd = x.double().numpy()
    order = np.stack([np.argsort(-row, kind="stable")[:top] for row in xd])
    np.testing.assert_array_equal(got["top_id"].cpu().numpy(), order)
    mx = xd.max(axis=1, keepdims=True)
    lp = (xd - mx) - np.log(np.exp(xd - mx).sum(axis=1, keepdims=True))
    want = {"logprob": lp[:, v - 1], "entropy": -(np.exp(lp) * lp).sum(axis=1)}
    lp_b, ent_b, rs = _lp_bounds(xd, want)
    assert np.all(np.abs(got["logprob"].double().cpu().numpy() - want["logprob"]) <= lp_b)
    assert np.all(np.abs(got["entropy"].double().cpu().numpy() - want["entropy"]) <= ent_b)
    wl = np.take_along_axis(lp, order, axis=1)
    err = np.abs(got["top_logprob"].double().cpu().numpy() - wl)
    assert np.all(err <= rs[:, None] + 2.0 ** -22 * (1 + np.abs(wl)))


def test_token_logprobs_of_the_most_rows(slim):
    t, v = 1 << 23, 3
    print(f"token_logprobs t={t} v={v}", flush=True)
    gen = torch.Generator(device="cuda:0")
    gen.manual_seed(106)
    x = 3 * torch.randn((t, v), generator=gen, device="cuda:0")
    ids = torch.randint(0, v, (t,), generator=gen, device="cuda:0")
    got = slim.token_logprobs(x, ids, top=2)
    d = x.double() - x.double().amax(dim=1, keepdim=True)
    lp = d - d.exp().sum(dim=1, keepdim=True).log()
    # the bounds of _lp_bounds with the spread of all rows
    spread = float((-d).max())
    rs = 2.0 ** -24 * (v / 64 + 40 + 4 * (1 + spread))
    want = lp.gather(1, ids[:, None])[:, 0]
    assert ((got["logprob"].double() - want).abs() <= rs + 2.0 ** -22 * (1 + want.abs())).all()
    ent = -(lp.exp() * lp).sum(dim=1)
    assert ((got["entropy"].double() - ent).abs() <= 2 * rs * (1 + ent) + 2.0 ** -21 * (1 + ent + spread)).all()
    order = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :2]
    assert torch.equal(got["top_id"].long(), order)


@pytest.mark.parametrize("t,n,m,g", [(3, 64, 256, 128), (20, 96, 160, 32), (1290, 2320, 384, 128)])
@pytest.mark.parametrize("xdt", ["bf16", "f32"])
@pytest.mark.parametrize("size", [2.0 ** -100, 2.0 ** -115, 2.0 ** -125, 2.0 ** -130])
def test_q4_linear_of_tiny_rows(slim, t, n, m, g, xdt, size):
    # bfloat16 X is exact down to its least value, float32 X enters to its multiples, 2^-133 (truncated)
    codes, scale, zero = _layer(110, 1, n, m, g)
    scale *= np.float32(2.0 ** 90)
    X = (size * _x(111, t, m, "f32").double()).to(DT[xdt])
    Y = slim.q4_linear(X.to("cuda:0"), slim.pack4(_gpu(codes), _gpu(scale), _gpu(zero), g), n, g)
    x = X.double().numpy()
    exact = x @ oracle.q4_weight(codes[0], scale[0], zero[0], g).T
    bound = _bound(x, codes[0], scale[0], zero[0], g, xdt, "f32", exact)
    if xdt == "f32":
        bound += 2.0 ** -133 * (codes[0] * np.repeat(scale[0], g, -1).astype(np.float64)).sum(axis=1)
    # what is below float32's normal range before the scale: a group's sums, to half of 2^-149 a term
    bound += 2.0 ** -149 * (3 * g + 32 * 2) * np.abs(scale[0].astype(np.float64)).sum(axis=1)
    err = np.abs(Y.double().cpu().numpy() - exact)
    assert np.all(err <= bound), float(np.max(err / bound))


# ------------------------------------------------------------------ two calls at once
def test_two_threads_on_two_streams(slim):
    """Every operator from two host threads, each on a stream of its own, against what it gives alone."""
    import threading
    n, m, g = 1410, 576, 64
    codes, scale, zero = _layer(120, 2, n, m, g)
    packed = slim.pack4(_gpu(codes), _gpu(scale), _gpu(zero), g)
    one = slim.pack4(_gpu(codes[0]), _gpu(scale[0]), _gpu(zero[0]), g)
    big, small = _x(121, 2310, m, "bf16").to("cuda:0"), _x(122, 5, m, "f32").to("cuda:0")
    off = torch.tensor([0, 1000, 2310], dtype=torch.int32, device="cuda:0")
    ids = torch.arange(2310, device="cuda:0") % n
    logits = _logits(123, 3, 40000, 0, 0, "f32").to("cuda:0")
    assert slim.load_library().slim_q4_linear_workspace(2310, n, m, g, 1) > 0       # a tile kernel
    assert slim.load_library().slim_token_logprobs_workspace(3, 40000, 4) > 0       # rows in segments

    def calls():
        s = slim.score_tokens(big, ids, one, n, g, top=3, block=1000)
        p = slim.token_logprobs(logits, ids[:3], top=4)
        return [slim.q4_linear(big, one, n, g), slim.q4_linear(small, one, n, g),
                slim.q4_experts(big, off, packed, n, g), *s.values(), *p.values()]
    want = calls()
    torch.cuda.synchronize()
    bad = []

    def work():
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(5):
                got = calls()
                stream.synchronize()
                bad.extend(i for i, (a, b) in enumerate(zip(got, want)) if not torch.equal(a, b))
    threads = [threading.Thread(target=work) for _ in range(2)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not bad, bad


@pytest.mark.parametrize("how", ["gptq", "hinv"])
def test_nibbles_of_every_way_to_quantize(slim, how):
    n, m, g, avg = 96, 512, 128, 3
    W = (0.02 * _x(130, n, m, "f32")).to(torch.bfloat16).to("cuda:0")
    X = _x(131, 300, m, "bf16").to("cuda:0")
    if how == "gptq":
        q = slim.quantize_layer(X, W, g, avg, gptq=True, nibbles=True)
    else:
        first = slim.quantize_layer(X, W, g, avg)
        q = slim.quantize_layer(X, W, g, avg, H=first["H"], hinv=first["hinv"], nibbles=True)
    assert int(q["info"]) == 0 and int(q["pack_info"]) == 0 and int(q["codes"].max()) < 16
    codes, scale, zero = (q[k].cpu().numpy() for k in ("codes", "scale", "zero"))
    np.testing.assert_array_equal(q["packed4"].cpu().numpy().view(np.uint32),
                                  oracle.pack4(codes[None], scale[None], zero[None], g))
    x = X[:9].double().cpu().numpy()
    exact = x @ oracle.q4_weight(codes, scale, zero, g).T
    Y = slim.q4_linear(X[:9].contiguous(), q["packed4"], n, g).double().cpu().numpy()
    assert np.all(np.abs(Y - exact) <= _bound(x, codes, scale, zero, g, "bf16", "f32", exact))

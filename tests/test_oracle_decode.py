"""Pins of the oracle's cache, attention and draft verification: against
definitions worked another way and against torch's attention on the CPU."""
import numpy as np
import pytest

import oracle

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("dim,group", [(64, 32), (128, 128), (256, 64)])
def test_quantizer_covers_and_rounds(dim, group):
    x = np.random.default_rng(1).standard_normal((50, 3, dim)).astype(np.float32) * 10
    x[0] = 2.5                                       # constant, a bfloat16 value
    x[1] = np.float32(0.1)                           # constant, not one
    codes, step, low = oracle.kv4_quantize(x, group)
    y = oracle.kv4_values(codes, step, low, group)
    s = np.repeat(step, group, -1)
    assert np.all(np.abs(y - x) <= 0.5001 * s + 1e-6)          # the grid covers every entry
    assert np.all(y[0] == 2.5) and np.all(step[0] == 0)
    assert np.all(np.abs(y[1] - 0.1) <= 0.1 * 2.0 ** -7)
    assert codes.max() == 15 and codes.min() == 0
    # steps and low ends are bfloat16 values, at most one unit outwards
    for z in (step, low):
        assert np.all(z.view(np.uint32) & 0xFFFF == 0)
    xg = x.reshape(50, 3, dim // group, group)
    lo, hi = xg.min(-1), xg.max(-1)
    assert np.all(low <= lo) and np.all(lo - low <= np.abs(lo) * 2.0 ** -7)
    true = (hi.astype(np.float64) - low) / 15
    assert np.all(step >= true * (1 - 2.0 ** -23)) and np.all(step <= true * (1 + 2.0 ** -7) + 1e-37)


def test_quantizer_of_what_has_no_grid():
    x = np.zeros((5, 1, 64), np.float32)
    x[0, 0, 3], x[1, 0, 40], x[2, 0, 0], x[3, 0, 0] = np.nan, np.inf, 3.3e38, 1e-42
    x[2, 0, 1] = -3.3e38
    codes, step, low = oracle.kv4_quantize(x, 32)
    y = oracle.kv4_values(codes, step, low, 32)
    assert np.isnan(y[0, 0, :32]).all() and np.all(y[0, 0, 32:] == 0)
    assert np.isnan(y[1, 0, 32:]).all() and np.isnan(y[2, 0, :32]).all()
    assert step[3, 0, 0] == np.float32(2.0 ** -126) and np.all(np.abs(y[3]) <= 1e-42) and np.all(y[4] == 0)


@pytest.mark.parametrize("page,dim,group", [(16, 64, 32), (32, 128, 64)])
def test_layout_decodes(page, dim, group):
    rng = np.random.default_rng(2)
    heads, ng = 2, dim // group
    cache = np.zeros((3, heads, oracle.kv4_words(page, dim, group)), np.uint32)
    slots = [0, 17, 2 * page + 7, 3 * page - 1]
    held = {}
    for s in slots:
        held[s] = [oracle.kv4_quantize(rng.standard_normal((heads, dim)).astype(np.float32), group) for _ in "kv"]
        oracle.kv4_put(cache, s, page, dim, group, *held[s])
    rec_words = 4 * dim + 32 * ng
    for s in slots:
        for h in range(heads):
            rec = cache[s // page, h, s % page // 16 * rec_words:][:rec_words]
            t = s % 16
            for c in (0, 5, 31, 33, dim - 1):
                j, lg, e = c // 32, c % 32 // 8, c % 8
                word = int(rec[(16 * lg + t) * (dim // 32) + j])
                assert (word >> (8 * (e % 4) + 4 * (e // 4))) & 15 == held[s][0][0][h, c]
                word = int(rec[2 * dim + (16 * (t // 4) + c % 32 // 2) * (dim // 32) + c // 32])
                assert (word >> (8 * (t % 4) + 4 * (c % 2))) & 15 == held[s][1][0][h, c]
            for q in range(ng):
                for x in (0, 1):
                    word = rec[4 * dim + 16 * ng * x + 16 * q + t]
                    assert np.uint32(word << np.uint32(16)).view(np.float32) == held[s][x][1][h, q]
                    assert np.uint32(word & np.uint32(0xFFFF0000)).view(np.float32) == held[s][x][2][h, q]


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_complex_product(interleaved):
    rng = np.random.default_rng(3)
    x = rng.standard_normal((4, 2, 64)).astype(np.float32)
    a = rng.uniform(0, 6, (9, 16))
    table = np.concatenate([np.cos(a), np.sin(a)], axis=1).astype(np.float32)
    pos = [3, 0, 8, 9]
    y = oracle.rotate(x, table, pos, interleaved)
    assert np.all(y[:3, :, 32:] == x[:3, :, 32:]) and np.isnan(y[3]).all()
    for i in range(3):
        u = table[pos[i], :16].astype(np.float64) + 1j * table[pos[i], 16:]
        z = x[i, :, 0:32:2] + 1j * x[i, :, 1:32:2] if interleaved else x[i, :, :16] + 1j * x[i, :, 16:32]
        w = z * u
        got = y[i, :, 0:32:2] + 1j * y[i, :, 1:32:2] if interleaved else y[i, :, :16] + 1j * y[i, :, 16:32]
        np.testing.assert_allclose(got, w, rtol=0, atol=1e-6)


@pytest.mark.parametrize("causal", [True, False])
def test_attention_matches_torch(causal):
    rng = np.random.default_rng(4)
    n, length, hq, heads, dim = 3, 11, 4, 2, 64
    q, k, v = (rng.standard_normal(s) for s in ((n, hq, dim), (length, heads, dim), (length, heads, dim)))
    out = oracle.attention(q, k, v, 0.125, causal)
    kk, vv = (torch.from_numpy(x).repeat_interleave(2, dim=1).permute(1, 0, 2) for x in (k, v))
    mask = torch.ones(n, length, dtype=torch.bool).tril(length - n) if causal else None
    want = torch.nn.functional.scaled_dot_product_attention(torch.from_numpy(q).permute(1, 0, 2), kk, vv, attn_mask=mask,
                                                            scale=0.125)
    np.testing.assert_allclose(out, want.permute(1, 0, 2).numpy(), atol=1e-12)
    assert np.all(oracle.attention(q, k[:1], v[:1], 1.0, True)[:2] == 0)     # more queries than tokens


def test_draft_decisions():
    # two tokens, target half and half, draft 3/4 : 1/4
    t = np.log(np.array([[[0.5, 0.5], [0.9, 0.1]]]))
    d = np.log(np.array([[[0.75, 0.25]]]))
    run = lambda tok, u, w, **kw: [x.tolist() for x in oracle.verify_draft(t, np.array([[tok]]), np.array([[u, w]]), **kw)[:2]]  # noqa: E731,E501
    assert run(0, 0.6, 0.95, draft=d) == [[1], [[0, 1]]]       # 0.45 < 0.5: taken, then from the target's next row
    assert run(0, 0.7, 0.3, draft=d) == [[0], [[1, -1]]]       # 0.525: refused, what is left is token 1
    assert run(1, 0.99, 0.5, draft=d) == [[1], [[1, 0]]]       # p > q: always taken
    assert run(0, 0.49, 0.5) == [[1], [[0, 0]]]                # no probabilities: taken below p
    assert run(0, 0.51, 0.0) == [[0], [[1, -1]]]
    assert run(-1, 0.0, 0.7, draft=d) == [[0], [[1, -1]]]      # no draft: from the target
    assert run(2, 0.0, 0.2, draft=d) == [[0], [[1, -1]]]       # outside the vocabulary


def test_draft_keeps_the_targets_distribution():
    rng = np.random.default_rng(5)
    p, q = np.array([0.5, 0.3, 0.15, 0.05]), np.array([0.1, 0.2, 0.3, 0.4])
    n = 20000
    x = rng.choice(4, size=n, p=q)
    acc, ids, _ = oracle.verify_draft(np.broadcast_to(np.log([p, p]), (n, 2, 4)), x[:, None], rng.random((n, 2)),
                                      draft=np.broadcast_to(np.log(q), (n, 1, 4)))
    seen = np.bincount(ids[:, 0], minlength=4) / n
    assert np.all(np.abs(seen - p) < 5 * np.sqrt(p * (1 - p) / n))

"""Pins of the oracle's serving operators: against dequantization and matrix
products done another way, and against scipy's softmax functions."""
import numpy as np
import pytest
from scipy import special

import oracle


def _layer(seed, e, n, m, g):
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 16, size=(e, n, m), dtype=np.uint8)
    scale = rng.uniform(1e-3, 1e-2, size=(e, n, m // g)).astype(np.float32)
    zero = rng.uniform(0, 15, size=(e, n, m // g)).astype(np.float32)
    return codes, scale, zero


@pytest.mark.parametrize("e,n,m,g", [(1, 16, 128, 128), (2, 5, 96, 32), (1, 33, 320, 64)])
def test_pack4_layout_decodes(e, n, m, g):
    codes, scale, zero = _layer(1, e, n, m, g)
    words = oracle.pack4(codes, scale, zero, g)
    nrb, nch = -(-n // 16), -(-m // 128)
    rec = words.reshape(e, nrb, nch, 256 + 32 * (128 // g))
    for x in range(e):
        for i in (0, n // 2, n - 1):
            for c in (0, 3, 4, 31, m // 2, m - 1):
                ch, o = divmod(c, 128)
                word = rec[x, i // 16, ch, 4 * (16 * (o % 32 // 8) + i % 16) + o // 32]
                nib = int(word).to_bytes(4, "little")[o % 4]
                assert (nib >> (4 if o % 8 >= 4 else 0)) & 15 == codes[x, i, c]
                q = o // g
                assert rec[x, i // 16, ch, 256 + 2 * (16 * q + i % 16)].view(np.float32) == scale[x, i, c // g]
                assert rec[x, i // 16, ch, 257 + 2 * (16 * q + i % 16)].view(np.float32) == zero[x, i, c // g]
    # what lies past n and m is zero
    assert sum(int(w).bit_count() if hasattr(int, "bit_count") else bin(int(w)).count("1") for w in
               rec[:, :, :, :256].reshape(-1)) == sum(bin(int(c)).count("1") for c in codes.reshape(-1))


def test_products_match_loops():
    codes, scale, zero = _layer(2, 3, 7, 64, 32)
    X = np.random.default_rng(3).standard_normal((6, 64)).astype(np.float32)
    Y = oracle.q4_linear(X, codes[0], scale[0], zero[0], 32)
    for a in range(6):
        for i in range(7):
            y = sum(float(X[a, c]) * (float(codes[0, i, c]) - float(zero[0, i, c // 32])) * float(scale[0, i, c // 32])
                    for c in range(64))
            assert abs(y - Y[a, i]) < 1e-12
    rows, gates = [5, 0, 2, 2], np.array([0.5, 1.0, 2.0, -1.0], np.float32)
    out = oracle.q4_experts(X, [0, 1, 1, 4], codes, scale, zero, 32, rows, gates)
    assert sorted(out) == [0, 1, 2, 3]
    np.testing.assert_allclose(out[0], 0.5 * oracle.q4_linear(X[5:6], codes[0], scale[0], zero[0], 32)[0])
    np.testing.assert_allclose(out[3], -oracle.q4_linear(X[2:3], codes[2], scale[2], zero[2], 32)[0])


def test_logprobs_match_scipy():
    rng = np.random.default_rng(4)
    x = (3 * rng.standard_normal((5, 40))).astype(np.float32)
    x[1, ::2] = -np.inf
    x[2] = -np.inf
    ids = np.array([3, 1, 0, -1, 40])
    out = oracle.token_logprobs(x, ids, top=4)
    lp = special.log_softmax(x.astype(np.float64), axis=1)
    p = special.softmax(x.astype(np.float64), axis=1)
    assert abs(out["logprob"][0] - lp[0, 3]) < 1e-12 and abs(out["logprob"][1] - lp[1, 1]) < 1e-12
    assert np.isnan(out["logprob"][2]) and out["logprob"][3] == 0 and np.isnan(out["logprob"][4])
    for a in (0, 1, 3, 4):
        assert abs(out["entropy"][a] - special.entr(p[a]).sum()) < 1e-12
        np.testing.assert_array_equal(out["top_id"][a], np.argsort(-x[a], kind="stable")[:4])
        np.testing.assert_allclose(out["top_logprob"][a], lp[a][out["top_id"][a]])
    assert np.all(out["top_id"][2] == -1)

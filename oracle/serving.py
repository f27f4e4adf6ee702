"""Products from 4-bit codes, grouped by expert or not, and token log
probabilities.  TEST INFRASTRUCTURE (oracle).

The dequantized weight is (q - zero) * scale (rkmt.cn digest, FAQ on storage
and deployment); here it and the product are taken in float64.  Perplexity,
the metric of the digest's evaluation, is the mean of -ln p of the given
tokens.  Everything below is written from these definitions with loops where
they are short; it shares nothing with the kernels.
"""
import numpy as np

from .decode import as_f64


def pack4(codes, scale, zero, group: int) -> np.ndarray:
    """The 4-bit layout as slim.h states it, uint32 words, codes [e, n, m]."""
    e, n, m = codes.shape
    nrb, nch, gpc = -(-n // 16), -(-m // 128), 128 // group
    rec_words = 256 + 32 * gpc
    full = np.zeros((e, nrb * 16, nch * 128), dtype=np.uint32)
    full[:, :n, :m] = codes & 15
    s = np.zeros((e, nrb * 16, nch * gpc), dtype=np.float32)
    z = np.zeros_like(s)
    s[:, :n, :m // group] = scale
    z[:, :n, :m // group] = zero
    out = np.zeros((e * nrb * nch, rec_words), dtype=np.uint32)
    for x in range(e):
        for rb in range(nrb):
            for ch in range(nch):
                rec = out[(x * nrb + rb) * nch + ch]
                for lg in range(4):
                    for r in range(16):
                        for i in range(4):
                            c0 = 128 * ch + 32 * i + 8 * lg
                            q = full[x, 16 * rb + r, c0:c0 + 8]
                            rec[4 * (16 * lg + r) + i] = sum(int(q[b] + 16 * q[b + 4]) << (8 * b) for b in range(4))
                for q in range(gpc):
                    for r in range(16):
                        rec[256 + 2 * (16 * q + r)] = s[x, 16 * rb + r, ch * gpc + q].view(np.uint32)
                        rec[257 + 2 * (16 * q + r)] = z[x, 16 * rb + r, ch * gpc + q].view(np.uint32)
    return out.reshape(-1)


def q4_weight(codes, scale, zero, group: int) -> np.ndarray:
    """(q - zero) * scale in float64, [n, m]."""
    z = np.repeat(np.asarray(zero, dtype=np.float64), group, axis=-1)
    s = np.repeat(np.asarray(scale, dtype=np.float64), group, axis=-1)
    return (np.asarray(codes, dtype=np.float64) - z) * s


def q4_linear(X, codes, scale, zero, group: int) -> np.ndarray:
    return as_f64(X) @ q4_weight(codes, scale, zero, group).T


def q4_experts(X, offsets, codes, scale, zero, group: int, rows=None, row_scale=None) -> dict:
    """{row of Y: float64 [n]} for the rows the offsets cover."""
    x = as_f64(X)
    out = {}
    for j in range(len(offsets) - 1):
        w = q4_weight(codes[j], scale[j], zero[j], group)
        for a in range(offsets[j], offsets[j + 1]):
            src = a if rows is None else rows[a]
            out[a] = w @ x[src] * (1.0 if row_scale is None else float(row_scale[a]))
    return out


def token_logprobs(logits, ids, top: int = 0) -> dict:
    """float64 log probability, entropy and the top entries, row by row."""
    t, v = np.shape(logits)
    x = as_f64(logits)
    out = {"logprob": np.zeros(t), "entropy": np.zeros(t), "top_logprob": np.zeros((t, top)),
           "top_id": np.zeros((t, top), dtype=np.int32)}
    for a in range(t):
        row = x[a]
        if np.isnan(row).any() or np.isposinf(row).any() or np.isneginf(row).all():
            out["logprob"][a] = 0.0 if ids[a] < 0 else np.nan
            out["entropy"][a] = np.nan
            out["top_logprob"][a] = np.nan
            out["top_id"][a] = -1
            continue
        m = row.max()
        # (x - m) - ln S, not x - (m + ln S): next to a maximum of -3.4e38 the sum loses ln S
        lp = (row - m) - np.log(np.exp(row - m).sum())
        p = np.exp(lp)
        out["entropy"][a] = -np.sum(p[p > 0] * lp[p > 0])
        out["logprob"][a] = 0.0 if ids[a] < 0 else np.nan if ids[a] >= v else lp[ids[a]]
        order = sorted(range(v), key=lambda j: (-row[j], j))[:top]
        out["top_id"][a] = order
        out["top_logprob"][a] = lp[order]
    return out

"""Verification of drafted tokens.  TEST INFRASTRUCTURE (oracle).

Token by token from the definition in slim.h, in float64; it shares nothing
with the kernels.
"""
import numpy as np

from .decode import as_f64


def _softmax(row, temperature):
    x = as_f64(row)
    if np.isnan(x).any() or np.isposinf(x).any() or np.isneginf(x).all():
        return None
    e = np.exp((x - x.max()) / temperature)
    return e / e.sum()


def verify_draft(target, tokens, uniform, draft=None, temperature: float = 1.0):
    """-> accepted int32 [b], ids int64 [b, k + 1], margin [b]: how far (relative to the whole) the last
    decision or the drawn border was from its border, for near ties."""
    b, k1, v = np.shape(target)
    k = k1 - 1
    accepted, ids, margin = np.zeros(b, np.int32), np.full((b, k1), -1, np.int64), np.full(b, np.inf)
    for i in range(b):
        j = 0
        while True:
            p = _softmax(target[i][j], temperature)
            x = int(tokens[i, j]) if j < k else -1
            if x < 0:
                mass = p
                break
            if draft is None:
                q = np.zeros(v)
                if x < v:
                    q[x] = 1.0
            else:
                q = _softmax(draft[i][j], temperature)
            if p is None or q is None:
                mass = None
                break
            px, qx = (p[x], q[x]) if x < v else (0.0, 0.0)
            bar = float(uniform[i, j]) * qx
            if x < v and (px or bar):            # two powers of 0 are that exactly, on either side
                margin[i] = min(margin[i], abs(bar - px) / max(px, bar, 1e-300))
            if bar < px:
                ids[i, j] = x
                j += 1
                continue
            mass = np.where(p - q > 2.0 ** -44 * p, p - q, 0.0)
            break
        accepted[i] = j
        if mass is None or not mass.sum() > 0:
            continue
        run = np.cumsum(mass)
        want = float(uniform[i, k]) * run[-1]
        ids[i, j] = int(np.argmax(run > want))
        margin[i] = min(margin[i], np.abs(run - want).min() / run[-1])
    return accepted, ids, margin

"""The 4-bit key/value cache and attention over it.  TEST INFRASTRUCTURE (oracle).

The quantizer of the cache is a fixed float32 operation sequence (low end and
step rounded to bfloat16 outwards), so codes are comparable bit for bit; the
rotation and the attention are float64.  Written from the definitions in
slim.h with plain loops; it shares nothing with the kernels.
"""
import numpy as np

from .decode import as_f32, as_f64


def _bf16_down(x):
    u = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    neg = u >> 31 == 1
    u = np.where(neg, u + 0xFFFF, u) & 0xFFFF0000
    return u.astype(np.uint32).view(np.float32)


def _bf16_up(x):
    """Of numbers >= 0."""
    u = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    return ((u + 0xFFFF) & 0xFFFF0000).astype(np.uint32).view(np.float32)


def kv4_quantize(x, group: int):
    """float32 [..., dim] -> codes uint8 [..., dim], step and low float32 [..., dim / group]."""
    x = np.asarray(x, dtype=np.float32)
    xg = x.reshape(*x.shape[:-1], x.shape[-1] // group, group)
    with np.errstate(all="ignore"):
        good = np.isfinite(xg).all(axis=-1)
        safe = np.where(good[..., None], xg, np.float32(0))
        low = _bf16_down(safe.min(axis=-1))
        step = _bf16_up((safe.max(axis=-1) - low) / np.float32(15))
        good &= np.isfinite(low) & np.isfinite(step)
        step = np.where(step > 0, np.maximum(step, np.float32(2.0 ** -126)), step)
        step = np.where(good, step, np.float32(np.nan)).astype(np.float32)
        low = np.where(good, low, np.float32(0)).astype(np.float32)
        inv = np.where(step > 0, np.float32(1) / step, np.float32(0)).astype(np.float32)
        n = np.rint((safe - low[..., None]) * inv[..., None])
        codes = np.where(good[..., None], np.clip(n, 0, 15), 0).astype(np.uint8)
    return codes.reshape(x.shape), step, low


def kv4_values(codes, step, low, group: int) -> np.ndarray:
    """float32 fl(code step + low): the product is exact."""
    s = np.repeat(step.astype(np.float64), group, axis=-1)
    lo = np.repeat(low.astype(np.float64), group, axis=-1)
    return (codes.astype(np.float64) * s + lo).astype(np.float32)


def rotate(x, rotary, positions, interleaved: bool) -> np.ndarray:
    """[t, heads, dim] stored rows -> float32, the first rot channels of every head turned."""
    y = as_f64(x).copy()
    if rotary is None:
        return y.astype(np.float32)
    rot = rotary.shape[1]
    for i, p in enumerate(positions):
        if not 0 <= p < rotary.shape[0]:
            y[i] = np.nan
            continue
        for j in range(rot // 2):
            a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + rot // 2)
            c, s = float(rotary[p, j]), float(rotary[p, rot // 2 + j])
            u, w = y[i, :, a].copy(), y[i, :, b].copy()
            y[i, :, a], y[i, :, b] = u * c - w * s, w * c + u * s
    return y.astype(np.float32)


def kv4_words(page: int, dim: int, group: int) -> int:
    return page // 16 * (4 * dim + 32 * (dim // group))


def kv4_put(cache, slot: int, page: int, dim: int, group: int, k, v):
    """One token's quantized key and value, (codes, step, low) [heads, ..] each, into uint32 words."""
    k_codes, k_step, k_low = k
    v_codes, v_step, v_low = v
    ng, rec_words = dim // group, 4 * dim + 32 * (dim // group)
    t = slot % 16
    bits = lambda s, lo: int(np.float32(s).view(np.uint32) >> 16) | int(np.float32(lo).view(np.uint32))  # noqa: E731
    for h in range(cache.shape[1]):
        rec = cache[slot // page, h].reshape(page // 16, rec_words)[slot % page // 16]
        for lg in range(4):
            for j in range(dim // 32):
                c = 32 * j + 8 * lg
                rec[(16 * lg + t) * (dim // 32) + j] = sum(
                    (int(k_codes[h, c + b]) + 16 * int(k_codes[h, c + 4 + b])) << (8 * b) for b in range(4))
        as_bytes = rec[2 * dim:4 * dim].view(np.uint8)
        for r in range(16):
            for a in range(dim // 32):
                c = 32 * a + 2 * r
                as_bytes[4 * ((16 * (t // 4) + r) * (dim // 32) + a) + t % 4] = v_codes[h, c] + 16 * v_codes[h, c + 1]
        for q in range(ng):
            rec[4 * dim + 16 * q + t] = bits(k_step[h, q], k_low[h, q])
            rec[4 * dim + 16 * ng + 16 * q + t] = bits(v_step[h, q], v_low[h, q])


def attention(q, k, v, scale: float, causal: bool) -> np.ndarray:
    """One sequence: q [n, hq, dim], the last n tokens' queries; k, v [len, heads, dim] values -> float64.
    A row that attends to nothing is 0."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    n, hq, _ = q.shape
    out = np.zeros(q.shape)
    for i in range(n):
        reach = len(k) - n + i + 1 if causal else len(k)
        if reach <= 0:
            continue
        for h in range(hq):
            hh = h // (hq // k.shape[1])
            s = scale * (k[:reach, hh] @ q[i, h])
            p = np.exp(s - s.max())
            out[i, h] = (p / p.sum()) @ v[:reach, hh]
    return out

"""One linear layer through the whole path, enqueued on the current stream.

Stage order as in the SliM-LLM blog digest (rkmt.cn), core design: Hessian
from calibration activations, salience, SBA bit allocation, SQC calibration,
then group-structured storage.  Nothing is copied back to the host between
stages; the caller synchronises once and may inspect ``info``.
"""
from __future__ import annotations

from . import _lib


def quantize_layer(X, W, group: int = 128, avg_bits: int = 2, lam: float = 0.1, n_tau: int = 50,
                   damp_frac: float = 0.01, H=None, gptq: bool = False, hinv=None, nibbles: bool = False):
    """X [T, m], W [n, m] (bf16 or f32, GPU).  If H is given the Hessian stage is
    skipped (a Hessian shared by several linears of one input width); if hinv,
    that H's diag((H + a I)^-1) from an earlier call, is given too, the
    factorisation is skipped as well and only the group means are formed.
    With gptq set, the groups are calibrated and quantized inside GPTQ's
    error-compensating sweep (the backbone the digest names) instead of
    independently (it reads the factor, so hinv is not taken then).  With nibbles
    the codes are also laid out for the 4-bit products (packed4, for q4_linear;
    avg_bits at most 3, so that no width is above 4)."""
    if nibbles and avg_bits > 3:
        raise _lib.SlimError(f"nibbles: widths up to {avg_bits + 1} do not fit 4 bits")
    if hinv is not None and (H is None or gptq):
        raise _lib.SlimError("hinv is taken with the H it came from, and not with gptq")
    if H is None:
        H = _lib.hessian(X)
    if gptq:   # the salience sweep also yields the factor GPTQ reads
        hinv, gsal, info, _, U = _lib.salience(H, W, group, damp_frac, want_u=True)
    elif hinv is not None:
        gsal, info, _ = _lib.group_salience(hinv, W, group)
    else:
        hinv, gsal, info, _ = _lib.salience(H, W, group, damp_frac)
    bits, kl, r_star = _lib.sba_search(X, W, gsal, group, avg_bits)
    if gptq:
        sq = _lib.gptq_quantize(None, W, bits, hinv, group, damp_frac, lam, n_tau, U=U)
        sq["gptq_info"] = sq.pop("info")
    else:
        sq = _lib.sqc_calibrate(W, bits, hinv, group, lam, n_tau)
    packed, pinfo = _lib.pack(sq["codes"], bits, group, avg_bits)
    out = {"H": H, "hinv": hinv, "group_sal": gsal, "info": info, "bits": bits, "kl": kl, "r_star": r_star,
           "pack_info": pinfo, "packed": packed, **sq}
    if nibbles:
        out["packed4"] = _lib.pack4(sq["codes"], sq["scale"], sq["zero"], group)
    return out


def score_tokens(X, ids, packed4, n: int, group: int, top: int = 0, block: int = 2048):
    """Scores of given tokens under an output layer in the 4-bit layout (perplexity is the
    exponential of minus their mean log probability; the metric of the digest's evaluation).
    X [T, m] (the layer's inputs, bf16 or f32), ids int64 [T] (negative: padding), packed4 of the
    n x m layer -> as token_logprobs.  The logits, float32 [T, n], are formed and scored a block
    of rows at a time in one buffer; at the default block of 2048 rows they take 2048 n floats."""
    import torch
    if block < 1:
        raise _lib.SlimError(f"block {block} must be at least 1")
    if not isinstance(X, torch.Tensor) or not isinstance(ids, torch.Tensor) or X.dim() != 2 or ids.dim() != 1 \
            or ids.shape[0] != X.shape[0]:
        raise _lib.SlimError("X: expected [T, m] and ids: expected [T]")
    T, m = X.shape
    # what can be refused, before the buffer of a block's logits is made
    packed4 = _lib._arg(packed4, "packed", (_lib._words4(1, n, m, group),), (torch.int32,))
    if not 0 <= top <= min(n, _lib.LOGPROB_MAX_TOP):
        raise _lib.SlimError(f"top {top} must lie in 0 .. {min(n, _lib.LOGPROB_MAX_TOP)}")
    if not (X.is_cuda and packed4.is_cuda and ids.is_cuda):
        raise _lib.SlimError("tensors must live in GPU memory")
    if T <= block:
        return _lib.token_logprobs(_lib.q4_linear(X, packed4, n, group), ids, top)
    buf = torch.empty((block, n), dtype=torch.float32, device=X.device)
    parts = []
    for a in range(0, T, block):
        b = min(T, a + block)
        logits = _lib.q4_linear(X[a:b], packed4, n, group, Y=buf[:b - a])
        parts.append(_lib.token_logprobs(logits, ids[a:b], top))
    return {k: torch.cat([p[k] for p in parts]) for k in parts[0]}

"""SliM-LLM per-layer quantizer path for MI355X (gfx950).

Five stages, each one C-ABI call into libslim.so (include/slim.h) running
hand-written HIP kernels:

    hessian        H = 2 X^T X                                  (MFMA bf16/f32)
    salience       d = diag((H + a I)^-1), group-mean w^2/d^2   (fp64 MFMA Cholesky)
    sba_search     balanced N-1/N/N+1 allocation scored by output KL (fused MFMA + softmax)
                   (sba_search_ex: output-MSE objective or a given group order, for the ablations)
    sqc_calibrate  3-sigma mask + tau grid over scale and zero  (wave-level, VALU)
                   (gptq_quantize: the same quantizer inside GPTQ's error-compensating sweep;
                    lwc_calibrate: SliM-LLM+, learnable weight clipping in its place)
    pack           group-structured bit-planes                  (HBM)
    qlinear        Y = X W_hat^T read from the planes (decode-sized batches)
                   (qlinear_noalloc: the same with no workspace, for callers that cannot allocate)

    pack4          codes of up to 4 bits with scales and zeros in one streamable buffer
    q4_linear      Y = X W_hat^T read from it, decode batches to prefill (MFMA bf16)
    q4_experts     the same grouped by expert over rows sorted by expert
    token_logprobs log probability of given tokens, entropy and best entries of logits (HBM)

    kv4_cache      an empty paged cache of keys and values in 4 bits
    kv4_append     keys and values into it, rotated to their positions on the way (kv4_read: what slots hold)
    kv4_attention  attention over it, single tokens to prompts (MFMA bf16, HBM)
    verify_draft   drafted tokens against the target's probabilities, from given random numbers

``quantize_layer`` chains the five stages on the current stream; ``score_tokens`` chains an output
layer's 4-bit product and the scores of its logits.  PyTorch only provides
device memory and the stream.
"""
from ._lib import (SlimError, load_library, hessian, salience, group_salience, sba_search, sba_search_ex, sqc_calibrate, gptq_quantize,
                   lwc_calibrate, pack, qlinear, qlinear_noalloc, pack4, q4_linear, q4_experts,
                   token_logprobs, kv4_cache, kv4_append, kv4_read, kv4_attention, verify_draft, tau_table,
                   timing_enable, timing_select, timing_reset, timing_read, SLIM_F32, SLIM_BF16)
from .layer import quantize_layer, score_tokens

__all__ = ["SlimError", "load_library", "hessian", "salience", "group_salience", "sba_search", "sba_search_ex", "sqc_calibrate",
           "gptq_quantize", "lwc_calibrate", "pack", "qlinear", "qlinear_noalloc", "pack4", "q4_linear", "q4_experts",
           "token_logprobs", "kv4_cache", "kv4_append", "kv4_read", "kv4_attention", "verify_draft", "tau_table", "timing_enable", "timing_select", "timing_reset", "timing_read", "quantize_layer", "score_tokens", "SLIM_F32",
           "SLIM_BF16"]

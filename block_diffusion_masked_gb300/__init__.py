"""Block-diffusion attention on GB300 (sm_103a).

Exact softmax attention over a [noisy | clean] sequence of length 2n under the
block-diffusion mask, forward and backward, in hand-written tcgen05/TMA CUDA
kernels behind the C ABI of ``libdfa.so`` (``include/dfa.h``).  PyTorch only
provides device memory, streams and autograd plumbing.

    from block_diffusion_masked_gb300 import diffusion_attn_func
    out = diffusion_attn_func(q, k, v, block_size=4)  # (batch, 2n, heads, headdim) bf16

Sampling, block by block, over a paged 8-bit (or 4-bit: bits=4) cache of the
finished tokens:

    from block_diffusion_masked_gb300 import KVCache, PageTable, rotary_func, rotary_table
    pages = PageTable(batch, max_pages, num_pages, page_size)
    cache = KVCache(num_pages, page_size, kv_heads, headdim)   # one per layer
    step = pages.plan(new_lens, rows, max_new)                 # one per step
    q, k = rotary_func(q, k, table, step.positions)            # packed rows
    out, lse = cache.attend(q, step, k, v, block_size)
    cache.append(k, v, step)                                   # the block is finished
    pages.advance(step)
    k, v = cache.read(pages, cu_rows, rows)                    # tokens back as bf16

Scores of tokens, for a sampler's choice by confidence and for the loss, which is
differentiable in the logits:

    from block_diffusion_masked_gb300 import token_logprobs_func
    logprobs, entropy, top_logprobs, top_tokens = token_logprobs_func(logits, tokens, top=8)

The binding is imported lazily so that ``inputs`` can be used without CUDA.
"""

from __future__ import annotations

__all__ = ["diffusion_attn_func", "diffusion_attn_varlen_func", "causal_attn_func",
           "rotary_func", "rotary_table", "token_logprobs_func", "PageTable", "KVCache", "binding"]


def __getattr__(name):
    import importlib

    if name in ("rotary_table", "PageTable", "KVCache"):
        value = getattr(importlib.import_module(__name__ + ".sampling"), name)
    elif name in ("diffusion_attn_func", "diffusion_attn_varlen_func", "causal_attn_func",
                  "rotary_func", "token_logprobs_func", "DiffusionAttnFunc",
                  "DiffusionAttnVarlenFunc", "CausalAttnFunc", "RotaryFunc",
                  "TokenLogprobsFunc"):
        value = getattr(importlib.import_module(__name__ + ".autograd"), name)
    elif name in ("binding", "autograd", "inputs", "build", "sampling"):
        return importlib.import_module(__name__ + "." + name)
    else:
        raise AttributeError(name)
    globals()[name] = value  # not looked up again
    return value

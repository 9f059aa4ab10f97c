"""Block-diffusion attention on GB300 (sm_103a).

Exact softmax attention over a [noisy | clean] sequence of length 2n under the
block-diffusion mask, forward and backward, in hand-written tcgen05/TMA CUDA
kernels behind the C ABI of ``libdfa.so`` (``include/dfa.h``).  PyTorch only
provides device memory, streams and autograd plumbing.

    from block_diffusion_masked_gb300 import diffusion_attn_func
    out = diffusion_attn_func(q, k, v, block_size=4)  # (batch, 2n, heads, headdim) bf16

Sampling, block by block, over a paged 8-bit cache of the finished tokens:

    from block_diffusion_masked_gb300 import KVCache, PageTable, rotary_func, rotary_table
    pages = PageTable(batch, max_pages, num_pages, page_size)
    cache = KVCache(num_pages, page_size, kv_heads, headdim)   # one per layer
    step = pages.plan(new_lens, rows, max_new)                 # one per step
    q, k = rotary_func(q, k, table, step.positions)            # packed rows
    out, lse = cache.attend(q, step, k, v, block_size)
    cache.append(k, v, step)                                   # the block is finished
    pages.advance(step)

The binding is imported lazily so that ``inputs`` can be used without CUDA.
"""

from __future__ import annotations

__all__ = ["diffusion_attn_func", "diffusion_attn_varlen_func", "causal_attn_func",
           "rotary_func", "rotary_table", "PageTable", "KVCache", "binding"]


def __getattr__(name):
    import importlib

    if name in ("rotary_table", "PageTable", "KVCache"):
        return getattr(importlib.import_module(__name__ + ".sampling"), name)
    if name in ("diffusion_attn_func", "diffusion_attn_varlen_func", "causal_attn_func",
                "rotary_func", "DiffusionAttnFunc", "DiffusionAttnVarlenFunc", "CausalAttnFunc",
                "RotaryFunc"):
        return getattr(importlib.import_module(__name__ + ".autograd"), name)
    if name in ("binding", "autograd", "inputs", "build", "sampling"):
        return importlib.import_module(__name__ + "." + name)
    raise AttributeError(name)

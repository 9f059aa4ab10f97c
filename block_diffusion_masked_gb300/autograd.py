"""torch.autograd wrappers over the C ABI (the pages' ``diffusion_attn_func``).

``diffusion_attn_func(q, k, v, block_size)`` mirrors the API of "Fast
Diffusion Attention" (section "Try it"): q, k, v are (batch, 2n, heads,
headdim) bf16 tensors ordered [noisy | clean] (k and v may carry fewer
heads, a divisor of q's: grouped-query / multi-query attention, query head h
reading key/value head h // (heads // kv_heads)); the forward saves out and the
log-sum-exp, and the backward recomputes from them (section 4.5 of
"FlashAttention: Exact Attention Without Materialization").
"""

from __future__ import annotations

import torch
import torch.autograd.forward_ad as forward_ad

from . import binding


def _strided(t):
    """t itself where the kernels can read its strides (heads of whole 16-byte
    pieces), else a contiguous copy."""
    if t.data_ptr() % 16 == 0:
        if t.is_contiguous():
            return t
        s = t.stride()
        if s[-1] == 1 and not any([x & 7 for x in s[:-1]]):
            return t
    return t.clone(memory_format=torch.contiguous_format)


def _followed():
    """Whether autograd follows what is computed: backward, or with tangents."""
    return torch.is_grad_enabled() or forward_ad._current_level >= 0


class RotaryFunc(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, table, positions, period, flags):
        ctx.set_materialize_grads(False)
        ctx.save_for_backward(table, positions)
        ctx.save_for_forward(table, positions)
        sizes = binding._rotary_sizes(q, k, table, positions, period)
        ctx.how, ctx.has_k = (sizes, flags), k is not None
        return binding._rotary_launch(q, k, table, positions, sizes, flags)

    @staticmethod
    def jvp(ctx, tq, tk, *_):
        # The map is linear: a tangent turns as its input does, or stays zero.
        table, positions = ctx.saved_tensors
        (_, _, period, heads, kv_heads, d, _, _), flags = ctx.how
        if tq is None:
            yq = tk.new_zeros((*tk.shape[:-2], heads, d))
            return yq, RotaryFunc.apply(_strided(tk), None, table, positions, period, flags)[0]
        yq, yk = RotaryFunc.apply(_strided(tq), None if tk is None else _strided(tk), table,
                                  positions, period, flags)
        if tk is None and ctx.has_k:
            yk = tq.new_zeros((*tq.shape[:-2], kv_heads, d))
        return yq, yk

    @staticmethod
    def backward(ctx, dq, dk):
        # Gradients have the outputs' shapes and types, checked in the forward.
        table, positions = ctx.saved_tensors
        sizes, flags = ctx.how
        flags ^= binding.DFA_ROTARY_INVERSE
        if not ctx.needs_input_grad[0]:
            dq = None
        if not ctx.needs_input_grad[1]:
            dk = None
        if _followed():  # the gradients are to have gradients: linear again
            if dq is not None:
                dq, dk = RotaryFunc.apply(_strided(dq), None if dk is None else _strided(dk),
                                          table, positions, sizes[2], flags)
            elif dk is not None:
                dk = RotaryFunc.apply(_strided(dk), None, table, positions, sizes[2], flags)[0]
        elif dq is not None:
            dq, dk = binding._rotary_launch(_strided(dq), None if dk is None else _strided(dk),
                                            table, positions,
                                            sizes if dk is not None else (*sizes[:4], 0, *sizes[5:]),
                                            flags)
        elif dk is not None:
            sizes = (*sizes[:3], sizes[4], 0, *sizes[5:])
            dk = binding._rotary_launch(_strided(dk), None, table, positions, sizes, flags)[0]
        return dq, dk, None, None, None, None


def rotary_func(q, k, table, positions=None, interleaved=False, period=None):
    """Rotary positions of queries and keys; differentiable, backward and with
    tangents (``torch.autograd.forward_ad``).

    q (B, L, H, d) and k (B, L, Hk, d), or packed (rows, heads, d) with
    ``positions`` (rows,); bf16, strided views (the slices of a fused
    projection) are read in place.  k may be None.  ``table``: see
    :func:`rotary_table`.  ``positions``: int32, a negative one marks a row
    that is not in use (its output is 0).  Without positions row r has
    position r mod ``period``; the default period L // 2 is the [noisy |
    clean] layout, both halves counted from 0.  ``table`` gets no gradient.  A
    backward pass is captured into a CUDA graph only while no eager graph of
    the same leaves is alive (a rule of autograd's, for any function).
    """
    q = _strided(q)
    if k is not None:
        k = _strided(k)
    flags = binding.DFA_ROTARY_CLEAR | (binding.DFA_ROTARY_INTERLEAVED if interleaved else 0)
    if forward_ad._current_level >= 0 or torch.is_grad_enabled() and (
            q.requires_grad or (k is not None and k.requires_grad)):
        return RotaryFunc.apply(q, k, table, positions, period, flags)
    return binding._rotary_launch(q, k, table, positions,
                                  binding._rotary_sizes(q, k, table, positions, period), flags)


class DiffusionAttnFunc(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, block_size):
        q, k, v = (t.contiguous() for t in (q, k, v))
        if k.shape[2] == q.shape[2]:
            out, lse = binding.dfa_forward(q, k, v, block_size)
        else:
            out, lse = binding.dfa_forward_gqa(q, k, v, block_size)
        ctx.save_for_backward(q, k, v, out, lse)
        ctx.block_size = block_size
        return out

    @staticmethod
    def backward(ctx, dout):
        q, k, v, out, lse = ctx.saved_tensors
        bwd = binding.dfa_backward if k.shape[2] == q.shape[2] else binding.dfa_backward_gqa
        dq, dk, dv = bwd(q, k, v, out, dout.contiguous(), lse, ctx.block_size)
        return dq, dk, dv, None


class CausalAttnFunc(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v):
        q, k, v = (t.contiguous() for t in (q, k, v))
        out, lse = binding.dfa_causal_forward(q, k, v)
        ctx.save_for_backward(q, k, v, out, lse)
        return out

    @staticmethod
    def backward(ctx, dout):
        q, k, v, out, lse = ctx.saved_tensors
        dq, dk, dv = binding.dfa_causal_backward(q, k, v, out, dout.contiguous(), lse)
        return dq, dk, dv


class DiffusionAttnVarlenFunc(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, cu_seqlens, block_size):
        q, k, v = (t.contiguous() for t in (q, k, v))
        cu = [int(x) for x in (cu_seqlens.tolist() if isinstance(cu_seqlens, torch.Tensor)
                               else cu_seqlens)]
        out, lse = binding.dfa_forward_varlen(q, k, v, cu, block_size)
        ctx.save_for_backward(q, k, v, out, lse)
        ctx.cu = cu
        ctx.block_size = block_size
        return out

    @staticmethod
    def backward(ctx, dout):
        q, k, v, out, lse = ctx.saved_tensors
        dq, dk, dv = binding.dfa_backward_varlen(q, k, v, out, dout.contiguous(), lse, ctx.cu,
                                                 ctx.block_size)
        return dq, dk, dv, None, None


def diffusion_attn_varlen_func(q, k, v, cu_seqlens, block_size, rotary_table=None,
                               positions=None, interleaved=False):
    """Block-diffusion attention on a packed batch (the pages' varlen API).

    q: (rows, heads, headdim), k, v: (rows, kv_heads, headdim) bf16; sample b
    is rows [cu_seqlens[b], cu_seqlens[b+1]), [noisy | clean], even length.
    ``rotary_table`` with ``positions`` (int32 (rows,)): q and k get rotary
    positions first (:func:`rotary_func`).
    """
    if rotary_table is not None:
        q, k = rotary_func(q, k, rotary_table, positions, interleaved)
    elif positions is not None:
        raise ValueError("positions need a rotary_table")
    return DiffusionAttnVarlenFunc.apply(q, k, v, cu_seqlens, block_size)


def diffusion_attn_func(q, k, v, block_size, rotary_table=None, interleaved=False):
    """Attention under the block-diffusion mask; differentiable.

    ``rotary_table``: q and k get rotary positions first, 0 .. n - 1 in either
    half (:func:`rotary_func`).
    """
    if rotary_table is not None:
        q, k = rotary_func(q, k, rotary_table, interleaved=interleaved)
    return DiffusionAttnFunc.apply(q, k, v, block_size)


def causal_attn_func(q, k, v, rotary_table=None, interleaved=False):
    """Causal attention on (Bc, L, H, d), any Bc; the yardstick kernels.

    ``rotary_table``: q and k get rotary positions 0 .. L - 1 first.
    """
    if rotary_table is not None:
        q, k = rotary_func(q, k, rotary_table, interleaved=interleaved, period=max(q.shape[1], 1))
    return CausalAttnFunc.apply(q, k, v)

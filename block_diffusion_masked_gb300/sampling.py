"""Sampling block by block: rotary tables, page tables, the 8-bit and 4-bit caches.

A block-diffusion sampler denoises one block of tokens at a time against the
clean tokens of the blocks before it ("Fast Diffusion Attention", "Block
diffusion in one picture": a block sees itself and the earlier clean blocks).
``PageTable`` holds the requests' pages and lengths, shared by all layers;
``KVCache`` holds one layer's keys and values in e4m3 with a power-of-two
scale per page and head, or in 4 bits with a scale per token and 32 dims.  All
state lives on the GPU and every step is a few launches of fixed shape, so a
step can be captured into a CUDA graph.
"""

from __future__ import annotations

import dataclasses
import math

import torch

from . import binding


def rotary_table(max_pos, rot_dim, base=10000.0, scaling=None, factor=1.0, original_max_pos=None,
                 beta_fast=32.0, beta_slow=1.0, device="cuda"):
    """Cosines and sines of positions 0 .. max_pos - 1: float32 (max_pos, rot_dim).

    Frequency i is base^(-2i / rot_dim); angles are computed in float64.
    ``scaling`` for contexts longer than those trained on, by ``factor``:

    * ``"linear"``: positions divided by ``factor``;
    * ``"base"``: base * factor^(rot_dim / (rot_dim - 2)), so that the lowest
      frequency is divided by ``factor`` and the highest is kept;
    * ``"parts"``: a frequency that turns more than ``beta_fast`` times within
      ``original_max_pos`` is kept, one that turns less than ``beta_slow`` times
      is divided by ``factor``, and the part that is divided grows linearly with
      i between (from the whole i below to the one above); cosines and sines are
      multiplied by 0.1 ln(factor) + 1.  After "YaRN: Efficient Context Window
      Extension of Large Language Models", sections 3.2 and 3.4, whose ramp is
      linear in the number of turns instead.
    """
    if max_pos < 1 or rot_dim < 16 or rot_dim % 16:
        raise ValueError("max_pos must be at least 1 and rot_dim a multiple of 16")
    if factor <= 0 or base <= 1:
        raise ValueError("factor must be positive and base above 1")
    i = torch.arange(rot_dim // 2, dtype=torch.float64, device=device)
    mult = 1.0
    if scaling == "base":
        base = base * factor ** (rot_dim / (rot_dim - 2))
    freq = base ** (-2.0 * i / rot_dim)
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "parts":
        if original_max_pos is None:
            raise ValueError("scaling 'parts' needs original_max_pos")

        def index_of(turns):  # the i whose frequency turns that often
            return rot_dim * math.log(original_max_pos / (turns * 2 * math.pi)) / \
                (2 * math.log(base))

        lo, hi = math.floor(index_of(beta_fast)), math.ceil(index_of(beta_slow))
        ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        freq = freq * (1 - ramp) + freq / factor * ramp
        mult = 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0
    elif scaling not in (None, "base"):
        raise ValueError("scaling must be None, 'linear', 'base' or 'parts'")
    angle = torch.arange(max_pos, dtype=torch.float64, device=device)[:, None] * freq
    return (torch.cat([angle.cos(), angle.sin()], 1) * mult).float()


@dataclasses.dataclass
class Step:
    """One sampling step's rows (see ``dfa_cache_plan``).

    ``cache_lens`` and ``block_table`` are the page table's own tensors: a step
    is over once :meth:`PageTable.advance` or :meth:`PageTable.release` has run.
    """

    cu_new: torch.Tensor      # (batch + 1,) first row of each request
    positions: torch.Tensor   # (rows,), -1 behind the last request
    cache_lens: torch.Tensor  # (batch,) tokens held before the step
    block_table: torch.Tensor
    next_lens: torch.Tensor
    next_free: torch.Tensor
    missing: torch.Tensor     # (1,) pages that were not to be had
    max_new: int
    # the page table's turn at the plan, negative: at the advance; 0: not known,
    # for replays of a captured plan are not seen on the host
    turn: int = 0


def _capturing(t):
    return t.is_cuda and torch.cuda.is_current_stream_capturing()


class PageTable:
    """Pages and lengths of a batch of requests, on the GPU."""

    def __init__(self, batch, max_pages, num_pages, page_size=64, device="cuda"):
        dev = torch.device(device)
        if dev.index is None and dev.type == "cuda":
            dev = torch.device("cuda", torch.cuda.current_device())
        i32 = dict(dtype=torch.int32, device=dev)
        self.page_size = page_size
        self.block_table = torch.full((batch, max_pages), -1, **i32)
        self.cache_lens = torch.zeros(batch, **i32)
        self.free_pages = torch.arange(num_pages, **i32).flip(0).contiguous()
        self.free_count = torch.full((1,), num_pages, **i32)
        self._turn = 1  # counts what makes planned steps stale: advance, release

    def plan(self, new_lens, rows, max_new):
        """Pages and positions for ``new_lens`` (int32 (batch,)) more tokens in
        ``rows`` packed rows; no request adds more than ``max_new``.  The same
        step may be planned again until :meth:`advance`."""
        got = binding.dfa_cache_plan(self.cache_lens, new_lens, self.block_table, self.free_pages,
                                     self.free_count, self.page_size, rows)
        table, cu_new, positions, next_lens, next_free, missing = got
        return Step(cu_new, positions, self.cache_lens, table, next_lens, next_free, missing,
                    max_new, 0 if _capturing(new_lens) else self._turn)

    def advance(self, step):
        """The step's tokens are in the caches: they count as held from now on.
        Copied in place, so captured graphs see the new lengths.

        A step that was planned before the last :meth:`advance` or :meth:`release`
        is refused: its lengths and free pages are not the table's any more.  Not
        so the step of a plan that was captured into a graph, which each replay
        plans anew: there a release between the plan's replay and the advance
        loses pages."""
        if step.turn != -self._turn:  # not the one whose advance came last
            if step.turn not in (0, self._turn):
                raise ValueError("the step was planned before the last advance or release: "
                                 "plan it again")
            self._turn += 1
            if step.turn:
                step.turn = -self._turn
        self.cache_lens.copy_(step.next_lens)
        self.free_count.copy_(step.next_free)

    def release(self, finished):
        """Requests with finished != 0 (int32 (batch,)) give their pages back.
        Steps that are planned and not advanced are over: plan them again."""
        self._turn += 1
        binding.dfa_cache_release(finished, self.cache_lens, self.block_table, self.free_pages,
                                  self.free_count, self.page_size)


class KVCache:
    """One layer's keys and values: pages of 8 or 4 bits a value.

    ``bits=8``: k, v e4m3 (pages, kv_heads, page_size, headdim), k_scale, v_scale
    float32 (pages, kv_heads), a power-of-two scale for each page and head.
    ``bits=4``: k, v uint8 (pages, kv_heads, page_size, headdim / 2), k_scale, v_scale
    float8_e5m2 (pages, kv_heads, headdim / 32, page_size), a scale for each token, head
    and 32 dims (``dfa_cache4_append``): 4.25 bits a value, an error of up to 5/64 of the
    largest of the 32 values (an 8th for one of the other sign), where that is within
    2^-11 and 7168.
    """

    def __init__(self, num_pages, page_size, kv_heads, headdim, device="cuda", bits=8):
        if bits not in (4, 8):
            raise ValueError("bits must be 4 or 8")
        self.bits = bits
        shape = (num_pages, kv_heads, page_size, headdim * bits // 8)
        self.k, self.v = (torch.zeros(shape, dtype=torch.uint8, device=device) for _ in range(2))
        if bits == 8:
            self.k, self.v = (x.view(torch.float8_e4m3fn) for x in (self.k, self.v))
            self.k_scale, self.v_scale = (
                torch.ones(shape[:2], dtype=torch.float32, device=device) for _ in range(2))
        else:
            scales = (num_pages, kv_heads, headdim // 32, page_size)
            self.k_scale, self.v_scale = (
                torch.zeros(scales, dtype=torch.uint8, device=device).view(torch.float8_e5m2)
                for _ in range(2))

    def append(self, k, v, step):
        """Keep the step's tokens: k, v packed (rows, kv_heads, headdim) bf16."""
        append = binding.dfa_cache_append if self.bits == 8 else binding.dfa_cache4_append
        append(k, v, step.cu_new, step.cache_lens, step.block_table, self.k,
               self.v, self.k_scale, self.v_scale, step.max_new)

    def attend(self, q, step, k=None, v=None, block_size=1, **kwargs):
        """Attention of the step's rows over the tokens held before it and, with
        k and v, over their own blocks; returns (out, lse), detached from autograd
        (``dfa_cache_forward``, ``dfa_cache4_forward``)."""
        forward = binding.dfa_cache_forward if self.bits == 8 else binding.dfa_cache4_forward
        return forward(q, self.k, self.v, self.k_scale, self.v_scale,
                       step.block_table, step.cache_lens, step.cu_new,
                       step.max_new, k=k, v=v, block_size=block_size, **kwargs)

    def read(self, pages, cu_rows, rows, first=None, **kwargs):
        """Tokens that ``pages`` (a :class:`PageTable`) counts as held, as the cache
        holds them: request b's from first[b] (None: 0) on, in rows [cu_rows[b],
        cu_rows[b + 1]) of k, v (rows, kv_heads, headdim) bf16 (``dfa_cache_read``).
        A 4-bit cache that they are appended to again may round them once more."""
        read = binding.dfa_cache_read if self.bits == 8 else binding.dfa_cache4_read
        return read(self.k, self.v, self.k_scale, self.v_scale, pages.block_table,
                    pages.cache_lens, cu_rows, rows, first=first, **kwargs)

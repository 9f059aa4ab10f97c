"""Sampling operators on the host: refusals of the C ABI before any launch,
the arithmetic the kernels share, rotary tables, and the oracle's own pins."""

import ctypes
import math

import numpy as np
import pytest
import torch

from block_diffusion_masked_gb300 import build as build_mod
from oracle import sampling as osam


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    from block_diffusion_masked_gb300 import binding

    return binding.lib()


P, NULL, ODD = ctypes.c_void_p(0x1000), None, ctypes.c_void_p(0x1008)
EINVAL, EUNSUPPORTED = -1, -2


def _rotary(lib, **kw):
    a = dict(q=P, k=P, qo=P, ko=P, table=P, pos=NULL, batch=1, rows=8, period=4, heads=2,
             kv_heads=2, headdim=64, rot=64, max_pos=4, qs=NULL, ks=NULL, flags=0)
    a.update(kw)
    return lib.dfa_rotary(*a.values(), NULL)


def test_rotary_refusals(lib):
    for kw in (dict(q=NULL), dict(k=NULL), dict(qo=NULL), dict(ko=ODD), dict(q=ODD),
               dict(table=NULL), dict(table=ODD), dict(batch=-1), dict(rows=-1), dict(heads=-1),
               dict(heads=0, kv_heads=0), dict(rot=0), dict(rot=24), dict(rot=80), dict(max_pos=0),
               dict(max_pos=3), dict(period=0), dict(flags=8),
               dict(pos=ctypes.c_void_p(0x1002)),
               dict(qs=(ctypes.c_longlong * 3)(64, 12, 8))):
        assert _rotary(lib, **kw) == EINVAL, kw
    for d in (0, 32, 96, 512):
        assert _rotary(lib, headdim=d) == EUNSUPPORTED
    assert _rotary(lib, batch=0) == 0 and _rotary(lib, rows=0) == 0


def _plan(lib, **kw):
    a = dict(lens=P, new=P, table=P, free=P, count=P, cu=P, pos=P, nxt=P, nfree=P, missing=P,
             batch=2, max_pages=4, num_free=8, ps=64, rows=8)
    a.update(kw)
    return lib.dfa_cache_plan(*a.values(), NULL)


def test_plan_and_release_refusals(lib):
    bad = ctypes.c_void_p(0x1002)
    for kw in (dict(lens=NULL), dict(new=NULL), dict(table=NULL), dict(free=NULL),
               dict(count=NULL), dict(cu=NULL), dict(pos=NULL), dict(nxt=NULL), dict(nfree=NULL),
               dict(missing=NULL), dict(batch=-1), dict(max_pages=0), dict(num_free=-1),
               dict(ps=48), dict(ps=0), dict(ps=256), dict(rows=-1),
               dict(max_pages=1 << 25, ps=64), dict(lens=bad), dict(pos=bad)):
        assert _plan(lib, **kw) == EINVAL, kw
    rel = lambda *a: lib.dfa_cache_release(*a, NULL)  # noqa: E731
    assert rel(P, P, P, P, NULL, 2, 4, 8, 64) == EINVAL
    assert rel(P, P, P, P, P, 2, 4, 8, 20) == EINVAL
    assert rel(P, P, bad, P, P, 2, 4, 8, 64) == EINVAL
    assert rel(P, P, P, P, P, 0, 4, 8, 64) == 0


def _append(lib, **kw):
    a = dict(k=P, v=P, cu=P, lens=P, table=P, kc=P, vc=P, ks=P, vs=P, batch=2, rows=8, max_new=4,
             heads=2, d=64, ps=16, pages=4, maxp=2, kst=NULL, vst=NULL)
    a.update(kw)
    return lib.dfa_cache_append(*a.values(), NULL)


def test_append_refusals(lib):
    for kw in (dict(k=NULL), dict(v=ODD), dict(cu=NULL), dict(lens=NULL), dict(table=NULL),
               dict(kc=NULL), dict(vc=ODD), dict(ks=NULL), dict(vs=NULL), dict(batch=-1),
               dict(rows=-1), dict(max_new=-1), dict(heads=0), dict(heads=65536), dict(ps=24),
               dict(pages=0), dict(maxp=0), dict(kst=(ctypes.c_longlong * 2)(128, 65)),
               dict(vst=(ctypes.c_longlong * 2)(100, 64)),
               dict(batch=20000, rows=1 << 21, max_new=1 << 21, heads=8)):  # too many blocks
        assert _append(lib, **kw) == EINVAL, kw
    assert _append(lib, d=96) == EUNSUPPORTED
    for kw in (dict(batch=0), dict(rows=0), dict(max_new=0)):
        assert _append(lib, **kw) == 0


def _forward(lib, **kw):
    a = dict(q=P, k=P, v=P, kc=P, vc=P, ks=P, vs=P, table=P, lens=P, cu=P, out=P, lse=P, work=P,
             nwork=1 << 40, batch=2, rows=8, max_new=4, heads=4, kv_heads=2, d=64, bs=4, ps=16,
             pages=4, maxp=2, qst=NULL, kst=NULL, vst=NULL)
    a.update(kw)
    return lib.dfa_cache_forward(*a.values(), NULL)


def test_forward_refusals(lib):
    for kw in (dict(q=NULL), dict(k=NULL), dict(v=NULL), dict(k=ODD), dict(kc=NULL), dict(vc=ODD),
               dict(ks=NULL), dict(vs=NULL), dict(table=NULL), dict(lens=NULL), dict(cu=NULL),
               dict(out=ODD), dict(lse=NULL), dict(work=ODD), dict(batch=-1),
               dict(batch=40000), dict(rows=-1), dict(max_new=-1), dict(heads=0),
               dict(kv_heads=3), dict(kv_heads=0), dict(kv_heads=8), dict(bs=0), dict(ps=8),
               dict(pages=0), dict(maxp=0), dict(maxp=1 << 27),
               dict(heads=1 << 16, kv_heads=1, rows=1 << 15, max_new=1 << 15)):
        assert _forward(lib, **kw) == EINVAL, kw
    assert _forward(lib, d=80) == EUNSUPPORTED
    for kw in (dict(batch=0), dict(rows=0), dict(max_new=0)):
        assert _forward(lib, **kw) == 0
    assert lib.dfa_cache_workspace_bytes(1, 8, 8, 4, 3, 64, 16, 2) == EINVAL
    assert lib.dfa_cache_workspace_bytes(1, 8, 8, 4, 2, 64, 24, 2) == EINVAL
    assert lib.dfa_cache_workspace_bytes(1, 8, 8, 4, 2, 72, 16, 2) == EUNSUPPORTED
    assert lib.dfa_cache_workspace_bytes(0, 8, 8, 4, 2, 64, 16, 2) == 0


def test_binding_refusals():
    """Wrong types, shapes and devices are refused before the library is asked."""
    from block_diffusion_masked_gb300 import binding as b
    from block_diffusion_masked_gb300 import diffusion_attn_varlen_func, rotary_func

    x = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    t = torch.zeros(4, 64)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        b.dfa_rotary(x, x, t)  # not on a GPU
    with pytest.raises(ValueError):
        rotary_func(x[0], x[0], t)  # packed rows need positions
    with pytest.raises(ValueError):
        diffusion_attn_varlen_func(x[0], x[0], x[0], i, 1, positions=i)  # without a table
    with pytest.raises(ValueError):
        b.dfa_cache_plan(i, i, torch.zeros(2, 2, dtype=torch.int32), i, i[:1], 64, 4)
    with pytest.raises(ValueError):
        b.dfa_cache_release(i, i, torch.zeros(2, 2, dtype=torch.int32), i, i[:1], 64)
    with pytest.raises(ValueError):
        b.dfa_cache_append(x[0], x[0], i, i, i, x, x, t, t, 1)
    with pytest.raises(ValueError):
        b.dfa_cache_forward(x[0], x, x, t, t, i, i, i, 1)


# ------------------------------------------------------------- shared arithmetic

def test_scale_exponent(lib):
    """Every bf16 magnitude against the definition."""
    bits = np.arange(0, 0x7f80, dtype=np.uint32)
    mag = (bits << 16).view(np.float32).astype(np.float64)
    for b, m in list(zip(bits.tolist(), mag.tolist()))[::7] + [(0x43e0, 448.0), (0x43e1, 450.0)]:
        e = lib.dfa_cache_scale_exp(b)
        assert m <= 448.0 * 2.0 ** e
        assert e == osam.MIN_EXP or m > 448.0 * 2.0 ** (e - 1)


def test_page_numbers(lib):
    ok = lambda p, n: lib.dfa_cache_page_ok(p, n)  # noqa: E731
    assert ok(0, 1) and ok(6, 7)
    for page, n in ((-1, 7), (7, 7), (2 ** 31 - 1, 7), (-2 ** 31, 7), (0, 0)):
        assert not ok(page, n)


@pytest.mark.parametrize("ps", [16, 32, 64, 128])
def test_append_spans(lib, ps):
    """The spans of the touched pages are the new tokens, page by page."""
    span = (ctypes.c_int * 2)()
    for length in (0, 1, ps - 1, ps, ps + 1, 5 * ps + 3, 2 ** 30 - 1):
        for n in (0, 1, 2, ps - 1, ps, ps + 1, 3 * ps + 2):
            got = []
            for j in range(lib.dfa_cache_append_pages(n, ps) + 1):
                assert lib.dfa_cache_append_span(length, n, j, ps, span) == 0
                if span[0] < span[1]:
                    page = length // ps + j
                    assert page * ps <= span[0] and span[1] <= (page + 1) * ps
                    got += range(span[0], span[1])
            assert got == list(range(length, length + n))


def test_runs_share_the_units(lib):
    """Blocks' runs are equal to within a unit, cover all units in order, and
    name their owners."""
    g = np.random.default_rng(0)
    for _ in range(200):
        B, limit = int(g.integers(1, 70)), int(g.integers(1, 400))
        lens = (2.0 ** g.uniform(0, 17, B)).astype(int) * (g.random(B) < 0.9)
        rows = (g.random(B) < 0.9).astype(int)
        units = [lib.dfa_cache_units(int(n), int(r), 128, 3) for n, r in zip(lens, rows)]
        assert units == [r * (3 - -int(n) // 128) for n, r in zip(lens, rows)]
        total = sum(units) * int(g.integers(1, 9))
        blocks = lib.dfa_cache_blocks(total, limit)
        if total == 0:
            assert blocks == 0
            continue
        assert blocks == min(limit, total)
        ends = [lib.dfa_cache_run(x, total, blocks) for x in range(blocks + 1)]
        assert ends[0] == 0 and ends[-1] == total
        sizes = np.diff(ends)
        assert sizes.min() >= 1 and sizes.max() - sizes.min() <= 1
        for w in {0, total - 1, *g.integers(0, total, 20).tolist(), *ends[:-1][::7]}:
            x = lib.dfa_cache_owner(w, total, blocks)
            assert ends[x] <= w < ends[x + 1]
    # 64-bit products: a batch of 32768 requests of 2^30 keys, 256 heads
    total = 32768 * 2 ** 23 * 256
    ends = [lib.dfa_cache_run(x, total, 304) for x in (0, 1, 303, 304)]
    assert ends == [x * total // 304 for x in (0, 1, 303, 304)]
    assert lib.dfa_cache_owner(total - 1, total, 304) == 303
    assert lib.dfa_cache_units(2 ** 30, 1, 128, 3) == 2 ** 23 + 3
    assert lib.dfa_cache_units(500, 4, 0, 1) == 1 and lib.dfa_cache_units(500, 0, 0, 1) == 0


def test_own_block_ends(lib):
    for length, n, bs in ((0, 7, 4), (3, 9, 4), (8, 4, 4), (5, 6, 1), (7, 5, 100),
                          (2 ** 30 - 8, 8, 3)):
        for i in range(n):
            want = sum((length + j) // bs <= (length + i) // bs for j in range(n))
            assert lib.dfa_cache_own_end(length, i, n, bs) == want


# ------------------------------------------------------------- rotary tables

def test_rotary_tables():
    from block_diffusion_masked_gb300 import rotary_table

    t = rotary_table(1000, 32, base=10000.0, device="cpu")
    for pos, i in ((0, 0), (1, 3), (999, 15), (500, 7)):
        a = pos * 10000.0 ** (-2 * i / 32)
        # one rounding to float32 of a value at most 1
        assert abs(t[pos, i] - math.cos(a)) <= 2.0 ** -24
        assert abs(t[pos, 16 + i] - math.sin(a)) <= 2.0 ** -24
    assert torch.equal(rotary_table(64, 32, scaling="linear", factor=4.0, device="cpu")[::4][:16],
                       rotary_table(16, 32, device="cpu"))
    b = rotary_table(64, 32, scaling="base", factor=4.0, device="cpu")
    assert torch.equal(b[:, 0], rotary_table(64, 32, device="cpu")[:, 0])
    low = 10000.0 ** (-30 / 32) / 4.0  # the lowest frequency is divided by the factor
    assert abs(b[63, 31] - math.sin(63 * low)) <= 2.0 ** -24
    p = rotary_table(64, 128, scaling="parts", factor=8.0, original_max_pos=4096, device="cpu")
    m = 0.1 * math.log(8.0) + 1.0
    assert abs(p[1, 0] - m * math.cos(1.0)) <= 2.0 ** -23
    assert abs(p[63, 127] - m * math.sin(63 * 10000.0 ** (-126 / 128) / 8)) <= 2.0 ** -23
    for kw in (dict(max_pos=0, rot_dim=32), dict(max_pos=4, rot_dim=24), dict(max_pos=4, rot_dim=8),
               dict(max_pos=4, rot_dim=32, scaling="else"),
               dict(max_pos=4, rot_dim=32, scaling="parts"),
               dict(max_pos=4, rot_dim=32, factor=0.0)):
        with pytest.raises(ValueError):
            rotary_table(device="cpu", **kw)


# ------------------------------------------------------------- the oracle's pins

def test_oracle_e4m3_rounding_is_the_types():
    """All halfway points and neighbours against torch's float8 conversion."""
    vals = torch.arange(0, 0x7f, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    mids = (vals[1:] + vals[:-1]) / 2
    x = torch.cat([vals, mids, mids * (1 + 2.0 ** -20), mids * (1 - 2.0 ** -20)])
    x = torch.cat([x, -x])
    want = x.float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(osam.round_e4m3(x.numpy()), want)


def test_oracle_cache_attention_is_the_training_mask():
    """A sampler's step sees what the training mask shows a noisy block: its own
    block and the clean blocks before it; the exact cache (values that e4m3
    holds) reproduces the noisy rows of the training forward."""
    import oracle

    g = np.random.default_rng(3)
    n, bs, H, d, ps = 12, 4, 2, 4, 16
    clean = [np.clip(g.integers(-8, 9, (n, H, d)), -8, 8).astype(float) for _ in range(2)]
    noisy = [g.standard_normal((n, H, d)) for _ in range(3)]
    q = np.concatenate([noisy[0], np.zeros((n, H, d))])[None]
    k = np.concatenate([noisy[1], clean[0]])[None]
    v = np.concatenate([noisy[2], clean[1]])[None]
    ref, lse = oracle.diffusion_forward(q, k, v, bs)
    one = np.ones((1, H))
    cache = [np.zeros((1, H, ps, d)) for _ in range(2)]
    for start in range(0, n, bs):
        for c, x in zip(cache, clean):
            c[0, :, :start] = x[:start].transpose(1, 0, 2)
        sl = slice(start, start + bs)
        out, l2, _, _ = osam.cache_attention(noisy[0][sl], cache[0], cache[1], one, one, [[0]],
                                             [start], [0, bs], noisy[1][sl], noisy[2][sl], bs)
        assert np.abs(out - ref[0, sl]).max() < 1e-12
        assert np.abs(l2 - lse[0, :, sl]).max() < 1e-12


def test_forward_bounds_on_the_rows_of_a_request(lib):
    """The limit holds for the rows there can be, not for a loose bound on them.
    (Sizes are looked at before the head dimension, which is refused here.)"""
    for m in (1 << 24, (1 << 24) + 1, (1 << 31) - 1):
        assert _forward(lib, max_new=m, d=80) == EUNSUPPORTED
        assert lib.dfa_cache_workspace_bytes(1, 8, m, 4, 2, 72, 16, 2) == EUNSUPPORTED
    for rows, m in (((1 << 24) + 1, (1 << 24) + 1), (1 << 30, (1 << 31) - 1)):
        assert _forward(lib, heads=1, kv_heads=1, rows=rows, max_new=m, d=80) == EINVAL
        assert lib.dfa_cache_workspace_bytes(1, rows, m, 1, 1, 72, 16, 2) == EINVAL


# ------------------------------------------------------------- steps of a page table

def test_stale_steps_are_refused(monkeypatch):
    """advance takes over a plan's lengths and free pages, so nothing may have
    changed them since: a release, or another step's advance."""
    from block_diffusion_masked_gb300 import PageTable, sampling

    def plan(lens, new, table, free, count, ps, rows):
        return table, None, None, lens + new, count - 1, None

    calls = []
    monkeypatch.setattr(sampling.binding, "dfa_cache_plan", plan)
    monkeypatch.setattr(sampling.binding, "dfa_cache_release", lambda *a: calls.append(a))
    pages = PageTable(2, 4, 8, 16, device="cpu")
    new = torch.tensor([3, 1], dtype=torch.int32)
    step = pages.plan(new, 4, 3)
    again = pages.plan(new, 4, 3)  # the same step may be planned again
    pages.advance(again)
    pages.advance(again)           # and advanced again: nothing changes
    assert pages.cache_lens.tolist() == [3, 1] and pages.free_count.item() == 7
    with pytest.raises(ValueError):
        pages.advance(step)
    step = pages.plan(new, 4, 3)
    pages.release(new)
    assert len(calls) == 1
    for stale in (step, again):
        with pytest.raises(ValueError):
            pages.advance(stale)
    assert pages.cache_lens.tolist() == [3, 1] and pages.free_count.item() == 7
    pages.advance(pages.plan(new, 4, 3))
    assert pages.cache_lens.tolist() == [6, 2] and pages.free_count.item() == 6


# ------------------------------------------------------------- the rotary autograd function

@pytest.mark.parametrize("frozen", ["q", "k", None])
def test_rotary_backward_leaves_frozen_inputs_out(monkeypatch, frozen):
    """No gradient is read or written for an input that needs none."""
    from block_diffusion_masked_gb300 import autograd

    launches = []

    def launch(q, k, table, positions, sizes, flags):
        launches.append((tuple(q.shape), None if k is None else tuple(k.shape), sizes[3:5]))
        return q.clone(), None if k is None else k.clone()

    monkeypatch.setattr(autograd.binding, "_rotary_sizes",
                        lambda q, k, *a: (1, 4, 2, q.shape[2], k.shape[2], 64, 64, 2))
    monkeypatch.setattr(autograd.binding, "_rotary_launch", launch)
    q, k = (torch.randn(1, 4, h, 64, dtype=torch.bfloat16).requires_grad_() for h in (3, 1))
    if frozen:
        (q if frozen == "q" else k).requires_grad_(False)
    yq, yk = autograd.rotary_func(q, k, torch.zeros(2, 64))
    (yq.sum() + yk.sum()).backward()
    assert (q.grad is None) == (frozen == "q") and (k.grad is None) == (frozen == "k")
    assert len(launches) == 2
    shapes, heads = launches[1][:2], launches[1][2]
    if frozen is None:
        assert shapes == (q.shape, k.shape) and heads == (3, 1)
    else:
        x = k if frozen == "q" else q
        assert shapes == (x.shape, None) and heads == (x.shape[2], 0)


def test_arguments_past_32_bits():
    """They are not wrapped to arguments that would be taken."""
    from block_diffusion_masked_gb300 import binding as b

    assert b._int32(2 ** 32 + 5) == b._int32(2 ** 40) == 2 ** 31 - 1
    assert b._int32(-2 ** 32 + 5) == b._int32(-2 ** 40) == -1 and b._int32(7) == 7
    good = [1, 8, 8, 4, 2, 64, 16, 2]
    for i, x in ((0, -2 ** 32 + 1), (1, 2 ** 32 + 8), (2, -2 ** 32 + 8), (3, 2 ** 32 + 4),
                 (4, 2 ** 32 + 2), (6, 2 ** 32 + 16), (7, 2 ** 32 + 2)):
        bad = list(good)
        bad[i] = x
        with pytest.raises(b.DfaError) as e:
            b.dfa_cache_workspace_bytes(*bad)
        assert e.value.code == b.DFA_EINVAL, i


@pytest.mark.parametrize("base,rot,length", [(10000.0, 128, 131072), (10000.0, 64, 4096),
                                             (500000.0, 128, 8192), (10000.0, 32, 128)])
def test_rotary_table_by_parts(base, rot, length):
    """Kept, divided, or in between by the frequency's place between the two that
    turn beta_fast and beta_slow times: also where those lie outside the table.
    Tolerance: an angle below 2 in float64, one rounding to float32 of at most m."""
    from block_diffusion_masked_gb300 import rotary_table

    factor, m = 8.0, 0.1 * math.log(8.0) + 1.0
    t = rotary_table(2, rot, base=base, scaling="parts", factor=factor, original_max_pos=length,
                     device="cpu").double()
    place = [rot * math.log(length / (turns * 2 * math.pi)) / (2 * math.log(base))
             for turns in (32.0, 1.0)]
    lo, hi = math.floor(place[0]), math.ceil(place[1])
    between = 0
    for i in range(rot // 2):
        f = base ** (-2 * i / rot)
        turns = length * f / (2 * math.pi)
        part = min(max((i - lo) / (hi - lo), 0.0), 1.0)
        if turns >= 32 and i <= lo:
            assert part == 0
        if turns <= 1 and i >= hi:
            assert part == 1
        between += 0 < part < 1
        a = f * (1 - part) + f / factor * part
        assert abs(t[1, i] - m * math.cos(a)) <= 2.0 ** -23
        assert abs(t[1, rot // 2 + i] - m * math.sin(a)) <= 2.0 ** -23
    assert between


def test_captured_plans_are_not_refused(monkeypatch):
    """A replay plans anew without the host: the captured step may be advanced
    after every one, releases in between or not, and makes other steps stale."""
    from block_diffusion_masked_gb300 import PageTable, sampling

    def plan(lens, new, table, free, count, ps, rows):
        return table, None, None, lens + new, count - 1, None

    monkeypatch.setattr(sampling.binding, "dfa_cache_plan", plan)
    monkeypatch.setattr(sampling.binding, "dfa_cache_release", lambda *a: None)
    pages = PageTable(2, 4, 8, 16, device="cpu")
    new = torch.tensor([3, 1], dtype=torch.int32)
    with monkeypatch.context() as m:
        m.setattr(sampling, "_capturing", lambda t: True)
        captured = pages.plan(new, 4, 3)
    eager = pages.plan(new, 4, 3)
    pages.advance(captured)
    with pytest.raises(ValueError):
        pages.advance(eager)
    pages.release(new)
    captured.next_lens += new  # what a replay does
    pages.advance(captured)
    assert pages.cache_lens.tolist() == [6, 2]

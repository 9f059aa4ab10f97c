"""The sampling cache on the GPU: plan, release, append and attention against
the float64 definitions, and a sampler's steps run together.

Tolerance of the attention.  A score is a sum of d products of exact f16 (or
bf16) operands in float32: at most (d + 2) * 2^-23 of scale * sum |q k|
(truncating adds included), and the exponential and its argument's rounding
add 2^-20 (1 + |s|); both act as a relative error delta on the probabilities.
Cached probabilities are rounded to f16 (2^-11), own ones to bf16 (2^-8), so
the output is off by at most (2^-8 + 2 delta) sum p |v| plus its own rounding,
2^-8 of it; without own keys 2^-11 stands for the first 2^-8.  Probabilities
below 2^-30 of the largest may be lost: keys * 2^-30 max |v|.  lse: delta +
2^-22 |lse|.
"""

import numpy as np
import pytest
import torch

from oracle import sampling as osam

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.fixture(scope="module")
def b():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from block_diffusion_masked_gb300 import binding, build

    build.build()
    binding.lib()
    return binding


def _f64(t):
    return t.detach().float().cpu().double().numpy()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------ plan

@pytest.mark.parametrize("B,ps,longest,most", [
    (1, 16, 0, 1), (5, 64, 300, 16), (3, 128, 1000, 700), (40, 32, 200, 33), (700, 16, 50, 9),
    (1300, 32, 90, 5)])
@pytest.mark.parametrize("short", [False, True])
def test_plan(b, B, ps, longest, most, short):
    g = np.random.default_rng(B + ps + most)
    lens = g.integers(0, longest + 1, B)
    new = g.integers(0, most + 1, B)
    maxp = int(-(-(longest + most) // ps)) + 1
    need = int(sum(-(-(o + a) // ps) - -(-o // ps) for o, a in zip(lens, new)))
    count = max(0, need - 3) if short else need + 2
    free = g.permutation(count + 5)
    table = np.full((B, maxp), -1)
    for i, o in enumerate(lens):
        table[i, :-(-o // ps)] = 5000 + g.integers(0, 1000, -(-o // ps))
    rows = int(new.sum()) + 11
    t = _i32(table)
    args = (_i32(lens), _i32(new), t, _i32(free), _i32([count]), ps, rows)
    ref = osam.plan(lens, new, table, free, count, ps, rows)
    for _ in range(2):  # again on the same state: the same
        got = b.dfa_cache_plan(*args)
        assert b.dfa_status() == 0
        assert got[0] is t
        for x, y in zip(got, ref):
            assert np.array_equal(x.cpu().numpy().ravel(), np.ravel(y))


def test_plan_full_tables_and_cut_rows(b):
    # request 0 wants three pages more than its table has; eight rows do not fit
    t = _i32([[4, -1], [-1, -1]])
    got = b.dfa_cache_plan(_i32([10, 0]), _i32([60, 20]), t, _i32(range(9)), _i32([9]), 16, 100)
    assert b.dfa_status() == 0
    assert t.tolist() == [[4, 8], [7, 6]]
    assert got[3].tolist() == [32, 20] and got[4].item() == 6 and got[5].item() == 3
    t = _i32([[-1, -1], [-1, -1]])
    got = b.dfa_cache_plan(_i32([0, 0]), _i32([12, 20]), t, _i32(range(9)), _i32([9]), 16, 24)
    assert b.dfa_status() == b.DFA_EDEVICE
    assert got[1].tolist() == [0, 12, 24] and got[3].tolist() == [12, 12]
    assert got[2].tolist() == list(range(12)) * 2


def test_plan_cut_rows_take_no_pages(b):
    """Rows that are cut take no pages: after every step the pages held and the
    pages free are all the pages there are."""
    lens, new = [3, 16, 0] * 300, [20, 17, 40] * 300
    lens, new = lens[:700], new[:700]
    n = sum(-(-x // 16) for x in lens)
    table = np.full((700, 4), -1)
    at = 0
    for i, x in enumerate(lens):
        for j in range(-(-x // 16)):
            table[i, j] = at
            at += 1
    free = list(range(n, n + 3000))
    for rows in (0, 30, 5000, 14000, sum(new)):
        t = _i32(table)
        got = b.dfa_cache_plan(_i32(lens), _i32(new), t, _i32(free), _i32([3000]), 16, rows)
        assert b.dfa_status() == (0 if rows == sum(new) else b.DFA_EDEVICE)
        ref = osam.plan(lens, new, table, free, 3000, 16, rows)
        for x, y in zip(got, ref):
            assert np.array_equal(x.cpu().numpy().ravel(), np.ravel(y))
        held = sum(-(-x // 16) for x in got[3].tolist())
        assert held + got[4].item() == n + 3000


def test_plan_bad_state(b):
    """Lengths and counts outside their ranges are errors; nothing is read
    through them."""
    for lens, new, count in (([-1, 3], [2, 2], 4), ([3, 33], [2, 0], 4), ([3, 3], [-5, 2], 4),
                             ([3, 3], [2, 2], 99), ([3, 3], [2, 2], -1)):
        t = _i32([[0, -1], [1, -1]])
        b.dfa_cache_plan(_i32(lens), _i32(new), t, _i32(range(8)), _i32([count]), 16, 9)
        assert b.dfa_status() == b.DFA_EDEVICE
        assert int(t.max()) < 8 and int(t.min()) >= -1


def test_plan_empty(b):
    got = b.dfa_cache_plan(_i32([]), _i32([]), torch.empty(0, 3, dtype=torch.int32, device=DEV),
                           _i32([7]), _i32([1]), 64, 3)
    assert b.dfa_status() == 0
    assert [x.tolist() for x in got[1:]] == [[0], [-1, -1, -1], [], [1], [0]]


@pytest.mark.parametrize("B", [1, 17, 50])
def test_release(b, B):
    from block_diffusion_masked_gb300 import PageTable

    g = np.random.default_rng(B)
    pages = PageTable(B, 40, 40 * B, 16)
    new = _i32(g.integers(0, 600, B))
    step = pages.plan(new, 600 * B, 600)
    pages.advance(step)
    table, lens = pages.block_table.cpu().numpy().copy(), pages.cache_lens.tolist()
    done = g.random(B) < 0.5
    done[0] = True
    before = int(pages.free_count)
    stack = pages.free_pages[:before].tolist()
    pages.release(_i32(done.astype(int)))
    assert b.dfa_status() == 0
    for i in range(B):
        n = -(-lens[i] // 16)
        if done[i]:
            stack += table[i, :n].tolist()
            table[i, :n] = -1
            lens[i] = 0
    assert pages.free_pages[:int(pages.free_count)].tolist() == stack
    assert pages.cache_lens.tolist() == lens
    assert np.array_equal(pages.block_table.cpu().numpy(), table)
    assert len(set(stack)) == len(stack)


# ------------------------------------------------------------------ append

def _cache(P, Hk, ps, d, seed):
    g = torch.Generator("cpu").manual_seed(seed)
    x = torch.randn((P, Hk, ps, d), generator=g).clamp(-4, 4) * 64
    e = torch.randint(-12, -4, (P, Hk), generator=g)
    return x.to(torch.float8_e4m3fn).to(DEV), (2.0 ** e.double()).float().to(DEV)


def _requests(lens, new, ps, seed, spare=2):
    """A page table with pages in random order, and cu_new."""
    g = np.random.default_rng(seed)
    need = [-(-(o + a) // ps) for o, a in zip(lens, new)]
    perm = g.permutation(sum(need) + spare)
    table, at = np.full((len(lens), max(max(need), 1)), -1), 0
    for i, n in enumerate(need):
        table[i, :n] = perm[at:at + n]
        at += n
    return table, [0] + np.cumsum(new).tolist(), sum(need) + spare


@pytest.mark.parametrize("d,ps,Hk", [(64, 16, 1), (64, 128, 3), (128, 32, 2), (128, 64, 1),
                                     (256, 16, 2), (256, 128, 1)])
@pytest.mark.parametrize("lens,new", [
    ([0], [1]), ([15, 16, 17], [1, 1, 1]), ([0, 130, 5, 64], [70, 0, 3, 200]),
    ([127, 3], [129, 300])])
def test_append(b, d, ps, Hk, lens, new):
    table, cu, P = _requests(lens, new, ps, d + ps)
    kc, ks = _cache(P, Hk, ps, d, 1)
    vc, vs = _cache(P, Hk, ps, d, 2)
    rows = cu[-1] + 3  # three rows behind the last request
    g = torch.Generator("cpu").manual_seed(5)
    amp = torch.exp(2 * torch.randn((rows, Hk, 1), generator=g))
    kv = (torch.randn((2, rows, Hk, d), generator=g) * amp).to(torch.bfloat16)
    kv[0, 0, 0, 0], kv[1, -4, 0, 1] = 0.0, 2.0 ** -120
    # slices of one projection's output: strided rows and heads
    both = torch.stack([kv[0], kv[1]], 2).to(DEV)  # (rows, Hk, 2, d)
    k, v = both[:, :, 0], both[:, :, 1]
    refs = [osam.append(_f64(x), cu, lens, table, _f64(c), _f64(s))
            for x, c, s in ((k, kc, ks), (v, vc, vs))]
    for _ in range(2):  # the second time on the appended cache: nothing changes
        b.dfa_cache_append(k, v, _i32(cu), _i32(lens), _i32(table), kc, vc, ks, vs, max(new))
        assert b.dfa_status() == 0
        for (rc, rs), c, s in ((refs[0], kc, ks), (refs[1], vc, vs)):
            assert np.array_equal(_f64(s), rs)
            assert np.array_equal(_f64(c), rc)


def test_append_values_that_are_not_finite(b):
    """They are kept as NaN and do not count for the scale; zeros take the
    smallest scale, the largest bf16 the largest."""
    lens, new, ps, d = [0, 0, 0, 0], [3, 2, 2, 1], 16, 64
    table, cu, P = _requests(lens, new, ps, 3)
    kc, ks = _cache(P, 1, ps, d, 4)
    vc, vs = _cache(P, 1, ps, d, 5)
    x = torch.ones((8, 1, d), dtype=torch.bfloat16, device=DEV)
    x[0, 0, 3], x[1, 0, 4], x[2, 0, 5] = float("inf"), float("-inf"), float("nan")
    x[3:5] = 0
    x[5:7] = torch.finfo(torch.bfloat16).max
    x[7] = float("nan")
    rc, rs = osam.append(_f64(x), cu, lens, table, _f64(kc), _f64(ks))
    b.dfa_cache_append(x, x, _i32(cu), _i32(lens), _i32(table), kc, vc, ks, vs, 3)
    assert b.dfa_status() == 0
    assert np.array_equal(_f64(kc), rc, equal_nan=True) and np.array_equal(_f64(ks), rs)
    assert rs[table[1][0], 0] == 2.0 ** -100 and rs[table[2][0], 0] == 2.0 ** 120


@pytest.mark.parametrize("what", ["page", "negative page", "table", "order", "rows", "max_new",
                                  "length"])
def test_append_bad_tables(b, what):
    """One bad request is an error and left out; the other is appended."""
    d, ps = 64, 16
    lens, new = [4, 20], [5, 6]
    table, cu, P = _requests(lens, new, ps, 6)
    maxn = 6
    if what == "page":
        table[0, 0] = P
    elif what == "negative page":
        table[0, 0] = -3
    elif what == "table":
        lens[0] = 10 ** 6
    elif what == "order":
        cu = [7, 5, 11]
    elif what == "rows":
        cu, new, lens = [0, 6, 400], [6, 394], lens[::-1]
        table, maxn = table[::-1].copy(), 500
    elif what == "max_new":
        maxn = 5
    else:
        lens[0] = -1
    kc, ks = _cache(P, 1, ps, d, 7)
    vc, vs = _cache(P, 1, ps, d, 8)
    was = kc.clone()
    x = torch.randn((11, 1, d), device=DEV).bfloat16()
    b.dfa_cache_append(x, x, _i32(cu), _i32(lens), _i32(table), kc, vc, ks, vs, maxn)
    assert b.dfa_status() == b.DFA_EDEVICE
    bad = 1 if what in ("rows", "max_new") else 0
    good = 1 - bad
    page = table[good][lens[good] // ps]
    assert not torch.equal(kc[page].view(torch.uint8), was[page].view(torch.uint8))
    for p in set(range(P)) - set(table[good].tolist()):
        assert torch.equal(kc[p].view(torch.uint8), was[p].view(torch.uint8))


# ------------------------------------------------------------------ attention

def _problem(lens, new, H, Hk, d, ps, seed=0, tail=0, own=True):
    table, cu, P = _requests(lens, new, ps, seed)
    kc, ks = _cache(P, Hk, ps, d, seed + 1)
    vc, vs = _cache(P, Hk, ps, d, seed + 2)
    ks *= 4.0
    g = torch.Generator("cpu").manual_seed(seed + 3)
    rows = cu[-1] + tail
    q = torch.randn((rows, H, d), generator=g).to(torch.bfloat16).to(DEV)
    k, v = (torch.randn((rows, Hk, d), generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
    # behind the last token of a request: bytes that are not numbers
    for i, n in enumerate(lens):
        if n % ps:
            for c in (kc, vc):
                c.view(torch.uint8)[int(table[i, n // ps]), :, n % ps:] = 0x7F
    return dict(table=table, cu=cu, lens=lens, new=new, kc=kc, ks=ks, vc=vc, vs=vs, q=q,
                k=k if own else None, v=v if own else None)


def _run(b, p, bs, **kw):
    return b.dfa_cache_forward(p["q"], p["kc"], p["vc"], p["ks"], p["vs"], _i32(p["table"]),
                               _i32(p["lens"]), _i32(p["cu"]), max(p["new"]), k=p["k"], v=p["v"],
                               block_size=bs, **kw)


def _check(p, bs, out, lse):
    d, n = p["q"].shape[2], p["cu"][-1]
    own = p["k"] is not None
    ref, rl, absout, big = osam.cache_attention(
        _f64(p["q"]), _f64(p["kc"]), _f64(p["vc"]), _f64(p["ks"]), _f64(p["vs"]), p["table"],
        p["lens"], p["cu"], _f64(p["k"]) if own else None, _f64(p["v"]) if own else None, bs)
    delta = (d + 2) * 2.0 ** -23 * big + 2.0 ** -20 * (1 + big)  # (H, rows)
    vmax = 2.0 ** -30 * (max(p["lens"]) + 1) * float(
        (p["vc"].float().nan_to_num(0).abs().amax((2, 3)) * p["vs"]).max())
    tol = 2.0 ** -8 * np.abs(ref) + ((2.0 ** -8 if own else 2.0 ** -11)
                                     + 2 * delta.T[..., None]) * absout + vmax
    err = np.abs(_f64(out) - ref)[:n]
    assert np.isfinite(_f64(out)[:n]).all()
    assert (err <= tol[:n]).all(), float((err - tol[:n]).max())
    got, want = lse.cpu().double().numpy()[:, :n], rl[:, :n]
    none = np.isneginf(want)
    assert (np.isneginf(got) == none).all()
    off = np.abs(got - want)[~none]
    assert (off <= (delta[:, :n] + 2.0 ** -22 * np.abs(want))[~none]).all(), off.max()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens,new,H,Hk,ps,bs", [
    ([1], [1], 1, 1, 16, 1),
    ([0], [3], 2, 1, 32, 4),
    ([33], [4], 4, 1, 16, 4),
    ([31, 0, 200, 17], [4, 4, 0, 3], 8, 2, 32, 4),
    ([300, 64], [5, 9], 4, 4, 64, 3),
    ([129, 500, 1], [16, 7, 16], 4, 2, 128, 16),
    ([700, 90], [33, 12], 2, 1, 16, 64),
    ([260], [40], 6, 3, 64, 1),
    ([0, 128, 257], [9, 5, 16], 16, 2, 32, 4),
    ([1000, 3], [150, 70], 2, 1, 128, 50)])
def test_attention(b, d, lens, new, H, Hk, ps, bs):
    p = _problem(lens, new, H, Hk, d, ps, seed=d + ps)
    out, lse = _run(b, p, bs)
    assert b.dfa_status() == 0
    _check(p, bs, out, lse)


@pytest.mark.parametrize("d,G,T", [(64, 1, 2), (128, 4, 3), (128, 8, 4), (128, 4, 20), (256, 2, 11),
                                   (256, 4, 16), (64, 8, 8)])
def test_attention_split_over_chunks(b, d, G, T):
    """Long requests beside short ones: several chunks joined, others not."""
    p = _problem([3001, 40, 1030], [T, T, 1], 2 * G, 2, d, 64, seed=G + T)
    out, lse = _run(b, p, T)
    assert b.dfa_status() == 0
    _check(p, T, out, lse)


@pytest.mark.parametrize("longest", [500, 1000])
@pytest.mark.parametrize("B,H,T", [(1, 4, 1), (80, 4, 1), (40, 16, 5), (3, 16, 20)])
def test_attention_short_tables(b, B, H, T, longest):
    """Tables of a few pages, few and many segments: whole segments and cut ones."""
    g = np.random.default_rng(B + longest)
    lens = g.integers(0, longest + 1, B).tolist()
    lens[0] = longest
    p = _problem(lens, [T] * B, H, 4, 64, 16, seed=B)
    out, lse = _run(b, p, 8)
    assert b.dfa_status() == 0
    _check(p, 8, out, lse)


@pytest.mark.parametrize("B,d,H,Hk,T", [(2100, 64, 2, 1, 1), (700, 128, 4, 1, 3),
                                        (600, 64, 16, 2, 7), (600, 128, 8, 1, 9),
                                        (150, 128, 16, 1, 20), (300, 256, 8, 1, 9)])
@pytest.mark.parametrize("longest", [0, 3000])
def test_attention_many_small_requests(b, B, d, H, Hk, T, longest):
    """Many pieces to a block, most of one tile: the rings and buffers turn over
    with every piece; with a long request among them, cut."""
    g = np.random.default_rng(B + d)
    lens = g.integers(0, 140, B) * (g.random(B) < 0.9)
    lens[B // 2] = longest
    new = g.integers(0, T + 1, B)
    new[B // 2] = T
    p = _problem(lens.tolist(), new.tolist(), H, Hk, d, 32, seed=B)
    out, lse = _run(b, p, 5)
    assert b.dfa_status() == 0
    _check(p, 5, out, lse)


@pytest.mark.parametrize("d,H", [(64, 8), (128, 8), (128, 2), (256, 8)])
@pytest.mark.parametrize("longest", [0, 3000])
def test_own_values_that_are_not_finite_stay_with_their_rows(b, d, H, longest):
    """Every seventh of many small requests has an infinite value: causal rows
    that do not see it, of that request or another, are as without it."""
    B, T = 300, 9
    g = np.random.default_rng(d)
    lens = g.integers(0, 140, B).tolist()
    lens[5] = longest
    p = _problem(lens, [T] * B, H, 1, d, 32, seed=d)
    want = _run(b, p, 1)
    sees = torch.zeros(B * T, dtype=torch.bool)
    v = p["v"].clone()
    for i in range(0, B, 7):
        j = i % T
        v[i * T + j, 0, 3] = float("inf")
        sees[i * T + j:(i + 1) * T] = True
    got = _run(b, dict(p, v=v), 1)
    assert b.dfa_status() == 0
    sees = sees.to(DEV)
    assert torch.equal(got[0][~sees], want[0][~sees]) and torch.equal(got[1], want[1])
    assert bool((got[0][sees][..., 3] == float("inf")).all())
    rest = [i for i in range(d) if i != 3]
    assert torch.equal(got[0][sees][..., rest], want[0][sees][..., rest])


@pytest.mark.parametrize("H", [4, 32])
@pytest.mark.parametrize("lens", [[0], [5], [0, 70, 0, 16], [1000, 0]])
def test_attention_without_own_keys(b, lens, H):
    """Rows of an empty cache see nothing: output 0, lse -inf."""
    new = [3] * len(lens)
    p = _problem(lens, new, H, 2, 64, 16, seed=9, own=False)
    out, lse = _run(b, p, 1)
    assert b.dfa_status() == 0
    _check(p, 1, out, lse)


@pytest.mark.parametrize("H", [4, 32])
def test_attention_leaves_rows_behind_the_last_request(b, H):
    p = _problem([40, 7], [3, 2], H, 2, 128, 32, seed=10, tail=6)
    out = torch.full_like(p["q"], 9.0)
    lse = torch.full((H, 11), 8.0, device=DEV)
    _run(b, p, 4, out=out, lse=lse)
    assert b.dfa_status() == 0
    assert (out[5:] == 9).all() and (lse[:, 5:] == 8).all()
    _check(p, 4, out, lse)


@pytest.mark.parametrize("H", [4, 16])
def test_attention_strided_and_large_magnitudes(b, H):
    """Slices of one projection; queries far above and below f16's range; page
    scales that differ by 2^20."""
    p = _problem([100, 300], [6, 4], H, 2, 128, 16, seed=11)
    qkv = torch.cat([p["q"], p["k"], p["v"]], 1)
    # scores stay below about 10: queries of 2^40 meet keys of 2^-40
    p["ks"] *= 2.0 ** -40
    qkv[:, :H] *= 2.0 ** 40
    qkv[:, H:H + 2] *= 2.0 ** -40
    p["vs"][::2] *= 2.0 ** 20
    p["q"], p["k"], p["v"] = qkv[:, :H], qkv[:, H:H + 2], qkv[:, H + 2:]
    out, lse = _run(b, p, 3)
    assert b.dfa_status() == 0
    _check(p, 3, out, lse)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("H", [4, 8])
def test_own_values_that_are_not_finite(b, d, bad, H):
    """They reach the rows that see them and no others."""
    p = _problem([20, 33], [12, 9], H, 2, d, 16, seed=12)
    clean = _run(b, p, 4)[0].clone()
    p["v"][9, 1, 5] = bad   # request 0, position 29: seen from block 7 (row 8) on
    p["k"][12 + 7, 0, 3] = float("nan")  # request 1, position 40: block 10, rows 7 ...
    out, lse = _run(b, p, 4)
    assert b.dfa_status() == 0
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[8:12, H // 2:, 5] = True
    hit[12 + 7:, :H // 2] = True
    assert not torch.isfinite(out[hit]).any()
    if bad == bad:
        assert (out[8:12, H // 2:, 5] == bad).all()
    assert torch.isfinite(out[~hit]).all()
    assert torch.equal(out[~hit], clean[~hit])


@pytest.mark.parametrize("what", ["page", "negative page", "length", "negative length", "order",
                                  "rows", "max_new"])
@pytest.mark.parametrize("H", [2, 10])
def test_attention_bad_tables(b, what, H):
    """A bad page counts as masked, a bad request as empty; the rest is right."""
    lens, new = [100, 50], [4, 5]
    p = _problem(lens, new, H, 1, 128, 16, seed=13)
    q = dict(p)
    q["table"], q["lens"], q["cu"] = p["table"].copy(), list(lens), list(p["cu"])
    maxn = 5
    if what == "page":
        q["table"][0, 2] = 10 ** 6
    elif what == "negative page":
        q["table"][0, 3] = -1
    elif what == "length":
        q["lens"][0] = 10 ** 8
    elif what == "negative length":
        q["lens"][0] = -5
    elif what == "order":
        q["cu"][0] = 6
    elif what == "rows":
        q["cu"], q["new"] = [0, 4, 500], [4, 496]
        maxn = 496
    else:
        maxn = 4
    out, lse = b.dfa_cache_forward(q["q"], q["kc"], q["vc"], q["ks"], q["vs"], _i32(q["table"]),
                                   _i32(q["lens"]), _i32(q["cu"]), maxn, k=q["k"], v=q["v"],
                                   block_size=4)
    assert b.dfa_status() == b.DFA_EDEVICE
    want, _ = _run(b, p, 4)
    assert b.dfa_status() == 0
    good = slice(0, 4) if what in ("rows", "max_new") else slice(4, 9)
    assert torch.equal(out[good], want[good])
    if "page" in what:
        assert torch.isfinite(out).all()


def test_refusals(b):
    p = _problem([10], [2], 4, 2, 64, 16)
    good = dict(k=p["k"], v=p["v"])
    args = [p["q"], p["kc"], p["vc"], p["ks"], p["vs"], _i32(p["table"]), _i32(p["lens"]),
            _i32(p["cu"]), 2]
    b.dfa_cache_forward(*args, **good)
    for i, x in ((0, p["q"].float()), (0, p["q"][:, :3]), (0, p["q"][..., :32]), (1, p["kc"][:1]),
                 (2, p["vc"].view(torch.uint8)), (3, p["ks"][:, :1]), (4, p["vs"].double()),
                 (5, _i32(p["table"]).long()), (6, _i32([1, 2])), (7, _i32([0]))):
        bad = list(args)
        bad[i] = x
        with pytest.raises((ValueError, b.DfaError)):
            b.dfa_cache_forward(*bad, **good)
    for kw in (dict(k=p["k"]), dict(k=p["k"], v=p["v"][:1]), dict(**good, block_size=0),
               dict(**good, out=torch.empty(2, 4, 64, device=DEV))):
        with pytest.raises((ValueError, b.DfaError)):
            b.dfa_cache_forward(*args, **kw)
    with pytest.raises(b.DfaError):
        b.dfa_cache_forward(*args[:8], -1, **good)
    with pytest.raises(ValueError):
        b.dfa_cache_append(p["k"], p["v"][:1], args[7], args[6], args[5], *args[1:5], 2)
    with pytest.raises(b.DfaError):  # pages of 24 tokens
        c = torch.zeros((3, 2, 24, 64), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
        s = torch.ones((3, 2), device=DEV)
        b.dfa_cache_append(p["k"], p["v"], args[7], args[6], args[5], c, c, s, s, 2)
    torch.cuda.synchronize()
    assert b.dfa_status() == 0


def test_workspaces(b):
    """Short tables need none; long ones one of the size that is asked for, which
    is then all that is written."""
    p = _problem([10], [2], 4, 2, 64, 16)
    assert b.dfa_cache_workspace_bytes(1, 2, 2, 4, 2, 64, 16, p["table"].shape[1]) == 0
    want = _run(b, p, 2)
    for n in (0, 16):
        got = _run(b, p, 2, workspace=torch.empty(n, dtype=torch.uint8, device=DEV))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for T, H in ((2, 4), (7, 8), (40, 8)):
        p = _problem([5000, 3], [T, T], H, 2, 64, 16)
        want = _run(b, p, 2)
        n = b.dfa_cache_workspace_bytes(2, 2 * T, T, H, 2, 64, 16, p["table"].shape[1])
        assert n > 0
        with pytest.raises(b.DfaError):
            _run(b, p, 2, workspace=torch.empty(n - 1, dtype=torch.uint8, device=DEV))
        buf = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device=DEV)
        got = _run(b, p, 2, workspace=buf[:n])
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert bool((buf[n:] == 0xA5).all())
    assert b.dfa_status() == 0


@pytest.mark.parametrize("block", [2 ** 31 - 1, 2 ** 31, 2 ** 32 + 1, 2 ** 40])
def test_block_sizes_past_32_bits(b, block):
    """A block of any size that covers the rows makes them one block."""
    p = _problem([70, 3], [5, 9], 4, 2, 64, 32)
    want = _run(b, p, 2 ** 30)
    got = _run(b, p, block)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    causal = _run(b, p, 1)
    assert not torch.equal(causal[0], want[0])


# ------------------------------------------------------------------ together

def _sampler(b, steps, T, bs, H, Hk, d, ps, table, pages, cache, qkv, stream=None):
    """Rotate, attend and append block after block; the outputs of all steps."""
    from block_diffusion_masked_gb300 import rotary_func

    outs = []
    for i in range(steps):
        rows = qkv[i].shape[0]
        step = pages.plan(T[i], rows, int(max(T[i].tolist())) if stream is None else rows)
        q, k, v = qkv[i][:, :H], qkv[i][:, H:H + Hk], qkv[i][:, H + Hk:]
        q, k = rotary_func(q, k, table, step.positions)
        out, lse = cache.attend(q, step, k, v, bs)
        cache.append(k, v, step)
        outs.append((q, k, v, out, lse, step))
        pages.advance(step)
    return outs


def test_sampler_steps(b):
    """Blocks of two requests, one of them released and begun again: every
    step's attention against the definition on the cache as it stood, and the
    cache against appends by the definition."""
    from block_diffusion_masked_gb300 import KVCache, PageTable, rotary_table

    H, Hk, d, ps, bs = 4, 2, 64, 16, 8
    pages, cache = PageTable(2, 8, 11, ps), KVCache(11, ps, Hk, d)
    table = rotary_table(128, d)
    g = torch.Generator("cpu").manual_seed(0)
    ref_k, ref_ks = _f64(cache.k), _f64(cache.k_scale)
    ref_v, ref_vs = _f64(cache.v), _f64(cache.v_scale)
    for i, new in enumerate([[8, 8], [8, 5], [8, 0], [8, 8], [3, 8]]):
        if i == 3:
            pages.release(_i32([0, 1]))
        rows = sum(new) + 2
        qkv = torch.randn((rows, H + 2 * Hk, d), generator=g).to(torch.bfloat16).to(DEV)
        before = pages.cache_lens.tolist()
        ((q, k, v, out, lse, step),) = _sampler(b, 1, [_i32(new)], bs, H, Hk, d, ps, table, pages,
                                                cache, [qkv])
        assert b.dfa_status() == 0 and int(step.missing) == 0
        cu, tab = step.cu_new.tolist(), step.block_table.cpu().numpy()
        pos = step.positions.tolist()
        want_q = osam.rotary(_f64(qkv[:, :H]), table.cpu().numpy(), pos)
        assert np.abs(_f64(q) - want_q).max() <= 2.0 ** -8 * np.abs(want_q).max() + 2.0 ** -20
        p = dict(table=tab, cu=cu, lens=before, new=new, q=q, k=k, v=v,
                 kc=torch.tensor(ref_k), ks=torch.tensor(ref_ks), vc=torch.tensor(ref_v),
                 vs=torch.tensor(ref_vs))
        _check(p, bs, out, lse)
        ref_k, ref_ks = osam.append(_f64(k), cu, before, tab, ref_k, ref_ks)
        ref_v, ref_vs = osam.append(_f64(v), cu, before, tab, ref_v, ref_vs)
        assert np.array_equal(_f64(cache.k), ref_k) and np.array_equal(_f64(cache.k_scale), ref_ks)
        assert np.array_equal(_f64(cache.v), ref_v) and np.array_equal(_f64(cache.v_scale), ref_vs)


def test_sampler_in_a_graph_and_on_two_streams(b):
    """A captured step replayed over growing lengths, and two samplers on two
    streams at once, give what the same steps give eagerly on one stream."""
    from block_diffusion_masked_gb300 import KVCache, PageTable, rotary_func, rotary_table

    H, Hk, d, ps, bs, B, steps = 8, 2, 128, 32, 4, 3, 6
    table = rotary_table(2048, d)
    new = _i32([4, 4, 3])
    rows = 12
    g = torch.Generator("cpu").manual_seed(1)
    data = [[torch.randn((rows, H + 2 * Hk, d), generator=g).to(torch.bfloat16).to(DEV)
             for _ in range(steps)] for _ in range(2)]
    prompt = [torch.randn((1100 * B, H + 2 * Hk, d), generator=g).to(torch.bfloat16).to(DEV)
              for _ in range(2)]

    def begin(i):
        pages, cache = PageTable(B, 64, 64 * B, ps), KVCache(64 * B, ps, Hk, d)
        step = pages.plan(_i32([1100, 37, 900]), 1100 * B, 1100)
        cache.append(prompt[i][:, H:H + Hk], prompt[i][:, H + Hk:], step)
        pages.advance(step)
        return pages, cache

    def one(pages, cache, qkv):
        step = pages.plan(new, rows, 4)
        q, k = rotary_func(qkv[:, :H], qkv[:, H:H + Hk], table, step.positions)
        out, lse = cache.attend(q, step, k, qkv[:, H + Hk:], bs)
        cache.append(k, qkv[:, H + Hk:], step)
        pages.advance(step)
        return out, lse

    want = []
    for i in range(2):
        state = begin(i)
        want.append([[x.clone() for x in one(*state, qkv)] for qkv in data[i]])
    torch.cuda.synchronize()

    # two streams at once
    streams = [torch.cuda.Stream() for _ in range(2)]
    states = [begin(i) for i in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for n in range(steps):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(one(*states[i], data[i][n]))
    torch.cuda.synchronize()
    assert b.dfa_status() == 0

    def same(a, c):
        return torch.equal(a[0][:11], c[0][:11]) and torch.equal(a[1][:, :11], c[1][:, :11])

    for i in range(2):
        assert all(same(a, c) for a, c in zip(got[i], want[i]))

    # two graphs, captured on one stream, replayed on two at once
    graphs, ins, outs, states = [], [], [], [begin(i) for i in range(2)]
    for i in range(2):
        ins.append(data[i][0].clone())
        saved = [x.clone() for x in (states[i][0].cache_lens, states[i][0].free_count)]
        one(*states[i], ins[i])  # warm-up
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(one(*states[i], ins[i]))
        # the warm-up's tokens are taken back: lengths and pages as they were
        states[i][0].cache_lens.copy_(saved[0])
        states[i][0].free_count.copy_(saved[1])
        graphs.append(graph)
    torch.cuda.synchronize()
    for n in range(steps):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                ins[i].copy_(data[i][n])
                graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert same(outs[i], want[i][n]), (n, i)
    assert b.dfa_status() == 0


def test_long_offsets(b):
    """A cache of more than 2^32 bytes: the last pages are reached."""
    Hk, ps, d = 8, 128, 256
    P = 2 ** 32 // (Hk * ps * d) + 40
    kc = torch.zeros((P, Hk, ps, d), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    vc = torch.zeros((P, Hk, ps, d), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    ks, vs = (torch.ones((P, Hk), device=DEV) for _ in range(2))
    g = torch.Generator("cpu").manual_seed(2)
    x = torch.randn((2, 200, Hk, d), generator=g).to(torch.bfloat16).to(DEV)
    table = _i32([[P - 1, P - 3]])
    cu, zero = _i32([0, 200]), _i32([0])
    b.dfa_cache_append(x[0], x[1], cu, zero, table, kc, vc, ks, vs, 200)
    q = torch.randn((4, Hk, d), generator=g).to(torch.bfloat16).to(DEV)
    out, lse = b.dfa_cache_forward(q, kc, vc, ks, vs, table, _i32([200]), _i32([0, 4]), 4)
    assert b.dfa_status() == 0
    small = [c[[P - 1, P - 3]] if c.dtype == torch.float32 else
             c.view(torch.uint8)[[P - 1, P - 3]].view(torch.float8_e4m3fn) for c in (kc, vc, ks, vs)]
    o2, l2 = b.dfa_cache_forward(q, *small, _i32([[0, 1]]), _i32([200]), _i32([0, 4]), 4)
    assert torch.equal(out, o2) and torch.equal(lse, l2) and bool(out.any())
    ref, _, _, _ = osam.cache_attention(_f64(q), _f64(small[0]), _f64(small[1]), _f64(small[2]),
                                        _f64(small[3]), [[0, 1]], [200], [0, 4])
    assert np.abs(_f64(out) - ref).max() <= 2.0 ** -6 * np.abs(ref).max()


# --------------------------------------------------- small, zero and large magnitudes

@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("H", [1, 6, 16])
@pytest.mark.parametrize("size", [2.0 ** -10, 2.0 ** -40, 2.0 ** -120, 0.0])
def test_attention_of_small_and_zero_queries(b, d, H, size):
    """Units of which a half or more is not there, pages of 16: a masked key has
    no weight however small the row's scores are."""
    p = _problem([5, 48, 97, 33], [4, 4, 4, 4], H, 1, d, 16, seed=20)
    p["q"] *= size
    p["q"][1] = 0
    for own in (True, False):
        if not own:
            p["k"] = p["v"] = None
        out, lse = _run(b, p, 2)
        assert b.dfa_status() == 0
        _check(p, 2, out, lse)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("H", [2, 16])
@pytest.mark.parametrize("zero", ["k", "qk", "qkv"])
def test_sampler_on_zeros(b, d, H, zero):
    """Zero queries, keys and values through append and attend: every key counts
    alike, lse is the logarithm of their number."""
    from block_diffusion_masked_gb300 import KVCache, PageTable

    Hk, ps, new = 1, 64, [3, 5]
    pages, cache = PageTable(2, 4, 8, ps), KVCache(8, ps, Hk, d)
    g = torch.Generator("cpu").manual_seed(d + H)

    def rand(name, rows, heads):
        x = torch.randn((rows, heads, d), generator=g) * (name not in zero)
        return x.to(torch.bfloat16).to(DEV)

    step = pages.plan(_i32([37, 70]), 107, 70)
    cache.append(rand("k", 107, Hk), rand("v", 107, Hk), step)
    pages.advance(step)
    step = pages.plan(_i32(new), 8, 5)
    q, k, v = rand("q", 8, H), rand("k", 8, Hk), rand("v", 8, Hk)
    for own in (True, False):
        out, lse = cache.attend(q, step, *((k, v) if own else ()), block_size=64)
        assert b.dfa_status() == 0
        p = dict(table=step.block_table.cpu().numpy(), cu=[0, 3, 8], lens=[37, 70], new=new, q=q,
                 k=k if own else None, v=v if own else None, kc=cache.k, vc=cache.v,
                 ks=cache.k_scale, vs=cache.v_scale)
        _check(p, 64, out, lse)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("H", [2, 16])
@pytest.mark.parametrize("size", [1.0, 2.0 ** -10, 0.0])
@pytest.mark.parametrize("page", [-1, 10 ** 6])
def test_attention_refused_pages_and_small_queries(b, d, H, size, page):
    """Keys of a page that may not be followed count as masked: as if the request
    did not hold them (own rows one block, so that positions do not matter)."""
    p = _problem([100, 50], [4, 5], H, 1, d, 16, seed=21)
    p["q"] *= size
    table = p["table"].copy()
    table[0, 2] = page
    out, lse = _run(b, dict(p, table=table), 2 ** 20)
    assert b.dfa_status() == b.DFA_EDEVICE
    rest = p["table"].copy()
    rest[0, 2:6] = p["table"][0, 3:7]
    _check(dict(p, table=rest, lens=[84, 50]), 2 ** 20, out, lse)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("H", [1, 6, 16])
@pytest.mark.parametrize("e", [-60, -30, 60])
@pytest.mark.parametrize("many", [False, True])
def test_attention_scales_with_its_values(b, d, H, e, many):
    """The output is linear in the values: own ones and the pages' scales times a
    power of two give the same bits times that power, whatever its size.  Short
    tables, whose segments are not cut, and many requests beside a long one."""
    lens, new = [300, 40, 0, 500], [4, 5, 3, 4]
    if many:
        g = np.random.default_rng(d + H)
        lens, new = g.integers(0, 400, 150).tolist(), g.integers(0, 6, 150).tolist()
        lens[7], new[7] = 3000, 5
    p = _problem(lens, new, H, 1, d, 32, seed=22)
    p["q"] *= 2.0 ** -5  # scores of about 1: every key counts
    want = _run(b, p, 2)
    got = _run(b, dict(p, v=p["v"] * 2.0 ** e, vs=p["vs"] * 2.0 ** e), 2)
    assert b.dfa_status() == 0
    assert torch.equal(got[0].double(), want[0].double() * 2.0 ** e)
    assert torch.equal(got[1], want[1])


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("H", [1, 6, 16])
@pytest.mark.parametrize("own,cached", [(0, -40), (-40, 0), (0, 100), (122, 0), (100, -90),
                                        (122, -90), (-110, -90)])
def test_attention_own_and_cached_values_of_different_sizes(b, d, H, own, cached):
    """Own values of 2^own beside cached ones of 2^cached, over bf16's range; rows
    that see next to nothing of their own among them (scores of up to 30)."""
    p = _problem([300, 40, 0], [4, 5, 3], H, 1, d, 32, seed=23)
    p["v"] *= 2.0 ** own
    p["vs"] *= 2.0 ** cached
    out, lse = _run(b, p, 2)
    assert b.dfa_status() == 0
    _check(p, 2, out, lse)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [9, 16])
def test_own_values_that_are_not_finite_in_first_steps(b, d, T):
    """Empty caches: every piece is one tile of own keys, the next one's behind
    it.  Each request but every third has an infinite value, at every row in turn."""
    B, H = 1500, 8
    p = _problem([0] * B, [T] * B, H, 1, d, 32, seed=d + T)
    want = _run(b, p, 1)
    v, sees = p["v"].clone(), torch.zeros((B, T), dtype=torch.bool)
    for i in range(B):
        if i % 3:
            j = (i + i // 7) % T
            v[i * T + j, 0, i % d] = float("inf")
            sees[i, j:] = True
    sees = sees.reshape(-1).to(DEV)
    dim = (torch.arange(B, device=DEV) % d).repeat_interleave(T)
    hit = (sees[:, None] & (torch.arange(d, device=DEV) == dim[:, None]))[:, None].expand(-1, H, d)
    for _ in range(5):
        got = _run(b, dict(p, v=v), 1)
        assert bool((got[0][hit] == float("inf")).all())
        assert torch.equal(got[0][~hit], want[0][~hit]) and torch.equal(got[1], want[1])
    assert b.dfa_status() == 0


@pytest.mark.parametrize("H", [2, 16])
def test_loose_bounds_on_the_rows_of_a_request(b, H):
    """max_new is an upper bound: one far above the rows changes nothing."""
    p = _problem([700, 3], [5, 9], H, 1, 64, 32, seed=24)
    want = _run(b, p, 4)
    for bound in (14, 2 ** 24 + 1, 2 ** 31 - 1, 2 ** 40):
        got = _run(b, dict(p, new=[bound]), 4)
        assert b.dfa_status() == 0
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_release_between_plan_and_advance(b):
    """The planned step is refused; planned again, no page is lost and the released
    request begins anew."""
    from block_diffusion_masked_gb300 import PageTable

    pages = PageTable(2, 8, 12, 16)
    pages.advance(pages.plan(_i32([40, 20]), 60, 40))
    step = pages.plan(_i32([16, 16]), 32, 16)
    pages.release(_i32([1, 0]))
    with pytest.raises(ValueError):
        pages.advance(step)
    pages.advance(pages.plan(_i32([5, 16]), 21, 16))
    assert b.dfa_status() == 0
    assert pages.cache_lens.tolist() == [5, 36] and int(pages.free_count) == 12 - 1 - 3
    held = pages.block_table[0, :1].tolist() + pages.block_table[1, :3].tolist()
    assert sorted(held + pages.free_pages[:8].tolist()) == list(range(12))


def test_arguments_past_32_bits(b):
    """Page sizes, rows and bounds past 32 bits are refused, not wrapped."""
    p = _problem([10], [2], 4, 2, 64, 16)
    for bound in (-1, -2 ** 32 + 2):
        with pytest.raises(b.DfaError):
            _run(b, dict(p, new=[bound]), 2)
        with pytest.raises(b.DfaError):
            b.dfa_cache_append(p["k"], p["v"], _i32(p["cu"]), _i32([10]), _i32(p["table"]), p["kc"],
                               p["vc"], p["ks"], p["vs"], bound)
    with pytest.raises(b.DfaError):
        _run(b, p, -2 ** 32 + 2)
    state = (_i32([0]), _i32([1]), _i32([[-1]]), _i32([0]), _i32([1]))
    for ps, rows in ((2 ** 32 + 16, 4), (16, 2 ** 32 + 4), (16, -2 ** 32 + 4)):
        with pytest.raises((ValueError, b.DfaError)):
            b.dfa_cache_plan(*state, ps, rows)
    with pytest.raises(b.DfaError):
        b.dfa_cache_release(state[1], state[0], *state[2:], 2 ** 32 + 16)
    assert b.dfa_status() == 0


def test_captured_plan_advanced_outside_its_graph(b):
    """A graph of the plan alone, replayed; advances and releases between replays."""
    from block_diffusion_masked_gb300 import PageTable

    pages = PageTable(2, 8, 12, 16)
    new = _i32([20, 5])
    pages.plan(new, 25, 20)  # warm-up
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step = pages.plan(new, 25, 20)
    for lens in ([20, 5], [40, 10]):
        graph.replay()
        pages.advance(step)
        assert pages.cache_lens.tolist() == lens
    pages.release(_i32([1, 0]))
    graph.replay()
    pages.advance(step)
    assert b.dfa_status() == 0
    assert pages.cache_lens.tolist() == [20, 15] and int(pages.free_count) == 12 - 2 - 1
    held = pages.block_table[0, :2].tolist() + pages.block_table[1, :1].tolist()
    assert sorted(held + pages.free_pages[:9].tolist()) == list(range(12))

"""The 4-bit cache on the GPU -- append, reading back, attention -- against the float64
definitions, the reading back of the 8-bit cache, and a sampler's steps over either.

Appended codes and scales are those of the definition exactly, and so is what is read
back.  Attention: a cached value (n - 8) s is exact in f16, so the tolerance is that of
the 8-bit cache's products.  A score is a sum of d products of exact f16 (or bf16)
operands in float32: at most (d + 2) * 2^-23 of scale * sum |q k| (truncating adds
included), and the exponential and its argument's rounding add 2^-20 (1 + |s|); both act
as a relative error delta on the probabilities.  Cached probabilities are rounded to f16
(2^-11), own ones to bf16 (2^-8), so the output is off by at most (2^-8 + 2 delta)
sum p |v| plus its own rounding, 2^-8 of it; without own keys 2^-11 stands for the first
2^-8.  Probabilities below 2^-30 of the largest may be lost: keys * 2^-30 max |v|.
lse: delta + 2^-22 |lse|.
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
    return t.detach().double().cpu().numpy()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _codes(t):
    return osam.codes4(t.cpu().numpy())


def _e5m2(s):
    return torch.tensor(s).float().to(torch.float8_e5m2)


def _pack(codes):
    """Bytes (..., d / 2) of codes (..., d)."""
    c = codes.reshape(*codes.shape[:-1], -1, 8)
    word = sum(c[..., i] << (16 * (i % 2) + 4 * (i // 2)) for i in range(8))
    return torch.tensor(word.astype("<u4").view(np.uint8).reshape(*codes.shape[:-1], -1))


def _cache(P, Hk, ps, d, seed, e=(-4, 1)):
    """Random codes and scales of both signs, of sizes 2^e[0] .. 2^e[1]."""
    g = np.random.default_rng(seed)
    codes = g.integers(0, 16, (P, Hk, ps, d))
    s = g.integers(4, 8, (P, Hk, d // 32, ps)) * 2.0 ** g.integers(*e, (P, Hk, d // 32, ps)) / 16
    s *= g.choice([-1, 1], s.shape)
    return _pack(codes).to(DEV), _e5m2(s).to(DEV)


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


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("d,ps,Hk", [(64, 16, 1), (64, 128, 3), (128, 32, 2), (128, 64, 1),
                                     (128, 128, 1), (256, 16, 2), (256, 64, 1), (256, 128, 1)])
@pytest.mark.parametrize("lens,new", [
    ([0], [1]), ([15, 16, 17], [1, 1, 1]), ([0, 130, 5, 64], [70, 0, 3, 200]),
    ([127, 3], [129, 300]), ([2, 9], [12, 40])])
def test_append(b, d, ps, Hk, lens, new):
    """Codes and scales of the definition in their places, everything else as it was;
    values spread over many powers of two, with ties and both limits among them."""
    table, cu, P = _requests(lens, new, ps, d + ps)
    kc, ks = _cache(P, Hk, ps, d, 1)
    vc, vs = _cache(P, Hk, ps, d, 2)
    rows = cu[-1] + 3  # three rows behind the last request
    g = torch.Generator("cpu").manual_seed(5)
    amp = torch.exp(3 * torch.randn((rows, Hk, 1), generator=g))
    kv = torch.randn((2, rows, Hk, d), generator=g) * amp
    kv[1, :, :, ::3] = kv[1, :, :, ::3].round()          # whole and half scales
    kv[1, :, :, 0::32], kv[1, :, :, 1::32] = 8.0, 4.5
    kv = kv.to(torch.bfloat16)
    kv[0, 0, 0, :32], kv[0, 0, 0, 32] = 0.0, 2.0 ** -120
    kv[0, -4, 0, 1], kv[1, -4, 0, 33] = 3e4, -2.0 ** 100
    # slices of one projection's output: strided rows and heads
    both = torch.stack([kv[0], kv[1]], 2).to(DEV)  # (rows, Hk, 2, d)
    k, v = both[:, :, 0], both[:, :, 1]
    refs = [osam.append4(_f64(x), cu, lens, table, _codes(c), _f64(s))
            for x, c, s in ((k, kc, ks), (v, vc, vs))]
    for _ in range(2):  # the second time on the appended cache: nothing changes
        b.dfa_cache4_append(k, v, _i32(cu), _i32(lens), _i32(table), kc, vc, ks, vs, max(new))
        assert b.dfa_status() == 0
        for (rc, rs), c, s in ((refs[0], kc, ks), (refs[1], vc, vs)):
            assert np.array_equal(_f64(s), rs)
            assert np.array_equal(_codes(c), rc)


def test_append_every_value(b):
    """Every finite bf16 value beside every size of the largest one: the codes are those
    of the definition, ties too."""
    d, ps = 64, 128
    bits = np.arange(0, 0x7f80, 5, dtype=np.uint32)
    small = torch.tensor((bits << 16).view(np.float32)).to(torch.bfloat16)
    n = -(-small.numel() // 31) * 31
    rest = torch.cat([small, small[:n - small.numel()]]).view(-1, 31)
    rows = []
    for m in range(128, 256, 3):  # magnitudes of 8 significant bits
        top = torch.full((24, 1), m * 2.0 ** -7)
        steps = torch.arange(31)[None] * top / 31 * (torch.arange(24)[:, None] / 24 + 0.02)
        rows.append(torch.cat([top, steps], 1).to(torch.bfloat16))
        rows.append(-rows[-1])
    x = torch.cat(rows + [torch.cat([rest.amax(1, True), rest], 1)])
    x = torch.cat([x, x[:x.shape[0] % 2]]).view(-1, 1, d).to(DEV)
    T = x.shape[0]
    table, cu, P = _requests([0], [T], ps, 1)
    kc, ks = _cache(P, 1, ps, d, 1)
    vc, vs = _cache(P, 1, ps, d, 2)
    rc, rs = osam.append4(_f64(x), cu, [0], table, _codes(kc), _f64(ks))
    b.dfa_cache4_append(x, x, _i32(cu), _i32([0]), _i32(table), kc, vc, ks, vs, T)
    assert b.dfa_status() == 0
    assert np.array_equal(_f64(ks), rs) and np.array_equal(_codes(kc), rc)


def test_values_that_are_not_finite(b):
    """Their group is NaN, and no other."""
    d, ps, T = 128, 16, 6
    table, cu, P = _requests([3], [T], ps, 3)
    kc, ks = _cache(P, 2, ps, d, 4)
    vc, vs = _cache(P, 2, ps, d, 5)
    x = torch.randn((T, 2, d), device=DEV).bfloat16()
    x[0, 0, 3], x[2, 1, 64], x[5, 0, 127] = float("inf"), float("-inf"), float("nan")
    b.dfa_cache4_append(x, x, _i32(cu), _i32([3]), _i32(table), kc, vc, ks, vs, T)
    k, v = b.dfa_cache4_read(kc, vc, ks, vs, _i32(table), _i32([3 + T]), _i32([0, T]), T,
                             first=_i32([3]))
    assert b.dfa_status() == 0
    bad = torch.zeros((T, 2, d), dtype=torch.bool, device=DEV)
    bad[0, 0, :32] = bad[2, 1, 64:96] = bad[5, 0, 96:] = True
    assert torch.equal(k.isnan(), bad) and torch.equal(v.isnan(), bad)
    assert (k[~bad].float() - x[~bad].float()).abs().max() <= 0.5


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
    was, was_s = kc.clone(), ks.view(torch.uint8).clone()
    x = torch.randn((11, 1, d), device=DEV).bfloat16()
    b.dfa_cache4_append(x, x, _i32(cu), _i32(lens), _i32(table), kc, vc, ks, vs, maxn)
    assert b.dfa_status() == b.DFA_EDEVICE
    good = 0 if what in ("rows", "max_new") else 1
    page = table[good][lens[good] // ps]
    assert not torch.equal(kc[page], was[page])
    for p in set(range(P)) - set(table[good].tolist()):
        assert torch.equal(kc[p], was[p]) and torch.equal(ks.view(torch.uint8)[p], was_s[p])


# ------------------------------------------------------------------ read

@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("d,ps,Hk", [(64, 16, 1), (64, 128, 5), (128, 32, 2), (256, 64, 3)])
@pytest.mark.parametrize("lens,first,n", [
    ([1], None, [1]), ([40, 300, 7], [3, 0, 7], [37, 200, 0]), ([0, 70, 0, 129], [0, 69, 0, 64],
                                                                [0, 1, 0, 65]),
    ([200] * 70, list(range(70)), [i % 4 for i in range(70)])])
def test_read(b, bits, d, ps, Hk, lens, first, n):
    table, _, P = _requests(lens, [0] * len(lens), ps, d + ps)
    cu = [0] + np.cumsum(n).tolist()
    rows = cu[-1] + 4  # behind the last request: left as they are
    if bits == 4:
        kc, ks = _cache(P, Hk, ps, d, 1)
        vc, vs = _cache(P, Hk, ps, d, 2)
        values = [osam.values4(_codes(c), _f64(s)) for c, s in ((kc, ks), (vc, vs))]
    else:
        g = torch.Generator("cpu").manual_seed(3)
        kc, vc = (torch.randn((P, Hk, ps, d), generator=g).mul(64).clamp(-448, 448)
                  .to(torch.float8_e4m3fn).to(DEV) for _ in range(2))
        ks, vs = ((2.0 ** torch.randint(-100, 100, (P, Hk), generator=g).double()).float().to(DEV)
                  for _ in range(2))
        values = [_f64(c) * _f64(s)[:, :, None, None] for c, s in ((kc, ks), (vc, vs))]
    k, v = (torch.full((rows, Hk, d), 9.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    read = b.dfa_cache4_read if bits == 4 else b.dfa_cache_read
    got = read(kc, vc, ks, vs, _i32(table), _i32(lens), _i32(cu), rows,
               first=None if first is None else _i32(first), k=k, v=v)
    assert b.dfa_status() == 0 and got[0] is k and got[1] is v
    for x, c in ((k, values[0]), (v, values[1])):
        assert np.array_equal(_f64(x)[:cu[-1]],
                              osam.cache_read(c, table, first or [0] * len(lens), cu))
        assert (x[cu[-1]:] == 9).all()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("what", ["page", "negative page", "past the length", "before 0", "length",
                                  "order", "negative row"])
def test_read_bad_tables(b, bits, what):
    """Tokens that are not there are zeros, rows out of order are left alone, the other
    request's are right."""
    lens, ps, d = [40, 20], 16, 64
    table, _, P = _requests(lens, [0, 0], ps, 6)
    cu, first, want_lens = [0, 10, 16], [20, 3], list(lens)
    if bits == 4:
        kc, ks = _cache(P, 1, ps, d, 7)
        values = osam.values4(_codes(kc), _f64(ks))
    else:
        kc = torch.randn((P, 1, ps, d), device=DEV).to(torch.float8_e4m3fn)
        ks = torch.ones((P, 1), device=DEV)
        values = _f64(kc)
    right = osam.cache_read(values, table, first, cu)
    bad_table = table.copy()
    zero = slice(0, 10)
    if what == "page":
        bad_table[0, 1] = P  # tokens 16 .. 31: rows 0 .. 9 are tokens 20 .. 29
    elif what == "negative page":
        bad_table[0, 1] = -1
    elif what == "past the length":
        want_lens[0] = 25
        zero = slice(5, 10)
    elif what == "before 0":
        first[0] = -4
        right[4:10] = osam.cache_read(values, table, [0, 3], [0, 6, 12])[:6]
        zero = slice(0, 4)
    elif what == "length":
        want_lens[0] = 10 ** 8
    elif what == "order":
        cu = [12, 10, 16]
        zero = slice(0, 0)
    else:
        cu[0] = -3
        zero = slice(0, 0)
    out = torch.full((16, 1, d), 9.0, dtype=torch.bfloat16, device=DEV)
    other = out.clone()
    read = b.dfa_cache4_read if bits == 4 else b.dfa_cache_read
    read(kc, kc, ks, ks, _i32(bad_table), _i32(want_lens), _i32(cu), 16, first=_i32(first), k=out,
         v=other)
    assert b.dfa_status() == b.DFA_EDEVICE
    assert torch.equal(out, other)
    got = _f64(out)
    if what not in ("order", "negative row"):
        right[zero] = 0
        assert np.array_equal(got, right)
    else:
        assert (got[:10] == 9).all()
        if what == "negative row":
            assert np.array_equal(got[10:], right[10:])


# ------------------------------------------------------------------ attention

def _problem(lens, new, H, Hk, d, ps, seed=0, tail=0, own=True, e=(-4, 1)):
    table, cu, P = _requests(lens, new, ps, seed)
    kc, ks = _cache(P, Hk, ps, d, seed + 1, e)
    vc, vs = _cache(P, Hk, ps, d, seed + 2, e)
    g = torch.Generator("cpu").manual_seed(seed + 3)
    rows = cu[-1] + tail
    q = torch.randn((rows, H, d), generator=g).to(torch.bfloat16).to(DEV)
    k, v = (torch.randn((rows, Hk, d), generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
    p = dict(table=table, cu=cu, lens=lens, new=new, kc=kc, ks=ks, vc=vc, vs=vs, q=q,
             k=k if own else None, v=v if own else None)
    p["values"] = [osam.values4(_codes(c), _f64(s)) for c, s in ((kc, ks), (vc, vs))]
    # behind the last token of a request, and in pages that none has: scales that are not
    # numbers, infinities and codes of any kind
    for i, n in enumerate(lens):
        if n % ps:
            page = int(table[i, n // ps])
            for s in (ks, vs):
                s.view(torch.uint8)[page, :, :, n % ps:] = 0x7F if i % 2 else 0x7C
    for page in set(range(P)) - set(table.reshape(-1).tolist()):
        ks.view(torch.uint8)[page] = vs.view(torch.uint8)[page] = 0xFE
    return p


def _run(b, p, bs, **kw):
    return b.dfa_cache4_forward(p["q"], p["kc"], p["vc"], p["ks"], p["vs"], _i32(p["table"]),
                                _i32(p["lens"]), _i32(p["cu"]), max(p["new"]), k=p["k"], v=p["v"],
                                block_size=bs, **kw)


def _check(p, bs, out, lse):
    d, n = p["q"].shape[2], p["cu"][-1]
    own = p["k"] is not None
    kv, vv = p["values"]
    ones = np.ones(kv.shape[:2])
    ref, rl, absout, big = osam.cache_attention(
        _f64(p["q"]), kv, vv, ones, ones, p["table"], p["lens"], p["cu"],
        _f64(p["k"]) if own else None, _f64(p["v"]) if own else None, bs)
    delta = (d + 2) * 2.0 ** -23 * big + 2.0 ** -20 * (1 + big)  # (H, rows)
    vmax = 2.0 ** -30 * (max(p["lens"]) + 1) * np.abs(vv).max()
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


@pytest.mark.parametrize("ps", [16, 64, 128])
@pytest.mark.parametrize("d,G,T", [(64, 1, 2), (128, 4, 3), (128, 8, 4), (128, 4, 20), (256, 2, 11),
                                   (256, 4, 16), (64, 8, 8)])
def test_attention_split_over_chunks(b, d, G, T, ps):
    """Long requests beside short ones: several chunks joined, others not."""
    p = _problem([3001, 40, 1030], [T, T, 1], 2 * G, 2, d, ps, seed=G + T)
    out, lse = _run(b, p, T)
    assert b.dfa_status() == 0
    _check(p, T, out, lse)


@pytest.mark.parametrize("longest", [500, 1000])
@pytest.mark.parametrize("B,H,T", [(1, 4, 1), (80, 4, 1), (40, 16, 5), (3, 16, 20)])
def test_attention_short_tables(b, B, H, T, longest):
    g = np.random.default_rng(B + T)
    lens = g.integers(0, longest, B).tolist()
    lens[0] = longest
    p = _problem(lens, [T] * B, H, 2, 64, 32, seed=B)
    out, lse = _run(b, p, T)
    assert b.dfa_status() == 0
    _check(p, T, out, lse)


@pytest.mark.parametrize("H", [4, 32])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens", [[0], [5], [0, 70, 0, 16], [1000, 0]])
def test_attention_without_own_keys(b, lens, d, H):
    """Rows of an empty cache see nothing: output 0, lse -inf."""
    p = _problem(lens, [3] * len(lens), H, 2, d, 16, seed=9, own=False)
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


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("H", [4, 16, 64])
def test_attention_at_the_limits_of_the_scales(b, d, H):
    """Strided queries and own rows; scales over all of their range, 2^-14 to 896: values
    up to 7168 and down to 2^-14, queries such that scores stay moderate."""
    p = _problem([100, 300], [6, 4], H, 2, d, 16, seed=11, e=(-12, 12))
    qkv = torch.cat([p["q"] * 2.0 ** -12, p["k"], p["v"]], 1)
    p["q"], p["k"], p["v"] = qkv[:, :H], qkv[:, H:H + 2], qkv[:, H + 2:]
    assert np.abs(p["values"][0]).max() > 4096
    out, lse = _run(b, p, 3)
    assert b.dfa_status() == 0
    _check(p, 3, out, lse)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("H", [1, 6, 16])
@pytest.mark.parametrize("size", [2.0 ** -40, 2.0 ** -120, 0.0, 2.0 ** 6])
def test_attention_of_small_and_large_queries(b, d, H, size):
    """Scores of 0, and of some hundreds: one key has nearly all of the probability."""
    p = _problem([300, 40], [3, 8], H, 1, d, 32, seed=14)
    p["q"] *= size
    out, lse = _run(b, p, 8)
    assert b.dfa_status() == 0
    _check(p, 8, out, lse)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("H", [2, 16, 40])
@pytest.mark.parametrize("own,cached", [(0, -12), (-40, 0), (100, 0), (122, 6)])
def test_attention_own_and_cached_values_of_different_sizes(b, d, H, own, cached):
    """Own values of one size beside cached ones of another: neither loses more than its
    own rounding."""
    p = _problem([200, 33], [8, 3], H, 2, d, 16, seed=15, e=(cached, cached + 2))
    p["q"] *= 2.0 ** -max(cached, 0)
    p["v"] = (p["v"].double() * 2.0 ** own).to(torch.bfloat16)
    out, lse = _run(b, p, 8)
    assert b.dfa_status() == 0
    _check(p, 8, out, lse)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("H", [2, 16, 64])
def test_cached_groups_that_are_not_numbers(b, d, H):
    """A value group that is NaN reaches its dims of the rows that see it; a key group
    that is, all dims of the rows of its head."""
    p = _problem([90, 50], [4, 3], H, 2, d, 16, seed=16)
    clean = _run(b, p, 4)[0].clone()
    page, key = p["table"][0][2], p["table"][1][1]
    p["vs"].view(torch.uint8)[int(page), 1, d // 32 - 1, 5] = 0x7F
    p["ks"].view(torch.uint8)[int(key), 0, 0, 3] = 0x7F
    out, lse = _run(b, p, 4)
    assert b.dfa_status() == 0
    hit = torch.zeros_like(out, dtype=torch.bool)
    hit[:4, H // 2:, d - 32:] = True
    hit[4:, :H // 2] = True
    assert out[hit].isnan().all()
    assert torch.equal(out[~hit], clean[~hit])
    assert lse[:H // 2, 4:].isnan().all() and lse[H // 2:].isfinite().all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("H", [4, 8, 32])
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
    assert torch.equal(out[~hit], clean[~hit])


@pytest.mark.parametrize("what", ["page", "negative page", "length", "negative length", "order",
                                  "rows", "max_new"])
@pytest.mark.parametrize("d,H,ps", [(128, 2, 16), (128, 10, 16), (256, 10, 64), (64, 2, 32)])
def test_attention_bad_tables(b, what, d, H, ps):
    """A bad page counts as masked, a bad request as empty; the rest is right."""
    lens, new = [200, 50], [4, 5]
    p = _problem(lens, new, H, 1, d, ps, seed=13)
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
    out, lse = b.dfa_cache4_forward(q["q"], q["kc"], q["vc"], q["ks"], q["vs"], _i32(q["table"]),
                                    _i32(q["lens"]), _i32(q["cu"]), maxn, k=q["k"], v=q["v"],
                                    block_size=4)
    assert b.dfa_status() == b.DFA_EDEVICE
    want, _ = _run(b, p, 4)
    assert b.dfa_status() == 0
    i = 0 if what in ("rows", "max_new") else 1
    good = slice(0, 4) if i == 0 else slice(4, 9)
    if i:  # with another max_new, tiles have other rows, and sums another order
        assert torch.equal(out[good], want[good])
    r = dict(p, cu=[0, 4, 4] if i == 0 else [0, 0, 5])
    r["q"], r["k"], r["v"] = p["q"][good], p["k"][good], p["v"][good]
    _check(r, 4, out[good], lse[:, good])
    if "page" in what:
        assert torch.isfinite(out).all()
        # the definition, with that page's keys left out; the own rows' blocks of four
        # begin where they did
        at = 2 if what == "page" else 3
        left = 200 - min(ps, 200 - at * ps)
        assert left % 4 == 0
        r = dict(p, table=np.delete(p["table"], at, 1), lens=[left, 50], cu=[0, 4, 4], new=[4, 0])
        r["q"], r["k"], r["v"] = p["q"][:4], p["k"][:4], p["v"][:4]
        _check(r, 4, out[:4], lse[:, :4])


def test_workspaces(b):
    """Short tables need none; long ones one of the size that is asked for, which
    is then all that is written."""
    p = _problem([10], [2], 4, 2, 64, 16)
    assert b.dfa_cache4_workspace_bytes(1, 2, 2, 4, 2, 64, 16, p["table"].shape[1]) == 0
    for T, H in ((2, 4), (7, 8), (40, 8)):
        p = _problem([5000, 3], [T, T], H, 2, 64, 16)
        want = _run(b, p, 2)
        n = b.dfa_cache4_workspace_bytes(2, 2 * T, T, H, 2, 64, 16, p["table"].shape[1])
        assert n > 0
        with pytest.raises(b.DfaError):
            _run(b, p, 2, workspace=torch.empty(n - 1, dtype=torch.uint8, device=DEV))
        buf = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device=DEV)
        got = _run(b, p, 2, workspace=buf[:n])
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert bool((buf[n:] == 0xA5).all())
    assert b.dfa_status() == 0


def test_refusals(b):
    p = _problem([10], [2], 4, 2, 64, 16)
    good = dict(k=p["k"], v=p["v"])
    args = [p["q"], p["kc"], p["vc"], p["ks"], p["vs"], _i32(p["table"]), _i32(p["lens"]),
            _i32(p["cu"]), 2]
    b.dfa_cache4_forward(*args, **good)
    for i, x in ((0, p["q"].float()), (0, p["q"][:, :3]), (0, p["q"][..., :32]), (1, p["kc"][:1]),
                 (2, p["vc"].view(torch.int8)), (3, p["ks"][:, :1]),
                 (4, p["vs"].view(torch.uint8)), (5, _i32(p["table"]).long()), (6, _i32([1, 2])),
                 (7, _i32([0]))):
        bad = list(args)
        bad[i] = x
        with pytest.raises((ValueError, b.DfaError)):
            b.dfa_cache4_forward(*bad, **good)
        if i:
            with pytest.raises((ValueError, b.DfaError)):
                b.dfa_cache4_append(p["k"], p["v"], bad[7], bad[6], bad[5], *bad[1:5], 2)
        if 0 < i:
            with pytest.raises((ValueError, b.DfaError)):
                b.dfa_cache4_read(*bad[1:8], 2)
    for kw in (dict(first=_i32([0, 0])), dict(first=torch.zeros(1, device=DEV)),
               dict(k=torch.empty(2, 2, 64, device=DEV)), dict(v=p["v"][:1])):
        with pytest.raises(ValueError):
            b.dfa_cache4_read(*args[1:8], 2, **kw)
    with pytest.raises(ValueError):
        b.dfa_cache4_read(*args[1:8], -1)
    with pytest.raises((ValueError, b.DfaError)):  # the other format's cache
        b.dfa_cache_forward(*args, **good)
    torch.cuda.synchronize()
    assert b.dfa_status() == 0


def test_long_offsets(b):
    """A cache of more than 2^32 bytes: the last pages are reached."""
    Hk, ps, d = 8, 128, 256
    P = 2 ** 32 // (Hk * ps * d // 2) + 40
    kc, vc = (torch.zeros((P, Hk, ps, d // 2), dtype=torch.uint8, device=DEV) for _ in range(2))
    ks, vs = (torch.zeros((P, Hk, d // 32, ps), dtype=torch.uint8, device=DEV)
              .view(torch.float8_e5m2) for _ in range(2))
    g = torch.Generator("cpu").manual_seed(2)
    x = torch.randn((2, 200, Hk, d), generator=g).to(torch.bfloat16).to(DEV)
    table = _i32([[P - 1, P - 3]])
    b.dfa_cache4_append(x[0], x[1], _i32([0, 200]), _i32([0]), table, kc, vc, ks, vs, 200)
    q = torch.randn((4, Hk, d), generator=g).to(torch.bfloat16).to(DEV)
    out, lse = b.dfa_cache4_forward(q, kc, vc, ks, vs, table, _i32([200]), _i32([0, 4]), 4)
    k, v = b.dfa_cache4_read(kc, vc, ks, vs, table, _i32([200]), _i32([0, 200]), 200)
    assert b.dfa_status() == 0
    n, s = osam.quantise4(_f64(x))
    assert np.array_equal(_f64(torch.stack([k, v])), (n - 8) * np.repeat(s, 32, -1))
    small = [c.view(torch.uint8)[[P - 1, P - 3]].view(c.dtype) for c in (kc, vc, ks, vs)]
    o2, l2 = b.dfa_cache4_forward(q, *small, _i32([[0, 1]]), _i32([200]), _i32([0, 4]), 4)
    assert torch.equal(out, o2) and torch.equal(lse, l2) and bool(out.any())


# ------------------------------------------------------------------ together

def test_sampler_steps(b):
    """Blocks of two requests, one of them released and begun again: every step's
    attention against the definition on the cache as it stood, the cache against appends
    by the definition, and all of it read back."""
    from block_diffusion_masked_gb300 import KVCache, PageTable, rotary_func, rotary_table

    H, Hk, d, ps, bs = 4, 2, 64, 16, 8
    pages, cache = PageTable(2, 8, 11, ps), KVCache(11, ps, Hk, d, bits=4)
    table = rotary_table(128, d)
    g = torch.Generator("cpu").manual_seed(0)
    ref = [[_codes(c), _f64(s)] for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale))]
    for i, new in enumerate([[8, 8], [8, 5], [8, 0], [8, 8], [3, 8]]):
        if i == 3:
            pages.release(_i32([0, 1]))
        rows = sum(new) + 2
        qkv = torch.randn((rows, H + 2 * Hk, d), generator=g).to(torch.bfloat16).to(DEV)
        before = pages.cache_lens.tolist()
        step = pages.plan(_i32(new), rows, max(new))
        q, k = rotary_func(qkv[:, :H], qkv[:, H:H + Hk], table, step.positions)
        v = qkv[:, H + Hk:]
        out, lse = cache.attend(q, step, k, v, bs)
        cache.append(k, v, step)
        cu, tab = step.cu_new.tolist(), step.block_table.cpu().numpy()
        pages.advance(step)
        assert b.dfa_status() == 0 and int(step.missing) == 0
        p = dict(table=tab, cu=cu, lens=before, new=new, q=q, k=k, v=v,
                 values=[osam.values4(c, s) for c, s in ref])
        _check(p, bs, out, lse)
        ref = [list(osam.append4(_f64(x), cu, before, tab, c, s))
               for x, (c, s) in zip((k, v), ref)]
        for (c, s), mine, scale in zip(ref, (cache.k, cache.v), (cache.k_scale, cache.v_scale)):
            assert np.array_equal(_codes(mine), c) and np.array_equal(_f64(scale), s)
        lens = pages.cache_lens.tolist()
        cu = [0] + np.cumsum(lens).tolist()
        got = cache.read(pages, _i32(cu), cu[-1])
        assert b.dfa_status() == 0
        for x, (c, s) in zip(got, ref):
            assert np.array_equal(_f64(x), osam.cache_read(osam.values4(c, s), tab, [0, 0], cu))


@pytest.mark.parametrize("bits", [4, 8])
def test_tokens_taken_out_and_put_back(b, bits):
    """A request's tokens are read back, its pages given away, and the tokens appended to
    other pages: a row's attention over them is that of the definition on the new cache."""
    from block_diffusion_masked_gb300 import KVCache, PageTable

    Hk, d, ps = 2, 128, 32
    pages, cache = PageTable(2, 16, 24, ps), KVCache(24, ps, Hk, d, bits=bits)
    x = torch.randn((2, 300, Hk, d), device=DEV).bfloat16()
    step = pages.plan(_i32([200, 100]), 300, 200)
    cache.append(x[0], x[1], step)
    pages.advance(step)
    k, v = cache.read(pages, _i32([0, 0, 100]), 100)
    pages.release(_i32([0, 1]))
    step = pages.plan(_i32([64, 0]), 64, 64)
    cache.append(x[0][:64], x[1][:64], step)
    pages.advance(step)
    step = pages.plan(_i32([0, 100]), 100, 100)
    cache.append(k, v, step)
    pages.advance(step)
    back = cache.read(pages, _i32([0, 0, 100]), 100)
    assert b.dfa_status() == 0
    if bits == 8:  # a power of two costs e4m3 nothing but subnormals
        assert (back[0].float() - k.float()).abs().max() <= 2.0 ** -9
    else:
        n, s = osam.quantise4(_f64(torch.stack([k, v])))
        assert np.array_equal(_f64(torch.stack(back)), (n - 8) * np.repeat(s, 32, -1))


@pytest.mark.parametrize("T", [4, 40])
def test_sampler_in_a_graph_and_on_two_streams(b, T):
    """A captured step replayed over growing lengths, and two samplers on two streams at
    once, give what the same steps give eagerly on one stream."""
    from block_diffusion_masked_gb300 import KVCache, PageTable, rotary_func, rotary_table

    H, Hk, d, ps, B, steps = 8, 2, 128, 32, 3, 5
    table = rotary_table(2048, d)
    new, rows = _i32([T, T, T - 1]), 3 * T
    g = torch.Generator("cpu").manual_seed(1)
    data = [[torch.randn((rows, H + 2 * Hk, d), generator=g).to(torch.bfloat16).to(DEV)
             for _ in range(steps)] for _ in range(2)]
    prompt = [torch.randn((1100 * B, H + 2 * Hk, d), generator=g).to(torch.bfloat16).to(DEV)
              for _ in range(2)]
    cu_read = _i32([0, 9, 9, 29])
    first = _i32([1000, 0, 880])

    def begin(i):
        pages, cache = PageTable(B, 64, 64 * B, ps), KVCache(64 * B, ps, Hk, d, bits=4)
        step = pages.plan(_i32([1100, 37, 900]), 1100 * B, 1100)
        cache.append(prompt[i][:, H:H + Hk], prompt[i][:, H + Hk:], step)
        pages.advance(step)
        return pages, cache

    def one(pages, cache, qkv):
        step = pages.plan(new, rows, T)
        q, k = rotary_func(qkv[:, :H], qkv[:, H:H + Hk], table, step.positions)
        out, lse = cache.attend(q, step, k, qkv[:, H + Hk:], 4)
        cache.append(k, qkv[:, H + Hk:], step)
        pages.advance(step)
        return (out, lse, *cache.read(pages, cu_read, 29, first=first))

    def same(a, c):
        n = rows - 1
        return (torch.equal(a[0][:n], c[0][:n]) and torch.equal(a[1][:, :n], c[1][:, :n])
                and torch.equal(a[2], c[2]) and torch.equal(a[3], c[3]))

    want = []
    for i in range(2):
        state = begin(i)
        want.append([[x.clone() for x in one(*state, qkv)] for qkv in data[i]])
    torch.cuda.synchronize()
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


def _winners(p, bs):
    """Values (rows, H, d) of each row's likeliest key, and where that key is ahead of the
    next one by more than the scores may be off, and by 40 besides."""
    k, v = p["values"]
    n, ps, (H, d) = p["cu"][-1], k.shape[2], p["q"].shape[1:]
    q = _f64(p["q"])
    best, clear = np.zeros((n, H, d)), np.zeros((n, H), bool)
    for b, o in enumerate(p["lens"]):
        pages = [int(x) for x in p["table"][b][:-(-o // ps)]]
        for row in range(p["cu"][b], p["cu"][b + 1]):
            at = row - p["cu"][b]
            own = min(p["new"][b], ((o + at) // bs + 1) * bs - o) if p["k"] is not None else 0
            for h in range(H):
                hk = h // (H // k.shape[1])
                kv = []
                for c, x in ((k, p["k"]), (v, p["v"])):
                    y = np.concatenate([c[i, hk] for i in pages])[:o]
                    if own:
                        y = np.concatenate([y, _f64(x[p["cu"][b]:p["cu"][b] + own, hk])])
                    kv.append(y)
                s = kv[0] @ q[row, h] / np.sqrt(d)
                off = (d + 2) * 2.0 ** -23 * (np.abs(kv[0]) @ np.abs(q[row, h])).max() / np.sqrt(d)
                first, second = np.argsort(s)[:-3:-1]
                best[row, h] = kv[1][first]
                clear[row, h] = s[first] - s[second] > 2 * off + 2.0 ** -21 * np.abs(s).max() + 40
    return best, clear


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("H", [1, 6, 16, 40])
@pytest.mark.parametrize("own", [False, True])
@pytest.mark.parametrize("e", [24, 28, 34, 40, 60, 100, 118])
def test_attention_of_huge_queries(b, d, H, own, e):
    """Queries of 2^e on keys of some 2^-12: finite scores of up to 2^117.  The likeliest key
    has all of the probability, lse is its score, and nothing is off by a power of two or not
    a number."""
    p = _problem([300, 40], [3, 8], H, 1, d, 32, seed=17, own=own, e=(-12, -11))
    p["q"] = (p["q"].double().clamp(-1.9, 1.9) * 2.0 ** e).to(torch.bfloat16)
    if own:
        p["k"] = (p["k"].double() * 2.0 ** -11).to(torch.bfloat16)
    out, lse = _run(b, p, 8)
    assert b.dfa_status() == 0
    assert lse[:, :p["cu"][-1]].isfinite().all()
    _check(p, 8, out, lse)
    best, clear = _winners(p, 8)
    assert clear.mean() > 0.8
    off = np.abs(_f64(out)[:len(best)] - best)[clear]
    tol = (2.0 ** -8 + 2.0 ** -8 * own) * np.abs(best[clear]) + 2.0 ** -21
    assert (off <= tol).all(), off.max()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("H", [1, 6, 16, 40])
@pytest.mark.parametrize("e", [20, 30, 40, 100])
@pytest.mark.parametrize("far", ["first", "last", "all", "ahead"])
def test_attention_of_scores_far_apart(b, d, H, e, far):
    """Some keys' scores are some -2^e exactly, the first ones', the last ones' or all, the
    others' 0; or five keys' are 2^e: the likeliest keys' values have equal weights, whatever
    the reference of a row was before they came."""
    n, T = 700, 3
    p = _problem([n], [T], H, 1, d, 32, seed=18, own=False)
    at = np.arange(n)
    far_ones = {"first": at < 400, "last": at >= 300, "all": at >= 0, "ahead": at % 150 == 77}[far]
    # every code 8 (0), but for dim 0 of those keys: code 0, -8 scales of 2^-3
    codes = np.full((p["kc"].shape[0], 1, 32, d), 8)
    pages = p["table"][0]
    for i in at[far_ones]:
        codes[pages[i // 32], 0, i % 32, 0] = 0
    p["kc"] = _pack(codes).to(DEV)
    live = p["ks"].view(torch.uint8)
    for i, page in enumerate(pages[:-(-n // 32)]):
        live[int(page), :, :, :min(32, n - 32 * i)] = 0x30  # 2^-3
    p["q"].zero_()  # nothing else, so that the scores are exact
    p["q"][:, :, 0] = -2.0 ** e if far == "ahead" else 2.0 ** e
    out, lse = _run(b, p, T)
    assert b.dfa_status() == 0
    best = far_ones if far in ("all", "ahead") else ~far_ones
    score = (2.0 ** e if far == "ahead" else -2.0 ** e if far == "all" else 0.0) / np.sqrt(d)
    v = np.concatenate([p["values"][1][int(i), 0] for i in pages])[:n][best]
    # weights are f16 (2^-11), sums of n of them float32, the output bf16; a request's pieces
    # are joined by their lse, which is off by 2^-22 of itself, and so by that factor's power
    # of e: past 2^22 the pieces' weights may be any, but the output is among the values
    off = np.abs(_f64(out) - v.mean(0))
    piece = 2 * min(1, np.exp(2.0 ** -22 * abs(score)) - 1) if abs(score) < 2.0 ** 22 else 2
    assert (off <= 2.0 ** -8 * np.abs(v.mean(0))
            + (2.0 ** -10 + piece) * np.abs(v).mean(0)).all(), off.max()
    room = 2.0 ** -7 * np.abs(v).max(0)
    assert (_f64(out) <= v.max(0) + room).all() and (_f64(out) >= v.min(0) - room).all()
    want = score + np.log(best.sum())
    assert (lse.double().cpu() - want).abs().max() <= 2.0 ** -18 * (1 + abs(want))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("H", [1, 6, 16, 40])
@pytest.mark.parametrize("own", [False, True])
@pytest.mark.parametrize("e", [121, 122, 124, 126])
def test_attention_of_queries_near_the_largest(b, d, H, own, e):
    """The same for queries of up to 2^127, whose scores are still float32 numbers."""
    test_attention_of_huge_queries(b, d, H, own, e)


@pytest.mark.parametrize("e", [-14, -3, 7])
def test_append_every_significand_beside_every_scale(b, e):
    """All 128 significands of bf16, of either sign, beside every significand and sign of a
    scale, over all powers of two that give |x / s| from 1/4 to 8: the codes and scales are
    the definition's, every tie among them."""
    d, ps = 64, 128
    m = np.arange(128, 256) / 128.0
    sizes = np.concatenate([m * 2.0 ** k for k in range(-2, 4)])
    rows = []
    for scale in (4, 5, 6, 7):
        s = scale / 4 * 2.0 ** e  # 8 s is the largest magnitude of its groups
        for sign in (1, -1):
            x = np.concatenate([sizes, -sizes]) * 2.0 ** e
            x = x[(np.abs(x) < 8 * s)]  # the largest one stands alone
            x = np.concatenate([x, np.zeros(-x.size % 31)]).reshape(-1, 31)
            rows.append(np.concatenate([np.full((len(x), 1), sign * 8 * s), x], 1))
    x = torch.tensor(np.concatenate(rows))
    x = torch.cat([x, x[:x.shape[0] % 2]]).view(-1, 1, d)
    assert torch.equal(x.bfloat16().double(), x)
    x = x.bfloat16().to(DEV)
    T = x.shape[0]
    table, cu, P = _requests([0], [T], ps, 1)
    kc, ks = _cache(P, 1, ps, d, 1)
    vc, vs = _cache(P, 1, ps, d, 2)
    rc, rs = osam.append4(_f64(x), cu, [0], table, _codes(kc), _f64(ks))
    ratio = _f64(x) / np.repeat(osam.quantise4(_f64(x))[1], 32, -1)
    assert (np.abs(ratio) % 1 == 0.5).sum() >= 128 and np.abs(ratio).max() == 8
    b.dfa_cache4_append(x, -x, _i32(cu), _i32([0]), _i32(table), kc, vc, ks, vs, T)
    assert b.dfa_status() == 0
    assert np.array_equal(_f64(ks), rs) and np.array_equal(_codes(kc), rc)
    rc, rs = osam.append4(-_f64(x), cu, [0], table, _codes(vc), _f64(vs))
    assert np.array_equal(_f64(vs), rs) and np.array_equal(_codes(vc), rc)


@pytest.mark.parametrize("bits", [4, 8])
def test_read_of_more_rows_than_there_are(b, bits):
    """cu_rows past the rows of k and v is an error; the rows that there are are right."""
    lens, ps, d = [40, 20], 16, 64
    table, _, P = _requests(lens, [0, 0], ps, 6)
    if bits == 4:
        kc, ks = _cache(P, 1, ps, d, 7)
        values = osam.values4(_codes(kc), _f64(ks))
    else:
        kc = torch.randn((P, 1, ps, d), device=DEV).to(torch.float8_e4m3fn)
        ks = torch.ones((P, 1), device=DEV)
        values = _f64(kc)
    cu, first = [0, 10, 16], [20, 3]
    read = b.dfa_cache4_read if bits == 4 else b.dfa_cache_read
    args = (kc, kc, ks, ks, _i32(table), _i32(lens), _i32(cu))
    k, _ = read(*args, 12, first=_i32(first))
    assert b.dfa_status() == b.DFA_EDEVICE
    right = osam.cache_read(values, table, first, cu)
    assert np.array_equal(_f64(k), right[:12])
    assert np.array_equal(_f64(read(*args, 16, first=_i32(first))[0]), right)
    assert b.dfa_status() == 0

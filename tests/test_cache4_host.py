"""The 4-bit cache and the reading back: format arithmetic against the definition, and
refusals.  No GPU."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import sampling as osam

EINVAL, EUNSUPPORTED = -1, -2
P, NULL = ctypes.c_void_p(1 << 20), None
ODD, HALF = ctypes.c_void_p((1 << 20) + 1), ctypes.c_void_p((1 << 20) + 8)


@pytest.fixture(scope="module")
def lib():
    from block_diffusion_masked_gb300 import binding, build

    build.build()
    return binding.lib()


def test_scale_bytes(lib):
    """Every bf16 value as the largest of a group, against the definition."""
    bits = np.arange(1 << 16, dtype=np.uint32)
    value = (bits << 16).view(np.float32).astype(np.float64)
    got = np.array([lib.dfa_cache4_scale_byte(int(2 * (b & 0x7fff) + (b >> 15))) for b in bits],
                   dtype=np.uint8)
    got = torch.tensor(got).view(torch.float8_e5m2).double().numpy()
    sizes = np.array([m * 2.0 ** e for e in range(-16, 8) for m in (4, 5, 6, 7)])
    with np.errstate(invalid="ignore"):
        want = sizes[np.minimum(np.searchsorted(8 * sizes, np.abs(value)), len(sizes) - 1)]
    want = np.where(np.isfinite(value), np.where(value > 0, -want, want), np.nan)
    assert np.array_equal(got, want, equal_nan=True)


def test_definition():
    """The largest magnitude's code, ties, the other sign, zeros, limits, other values."""
    x = np.zeros((9, 32))
    x[0, :4] = 8.0, -1.0, 0.5, -0.5       # s -1: ties away from 0
    x[1, :4] = -8.0, 7.5, 8.0, 1.5        # s 1, and 8 has no code of its own
    x[2, 0] = 1e6                         # cut
    x[3, 0] = 2.0 ** -16                  # lost
    x[4, :2] = 9.0, -9.0                  # s 1.25
    x[5, 31] = np.inf
    x[6, 5] = np.nan
    x[7] = -0.0
    n, s = osam.quantise4(x)
    assert s[:, 0].tolist()[:5] == [-1.0, 1.0, -896.0, -2.0 ** -14, 1.25]
    assert np.isnan(s[5:7]).all() and s[7, 0] == s[8, 0] == 2.0 ** -14
    v = (n - 8) * np.repeat(s, 32, -1)
    assert v[0, :4].tolist() == [8.0, -1.0, 1.0, -1.0]
    assert v[1, :4].tolist() == [-8.0, 7.0, 7.0, 2.0]
    assert v[2, 0] == 7168 and v[3, 0] == 0
    assert v[4, :2].tolist() == [8.75, -8.75]
    assert (v[7:] == 0).all()


def test_error_bound():
    """Within the range no value is off by more than half a scale, but those of the other
    sign past 7.5 scales, which are off by at most one."""
    g = np.random.default_rng(0)
    x = torch.tensor(g.standard_normal((400, 64)) * np.exp(g.standard_normal((400, 1))))
    x = x.to(torch.bfloat16).double().numpy()
    n, s = osam.quantise4(x)
    s = np.repeat(s, 32, -1)
    off = np.abs((n - 8) * s - x) / np.abs(s)
    past = x / s > 7.5
    assert off[~past].max() <= 0.5 and off[past].max() <= 1.0 and past.any()
    assert (np.abs(s) * 8 >= np.abs(x)).all()


def test_packing_is_the_headers():
    """Code of dim 2i in bits 4i of a word, of dim 2i + 1 in bits 16 + 4i."""
    codes = np.array([3, 14, 0, 7, 9, 1, 15, 8])
    word = sum(int(c) << (16 * (i & 1) + 4 * (i >> 1)) for i, c in enumerate(codes))
    assert osam.codes4(np.frombuffer(word.to_bytes(4, "little"), np.uint8)).tolist() == \
        codes.tolist()


def _append(lib, **kw):
    a = dict(k=P, v=P, cu=P, lens=P, table=P, kc=P, vc=P, ks=P, vs=P, batch=2, rows=8, max_new=4,
             heads=2, d=64, ps=16, pages=4, maxp=2, kst=NULL, vst=NULL)
    a.update(kw)
    return lib.dfa_cache4_append(*a.values(), NULL)


def test_append_refusals(lib):
    for kw in (dict(k=NULL), dict(v=ODD), dict(cu=NULL), dict(lens=NULL), dict(table=NULL),
               dict(kc=NULL), dict(vc=ODD), dict(ks=NULL), dict(vs=HALF), dict(batch=-1),
               dict(rows=-1), dict(max_new=-1), dict(heads=0), dict(heads=65536), dict(ps=24),
               dict(pages=0), dict(maxp=0), dict(kst=(ctypes.c_longlong * 2)(128, 65)),
               dict(vst=(ctypes.c_longlong * 2)(100, 64)),
               dict(batch=20000, rows=1 << 21, max_new=1 << 21, heads=8)):
        assert _append(lib, **kw) == EINVAL, kw
    assert _append(lib, d=96) == EUNSUPPORTED
    for kw in (dict(batch=0), dict(rows=0), dict(max_new=0)):
        assert _append(lib, **kw) == 0


def _forward(lib, **kw):
    a = dict(q=P, k=P, v=P, kc=P, vc=P, ks=P, vs=P, table=P, lens=P, cu=P, out=P, lse=P, work=P,
             nwork=1 << 40, batch=2, rows=8, max_new=4, heads=4, kv_heads=2, d=64, bs=4, ps=16,
             pages=4, maxp=2, qst=NULL, kst=NULL, vst=NULL)
    a.update(kw)
    return lib.dfa_cache4_forward(*a.values(), NULL)


def test_forward_refusals(lib):
    for kw in (dict(q=NULL), dict(k=NULL), dict(v=NULL), dict(k=ODD), dict(kc=NULL), dict(vc=ODD),
               dict(ks=NULL), dict(vs=HALF), dict(table=NULL), dict(lens=NULL), dict(cu=NULL),
               dict(out=ODD), dict(lse=NULL), dict(work=ODD), dict(batch=-1),
               dict(batch=40000), dict(rows=-1), dict(max_new=-1), dict(heads=0),
               dict(kv_heads=3), dict(kv_heads=0), dict(kv_heads=8), dict(bs=0), dict(ps=8),
               dict(pages=0), dict(maxp=0), dict(maxp=1 << 27),
               dict(heads=1 << 16, kv_heads=1, rows=1 << 15, max_new=1 << 15)):
        assert _forward(lib, **kw) == EINVAL, kw
    assert _forward(lib, d=80) == EUNSUPPORTED
    for kw in (dict(batch=0), dict(rows=0), dict(max_new=0)):
        assert _forward(lib, **kw) == 0
    assert lib.dfa_cache4_workspace_bytes(1, 8, 8, 4, 3, 64, 16, 2) == EINVAL
    assert lib.dfa_cache4_workspace_bytes(1, 8, 8, 4, 2, 72, 16, 2) == EUNSUPPORTED
    assert lib.dfa_cache4_workspace_bytes(0, 8, 8, 4, 2, 64, 16, 2) == 0


@pytest.mark.parametrize("bits", [8, 4])
def test_read_refusals(lib, bits):
    def read(**kw):
        a = dict(kc=P, vc=P, ks=P, vs=P, table=P, lens=P, first=NULL, cu=P, k=P, v=P, batch=2,
                 rows=8, heads=2, d=64, ps=16, pages=4, maxp=2)
        a.update(kw)
        return (lib.dfa_cache_read if bits == 8 else lib.dfa_cache4_read)(*a.values(), NULL)

    for kw in (dict(kc=NULL), dict(vc=ODD), dict(ks=NULL), dict(vs=ODD), dict(table=NULL),
               dict(lens=ODD), dict(first=ODD), dict(cu=NULL), dict(k=NULL), dict(v=HALF),
               dict(batch=-1), dict(batch=40000), dict(rows=-1), dict(heads=0),
               dict(heads=65536), dict(ps=24), dict(pages=0), dict(maxp=0), dict(maxp=1 << 27)):
        assert read(**kw) == EINVAL, kw
    assert read(d=96) == EUNSUPPORTED
    for kw in (dict(batch=0), dict(rows=0)):
        assert read(**kw) == 0


def test_binding_refusals():
    from block_diffusion_masked_gb300 import KVCache
    from block_diffusion_masked_gb300 import binding as b

    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    c = KVCache(3, 16, 2, 64, device="cpu", bits=4)
    assert c.k.shape == (3, 2, 16, 32) and c.v_scale.shape == (3, 2, 2, 16)
    i = torch.zeros(2, dtype=torch.int32)
    args = (c.k, c.v, c.k_scale, c.v_scale)
    with pytest.raises(ValueError):
        KVCache(3, 16, 2, 64, device="cpu", bits=5)
    with pytest.raises(ValueError):
        b.dfa_cache4_append(x, x, i, i, i, *args, 1)  # not on a GPU
    with pytest.raises(ValueError):
        b.dfa_cache4_forward(x, *args, i, i, i, 1)
    with pytest.raises(ValueError):
        b.dfa_cache4_read(*args, i, i, i, 1)
    with pytest.raises(ValueError):
        b.dfa_cache_read(*args, i, i, i, 1)


def test_error_bound_by_the_largest_value():
    """Where a group's largest magnitude is within 2^-11 and 7168, its scale is at most 5/4 of
    an 8th of that: values are off by 5/64 of it at most, those of the sign that has no code
    -8 by an 8th.  A 16th would be too little."""
    g = np.random.default_rng(1)
    x = torch.tensor(g.standard_normal((500, 64)) * np.exp2(g.integers(-8, 10, (500, 1))))
    x[:64, 0] = torch.linspace(1, 1.984375, 64).double() * 16  # largest ones of each size
    x = x.to(torch.bfloat16).double().numpy()
    n, s = osam.quantise4(x)
    s = np.repeat(s, 32, -1)
    top = np.repeat(np.abs(x).reshape(500, 2, 32).max(-1), 32, -1)
    assert top.min() > 2.0 ** -11 and top.max() < 7168
    off, other = np.abs((n - 8) * s - x) / top, x / s > 0
    assert off[~other].max() <= 5 / 64 and off[other].max() <= 1 / 8
    assert off[~other].max() > 1 / 16


def test_values_appended_again():
    """What was read back and is appended again is rounded once more at most: some groups get a
    smaller scale, by the definition, and keep it."""
    g = np.random.default_rng(0)
    x = torch.tensor(g.standard_normal((500, 64))).to(torch.bfloat16).double().numpy()
    seen = [x]
    for _ in range(3):
        n, s = osam.quantise4(seen[-1])
        seen.append((n - 8) * np.repeat(s, 32, -1))
    changed = (seen[2] != seen[1]).reshape(500, 2, 32).any(-1).mean()
    assert 0 < changed < 0.15 and np.array_equal(seen[3], seen[2])

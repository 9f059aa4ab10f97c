"""Rotary positions on the GPU against the float64 definition.

Tolerance.  With x1, x2 exact in float32 and c, s float32, c x1 - s x2 is one
product and one fused multiply-add (or two roundings more): at most
3 * 2^-24 (|c x1| + |s x2|) <= 2^-22 max(|c|, |s|) max(|x1|, |x2|), then one
rounding to bf16, at most 2^-8 of the value (half of eps 2^-7), plus the
float32 error carried through it.
"""

import numpy as np
import pytest
import torch

from oracle import sampling as osam

pytestmark = pytest.mark.gpu


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


def _randn(shape, seed):
    g = torch.Generator("cpu").manual_seed(seed)
    return torch.randn(shape, generator=g).to(torch.bfloat16).cuda()


def _check(got, x, table, pos, inter, inverse=False):
    """got, x (rows, heads, d)."""
    ref = osam.rotary(_f64(x), table.cpu().numpy(), pos, inter, inverse)
    rot = table.shape[1]
    big = np.abs(_f64(x)).max(-1, keepdims=True) * max(1.0, float(table.abs().max()))
    tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -22 * big
    err = np.abs(_f64(got) - ref)
    used = np.asarray(pos) >= 0
    assert (err[used] <= tol[used]).all(), (err - tol)[used].max()
    # values past the turned ones are copied bit by bit
    assert torch.equal(got[torch.tensor(used)][..., rot:], x[torch.tensor(used)][..., rot:])


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("B,n,H,Hk,d,rot", [
    (1, 1, 1, 1, 64, 64), (2, 5, 3, 1, 64, 16), (1, 33, 8, 2, 128, 128), (3, 7, 5, 5, 128, 96),
    (1, 9, 4, 2, 256, 64), (2, 3, 1, 1, 256, 256), (1, 130, 6, 2, 128, 32)])
def test_layouts_and_gradients(b, B, n, H, Hk, d, rot, inter):
    from block_diffusion_masked_gb300 import rotary_func, rotary_table

    table = rotary_table(n, rot, base=100.0)
    q, k = _randn((B, 2 * n, H, d), 1).requires_grad_(), _randn((B, 2 * n, Hk, d), 2).requires_grad_()
    yq, yk = rotary_func(q, k, table, interleaved=inter)
    gq, gk = _randn(yq.shape, 3), _randn(yk.shape, 4)
    dq, dk = torch.autograd.grad((yq, yk), (q, k), (gq, gk))
    assert b.dfa_status() == 0
    pos = list(range(n)) * 2
    for i in range(B):
        for y, x, inverse in ((yq, q, False), (yk, k, False), (dq, gq, True), (dk, gk, True)):
            _check(y[i], x[i], table, pos, inter, inverse)


@pytest.mark.parametrize("inter", [False, True])
def test_gradient_against_differences(b, inter):
    """<g, R(x + e) - R(x)> = <dx, e> for a linear map: in float64 up to the
    bf16 roundings of R(x + e), R(x) and dx."""
    from block_diffusion_masked_gb300 import rotary_func, rotary_table

    n, H, d = 4, 2, 64
    table = rotary_table(n, d)
    x = _randn((1, 2 * n, H, d), 5).requires_grad_()
    g = _randn(x.shape, 6)
    y, _ = rotary_func(x, None, table, interleaved=inter)
    (dx,) = torch.autograd.grad(y, x, g)
    for seed in range(4):
        e = _randn(x.shape, 20 + seed)
        z, _ = rotary_func((x.detach().float() + 8 * e.float()).bfloat16(), None, table,
                           interleaved=inter)
        step = (x.detach().float() + 8 * e.float()).bfloat16().double() - x.detach().double()
        lhs = float((g.double() * (z.double() - y.detach().double())).sum())
        rhs = float((dx.double() * step).sum())
        tol = 2.0 ** -8 * float((g.double().abs() * (z.double().abs() + y.detach().double().abs()))
                                .sum() + (dx.double().abs() * step.abs()).sum()) * 1.01
        assert abs(lhs - rhs) <= tol


def test_gradients_of_gradients(b):
    """The map is linear in the gradients too: differentiating the backward
    pass turns forward again; q and k, either alone."""
    from block_diffusion_masked_gb300 import rotary_func, rotary_table

    table = rotary_table(3, 64)
    q, k = _randn((1, 6, 2, 64), 1).requires_grad_(), _randn((1, 6, 1, 64), 2).requires_grad_()
    gq, gk = _randn(q.shape, 3).requires_grad_(), _randn(k.shape, 4).requires_grad_()
    zq, zk = _randn(q.shape, 5), _randn(k.shape, 6)
    yq, yk = rotary_func(q, k, table)
    dq, dk = torch.autograd.grad((yq, yk), (q, k), (gq, gk), create_graph=True)
    aq, ak = torch.autograd.grad((dq, dk), (gq, gk), (zq, zk))
    pos = [0, 1, 2] * 2
    for got, x in ((aq, zq), (ak, zk)):
        _check(got[0], x[0], table, pos, False, False)
    yq, yk = rotary_func(q, k, table)
    (dk,) = torch.autograd.grad(yk, k, gk, create_graph=True)
    (ak,) = torch.autograd.grad(dk, gk, zk)
    _check(ak[0], zk[0], table, pos, False, False)
    assert b.dfa_status() == 0


def test_broadcast_inputs(b):
    """A batch and heads that are one in memory: read in place, and their
    gradient is the sum (float32 in between: half a bf16 step of each term, and
    of each partial sum)."""
    from block_diffusion_masked_gb300 import rotary_func, rotary_table

    table = rotary_table(5, 64)
    q = _randn((1, 10, 1, 64), 1).requires_grad_()
    k = _randn((1, 10, 1, 64), 2).requires_grad_()
    gq, gk = _randn((3, 10, 4, 64), 3), _randn((3, 10, 2, 64), 4)
    y = rotary_func(q.expand(3, 10, 4, 64), k.expand(3, 10, 2, 64), table)
    d = torch.autograd.grad(y, (q, k), (gq, gk))
    assert b.dfa_status() == 0
    pos = [0, 1, 2, 3, 4] * 2
    for got, x, g, out in ((d[0], q, gq, y[0]), (d[1], k, gk, y[1])):
        for i in range(3):
            _check(out[i].detach(), x[0].detach().expand(out.shape[1:]), table, pos, False, False)
        terms = np.stack([osam.rotary(_f64(g[i]), table.cpu().numpy(), pos, False, True)
                          for i in range(3)])
        want, size = terms.sum((0, 2)), np.abs(terms).sum((0, 2))
        n = terms.shape[0] * terms.shape[2]
        assert (np.abs(_f64(got)[0, :, 0] - want) <= 2.0 ** -8 * (n + 1) * size).all()


def test_captured_forward_and_backward(b):
    from block_diffusion_masked_gb300 import rotary_func, rotary_table

    table = rotary_table(9, 64)
    q, k = (_randn((2, 18, h, 64), h).requires_grad_() for h in (3, 1))
    g = [_randn(x.shape, 7) for x in (q, k)]
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):  # warm-up, its graph gone before the capture
        torch.autograd.grad(rotary_func(q, k, table), (q, k), g)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        y = rotary_func(q, k, table)
        d = torch.autograd.grad(y, (q, k), g)
    for seed in (20, 30):
        with torch.no_grad():
            for x in (q, k, *g):
                x.copy_(_randn(x.shape, seed))
        graph.replay()
        torch.cuda.synchronize()
        for i in range(2):
            for got, x, inverse in zip((*y, *d), (q, k, *g), (False, False, True, True)):
                _check(got[i].detach(), x[i].detach(), table, list(range(9)) * 2, False, inverse)
    assert b.dfa_status() == 0


@pytest.mark.parametrize("d,inter", [(64, False), (128, True), (256, False)])
def test_strided_views_and_packed_rows(b, d, inter):
    """Slices of a fused projection, far positions, rows that are not in use."""
    from block_diffusion_masked_gb300 import rotary_func, rotary_table

    rows, H, Hk = 21, 4, 2
    table = rotary_table(50000, d // 2, base=500000.0)
    qkv = _randn((rows, H + 2 * Hk, d), 7)
    q, k = qkv[:, :H], qkv[:, H:H + Hk]
    pos = [0, 49999, 31, -1, 777] + list(range(1000, 1012)) + [-1, 5, 5, -7]
    p = torch.tensor(pos, dtype=torch.int32, device="cuda")
    yq, yk = rotary_func(q, k, table, p, inter)
    assert b.dfa_status() == 0
    assert yq.is_contiguous() and yk.is_contiguous()
    _check(yq, q, table, pos, inter)
    _check(yk, k, table, pos, inter)
    for r in (3, 17, 20):  # unused: zero here, left alone by the binding
        assert not yq[r].any() and not yk[r].any()
    out = torch.full((1, rows, H, d), 7.0, dtype=torch.bfloat16, device="cuda")
    b.dfa_rotary(q[None], None, table, p[None], interleaved=inter, q_out=out)
    assert (out[0, 3] == 7).all() and (out[0, 17] == 7).all()
    assert torch.equal(out[0, :3], yq[:3])


def test_in_place_and_alone(b):
    from block_diffusion_masked_gb300 import rotary_table

    table = rotary_table(8, 128)
    x, k = _randn((2, 16, 3, 128), 8), _randn((2, 16, 1, 128), 9)
    want, wk = b.dfa_rotary(x, k, table)
    y = x.clone()
    got, none = b.dfa_rotary(y, None, table, q_out=y)
    assert none is None and got is y and torch.equal(y, want)
    # a plain sequence: positions 0 .. L - 1
    t16 = rotary_table(16, 128)
    p16 = torch.arange(16, dtype=torch.int32, device="cuda").expand(2, 16).contiguous()
    a, _ = b.dfa_rotary(x, k, t16, period=16)
    c, _ = b.dfa_rotary(x, k, t16, p16)
    assert torch.equal(a, c)
    assert b.dfa_status() == 0


def test_positions_past_the_table(b):
    from block_diffusion_masked_gb300 import rotary_table

    table = rotary_table(8, 64)
    x = _randn((1, 3, 2, 64), 10)
    pos = torch.tensor([[7, 8, 2 ** 31 - 1]], dtype=torch.int32, device="cuda")
    out = torch.full_like(x, 3.0)
    b.dfa_rotary(x, None, table, pos, q_out=out)
    assert b.dfa_status() == b.DFA_EDEVICE
    assert (out[0, 1:] == 3).all() and not (out[0, 0] == 3).all()
    b.dfa_rotary(x, None, table, pos, q_out=out, clear=True)
    assert b.dfa_status() == b.DFA_EDEVICE and not out[0, 1:].any()


def test_refusals(b):
    from block_diffusion_masked_gb300 import rotary_table

    table = rotary_table(4, 64)
    x = _randn((1, 8, 2, 64), 11)
    with pytest.raises(ValueError):
        b.dfa_rotary(x.float(), None, table)
    with pytest.raises(ValueError):
        b.dfa_rotary(x[:, :7], None, table)  # odd length without a period
    with pytest.raises(ValueError):
        b.dfa_rotary(x, x[:, :4], table)
    with pytest.raises(ValueError):
        b.dfa_rotary(x, None, table.double())
    with pytest.raises(ValueError):
        b.dfa_rotary(x, None, table, torch.zeros(8, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        b.dfa_rotary(x.transpose(2, 3), None, table)
    with pytest.raises(b.DfaError):
        b.dfa_rotary(x, None, rotary_table(3, 64))  # four positions, a table of three
    with pytest.raises(b.DfaError):
        b.dfa_rotary(x, None, table[:, :24].contiguous())


@pytest.mark.parametrize("kind", ["diffusion", "varlen", "causal"])
def test_attention_with_positions(b, kind):
    """The attention functions turn q and k first: the same outputs and
    gradients as the two calls one after the other."""
    import block_diffusion_masked_gb300 as m

    table = m.rotary_table(64, 64)
    shape = (1, 64, 2, 64)
    q, k, v = (_randn(shape, 30 + i).requires_grad_() for i in range(3))
    g = _randn(shape, 33)
    if kind == "diffusion":
        one = m.diffusion_attn_func(q, k, v, 4, rotary_table=table)
        two = m.diffusion_attn_func(*m.rotary_func(q, k, table), v, 4)
    elif kind == "causal":
        one = m.causal_attn_func(q, k, v, rotary_table=table)
        two = m.causal_attn_func(*m.rotary_func(q, k, table, period=64), v)
    else:
        pos = torch.tensor(list(range(20)) * 2 + list(range(12)) * 2, dtype=torch.int32,
                           device="cuda")
        one = m.diffusion_attn_varlen_func(q[0], k[0], v[0], [0, 40, 64], 4, rotary_table=table,
                                           positions=pos)[None]
        a, c = m.rotary_func(q[0], k[0], table, pos)
        two = m.diffusion_attn_varlen_func(a, c, v[0], [0, 40, 64], 4)[None]
    assert torch.equal(one, two)
    g1 = torch.autograd.grad(one, (q, k, v), g)
    g2 = torch.autograd.grad(two, (q, k, v), g)
    assert torch.equal(g1[1], g2[1]) and torch.equal(g1[2], g2[2])
    # dq sums float32 atomics in any order, then two roundings to bf16
    err = (g1[0].float() - g2[0].float()).abs().max() / g2[0].float().abs().max()
    assert float(err) <= 2 * 2.0 ** -8
    assert b.dfa_status() == 0


@pytest.mark.parametrize("packed", [False, True])
def test_forward_mode_tangents(b, packed):
    """A tangent turns like its input: the map is linear.  q and k, either alone,
    and beside a backward pass of the tangent."""
    import torch.autograd.forward_ad as fwad

    from block_diffusion_masked_gb300 import rotary_func, rotary_table

    table = rotary_table(5, 64)
    q, k, tq, tk = (_randn((1, 10, h, 64), s) for s, h in enumerate((3, 1, 3, 1)))
    pos, at = None, list(range(5)) * 2
    if packed:
        at = [0, 4, 2, 2, 1, 0, 3, 3, 4, 1]
        pos = torch.tensor(at, dtype=torch.int32, device="cuda")
        q, k, tq, tk = q[0], k[0], tq[0], tk[0]

    def rows(x):
        return x if packed else x[0]

    for with_q, with_k in ((True, True), (True, False), (False, True)):
        with fwad.dual_level():
            a = fwad.make_dual(q, tq) if with_q else q
            c = fwad.make_dual(k, tk) if with_k else k
            (yq, dyq), (yk, dyk) = (fwad.unpack_dual(y) for y in rotary_func(a, c, table, pos))
        for y, x in ((yq, q), (yk, k)):
            _check(rows(y), rows(x), table, at, False)
        if with_q:
            _check(rows(dyq), rows(tq), table, at, False)
        else:
            assert dyq is None or not dyq.any()
        if with_k:
            _check(rows(dyk), rows(tk), table, at, False)
        else:
            assert dyk is None or not dyk.any()
    with fwad.dual_level():  # q alone
        y, none = rotary_func(fwad.make_dual(q, tq), None, table, pos)
        assert none is None
        _check(rows(fwad.unpack_dual(y).tangent), rows(tq), table, at, False)
    # the gradient's tangent, and the gradient of a tangent
    x = q.clone().requires_grad_()
    with fwad.dual_level():
        y, _ = rotary_func(x, k, table, pos)
        (dx,) = torch.autograd.grad(y, x, fwad.make_dual(q, tq))
        primal, tangent = fwad.unpack_dual(dx)
    _check(rows(primal), rows(q), table, at, False, True)
    _check(rows(tangent), rows(tq), table, at, False, True)
    t = tq.clone().requires_grad_()
    with fwad.dual_level():
        y, _ = rotary_func(fwad.make_dual(q, t), k, table, pos)
        (dt,) = torch.autograd.grad(fwad.unpack_dual(y).tangent, t, q)
    _check(rows(dt), rows(q), table, at, False, True)
    assert b.dfa_status() == 0


@pytest.mark.parametrize("frozen", ["q", "k"])
def test_gradients_beside_a_frozen_input(b, frozen):
    from block_diffusion_masked_gb300 import rotary_func, rotary_table

    table = rotary_table(5, 64)
    q, k = _randn((1, 10, 3, 64), 1), _randn((1, 10, 1, 64), 2)
    gq, gk = _randn(q.shape, 3), _randn(k.shape, 4)
    x, g = (k, gk) if frozen == "q" else (q, gq)
    x.requires_grad_()
    y = rotary_func(q, k, table)
    torch.autograd.backward(y, (gq, gk))
    assert (q.grad is None) == (frozen == "q") and (k.grad is None) == (frozen == "k")
    _check(x.grad[0], g[0], table, list(range(5)) * 2, False, True)
    assert b.dfa_status() == 0


def test_periods_past_32_bits(b):
    """A period above the rows leaves their positions, however large it is; one
    below 1 is refused, however small."""
    from block_diffusion_masked_gb300 import rotary_func, rotary_table

    table = rotary_table(16, 64)
    x = _randn((1, 16, 2, 64), 12)
    want, _ = b.dfa_rotary(x, None, table, period=16)
    for period in (17, 2 ** 31 - 1, 2 ** 31, 2 ** 32 + 5, 2 ** 40 + 1):
        assert torch.equal(b.dfa_rotary(x, None, table, period=period)[0], want)
        assert torch.equal(rotary_func(x, None, table, period=period)[0], want)
    for period in (0, -1, -2 ** 32 + 5, -2 ** 40 + 16):
        with pytest.raises(b.DfaError):
            b.dfa_rotary(x, None, table, period=period)
    assert b.dfa_status() == 0

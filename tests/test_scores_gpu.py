"""Scores of tokens on the GPU against the float64 definitions: log probabilities,
entropies, alternatives, gradients.

Tolerances.  A term exp(x - m) is off by 2^-22 (1 + |x - m|) of itself: the exponential's
own error, and the rounding of its argument, a product of an exact difference's rounding
with a constant's.  Sums of a row of V are those of 256 threads or more, one after another
over at most V / 256 + 8 vectors' values each, then a tree of 16: at most n = V / 256 + 32
roundings of 2^-24 of the sum.  With D = sum p |log p - max log p| the logarithm of the
sum is off by at most

    e = 2^-22 (1 + D) + n 2^-24 + 2^-22 (1 + |ln S|),

the last for the logarithm itself.  A log probability adds two roundings, 2^-23 |log p|.
The entropy is ln S less a mean: its sum's terms weigh |x - m| times as much, so it is off
by e + 2^-22 sum p |x - m| (1 + |x - m|) + (n 2^-24 + 2^-22) (D + 1).  A probability in the
gradient is off by p (e + 2^-22 (2 + |log p|)), its product with the row's gradients by
2^-22 of it, and the result is rounded to the logits' type, half a step: eps / 2 of it,
and half of the type's smallest number.
"""

import math

import numpy as np
import pytest
import torch

from oracle import scores as osc

pytestmark = pytest.mark.gpu

DEV = "cuda"
TYPES = [torch.bfloat16, torch.float16, torch.float32]


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


def _logits(rows, V, dtype, seed=0, pad=0, lead=0, size=3.0, masked=0.1):
    """A slice of (rows, lead + V + pad), some tokens masked, one row nearly even."""
    g = torch.Generator("cpu").manual_seed(seed)
    x = size * torch.randn((rows, lead + V + pad), generator=g)
    x[torch.rand(x.shape, generator=g) < masked] = -math.inf
    if rows > 2:
        x[1] *= 0.01
    x[:, lead] = 1.0
    x = x.to(dtype).to(DEV)
    if pad or lead:
        x[:, :lead], x[:, lead + V:] = math.nan, math.inf  # not the rows' own
    return x[:, lead:lead + V]


def _errors(x, lp):
    """e of every row, and the entropy's bound, for log probabilities lp (rows, V)."""
    V = x.shape[1]
    n = (V / 256 + 32) * 2.0 ** -24
    with np.errstate(invalid="ignore"):
        p = np.exp(lp)
        dist = np.where(p > 0, lp.max(1, keepdims=True) - lp, 0)
        mean, square = (p * dist).sum(1), (p * dist * (1 + dist)).sum(1)
    log_s = -lp.max(1)
    e = 2.0 ** -22 * (1 + mean) + n + 2.0 ** -22 * (1 + log_s)
    return e, e + 2.0 ** -22 * square + (n + 2.0 ** -22) * (mean + 1)


def _check(x, t, top, lp, ent, best, which):
    x = _f64(x)
    rl, re, rb, rw = osc.token_logprobs(x, t, top)
    table = np.stack([osc.log_softmax(r) for r in x])
    e, eh = _errors(x, table)

    def near(got, want, tol):
        got = _f64(got)
        same = (got == want) | (np.isnan(got) & np.isnan(want))
        with np.errstate(invalid="ignore"):
            off = np.where(same, 0, np.abs(got - want))
            bound = np.where(same, 0, tol)
        assert (off <= bound).all(), (off - bound).max()

    finite = np.where(np.isfinite(rl), np.abs(rl), 0)
    if lp is not None:
        near(lp, rl, e + 2.0 ** -23 * finite)
    near(ent, re, eh)
    assert np.array_equal(which.cpu().numpy(), rw.reshape(which.shape))
    near(best, rb.reshape(best.shape),
         e[:, None] + 2.0 ** -23 * np.where(np.isfinite(rb), np.abs(rb), 0).reshape(best.shape))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,V,pad,lead,top", [
    (1, 1, 0, 0, 1), (3, 2, 0, 0, 3), (5, 7, 1, 1, 4), (2, 15, 0, 3, 32), (9, 33, 7, 0, 5),
    (20, 4099, 1, 0, 8), (4, 32768, 0, 0, 32), (2, 65003, 5, 2, 32), (700, 1000, 24, 0, 1),
    (1, 131001, 0, 0, 16), (2500, 40, 0, 0, 7), (3, 9001, 0, 5, 0)])
def test_scores(b, dtype, rows, V, pad, lead, top):
    x = _logits(rows, V, dtype, rows + V, pad, lead)
    g = torch.Generator("cpu").manual_seed(7)
    t = torch.randint(-1, V, (rows,), generator=g)
    kind = torch.int32 if V % 2 else torch.int64
    lp, ent, stats, best, which = b.dfa_token_logprobs(x, t.to(kind).to(DEV), top)
    assert b.dfa_status() == 0
    _check(x, t.tolist(), top, lp, ent, best, which)
    none = b.dfa_token_logprobs(x, None, top)
    assert none[0] is None
    for u, v in zip((ent, stats, best, which), none[1:]):
        assert torch.equal(u, v)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", ["equal", "up", "down", "few values", "one", "far", "large",
                                  "tail", "stripe", "lowest", "lowest mask", "highest"])
@pytest.mark.parametrize("V", [300, 40000])
def test_scores_of_unusual_rows(b, dtype, kind, V):
    """All alike, in order either way, many ties, one possible token, logits far apart or
    large against their spread, the largest ones all at the end or all in one thread's
    share; rows of the type's lowest value, masks of it, its highest value."""
    at = torch.arange(V, dtype=torch.float64)
    if kind == "equal":
        x = torch.full((V,), 0.5)
    elif kind in ("up", "down"):
        x = at / V * 20 * (1 if kind == "up" else -1)
    elif kind == "few values":
        x = (at * 7 % 5 == 0).double() - (at * 3 % 11 == 0).double() * 0.0
        x = torch.where(at % 13 == 0, -0.0 * x, x)
    elif kind == "one":
        x = torch.where(at == V - 3, 1.0, -math.inf)
    elif kind == "far":
        x = torch.where(at % 100 == 7, 3e4, -3e4)
    elif kind == "large":
        x = 2e4 + 64 * (at % 17)
    elif kind == "lowest":
        x = torch.full((V,), torch.finfo(dtype).min)
        x[::3] = -math.inf
    elif kind == "lowest mask":
        x = torch.where(at % 5 == 0, at % 7, torch.finfo(dtype).min)
    elif kind == "highest":
        x = torch.where(at % 90 == 4, torch.finfo(dtype).max, at % 7)
    elif kind == "tail":
        x = torch.where(at >= V - 40, 5 + at / V, 0.0)
    else:
        x = torch.where(at.long() // 8 % 256 == 9, 6 + at / V, at / V)
    x = x.to(dtype)[None].repeat(3, 1).to(DEV)
    x[1] = x[1].roll(1)
    lp, ent, _, best, which = b.dfa_token_logprobs(x, torch.tensor([0, V - 3, V - 1], device=DEV),
                                                   32)
    assert b.dfa_status() == 0
    _check(x, [0, V - 3, V - 1], 32, lp, ent, best, which)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V", [5, 20000])
def test_rows_that_are_not_numbers(b, dtype, V):
    """A NaN or +inf makes a row's scores NaN; a row of -inf has none; the others are
    right.  Their gradients: NaN, zeros, the others'."""
    x = _logits(6, V, dtype, 3, masked=0)
    x[1, V - 1], x[2, 0], x[3] = math.nan, math.inf, -math.inf
    x[4, 1] = -math.inf
    t = [0, 0, 1, 2, 1, V - 1]
    td = torch.tensor(t, device=DEV)
    lp, ent, stats, best, which = b.dfa_token_logprobs(x, td, 3)
    assert b.dfa_status() == 0
    _check(x, t, 3, lp, ent, best, which)
    assert lp[3] == -math.inf and lp[4] == -math.inf and ent[3] == 0
    ones = torch.ones(6, device=DEV)
    g = b.dfa_token_logprobs_backward(x, td, stats, ent, ones, ones)
    assert g[1:3].isnan().all() and (g[3] == 0).all() and g[[0, 4, 5]].isfinite().all()
    ones[1:3] = 0  # rows that take no part
    g = b.dfa_token_logprobs_backward(x, td, stats, ent, ones, ones)
    assert (g[1:4] == 0).all() and g.isfinite().all()


def test_tokens_that_there_are_not(b):
    x = _logits(4, 50, torch.float32)
    for kind in (torch.int32, torch.int64):
        t = torch.tensor([3, 50, 2 ** 31 - 1, -7], dtype=kind, device=DEV)
        lp, ent, stats, _, _ = b.dfa_token_logprobs(x, t)
        assert b.dfa_status() == b.DFA_EDEVICE
        assert (lp[1:] == 0).all() and lp[0] != 0 and ent.isfinite().all()
        one = torch.ones(4, device=DEV)
        g = b.dfa_token_logprobs_backward(x, t, stats, ent, one)
        assert (g[1:] == 0).all() and (g[0] != 0).any()
    t = torch.tensor([2 ** 40, 2 ** 32, -2 ** 40, 3], device=DEV)
    lp = b.dfa_token_logprobs(x, t)[0]
    assert b.dfa_status() == b.DFA_EDEVICE and (lp[:3] == 0).all() and lp[3] != 0


# ------------------------------------------------------------------ gradients

def _grad_check(x, t, gl, ge, got, dtype):
    x, gl, ge = _f64(x), _f64(gl), _f64(ge)
    want = osc.token_logprobs_grad(x, t, gl, ge)
    table = np.stack([osc.log_softmax(r) for r in x])
    e, eh = _errors(x, table)
    p = np.exp(table)
    lp = np.where(p > 0, table, 0)
    ent = np.array([osc.entropy(r) for r in table])
    gl = np.where(np.array(t) >= 0, gl, 0)
    inner = np.abs(gl)[:, None] + np.abs(ge)[:, None] * (np.abs(lp) + ent[:, None])
    tol = p * inner * (e[:, None] + 2.0 ** -22 * (4 + np.abs(lp)))
    tol += p * np.abs(ge)[:, None] * (e + eh)[:, None]
    tol += 2.0 ** -23 * np.abs(gl)[:, None] * p  # the token's own sum
    info = torch.finfo(dtype)
    # a float32 result below the smallest normal number may be lost
    tiny = info.smallest_normal if dtype != torch.float16 else info.smallest_normal * info.eps / 2
    tol += info.eps / 2 * (np.abs(want) + tol) + tiny
    at = np.array(t)
    rows = np.nonzero(at >= 0)[0]
    tol[rows, at[rows]] += 2.0 ** -23 * np.abs(gl[rows])
    off = np.abs(_f64(got) - want)
    assert (off <= tol).all(), (off - tol).max()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,V,pad,lead", [
    (1, 1, 0, 0), (3, 2, 0, 0), (5, 7, 1, 1), (9, 33, 7, 0), (20, 4099, 1, 0), (2, 65003, 0, 2),
    (700, 1000, 24, 0), (2, 32768, 0, 0)])
@pytest.mark.parametrize("which", ["logprobs", "entropy", "both"])
def test_gradients(b, dtype, rows, V, pad, lead, which):
    from block_diffusion_masked_gb300 import token_logprobs_func

    x = _logits(rows, V, dtype, rows + V, pad, lead).detach().requires_grad_()
    g = torch.Generator("cpu").manual_seed(8)
    t = torch.randint(-1, V, (rows,), generator=g)
    gl, ge = (torch.randn((rows,), generator=g).to(DEV) for _ in range(2))
    if rows > 3:
        gl[2] = ge[2] = 0
    lp, ent, _, _ = token_logprobs_func(x, t.to(DEV))
    zero = torch.zeros_like(gl)
    if which == "logprobs":
        (got,), ge = torch.autograd.grad((lp,), (x,), (gl,)), zero
    elif which == "entropy":
        (got,), gl = torch.autograd.grad((ent,), (x,), (ge,)), zero
    else:
        (got,) = torch.autograd.grad((lp, ent), (x,), (gl, ge))
    assert b.dfa_status() == 0
    assert got.dtype == dtype and got.shape == x.shape
    _grad_check(x, t.tolist(), gl, ge, got, dtype)


def test_gradient_against_differences(b):
    """float32 logits along random directions.  A central difference over steps of h is
    off by h^2 / 6 of the third derivative, which for unit-size directions and weights is
    below 16 per row here, and by the scores' own error over h."""
    from block_diffusion_masked_gb300 import token_logprobs_func

    rows, V, h = 12, 300, 2.0 ** -5
    x = _logits(rows, V, torch.float32, 4, masked=0).detach().requires_grad_()
    t = torch.arange(rows, device=DEV) * 20
    gl, ge = torch.rand(rows, device=DEV), torch.rand(rows, device=DEV)

    def total(y):
        lp, ent, _, _ = token_logprobs_func(y, t)
        return gl.double() * lp.double() + ge.double() * ent.double()

    (grad,) = torch.autograd.grad(total(x).sum(), (x,))
    way = torch.rand((rows, V), device=DEV) - 0.5
    diff = (total((x + h * way).detach()) - total((x - h * way).detach())) / (2 * h)
    assert ((grad.double() * way.double()).sum(1) - diff).abs().max() <= 16 * h * h / 6 + 2e-4


def test_shapes_and_expanded_logits(b):
    """Leading dimensions, one row, no rows, a broadcast row, a transposed vocabulary:
    what the flat call gives."""
    from block_diffusion_masked_gb300 import token_logprobs_func

    x = _logits(6, 40, torch.bfloat16, 5)
    t = torch.tensor([1, -1, 3, 4, 5, 6], device=DEV)
    flat = token_logprobs_func(x, t, 3)
    many = token_logprobs_func(x.view(2, 3, 40), t.view(2, 3), 3)
    for u, v in zip(flat, many):
        assert torch.equal(u, v.flatten(0, 1))
    one = token_logprobs_func(x[0], t[0], 3)
    assert one[0].shape == () and one[0] == flat[0][0] and torch.equal(one[3], flat[3][0])
    far = token_logprobs_func(x.t().contiguous().t(), t, 3)
    assert all(torch.equal(u, v) for u, v in zip(flat, far))
    empty = token_logprobs_func(x[:0], t[:0], 3)
    assert [tuple(y.shape) for y in empty] == [(0,), (0,), (0, 3), (0, 3)]
    base = x[:1].detach().clone().requires_grad_()
    lp, _, _, _ = token_logprobs_func(base.expand(6, 40), t)
    (got,) = torch.autograd.grad(lp.sum(), (base,))
    copy = x[:1].repeat(6, 1).requires_grad_()
    lp, _, _, _ = token_logprobs_func(copy, t)
    (rows,) = torch.autograd.grad(lp.sum(), (copy,))
    assert torch.equal(got, rows.sum(0, keepdim=True))
    z = x[:0].detach().requires_grad_()
    lp, ent, _, _ = token_logprobs_func(z, t[:0])
    assert torch.autograd.grad((lp.sum() + ent.sum()), (z,))[0].shape == (0, 40)


def test_autograd_rules(b):
    """Alternatives have no gradient; a second derivative is refused; without tokens the
    entropy alone has a gradient."""
    from block_diffusion_masked_gb300 import token_logprobs_func

    x = _logits(4, 30, torch.float32, 6).detach().requires_grad_()
    lp, ent, best, which = token_logprobs_func(x, torch.zeros(4, dtype=torch.int32, device=DEV), 2)
    assert lp.requires_grad and ent.requires_grad
    assert not best.requires_grad and not which.requires_grad
    (g,) = torch.autograd.grad(lp.sum(), (x,), create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(g.square().sum(), (x,))
    none, ent, _, _ = token_logprobs_func(x)
    assert none is None
    (g,) = torch.autograd.grad(ent.sum(), (x,))
    assert (g != 0).any()
    with torch.no_grad():
        assert not token_logprobs_func(x)[1].requires_grad


def test_tangents_are_refused(b):
    """Forward-mode tangents are not dropped silently; a level alone changes nothing."""
    import torch.autograd.forward_ad as fwad
    from block_diffusion_masked_gb300 import token_logprobs_func

    x, t = _logits(4, 30, torch.float32, 6), torch.zeros(4, dtype=torch.int64, device=DEV)
    want = token_logprobs_func(x, t)[0]
    with fwad.dual_level():
        assert torch.equal(token_logprobs_func(x, t)[0], want)
        with pytest.raises(RuntimeError):
            token_logprobs_func(fwad.make_dual(x, torch.ones_like(x)), t)


def test_sizes_past_32_bits_are_not_wrapped(b):
    """2^32 + 5 rows (of one value, expanded) are refused, not taken as 5."""
    x = torch.zeros((1, 1), device=DEV).expand(2 ** 32 + 5, 1)
    with pytest.raises(ValueError):
        b.dfa_token_logprobs(x)
    with pytest.raises(ValueError):
        b.dfa_token_logprobs_backward(x, None, x, x)


def test_refusals(b):
    x, t = _logits(4, 30, torch.float32), torch.zeros(4, dtype=torch.int64, device=DEV)
    _, ent, stats, _, _ = b.dfa_token_logprobs(x, t)
    for bad in (x.double(), x[0], x.t(), x.cpu(), x[:, :0]):
        with pytest.raises((ValueError, b.DfaError)):
            b.dfa_token_logprobs(bad, t)
    for bad in (t[:3], t.float(), t.cpu(), t.to(torch.int16), torch.zeros(8, device=DEV).long()[::2]):
        with pytest.raises(ValueError):
            b.dfa_token_logprobs(x, bad)
    for top in (-1, 33, 2 ** 32):
        with pytest.raises(ValueError):
            b.dfa_token_logprobs(x, t, top)
    g = torch.ones(4, device=DEV)
    for kw in (dict(dlogprobs=g[:3]), dict(dlogprobs=g.double()), dict(dentropy=g[::2]),
               dict(dlogits=x[:, :29]), dict(dlogits=x.bfloat16())):
        with pytest.raises(ValueError):
            b.dfa_token_logprobs_backward(x, t, stats, ent, **kw)
    with pytest.raises(ValueError):
        b.dfa_token_logprobs_backward(x, t, stats[:, :1], ent, g)
    big = _logits(2, 65003, torch.float32)
    n = b.dfa_token_logprobs_workspace_bytes(2, 65003, 4, torch.float32)
    assert n > 0
    with pytest.raises(b.DfaError):
        b.dfa_token_logprobs(big, None, 4, workspace=torch.empty(n - 1, dtype=torch.uint8,
                                                                 device=DEV))
    buf = torch.full((n + 256,), 0xA5, dtype=torch.uint8, device=DEV)
    got = b.dfa_token_logprobs(big, None, 4, workspace=buf[:n])
    assert torch.equal(got[4], b.dfa_token_logprobs(big, None, 4)[4])
    assert (buf[n:] == 0xA5).all() and b.dfa_status() == 0


def test_on_two_streams_and_in_graphs(b):
    """Calls on two streams at once, a captured call and a captured training step, replayed
    on new logits, give what calls one after another give, bit by bit."""
    from block_diffusion_masked_gb300 import token_logprobs_func

    xs = [_logits(6, 65003, torch.bfloat16, 10 + i) for i in range(8)]
    t = torch.arange(6, device=DEV)
    want = [[y.clone() for y in token_logprobs_func(x, t, 5)] for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i, x in enumerate(xs):
        with torch.cuda.stream(streams[i % 2]):
            got.append(token_logprobs_func(x, t, 5))
    torch.cuda.synchronize()
    for u, v in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(u, v))

    graphs, outs, ins = [], [], [xs[0].clone() for _ in range(2)]
    token_logprobs_func(ins[0], t, 5)
    torch.cuda.synchronize()
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(token_logprobs_func(ins[i], t, 5))
        graphs.append(graph)
    for n in range(4):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                ins[i].copy_(xs[2 * n + i])
                graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert all(torch.equal(p, q) for p, q in zip(outs[i], want[2 * n + i]))

    weight = torch.rand(6, device=DEV)
    grads = []
    for x in xs[:3]:
        y = x.detach().clone().requires_grad_()
        lp, ent, _, _ = token_logprobs_func(y, t)
        grads.append(torch.autograd.grad((lp * weight + ent).sum(), (y,))[0])
        del lp, ent, y
    leaf = xs[0].detach().clone().requires_grad_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lp, ent, _, _ = token_logprobs_func(leaf, t)
        (out,) = torch.autograd.grad((lp * weight + ent).sum(), (leaf,))
    for x, g in zip(xs, grads):
        with torch.no_grad():
            leaf.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, g)
    assert b.dfa_status() == 0


def test_long_rows_and_offsets(b):
    """Offsets past 2^32 bytes: the last of many rows; a vocabulary of millions."""
    rows, V = 2 ** 17 + 3, 2 ** 14 + 1
    x = torch.zeros((rows, V), dtype=torch.bfloat16, device=DEV)
    x[-1] = _logits(1, V, torch.bfloat16, 20)[0]
    t = torch.full((rows,), -1, device=DEV)
    t[-1] = 5
    lp, ent, stats, best, which = b.dfa_token_logprobs(x, t, 2)
    _check(x[-1:], [5], 2, lp[-1:], ent[-1:], best[-1:], which[-1:])
    assert (which[:-1] == torch.tensor([0, 1], device=DEV)).all()
    g = torch.zeros(rows, device=DEV)
    g[-1] = 1
    got = b.dfa_token_logprobs_backward(x, t, stats, ent, g)
    _grad_check(x[-1:], [5], g[-1:], 0 * g[-1:], got[-1:], torch.bfloat16)
    assert not got[:-1].any()
    del x, got
    x = _logits(1, 3_000_001, torch.float16, 21)
    lp, ent, _, best, which = b.dfa_token_logprobs(x, torch.tensor([2_999_999], device=DEV), 32)
    assert b.dfa_status() == 0
    _check(x, [2_999_999], 32, lp, ent, best, which)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("size", [-2.0 ** 21, -2.0 ** 22 + 0.25, -2.0 ** 22, -2.0 ** 22 - 0.5,
                                  -1e9, -5e9, -1e10, -1e12, -1e20, -1e30, -2e30, 1e7, 1e10, 1e30])
def test_scores_of_large_finite_logits(b, dtype, size):
    """A finite mask value of any size, in whole vectors, whole threads' shares and whole
    pieces beside ordinary logits; rows of nothing else; rows whose largest logit it is; a
    row that passes through such sizes on its way up.  Forward and gradient.

    The bounds are those of ordinary rows: a difference to the row's maximum has one
    rounding, of itself, whatever the size of the two."""
    V = 40000
    at = torch.arange(V, dtype=torch.float64)
    plain = at * 7 % 31 / 4
    rows = [torch.full((V,), size),
            torch.where(at % 5 == 0, plain, size),       # within every vector
            torch.where(at < 30000, size, plain),        # a piece's beginning, whole pieces
            torch.where(at < 10000, plain, size),        # ... its end
            torch.where(at // 8 % 256 < 40, plain, size),  # all of most threads' shares
            torch.where(at == V - 2, plain, size),       # but for one token
            torch.where(at % 3 == 0, size, -math.inf),
            -2.0 ** (101 - at // 400)]                   # -2^101 ... -2^2
    x = torch.stack([r.double() for r in rows]).to(dtype).to(DEV)
    t = [3, 5, 30001, 7, 9, V - 2, 0, V - 1]
    td = torch.tensor(t, device=DEV)
    lp, ent, stats, best, which = b.dfa_token_logprobs(x, td, 32)
    assert b.dfa_status() == 0
    _check(x, t, 32, lp, ent, best, which)
    none = b.dfa_token_logprobs(x, td, 0)  # the kernel without alternatives
    _check(x, t, 0, none[0], none[1], none[3], none[4])
    # rows of many pieces, and one piece to a row
    many = x.repeat(100, 1)
    got = b.dfa_token_logprobs(many, td.repeat(100), 3)
    _check(x, t, 3, *(got[i][:8] for i in (0, 1, 3, 4)))
    assert all(torch.equal(got[i][:8].repeat(100, *[1] * (got[i].dim() - 1)), got[i])
               for i in (0, 1, 3, 4))
    gl, ge = torch.linspace(0.5, 1, 8, device=DEV), torch.linspace(1, 0.25, 8, device=DEV)
    g = b.dfa_token_logprobs_backward(x, td, stats, ent, gl, ge)
    _grad_check(x, t, gl, ge, g, dtype)

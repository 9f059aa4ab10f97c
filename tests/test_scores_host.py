"""Scores of tokens: the float64 definitions against PyTorch and against differences,
and the refusals of the entry points.  No GPU."""

import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import scores as osc

EINVAL = -1
P, NULL, ODD = ctypes.c_void_p(1 << 20), None, ctypes.c_void_p((1 << 20) + 1)


@pytest.fixture(scope="module")
def lib():
    from block_diffusion_masked_gb300 import binding, build

    build.build()
    return binding.lib()


def _logits(rows, V, seed=0):
    g = np.random.default_rng(seed)
    x = 3 * g.standard_normal((rows, V))
    x[g.random((rows, V)) < 0.1] = -math.inf
    x[:, 0] = 1.0
    return x


def test_definitions_are_softmax_and_categorical():
    x = _logits(7, 33)
    t = np.array([0, 0, -1, 0, 0, 0, 0])
    lp, ent, best, which = osc.token_logprobs(x, t, 5)
    ref = torch.distributions.Categorical(logits=torch.tensor(x))
    assert np.allclose(lp, np.where(t < 0, 0, ref.logits[:, 0].numpy()), rtol=0, atol=1e-13)
    p = ref.probs.numpy()
    assert np.allclose(ent, -(p * np.log(np.where(p > 0, p, 1))).sum(1), rtol=0, atol=1e-13)
    top = torch.tensor(x).topk(5)
    assert np.array_equal(which, top.indices.numpy())
    assert np.allclose(np.exp(best).sum(1), np.take_along_axis(p, which, 1).sum(1))


def test_definitions_of_ties_and_impossible_tokens():
    x = np.array([[1.0, 2.0, 2.0, 1.0], [-math.inf, 0.0, -math.inf, -0.0],
                  [-math.inf] * 4, [0.0, math.inf, 0.0, 0.0], [0.0, math.nan, 0.0, 0.0]])
    lp, ent, best, which = osc.token_logprobs(x, [1, 0, 2, 0, -1], 3)
    assert which.tolist() == [[1, 2, 0], [1, 3, -1], [-1] * 3, [-1] * 3, [-1] * 3]
    assert best[1].tolist() == [math.log(0.5)] * 2 + [-math.inf]
    assert lp[1] == -math.inf and lp[2] == -math.inf and ent[2] == 0 and ent[1] == math.log(2)
    assert np.isnan([lp[3], ent[3], ent[4]]).all() and lp[4] == 0


def test_gradient_against_differences():
    x = _logits(5, 9, seed=1)
    t = [0, 3, -1, 0, 0]
    x[1, 3] = 0.25
    g = np.random.default_rng(2)
    gl, ge = g.standard_normal(5), g.standard_normal(5)
    ge[3] = 0

    def total(y):
        lp, ent, _, _ = osc.token_logprobs(y, t)
        return float((gl * lp + ge * ent).sum())

    grad, h = osc.token_logprobs_grad(x, t, gl, ge), 1e-5
    for at in np.ndindex(x.shape):
        if x[at] == -math.inf:
            assert grad[at] == 0
            continue
        up, down = x.copy(), x.copy()
        up[at] += h
        down[at] -= h
        assert abs((total(up) - total(down)) / (2 * h) - grad[at]) < 1e-8


def _forward(lib, **kw):
    a = dict(x=P, t=P, tb=8, lp=P, ent=P, st=P, tl=P, tt=P, work=P, nwork=1 << 40, rows=3, V=9,
             top=2, stride=9, dtype=0)
    a.update(kw)
    return lib.dfa_token_logprobs(*a.values(), NULL)


def _backward(lib, **kw):
    a = dict(x=P, t=P, tb=8, st=P, ent=P, gl=P, ge=P, dx=P, rows=3, V=9, stride=9, dtype=0)
    a.update(kw)
    return lib.dfa_token_logprobs_backward(*a.values(), NULL)


def test_refusals(lib):
    same = (dict(x=NULL), dict(x=ODD), dict(t=ODD), dict(tb=2), dict(rows=-1),
            dict(rows=(1 << 24) + 1), dict(V=0), dict(V=(1 << 30) + 1), dict(stride=-1),
            dict(stride=(1 << 40) + 1), dict(dtype=3), dict(dtype=-1), dict(st=NULL),
            dict(st=ctypes.c_void_p((1 << 20) + 4)))
    for kw in same + (dict(lp=NULL), dict(lp=ODD), dict(ent=NULL), dict(tl=NULL), dict(tt=ODD),
                      dict(top=-1), dict(top=33), dict(work=ctypes.c_void_p((1 << 20) + 4))):
        assert _forward(lib, **kw) == EINVAL, kw
    for kw in same + (dict(dx=NULL), dict(dx=ctypes.c_void_p((1 << 20) + 8)), dict(gl=ODD),
                      dict(ge=ODD), dict(ent=NULL)):
        assert _backward(lib, **kw) == EINVAL, kw
    assert _forward(lib, rows=0) == 0 and _backward(lib, rows=0) == 0
    size = lib.dfa_token_logprobs_workspace_bytes
    for a in ((-1, 9, 0, 0), (3, 0, 0, 0), (3, 9, 33, 0), (3, 9, -1, 0), (3, 9, 0, 7)):
        assert size(*a) == EINVAL, a
    assert size(0, 9, 0, 0) == 0


def test_binding_refusals():
    from block_diffusion_masked_gb300 import binding as b
    from block_diffusion_masked_gb300 import token_logprobs_func

    x, t = torch.zeros(3, 5), torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError):
        b.dfa_token_logprobs(x, t)  # not on a GPU
    with pytest.raises(ValueError):
        b.dfa_token_logprobs_backward(x, t, x, x)
    for bad in (t[:2], t[:, None], 7):
        with pytest.raises(ValueError):
            token_logprobs_func(x, bad)
    for bad in (torch.zeros(()), torch.zeros(3, 0), None):
        with pytest.raises(ValueError):
            token_logprobs_func(bad)

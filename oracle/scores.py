"""Plain float64 definitions of the scores of tokens.

TEST INFRASTRUCTURE ONLY, like ``oracle.attention``: log probabilities, entropies,
alternatives and gradients from logits, row by row with NumPy.
"""

from __future__ import annotations

import math

import numpy as np


def log_softmax(x):
    """log p of one row; every logit -inf: all -inf; a NaN or +inf: all NaN."""
    x = np.asarray(x, np.float64)
    if np.isnan(x).any() or np.isposinf(x).any():
        return np.full(x.shape, np.nan)
    m = x.max()
    if m == -math.inf:
        return np.full(x.shape, -math.inf)
    return x - m - math.log(np.exp(x - m).sum())


def entropy(lp):
    if np.isnan(lp).any():
        return math.nan
    p = np.exp(lp)
    return float(-(p[p > 0] * lp[p > 0]).sum())


def alternatives(x, lp, top):
    """The ``top`` likeliest tokens of a row, equal ones lowest index first."""
    if np.isnan(lp).any():
        return np.full(top, np.nan), np.full(top, -1)
    order = [i for i in np.argsort(-np.asarray(x, np.float64), kind="stable")
             if x[i] > -math.inf][:top]
    best, which = np.full(top, -math.inf), np.full(top, -1)
    best[:len(order)], which[:len(order)] = lp[order], order
    return best, which


def token_logprobs(x, tokens, top=0):
    """(logprobs, entropy, top_logprobs, top_tokens) of logits x (rows, vocab)."""
    got = []
    for row, t in zip(np.asarray(x, np.float64), tokens):
        lp = log_softmax(row)
        got.append((lp[t] if t >= 0 else 0.0, entropy(lp), *alternatives(row, lp, top)))
    return [np.array(c) for c in zip(*got)]


def token_logprobs_grad(x, tokens, dlogprobs, dentropy):
    """Gradient in x of sum(dlogprobs * logprobs + dentropy * entropy)."""
    x = np.asarray(x, np.float64)
    out = np.zeros(x.shape)
    for r, t in enumerate(tokens):
        g, h = (dlogprobs[r] if t >= 0 else 0.0), dentropy[r]
        lp = log_softmax(x[r])
        if (g == 0 and h == 0) or np.isneginf(lp).all():
            continue
        p = np.exp(lp)
        plp = np.where(p > 0, p * np.where(p > 0, lp, 0.0), 0.0 * p)
        out[r] = -g * p - h * (plp + p * entropy(lp))
        if g != 0:
            out[r, t] += g
    return out

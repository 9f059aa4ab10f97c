"""Plain float64 definitions of the sampling operators.

TEST INFRASTRUCTURE ONLY, like ``oracle.attention``: rotary positions, the
page plan, the append to a paged 8-bit cache and attention over that cache,
each written out request by request with NumPy.  A page is a Python-level
object here: no tiling, no online softmax, no packing tricks.
"""

from __future__ import annotations

import math

import numpy as np

E4M3_MAX = 448.0
MIN_EXP = -100


def rotary(x, table, positions, interleaved=False, inverse=False):
    """x (rows, heads, d), table (max_pos, rot), positions (rows,): float64."""
    x, table = np.asarray(x, np.float64), np.asarray(table, np.float64)
    rot = table.shape[1]
    y = x.copy()
    for r, pos in enumerate(positions):
        if pos < 0:
            y[r] = 0
            continue
        for i in range(rot // 2):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
            c, s = table[pos, i], table[pos, rot // 2 + i]
            if inverse:
                s = -s
            y[r, :, a] = c * x[r, :, a] - s * x[r, :, b]
            y[r, :, b] = s * x[r, :, a] + c * x[r, :, b]
    return y


def plan(cache_lens, new_lens, table, free_pages, free_count, page_size, rows):
    """(table, cu_new, positions, next_lens, next_free, missing) as lists/arrays."""
    table = np.array(table)
    top, missing = int(free_count), 0
    cu, positions, next_lens = [0], [], []
    for b, (n0, n) in enumerate(zip(cache_lens, new_lens)):
        n = min(n, rows - cu[-1])
        have = -(-n0 // page_size)
        for j in range(have, -(-(n0 + n) // page_size)):
            if j >= table.shape[1]:
                missing += 1
                continue
            if top > 0:
                top -= 1
                table[b, j] = free_pages[top]
                have = j + 1
            else:
                table[b, j] = -1
                missing += 1
        positions += range(n0, n0 + n)
        cu.append(cu[-1] + n)
        next_lens.append(min(n0 + n, have * page_size))
    positions += [-1] * (rows - len(positions))
    return table, cu, positions, next_lens, top, missing


def round_e4m3(x):
    """Nearest e4m3 value (ties to even) of float64 values within +-448; NaN kept."""
    x = np.asarray(x, np.float64)
    out = np.full(x.shape, np.nan)
    ok = np.isfinite(x)
    mag = np.abs(x[ok])
    exp = np.floor(np.log2(np.where(mag > 0, mag, 1.0)))
    exp = np.where(2.0 ** exp > mag, exp - 1, exp)
    exp = np.where(2.0 ** (exp + 1) <= mag, exp + 1, exp)
    step = 2.0 ** (np.maximum(exp, -6) - 3)  # 3 mantissa bits, smallest normal 2^-6
    out[ok] = np.sign(x[ok]) * np.round(mag / step) * step  # np.round: ties to even
    assert not (np.abs(out[ok]) > E4M3_MAX).any()
    return out


def page_scale(amax):
    """Smallest 2^e, e >= MIN_EXP, with amax <= 448 * 2^e."""
    e = MIN_EXP
    while amax > E4M3_MAX * 2.0 ** e:
        e += 1
    return 2.0 ** e


def append(x, cu_new, cache_lens, table, cache, scale):
    """Append packed x (rows, kv_heads, d) to cache (pages, kv_heads, ps, d), float64
    e4m3 values, and scale (pages, kv_heads); returns new copies."""
    cache, scale = np.array(cache, np.float64), np.array(scale, np.float64)
    x = np.asarray(x, np.float64)
    ps = cache.shape[2]
    for b, n0 in enumerate(cache_lens):
        end = n0 + cu_new[b + 1] - cu_new[b]
        for j in range(n0 // ps, -(-end // ps)):
            lo, hi = max(n0, j * ps), min(end, (j + 1) * ps)
            if lo >= hi:
                continue
            page, held = table[b][j], lo - j * ps
            for h in range(cache.shape[1]):
                new = x[cu_new[b] + lo - n0:cu_new[b] + hi - n0, h]
                fin = np.abs(new[np.isfinite(new)])
                s = page_scale(fin.max() if fin.size else 0.0)
                if held:
                    old = scale[page, h]
                    if old >= s:
                        s = old
                    else:
                        cache[page, h, :held] = round_e4m3(cache[page, h, :held] * (old / s))
                scale[page, h] = s
                cache[page, h, held:held + hi - lo] = round_e4m3(new / s)
    return cache, scale


def quantise4(x):
    """Codes 0 .. 15 and scales of x (..., d) in groups of 32 along d: the scale's size
    is the smallest of {4, 5, 6, 7} 2^e, within [2^-14, 896], that is at least the
    largest magnitude over 8; negative where a positive value alone has that magnitude.
    Codes are 8 + x / scale to the nearest, ties away from 0, within 0 .. 15.  A group
    with a value that is not finite has scale NaN (and codes of no meaning)."""
    x = np.asarray(x, np.float64)
    g = x.reshape(*x.shape[:-1], -1, 32)
    codes, scales = np.zeros(g.shape, np.int64), np.full(g.shape[:-1], np.nan)
    sizes = [m * 2.0 ** e for e in range(-16, 8) for m in (4, 5, 6, 7)]
    assert sizes[0] == 2.0 ** -14 and sizes[-1] == 896
    for at in np.ndindex(scales.shape):
        y = g[at]
        if not np.isfinite(y).all():
            continue
        top = np.abs(y).max()
        s = next((s for s in sizes if 8 * s >= top), sizes[-1])
        if top > 0 and -top not in y:
            s = -s
        n = np.sign(y / s) * np.floor(np.abs(y / s) + 0.5)
        codes[at], scales[at] = np.clip(n, -8, 7) + 8, s
    return codes.reshape(x.shape), scales


def codes4(packed):
    """Codes (..., d) of bytes (..., d / 2): eight to a little-endian 32-bit word, those
    of even dims in its low half, of odd ones in its high half."""
    words = np.ascontiguousarray(packed, np.uint8).view("<u4")
    at = [16 * (i % 2) + 4 * (i // 2) for i in range(8)]
    out = np.stack([(words >> a) & 15 for a in at], -1).astype(np.int64)
    return out.reshape(*words.shape[:-1], -1)


def values4(codes, scales):
    """Values (..., ps, d) of codes (..., ps, d) and scales (..., d / 32, ps)."""
    s = np.repeat(np.swapaxes(scales, -1, -2), 32, -1)
    return (np.asarray(codes, np.float64) - 8) * s


def append4(x, cu_new, cache_lens, table, codes, scales):
    """Append packed x (rows, kv_heads, d) to codes (pages, kv_heads, ps, d) and scales
    (pages, kv_heads, d / 32, ps); returns new copies."""
    codes, scales = np.array(codes), np.array(scales, np.float64)
    n, s = quantise4(x)
    ps = codes.shape[2]
    for b, n0 in enumerate(cache_lens):
        for row in range(cu_new[b], cu_new[b + 1]):
            pos = n0 + row - cu_new[b]
            page = table[b][pos // ps]
            codes[page, :, pos % ps] = n[row]
            scales[page, :, :, pos % ps] = s[row]
    return codes, scales


def cache_read(values, table, first, cu_rows):
    """Rows (rows, kv_heads, d) of the tokens first[b], first[b] + 1, ... of each
    request, from values (pages, kv_heads, ps, d); rows of no request are NaN."""
    ps = values.shape[2]
    out = np.full((cu_rows[-1], values.shape[1], values.shape[3]), np.nan)
    for b, f in enumerate(first):
        for row in range(cu_rows[b], cu_rows[b + 1]):
            pos = f + row - cu_rows[b]
            out[row] = values[table[b][pos // ps], :, pos % ps]
    return out


def cache_attention(q, k_cache, v_cache, k_scale, v_scale, table, cache_lens, cu_new, k=None,
                    v=None, block_size=1):
    """Attention of packed rows q (rows, H, d); caches are float64 e4m3 values.

    Returns out (rows, H, d), lse (H, rows) and, for error bounds, the sums
    sum_j p_j |v_j| (rows, H, d) and max_j scale * sum_i |q_i| |k_ji| (H, rows).
    Rows of no request are NaN.
    """
    q = np.asarray(q, np.float64)
    rows, H, d = q.shape
    Hk, ps = k_cache.shape[1], k_cache.shape[2]
    out, absout = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    lse, big = np.full((H, rows), np.nan), np.zeros((H, rows))
    for b, n0 in enumerate(cache_lens):
        for row in range(cu_new[b], cu_new[b + 1]):
            i = row - cu_new[b]
            own = 0
            if k is not None:
                end = ((n0 + i) // block_size + 1) * block_size
                own = min(cu_new[b + 1] - cu_new[b], end - n0)
            for h in range(H):
                hk = h // (H // Hk)
                ks, vs = [], []
                for j in range(0, n0, ps):
                    page, m = table[b][j // ps], min(ps, n0 - j)
                    ks.append(k_cache[page, hk, :m] * k_scale[page, hk])
                    vs.append(v_cache[page, hk, :m] * v_scale[page, hk])
                if own:
                    ks.append(np.asarray(k[cu_new[b]:cu_new[b] + own, hk], np.float64))
                    vs.append(np.asarray(v[cu_new[b]:cu_new[b] + own, hk], np.float64))
                if not ks:
                    out[row, h] = absout[row, h] = 0
                    lse[h, row] = -math.inf
                    continue
                kk, vv = np.concatenate(ks), np.concatenate(vs)
                s = kk @ q[row, h] / math.sqrt(d)
                top = s.max()
                p = np.exp(s - top)
                lse[h, row] = top + math.log(p.sum())
                p /= p.sum()
                out[row, h] = p @ vv
                absout[row, h] = p @ np.abs(vv)
                big[h, row] = (np.abs(kk) @ np.abs(q[row, h])).max() / math.sqrt(d)
    return out, lse, absout, big

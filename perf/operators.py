"""The operators of a block-diffusion sampler, as calls to be measured.

Four operators: rotary positions of queries and keys (forward and backward),
the page plan of a sampling step, the append of finished tokens to a paged
8-bit key/value cache, and attention of new rows over that cache.  ``run``
computes each in elementary torch operations, or, where ``own`` is true,
through the package.

Cache layout: k_cache, v_cache (pages, kv_heads, page_size, headdim) e4m3;
k_scale, v_scale (pages, kv_heads) float32 powers of two; block_table
(batch, max_pages) int32 page numbers; cache_lens (batch,) int32 tokens held.
New rows are packed: sequence b has rows [cu_new[b], cu_new[b + 1]), at the
positions that follow its cached tokens.
"""

import math

import torch

own = False

DEV = "cuda"
MIN_EXP = -100  # the smallest scale of a page is 2^MIN_EXP


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one decoding step's rows, far positions, packed: latency counts
        dict(name="rotary packed decode", op="rotary", B=1, L=64, H=32, Hk=8, d=128, rot=128,
             inter=False, back=False, packed=True, fused=True),
        # q and k of the mid training workload (B=4, n=2048, H=32), forward and backward
        dict(name="rotary train mid", op="rotary", B=4, L=4096, H=32, Hk=32, d=128, rot=128,
             inter=False, back=True, packed=False, fused=False),
        # the longest workload's odd neighbour: interleaved pairs on half of each head
        dict(name="rotary long interleaved", op="rotary", B=1, L=16382, H=16, Hk=4, d=256, rot=128,
             inter=True, back=True, packed=False, fused=True),
        # a handful of requests, one block of 16 tokens each
        dict(name="plan few requests", op="plan", B=5, ctx=700, new=16, ps=64, maxp=32),
        # a full batch of long requests
        dict(name="plan many requests", op="plan", B=1024, ctx=16000, new=32, ps=64, maxp=256),
        # one token for each of 64 requests (block_size 1)
        dict(name="append one token", op="append", B=64, ctx=1000, new=1, Hk=8, d=128, ps=64),
        # a finished block of 32 for each of 127 requests, pages partly filled
        dict(name="append blocks", op="append", B=127, ctx=2000, new=32, Hk=8, d=128, ps=32),
        # the prompts of 8 requests
        dict(name="append prompts", op="append", B=8, ctx=0, new=8190, Hk=8, d=128, ps=64),
        # one request, one token that was appended before: the latency of a step
        dict(name="attn one token", op="attn", B=1, ctx=500, new=1, H=16, Hk=4, d=128, ps=64, bs=1,
             ragged=False, mine=False),
        # ragged batch, blocks of 4 as in the mid workload, grouped heads
        dict(name="attn blocks of 4", op="attn", B=24, ctx=8000, new=4, H=32, Hk=8, d=128, ps=64,
             bs=4, ragged=True, mine=True),
        # blocks of 32 with four query heads to a key head: 128 rows for each key
        dict(name="attn blocks of 32", op="attn", B=32, ctx=8192, new=32, H=32, Hk=8, d=128, ps=64,
             bs=32, ragged=True, mine=True),
        # a single long context, headdim 64, a block of 16
        dict(name="attn long context", op="attn", B=1, ctx=131000, new=16, H=16, Hk=16, d=64,
             ps=128, bs=16, ragged=False, mine=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "plan", "append", "attn", "attn"])
    if op == "rotary":
        d = rng.choice([64, 128, 256])
        Hk = rng.choice([1, 2, 4, 8])
        H = Hk * rng.choice([1, 2, 4])
        B = rng.choice([1, 2, 3, 4])
        packed = rng.random() < 0.4
        L = _log(rng, 1, 8192) if packed else 2 * _log(rng, 1, 8192)
        L = min(L, 2 * (2 ** 26 // (B * H * d)))
        return dict(op=op, B=1 if packed else B, L=L, H=H, Hk=Hk, d=d,
                    rot=rng.choice([d, d // 2, 32]), inter=rng.random() < 0.5,
                    back=rng.random() < 0.5, packed=packed, fused=rng.random() < 0.5)
    if op == "plan":
        ps = rng.choice([16, 32, 64, 128])
        ctx, new = _log(rng, 1, 16000), _log(rng, 1, 128)
        return dict(op=op, B=_log(rng, 1, 1024), ctx=ctx, new=new, ps=ps,
                    maxp=(ctx + new) // ps + 1 + rng.randrange(8))
    if op == "append":
        B, Hk = _log(rng, 1, 128), rng.choice([1, 2, 4, 8])
        return dict(op=op, B=B, ctx=_log(rng, 1, 4000), new=_log(rng, 1, min(8190, 32768 // B)),
                    Hk=Hk, d=rng.choice([64, 128, 256]), ps=rng.choice([16, 32, 64, 128]))
    d, Hk, G = rng.choice([64, 128, 256]), rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 8])
    B, new = _log(rng, 1, 64), _log(rng, 1, 64)
    ctx = _log(rng, 1, 131000)
    # at most the keys and the products of the largest listed case
    ctx = max(1, min(ctx, 32 * 8192 * 8 * 128 // (B * Hk * d), 2 ** 28 // (B * Hk * G * new)))
    return dict(op="attn", B=B, ctx=ctx, new=new, H=Hk * G, Hk=Hk, d=d,
                ps=rng.choice([16, 32, 64, 128]), bs=rng.choice([1, 4, new, new]),
                ragged=rng.random() < 0.6, mine=rng.random() < 0.8)


def _lens(case):
    """Tokens cached and new of each request: from the case alone."""
    B, ctx, new = case["B"], case["ctx"], case["new"]
    if case["op"] == "attn" and not case["ragged"]:
        return [ctx] * B, [new] * B
    old = [int(ctx * (0.25 + 0.75 * ((0.6180339887 * b) % 1.0))) for b in range(B)]
    old[0] = ctx
    add = [new] * B
    if B > 6:
        old[3] = 0              # a request that has just begun
        add[5] = 0              # one that has nothing to add
        add[6] = (new + 1) // 2  # a short last block
    return old, add


def work(case):
    op = case["op"]
    if op == "rotary":
        heads, d = case["H"] + case["Hk"], case["d"]
        rows = case["B"] * case["L"]
        times = 2 if case["back"] else 1
        table = 4 * case["rot"] * (case["L"] if case["packed"] else case["L"] // 2)
        return {"bytes": times * (4 * rows * heads * d + table),
                "flops": times * 3 * rows * heads * case["rot"]}
    old, add = _lens(case)
    B, ps = case["B"], case.get("ps", 64)
    if op == "plan":
        pages = sum(-(-(o + a) // ps) - -(-o // ps) for o, a in zip(old, add))
        return {"bytes": 4 * (4 * B + sum(add) + 2 * pages), "flops": 0}
    Hk, d = case["Hk"], case["d"]
    if op == "append":
        return {"bytes": 2 * sum(add) * Hk * d * 3, "flops": 4 * sum(add) * Hk * d}
    H = case["H"]
    keys = sum(o for o, a in zip(old, add) if a)
    pairs = sum(a * o + case["mine"] * _own_pairs(o, a, case["bs"]) for o, a in zip(old, add))
    return {"bytes": 2 * keys * Hk * d + sum(add) * (4 * (H + case["mine"] * Hk) * d + 4 * H),
            "flops": 4 * pairs * H * d}


def _own_pairs(o, a, bs):
    """Pairs of own rows and own keys of the rows' blocks or earlier ones."""
    return sum(min(a, ((o + i) // bs + 1) * bs - o) for i in range(a))


# ------------------------------------------------------------------ the inputs

def _gen(seed):
    return torch.Generator(DEV).manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _scan(x):
    return [0] + torch.tensor(x).cumsum(0).tolist()


def _table(rows, rot, base=500000.0):
    """cos and sin of position * base^(-2i/rot), from 64-bit angles."""
    freq = base ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
    ang = torch.arange(rows, device=DEV, dtype=torch.float64)[:, None] * freq
    return torch.cat([ang.cos(), ang.sin()], 1).float()


def _pages(case, old, add, g):
    """Page numbers in random order for every request, unused entries -1."""
    ps, B = case["ps"], case["B"]
    need = [-(-(o + a) // ps) for o, a in zip(old, add)]
    maxp = max(1, max(need))
    total = sum(need) + 3
    perm = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    start = _ints(_scan(need)[:-1])[:, None]
    j = torch.arange(maxp, device=DEV)
    table = perm[(start + j).clamp(max=total - 1).long()]
    return torch.where(j < _ints(need)[:, None], table, -1).to(torch.int32).contiguous(), total


def _quantised(g, pages, Hk, ps, d):
    """Random e4m3 pages and their power-of-two scales."""
    x = _randn(g, pages, Hk, ps, d)
    x *= torch.exp(0.5 * _randn(g, pages, Hk, 1, 1))
    e = _exponent(x.abs().amax((2, 3)))
    return (x / _pow2(e)[:, :, None, None]).to(torch.float8_e4m3fn), _pow2(e)


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    if op == "rotary":
        B, L, H, Hk, d = (case[k] for k in ("B", "L", "H", "Hk", "d"))
        if case["fused"]:  # views of one projection's output
            qkv = _randn(g, B, L, H + 2 * Hk, d).bfloat16()
            q, k = qkv[:, :, :H], qkv[:, :, H:H + Hk]
        else:
            q, k = _randn(g, B, L, H, d).bfloat16(), _randn(g, B, L, Hk, d).bfloat16()
        s = dict(op=op, inter=case["inter"], rot=case["rot"], back=case["back"], pos=None)
        if case["packed"]:
            rows = 131072
            s["pos"] = torch.randint(0, rows, (L,), generator=g, device=DEV, dtype=torch.int32)
            q, k = q[0], k[0]
        else:
            rows = L // 2
        s["table"] = _table(rows, case["rot"])
        if case["back"]:
            q, k = q.detach().requires_grad_(), k.detach().requires_grad_()
            s["gq"] = _randn(g, *q.shape).bfloat16()
            s["gk"] = _randn(g, *k.shape).bfloat16()
        return dict(s, q=q, k=k)
    old, add = _lens(case)
    if op == "plan":
        ps, B = case["ps"], case["B"]
        table, total = _pages(dict(case), old, [0] * B, g)
        wide = torch.full((B, case["maxp"]), -1, dtype=torch.int32, device=DEV)
        n = min(case["maxp"], table.shape[1])
        wide[:, :n] = table[:, :n]
        spare = sum(-(-(o + a) // ps) - -(-o // ps) for o, a in zip(old, add))
        free = torch.randperm(total + spare + 9, generator=g, device=DEV).to(torch.int32)
        return dict(op=op, lens=_ints(old), new=_ints(add), table=wide, free=free,
                    count=_ints([spare + 5]), ps=ps, rows=sum(add) + 7)
    Hk, d, ps = case["Hk"], case["d"], case["ps"]
    table, total = _pages(case, old, add, g)
    kc, ks = _quantised(g, total, Hk, ps, d)
    vc, vs = _quantised(g, total, Hk, ps, d)
    rows = sum(add)
    amp = torch.exp(0.5 * _randn(g, rows, Hk, 1))
    k = (_randn(g, rows, Hk, d) * amp).bfloat16()
    v = (_randn(g, rows, Hk, d) * amp).bfloat16()
    s = dict(op=op, kc=kc, ks=ks, vc=vc, vs=vs, table=table, lens=_ints(old), cu=_ints(_scan(add)),
             k=k, v=v, max_new=max(add), ps=ps)
    if op == "append":
        return s
    # what lies behind a request's last token is not a number
    span = torch.arange(ps, device=DEV)
    for c in (kc, vc):
        j = torch.arange(table.shape[1], device=DEV)
        left = (s["lens"][:, None] - j * ps).clamp(0, ps)            # tokens of each page
        page = torch.where(table >= 0, table, total).long()
        keep = torch.zeros(total + 1, device=DEV, dtype=torch.int64)
        keep[page.reshape(-1)] = left.reshape(-1).long()
        dead = (span >= keep[:total, None])[:, None, :, None]
        c.view(torch.uint8).masked_fill_(dead, 0x7F)
    q = _randn(g, rows, case["H"], d).bfloat16()
    if not case["mine"]:  # the rows' own tokens are in the cache, or are none of its
        s["k"] = s["v"] = None
    return dict(s, q=q, bs=case["bs"], ctx=max(old))


# ------------------------------------------------------------------ one pass

def run(state):
    return {"rotary": _rotary, "plan": _plan, "append": _append, "attn": _attn}[state["op"]](state)


def _rotary(s):
    if own:
        import block_diffusion_masked_gb300 as m

        q, k = m.rotary_func(s["q"], s["k"], s["table"], positions=s["pos"], interleaved=s["inter"])
        if not s["back"]:
            return [q, k]
        dq, dk = torch.autograd.grad((q, k), (s["q"], s["k"]), (s["gq"], s["gk"]))
        return [q, k, dq, dk]
    got = [_turn(s["q"].detach(), s, 1.0), _turn(s["k"].detach(), s, 1.0)]
    if s["back"]:
        got += [_turn(s["gq"], s, -1.0), _turn(s["gk"], s, -1.0)]
    return got


def _turn(x, s, sign):
    """Rotate (sign 1) or rotate back (sign -1) the first rot values of each head."""
    rot, L = s["rot"], x.shape[-3]
    pos = s["pos"].long() if s["pos"] is not None else \
        torch.arange(L, device=x.device) % (L // 2)
    t = s["table"][pos]
    c, n = t[:, None, :rot // 2], sign * t[:, None, rot // 2:]
    y = x.float()
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if s["inter"] else \
        (y[..., :rot // 2], y[..., rot // 2:rot])
    u, w = c * a - n * b, n * a + c * b
    first = torch.stack([u, w], -1).flatten(-2) if s["inter"] else torch.cat([u, w], -1)
    return torch.cat([first, y[..., rot:]], -1).to(x.dtype)


def _plan(s):
    if own:
        from block_diffusion_masked_gb300 import binding

        return list(binding.dfa_cache_plan(s["lens"], s["new"], s["table"], s["free"], s["count"],
                                           s["ps"], s["rows"]))
    lens, new, ps = s["lens"].long(), s["new"].long(), s["ps"]
    has = (lens + ps - 1) // ps
    need = (lens + new + ps - 1) // ps - has
    before = need.cumsum(0) - need
    j = torch.arange(s["table"].shape[1], device=lens.device)
    local = j - has[:, None]
    at = (s["count"].long() - 1 - before[:, None] - local).clamp(0, s["free"].numel() - 1)
    table = torch.where((local >= 0) & (local < need[:, None]), s["free"][at], s["table"])
    ends = new.cumsum(0)
    cu = torch.cat([torch.zeros_like(ends[:1]), ends])
    r = torch.arange(s["rows"], device=lens.device)
    b = torch.searchsorted(ends, r, right=True).clamp(max=lens.numel() - 1)
    pos = torch.where(r < ends[-1], lens[b] + r - cu[b], -1)
    left = s["count"].long() - need.sum()
    i32 = torch.int32
    return [table, cu.to(i32), pos.to(i32), (lens + new).to(i32), left.clamp(min=0).to(i32),
            (-left).clamp(min=0).to(i32)]


def _exponent(amax):
    """The smallest e >= MIN_EXP with amax <= 448 * 2^e."""
    m, e = torch.frexp(amax)  # amax = m * 2^e, 0.5 <= m < 1; 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8)
    return torch.where(amax > 0, e, MIN_EXP).clamp(min=MIN_EXP)


def _pow2(e):
    """2^e as float32, -126 <= e <= 127, from its bits."""
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _row_owner(cu, rows):
    r = torch.arange(rows, device=cu.device)
    b = torch.searchsorted(cu[1:].contiguous(), r, right=True).clamp(max=cu.numel() - 2)
    return b, r - cu[b]


def _append(s):
    if own:
        from block_diffusion_masked_gb300 import binding

        binding.dfa_cache_append(s["k"], s["v"], s["cu"], s["lens"], s["table"], s["kc"], s["vc"],
                                 s["ks"], s["vs"], s["max_new"])
    else:
        _append_one(s, s["k"], s["kc"], s["ks"])
        _append_one(s, s["v"], s["vc"], s["vs"])
    return [s["kc"], s["vc"], s["ks"], s["vs"]]


def _append_one(s, x, cache, scale):
    ps, rows = s["ps"], x.shape[0]
    b, i = _row_owner(s["cu"].long(), rows)
    old = s["lens"].long()
    pos = old[b] + i
    page = s["table"][b, pos // ps].long()
    x = x.float()
    top = torch.zeros_like(scale)
    top.index_reduce_(0, page, x.abs().amax(-1), "amax")
    # the pages that get rows, and whether they held tokens before this call
    fresh = torch.zeros(scale.shape[0], device=x.device)
    fresh.index_reduce_(0, page, 1.0 + (old[b] <= pos // ps * ps), "amax")
    want = _pow2(_exponent(top))
    now = torch.where(fresh[:, None] == 0, scale,
                      torch.where(fresh[:, None] == 2, want, torch.maximum(scale, want)))
    grown = (fresh == 1)[:, None] & (now > scale)
    again = (cache.float() * (scale / now)[:, :, None, None]).to(torch.float8_e4m3fn)
    keep = torch.zeros(scale.shape[0], device=x.device, dtype=torch.int64)
    keep[page] = (old[b] - pos // ps * ps).clamp(0, ps)
    held = torch.arange(ps, device=x.device) < keep[:, None]
    redo = grown[:, :, None, None] & held[:, None, :, None]
    raw = cache.view(torch.uint8)
    raw.copy_(torch.where(redo, again.view(torch.uint8), raw))
    raw[page, :, pos % ps] = (x / now[page][:, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    scale.copy_(now)


def _attn(s):
    if own:
        from block_diffusion_masked_gb300 import binding

        return list(binding.dfa_cache_forward(
            s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["lens"], s["cu"],
            s["max_new"], k=s["k"], v=s["v"], block_size=s["bs"]))
    q, ps, bs, T, S = s["q"], s["ps"], s["bs"], s["max_new"], s["ctx"]
    rows, H, d = q.shape
    Hk = s["kc"].shape[1]
    lens, cu = s["lens"].long(), s["cu"].long()
    B = lens.numel()
    at = torch.arange(S, device=q.device)
    page = s["table"][:, at // ps].clamp(min=0).long()
    row = (cu[:-1, None] + torch.arange(T, device=q.device)).clamp(max=rows - 1)
    seen = at < lens[:, None]

    def keys(cache, scale, mine):
        x = cache.view(torch.uint8)[page, :, at % ps].view(torch.float8_e4m3fn).float()
        x = torch.where(seen[:, :, None, None], x * scale[page][..., None], 0.0)
        if mine is not None:
            x = torch.cat([x, mine[row].float()], 1)
        return x.transpose(1, 2)  # (B, Hk, S + T, d)

    qg = q[row].float().view(B, T, Hk, H // Hk, d).permute(0, 2, 3, 1, 4).reshape(B, Hk, -1, d)
    w = (qg @ keys(s["kc"], s["ks"], s["k"]).transpose(2, 3)) / math.sqrt(d)
    i = torch.arange(T, device=q.device)
    there = i < (cu[1:] - cu[:-1])[:, None]
    blk = (lens[:, None] + i) // bs
    mine = there[:, None, :] & (blk[:, None, :] <= blk[:, :, None])
    see = seen[:, None, :].expand(B, T, S)
    if s["k"] is not None:
        see = torch.cat([see, mine], 2)
    see = see[:, None, None].expand(B, 1, H // Hk, T, -1).reshape(B, 1, H // Hk * T, -1)
    w = w.masked_fill_(~see, -math.inf)
    m = w.amax(-1, keepdim=True).clamp(min=-1e30)
    w = w.sub_(m).exp_()
    den = w.sum(-1, keepdim=True)
    o = (w @ keys(s["vc"], s["vs"], s["v"])) / den.clamp(min=1e-38)
    lse = torch.where(den > 0, m + den.log(), -math.inf)
    shape = (B, Hk, H // Hk, T)
    o = o.view(*shape, d).permute(0, 3, 1, 2, 4).reshape(B, T, H, d)
    lse = lse.view(shape).permute(0, 3, 1, 2).reshape(B, T, H)
    b, i = _row_owner(cu, rows)
    return [o[b, i].to(q.dtype), lse[b, i].t().contiguous()]


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"rotary": _exact_rotary, "plan": _exact_plan, "append": _exact_append,
            "attn": _exact_attn}[s["op"]](s)


def _exact_rotary(s):
    def spin(x, back):
        L, rot = x.shape[-3], s["rot"]
        pos = s["pos"].long() if s["pos"] is not None else \
            torch.arange(L // 2, device=x.device).repeat(2)
        t = s["table"].double()[pos]
        z = torch.complex(t[:, :rot // 2], t[:, rot // 2:])
        z = (z.conj() if back else z)[:, None]
        y = x.detach().double()
        if s["inter"]:
            out = torch.view_as_real(torch.view_as_complex(
                y[..., :rot].unflatten(-1, (-1, 2)).contiguous()) * z).flatten(-2)
        else:
            out = torch.complex(y[..., :rot // 2].contiguous(),
                                y[..., rot // 2:rot].contiguous()) * z
            out = torch.cat([out.real, out.imag], -1)
        return torch.cat([out, y[..., rot:]], -1)

    got = [spin(s["q"], False), spin(s["k"], False)]
    return got + [spin(s["gq"], True), spin(s["gk"], True)] if s["back"] else got


def _exact_plan(s):
    lens, new, ps = s["lens"].tolist(), s["new"].tolist(), s["ps"]
    table, free, top = s["table"].cpu().numpy().copy(), s["free"].tolist(), s["count"].item()
    cu, pos = [0], []
    for b, (o, a) in enumerate(zip(lens, new)):
        for j in range(-(-o // ps), -(-(o + a) // ps)):
            top -= 1
            table[b, j] = free[top]
        pos += range(o, o + a)
        cu.append(cu[-1] + a)
    pos += [-1] * (s["rows"] - len(pos))
    return [_ints(x) for x in (table, cu, pos, [o + a for o, a in zip(lens, new)], [top], [0])]


def _exact_append(s):
    """Page by page: scales, then tokens; the cache's own values in 64 bits."""
    if s["cu"].numel() * s["max_new"] > 20000 or s["table"].numel() > 2000:
        return None
    got, ps = [], s["ps"]
    cu, lens, table = s["cu"].tolist(), s["lens"].tolist(), s["table"].tolist()
    for x, cache, scale in ((s["k"], s["kc"], s["ks"]), (s["v"], s["vc"], s["vs"])):
        cache, scale, x = cache.double(), scale.double(), x.double()
        for b, o in enumerate(lens):
            end = o + cu[b + 1] - cu[b]
            for j in range(o // ps, -(-end // ps)):
                lo, hi = max(o, j * ps), min(end, (j + 1) * ps)
                if lo >= hi:
                    continue
                new = x[cu[b] + lo - o:cu[b] + hi - o].transpose(0, 1)
                p, held = table[b][j], lo - j * ps
                # log2 of the ratio is rounded, so start low and step up to the definition
                e = torch.floor(torch.log2(new.abs().amax((1, 2)) / 448)) - 1
                e = e.clamp(min=MIN_EXP)
                for _ in range(3):
                    now = ((e.long() + 1023) << 52).view(torch.float64)
                    e = torch.where(new.abs().amax((1, 2)) > 448 * now, e + 1, e)
                now = ((e.long() + 1023) << 52).view(torch.float64)
                if held:
                    now = torch.maximum(now, scale[p])
                    was = cache[p, :, :held] * (scale[p] / now)[:, None, None]
                    cache[p, :, :held] = was.float().to(torch.float8_e4m3fn).double()
                cache[p, :, held:held + hi - lo] = \
                    (new / now[:, None, None]).float().to(torch.float8_e4m3fn).double()
                scale[p] = now
        got.append((cache, scale))
    return [got[0][0], got[1][0], got[0][1], got[1][1]]


def _exact_attn(s):
    q, ps, bs = s["q"].double(), s["ps"], s["bs"]
    rows, H, d = q.shape
    Hk = s["kc"].shape[1]
    out = torch.zeros(rows, H, d, dtype=torch.float64, device=q.device)
    lse = torch.zeros(H, rows, dtype=torch.float64, device=q.device)
    cu = s["cu"].tolist()
    for b, n in enumerate(s["lens"].tolist()):
        lo, hi = cu[b], cu[b + 1]
        if lo == hi:
            continue
        pages = s["table"][b, :-(-n // ps)].long()

        def side(cache, scale, new):
            x = cache[pages].double() * scale[pages].double()[:, :, None, None]
            x = x.transpose(0, 1).reshape(Hk, -1, d)[:, :n]
            return x if new is None else torch.cat([x, new[lo:hi].double().transpose(0, 1)], 1)

        k, v = side(s["kc"], s["ks"], s["k"]), side(s["vc"], s["vs"], s["v"])
        w = torch.einsum("ihgd,hjd->hgij", q[lo:hi].view(hi - lo, Hk, H // Hk, d), k) * d ** -0.5
        if not w.shape[-1]:  # no key at all
            lse[:, lo:hi] = -math.inf
            continue
        pos = torch.arange(n + hi - lo, device=q.device)
        see = (pos[None] < n) | (pos[None] // bs <= pos[n:, None] // bs)
        w = w.masked_fill(~see[:, :w.shape[-1]], -math.inf)
        z = w.logsumexp(-1)
        lse[:, lo:hi] = z.reshape(H, -1)
        o = torch.einsum("hgij,hjd->ihgd", (w - z[..., None]).exp(), v)
        out[lo:hi] = o.reshape(hi - lo, H, d)
    return [out, lse]

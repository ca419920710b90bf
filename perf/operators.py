"""Attention over a paged KV cache that is held in 8 bits with a scale per block, and
attention with modified scores: the cases that are measured, their plain forms and their
definitions in 64 bits.

Three operators, each reached through the package's public calls:

append   rope_append_block_scaled: the rotary embedding of new queries and keys, and the
         write of keys and values into E4M3 blocks that carry one power-of-two scale
         (E8M0) per block and KV head. A block's scale follows its largest element: where
         a new token needs a larger one, the block's earlier codes are rescaled.
decode   paged_attn_decode_ext: one query token per sequence over its paged cache (16-bit,
         or E4M3 with block scales), the scores capped by a tanh, with a bias by distance
         (ALiBi) or limited to a window of the last keys.
prefill  paged_attn_prefill_chunk_ext: the same for chunks of new query tokens, causal,
         with a prefix that every row sees where prefix lengths are given.

A case's lengths follow from the case alone; every value follows from the seed.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
E4M3 = torch.float8_e4m3fn
MIN_EXP = -60                 # smallest exponent that the append gives a block


# ---- cases ----------------------------------------------------------------------------

def listed():
    return [
        # one new token of one conversation: what the cache write of a single stream costs
        dict(name="append one token", op="append", n=1, lo=300, hi=300, qlo=1, qhi=1, hq=32, hkv=8,
             d=128, bs=16, dtype="bf16", rot=128, neox=True),
        # the serving batch's new tokens, one per sequence, each into a partly filled block
        dict(name="append batch of 128", op="append", n=128, lo=20, hi=900, qlo=1, qhi=1, hq=32,
             hkv=8, d=128, bs=16, dtype="bf16", rot=128, neox=True),
        # prompts arriving as chunks that start and end inside blocks; part of each head rotated
        dict(name="append ragged chunks", op="append", n=7, lo=400, hi=2500, qlo=150, qhi=2100,
             hq=28, hkv=4, d=128, bs=64, dtype="f16", rot=64, neox=False),
        # one conversation, a few hundred tokens in: latency alone
        dict(name="decode one sequence", op="decode", n=1, lo=700, hi=700, hq=32, hkv=8, d=128,
             bs=16, dtype="bf16", kv="block", softcap=0.0, window=0, alibi=False),
        # the serving batch over the 8-bit cache
        dict(name="decode batch of 128", op="decode", n=128, lo=1024, hi=8192, hq=32, hkv=8, d=128,
             bs=16, dtype="bf16", kv="block", softcap=0.0, window=0, alibi=False),
        # few very long contexts, blocks of 64
        dict(name="decode long contexts", op="decode", n=4, lo=32768, hi=131072, hq=32, hkv=8,
             d=128, bs=64, dtype="bf16", kv="block", softcap=0.0, window=0, alibi=False),
        # wide heads, capped scores, a window whose older blocks the cache has given back
        dict(name="decode capped window", op="decode", n=32, lo=500, hi=6000, hq=16, hkv=8, d=256,
             bs=32, dtype="bf16", kv="same", softcap=50.0, window=1024, alibi=False),
        # no grouping of heads, scores biased by distance
        dict(name="decode distance bias", op="decode", n=16, lo=100, hi=4000, hq=16, hkv=16, d=64,
             bs=16, dtype="f16", kv="same", softcap=0.0, window=0, alibi=True),
        # a 512-token chunk of a prompt over the 8-bit cache, as beside a decode batch
        dict(name="prefill one chunk", op="prefill", n=1, lo=2012, hi=2012, qlo=512, qhi=512, hq=16,
             hkv=8, d=128, bs=16, dtype="bf16", kv="block", softcap=0.0, window=0, alibi=False,
             prefix=False, pad=0),
        # a long prompt's later part over the 8-bit cache
        dict(name="prefill long chunk", op="prefill", n=1, lo=6144, hi=6144, qlo=2048, qhi=2048,
             hq=32, hkv=8, d=128, bs=64, dtype="bf16", kv="block", softcap=0.0, window=0,
             alibi=False, prefix=False, pad=0),
        # capped scores and a window, 16-bit cache
        dict(name="prefill capped window", op="prefill", n=2, lo=3500, hi=4096, qlo=1500, qhi=2048,
             hq=16, hkv=8, d=128, bs=16, dtype="bf16", kv="same", softcap=30.0, window=1024,
             alibi=False, prefix=False, pad=0),
        # prompts of several users, biased by distance, each with a prefix its rows all see
        dict(name="prefill prefix and bias", op="prefill", n=6, lo=90, hi=1300, qlo=60, qhi=700,
             hq=28, hkv=4, d=64, bs=32, dtype="f16", kv="same", softcap=0.0, window=0, alibi=True,
             prefix=True, pad=5),
    ]


def _log(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["append", "decode", "prefill"])
    hkv = rng.choice([1, 2, 4, 8])
    d = rng.choice([64, 128, 128, 256])
    g = rng.choice([1, 2, 3, 4, 7, 8] + ([16] if d < 256 else []))
    c = dict(op=op, hq=g * hkv, hkv=hkv, d=d, bs=rng.choice([16, 16, 32, 64]),
             dtype=rng.choice(["bf16", "f16"]))
    if op == "append":
        if rng.random() < 0.5:                    # new tokens of a batch
            lo = rng.randint(1, 300)
            return dict(c, n=_log(rng, 1, 256), lo=lo, hi=lo + rng.randint(0, 600), qlo=1, qhi=1,
                        rot=rng.choice([16, d // 2, d]), neox=rng.random() < 0.5)
        qlo = _log(rng, 2, 1000)                  # chunks, up to 16 of them
        qhi = min(2100, qlo + rng.randint(0, 1100))
        n = _log(rng, 1, 4)
        # at most about the bytes of the largest listed case
        qhi = max(2, min(qhi, int(1.2e8 / (n * d * (4 * c["hq"] + 6 * hkv)))))
        qlo = min(qlo, qhi)
        return dict(c, n=n, lo=qhi, hi=qhi + rng.randint(0, 700), qlo=qlo, qhi=qhi,
                    rot=rng.choice([16, d // 2, d]), neox=rng.random() < 0.5)
    c.update(kv=rng.choice(["block", "block", "same"]),
             softcap=rng.choice([0.0, 0.0, 20.0, 50.0]), alibi=rng.random() < 0.25,
             window=_log(rng, 8, 4096) if rng.random() < 0.3 else 0)
    if op == "decode":
        lo = _log(rng, 1, 6000)
        hi = min(8000, lo + rng.randint(0, lo + 40))
        # at most about the bytes of the largest listed case
        n = max(1, min(_log(rng, 1, 96), int(1e9 / (hi * hkv * d * (2 if c["kv"] == "block" else 4)))))
        return dict(c, n=n, lo=lo, hi=hi)
    n = _log(rng, 1, 6)
    qlo = _log(rng, 1, 1200)
    qhi = min(1500, qlo + rng.randint(0, qlo))
    ctx = qhi + (0 if rng.random() < 0.2 else _log(rng, 1, 2000))
    # at most about the pairs of the largest listed case
    n = max(1, min(n, int(3.2e8 / (c["hq"] * qhi * ctx))))
    return dict(c, n=n, lo=ctx, hi=ctx + rng.randint(0, 200), qlo=qlo, qhi=qhi,
                prefix=rng.random() < 0.25, pad=rng.choice([0, 0, 3]))


def _lens(c):
    """Context lengths and new tokens of each sequence: the case's own, whatever the seed."""
    r = random.Random("%s %d %d %d" % (c["op"], c["n"], c["lo"], c["hi"]))
    ctx = [r.randint(c["lo"], c["hi"]) for _ in range(c["n"])]
    ctx[-1] = c["hi"]
    if c["op"] == "decode":
        return ctx, [1] * c["n"]
    q = [min(x, r.randint(c["qlo"], c["qhi"])) for x in ctx]
    q[-1] = min(ctx[-1], c["qhi"])
    return ctx, q


def _prefixes(c):
    """Prefix lengths: some within the cached part, some into the chunk, some none."""
    ctx, _ = _lens(c)
    r = random.Random("prefix %d" % c["hi"])
    return [r.choice([0, x // 3, x // 2, x]) for x in ctx]


def work(c):
    ctx, ql = _lens(c)
    hq, hkv, d, n = c["hq"], c["hkv"], c["d"], c["n"]
    t = sum(ql)
    if c["op"] == "append":
        # queries read and written, keys and values read, their codes written, the scales of
        # the blocks, the table's rows of the rotary angles
        blocks = sum((x - 1) // c["bs"] - (x - q) // c["bs"] + 1 for x, q in zip(ctx, ql))
        return {"bytes": t * d * (4 * hq + 4 * hkv + 2 * hkv) + 4 * blocks * hkv + 4 * t * c["rot"],
                "flops": 3.0 * t * c["rot"] * (hq + hkv)}
    pre = _prefixes(c) if c.get("prefix") else [0] * n
    w = c["window"] or 1 << 30
    keys = sum(min(x, w + q - 1) for x, q in zip(ctx, ql))
    pairs = 0
    for x, q, f in zip(ctx, ql, pre):
        for p in range(x - q, x):
            pairs += max(p + 1, f) - max(0, p + 1 - w)
    elt = 1 if c["kv"] == "block" else 2
    return {"bytes": keys * hkv * d * 2 * elt + 4 * t * hq * d +
            (2 * keys * hkv // c["bs"] if elt == 1 else 0),
            "flops": 4.0 * pairs * hq * d}


# ---- inputs ---------------------------------------------------------------------------

class State:
    pass


def _exponent(amax):
    """The smallest e with amax <= 448 * 2^e, at least MIN_EXP (whole numbers, int32)."""
    m, e = torch.frexp(amax)
    need = e - 9 + (m > 0.875).to(e.dtype)
    return torch.where(amax > 0, need, MIN_EXP).clamp_min(MIN_EXP).to(torch.int32)


def _power(e):
    """2^e in fp32 for exponents from -126 to 127."""
    return ((e + 127) << 23).view(torch.float32)


def _pool(nb, hkv, bs, d, g, dev):
    """Keys or values of a whole pool [nb, hkv, bs, d]: heads and blocks of other sizes, and
    a few channels that stand out, as keys have them."""
    x = torch.randn(nb, hkv, bs, d, generator=g, device=dev)
    x *= torch.exp2(torch.rand(nb, hkv, 1, 1, generator=g, device=dev) * 3 - 2)
    x[..., :: d // 4] *= 4
    return x


def _quantised(x):
    e = _exponent(x.abs().amax((2, 3)))
    return (x * _power(-e)[..., None, None]).to(E4M3), (e + 127).to(torch.uint8)


def prepare(c, seed):
    dev = "cuda"
    g = torch.Generator(dev).manual_seed(seed)
    ctx, ql = _lens(c)
    n, hq, hkv, d, bs, dt = c["n"], c["hq"], c["hkv"], c["d"], c["bs"], DT[c["dtype"]]
    s = State()
    s.c = c
    need = [-(-x // bs) for x in ctx]
    s.maxb = max(need) + 1
    nb = sum(need) + 3
    order = torch.randperm(nb, generator=g, device=dev).to(torch.int32)
    first = torch.tensor([0] + need).cumsum(0)[:n].to(dev)
    need = torch.tensor(need, device=dev)
    j = torch.arange(s.maxb, device=dev)
    has = j[None] < need[:, None]
    s.tables = torch.where(has, order[(first[:, None] + j[None]).clamp_max(nb - 1)], -1)
    s.seq_lens = torch.tensor(ctx, dtype=torch.int32, device=dev)
    cu = [0]
    for q in ql:
        cu.append(cu[-1] + q)
    s.cu = torch.tensor(cu, dtype=torch.int32, device=dev)
    s.max_q, s.max_ctx, t = max(ql), max(ctx), cu[-1]
    last = s.tables[torch.arange(n, device=dev), need - 1].long()
    if c["op"] == "append":
        # what stands in the cache is a little smaller than what comes, so some scales grow
        s.k, s.ks = _quantised(_pool(nb, hkv, bs, d, g, dev) * 0.7)
        s.v, s.vs = _quantised(_pool(nb, hkv, bs, d, g, dev) * 0.7)
        size = torch.exp2(torch.rand(t, hkv, 1, generator=g, device=dev) * 2 - 1)
        s.key = (torch.randn(t, hkv, d, generator=g, device=dev) * size).to(dt)
        s.value = (torch.randn(t, hkv, d, generator=g, device=dev) * size).to(dt)
        s.query = torch.randn(t, hq, d, generator=g, device=dev).to(dt)
        s.query_out = torch.empty_like(s.query)
        half = c["rot"] // 2
        inv = 10000.0 ** (-torch.arange(half, device=dev, dtype=torch.float64) / half)
        a = torch.arange(s.max_ctx + 1, device=dev, dtype=torch.float64)[:, None] * inv[None]
        s.cos_sin = torch.cat([a.cos(), a.sin()], 1).float()
        return s
    t += c.get("pad", 0)
    s.q = (torch.randn(t, hq, d, generator=g, device=dev) * 1.5).to(dt)
    s.out = torch.zeros_like(s.q)
    s.scale = d ** -0.5
    k, v = _pool(nb, hkv, bs, d, g, dev), _pool(nb, hkv, bs, d, g, dev)
    if c["kv"] == "block":
        (s.k, s.ks), (s.v, s.vs) = _quantised(k), _quantised(v)
    else:
        s.k, s.v, s.ks, s.vs = k.to(dt), v.to(dt), None, None
    # what lies behind a context in its last block is nobody's: NaN
    tail = (torch.arange(bs, device=dev)[None] > ((s.seq_lens - 1) % bs)[:, None])[:, None, :, None]
    for x in (s.k, s.v):
        b = x[last].float().masked_fill(tail, math.nan)
        x[last] = b.to(x.dtype)
    if c["window"]:
        # blocks that no row's window reaches were given back
        low = s.seq_lens - torch.tensor(ql, device=dev) - c["window"] + 1
        s.tables = torch.where((j[None] + 1) * bs <= low[:, None], -1, s.tables)
    s.slopes = None
    if c["alibi"]:
        s.slopes = torch.exp2(-8.0 * torch.arange(1, hq + 1, device=dev) / hq).float()
    s.prefix = torch.tensor(_prefixes(c), dtype=torch.int32, device=dev) if c.get("prefix") else None
    s.tables = s.tables.to(torch.int32).contiguous()
    s.workspace = None
    return s


# ---- one pass -------------------------------------------------------------------------

def run(s):
    c = s.c
    if own:
        import paged_kv_decode_11_gb300 as P
        if c["op"] == "append":
            P.rope_append_block_scaled(s.key, s.value, s.k, s.v, s.ks, s.vs, s.tables, s.seq_lens,
                                       s.cu, query=s.query, query_out=s.query_out,
                                       cos_sin_cache=s.cos_sin, neox_style=c["neox"])
            return {"query": s.query_out, "k": s.k, "v": s.v, "ks": s.ks, "vs": s.vs}
        if c["op"] == "decode":
            if s.workspace is None:               # the program's own: zeroed once, then kept
                size = P.paged_attn_decode_ext_workspace_size(c["n"], c["hq"], c["hkv"], c["d"],
                                                              s.max_ctx, c["window"])
                s.workspace = torch.zeros(size, dtype=torch.uint8, device="cuda")
            P.paged_attn_decode_ext(s.out, s.q, s.k, s.v, s.tables, s.seq_lens, s.scale, s.max_ctx,
                                    s.ks, s.vs, softcap=c["softcap"], window=c["window"],
                                    alibi_slopes=s.slopes, workspace=s.workspace)
            return s.out
        P.paged_attn_prefill_chunk_ext(s.out, s.q, s.k, s.v, s.tables, s.seq_lens, s.cu, s.scale,
                                       s.max_q, s.ks, s.vs, softcap=c["softcap"],
                                       window=c["window"], alibi_slopes=s.slopes,
                                       prefix_lens=s.prefix)
        return s.out
    return _append(s) if c["op"] == "append" else _attention(s)


def _rows(s):
    """Of each row of q: its sequence, its place among that sequence's new tokens, and
    whether a sequence owns it at all (rows behind the last one belong to nobody)."""
    t = s.key.shape[0] if s.c["op"] == "append" else s.q.shape[0]
    r = torch.arange(t, device="cuda", dtype=torch.int32)
    n = s.c["n"]
    seq = torch.searchsorted(s.cu, r, right=True) - 1
    mine = seq < n
    seq = seq.clamp_max(n - 1)
    return seq, r - s.cu[seq], mine


def _rotate(x, cs, rot, neox):
    """Rotary embedding in 64 bits, where a rounding to 16 bits next to a border is safe."""
    half = rot // 2
    y = x.double()
    co, si = cs[:, None, :half].double(), cs[:, None, half:].double()
    if neox:
        a, b = y[..., :half], y[..., half:rot]
        z = torch.cat([a * co - b * si, b * co + a * si], -1)
    else:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        z = torch.stack([a * co - b * si, b * co + a * si], -1).flatten(-2)
    return torch.cat([z, y[..., rot:]], -1).to(x.dtype)


def _append(s):
    c = s.c
    n, bs = c["n"], c["bs"]
    seq, i, _ = _rows(s)
    start = s.seq_lens - (s.cu[1:] - s.cu[:-1])
    pos = start[seq] + i
    cs = s.cos_sin[pos.long()]
    query = _rotate(s.query, cs, c["rot"], c["neox"])
    key = _rotate(s.key, cs, c["rot"], c["neox"])
    j = torch.div(pos, bs, rounding_mode="floor")
    block = s.tables[seq, j.long()].long()
    off = (pos % bs).long()
    nt = (s.max_q + bs - 2) // bs + 1
    w = (seq * nt + j - (start // bs)[seq]).long()
    base = s.tables[torch.arange(n, device="cuda"), (start // bs).long()].long()
    fresh = (start % bs == 0)[:, None]
    for x, cache, scales in ((key, s.k, s.ks), (s.value, s.v, s.vs)):
        x = x.float()
        big = torch.where(x.isfinite(), x.abs(), 0).amax(-1)
        amax = torch.zeros(n * nt, x.shape[1], device="cuda")
        amax = amax.scatter_reduce(0, w[:, None].expand_as(big), big, "amax")
        new = _exponent(amax).view(n, nt, -1)
        old = scales[base].to(torch.int32) - 127
        new[:, 0] = torch.where(fresh, new[:, 0], torch.maximum(new[:, 0], old))
        # the codes that stand in a sequence's first block, to that block's new scale
        factor = torch.where(fresh, 1.0, _power(torch.where(fresh, 0, old - new[:, 0]).clamp_min(-126)))
        codes = cache[base]
        cache[base] = torch.where(factor[..., None, None] == 1, codes.float(),
                                  codes.float() * factor[..., None, None]).to(E4M3)
        e = new.view(n * nt, -1)[w]
        y = x * _power(-e)[..., None]
        cache[block, :, off] = y.clamp(-448, 448).to(E4M3)
        scales[block] = (e + 127).to(torch.uint8)
    return {"query": query, "k": s.k, "v": s.v, "ks": s.ks, "vs": s.vs}


def _dense(s, cache, scales):
    """The cache in fp32 as the tables lay it out, [n, hkv, tokens, d]."""
    ids = s.tables.clamp_min(0).long()
    x = cache[ids].float()
    if scales is not None:
        x = x * _power(scales[ids].to(torch.int32) - 127)[..., None, None]
    n, m, h, b, d = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(n, h, m * b, d)


def _attention(s):
    c = s.c
    n, hq, hkv, d = c["n"], c["hq"], c["hkv"], c["d"]
    lq = s.max_q
    k, v = _dense(s, s.k, s.ks), _dense(s, s.v, s.vs)
    i = torch.arange(lq, device="cuda", dtype=torch.int32)
    ql = s.cu[1:] - s.cu[:-1]
    rows = (s.cu[:-1, None] + i[None]).clamp_max(s.q.shape[0] - 1).long()
    q = s.q[rows].float().view(n, lq, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4)
    x = torch.einsum("nhgid,nhjd->nhgij", q, k) * s.scale
    if c["softcap"]:
        x = torch.tanh(x / c["softcap"]) * c["softcap"]
    pos = ((s.seq_lens - ql)[:, None] + i[None])[:, :, None]
    j = torch.arange(k.shape[2], device="cuda", dtype=torch.int32)[None, None, :]
    if s.slopes is not None:
        x = x - s.slopes.view(1, hkv, -1, 1, 1) * (pos - j).abs()[:, None, None].float()
    see = j <= pos
    if s.prefix is not None:
        see = see | (j < s.prefix[:, None, None])
    if c["window"]:
        see = see & (pos - j < c["window"])
    see = (see & (j < s.seq_lens[:, None, None]))[:, None, None]
    x = x.masked_fill(~see, -math.inf)
    v = v.masked_fill(~see.any(3).view(n, 1, -1, 1), 0.0)
    m = x.amax(-1, keepdim=True).clamp_min(torch.finfo(torch.float32).min)
    p = torch.exp(x - m)
    o = torch.einsum("nhgij,nhjd->nhgid", p, v) / p.sum(-1, keepdim=True).clamp_min(1e-37)
    o = o.permute(0, 3, 1, 2, 4).reshape(n, lq, hq, d)
    seq, at, mine = _rows(s)
    return torch.where(mine[:, None, None], o[seq.long(), at.clamp_max(lq - 1).long()], 0.0).to(s.q.dtype)


# ---- the definitions in 64 bits -----------------------------------------------------------

def _exact_e4m3(x):
    """The nearest of the values that 4 exponent and 3 mantissa bits hold, ties to even."""
    _, e = torch.frexp(x.abs())
    step = torch.exp2(torch.clamp(e - 1, min=-6).double() - 3)
    return torch.clamp(torch.round(x / step) * step, -448, 448)


def _exact_exponent(a):
    """Smallest whole e >= MIN_EXP with a <= 448 * 2^e, of one number."""
    if a <= 0:
        return MIN_EXP
    e = math.floor(math.log2(a / 448.0)) - 1
    while a > 448.0 * 2.0 ** e:
        e += 1
    return max(MIN_EXP, e)


def exact(c, seed):
    s = prepare(c, seed)
    ctx, ql = _lens(c)
    n, hq, hkv, d, bs = c["n"], c["hq"], c["hkv"], c["d"], c["bs"]
    cu = [0]
    for q in ql:
        cu.append(cu[-1] + q)
    tables = s.tables.cpu()
    if c["op"] == "append":
        half = c["rot"] // 2
        first = list(range(half)) if c["neox"] else list(range(0, c["rot"], 2))
        second = list(range(half, c["rot"])) if c["neox"] else list(range(1, c["rot"], 2))

        def turned(x, p):
            co, si = s.cos_sin[p, :half].double(), s.cos_sin[p, half:].double()
            y = x.double().clone()
            y[..., first] = x[..., first].double() * co - x[..., second].double() * si
            y[..., second] = x[..., second].double() * co + x[..., first].double() * si
            return y
        query = torch.empty(cu[-1], hq, d, dtype=torch.float64, device="cuda")
        kd, vd = s.k.double(), s.v.double()
        for b in range(n):
            p0 = ctx[b] - ql[b]
            at = torch.arange(p0, ctx[b], device="cuda")
            r = slice(cu[b], cu[b + 1])
            query[r] = turned(s.query[r], at[:, None])
            rows_k = turned(s.key[r], at[:, None]).to(s.key.dtype).double()
            rows_v = s.value[r].double()
            for j in range(p0 // bs, (ctx[b] - 1) // bs + 1):
                lo, hi = max(p0, j * bs), min(ctx[b], (j + 1) * bs)
                block = int(tables[b, j])
                for rows, cache, scales in ((rows_k, kd, s.ks), (rows_v, vd, s.vs)):
                    new = rows[lo - p0:hi - p0].transpose(0, 1)              # [hkv, tokens, d]
                    tops, olds = new.abs().amax((1, 2)).tolist(), scales[block].tolist()
                    es = [_exact_exponent(a) for a in tops]
                    if lo > j * bs:
                        es = [max(e, o - 127) for e, o in zip(es, olds)]
                        f = torch.tensor([2.0 ** (o - 127 - e) for o, e in zip(olds, es)],
                                         dtype=torch.float64, device="cuda")
                        cache[block] = _exact_e4m3(cache[block] * f[:, None, None])
                    f = torch.tensor([2.0 ** -e for e in es], dtype=torch.float64, device="cuda")
                    cache[block][:, lo - j * bs:hi - j * bs] = _exact_e4m3(new * f[:, None, None])
        return {"query": query, "k": kd, "v": vd, "ks": None, "vs": None}
    out = torch.zeros(s.q.shape, dtype=torch.float64, device="cuda")
    pre = _prefixes(c) if c.get("prefix") else [0] * n
    for b in range(n):
        p0 = ctx[b] - ql[b]
        low = max(0, p0 - c["window"] + 1) if c["window"] else 0
        j = torch.arange(low, ctx[b], device="cuda")
        block, off = s.tables[b, j // bs].long(), j % bs
        k, v = s.k[block, :, off].double(), s.v[block, :, off].double()      # [keys, hkv, d]
        if s.ks is not None:
            k = k * torch.exp2(s.ks[block].double() - 127)[..., None]
            v = v * torch.exp2(s.vs[block].double() - 127)[..., None]
        for i0 in range(0, ql[b], 256):
            i = torch.arange(i0, min(ql[b], i0 + 256), device="cuda")
            q = s.q[cu[b] + i].double().view(len(i), hkv, -1, d)
            x = torch.einsum("ihgd,jhd->hgij", q, k) * s.scale
            if c["softcap"]:
                x = c["softcap"] * torch.tanh(x / c["softcap"])
            pos = (p0 + i)[:, None]
            gap = pos - j[None]
            if s.slopes is not None:
                x = x - s.slopes.double().view(hkv, -1, 1, 1) * gap.abs()
            see = (gap >= 0) | (j[None] < pre[b])
            if c["window"]:
                see = see & (gap < c["window"])
            p = torch.softmax(x.masked_fill(~see, -math.inf), -1)
            out[cu[b] + i] = torch.einsum("hgij,jhd->ihgd", p, v).reshape(len(i), hq, d)
    return out

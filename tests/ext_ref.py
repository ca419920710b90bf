"""The block-scaled append and the attentions with block scales or modified
scores, from their definitions in 64 bits with plain torch, sequence by
sequence; shares no code with the library."""
import math

import torch

MIN_EXP = -60


def e4m3(x):
    """The nearest E4M3 value of each double (ties to even, saturating; NaN stays)."""
    _, e = torch.frexp(x.abs())
    step = torch.exp2(torch.clamp(e - 1, min=-6).double() - 3)
    y = torch.clamp(torch.round(x / step) * step, -448.0, 448.0)
    y = torch.where(torch.isinf(x), torch.sign(x) * 448.0, y)
    return torch.where(torch.isnan(x), torch.nan, y)


def exponent(amax):
    """Smallest whole e >= -60 with amax <= 448 * 2^e, of each double."""
    e = torch.full_like(amax, MIN_EXP)
    for k in range(MIN_EXP + 1, 128):
        e = torch.where(amax > 448.0 * 2.0 ** (k - 1), float(k), e)
    return e


def round16(x, dtype):
    """Doubles to the nearest fp32 value, then to the nearest value of a 16-bit type: the
    rounding the append defines for rotated elements."""
    return x.float().to(dtype)


def rotate(x, pos, cos_sin, neox):
    """Rows x [t, heads, d] turned by the angles of their positions, exact in double."""
    rot = cos_sin.shape[1]
    half = rot // 2
    co = cos_sin[pos, :half].double()[:, None]
    si = cos_sin[pos, half:].double()[:, None]
    y = x.double().clone()
    a, b = (y[..., :half], y[..., half:rot]) if neox else (y[..., 0:rot:2], y[..., 1:rot:2])
    a2, b2 = a * co - b * si, b * co + a * si
    if neox:
        y[..., :half], y[..., half:rot] = a2, b2
    else:
        y[..., 0:rot:2], y[..., 1:rot:2] = a2, b2
    return y


def append(key, value, k, v, ks, vs, tables, seq_lens, cu, query=None, cos_sin=None, neox=True,
           skip=()):
    """Updates copies of the caches (as doubles) and scales (as int64 bytes); returns them and
    the rotated queries."""
    k, v = k.view(torch.float8_e4m3fn).double(), v.view(torch.float8_e4m3fn).double()
    ks, vs = ks.view(torch.uint8).long().clone(), vs.view(torch.uint8).long().clone()
    query = query.clone() if query is not None else None
    bs = k.shape[2]
    tables, seq_lens, cu = tables.tolist(), seq_lens.tolist(), cu.tolist()
    for n, ctx in enumerate(seq_lens):
        L = cu[n + 1] - cu[n]
        if L <= 0 or n in skip:
            continue
        p0 = ctx - L
        rows = slice(cu[n], cu[n + 1])
        pos = torch.arange(p0, ctx, device=key.device)
        kk, vv = key[rows], value[rows]
        if cos_sin is not None:
            kk = round16(rotate(kk, pos, cos_sin, neox), key.dtype)
            if query is not None:
                query[rows] = round16(rotate(query[rows], pos, cos_sin, neox), query.dtype)
        for j in range(p0 // bs, (ctx - 1) // bs + 1):
            lo, hi = max(p0, j * bs), min(ctx, (j + 1) * bs)
            block = tables[n][j]
            if not 0 <= block < k.shape[0]:
                continue
            for x, cache, scales in ((kk, k, ks), (vv, v, vs)):
                new = x[lo - p0:hi - p0].double().transpose(0, 1)          # [hkv, tokens, d]
                big = torch.where(torch.isfinite(new), new.abs(), 0.0).amax((1, 2))
                e = exponent(big)
                if lo > j * bs:
                    old = torch.clamp(scales[block], max=254).double() - 127
                    e = torch.maximum(e, old)
                    f = torch.exp2(old - e)[:, None, None]
                    cache[block] = torch.where(f < 1, e4m3(cache[block] * f), cache[block])
                cache[block][:, lo - j * bs:hi - j * bs] = e4m3(new * torch.exp2(-e)[:, None, None])
                scales[block] = (e + 127).long()
    return k, v, ks, vs, query


class Attn:
    """out, lse and, for the tolerances, sum_j p_j |v_j| and the largest sum_d |q_d k_d|."""

    def __init__(self, shape, device):
        self.out = torch.zeros(shape, dtype=torch.float64, device=device)
        self.lse = torch.full(shape[:2], -math.inf, dtype=torch.float64, device=device)
        self.mass = torch.zeros(shape, dtype=torch.float64, device=device)
        self.size = torch.zeros(shape[:2], dtype=torch.float64, device=device)
        self.bias = torch.zeros(shape[:2], dtype=torch.float64, device=device)


def values(cache, scales):
    """The numbers a cache stands for, as doubles: scales None, fp32 [hkv] or E8M0 [nb, hkv]."""
    if cache.dtype in (torch.uint8, torch.float8_e4m3fn):
        x = cache.view(torch.float8_e4m3fn).double()
        if scales.dim() == 1:
            return x * scales.double()[None, :, None, None]
        s = scales.view(torch.uint8).double()
        return x * torch.where(s == 255, torch.nan, torch.exp2(s - 127))[..., None, None]
    return cache.double()


def attention(q, k, v, tables, seq_lens, cu, scale, ks=None, vs=None, softcap=0.0, window=0,
              slopes=None, prefix=None, skip=()):
    """Rows cu[n] .. cu[n+1]-1 of q are the last tokens of sequence n."""
    hq, d = q.shape[1:]
    hkv, bs = k.shape[1], k.shape[2]
    res = Attn(q.shape, q.device)
    cu = cu.tolist()
    for n, ctx in enumerate(seq_lens.tolist()):
        L = cu[n + 1] - cu[n]
        if L <= 0 or ctx <= 0 or n in skip:
            continue
        p0 = ctx - L
        low = max(0, p0 - window + 1) if window else 0
        j = torch.arange(low, ctx, device=q.device)
        block, off = tables[n, j // bs].long(), j % bs
        kk = values(k[block], ks if ks is None or ks.dim() == 1 else ks[block])
        vv = values(v[block], vs if vs is None or vs.dim() == 1 else vs[block])
        at = torch.arange(len(j), device=q.device)
        kk, vv = kk[at, :, off], vv[at, :, off]                            # [keys, hkv, d]
        rows = slice(cu[n], cu[n + 1])
        qq = q[rows].double().view(L, hkv, hq // hkv, d)
        x = torch.einsum("ihgd,jhd->hgij", qq, kk) * scale
        size = torch.einsum("ihgd,jhd->hgij", qq.abs(), kk.abs()) * scale
        if softcap:
            x = softcap * torch.tanh(x / softcap)
        gap = torch.arange(p0, ctx, device=q.device)[:, None] - j[None]
        bias = torch.zeros_like(x)
        if slopes is not None:
            bias = slopes.double().view(hkv, -1, 1, 1) * gap.abs()
            x = x - bias
        see = gap >= 0
        if prefix is not None:
            see = see | (j[None] < int(prefix[n]))
        if window:
            see = see & (gap < window)
        x = x.masked_fill(~see, -math.inf)
        p = torch.softmax(x, -1)
        res.out[rows] = torch.einsum("hgij,jhd->ihgd", p, vv).reshape(L, hq, d)
        res.mass[rows] = torch.einsum("hgij,jhd->ihgd", p, vv.abs()).reshape(L, hq, d)
        res.lse[rows] = torch.logsumexp(x, -1).permute(2, 0, 1).reshape(L, hq)
        res.size[rows] = size.masked_fill(~see, 0).amax(-1).permute(2, 0, 1).reshape(L, hq)
        res.bias[rows] = bias.masked_fill(~see, 0).amax(-1).permute(2, 0, 1).reshape(L, hq)
    return res


# Rounding of a type: half a step, relative.
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def score_error(ref, softcap=0.0):
    """Bound on a score's error in fp32 (natural log units), per row: tensor-core sums of D
    products (at most 2 * 17 partial sums, each within 2^-23 of sum |q k|), the conversions to
    log2 units and back (a few 2^-24 of the score and the bias), the cap's 1 - 2/(E+1) (2^-21
    of the cap), the exponentials (2^-21)."""
    x = ref.size + ref.bias + abs(softcap)
    return 2.0 ** -23 * (40 * ref.size + 4 * ref.bias + 4 * abs(softcap) + 4 * x.clamp(max=1e4) + 8)


def tolerance(ref, q_dtype, p_dtype, softcap=0.0):
    """Elementwise bound on |out - ref.out|: the weights rounded to p_dtype, every score off by
    score_error (a weight and the sum by that much each), the output rounded to q_dtype."""
    e = score_error(ref, softcap)[..., None]
    return (U[p_dtype] + 3 * e) * ref.mass * 1.01 + U[q_dtype] * ref.out.abs() * 1.01 + 2.0 ** -24


def lse_tolerance(ref, softcap=0.0):
    return score_error(ref, softcap) + 2.0 ** -21 * (1 + ref.lse.abs().nan_to_num(posinf=0))

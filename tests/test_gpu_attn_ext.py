"""paged_attn_decode_ext and paged_attn_prefill_chunk_ext against attention in 64 bits
(tests/ext_ref.py, which derives the tolerances): types, head layouts, lengths, block
scales, caps, biases, windows, prefixes, and what must not reach the result."""
import numpy as np
import pytest
import torch

import paged_kv_decode_11_gb300 as P
from tests import ext_ref as R

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
SEQ_LEN, QLEN, BLOCK_ID = 0x4, 0x10, 0x1


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from paged_kv_decode_11_gb300 import build
    build.build()
    P.load()
    torch.cuda.init()
    P.pkv_get_device_error()


class Case:
    """seqs: (cached tokens, query tokens) of each sequence. kv: "same", "head" (fp32 scale
    per head) or "block". What no row sees is NaN in the caches, and blocks that no row
    reaches have no table entry."""

    def __init__(self, seed, seqs, hq=8, hkv=2, d=128, bs=16, dtype="bf16", kv="block", softcap=0.0,
                 window=0, alibi=False, prefix=None, qsize=1.0, spread=3, pad=0, pool=None):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        dt = DT[dtype]
        ctx, ql = [p + q for p, q in seqs], [q for _, q in seqs]
        need = [-(-x // bs) for x in ctx]
        nb = sum(need) + 4 if pool is None else pool
        maxb = max(need + [1]) + 1
        ids = (nb - 1 - np.arange(sum(need))) if pool else rng.permutation(nb)
        t = np.full((len(seqs), maxb), -1, dtype=np.int32)
        at = 0
        for i, m in enumerate(need):
            t[i, :m] = ids[at:at + m]
            at += m
        used = torch.from_numpy(ids[:at].astype(np.int64).copy())
        cu = np.concatenate([[0], np.cumsum(ql)])
        rows = int(cu[-1]) + pad
        self.q = (torch.randn(rows, hq, d, generator=g) * qsize).to(dt).cuda()
        x = torch.randn(2, at, hkv, bs, d, generator=g)
        x *= torch.exp2((torch.rand(2, at, hkv, 1, 1, generator=g) - 0.5) * 2 * spread)
        self.ks = self.vs = None
        if kv == "same":
            x = x.to(dt)
        elif kv == "head":
            s = x.abs().amax((1, 3, 4)) / 448.0                         # [2, hkv]
            x = (x / s[:, None, :, None, None]).to(torch.float8_e4m3fn)
            self.ks, self.vs = s.float().cuda()
        else:
            e = R.exponent(x.abs().amax((3, 4)).double())
            x = (x.double() * torch.exp2(-e)[..., None, None]).float().to(torch.float8_e4m3fn)
            s = torch.full((2, nb, hkv), 255, dtype=torch.uint8)
            s[:, used] = (e + 127).to(torch.uint8)
            self.ks, self.vs = s.cuda()
        shape = (2, nb, hkv, bs, d)
        pool_kv = (torch.empty(shape, dtype=x.dtype, device="cuda") if pool else
                   torch.full(shape, float("nan")).to(x.dtype).cuda())
        pool_kv[:, used.cuda()] = x.cuda()
        # slots behind a context, and before the first key any row sees, hold NaN
        for i, (p, q) in enumerate(seqs):
            lo = max(0, p - window + 1) if window and q else 0
            for j in range(need[i]):
                for o in range(bs):
                    if not lo <= j * bs + o < ctx[i]:
                        pool_kv[:, t[i, j], :, o] = torch.tensor(float("nan")).to(x.dtype)
                if (j + 1) * bs <= lo:
                    t[i, j] = -1 if i % 2 else nb + 7
        self.k, self.v = pool_kv
        self.tables = torch.from_numpy(t).cuda()
        self.seq_lens = torch.tensor(ctx, dtype=torch.int32).cuda()
        self.cu = torch.tensor(cu, dtype=torch.int32).cuda()
        self.max_q, self.max_ctx = max(ql + [0]), max(ctx + [0])
        self.scale, self.softcap, self.window = d ** -0.5, softcap, window
        self.slopes = None
        if alibi:
            self.slopes = torch.exp2(-8.0 * torch.arange(1, hq + 1) / hq).float().cuda()
        self.prefix = None if prefix is None else torch.tensor(prefix, dtype=torch.int32).cuda()
        self.p_dtype = torch.float16 if kv != "same" else dt       # the type weights are rounded to

    def opts(self):
        return dict(softcap=self.softcap, window=self.window, alibi_slopes=self.slopes)

    def decode(self, part=0, lse=True, **kw):
        out = torch.full_like(self.q, 9.0)
        le = torch.full(self.q.shape[:2], 9.0, device="cuda") if lse else None
        kw = {**self.opts(), **kw}
        P.paged_attn_decode_ext(out, self.q, self.k, self.v, self.tables, self.seq_lens, self.scale,
                                kw.pop("max_seq_len", self.max_ctx), self.ks, self.vs,
                                partition_tokens=part, out_lse=le, **kw)
        return out, le

    def prefill(self, lse=True, **kw):
        out = torch.full_like(self.q, 9.0)
        le = torch.full(self.q.shape[:2], 9.0, device="cuda") if lse else None
        kw = {**self.opts(), **kw}
        P.paged_attn_prefill_chunk_ext(out, self.q, self.k, self.v, self.tables, self.seq_lens,
                                       self.cu, self.scale, kw.pop("max_q_len", self.max_q), self.ks,
                                       self.vs, prefix_lens=self.prefix, out_lse=le, **kw)
        return out, le

    def want(self, skip=()):
        return R.attention(self.q, self.k, self.v, self.tables, self.seq_lens, self.cu, self.scale,
                           self.ks, self.vs, self.softcap, self.window, self.slopes, self.prefix,
                           skip)

    def check(self, got, ref=None, rows=None):
        ref = self.want() if ref is None else ref
        out, lse = got
        rows = slice(0, int(self.cu[-1])) if rows is None else rows
        err = (out.double() - ref.out).abs()[rows]
        tol = R.tolerance(ref, self.q.dtype, self.p_dtype, self.softcap)[rows]
        assert out[rows].isfinite().all()
        bad = err > tol
        assert not bad.any(), f"{int(bad.sum())} off, worst {float((err / tol).max()):.2f} of the bound"
        if lse is not None:
            w, tol = ref.lse[rows], R.lse_tolerance(ref, self.softcap)[rows]
            g = lse.double()[rows]
            assert torch.equal(g.isinf(), w.isinf()) and not g.isnan().any()
            off = ((g - w).abs() > tol) & w.isfinite()
            assert not off.any()


def ok():
    torch.cuda.synchronize()
    assert P.pkv_get_device_error() == 0


LENS = [1, 2, 15, 16, 17, 31, 100, 257, 700]

DECODE = [
    dict(kv="block"),
    dict(kv="block", dtype="f16", hq=7, hkv=1),
    dict(kv="block", d=64, bs=32, hq=16, hkv=1),
    dict(kv="block", d=256, bs=64, hq=8, hkv=1),
    dict(kv="block", bs=64, hq=32, hkv=2, softcap=20.0, alibi=True),
    dict(kv="block", window=40),
    dict(kv="block", window=1, bs=32),
    dict(kv="block", d=64, window=200, softcap=5.0, qsize=4.0),
    dict(kv="head", softcap=30.0),
    dict(kv="head", d=256, dtype="f16", window=33, alibi=True, hq=2, hkv=2),
    dict(kv="same", softcap=50.0, qsize=6.0, spread=1),
    dict(kv="same", dtype="f16", alibi=True, hq=12, hkv=4, d=64, spread=1),
    dict(kv="same", d=256, window=64, hq=16, hkv=8, spread=1),
    dict(kv="same", dtype="f16", bs=64, window=5, alibi=True, softcap=2.0, hq=13, hkv=1, spread=1),
    dict(kv="same", spread=1),
]


@pytest.mark.parametrize("i", range(len(DECODE)))
@pytest.mark.parametrize("part", [0, 64])
def test_decode(i, part):
    c = Case(i, [(n - 1, 1) for n in LENS], **DECODE[i])
    got = c.decode(part)
    ok()
    c.check(got)


@pytest.mark.parametrize("lens,kw", [
    ([1], {}), ([5000], dict(hkv=1, hq=8)), ([4096, 1], dict(bs=64)),
    ([513] * 40, {}),                                  # one partition plans, and split ones
    ([3000, 10, 2500, 1200], dict(window=1000)), ([9000], dict(kv="same", spread=1, alibi=True)),
    ([2000] * 80, dict(hq=4, hkv=2, d=64)),
])
def test_decode_plans(lens, kw):
    c = Case(77, [(n - 1, 1) for n in lens], **kw)
    for part in (0, 16, 512):
        got = c.decode(part)
        ok()
        c.check(got)


def test_decode_max_seq_len_above_the_contexts():
    c = Case(5, [(99, 1), (30, 1)], window=50)
    for msl in (100, 131, 4000, 100000):
        got = c.decode(max_seq_len=msl)
        ok()
        c.check(got)


def test_decode_empty_and_bad_lengths():
    c = Case(6, [(49, 1), (0, 1), (20, 1)], window=30, softcap=9.0)
    c.seq_lens[1] = 0
    got = c.decode()
    ok()
    assert (got[0][1] == 0).all() and (got[1][1] == -np.inf).all()
    ref = c.want()
    c.check(got, ref, [0, 2])
    c.seq_lens[1] = -3
    got = c.decode()
    torch.cuda.synchronize()
    assert P.pkv_get_device_error() == SEQ_LEN
    assert (got[0][1] == 0).all()
    c.check(got, ref, [0, 2])
    c.seq_lens[1] = 1
    c.tables[1, 0] = c.k.shape[0]
    c.decode()
    torch.cuda.synchronize()
    assert P.pkv_get_device_error() == BLOCK_ID


def test_decode_block_scales_far_apart():
    # V scales of one context 2^80 apart with the weight on the small ones: the result is theirs
    c = Case(8, [(99, 1), (600, 1)], spread=0)
    ref0 = c.want()
    first = c.tables[:, 0].long()
    lo, hi = c.vs.clone(), c.vs.clone()
    for b in range(2):
        rows = c.tables[b][c.tables[b] >= 0].long()
        hi[rows] = c.vs[rows] - 40
        hi[rows[0]] = c.vs[rows[0]] + 40
        lo[rows] = c.vs[rows] - 60
    # keys of the first block (the large V scale) get scores far below the others'
    kk = c.k[first].double().abs() * -1
    c.k[first] = kk.to(c.k.dtype)
    c.q.abs_()
    c.ks[first] += 8
    c.vs = hi
    got = c.decode()
    ok()
    c.check(got)
    c.vs = lo
    got = c.decode()
    ok()
    ref = c.want()
    err = (got[0].double() - ref.out).abs()
    tol = R.tolerance(ref, c.q.dtype, c.p_dtype) - 2.0 ** -24       # values near 2^-60: no floor
    assert (err <= tol).all()
    assert ref0.out.isfinite().all()


@pytest.mark.parametrize("kw", [dict(), dict(kv="head"), dict(kv="same", dtype="f16", spread=1),
                                dict(d=256), dict(d=64, bs=64)])
def test_small_weights_where_the_largest_meet_zeros(kw):
    # A steep bias: weights fall by 2^-1 a key, and V is 0 for the last 18 keys of a row, so what
    # is left has weights from 2^-18 on. The largest weight is held as 2^7 or more, so one is off by
    # 2^-11 of itself or, below f16's normal range (2^-14 against 2^7), by half of its
    # subnormal step 2^-24: 2^-32 of the largest weight, for each key. (Keys more than 40
    # back weigh less than 2^-40 each, 300 of them, and may be lost.) With block scales what is
    # held is the weight times the V scale 2^ev of its block: 2^-32 of the largest
    # of those, which in units of a key's own weight is at most 2^(largest ev - its ev) more.
    seqs = [(300, 1), (70, 1), (41, 1)]
    for lens, run in ((seqs, "decode"), ([(299, 2), (69, 2), (40, 2)], "prefill")):
        c = Case(21, lens, qsize=0.1, alibi=True, **kw)
        c.slopes = torch.full_like(c.slopes, 0.6931)
        bs, hkv = c.v.shape[2], c.v.shape[1]
        near = torch.zeros(c.q.shape, dtype=torch.float64, device="cuda")
        for n, (p, q) in enumerate(lens):
            for j in range(p + q - 18, p + q):
                c.v[c.tables[n, j // bs].long(), :, j % bs] = 0
            j = torch.arange(p + q - 41, p + q, device="cuda")
            block = c.tables[n, j // bs].long()
            vs = c.vs if c.vs is None or c.vs.dim() == 1 else c.vs[block]
            v = R.values(c.v[block], vs)[torch.arange(41, device="cuda"), :, j % bs].abs()
            if c.vs is not None and c.vs.dim() == 2:
                ev = c.vs[block].double()
                v = v * torch.exp2(ev.amax(0) - ev)[..., None]
            near[int(c.cu[n]):int(c.cu[n + 1])] = v.sum(0).repeat_interleave(c.q.shape[1] // hkv, 0)
        out, _ = getattr(c, run)()
        ok()
        ref = c.want()
        err = (out.double() - ref.out).abs()
        tol = R.tolerance(ref, c.q.dtype, c.p_dtype) - 2.0 ** -24 + 2.0 ** -32 * near + 2.0 ** -31
        assert ref.mass.max() < 2.0 ** -11          # nothing but small weights is left
        if c.q.dtype == torch.float16:               # f16 outputs that small are subnormal
            tol = tol + 2.0 ** -25
        assert (err <= tol).all()


def test_nan_scale_reaches_its_sequence_alone():
    c = Case(9, [(99, 1), (60, 1)])
    ref = c.want()
    c.vs[c.tables[0, 2].long(), 1] = 255
    out, _ = c.decode()
    ok()
    assert out[0, 4:].isnan().all()
    c.check((out, None), ref, [1])
    assert ((out[0, :4].double() - ref.out[0, :4]).abs() <=
            R.tolerance(ref, c.q.dtype, c.p_dtype)[0, :4]).all()


PREFILL = [
    dict(kv="block"),
    dict(kv="block", dtype="f16", hq=7, hkv=1, bs=64),
    dict(kv="block", d=64, bs=32, hq=16, hkv=1),
    dict(kv="block", d=256, hq=8, hkv=2),
    dict(kv="block", d=256, hq=3, hkv=3, window=30, softcap=8.0, dtype="f16", qsize=3.0),
    dict(kv="block", softcap=15.0, alibi=True, prefix=[0, 3, 900, 40, 16, -5, 1], hq=12, hkv=4),
    dict(kv="block", window=40),
    dict(kv="block", window=1, bs=32, d=64),
    dict(kv="block", window=100, prefix=[5, 1, 8, 333, 99, 0, 60], hq=5, hkv=1),
    dict(kv="head", softcap=30.0, qsize=4.0),
    dict(kv="head", d=64, dtype="f16", window=33, alibi=True, hq=2, hkv=2),
    dict(kv="head", d=256, alibi=True),
    dict(kv="same", softcap=50.0, qsize=6.0, spread=1),
    dict(kv="same", dtype="f16", alibi=True, hq=12, hkv=4, d=64, spread=1,
         prefix=[1, 0, 2, 50, 64, 700, 7]),
    dict(kv="same", d=256, window=64, hq=16, hkv=8, spread=1, bs=32),
    dict(kv="same", dtype="f16", window=5, alibi=True, softcap=2.0, hq=13, hkv=1, spread=1),
    dict(kv="same", window=300, hq=16, hkv=1, spread=1, prefix=[0, 3, 9, 40, 16, 600, 1]),
    dict(kv="same", spread=1),
]
CHUNKS = [(0, 1), (0, 3), (10, 7), (300, 130), (63, 65), (500, 300), (127, 1)]


@pytest.mark.parametrize("i", range(len(PREFILL)))
def test_prefill(i):
    c = Case(50 + i, CHUNKS, pad=3, **PREFILL[i])
    got = c.prefill()
    ok()
    c.check(got)
    assert (got[0][-3:] == 9).all() and (got[1][-3:] == 9).all()


@pytest.mark.parametrize("seqs,kw", [
    ([(1500, 512)], dict(hq=16, hkv=8)), ([(1500, 512)], dict(hq=16, hkv=8, kv="same", spread=1,
                                                               softcap=30.0, window=256)),
    ([(0, 2000)], dict(hq=4, hkv=1)), ([(3000, 20)], dict(kv="same", spread=1, alibi=True)),
    ([(3000, 20)], dict(kv="head", window=700)), ([(100, 0), (5, 40), (0, 0)], {}),
    ([(40, 900)], dict(kv="block", prefix=[500], d=64)),
    ([(0, 1100)], dict(kv="same", spread=1, window=2000, softcap=1.0, d=256, hq=2, hkv=1)),
])
def test_prefill_sizes(seqs, kw):
    c = Case(91, seqs, **kw)
    got = c.prefill()
    ok()
    c.check(got)


# few query rows on long contexts: the keys of a query tile are shared out over the CTAs of a
# cluster, some of which (the short sequences, the windows) get none
@pytest.mark.parametrize("kw", [
    dict(), dict(dtype="f16", softcap=20.0, alibi=True), dict(window=1200), dict(window=300),
    dict(prefix=[2000, 0, 700, 1, 5, 900]), dict(d=64), dict(d=64, alibi=True, bs=32),
    dict(d=256, hq=3, hkv=1), dict(d=256, softcap=4.0, window=600),
    dict(kv="head", alibi=True), dict(kv="head", d=64, dtype="f16", window=2100),
    dict(kv="head", d=256, softcap=30.0), dict(kv="same", spread=1, softcap=30.0),
    dict(kv="same", spread=1, d=64, dtype="f16", alibi=True),
    dict(kv="same", spread=1, d=256, prefix=[3, 1, 2400, 0, 0, 64])])
def test_prefill_few_rows_of_long_contexts(kw):
    c = Case(131, [(2500, 3), (40, 5), (4100, 1), (0, 2), (1027, 30), (2047, 1)], **kw)
    got = c.prefill()
    ok()
    c.check(got)
    again = c.prefill()
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


def test_prefill_block_scales_far_apart():
    # neighbouring blocks' V scales 2^70 apart, the weight on the small ones
    c = Case(12, [(200, 60)], spread=0, hq=4, hkv=2)
    even = c.tables[0, 0:16:2].long()
    c.k[even] = (c.k[even].double().abs() * -1).to(c.k.dtype)
    c.q.abs_()
    c.ks[even] += 8
    c.vs[even] += 30
    odd = c.tables[0, 1:16:2].long()
    c.vs[odd] -= 40
    c.scale = 1.0
    out, _ = got = c.prefill()
    ok()
    ref = c.want()
    rows = slice(16, 60)
    err = (out.double() - ref.out).abs()[rows]
    tol = (R.tolerance(ref, c.q.dtype, c.p_dtype) - 2.0 ** -24)[rows]
    assert (err <= tol).all()


@pytest.mark.parametrize("kw", [dict(), dict(softcap=9.0), dict(d=64), dict(d=256), dict(bs=64)])
@pytest.mark.parametrize("which", ["ks", "vs"])
def test_prefill_nan_scale_reaches_the_rows_that_see_it(which, kw):
    c = Case(19, [(20, 180), (30, 20)], **kw)
    ref = c.want()
    bs = c.k.shape[2]
    block = 100 // bs
    getattr(c, which)[c.tables[0, block].long(), 1] = 255
    out, _ = c.prefill()
    ok()
    first = max(0, block * bs - 20)                    # the first row that sees the block
    assert out[first:180, 4:].isnan().all()
    c.check((out, None), ref, list(range(first)) + list(range(180, 200)))
    tol = R.tolerance(ref, c.q.dtype, c.p_dtype, c.softcap)
    assert ((out.double() - ref.out).abs() <= tol)[:, :4].all()


@pytest.mark.parametrize("kw", [dict(), dict(kv="same", spread=1, alibi=True), dict(d=256)])
def test_largest_window_sees_everything(kw):
    c = Case(20, [(200, 70), (0, 33), (5, 1)], **kw)
    for w in (2 ** 31 - 1, 271):
        c.prefix = None
        got = c.prefill(window=w)
        c.check(got)
        c.prefix = torch.tensor([260, 33, -1], dtype=torch.int32).cuda()
        got = c.prefill(window=w)
        c.check(got)
    ok()


@pytest.mark.parametrize("kw", [
    dict(kv="same", spread=1, softcap=30.0), dict(kv="same", spread=1, softcap=3.0, window=200),
    dict(kv="same", spread=1, softcap=3.0, d=256, dtype="f16"), dict(kv="head", softcap=3.0, d=64),
    dict(softcap=3.0, alibi=True), dict(softcap=30.0, d=64, bs=32), dict(), dict(window=70),
    dict(kv="same", spread=1, alibi=True)])
def test_prefill_rows_do_not_depend_on_keys_they_do_not_see(kw):
    # the last 20 tokens' keys and values change, and the slots behind them: not one bit of the
    # rows before them does
    seqs = [(300, 100), (0, 70), (650, 45), (33, 21)]
    c = Case(137, seqs, **kw)
    out, lse = c.prefill()
    ok()
    bs = c.k.shape[2]
    big = torch.tensor(64.0).to(c.k.dtype).cuda()
    for i, (p, q) in enumerate(seqs):
        for j in range(p + q - 20, -(-(p + q) // bs) * bs):
            b = int(c.tables[i, j // bs])
            c.k[b, :, j % bs, ::2] = big
            c.k[b, :, j % bs, 1::2] = big / 2 if c.k.dtype != torch.float8_e4m3fn else big
            c.v[b, :, j % bs] = big
    out2, lse2 = c.prefill()
    ok()
    at = 0
    for p, q in seqs:
        rows = slice(at, at + q - 20)
        assert torch.equal(out[rows], out2[rows]) and torch.equal(lse[rows], lse2[rows])
        assert not torch.equal(out[at + q - 20:at + q], out2[at + q - 20:at + q])
        at += q


@pytest.mark.parametrize("cap", [300.0, 1e6, 1e30, 2e38])
@pytest.mark.parametrize("kw", [dict(), dict(kv="same", spread=1), dict(kv="head", d=64, dtype="f16"),
                                dict(kv="same", spread=1, d=256)])
def test_a_cap_far_above_the_scores(cap, kw):
    # inside the cap tanh is right to 2e-7 of itself, so of the score: less than the 4 * 2^-23 of
    # it that lse_tolerance and tolerance have for conversions. Nothing in the bound grows
    # with the cap
    c = Case(151, [(p + q - 1, 1) for p, q in CHUNKS], softcap=cap, **kw)
    ref = c.want()
    assert float(ref.size.max()) < 250                # sum |q k| * scale: no score reaches a cap
    for out, lse in (c.decode(), c.prefill()):
        ok()
        err = (out.double() - ref.out).abs()
        assert not (err > R.tolerance(ref, c.q.dtype, c.p_dtype)).any()
        assert not ((lse.double() - ref.lse).abs() > R.lse_tolerance(ref)).any()


def test_prefill_bad_sequences():
    c = Case(13, [(50, 10), (3, 20), (70, 8)])
    ref = c.want()
    c.seq_lens[1] = 12                              # shorter than its chunk
    out, lse = c.prefill()
    torch.cuda.synchronize()
    assert P.pkv_get_device_error() == QLEN
    rows = list(range(10)) + list(range(30, 38))
    c.check((out, lse), ref, rows)
    assert (out[10:30] == 9).all()
    c.seq_lens[1] = 23
    out, _ = c.prefill(max_q_len=15)                # one chunk longer than said
    torch.cuda.synchronize()
    assert P.pkv_get_device_error() == QLEN
    c.check((out, None), ref, rows)
    assert (out[10:30] == 9).all()
    c.tables[0, 0] = -1
    c.prefill()
    torch.cuda.synchronize()
    assert P.pkv_get_device_error() == BLOCK_ID


def test_offsets_past_32_bits():
    # a pool of more than 2^32 bytes a cache, the tokens in its last blocks
    nb = (1 << 32) // (2 * 64 * 256) + 9
    c = Case(14, [(70, 5), (300, 1)], hq=4, hkv=2, d=256, bs=64, pool=nb)
    got = c.prefill()
    ok()
    c.check(got)
    d = Case(15, [(70, 1), (300, 1)], hq=4, hkv=2, d=256, bs=64, pool=nb)
    got = d.decode()
    ok()
    d.check(got)
    key = torch.randn(6, 2, 256, device="cuda").bfloat16()
    st = [c.k, c.v, c.ks, c.vs]
    b = c.tables[c.tables >= 0].long()
    sub = [x[b].clone() for x in st]
    at = torch.full(c.tables.shape, -1, dtype=torch.int32, device="cuda")
    at[c.tables >= 0] = torch.arange(len(b), dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 5, 6], dtype=torch.int32, device="cuda")
    P.rope_append_block_scaled(key, key, *st, c.tables, c.seq_lens, cu)
    ok()
    k, v, ks, vs, _ = R.append(key, key, *sub, at, c.seq_lens, cu)
    for x, y in ((st[0][b].double(), k), (st[1][b].double(), v)):
        assert torch.equal(x.nan_to_num(500), y.nan_to_num(500))
    assert torch.equal(st[2][b].long(), ks) and torch.equal(st[3][b].long(), vs)


def test_other_stream_and_bitwise_repeat():
    c = Case(16, [(n - 1, 1) for n in LENS + [5000]])
    a = c.decode()
    ws = torch.zeros(P.paged_attn_decode_ext_workspace_size(len(LENS) + 1, 8, 2, 128, c.max_ctx),
                     dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = c.decode(workspace=ws)
    out = torch.empty_like(c.q)
    P.paged_attn_decode_ext(out, c.q, c.k, c.v, c.tables, c.seq_lens, c.scale, c.max_ctx, c.ks, c.vs,
                            workspace=torch.zeros_like(ws), stream=s.cuda_stream)
    ok()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.equal(a[0], out)
    p = Case(17, CHUNKS)
    x = p.prefill()
    with torch.cuda.stream(s):
        y = p.prefill()
    ok()
    assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


def test_binding_refuses():
    c = Case(18, [(20, 1), (30, 1)])

    def call(**kw):
        a = dict(out=torch.empty_like(c.q), q=c.q, k_cache=c.k, v_cache=c.v, block_tables=c.tables,
                 seq_lens=c.seq_lens, scale=c.scale, max_seq_len=64, k_scales=c.ks, v_scales=c.vs)
        a.update(kw)
        P.paged_attn_decode_ext(**a)
    call()
    ok()
    half = torch.zeros(c.k.shape, dtype=torch.bfloat16, device="cuda")
    for bad in (dict(q=c.q[:1]), dict(out=c.q.half()), dict(v_cache=c.v[:-1]), dict(k_scales=c.ks[0]),
                dict(v_scales=c.vs.float()), dict(k_cache=half, v_cache=half),
                dict(block_tables=c.tables[:1]), dict(seq_lens=c.seq_lens[:1]),
                dict(alibi_slopes=torch.zeros(3, device="cuda")),
                dict(out_lse=torch.zeros(2, 4, device="cuda")), dict(q=c.q.cpu()),
                dict(seq_lens=c.seq_lens.cpu()), dict(k_scales=c.ks.t())):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(scale=-1.0), dict(softcap=-1.0), dict(window=-1), dict(partition_tokens=8),
                dict(workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(P.PkvError):
            call(**bad)
    p = dict(out=torch.empty_like(c.q), q=c.q, k_cache=c.k, v_cache=c.v, block_tables=c.tables,
             seq_lens=c.seq_lens, scale=c.scale, max_q_len=1, k_scales=c.ks, v_scales=c.vs)
    for bad in (dict(cu_q_lens=c.cu[:2]), dict(cu_q_lens=c.cu.long()),
                dict(cu_q_lens=c.cu, prefix_lens=c.cu)):
        with pytest.raises(ValueError):
            P.paged_attn_prefill_chunk_ext(**{**p, **bad})

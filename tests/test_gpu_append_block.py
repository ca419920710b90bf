"""rope_append_block_scaled against its definition in 64 bits: codes, scales and
rotated queries equal value for value, whatever the blocks held before."""
import numpy as np
import pytest
import torch

import paged_kv_decode_11_gb300 as P
from tests import ext_ref as R

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}
QLEN, POSITION, BLOCK_ID = 0x10, 0x20, 0x1


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from paged_kv_decode_11_gb300 import build
    build.build()
    P.load()
    torch.cuda.init()
    P.pkv_get_device_error()


class Case:
    """seqs: (cached tokens, new tokens) of each sequence; `extra` rows before and behind all."""

    def __init__(self, seed, seqs, hq=8, hkv=2, d=128, bs=16, dtype="bf16", rot=128, neox=True,
                 extra=(0, 0), size=1.0):
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        dt = DT[dtype]
        need = [-(-(p + q) // bs) for p, q in seqs]
        nb = sum(need) + 4
        maxb = max(need + [1]) + 1
        ids = rng.permutation(nb)
        t = torch.full((len(seqs), maxb), -1, dtype=torch.int32)
        at = 0
        for i, m in enumerate(need):
            t[i, :m] = torch.from_numpy(ids[at:at + m].astype(np.int32))
            at += m
        cu = np.concatenate([[extra[0]], extra[0] + np.cumsum([q for _, q in seqs])])
        rows = int(cu[-1]) + extra[1]
        self.tables, self.seq_lens = t.cuda(), torch.tensor([p + q for p, q in seqs],
                                                            dtype=torch.int32).cuda()
        self.cu = torch.tensor(cu, dtype=torch.int32).cuda()
        codes = torch.randn(2, nb, hkv, bs, d, generator=g) * 100
        self.k, self.v = codes.to(torch.float8_e4m3fn).cuda()
        # stored scales around the size of what comes: some blocks grow, some do not
        self.ks, self.vs = torch.randint(110, 128, (2, nb, hkv), generator=g).to(torch.uint8).cuda()
        spread = torch.exp2(torch.randint(-6, 7, (rows, hkv, 1), generator=g).float()) * size
        self.key = (torch.randn(rows, hkv, d, generator=g) * spread).to(dt).cuda()
        self.value = (torch.randn(rows, hkv, d, generator=g) * spread).to(dt).cuda()
        self.query = torch.randn(rows, hq, d, generator=g).to(dt).cuda()
        self.neox = neox
        self.cos_sin = None
        if rot:
            inv = 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) / (rot // 2))
            a = torch.arange(maxb * bs + 1, dtype=torch.float64)[:, None] * inv
            self.cos_sin = torch.cat([a.cos(), a.sin()], 1).float().cuda()

    def state(self):
        return [x.clone() for x in (self.k, self.v, self.ks, self.vs)]

    def call(self, st, query_out=None, **kw):
        q = self.query if self.cos_sin is not None else None
        P.rope_append_block_scaled(self.key, self.value, *st, self.tables, self.seq_lens, self.cu,
                                   query=q, query_out=query_out if q is not None else None,
                                   cos_sin_cache=self.cos_sin, neox_style=self.neox, **kw)

    def want(self, st=None, skip=()):
        q = self.query if self.cos_sin is not None else None
        return R.append(self.key, self.value, *(st or self.state()), self.tables, self.seq_lens,
                        self.cu, q, self.cos_sin, self.neox, skip)


def check(st, want):
    k, v, ks, vs, _ = want
    assert torch.equal(st[2].long(), ks) and torch.equal(st[3].long(), vs)
    for got, ref in ((st[0], k), (st[1], v)):
        got = got.view(torch.float8_e4m3fn).double()
        assert torch.equal(got.isnan(), ref.isnan())
        assert torch.equal(got.nan_to_num(0), ref.nan_to_num(0))


SHAPES = [
    # one token at each place of a block; a chunk from an empty cache; blocks' borders
    dict(seqs=[(0, 1)]),
    dict(seqs=[(15, 1), (16, 1), (17, 1), (31, 1), (200, 1)], rot=64),
    dict(seqs=[(0, 16), (0, 17), (5, 11), (5, 12), (16, 48), (3, 100)], neox=False),
    dict(seqs=[(0, 0), (40, 3), (7, 0), (0, 5), (33, 0)], extra=(2, 3)),
    dict(seqs=[(0, 64), (63, 1), (63, 2), (10, 300)], bs=64, d=64, dtype="f16", rot=16),
    dict(seqs=[(31, 40), (0, 33)], bs=32, d=256, hq=7, hkv=1, rot=256),
    dict(seqs=[(31, 40), (64, 3)], bs=64, d=256, hq=3, hkv=3, rot=0),
    dict(seqs=[(i, 1) for i in range(70)], hkv=8, hq=16, dtype="f16", rot=128, neox=False),
    # a decode batch behind a chunk, and chunks long enough for several rows a CTA
    dict(seqs=[(100, 1), (5, 1500), (99, 1), (3, 1300), (0, 1)], hkv=8, hq=8, bs=16),
    dict(seqs=[(9, 2500), (3, 1)] + [(i, 1) for i in range(40)], hkv=8, hq=8, bs=64, rot=64),
]


@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_append_equals_definition(i):
    c = Case(100 + i, **SHAPES[i])
    st = c.state()
    qo = torch.full_like(c.query, 7.0)
    c.call(st, qo)
    torch.cuda.synchronize()
    assert P.pkv_get_device_error() == 0
    want = c.want()
    check(st, want)
    if c.cos_sin is not None:
        lo, hi = int(c.cu[0]), int(c.cu[-1])
        assert torch.equal(qo[lo:hi], want[4][lo:hi])
        assert (qo[:lo] == 7).all() and (qo[hi:] == 7).all()     # rows of nobody: left alone


def test_append_in_place_queries_and_again():
    c = Case(3, [(20, 1), (0, 40)])
    want = c.want()
    st = c.state()
    q = c.query.clone()
    P.rope_append_block_scaled(c.key, c.value, *st, c.tables, c.seq_lens, c.cu, query=q,
                               cos_sin_cache=c.cos_sin)
    assert torch.equal(q, want[4])
    check(st, want)
    c.call(st, torch.empty_like(q))            # the same tokens once more change nothing
    check(st, want)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_append_odd_values(dtype):
    c = Case(4, [(0, 20), (8, 8), (24, 1), (40, 1)], rot=0, dtype=dtype)
    big = torch.finfo(DT[dtype]).max
    c.key[0, 0, :4] = torch.tensor([np.inf, -np.inf, np.nan, 1.0])
    c.key[1, 1] = 0.0
    c.value[:16] = 0.0                           # a whole block of zeros
    c.value[16:20, 0] = np.nan                   # nothing finite
    c.value[20:28] = torch.finfo(DT[dtype]).tiny
    c.value[28] = big
    c.key[29, :, 0] = -big
    st = c.state()
    c.ks[:, 0] = 0                               # scales never written before
    c.vs[:, 1] = 255
    st[2][:, 0] = 0
    st[3][:, 1] = 255
    c.call(st)
    assert P.pkv_get_device_error() == 0
    check(st, c.want())


def test_scale_borders():
    # amax = 448 * 2^e takes e, the next larger value e + 1
    c = Case(5, [(0, 1), (0, 1), (0, 1), (0, 1)], rot=0, dtype="f16", hkv=1)
    c.key.zero_()
    c.value.zero_()
    c.key[0, 0, 3], c.key[1, 0, 3] = 448.0, 448.5
    c.value[2, 0, 5], c.value[3, 0, 5] = 3.5, -3.501953125
    st = c.state()
    c.call(st)
    check(st, c.want())
    b = c.tables[:, 0].long()
    assert st[2][b, 0].tolist() == [127, 128, 67, 67]
    assert st[3][b, 0].tolist() == [67, 67, 120, 121]


def test_token_by_token_ends_at_the_scale_of_the_whole():
    # the scale of a block is that of its largest element, however the tokens came
    one = Case(6, [(0, 40)], rot=0)
    st = one.state()
    one.call(st)
    steps = one.state()
    for i in range(40):
        n = torch.tensor([i + 1], dtype=torch.int32, device="cuda")
        cu = torch.tensor([i, i + 1], dtype=torch.int32, device="cuda")
        P.rope_append_block_scaled(one.key, one.value, *steps, one.tables, n, cu)
    used = one.tables[0, :3].long()
    for a, b in ((0, 2), (1, 3)):
        assert torch.equal(st[b][used], steps[b][used])
        # a code re-encoded on the way is off by at most its subnormal step each time the
        # scale grew (2^-10 of a unit of the scale, half a step, at most 40 times) on top of a half step
        # (offsets 8 to 15 of the third block hold no token)
        x, y = (s[a][used].double().transpose(1, 2).flatten(0, 1)[:40] for s in (st, steps))
        grow = 2.0 ** -10 * 40
        assert ((x - y).abs() <= 2 * x.abs() * 2.0 ** -4 + grow).all()


def test_bad_sequences_are_flagged_and_skipped():
    c = Case(7, [(10, 5), (0, 6), (20, 4), (3, 2)])
    st, keep = c.state(), c.state()
    c.seq_lens[1] = 4                            # shorter than its chunk
    qo = torch.full_like(c.query, 7.0)
    c.call(st, qo)
    assert P.pkv_get_device_error() == QLEN
    want = c.want(keep, skip=(1,))
    check(st, want)
    assert (qo[5:11] == 7).all() and torch.equal(qo[11:], want[4][11:])

    c = Case(8, [(10, 5), (100, 6)])
    st, keep = c.state(), c.state()
    c.cos_sin = c.cos_sin[:100].contiguous()     # the second context is past the table
    c.call(st, torch.empty_like(c.query))
    assert P.pkv_get_device_error() == POSITION
    c2 = Case(8, [(10, 5), (100, 6)])
    check(st, c2.want(keep, skip=(1,)))

    c = Case(9, [(10, 25), (30, 3)], rot=0)
    c.tables[0, 1] = c.k.shape[0]                # one block of the first sequence: outside
    c.tables[1, 1] = -5
    st, keep = c.state(), c.state()
    c.call(st)
    assert P.pkv_get_device_error() == BLOCK_ID
    check(st, c.want(keep))


@pytest.mark.parametrize("cu", [[0, 5, 3, 9], [-2, 4, 6, 9], [0, 5, 6, 400], [3, 3, 3, 3]])
def test_bad_offsets_touch_nothing_else(cu):
    # offsets that decrease or leave the rows: no access out of range, the sound sequences done
    c = Case(10, [(10, 5), (20, 1), (30, 3)], rot=0)
    c.cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    st = c.state()
    c.call(st)
    bits = P.pkv_get_device_error()
    assert bits == (0 if cu == [3, 3, 3, 3] else QLEN)
    free = torch.ones(c.k.shape[0], dtype=torch.bool, device="cuda")
    free[c.tables[c.tables >= 0].long()] = False
    for a, b in zip(st, c.state()):
        assert torch.equal(a.view(torch.uint8)[free], b.view(torch.uint8)[free])


def test_binding_refuses():
    c = Case(11, [(10, 5)])
    st = c.state()

    def call(**kw):
        a = dict(key=c.key, value=c.value, k_cache=st[0], v_cache=st[1], k_scales=st[2],
                 v_scales=st[3], block_tables=c.tables, seq_lens=c.seq_lens, cu_q_lens=c.cu,
                 query=c.query, cos_sin_cache=c.cos_sin)
        a.update(kw)
        P.rope_append_block_scaled(**a)
    for bad in (dict(value=c.value[:, :1]), dict(k_scales=st[2].float()), dict(v_scales=st[3][:-1]),
                dict(cu_q_lens=c.cu[:1]), dict(seq_lens=c.seq_lens.long()),
                dict(query=c.query[..., :64]), dict(query_out=c.query[:-1]),
                dict(cos_sin_cache=None), dict(query=None, query_out=c.query),
                dict(key=c.key.cpu()), dict(k_cache=st[0].half()),
                dict(key=c.key.transpose(1, 2).contiguous().transpose(1, 2)),
                dict(value=c.value.to(torch.float32))):
        with pytest.raises(ValueError):
            call(**bad)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(st, c.state()))

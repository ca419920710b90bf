"""paged_attn_tree where its softmax and its masks are at their limits, against attention in 64 bits
(tests/tree_ref.py, tolerances of tests/ext_ref.py)."""
import numpy as np
import pytest
import torch

import paged_kv_decode_11_gb300 as P
from tests import ext_ref as R
from tests import tree_ref as T
from tests.test_gpu_tree import QLEN, Case, ok

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from paged_kv_decode_11_gb300 import build
    build.build()
    P.load()
    torch.cuda.init()
    P.pkv_get_device_error()


@pytest.mark.parametrize("log2_score", [250, 1500, 4100, 8200, 33000])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("kw", [dict(kv="same", dtype="f16"), dict(kv="same"), dict(kv="same", d=64),
                                dict(kv="head"), dict(kv="head", dtype="f16", d=64), dict(kv="block"),
                                dict(kv="block", dtype="f16", d=64), dict(kv="same", dtype="f16", d=256)])
def test_large_scores_that_lie_close_together(kw, sign, log2_score):
    # every key of a row has about the same large score, so that several keys share its weight:
    # the reference of the weights has to follow the row's maximum exactly
    c = Case(50, [(3, 4), (1, 1), (40, 13), (0, 40), (700, 5)], **kw)
    d = c.q.shape[2]
    g = torch.Generator().manual_seed(51)
    unseen = c.k.float().isnan()
    k = torch.randn(c.k.shape, generator=g)
    k[..., 0] = 128.0
    c.k = k.to(c.k.dtype).cuda()
    c.k.view(torch.uint8 if c.k.element_size() == 1 else torch.int16)[unseen] = 0x7F if kw["kv"] != "same" else -1
    if kw["kv"] == "head":
        c.ks = torch.ones_like(c.ks)
    elif kw["kv"] == "block":
        c.ks = torch.full_like(c.ks, 127)
    c.q = torch.randn(c.q.shape, generator=g).to(c.q.dtype).cuda()
    # score = scale * (128 q0 + a sum of d - 1 products of N(0, 1)); log2 units
    q0 = log2_score * d ** 0.5 / (128 * 1.4427)
    c.q[..., 0] = sign * q0
    got = c.run()
    ok()
    c.check(got)


def sees(c, n, m):
    """Of sequence n's rows (of q), those that see its node m (below 0: its context)."""
    lo, hi = c.cu[n:n + 2].tolist()
    i = torch.arange(hi - lo)
    mine = (m <= i) if c.masks is None or m < 0 else c.masks[lo:hi, m]
    rows = torch.zeros(c.q.shape[0], dtype=torch.bool)
    rows[lo:hi] = mine
    return rows.cuda()


@pytest.mark.parametrize("masks", ["tree", "chain", "random"])
@pytest.mark.parametrize("kw", [dict(kv="same"), dict(kv="same", dtype="f16", d=64), dict(kv="same", d=256),
                                dict(kv="same", hq=32), dict(kv="same", dtype="f16", hq=32, bs=64),
                                dict(kv="head"), dict(kv="head", hq=32, d=64), dict(kv="head", d=256),
                                dict(kv="block", spread=3), dict(kv="block", hq=32, bs=32)])
def test_values_that_are_no_numbers_reach_the_rows_that_see_them(kw, masks):
    # elements of V, in the element of the output alone: of nodes, the rows whose masks have them,
    # of the context, all of the sequence's (trees of one tile and two, items of one part and more)
    seqs = [(200, 20), (9000, 5), (0, 17), (40, 70), (120, 16), (1300, 33)]
    c = Case(60, seqs, masks=masks, pad=2, **kw)
    ref = c.want()
    d, hkv = c.q.shape[2], c.k.shape[1]
    group = c.q.shape[1] // hkv
    odd = [float("inf"), -float("inf"), float("nan")] if kw["kv"] == "same" else [float("nan")]
    want = ref.out.clone()
    spots = [(n, p + m, k) for n, (p, l) in enumerate(seqs) for k, m in enumerate(range(0, l, 3)) if n != 4]
    spots += [(4, 120, 0), (4, 121, 1), (4, 135, 2), (1, 4000, 0), (5, 1299, 0)]     # (5: a context's last)
    for n, pos, k in spots:
        P0 = seqs[n][0]
        rows = sees(c, n, pos - P0)
        if not bool(rows.any()):
            continue                                          # (NaN already)
        for head in range(hkv):
            col, x = (7 * k + 13 * n + 5 * head) % d, odd[(k + n + head) % len(odd)]
            at = int(c.tables[n, pos // c.k.shape[2]]), head, pos % c.k.shape[2]
            c.v[at][col] = x
            want[rows, head * group:(head + 1) * group, col] += x
    out, lse = c.run()
    ok()
    assert (out[-2:] == 9).all()
    out, want, tol = out[:-2].double(), want[:-2], R.tolerance(ref, c.q.dtype, c.p_dtype)[:-2]
    # (an infinity comes out as itself or, where a copy of the row or a part of the item has no weight
    # for its key, as NaN)
    assert torch.equal(out.isfinite(), want.isfinite()) and out[want.isnan()].isnan().all()
    assert (out[out.isinf()] == want[out.isinf()]).all()
    near = (out - want).abs() <= tol
    assert near[want.isfinite()].all()
    assert ((lse.double() - ref.lse).abs()[:-2] <= R.lse_tolerance(ref)[:-2])[ref.lse[:-2].isfinite()].all()


@pytest.mark.parametrize("kw", [dict(kv="same"), dict(kv="same", dtype="f16", d=64, hq=32), dict(kv="same", d=256),
                                dict(kv="head"), dict(kv="head", d=256), dict(kv="block", spread=3, hq=32)])
def test_keys_that_are_no_numbers_reach_the_rows_that_see_them(kw):
    # NaN, or a score of +inf: NaN in the row's out and lse; a score of -inf: no weight; rows that
    # do not see the key, as if it were not there
    seqs = [(200, 20), (9000, 5), (3, 17), (40, 70), (130, 33), (77, 50)]
    c = Case(61, seqs, masks="tree", **kw)
    bad = torch.zeros(c.q.shape[:2], dtype=torch.bool, device="cuda")
    without = c.masks.clone()
    for n, (m, x) in enumerate(((7, "nan"), (2, "inf"), (15, "-inf"), (64, "nan"), (13, "inf"), (31, "-inf"))):
        x = float(x) if kw["kv"] == "same" else float("nan")
        pos = seqs[n][0] + m
        c.k[int(c.tables[n, pos // c.k.shape[2]]), :, pos % c.k.shape[2], 5] = x
        rows = sees(c, n, m)
        bad |= rows[:, None] & ~(c.q[:, :, 5].float() * x == -float("inf"))
        without[rows.cpu(), m] = False
    out, lse = c.run()
    ok()
    assert bad.any() and out[bad].isnan().all() and lse[bad].isnan().all()
    ref = T.attention(c.q, c.k, c.v, c.tables, c.seq_lens, c.cu, c.scale, without, c.ks, c.vs)
    assert ((out.double() - ref.out).abs() <= R.tolerance(ref, c.q.dtype, c.p_dtype))[~bad].all()
    assert ((lse.double() - ref.lse).abs() <= R.lse_tolerance(ref))[~bad].all()


@pytest.mark.parametrize("kv", ["same", "head", "block"])
def test_what_was_no_number_is_forgotten_by_the_next_call(kv):
    # eager, and replayed from a graph, with a workspace that another call has used in between
    c, other = Case(62, [(700, 20), (9000, 9), (60, 40)], kv=kv), Case(63, [(3000, 12)], kv=kv)
    ws = torch.empty(P.paged_attn_tree_workspace_size(8, 2, 128), dtype=torch.uint8, device="cuda")
    clean = c.run(lse=False, workspace=ws)[0].clone()
    out = torch.empty_like(clean)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(lse=False, out=out, workspace=ws)
    spots = [(int(c.tables[n, pos // 16]), slice(None), pos % 16, 3) for n, pos in ((0, 703), (1, 9008), (2, 65))]
    was = [c.v[s].clone() for s in spots]
    for call in (graph.replay, lambda: c.run(lse=False, out=out, workspace=ws)):
        for s in spots:
            c.v[s] = float("nan")
        call()
        seen = torch.stack([sees(c, n, m) for n, m in ((0, 3), (1, 8), (2, 5))]).any(0)
        assert torch.equal(out[:, :, 3].isnan(), seen[:, None].expand(-1, 8))
        assert torch.equal(torch.where(out.isnan(), clean, out), clean)
        for s, x in zip(spots, was):
            c.v[s] = x
        other.run(workspace=ws)
        call()
        assert torch.equal(out, clean)
    ok()


def test_sequences_beside_refused_ones():
    def values(c, rows, skip):
        out, lse = c.run()
        torch.cuda.synchronize()
        assert P.pkv_get_device_error() == QLEN
        ref = c.want(skip)
        for r in rows:
            c.check((out, lse), ref, r)
        return out, lse

    seqs = [(40, 10), (30, 6), (700, 7)]
    c = Case(16, seqs)
    c.cu[3] = 60                                              # past the rows of q
    out, lse = values(c, [slice(0, 16)], (2,))
    assert (out[16:] == 9).all() and (lse[16:] == 9).all()
    # offsets that fall: the first sequence's tree of 17 nodes, the second's of -1, and one row
    # that the first and the third both write
    c = Case(16, seqs)
    c.masks = torch.nn.functional.pad(c.masks, (0, 22))
    c.cu[1] = 17
    values(c, [slice(0, 16), slice(17, 23)], (1,))


@pytest.mark.parametrize("masks", ["tree", "random"])
@pytest.mark.parametrize("kw", [dict(d=256), dict(d=256, dtype="f16", hq=25, hkv=5, bs=64), dict(d=256, hq=64, hkv=8),
                                dict(d=128, hkv=5, hq=15), dict(d=128, dtype="f16", hq=32, bs=32), dict(d=64, hq=32),
                                dict(kv="head", d=256), dict(kv="block", hq=32)])
def test_segments_of_few_tiles(kw, masks):
    # tails of trees a tile or two behind one another, in ring stages that the tiles before have
    # just left or not yet reached: what lies behind a context, and nodes that nobody sees, are NaN
    rng = np.random.default_rng(70)
    for seed in range(6):
        seqs = [(int(rng.choice([0, 1, 15, 63, 64, 127, 128, 129, 500])), int(rng.integers(1, 66)))
                for _ in range(int(rng.integers(5, 60)))]
        c = Case(70 + seed, seqs, masks=masks, pad=seed % 2, qsize=float(2.0 ** rng.integers(-3, 3)), **kw)
        got = c.run()
        ok()
        c.check(got)

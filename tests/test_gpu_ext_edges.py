"""paged_attn_decode_ext, paged_attn_prefill_chunk_ext and the step that composes them where a
row's keys are NaN, where calls of other sizes share a workspace, and at bounds of the arguments."""
import pytest
import torch

import paged_kv_decode_11_gb300 as P
from tests import ext_ref as R
from tests.test_gpu_attn_ext import Case, ok

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from paged_kv_decode_11_gb300 import build
    build.build()
    P.load()
    torch.cuda.init()
    P.pkv_get_device_error()


def nan_blocks(c, n, first, which, head=1):
    """NaN scales for one KV head on the blocks of sequence n from number `first` on."""
    ids = c.tables[n].tolist()                  # (blocks before a window have no entry)
    blocks = [b for b in ids if 0 <= b < c.k.shape[0]][first:]
    getattr(c, which)[blocks, head] = 255


# (cached, new tokens) and the first position whose blocks are NaN: a row that sees nothing
# else (the only block; the whole context), the page behind a border between key tiles (of 128
# keys, 64 at head_dim 256), the last tiles of a long context whose tiles a cluster's CTAs share
NAN_PLACES = [([(0, 20)], 0), ([(5, 11)], 0), ([(0, 130)], 128), ([(127, 3)], 128), ([(60, 6)], 64),
              ([(0, 400)], 384), ([(4090, 7)], 0), ([(4090, 7)], 3840), ([(4090, 7)], 2048),
              ([(4090, 7)], 4096)]


@pytest.mark.parametrize("kw", [dict(), dict(softcap=9.0, alibi=True), dict(d=64), dict(d=256),
                                dict(dtype="f16", bs=64)])
@pytest.mark.parametrize("which", ["ks", "vs"])
@pytest.mark.parametrize("seqs,at", NAN_PLACES)
def test_prefill_nan_scales_are_all_a_share_sees(seqs, at, which, kw):
    # as many copies of the sequence as make clusters of eight, four, two and one CTA per tile
    for copies in (1, 12, 24, 60) if sum(seqs[0]) > 4000 else (1,):
        c = Case(200, seqs * copies, **kw)
        ref = c.want()
        p, q = seqs[0]
        bs = c.k.shape[2]
        for n in {0, copies - 1}:
            nan_blocks(c, n, at // bs, which)
        out, lse = c.prefill()
        ok()
        sees = torch.arange(p, p + q).cuda() >= at // bs * bs
        tol = R.tolerance(ref, c.q.dtype, c.p_dtype, c.softcap)
        near = (out.double() - ref.out).abs() <= tol
        lse_near = (lse.double() - ref.lse).abs() <= R.lse_tolerance(ref, c.softcap)
        for n in range(copies):
            rows = slice(n * q, (n + 1) * q)
            bad = torch.zeros(q, c.q.shape[1], dtype=torch.bool, device="cuda")
            if n in (0, copies - 1):
                bad[sees, 4:] = True
            assert out[rows][bad].isnan().all()
            assert near[rows][~bad].all() and lse_near[rows][~bad].all()
            if which == "ks":
                assert lse[rows][bad].isnan().all()


@pytest.mark.parametrize("kw", [dict(), dict(softcap=9.0, alibi=True), dict(d=64), dict(d=256),
                                dict(dtype="f16", window=600)])
@pytest.mark.parametrize("seqs,at", NAN_PLACES)
def test_prefill_nan_v_scales_leave_lse_alone(seqs, at, kw):
    # lse is a sum over scores, in which V has no part
    many = (1, 12) if "window" in kw else (1, 12, 24, 60)
    for copies in many if sum(seqs[0]) > 4000 else (1,):
        c = Case(204, seqs * copies, **kw)
        ref = c.want()
        for n in {0, copies - 1}:
            nan_blocks(c, n, 0 if c.window else at // c.k.shape[2], "vs")
        out, lse = c.prefill()
        ok()
        assert out[0 if c.window else -1, 4:].isnan().all()
        assert ((lse.double() - ref.lse).abs() <= R.lse_tolerance(ref, c.softcap)).all()


@pytest.mark.parametrize("kw", [
    dict(), dict(dtype="f16", softcap=9.0), dict(d=64, alibi=True), dict(d=256),
    dict(kv="head", softcap=9.0), dict(kv="head", d=256, dtype="f16", window=20),
    dict(kv="same", spread=1, softcap=9.0), dict(kv="same", spread=1, alibi=True, dtype="f16", d=64),
    dict(kv="same", spread=1, d=256), dict(kv="same", spread=1, window=30, prefix=[3, 700, 0])])
def test_prefill_nan_query_rows_stay_nan(kw):
    c = Case(201, [(10, 5), (0, 300), (3000, 4)], **kw)
    ref = c.want()
    at = [(2, 0), (7, 5), (100, 3), (304, 7), (306, 4)]
    for row, head in at:
        c.q[row, head, row % 64] = float("nan")
    out, lse = c.prefill()
    ok()
    bad = torch.zeros(c.q.shape[:2], dtype=torch.bool, device="cuda")
    for row, head in at:
        bad[row, head] = True
    assert out[bad].isnan().all() and lse[bad].isnan().all()
    tol = R.tolerance(ref, c.q.dtype, c.p_dtype, c.softcap)
    assert ((out.double() - ref.out).abs() <= tol)[~bad].all()
    assert ((lse.double() - ref.lse).abs() <= R.lse_tolerance(ref, c.softcap))[~bad].all()


@pytest.mark.parametrize("part", [0, 16, 512])
@pytest.mark.parametrize("kw", [dict(), dict(softcap=9.0, alibi=True), dict(d=64, window=900),
                                dict(d=256, bs=32), dict(softcap=300.0)])
@pytest.mark.parametrize("which", ["ks", "vs"])
def test_decode_nan_scales_and_their_lse(which, kw, part):
    # the NaN blocks: the whole context, the last page alone (one warp's, or one partition's), the
    # later half. A NaN K scale makes scores NaN, so out and lse; a NaN V scale out alone
    lens, first = [5, 16, 33, 700, 2500, 2500, 2500], [0, 0, 32, 688, 0, 2496, 1300]
    c = Case(202, [(n - 1, 1) for n in lens + [300]], **kw)
    ref = c.want()
    for n, at in enumerate(first):
        nan_blocks(c, n, 0 if c.window else at // c.k.shape[2], which)
    out, lse = c.decode(part)
    ok()
    bad = torch.zeros(c.q.shape[:2], dtype=torch.bool, device="cuda")
    bad[:len(lens), 4:] = True
    assert out[bad].isnan().all()
    tol = R.tolerance(ref, c.q.dtype, c.p_dtype, c.softcap)
    assert ((out.double() - ref.out).abs() <= tol)[~bad].all()
    near = (lse.double() - ref.lse).abs() <= R.lse_tolerance(ref, c.softcap)
    assert near[~bad].all()
    assert lse[bad].isnan().all() if which == "ks" else near.all()


@pytest.mark.parametrize("part", [0, 16])
@pytest.mark.parametrize("kw", [
    dict(dtype="f16", softcap=9.0), dict(kv="head", d=256, dtype="f16", window=20),
    dict(kv="same", spread=1, softcap=9.0), dict(kv="same", spread=1, alibi=True, dtype="f16", d=64),
    dict(kv="same", spread=1, d=256), dict(hq=2), dict(kv="head", hq=2, softcap=400.0)])
def test_decode_nan_query_rows_stay_nan(kw, part):
    # (over an E4M3 cache a KV head's bf16 queries share a power of two: one of a group alone)
    c = Case(203, [(n - 1, 1) for n in (1, 40, 700, 3000)], **kw)
    ref = c.want()
    bad = torch.zeros(c.q.shape[:2], dtype=torch.bool, device="cuda")
    bad[0, 0] = bad[2, 1] = bad[3, c.q.shape[1] - 1] = True
    c.q[..., 3].masked_fill_(bad, float("nan"))
    out, lse = c.decode(part)
    ok()
    assert out[bad].isnan().all() and lse[bad].isnan().all()
    tol = R.tolerance(ref, c.q.dtype, c.p_dtype, c.softcap)
    assert ((out.double() - ref.out).abs() <= tol)[~bad].all()
    assert ((lse.double() - ref.lse).abs() <= R.lse_tolerance(ref, c.softcap))[~bad].all()


@pytest.mark.parametrize("cap", [300.0, 1e4, 1e6, 1e30])
@pytest.mark.parametrize("kw", [dict(kv="same", spread=1), dict(kv="same", spread=1, d=256),
                                dict(kv="same", spread=1, d=64, window=90), dict()])
def test_a_score_below_minus_the_cap_leaves_the_others_alone(cap, kw):
    # Keys whose scores lie far below -cap weigh nothing (e^-cap at most), so the bound is that of
    # the other keys: nothing in it grows with the cap, or with those scores
    seqs = [(40, 60), (0, 100), (300, 1)]
    c = Case(205, seqs, softcap=cap, **kw)
    c.q[..., 0] = 8.0
    c.k[..., 0] = 0
    size = c.want().size
    big = 2.0 ** torch.tensor(3 * cap / (8 * c.scale)).log2().ceil().item()   # a score of -3 cap or below
    bs = c.k.shape[2]
    for n, (p, q) in enumerate(seqs):
        j = max(0, p + q - 30) // bs * bs                   # within every row's window, if it sees it
        block = int(c.tables[n, j // bs])
        if c.ks is not None:
            c.k[block] = 0
            c.k[block, ..., 0] = -1
            c.ks[block] = 127 + int(torch.tensor(big).log2().item())
        else:
            c.k[block, :, 3, 0] = -big
    ref = c.want()
    # rows that see nothing else (the first of an empty context may) are no test of this
    rows = ref.lse.min(1).values > -cap / 2
    assert rows.sum() > 100
    ref.size = size
    for out, lse in (c.prefill(),):
        ok()
        assert ((out.double() - ref.out).abs() <= R.tolerance(ref, c.q.dtype, c.p_dtype))[rows].all()
        assert ((lse.double() - ref.lse).abs() <= R.lse_tolerance(ref))[rows].all()


def test_calls_of_other_sizes_share_a_workspace_in_turn():
    # a buffer made for the largest call serves all of them, whichever ran before: the
    # partial results of one lie where another has its counters
    shapes = [dict(lens=[5000], hq=32, hkv=8), dict(lens=[2100] * 128, hq=8, hkv=1),
              dict(lens=[4000, 300, 2000], hq=8, hkv=2, d=64), dict(lens=[6000, 10], hq=16, hkv=2, d=256),
              dict(lens=[2100] * 40, hq=8, hkv=2, kv="same", spread=1, alibi=True),
              dict(lens=[700], hq=32, hkv=8, window=500)]
    cases = []
    for i, kw in enumerate(shapes):
        kw = dict(kw)
        cases.append(Case(210 + i, [(n - 1, 1) for n in kw.pop("lens")], **kw))
    size = max(P.paged_attn_decode_ext_workspace_size(len(c.seq_lens), c.q.shape[1], c.k.shape[1],
                                                      c.q.shape[2], c.max_ctx, c.window, part)
               for c in cases for part in (0, 64))
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    want = [[c.decode(part) for part in (0, 64)] for c in cases]
    for c, w in zip(cases, want):
        for got in w:
            c.check(got)
    ok()
    for order in ([0, 1, 0, 2, 1, 3, 4, 5, 1], [5, 4, 1, 3, 2, 0, 1, 1, 0]):
        for i in order:
            for part, w in zip((0, 64), want[i]):
                got = cases[i].decode(part, workspace=ws)
                assert torch.equal(got[0], w[0]) and torch.equal(got[1], w[1])
    ok()


def test_graphs_of_other_sizes_share_a_workspace():
    a = Case(220, [(6000, 1)], hq=32, hkv=8)
    b = Case(221, [(2500, 1)] * 100, hq=4, hkv=1)
    size = max(P.paged_attn_decode_ext_workspace_size(len(c.seq_lens), c.q.shape[1], c.k.shape[1],
                                                      128, c.max_ctx) for c in (a, b))
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    want, graphs = [c.decode() for c in (a, b)], []
    outs = [torch.zeros_like(c.q) for c in (a, b)]
    for c, out in zip((a, b), outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            P.paged_attn_decode_ext(out, c.q, c.k, c.v, c.tables, c.seq_lens, c.scale, c.max_ctx,
                                    c.ks, c.vs, workspace=ws)
        graphs.append(g)
    for _ in range(4):
        for i in (0, 1, 1, 0):
            outs[i].zero_()
            graphs[i].replay()
            assert torch.equal(outs[i], want[i][0])
    ok()


def test_a_workspace_for_a_large_batch_serves_the_smaller_ones():
    ws = torch.zeros(P.paged_attn_decode_ext_workspace_size(64, 16, 2, 128, 3000), dtype=torch.uint8,
                     device="cuda")
    for n in (64, 50, 33, 8, 5, 2, 1):
        c = Case(230 + n, [(2999, 1)] * n, hq=16, hkv=2)
        c.check(c.decode(workspace=ws))
    ok()


@pytest.mark.parametrize("kw", [dict(hq=16, hkv=1), dict(hq=8, hkv=1, d=256), dict(hq=7, hkv=1, d=64)])
def test_merges_of_many_chunks_repeat_themselves(kw):
    # hundreds of partitions: the merging CTA refills one staging space many times, right behind
    # its own use of it
    c = Case(240, [(5999, 1), (4000, 1), (777, 1)], **kw)
    first = c.decode(16)
    c.check(first)
    for _ in range(50):
        again = c.decode(16)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    ok()


@pytest.mark.parametrize("kw", [dict(), dict(kv="same", spread=1, softcap=9.0), dict(kv="head", window=9)])
def test_prefill_without_a_bound_flags_every_chunk(kw):
    c = Case(250, [(50, 10), (300, 0), (0, 3)], **kw)
    out, lse = c.prefill(max_q_len=0)
    torch.cuda.synchronize()
    assert P.pkv_get_device_error() == 0x10         # PKV_DEVERR_QLEN
    assert (out == 9).all() and (lse == 9).all()
    c = Case(251, [(50, 0), (0, 0)], pad=4, **kw)    # rows, but no chunk has one
    out, _ = c.prefill(max_q_len=0)
    ok()
    assert (out == 9).all()


@pytest.mark.parametrize("handle", [lambda s: s, lambda s: s.cuda_stream, lambda s: 0, lambda s: None])
def test_a_workspace_of_the_calls_own_lives_on_its_stream(handle, monkeypatch):
    # without a workspace argument: filled, and given back, in the order of the stream that the call
    # runs on, whichever stream is current
    c = Case(260, [(5000, 1), (800, 1)])
    old = Case(261, [(5000, 1), (800, 1)], kv="same", spread=1)
    key, slots = torch.randn(2, 2, 128, device="cuda").bfloat16(), torch.full((2,), -1, device="cuda")
    qsl = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    want = {s: s, 0: torch.cuda.default_stream()}.get(handle(s), s)
    if handle(s) is None:
        want = torch.cuda.current_stream()
    seen, zeros = [], torch.zeros

    def watched(*a, **kw):
        seen.append(torch.cuda.current_stream().cuda_stream)
        return zeros(*a, **kw)
    out = torch.empty_like(c.q)
    args = (old.q, old.k, old.v, old.tables, old.seq_lens)
    olds = [torch.empty_like(old.q) for _ in range(3)]
    ref, plain = c.decode(), old.decode()
    torch.cuda.synchronize()
    monkeypatch.setattr(torch, "zeros", watched)
    P.paged_attn_decode_ext(out, c.q, c.k, c.v, c.tables, c.seq_lens, c.scale, c.max_ctx, c.ks, c.vs,
                            stream=handle(s))
    P.paged_attn_decode(olds[0], *args, old.scale, old.max_ctx, stream=handle(s))
    P.paged_attn_decode_step(key, key, slots, olds[1], *args, old.scale, old.max_ctx, stream=handle(s))
    P.paged_attn_varlen(olds[2], *args, qsl, 2, old.scale, 0, old.max_ctx, stream=handle(s))
    junk = [torch.full((1 << 20,), 1.5, device="cuda") for _ in range(50)]     # the current stream's memory
    ok()
    assert seen == [want.cuda_stream] * 4 and len(junk) == 50
    assert torch.equal(out, ref[0])
    tol = R.tolerance(old.want(), old.q.dtype, old.p_dtype)
    for x in olds:
        assert ((x.double() - plain[0].double()).abs() <= 2 * tol).all()

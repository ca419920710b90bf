"""The append and the attentions over block scales together, as a step uses them: conversations
that grow token by token and chunk by chunk, eagerly, from captured graphs, and beside each
other on two streams; against the definitions in 64 bits."""
import numpy as np
import pytest
import torch

import paged_kv_decode_11_gb300 as P
from paged_kv_decode_11_gb300.step import BlockScaledStep
from tests import ext_ref as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from paged_kv_decode_11_gb300 import build
    build.build()
    P.load()
    torch.cuda.init()
    P.pkv_get_device_error()


def table(max_pos, rot=128):
    inv = 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) / (rot // 2))
    a = torch.arange(max_pos, dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float().cuda()


class Batch:
    """Caches, tables and growing sequences; the reference caches beside them."""

    def __init__(self, seed, start, room, hq=8, hkv=2, d=128, bs=16):
        self.g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.hq, self.hkv, self.d, self.bs = hq, hkv, d, bs
        per = -(-room // bs)
        nb = per * len(start) + 3
        self.tables = torch.from_numpy(rng.permutation(nb)[:per * len(start)].astype(np.int32)
                                       ).view(len(start), per).cuda()
        shape = (nb, hkv, bs, d)
        nan = torch.full(shape, float("nan")).to(torch.float8_e4m3fn)     # fresh blocks: anything
        self.k, self.v = nan.clone().cuda(), nan.clone().cuda()
        self.ks, self.vs = (torch.zeros(nb, hkv, dtype=torch.uint8).cuda() for _ in range(2))
        self.ref = [x.clone() for x in (self.k, self.v, self.ks, self.vs)]
        self.lens = [0] * len(start)
        self.cos_sin = table(room)
        self.opts = dict(softcap=0.0, window=0, slopes=None)

    def tokens(self, n):
        r = lambda h, s: (torch.randn(n, h, self.d, generator=self.g) * s).bfloat16().cuda()  # noqa: E731
        size = float(2.0 ** torch.randint(-2, 3, (1,), generator=self.g))
        return r(self.hq, 1.0), r(self.hkv, size), r(self.hkv, size)

    def step(self, new, num_decode, stream=None, **opts):
        """new: tokens that each sequence gets."""
        q, k, v = self.tokens(sum(new))
        self.lens = [a + b for a, b in zip(self.lens, new)]
        lens = torch.tensor(self.lens, dtype=torch.int32).cuda()
        cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32).cuda()
        s = BlockScaledStep(self.k, self.v, self.ks, self.vs, q, k, v, self.tables, lens, cu,
                            num_decode, self.d ** -0.5, max(self.lens), max(new),
                            cos_sin=self.cos_sin, **opts)
        return s

    def expect(self, s):
        """Append to the reference caches, then attention over them."""
        k, v, ks, vs, q = R.append(s.new_k, s.new_v, *self.ref, self.tables, s.seq_lens,
                                   s.cu_q_lens, s.q, self.cos_sin)
        to8 = lambda x: x.float().to(torch.float8_e4m3fn)                 # noqa: E731
        self.ref = [to8(k), to8(v), ks.to(torch.uint8), vs.to(torch.uint8)]
        return R.attention(q, *self.ref[:2], self.tables, s.seq_lens, s.cu_q_lens, s.scale,
                           *self.ref[2:], s.opts["softcap"], s.opts["window"],
                           s.opts["alibi_slopes"])

    def check(self, s, ref):
        assert P.pkv_get_device_error() == 0
        for a, b in zip((self.k, self.v, self.ks, self.vs), self.ref):
            a, b = a.view(b.dtype).float(), b.float()
            assert torch.equal(a.nan_to_num(500), b.nan_to_num(500))
        tol = R.tolerance(ref, s.q.dtype, torch.float16, s.opts["softcap"])
        assert ((s.out.double() - ref.out).abs() <= tol).all()


@pytest.mark.parametrize("opts", [{}, dict(softcap=20.0, window=50),
                                  dict(alibi=True)])
def test_conversations_grow(opts):
    b = Batch(1, [0] * 5, 400)
    opts = dict(opts)
    if opts.pop("alibi", False):
        opts["alibi_slopes"] = torch.exp2(-torch.arange(1, 9).float()).cuda()
    for new, nd in (([40, 1, 17, 100, 16], 0), ([1, 1, 1, 1, 1], 5), ([1, 1, 30, 5, 64], 2),
                    ([1, 1, 1, 0, 200], 3), ([1, 1, 1, 1, 1], 5), ([1, 1, 1, 1, 1], 5)):
        s = b.step(new, nd, **opts)
        s.run()
        b.check(s, b.expect(s))


def test_captured_decode_steps_replay():
    # one graph replayed as the sequences grow across block borders, its inputs copied in
    b = Batch(2, [0] * 4, 300)
    s = b.step([30, 15, 16, 100], 0)
    s.run()
    b.check(s, b.expect(s))
    s = b.step([1, 1, 1, 1], 4)
    s.max_seq_len = 160
    ws = P.paged_attn_decode_ext_workspace_size(4, 8, 2, 128, 160)
    s.workspace = torch.zeros(ws, dtype=torch.uint8, device="cuda")
    s.run()                                      # warm, and the first of the steps
    b.check(s, b.expect(s))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        s.run()
    for _ in range(20):
        q, k, v = b.tokens(4)
        b.lens = [x + 1 for x in b.lens]
        s.q.copy_(q), s.new_k.copy_(k), s.new_v.copy_(v)
        s.seq_lens.copy_(torch.tensor(b.lens, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        b.check(s, b.expect(s))


def test_captured_mixed_step_replays_the_same():
    b = Batch(3, [0] * 4, 600, hq=16, hkv=4)
    s = b.step([50, 200, 300, 7], 0)
    s.run()
    b.check(s, b.expect(s))
    s = b.step([1, 1, 100, 130], 2, softcap=30.0)
    s.run()
    ref = b.expect(s)
    b.check(s, ref)
    first = s.out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.run()
    for _ in range(3):                           # appending the same tokens again changes nothing
        s.out.fill_(3.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(s.out, first)
        b.check(s, ref)


def test_two_graphs_share_a_workspace_in_turn():
    b = Batch(4, [0] * 3, 3000)
    s = b.step([2000, 2500, 900], 0)
    s.run()
    b.check(s, b.expect(s))
    s = b.step([1, 1, 1], 3)
    s.run()
    ref = b.expect(s)
    b.check(s, ref)
    want = s.out.clone()
    other = BlockScaledStep(b.k, b.v, b.ks, b.vs, s.q, s.new_k, s.new_v, b.tables, s.seq_lens,
                            s.cu_q_lens, 3, s.scale, s.max_seq_len, cos_sin=b.cos_sin)
    other.workspace = s.workspace
    graphs = []
    for x in (s, other):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x.run()
        graphs.append(g)
    for _ in range(5):
        for g, x in zip(graphs, (s, other)):
            x.out.zero_()
            g.replay()
            assert torch.equal(x.out, want)
    assert P.pkv_get_device_error() == 0


def test_two_streams_with_their_own_workspaces():
    b1, b2 = Batch(5, [0] * 3, 1200), Batch(6, [0] * 2, 1200)
    steps = [b1.step([900, 1000, 70], 0), b2.step([1100, 3], 0)]
    for s in steps:
        s.run()
    for b, s in zip((b1, b2), steps):
        b.check(s, b.expect(s))
    steps = [b1.step([1, 1, 1], 3), b2.step([1, 1], 2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        for s, st in zip(steps, streams):
            s.run(stream=st)
    torch.cuda.synchronize()
    for b, s in zip((b1, b2), steps):
        b.check(s, b.expect(s))


def test_old_reader_of_a_block_scaled_cache_with_one_scale():
    # every block at one scale: the per-head calls read the same codes to the same result
    b = Batch(7, [0] * 2, 300)
    q, k, v = b.tokens(2 * 128)
    k.clamp_(-3, 3), v.clamp_(-3, 3)
    k[:, :, 0], v[:, :, 0] = 3.5, 3.5            # every block's largest element
    lens = torch.tensor([128, 128], dtype=torch.int32).cuda()
    cu = torch.tensor([0, 128, 256], dtype=torch.int32).cuda()
    P.rope_append_block_scaled(k, v, b.k, b.v, b.ks, b.vs, b.tables, lens, cu)
    used = b.tables[:, :8].flatten().long()
    assert (b.ks[used] == b.ks[used[0]]).all() and (b.vs[used] == b.vs[used[0]]).all()
    one = 2.0 ** (b.ks[used[0]].float() - 127)
    q = q[:2].contiguous()
    a, c = torch.empty_like(q), torch.empty_like(q)
    P.paged_attn_decode(a, q, b.k, b.v, b.tables, lens, 128 ** -0.5, 128, one, one)
    P.paged_attn_decode_ext(c, q, b.k, b.v, b.tables, lens, 128 ** -0.5, 128, b.ks, b.vs)
    # both round their weights to f16 against a reference of their own, and the output once
    assert ((a.double() - c.double()).abs() <= 2 * (2.0 ** -11 * 3.5 + 2.0 ** -8 * a.double().abs())).all()

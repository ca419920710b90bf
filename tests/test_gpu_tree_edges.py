"""paged_attn_tree where its softmax and its masks are at their limits, against attention in 64 bits
(tests/tree_ref.py, tolerances of tests/ext_ref.py)."""
import pytest
import torch

import paged_kv_decode_11_gb300 as P
from tests.test_gpu_tree import Case, ok

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

"""Argument checks of the block-scaled append and the _ext attentions that need
no GPU: every call returns its status before anything is launched."""
import pytest

import paged_kv_decode_11_gb300 as P
from paged_kv_decode_11_gb300 import build

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
F16, BF16, FP8, BLOCK = 0, 1, 2, 3
FAKE = 0x10000          # never dereferenced: every call below fails its checks first
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lib():
    build.build()
    return P.load()


def _decode(lib, **kw):
    a = dict(out=FAKE, q=FAKE, q_dtype=BF16, k=FAKE, v=FAKE, kv_dtype=BLOCK, bt=FAKE, sl=FAKE, B=4,
             Hq=8, Hkv=2, D=128, BS=16, maxb=8, nb=64, msl=128, scale=0.1, ks=FAKE, vs=FAKE,
             cap=0.0, win=0, slopes=None, part=0, lse=None, ws=None, wsb=0, stream=None)
    a.update(kw)
    return lib.paged_attn_decode_ext(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(D=96), UNSUPPORTED), (dict(D=256, Hq=32, Hkv=2), UNSUPPORTED), (dict(BS=8), UNSUPPORTED),
    (dict(BS=128), UNSUPPORTED), (dict(BS=24), UNSUPPORTED), (dict(Hq=34, Hkv=2), UNSUPPORTED),
    (dict(Hq=9, Hkv=2), INVALID), (dict(q_dtype=FP8), UNSUPPORTED), (dict(q_dtype=BLOCK), UNSUPPORTED),
    (dict(q_dtype=F16, kv_dtype=BF16), UNSUPPORTED), (dict(kv_dtype=4), UNSUPPORTED),
    (dict(part=24), INVALID), (dict(part=8192 + 16), INVALID), (dict(part=-16), INVALID),
    (dict(win=-1), INVALID), (dict(cap=-1.0), INVALID), (dict(cap=NAN), INVALID),
    (dict(cap=INF), INVALID), (dict(cap=3e38), INVALID), (dict(cap=1e-40), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=-0.1), INVALID), (dict(scale=NAN), INVALID),
    (dict(scale=INF), INVALID), (dict(ks=None), INVALID), (dict(vs=None), INVALID),
    (dict(kv_dtype=FP8, ks=None), INVALID), (dict(kv_dtype=BF16, ks=None, vs=None), WORKSPACE),
    (dict(out=None), INVALID), (dict(q=FAKE + 8), INVALID), (dict(k=FAKE + 4), INVALID),
    (dict(bt=None), INVALID), (dict(sl=None), INVALID), (dict(B=-1), INVALID),
    (dict(B=70000), UNSUPPORTED), (dict(nb=0), INVALID), (dict(maxb=0), INVALID),
    (dict(msl=-1), INVALID), (dict(nb=2 ** 30, BS=64), INVALID), (dict(B=0, out=None, q=None), OK),
])
def test_decode_ext_argument_checks(lib, kw, want):
    assert _decode(lib, **kw) == want


def test_decode_ext_workspace(lib):
    size = P.paged_attn_decode_ext_workspace_size
    need = size(4, 8, 2, 128, 4096, 0, 64)
    assert need == P.paged_attn_decode_workspace_size(4, 8, 2, 128, 4096, 64)
    a = dict(part=64, msl=4096)
    assert _decode(lib, **a, ws=FAKE, wsb=need - 1) == WORKSPACE
    assert _decode(lib, **a, ws=FAKE + 16, wsb=need) == WORKSPACE
    assert _decode(lib, **a, ws=None, wsb=need) == WORKSPACE
    # a window needs room for its keys and the rest of their first page alone
    assert size(4, 8, 2, 128, 4096, 100, 64) == size(4, 8, 2, 128, 115, 0, 64) < need
    assert size(4, 8, 2, 128, 100, 4096, 64) == size(4, 8, 2, 128, 100, 0, 64)
    assert size(4, 8, 2, 128, 4096, 2 ** 31 - 1, 64) == need
    assert size(4, 8, 2, 128, 4096, -1, 64) == 0
    assert size(4, 8, 2, 128, -1, 0, 64) == 0


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 8, 8), (128, 32, 8), (256, 16, 2)])
def test_decode_ext_workspace_is_that_of_the_type_with_most_parts(lib, D, Hq, Hkv):
    # the size is that of the type with the most partitions, and one byte less is refused for it
    # (calls that would pass the check are made where there are real buffers)
    for B in (1, 3, 17, 200):
        for msl in (1, 15, 700, 4096, 131072):
            for win in (0, 1, 300, 5000):
                need = P.paged_attn_decode_ext_workspace_size(B, Hq, Hkv, D, msl, win)
                span = min(msl, win + 15) if win else msl
                # room for the output rows of every partition, at least 64 keys each
                assert need >= B * Hkv * 8 + B * Hq * (4 * D + 4)
                assert need <= 768 + B * Hkv * 8 + B * Hq * (4 * D + 4) * (span // 64 + 1)
                a = dict(B=B, Hq=Hq, Hkv=Hkv, D=D, msl=msl, win=win, ws=FAKE)
                for kv in (BF16, FP8, BLOCK):
                    assert _decode(lib, **a, kv_dtype=kv, wsb=255) == WORKSPACE
                assert _decode(lib, **a, kv_dtype=BLOCK, wsb=need - 1) == WORKSPACE
                assert _decode(lib, **a, kv_dtype=FP8, wsb=need - 1) == WORKSPACE


def _prefill(lib, **kw):
    a = dict(out=FAKE, q=FAKE, q_dtype=BF16, k=FAKE, v=FAKE, kv_dtype=BLOCK, bt=FAKE, sl=FAKE,
             cu=FAKE, n=1, T=10, maxq=10, Hq=8, Hkv=2, D=128, BS=16, maxb=8, nb=64, scale=0.1,
             ks=FAKE, vs=FAKE, cap=0.0, win=0, slopes=None, prefix=None, lse=None, stream=None)
    a.update(kw)
    return lib.paged_attn_prefill_chunk_ext(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(D=320), UNSUPPORTED), (dict(cu=None), INVALID), (dict(ks=None), INVALID),
    (dict(BS=8), UNSUPPORTED), (dict(Hq=7, Hkv=2), INVALID), (dict(scale=0.0), INVALID),
    (dict(cap=-2.0), INVALID), (dict(win=-5), INVALID), (dict(T=-1), INVALID),
    (dict(maxq=-1), INVALID), (dict(q=FAKE + 2), INVALID), (dict(v=None), INVALID),
    (dict(kv_dtype=7), UNSUPPORTED), (dict(T=0, out=None), OK), (dict(n=0, out=None), OK),
    (dict(maxq=0, out=None), OK),
])
def test_prefill_ext_argument_checks(lib, kw, want):
    assert _prefill(lib, **kw) == want


def _append(lib, **kw):
    a = dict(key=FAKE, value=FAKE, src=BF16, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, bt=FAKE, sl=FAKE,
             cu=FAKE, n=2, T=4, qo=FAKE, q=FAKE, cs=FAKE, maxpos=4096, rot=128, neox=1, Hq=8,
             Hkv=2, D=128, BS=16, maxb=8, nb=64, stream=None)
    a.update(kw)
    return lib.rope_append_block_scaled(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(src=FP8), UNSUPPORTED), (dict(src=BLOCK), UNSUPPORTED), (dict(D=80), UNSUPPORTED),
    (dict(BS=8), UNSUPPORTED), (dict(rot=0), INVALID), (dict(rot=24), INVALID),
    (dict(rot=144), INVALID), (dict(maxpos=0), INVALID), (dict(q=None), INVALID),
    (dict(qo=None), INVALID), (dict(cs=FAKE + 4), INVALID), (dict(qo=FAKE + 8), INVALID),
    (dict(Hq=0), INVALID), (dict(key=None), INVALID), (dict(value=FAKE + 2), INVALID),
    (dict(ks=None), INVALID), (dict(vs=None), INVALID), (dict(bt=None), INVALID),
    (dict(sl=None), INVALID), (dict(cu=None), INVALID), (dict(kc=FAKE + 8), INVALID),
    (dict(T=-1), INVALID), (dict(n=-1), INVALID), (dict(nb=0), INVALID), (dict(maxb=0), INVALID),
    (dict(nb=2 ** 30, BS=64), INVALID), (dict(T=0, key=None), OK), (dict(n=0, key=None), OK),
])
def test_append_argument_checks(lib, kw, want):
    assert _append(lib, **kw) == want


def test_old_calls_refuse_block_scales(lib):
    assert lib.paged_attn_decode(FAKE, FAKE, BF16, FAKE, FAKE, BLOCK, FAKE, FAKE, 4, 8, 2, 128, 16, 8,
                                 64, 128, 0.1, FAKE, FAKE, 0, None, FAKE, 1 << 30, None) == UNSUPPORTED
    assert lib.reshape_and_cache(FAKE, FAKE, BF16, FAKE, FAKE, BLOCK, FAKE, 4, 2, 128, 16, 8, FAKE,
                                 FAKE, None) == UNSUPPORTED


def test_native_refuses_host_tensors(lib):
    import torch
    q = torch.zeros(1, 8, 128, dtype=torch.bfloat16)
    c = torch.zeros(2, 2, 16, 128, dtype=torch.uint8)
    s = torch.zeros(2, 2, dtype=torch.uint8)
    t, n = torch.zeros(1, 1, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    cu = torch.tensor([0, 1], dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        P.paged_attn_decode_ext(q, q, c, c, t, n, 0.1, 16, s, s, workspace=s)
    with pytest.raises(ValueError, match="CUDA"):
        P.paged_attn_prefill_chunk_ext(q, q, c, c, t, n, cu, 0.1, 1, s, s)
    with pytest.raises(ValueError, match="CUDA"):
        P.rope_append_block_scaled(q[:, :2], q[:, :2], c, c, s, s, t, n, cu)
    with pytest.raises(ValueError, match="dimensions"):
        P.paged_attn_prefill_chunk_ext(q, q[0], c, c, t, n, cu, 0.1, 1, s, s)
    with pytest.raises(ValueError, match="tensor"):
        P.paged_attn_prefill_chunk_ext(q, 5, c, c, t, n, cu, 0.1, 1, s, s)

"""Host side of the block-scaled append, the _ext attentions and their step; needs no GPU."""
import pytest

import paged_kv_decode_11_gb300 as P
from paged_kv_decode_11_gb300 import build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return P.load()


@pytest.mark.parametrize("Hq,Hkv,D", [(32, 8, 128), (8, 8, 64), (16, 2, 256), (28, 4, 128)])
@pytest.mark.parametrize("part", [0, 16, 512])
def test_a_larger_call_has_a_larger_workspace(lib, Hq, Hkv, D, part):
    size = P.paged_attn_decode_ext_workspace_size
    batches, lens = (1, 2, 3, 7, 8, 16, 17, 40, 128, 300), (1, 64, 65, 300, 700, 1000, 4096, 8192, 131072)
    table = [[size(b, Hq, Hkv, D, n, 0, part) for n in lens] for b in batches]
    for row in table:
        assert row == sorted(row)
    for col in zip(*table):
        assert list(col) == sorted(col)
    for b in batches:
        windows = [size(b, Hq, Hkv, D, 8192, w, part) for w in (1, 50, 51, 700, 5000, 8192, 0)]
        assert windows == sorted(windows)


def test_a_step_with_chunks_needs_their_bound():
    import torch
    from paged_kv_decode_11_gb300.step import BlockScaledStep
    c = torch.zeros(4, 2, 16, 128, dtype=torch.uint8)
    s, q, kv = torch.zeros(4, 2, dtype=torch.uint8), torch.zeros(6, 8, 128), torch.zeros(6, 2, 128)
    t, lens = torch.zeros(2, 2, dtype=torch.int32), torch.tensor([9, 5], dtype=torch.int32)
    cu = torch.tensor([0, 1, 6], dtype=torch.int32)
    for bound in ({}, dict(max_q_len=0), dict(max_q_len=-1)):
        with pytest.raises(ValueError, match="max_q_len"):
            BlockScaledStep(c, c, s, s, q, kv, kv, t, lens, cu, 1, 0.1, 32, **bound)
    BlockScaledStep(c, c, s, s, q, kv, kv, t, lens, cu, 1, 0.1, 32, max_q_len=5)
    BlockScaledStep(c, c, s, s, q[:2], kv[:2], kv[:2], t, lens, cu, 2, 0.1, 32)


def _elsewhere(tmp_path, code, without_native):
    """Runs code where a copy of the built package lies, with or without its _native module."""
    import os
    import shutil
    import subprocess
    import sys
    src = os.path.dirname(os.path.abspath(build.__file__))
    shutil.copytree(src, tmp_path / "paged_kv_decode_11_gb300", ignore=shutil.ignore_patterns(
        "csrc", "_build", "__pycache__", *(["_native.so"] if without_native else [])))
    r = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    return r.stdout.split("\n")


OLD_CALLS = """
import paged_kv_decode_11_gb300 as P
from paged_kv_decode_11_gb300 import _binding
{before}
L = P.load()
print(P.pkv_status_string(3), P.paged_attn_decode_workspace_size(4, 8, 2, 128, 128, 64),
      P.paged_attn_decode_ext_workspace_size(4, 8, 2, 128, 128, 0, 64))
try:
    P.rope_append_block_scaled(*[None] * 9)
except RuntimeError as e:
    print(e, e.__cause__)
"""


def test_old_calls_need_no_native_module(lib, tmp_path):
    size = P.paged_attn_decode_workspace_size(4, 8, 2, 128, 128, 64)
    out = _elsewhere(tmp_path, OLD_CALLS.format(before=""), True)
    assert str(size) in out[0] and "build.build()" in out[1]


def test_a_native_module_for_another_torch_is_not_used(lib, tmp_path):
    before = "_binding.native_target = lambda: 'torch 0.1, Python 3.0, other'"
    out = _elsewhere(tmp_path, OLD_CALLS.format(before=before), False)
    assert str(P.paged_attn_decode_workspace_size(4, 8, 2, 128, 128, 64)) in out[0]
    assert "built for " + build.native_target() in out[1] and "torch 0.1" in out[1]


def test_a_native_module_that_names_no_torch_is_not_used(lib, tmp_path):
    before = ("import sys, types\nP._native = types.ModuleType('_native')\n"
              "sys.modules['paged_kv_decode_11_gb300._native'] = P._native")
    out = _elsewhere(tmp_path, OLD_CALLS.format(before=before), True)
    assert str(P.paged_attn_decode_workspace_size(4, 8, 2, 128, 128, 64)) in out[0]
    assert "older version" in out[1]


def test_build_sees_that_torch_changed(lib, monkeypatch):
    assert build.up_to_date()
    monkeypatch.setattr(build, "native_target", lambda: "torch 0.1, Python 3.0, other")
    assert build.lib_up_to_date() and not build.native_up_to_date() and not build.up_to_date()


@pytest.mark.parametrize("part", [0, 512])
def test_bounds_above_the_longest_table(lib, part):
    # a row of a block table holds less than 2^30 tokens: a larger bound plans for no more, and the
    # 32-bit sums behind it do not wrap
    size = P.paged_attn_decode_ext_workspace_size
    top = size(1, 8, 2, 128, 2 ** 30, 0, part)
    parts = 2 ** 30 // (part or 2048)
    assert top >= parts * 8 * (4 * 128 + 4)
    for n in (2 ** 30 + 1, 2 ** 31 - 1000, 2 ** 31 - 1):
        assert size(1, 8, 2, 128, n, 0, part) == size(1, 8, 2, 128, n, n, part) == top

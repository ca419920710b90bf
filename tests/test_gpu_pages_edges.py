"""Paths, blocks and tables that are only partly there: entries that name no block, tokens that
cannot move, blocks that several rows share. Expectations by hand, or tests/tree_ref.py's walk of
what is left of the call."""
import ctypes

import pytest
import torch

import paged_kv_decode_11_gb300 as P
from tests.test_gpu_pages import i32, ok

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from paged_kv_decode_11_gb300 import build
    build.build()
    P.load()
    torch.cuda.init()
    P.pkv_get_device_error()


@pytest.mark.parametrize("kv", [1, 3])                        # bf16; E4M3 with block scales
def test_lengths_of_a_path_in_no_layer(kv):
    lib = P.load()
    tables, seq_lens, cu = i32([[0, 1], [2, -1]]), i32([20, 9]), i32([0, 6, 9])
    paths, path_lens, new = i32([[0, 3], [1, 1]]), i32([2, 0]), i32([-5, -5])
    stream = torch.cuda.current_stream().cuda_stream
    st = lib.kv_keep_path(None, None, kv, None, None, 0, tables.data_ptr(), seq_lens.data_ptr(), cu.data_ptr(),
                          paths.data_ptr(), path_lens.data_ptr(), 2, new.data_ptr(), 2, 2, 128, 16, 2, 4,
                          ctypes.c_void_p(stream))
    assert st == 0
    ok()
    assert new.tolist() == [16, 6]

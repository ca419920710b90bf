"""Paths, blocks and tables that are only partly there: entries that name no block, tokens that
cannot move, blocks that several rows share. Expectations by hand, or tests/tree_ref.py's walk of
what is left of the call."""
import ctypes

import pytest
import torch

import paged_kv_decode_11_gb300 as P
from tests.test_gpu_pages import BLOCK_ID, POOL, Keep, i32, ok

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from paged_kv_decode_11_gb300 import build
    build.build()
    P.load()
    torch.cuda.init()
    P.pkv_get_device_error()


def flagged():
    torch.cuda.synchronize()
    return P.pkv_get_device_error()


def fork(tables, lens, parents, refs, bs=16):
    tables, lens, refs = i32(tables), i32(lens), i32(refs)
    new, new_lens = torch.full_like(tables, 77), torch.full_like(lens, 77)
    copies = torch.full((len(parents), 2), 77, dtype=torch.int32, device="cuda")
    P.kv_fork_blocks(new, new_lens, tables, lens, i32(parents), refs, copies, bs)
    bits = flagged()
    return new.tolist(), new_lens.tolist(), refs.tolist(), copies.tolist(), bits


def test_fork_of_a_row_that_lacks_its_last_block():
    # the pool ran out when the row grew: its descendants lack the block too, and nothing is copied
    tables, lens, refs = i32([[2, 0, -1, -1], [1, 3, -1, -1]]), [32, 20], i32([1, 1, 1, 1, 0])
    P.kv_resize_blocks(tables, i32(lens), i32([33, 49]), refs, 16)
    assert flagged() == POOL and tables.tolist() == [[2, 0, 4, -1], [1, 3, -1, -1]]
    P.kv_resize_blocks(tables, i32([33, 49]), i32([0, 49]), refs, 16)
    ok()
    new, lens, refs, copies, bits = fork(tables.tolist(), [0, 49], [1, 1], refs.tolist())
    assert bits == 0 and lens == [49, 49]
    assert new == [[1, 3, -1, -1]] * 2 and refs == [0, 2, 0, 2, 0]
    assert copies == [[-1, -1]] * 2
    # one that has its block is copied beside it
    new, _, refs, copies, bits = fork([[1, 3, -1, -1], [2, 4, -1, -1], [-1] * 4, [-1] * 4],
                                      [49, 20, 0, 0], [0, 1, 0, 1], [0, 1, 1, 1, 1, 0])
    assert bits == 0 and refs == [1, 2, 2, 2, 1, 0]
    assert new == [[1, 3, -1, -1], [2, 4, -1, -1], [1, 3, -1, -1], [2, 0, -1, -1]]
    assert copies == [[-1, -1], [-1, -1], [-1, -1], [4, 0]]


def test_fork_of_a_row_whose_last_block_is_outside_the_pool():
    new, _, refs, copies, bits = fork([[1, 9, -1], [-1] * 3], [20, 0], [0, 0], [0, 1, 0, 0])
    assert bits == BLOCK_ID and refs == [0, 2, 0, 0]
    assert new == [[1, 9, -1], [1, -1, -1]] and copies == [[-1, -1]] * 2


def test_fork_flags_entries_outside_the_pool_that_stay():
    for parents in ([0, 1], [0, -1]):
        new, _, refs, _, bits = fork([[1, 9, 2], [0, -1, -1]], [48, 3], parents, [1, 1, 1, 0])
        assert bits == BLOCK_ID and new[0] == [1, 9, 2]
        assert refs == [1 if parents[1] == 1 else 0, 1, 1, 0]


@pytest.mark.parametrize("kv", ["bf16", "head", "block"])
def test_paths_with_blocks_outside_the_pool(kv):
    good = (33, 9, [2, 4])

    def check(seq, bad_entry, moved):
        # as if the path were `moved` alone, with all of its length
        p, l, path = seq
        for seed in (20, 21):
            c = Keep(seed, [good, seq, good], kv=kv)
            if kv != "bf16":                                  # what moves outgrows what it meets
                b, o = int(c.tables[1, (p + path[1]) // 16]), (p + path[1]) % 16
                c.caches[0].view(torch.uint8)[b, :, o] = 0x7E
                if kv == "block":
                    c.scales[0][b] = 150
            c.path_lens[1] = len(moved)
            assert path[:len(moved)] == moved
            want = c.want()
            want[2][1] = p + len(path)
            c.path_lens[1] = len(path)
            c.tables[1, bad_entry] = 10 ** 6
            c.run()
            assert flagged() == BLOCK_ID
            c.check(want)

    check((20, 40, [0, 14, 30]), 3, [0, 14])                   # the last one's source
    check((20, 44, [1, 14, 30, 43]), 3, [1, 14])
    check((32, 40, [20, 25]), 3, [])                          # every source of a fresh block
    check((20, 40, [13, 14, 15]), 1, [])                      # the destination
    check((30, 40, [1, 2]), 2, [1])                           # the last one's source, of larger values


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


def test_a_row_cut_into_a_block_that_it_shares():
    # two samples of a prompt of 40; the second goes back to 20 tokens, into a block that is the
    # first one's too: its own copy of that block comes of giving the block back, taking another
    # and copying
    bs, nb = 16, 12
    g = torch.Generator("cuda").manual_seed(1)
    k = torch.randn(nb, 2, bs, 64, generator=g, device="cuda").half()
    tables, lens, refs = i32([[5, 7, 2, -1], [-1] * 4]), i32([40, 0]), i32([0, 0, 1, 0, 0, 1, 0, 1] + [0] * 4)
    new, new_lens, copies = torch.empty_like(tables), torch.empty_like(lens), i32([[0, 0]] * 2)
    P.kv_fork_blocks(new, new_lens, tables, lens, i32([0, 0]), refs, copies, bs)
    P.kv_copy_blocks(k, copies)
    ok()
    assert new.tolist() == [[5, 7, 2, -1], [5, 7, 0, -1]]
    want = [k[b].clone() for b in (5, 7, 2)]
    before = new.clone()
    P.kv_resize_blocks(new, new_lens, i32([40, 16]), refs, bs)
    P.kv_resize_blocks(new, i32([40, 16]), i32([40, 20]), refs, bs)
    P.kv_copy_blocks(k, torch.stack([before[:, 1], new[:, 1]], 1).contiguous())
    ok()
    assert new.tolist() == [[5, 7, 2, -1], [5, 0, -1, -1]]
    assert refs.tolist() == [1, 0, 1, 0, 0, 2, 0, 1, 0, 0, 0, 0]
    assert torch.equal(k[0], want[1])
    k[int(new[1, 1]), :, 4:] = 9                              # what the second row writes next
    for b, w in zip((5, 7, 2), want):
        assert torch.equal(k[b], w)

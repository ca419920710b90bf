"""Outputs of the calls on pages that would be written while they are still read: refused before
anything is launched."""
import pytest

import paged_kv_decode_11_gb300 as P
from paged_kv_decode_11_gb300 import build
from tests.test_abi_tree import FAKE, INVALID, _fork, _keep


@pytest.fixture(scope="module")
def lib():
    build.build()
    return P.load()


@pytest.mark.parametrize("what", ["sl", "cu", "paths", "pl"])
def test_new_lengths_of_a_path_have_a_buffer_of_their_own(lib, what):
    others = {k: (2 + i) * FAKE for i, k in enumerate(("sl", "cu", "paths", "pl"))}
    assert _keep(lib, new=others[what], **others) == INVALID


def test_new_lengths_of_a_fork_are_not_its_parents(lib):
    assert _fork(lib, nl=4 * FAKE, p=4 * FAKE) == INVALID

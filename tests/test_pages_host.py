"""The page calls' refusals, without a GPU."""
import pytest
import torch

from sparse_long_context_dsa_b200 import build as B
from sparse_long_context_dsa_b200 import dsa

P, Q = 1 << 20, 1 << 22            # addresses that are never read: these calls return before any device access


@pytest.fixture(scope="module")
def lib():
    B.build()
    return dsa.lib()


@pytest.mark.parametrize("call,word", [
    (lambda L: L.dsa_pages_fork(P, P, 1, P, P, 1, 1, P, P, P, -1, None, 0, None, 0, None), "n out"),
    (lambda L: L.dsa_pages_fork(P, P, 1, P, P, 1, 1, P, P, P, 4097, None, 0, None, 0, None), "n out"),
    (lambda L: L.dsa_pages_fork(P, P, 0, P, P, 1, 1, P, P, P, 1, None, 0, None, 0, None), "n_pages"),
    (lambda L: L.dsa_pages_fork(P, P, 1 << 31, P, P, 1, 1, P, P, P, 1, None, 0, None, 0, None), "n_pages"),
    (lambda L: L.dsa_pages_fork(P, P, 1, P, P, 0, 1, P, P, P, 1, None, 0, None, 0, None), "max_pages"),
    (lambda L: L.dsa_pages_fork(P, P, 1, P, P, 1 << 25, 1, P, P, P, 1, None, 0, None, 0, None), "max_pages"),
    (lambda L: L.dsa_pages_fork(P, P, 1, P, P, 1, 0, P, P, P, 1, None, 0, None, 0, None), "n_req"),
    (lambda L: L.dsa_pages_fork(None, P, 1, P, P, 1, 1, P, P, P, 1, None, 0, None, 0, None), "NULL"),
    (lambda L: L.dsa_pages_fork(P, P + 2, 1, P, P, 1, 1, P, P, P, 1, None, 0, None, 0, None), "misaligned"),
    (lambda L: L.dsa_pages_fork(P, P + 4, 2, P, P, 1, 1, P, P, P, 1, None, 0, None, 0, None), "overlap"),
    (lambda L: L.dsa_pages_release(P, P, 4, P, P + 8, 3, 1, P, P, 1, None), "overlap"),
    (lambda L: L.dsa_pages_release(P, P, 4, P, P, 3, 1, P, P, -1, None), "n out"),
    (lambda L: L.dsa_pages_compact(P, P, 4, None, P, 3, 1, P, P, None, 0, None, 0, None), "NULL"),
    (lambda L: L.dsa_pages_compact(P, P, 0, P, P, 3, 1, P, P, None, 0, None, 0, None), "n_pages"),
])
def test_bad_arguments_are_rejected_on_the_host(lib, call, word):
    assert call(lib) == dsa.ERR_INVALID_ARG
    assert word in lib.dsa_last_error().decode()


def test_workspace_sizes(lib):
    assert lib.dsa_pages_fork_workspace_size(0) == 0 and lib.dsa_pages_fork_workspace_size(5) >= 24
    assert lib.dsa_pages_compact_workspace_size(0) == 0
    assert lib.dsa_pages_compact_workspace_size(1000) >= 12000


def test_the_binding_refuses_other_shapes_and_host_tensors():
    ref, table = torch.zeros(4, dtype=torch.int32), torch.zeros((2, 3), dtype=torch.int32)
    one = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        dsa.pages_release(ref, table, one, one)
    with pytest.raises(ValueError):
        dsa.pages_compact(ref, table, [torch.zeros((4, 16))])
    with pytest.raises(ValueError):
        dsa.pages_fork(ref, table, one, one, one, [])


@pytest.mark.parametrize("call,word", [
    # the counts and the table in one array
    (lambda L: L.dsa_pages_fork(P, P, 8, P + 16, P + 16, 3, 2, Q, Q, Q, 1, None, 0, None, 0, None), "overlap"),
    (lambda L: L.dsa_pages_release(P, P + 64, 8, P + 512, P + 80, 3, 2, Q, Q, 1, None), "overlap"),
    # what a compaction returns in place of what it reads
    (lambda L: L.dsa_pages_compact(P, P, 8, P + 512, P + 512, 3, 2, P, Q, None, 0, None, 0, None), "overlap"),
    (lambda L: L.dsa_pages_compact(P, P, 8, P + 512, P + 512, 3, 2, Q, P + 512, None, 0, None, 0, None), "overlap"),
    (lambda L: L.dsa_pages_compact(P, P, 8, P + 512, P + 512, 3, 2, Q, Q + 28, None, 0, None, 0, None), "overlap"),
])
def test_arrays_that_overlap_are_refused(lib, call, word):
    assert call(lib) == dsa.ERR_INVALID_ARG
    assert word in lib.dsa_last_error().decode()

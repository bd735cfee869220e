"""The page calls where the pools are more than a call takes, and where requests grow into pages of
their own, as a runtime with several layers runs them."""
import numpy as np
import pytest
import torch

from sparse_long_context_dsa_b200 import dsa

import _quant as Q

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def case(pages=40, pools=21, seed=3):
    gen = torch.Generator().manual_seed(seed)
    table = np.full((6, 8), -1, np.int32)
    t = Q.random_table([300, 64, 170], pages, seed)
    table[:3, :t.shape[1]] = t
    ref = np.zeros(pages, np.int32)
    ref[t[t >= 0]] = 1
    ps = [torch.randint(0, 256, (pages, 16 * (1 + i % 5)), dtype=torch.uint8, generator=gen) for i in range(pools)]
    return ref, table, ps


def test_more_pools_than_a_call_takes():
    # the calls' results are functions of the counts and the table alone: a call for every 8 pools,
    # from the same inputs into outputs of their own, moves every pool alike
    ref, table, ps = case()
    r, t, cu = i32(ref), i32(table), [p.cuda() for p in ps]
    args = i32([0, 2]), i32([4, 5]), i32([299, 130])
    outs = []
    for i in range(0, len(cu), dsa.MAX_PAGE_POOLS):
        outs.append(dsa.pages_fork(r, t, *args, cu[i:i + dsa.MAX_PAGE_POOLS], torch.empty_like(r), torch.empty_like(t)))
    dsa.check_device()
    for o in outs[1:]:
        assert torch.equal(o[0], outs[0][0]) and torch.equal(o[1], outs[0][1])
    r1, t1 = outs[0]
    for child, parent, page in ((4, 0, 4), (5, 2, 2)):
        for a, p in zip(cu, ps):
            assert torch.equal(a[int(t1[child, page])].cpu(), p[table[parent, page]])
    dsa.pages_release(r1, t1, i32([0]), i32([0]))
    kept = [p.cpu().clone() for p in cu]
    outs = []
    for i in range(0, len(cu), dsa.MAX_PAGE_POOLS):
        outs.append(dsa.pages_compact(r1, t1, cu[i:i + dsa.MAX_PAGE_POOLS], torch.empty_like(r), torch.empty_like(t)))
    dsa.check_device()
    for o in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(o, outs[0]))
    new, n_live = outs[0][2].cpu(), int(outs[0][3])
    for a, p in zip(cu, kept):
        for old in range(len(ref)):
            if new[old] >= 0:
                assert torch.equal(a[int(new[old])].cpu(), p[old])
    assert n_live == int((r1 > 0).sum())


def test_more_pools_than_a_call_takes_are_refused_in_one_call():
    ref, table, ps = case()
    with pytest.raises(ValueError, match="at most"):
        dsa.pages_fork(i32(ref), i32(table), i32([0]), i32([4]), i32([64]), [p.cuda() for p in ps])

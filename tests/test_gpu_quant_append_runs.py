"""Lists of the quantising append with two runs of one region: flagged, wherever the two stand; lists
without one are not, and write what the definition writes."""
import numpy as np
import pytest
import torch

from sparse_long_context_dsa_b200 import dsa

import _quant as Q

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def append(table, req, pos, pages, seed=1):
    """The call on an empty cache; returns the caches and the rows."""
    c, s = dsa.quant_cache(pages)
    x, y = Q.rows((len(pos), 4, 192), seed), Q.rows((len(pos), 4, 192), seed + 1)
    dsa.kv_append_quant(c, s, i32(table), i32(pos), x.cuda(), y.cuda(), q_req=i32(req))
    return c, s, x, y


def check(table, req, pos, pages):
    c, s, x, y = append(table, req, pos, pages)
    dsa.check_device()
    zero = np.zeros(tuple(c.shape), np.uint8), np.zeros(tuple(s.shape))
    wc, ws = Q.append(*zero, table, req, pos, x.double().numpy(), y.double().numpy())
    assert np.array_equal(c.cpu().numpy(), wc) and np.array_equal(s.cpu().double().numpy(), ws)


def flagged(table, req, pos, pages):
    append(table, req, pos, pages)
    with pytest.raises(dsa.DsaError, match="two runs"):
        dsa.check_device()


def test_a_list_ordered_step_by_step():
    # two requests, two tokens each: request by request, and token by token
    table = [[0, 1], [2, 3]]
    check(table, [0, 0, 1, 1], [5, 6, 9, 10], 4)
    flagged(table, [0, 1, 0, 1], [5, 9, 6, 10], 4)
    # step by step into regions of their own is no second run
    check(table, [0, 1, 0, 1], [7, 15, 8, 16], 4)


def test_a_page_of_two_requests():
    flagged([[0, 1], [2, 1]], [0, 1], [64, 70], 4)                  # the same region of page 1
    check([[0, 1], [2, 1]], [0, 1], [64, 72], 4)                    # two regions of it


def test_a_chunk_that_laps_a_ring():
    table = [list(np.arange(30) % 9)]
    # 576 tokens from 100 touch 73 regions (100 / 8 = 12 .. 675 / 8 = 84), the ring has 72: its first and
    # last are one; from 104 they touch 72
    flagged(table, [0] * 576, list(range(100, 676)), 9)
    check(table, [0] * 576, list(range(104, 680)), 9)
    flagged(table, [0] * 577, list(range(104, 681)), 9)


@pytest.mark.parametrize("n", [2, 300, 700, 2048, 2049, 6000])
def test_a_long_list_with_one_region_twice(n):
    # a token in each of n regions, in a random order; then one of them again, at the list's ends
    rng = np.random.default_rng(n)
    pages = (n + 7) // 8 + 1
    table = [rng.permutation(pages).tolist()]
    region = rng.permutation(n)
    pos = (region * 8 + rng.integers(0, 8, n)).tolist()
    c, s, x, y = append(table, [0] * n, pos, pages)
    dsa.check_device()
    got = Q.VALUE[c.cpu().numpy()]
    for i in rng.integers(0, n, 20):
        p, r = table[0][pos[i] // 64], pos[i] % 64 // 8
        sc = s[p, :, r].cpu().double().numpy()
        assert np.all(np.abs(got[p, :, r, 0, pos[i] % 8] * sc[:, :1] - x[i].double().numpy()) <= 2.0 ** -4 * np.abs(x[i].double().numpy()) + sc[:, :1] * 2.0 ** -10)
    again = pos[:-1] + [pos[0] // 8 * 8 + (pos[0] + 1) % 8]
    flagged(table, [0] * n, again, pages) if n > 2 else None
    flagged(table + table, [0] * n + [1], pos + [pos[0]], pages)


def test_many_requests_one_token_each():
    # a decode step's list that names its requests, in another order
    n = 4500
    rng = np.random.default_rng(3)
    req = rng.permutation(n).tolist()
    table = np.arange(n)[:, None].tolist()
    append(table, req, (np.asarray(req) % 64).tolist(), n)
    dsa.check_device()
    table[17] = table[4001]
    pos = np.asarray(req) % 64
    pos[req.index(17)] = pos[req.index(4001)] = 33
    flagged(table, req, pos.tolist(), n)


def test_runs_without_a_page_are_not_counted():
    # entries that are skipped (no page, no request, beyond the table) name no region
    append([[0, -1]], [0, 0, 0, 5, 5], [3, 70, 75, 1, 1], 1)
    with pytest.raises(dsa.DsaError) as e:
        dsa.check_device()
    assert "two runs" not in str(e.value)

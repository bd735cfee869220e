"""8-bit window attention on each side of its rules: many requests' decode steps (more rows than CTAs at
once, each taking several; what is left of the last round split in a launch of its own), chunks row by
row and with shared windows, whatever the block table's number of rows, against the same in 64 bits."""
import numpy as np
import pytest
import torch

from sparse_long_context_dsa_b200 import dsa

import _quant as Q

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def resident():
    """CTAs of the row kernel that the GPU holds at once."""
    return 2 * torch.cuda.get_device_properties(0).multi_processor_count


def window(cache, scale, table, q, req, pos, w):
    lse = torch.full((len(pos), 64), 7.0, dtype=torch.float32, device="cuda")
    out = torch.full((len(pos), 64, 192), 7.0, dtype=torch.bfloat16, device="cuda")
    dsa.window_attn_quant(q.cuda(), cache.cuda(), scale.cuda(), i32(table), i32(pos), w,
                          q_req=None if req is None else i32(req), out=out, lse=lse)
    dsa.check_device()
    return out, lse


def check(cache, scale, table, q, req, pos, w):
    out, lse = window(cache, scale, table, q, req, pos, w)
    req = range(len(pos)) if req is None else req
    ref = Q.attention(q.double().numpy(), cache.numpy(), scale.numpy(), table, req, pos, Q.window_tokens(pos, w), 2.0 ** -17)
    Q.check_attention(out, lse, ref)
    for i, p in enumerate(pos):
        if p < 0:
            assert not out[i].any() and torch.isinf(lse[i]).all()
    return out, lse


@pytest.mark.parametrize("rounds,w", [(1.08, 1), (1.08, 100), (1.3, 512), (2.1, 64), (2.7, 9), (1.08, 1024), (1.4, 1100),
                                      (2.05, 1300)])
def test_decode_steps_of_many_requests(rounds, w):
    # rows behind the last full round are split from 97 regions (windows above some 800) on
    n = int(resident() * rounds / 4)
    assert n * 4 > resident()
    rng = np.random.default_rng(n + w)
    pos = rng.integers(0, 1500, n)
    pos[:6] = [0, 1, 7, 8, 63, 64]
    pos[rng.random(n) < 0.12] = -1                                 # slots without a request
    pos[10:14] = -1
    pos = pos.tolist()
    pages = 60                                                     # requests share pages: reads alone
    table = rng.integers(0, pages, (n, 24)).astype(np.int32)
    cache, scale = Q.filled_cache(pages, n)
    check(cache, scale, table, Q.rows((n, 64, 192), w, 0.3), None, pos, w)


def test_decode_steps_with_nobody_there():
    n = resident() // 2
    cache, scale = Q.filled_cache(2, 1)
    out, lse = window(cache, scale, np.zeros((n, 1), np.int32), Q.rows((n, 64, 192), 2), None, [-1] * n, 512)
    assert not out.any() and torch.isinf(lse).all() and (lse < 0).all()


@pytest.mark.parametrize("extra_rows", [0, 100])
@pytest.mark.parametrize("w", [5, 127, 128, 512])
def test_chunks_on_both_sides_of_the_rules(w, extra_rows):
    # one request's chunk: row by row while its rows fit a round of CTAs (two below a window of 128),
    # with shared windows above; row by row with a block table of so many rows that few queries come to
    # one, where CTAs take several rows each
    edge = resident() // 4 * (2 if w < 128 else 1)
    table1 = Q.random_table([800], 13, 3)
    table = np.concatenate([table1, np.full((extra_rows, table1.shape[1]), -1, np.int32)])
    cache, scale = Q.filled_cache(13, 4)
    for n in (edge, edge + 1, edge + 41):
        pos = list(range(800 - n, 800))
        check(cache, scale, table, Q.rows((n, 64, 192), n, 0.3), [0] * n, pos, w)


def test_rows_without_tokens_between_others_row_by_row():
    # several rows per CTA, one and two and none of them with tokens
    n, w = resident() * 5 // 8, 1
    table = np.concatenate([Q.random_table([200], 4, 5), np.full((n, 4), -1, np.int32)])
    cache, scale = Q.filled_cache(4, 6)
    pos = [-1 if i % 5 in (1, 2, 4) or 60 < i < 140 else i for i in range(n)]
    assert n <= 200 and n * 4 > 2 * resident()
    q = Q.rows((n, 64, 192), 7, 0.3)
    for _ in range(5):
        check(cache, scale, table, q, [0] * n, pos, w)


@pytest.mark.parametrize("w", [1, 60, 512])
def test_one_query_alone_in_a_step_and_in_a_chunk(w):
    # the same query by itself, in a decode step of many requests, and inside a chunk whose windows are
    # shared: each within the bounds of the 64-bit form, so within two of them of another
    n = resident() // 4 + 6
    table = Q.random_table([1000], 16, 8)
    cache, scale = Q.filled_cache(16, 9)
    pos = list(range(1000 - n, 1000))
    q = Q.rows((n, 64, 192), 10, 0.3)
    chunk, cl = check(cache, scale, table, q, [0] * n, pos, w)
    steps, sl = check(cache, scale, np.repeat(table, n, 0), q, None, pos, w)
    again, al = window(cache, scale, np.repeat(table, n, 0), q, None, pos, w)
    assert torch.equal(steps, again) and torch.equal(sl, al)       # one call, one result
    for i in (0, 9, n - 1):
        alone, l = window(cache, scale, table, q[i:i + 1], [0], pos[i:i + 1], w)
        ref = Q.attention(q[i:i + 1].double().numpy(), cache.numpy(), scale.numpy(), table, [0], pos[i:i + 1],
                          Q.window_tokens(pos[i:i + 1], w), 2.0 ** -17)
        Q.check_attention(alone, l, ref)
        for other, ol in ((chunk, cl), (steps, sl)):
            d = (alone[0].double() - other[i].double()).abs().cpu().numpy()
            assert np.all(d <= 2 * ref[2][0])
            assert np.all((l[0].double() - ol[i].double()).abs().cpu().numpy() <= 2 * ref[3][0])

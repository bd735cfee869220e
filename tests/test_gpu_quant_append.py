"""GPU quantising append (dsa_kv_append_quant) against the definition in 64 bits: codes and scales
byte for byte, and nothing else of the cache touched."""
import numpy as np
import pytest
import torch

from sparse_long_context_dsa_b200 import dsa

import _quant as Q

pytestmark = pytest.mark.gpu


def run(cache, scale, table, req, pos, nk, nv, identity=False):
    """The call on the GPU and the plain form, compared over the whole cache; returns the GPU's."""
    c, s = cache.cuda(), scale.cuda()
    bt = torch.tensor(np.asarray(table), dtype=torch.int32, device="cuda")
    p = torch.tensor(pos, dtype=torch.int32, device="cuda")
    r = None if identity else torch.tensor(req, dtype=torch.int32, device="cuda")
    dsa.kv_append_quant(c, s, bt, p, nk.cuda(), nv.cuda(), q_req=r)
    wc, ws = Q.append(cache.numpy(), scale.double().numpy(), np.asarray(table), req, pos, nk.double().numpy(),
                      nv.double().numpy())
    gc, gs = c.cpu().numpy(), s.cpu().numpy()
    assert np.array_equal(gs.astype(np.float64), ws)
    # NaN has two codes; all else is one
    nan = np.isnan(Q.VALUE[wc])
    assert np.array_equal(np.isnan(Q.VALUE[gc]), nan)
    assert np.array_equal(gc[~nan], wc[~nan])
    return c.cpu(), s.cpu()


def new_rows(n, seed, spread=0.7):
    return Q.rows((n, Q.G, Q.D), seed, spread), Q.rows((n, Q.G, Q.D), seed + 1, spread)


@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 64, 65, 200, 2500])
@pytest.mark.parametrize("start", [0, 5, 64])
def test_consecutive_tokens_of_one_request(n, start):
    pages = (start + n + 63) // 64 + 2
    cache, scale = Q.filled_cache(pages, 10 + n)
    table = Q.random_table([start + n], pages, 11 + n)
    run(cache, scale, table, [0] * n, list(range(start, start + n)), *new_rows(n, 12 + n))
    dsa.check_device()


@pytest.mark.parametrize("batch", [1, 3, 8, 33])
def test_decode_steps_of_a_ragged_batch(batch):
    # 20 steps from lengths at every offset of a region; the caches of one step are the next one's
    lengths = [3 * b + (b * b) % 70 for b in range(batch)]
    pages = sum((L + 20 + 63) // 64 for L in lengths)
    table = Q.random_table([L + 20 for L in lengths], pages, batch)
    cache, scale = Q.filled_cache(pages, 20 + batch, spread=1.5)
    for step in range(20):
        pos = [L + step for L in lengths]
        cache, scale = run(cache, scale, table, list(range(batch)), pos, *new_rows(batch, 100 * step + batch, 1.5),
                           identity=True)
    dsa.check_device()


def test_ragged_requests_in_one_call():
    # runs of 0 .. 40 tokens of 9 requests, beginning anywhere
    counts = [1, 0, 40, 8, 3, 17, 0, 1, 25]
    starts = [70, 0, 5, 64, 6, 0, 9, 63, 31]
    pages = sum((s + c + 63) // 64 for s, c in zip(starts, counts)) + 1
    table = Q.random_table([s + c for s, c in zip(starts, counts)], pages, 5)
    req = [b for b, c in enumerate(counts) for _ in range(c)]
    pos = [s + j for s, c in zip(starts, counts) for j in range(c)]
    cache, scale = Q.filled_cache(pages, 6)
    run(cache, scale, table, req, pos, *new_rows(len(req), 7))
    dsa.check_device()


def test_ragged_requests_in_a_long_call():
    # runs of any length at any offset, at every place of 8 list entries; some entries skipped
    counts = [333, 1, 0, 95, 7, 410, 130]
    starts = [70, 3, 0, 61, 6, 5, 64]
    pages = sum((s + c + 63) // 64 for s, c in zip(starts, counts)) + 1
    table = Q.random_table([s + c for s, c in zip(starts, counts)], pages, 15)
    keep = [i for i in range(sum(counts)) if i % 41 not in (3, 17)]
    req = [b for b, c in enumerate(counts) for _ in range(c)]
    pos = [s + j for s, c in zip(starts, counts) for j in range(c)]
    req, pos = [req[i] for i in keep], [pos[i] for i in keep]
    cache, scale = Q.filled_cache(pages, 16)
    run(cache, scale, table, req, pos, *new_rows(len(req), 17))
    dsa.check_device()
    # entries of two bad pages among the others
    bad = np.array(table)
    bad[0, 3], bad[5, 4] = pages, -1
    x, y = new_rows(len(req), 18)
    c, s = cache.cuda(), scale.cuda()
    i32 = lambda v: torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")
    dsa.kv_append_quant(c, s, i32(bad), i32(pos), x.cuda(), y.cuda(), q_req=i32(req))
    with pytest.raises(dsa.DsaError):
        dsa.check_device()
    good = [i for i in range(len(req)) if (req[i], pos[i] // 64) not in ((0, 3), (5, 4))]
    assert 0 < len(good) < len(req)
    wc, ws = Q.append(cache.numpy(), scale.double().numpy(), bad, [req[i] for i in good], [pos[i] for i in good],
                      x[good].double().numpy(), y[good].double().numpy())
    assert np.array_equal(c.cpu().numpy(), wc) and np.array_equal(s.cpu().double().numpy(), ws)


def test_rows_of_a_run_may_leave_gaps():
    cache, scale = Q.filled_cache(2, 8)
    run(cache, scale, [[1, 0]], [0, 0, 0, 0], [1, 3, 6, 66], *new_rows(4, 9))
    dsa.check_device()


def test_ring_of_nine_pages():
    ring, batch = 9, 2
    table = (np.arange(batch)[:, None] * ring + np.arange(40)[None] % ring).astype(np.int32)
    cache, scale = Q.filled_cache(batch * ring, 10)
    for pos in ([511, 575], [512, 576], [580, 2000], [581, 2001]):
        cache, scale = run(cache, scale, table, [0, 1], pos, *new_rows(2, pos[0]))
    dsa.check_device()


@pytest.mark.parametrize("first", [0, 4])
def test_extreme_values(first):
    # zeros, the smallest and largest bf16, signed zeros, powers of two at a code's border
    vals = [0.0, 1e-40, 3.3e38, -3.3e38, 448.0, 449.0, -0.0, 2.0 ** -126, 2.0 ** -9, 1.0]
    cache, scale = Q.filled_cache(1, 11)
    if first == 0:
        cache.zero_()
        scale.zero_()
    for v in vals:
        x, y = new_rows(1, 12)
        x.fill_(v)
        y[:, :, ::2] = v
        run(cache, scale, [[0]], [0], [first], x, y)
    dsa.check_device()


def test_infinities_saturate_and_nan_stays():
    cache, scale = Q.filled_cache(1, 13)
    x, y = new_rows(3, 14)
    x[0, 0, 5] = float("inf")
    x[1, 1, 6] = float("nan")
    y[2, 2, 7] = float("-inf")
    y[2, 3] = float("nan")
    c, s = run(cache, scale, [[0]], [0, 0, 0], [0, 1, 2], x, y)
    assert float(s[0, 0, 0, 0]) == 2.0 ** 120 and Q.VALUE[c[0, 0, 0, 0, 0, 5]] == 448
    assert np.isfinite(s.numpy()).all()


def test_scales_that_are_no_powers_of_two_are_kept_or_raised():
    # a cache quantised elsewhere (absmax / 448): the old scale stays while it is the larger
    cache, scale = Q.filled_cache(1, 15)
    scale = scale * 1.37
    x, y = new_rows(1, 16, 0.0)
    c, s = cache.cuda(), scale.cuda()
    bt = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    dsa.kv_append_quant(c, s, bt, torch.tensor([3], dtype=torch.int32, device="cuda"), x.cuda(), y.cuda())
    dsa.check_device()
    new = torch.stack([x, y], 2)[0]                                # [4][2][192]
    want = torch.maximum(scale[0, :, 0], torch.tensor([[Q.block_scale(float(v.abs().max())) for v in g] for g in new]))
    assert torch.equal(s[0, :, 0].cpu(), want.float())
    # each code one rounding of x (2^-4 relative, or half a subnormal step), the product and the reciprocal 2^-23 more
    got = torch.from_numpy(Q.VALUE[c[0, :, 0, :, 3].cpu().numpy()]) * s[0, :, 0].cpu().double()[..., None]
    err = (got - new.double()).abs()
    assert (err <= new.double().abs() * (2.0 ** -4 + 2.0 ** -21) + s[0, :, 0].cpu().double()[..., None] * 2.0 ** -10).all()


@pytest.mark.parametrize("table,req,pos", [
    ([[0]], [0], [64]),              # beyond the block table
    ([[0]], [0], [-1]),
    ([[0]], [1], [3]),               # no such request
    ([[0]], [-1], [3]),
    ([[7]], [0], [3]),               # no such page
    ([[-1]], [0], [3]),
])
def test_bad_entries_are_flagged_and_skipped(table, req, pos):
    # beside a good entry, which is written
    cache, scale = Q.filled_cache(2, 17)
    x, y = new_rows(2, 18)
    c, s = cache.cuda(), scale.cuda()
    bt = torch.tensor([table[0] + [1]], dtype=torch.int32, device="cuda")[:, :2].contiguous()
    if pos == [64]:
        bt = torch.tensor([[0]], dtype=torch.int32, device="cuda")
    dsa.kv_append_quant(c, s, bt, torch.tensor(pos + [5], dtype=torch.int32, device="cuda"), x.cuda(), y.cuda(),
                        q_req=torch.tensor(req + [0], dtype=torch.int32, device="cuda"))
    with pytest.raises(dsa.DsaError):
        dsa.check_device()
    good = int(bt[0, 0])
    if 0 <= good < 2 and not (req == [0] and 0 <= pos[0] < 64):
        wc, ws = Q.append(cache.numpy(), scale.double().numpy(), [[good]], [0], [5], x[1:].double().numpy(),
                          y[1:].double().numpy())
    else:
        wc, ws = cache.numpy(), scale.double().numpy()
    assert np.array_equal(c.cpu().numpy(), wc) and np.array_equal(s.cpu().double().numpy(), ws)


@pytest.mark.parametrize("pos", [[3, 3], [4, 3], [1, 2, 2, 5], [0, 1, 2, 3, 4, 5, 6, 7, 7, 7]])
def test_entries_that_do_not_ascend_are_flagged_and_skipped(pos):
    cache, scale = Q.filled_cache(1, 19)
    x, y = new_rows(len(pos), 20)
    run(cache, scale, [[0]], [0] * len(pos), pos, x, y)
    with pytest.raises(dsa.DsaError, match="ascending"):
        dsa.check_device()


def test_pages_behind_four_gigabytes():
    # code offsets pass 2^32
    pages = (1 << 32) // (4 * 8 * 2 * 8 * 192) + 50
    c, s = dsa.quant_cache(pages)
    bt = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32, device="cuda")
    x, y = new_rows(70, 21)
    pos = list(range(70))
    dsa.kv_append_quant(c, s, bt, torch.tensor(pos, dtype=torch.int32, device="cuda"), x.cuda(), y.cuda(),
                        q_req=torch.zeros(70, dtype=torch.int32, device="cuda"))
    dsa.check_device()
    zero = np.zeros((2,) + tuple(c.shape[1:]), np.uint8), np.zeros((2,) + tuple(s.shape[1:]))
    wc, ws = Q.append(*zero, [[1, 0]], [0] * 70, pos, x.double().numpy(), y.double().numpy())
    assert np.array_equal(c[-2:].cpu().numpy(), wc) and np.array_equal(s[-2:].cpu().double().numpy(), ws)
    assert not c[:-2].any() and not s[:-2].any()


def test_on_a_side_stream_and_in_a_graph():
    cache, scale = Q.filled_cache(2, 22)
    x, y = new_rows(2, 23)
    want = Q.append(cache.numpy(), scale.double().numpy(), [[1], [0]], [0, 1], [6, 9], x.double().numpy(),
                    y.double().numpy())
    st = torch.cuda.Stream()
    bt = torch.tensor([[1], [0]], dtype=torch.int32, device="cuda")
    pos = torch.tensor([6, 9], dtype=torch.int32, device="cuda")
    xc, yc = x.cuda(), y.cuda()
    for graph in (False, True):
        c, s = cache.cuda(), scale.cuda()
        torch.cuda.synchronize()
        if graph:
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr):
                dsa.kv_append_quant(c, s, bt, pos, xc, yc)
            gr.replay()
        else:
            with torch.cuda.stream(st):
                dsa.kv_append_quant(c, s, bt, pos, xc, yc)
        torch.cuda.synchronize()
        dsa.check_device()
        assert np.array_equal(c.cpu().numpy(), want[0]) and np.array_equal(s.cpu().double().numpy(), want[1])

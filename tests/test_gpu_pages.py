"""GPU page calls (dsa_pages_fork, dsa_pages_release, dsa_pages_compact) against their definitions in
plain Python: counts, tables and pages equal, whole."""
import numpy as np
import pytest
import torch

from sparse_long_context_dsa_b200 import dsa

import _quant as Q

pytestmark = pytest.mark.gpu
PAGE = 64


def fork(ref, table, parent, child, length, pools):
    ref0, ref, table, pools = ref, ref.copy(), table.copy(), [p.copy() for p in pools]
    src_table, free, at = table.copy(), np.nonzero(ref0 <= 0)[0], 0
    errors = 0
    for i, (b, c, L) in enumerate(zip(parent, child, length)):
        ok = 0 <= b < len(table) and 0 <= c < len(table) and 0 <= L <= table.shape[1] * PAGE
        j = at
        if ok and L % PAGE:
            at += 1
        if not ok or c in parent or c in child[:i]:
            errors += 1
            continue
        full = L // PAGE
        row = np.full(table.shape[1], -1, np.int32)
        for v in range(full):
            p = src_table[b, v]
            if 0 <= p < len(ref) and ref0[p] > 0:
                row[v] = p
                ref[p] += 1
            else:
                errors += 1
        if L % PAGE:
            p = src_table[b, full]
            if 0 <= p < len(ref) and ref0[p] > 0 and j < len(free):
                row[full] = free[j]
                ref[free[j]] = 1
                for x in pools:
                    x[free[j]] = x[p]
            else:
                errors += 1
        table[c] = row
    return ref, table, pools, errors


def release(ref, table, req, keep):
    ref, table = ref.copy(), table.copy()
    errors = 0
    for i, (b, k) in enumerate(zip(req, keep)):
        if not 0 <= b < len(table) or k < 0 or b in req[:i]:
            errors += 1
            continue
        for v in range((k + PAGE - 1) // PAGE, table.shape[1]):
            p = table[b, v]
            table[b, v] = -1
            if p == -1:
                continue
            if not 0 <= p < len(ref) or ref[p] <= 0:
                errors += 1
            else:
                ref[p] -= 1
    return ref, table, errors


def compact(ref, table, pools):
    ref, pools = ref.copy(), [p.copy() for p in pools]
    live = ref > 0
    n_live = int(live.sum())
    movers = [p for p in range(len(ref) - 1, n_live - 1, -1) if live[p]]
    holes = [p for p in range(n_live) if not live[p]]
    new = np.where(live, np.arange(len(ref)), -1)
    for s, d in zip(movers, holes):
        new[s] = d
        ref[d], ref[s] = ref[s], 0
        for x in pools:
            x[d] = x[s]
    ok = (table >= 0) & (table < len(ref))
    out = np.where(ok, new[np.where(ok, table, 0)], -1).astype(np.int32)
    errors = int(((table != -1) & (out == -1)).sum())
    return ref, out, pools, new.astype(np.int32), n_live, errors


def pool_of(lengths, pages, seed, columns=None, rows=None, page_bytes=(96, 4096 * 5 + 32)):
    """ref, table (rows without a request: -1) and pools of these page sizes."""
    rng = np.random.default_rng(seed)
    rows = rows or len(lengths)
    columns = columns or max((L + PAGE - 1) // PAGE for L in lengths) + 1
    table = np.full((rows, columns), -1, np.int32)
    t = Q.random_table(lengths, pages, seed)
    table[:len(lengths), :t.shape[1]] = t
    ref = np.zeros(pages, np.int32)
    ref[t[t >= 0]] = 1
    pools = [rng.integers(0, 256, (pages, b), dtype=np.uint8) for b in page_bytes]
    return ref, table, pools


def cuda(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def outcome(errors):
    if errors:
        with pytest.raises(dsa.DsaError, match="pages"):
            dsa.check_device()
    else:
        dsa.check_device()


def run_fork(ref, table, parent, child, length, pools, in_place):
    want = fork(ref, table, parent, child, length, pools)
    r, t, ps = cuda(ref), cuda(table), [cuda(p) for p in pools]
    kw = {} if in_place else dict(ref_out=torch.full_like(r, 77), table_out=torch.full_like(t, 77))
    ro, to = dsa.pages_fork(r, t, i32(parent), i32(child), i32(length), ps, **kw)
    outcome(want[3])
    assert np.array_equal(ro.cpu().numpy(), want[0]) and np.array_equal(to.cpu().numpy(), want[1])
    for p, w in zip(ps, want[2]):
        assert np.array_equal(p.cpu().numpy(), w)
    if not in_place:
        assert np.array_equal(r.cpu().numpy(), ref) and np.array_equal(t.cpu().numpy(), table)
    return ro.cpu().numpy(), to.cpu().numpy(), [p.cpu().numpy() for p in ps]


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("pages", [40, 4096, 9001])
def test_fork(pages, in_place):
    ref, table, pools = pool_of([300, 64, 1000, 1], pages, pages, rows=20)
    run_fork(ref, table, [0, 0, 1, 2, 3, 2, 0], [4, 19, 7, 5, 6, 10, 11], [300, 256, 64, 130, 1, 0, 63], pools, in_place)


def test_many_forks_of_one_request():
    ref, table, pools = pool_of([700], 300, 1, rows=150)
    run_fork(ref, table, [0] * 149, list(range(1, 150)), [700 - i for i in range(149)], pools, True)


def test_fork_without_pools_and_without_forks():
    ref, table, pools = pool_of([300, 200], 20, 2, rows=4)
    run_fork(ref, table, [0, 1], [2, 3], [299, 128], [], True)
    run_fork(ref, table, [], [], [], pools, True)
    run_fork(ref, table, [], [], [], pools, False)


@pytest.mark.parametrize("parent,child,length", [
    ([0, 5], [2, 3], [70, 70]),              # no such parent
    ([0, -1], [2, 3], [70, 70]),
    ([0, 0], [2, 4], [70, 70]),              # no such child
    ([0, 0], [2, 3], [70, -1]),              # no such length
    ([0, 0], [2, 3], [70, 1 << 20]),
    ([0, 0, 1], [2, 2, 3], [70, 60, 50]),    # a child twice
    ([0, 2], [2, 3], [70, 60]),              # a child that is a parent
    ([0], [2], [400]),                       # behind the parent's pages: entries without a page
])
def test_bad_forks_are_flagged_and_do_nothing(parent, child, length):
    ref, table, pools = pool_of([300, 200], 30, 3, columns=8, rows=4)
    run_fork(ref, table, parent, child, length, pools, True)


def test_forks_without_a_free_page():
    ref, table, pools = pool_of([300, 200], 11, 4, rows=6)          # 9 pages held, 2 free
    run_fork(ref, table, [0, 1, 0, 1], [2, 3, 4, 5], [299, 199, 128, 190], pools, True)


def test_parents_entries_that_name_free_pages():
    # among them the pages that this call's forks copy into
    ref, table, pools = pool_of([300, 200, 700], 60, 14, rows=12)
    free = np.nonzero(ref <= 0)[0]
    table[0, 0], table[0, 4], table[1, 1], table[1, 3], table[2, 2] = free[0], free[1], free[2], free[0], free[9]
    for _ in range(5):
        run_fork(ref, table, [0, 1, 2, 0, 1, 2, 2], [4, 5, 6, 7, 8, 9, 10], [299, 198, 650, 256, 130, 699, 450], pools, True)


@pytest.mark.parametrize("in_place", [True, False])
def test_release(in_place):
    ref, table, pools = pool_of([300, 64, 1000, 1], 60, 5, rows=6)
    ref, table, _ = run_fork(ref, table, [2, 0], [4, 5], [900, 300], pools, True)
    req, keep = [2, 0, 4, 3], [0, 130, 64, 10 ** 9]
    want = release(ref, table, req, keep)
    r, t = cuda(ref), cuda(table)
    kw = {} if in_place else dict(ref_out=torch.full_like(r, 77), table_out=torch.full_like(t, 77))
    ro, to = dsa.pages_release(r, t, i32(req), i32(keep), **kw)
    outcome(want[2])
    assert want[2] == 0
    assert np.array_equal(ro.cpu().numpy(), want[0]) and np.array_equal(to.cpu().numpy(), want[1])
    if not in_place:
        assert np.array_equal(r.cpu().numpy(), ref) and np.array_equal(t.cpu().numpy(), table)


@pytest.mark.parametrize("req,keep", [([0, 0], [64, 0]), ([0, 9], [0, 0]), ([-1, 1], [0, 0]), ([0, 1], [-1, 0])])
def test_bad_releases_are_flagged_and_do_nothing(req, keep):
    ref, table, _ = pool_of([300, 64], 20, 6)
    want = release(ref, table, req, keep)
    r, t = dsa.pages_release(cuda(ref), cuda(table), i32(req), i32(keep))
    assert want[2] > 0
    outcome(want[2])
    assert np.array_equal(r.cpu().numpy(), want[0]) and np.array_equal(t.cpu().numpy(), want[1])


def test_release_of_pages_that_nobody_holds():
    ref, table, _ = pool_of([300, 64], 20, 7)
    ref[table[0, 1]] = 0
    table[0, 2] = 99
    want = release(ref, table, [0], [0])
    r, t = dsa.pages_release(cuda(ref), cuda(table), i32([0]), i32([0]))
    outcome(want[2])
    assert np.array_equal(r.cpu().numpy(), want[0]) and np.array_equal(t.cpu().numpy(), want[1])


def run_compact(ref, table, pools, in_place):
    want = compact(ref, table, pools)
    r, t, ps = cuda(ref), cuda(table), [cuda(p) for p in pools]
    kw = {} if in_place else dict(ref_out=torch.full_like(r, 77), table_out=torch.full_like(t, 77))
    ro, to, new, n_live = dsa.pages_compact(r, t, ps, **kw)
    outcome(want[5])
    assert int(n_live) == want[4]
    assert np.array_equal(ro.cpu().numpy(), want[0]) and np.array_equal(to.cpu().numpy(), want[1])
    assert np.array_equal(new.cpu().numpy(), want[3])
    for p, w in zip(ps, want[2]):
        assert np.array_equal(p.cpu().numpy()[:want[4]], w[:want[4]])
    if not in_place:
        assert np.array_equal(r.cpu().numpy(), ref) and np.array_equal(t.cpu().numpy(), table)


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("pages", [1, 2, 63, 100, 4095, 4096, 4097, 20011, 150000])
def test_compact(pages, in_place):
    rng = np.random.default_rng(pages)
    lengths = [max(1, int(x)) for x in rng.integers(1, 64 * max(1, pages // 16), 5)] if pages > 10 else [1]
    ref, table, _ = pool_of(lengths, pages, pages, page_bytes=())
    drop = rng.random(len(ref)) < 0.3                              # holes anywhere, tables to match
    held = table >= 0
    gone = np.zeros_like(held)
    gone[held] = drop[table[held]]
    ref[np.unique(table[gone])] = 0
    table[gone] = -1
    ref[ref > 0] += rng.integers(0, 3, int((ref > 0).sum())).astype(np.int32)
    pools = [rng.integers(0, 256, (pages, b), dtype=np.uint8) for b in (16, 176)]
    run_compact(ref, table, pools, in_place)


@pytest.mark.parametrize("kind", ["all free", "all live", "last live", "negative counts"])
def test_compact_extremes(kind):
    pages = 300
    rng = np.random.default_rng(8)
    pools = [rng.integers(0, 256, (pages, 48), dtype=np.uint8)]
    ref = np.zeros(pages, np.int32)
    table = np.full((2, 200), -1, np.int32)
    if kind == "all live":
        ref[:] = 2
        table[:, :150] = rng.permutation(pages).reshape(2, 150)
    elif kind == "last live":
        ref[-1] = 1
        table[1, 3] = pages - 1
    elif kind == "negative counts":
        ref[:100] = -3
        ref[200:] = 1
        table[0, :100] = np.arange(200, 300)
    run_compact(ref, table, pools, True)
    run_compact(ref, table, pools, False)


def test_compact_flags_entries_without_a_live_page():
    ref, table, pools = pool_of([300, 64], 20, 9)
    ref[table[0, 1]] = 0
    table[0, 2] = 99
    table[1, 0] = -7
    run_compact(ref, table, pools, True)


def test_a_large_page_and_offsets_behind_four_gigabytes():
    pages, size = 44000, 98304                                     # the cache's page: 4.3 GB in all
    pool = torch.zeros((pages, size), dtype=torch.uint8, device="cuda")
    row = torch.arange(size, device="cuda") % 251
    pool[pages - 1] = row.to(torch.uint8)
    ref = torch.ones(pages, dtype=torch.int32, device="cuda")
    ref[7] = 0
    table = i32([[pages - 1, 3], [-1, -1]])
    ro, to = dsa.pages_fork(ref, table, i32([0]), i32([1]), i32([63]), [pool])
    dsa.check_device()
    assert int(to[1, 0]) == 7 and torch.equal(pool[7], row.to(torch.uint8)) and int(ro[7]) == 1
    ro, to = dsa.pages_release(ro, to, i32([1]), i32([0]))
    pool[7] = 0
    ro, to, new, n_live = dsa.pages_compact(ro, to, [pool])
    dsa.check_device()
    assert int(n_live) == pages - 1 and int(to[0, 0]) == 7 and torch.equal(pool[7], row.to(torch.uint8))


def test_pools_that_overlap_are_refused():
    ref, table = torch.zeros(8, dtype=torch.int32, device="cuda"), i32([[-1, -1]] * 2)
    data = torch.zeros(9 * 64, dtype=torch.uint8, device="cuda")
    a, b = data[:512].view(8, 64), data[64:].view(8, 64)
    for pools in ([a, b], [a, a]):
        with pytest.raises(dsa.DsaError, match="overlap"):
            dsa.pages_compact(ref, table, pools)
        with pytest.raises(dsa.DsaError, match="overlap"):
            dsa.pages_fork(ref, table, i32([0]), i32([1]), i32([0]), pools)


def test_streams_and_graphs():
    ref, table, pools = pool_of([300, 500], 60, 10, rows=5)
    want = fork(ref, table, [0, 1, 1], [2, 3, 4], [290, 400, 500], pools)
    r, t, ps = cuda(ref), cuda(table), [cuda(p) for p in pools]
    args = [(torch.empty_like(r), torch.empty_like(t)) for _ in range(2)]
    pa, ch, le = i32([0, 1, 1]), i32([2, 3, 4]), i32([290, 400, 500])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dsa.pages_fork(r, t, pa, ch, le, ps, *args[0])
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        dsa.pages_fork(r, t, pa, ch, le, ps, *args[1])
    graph.replay()
    torch.cuda.synchronize()
    dsa.check_device()
    for ro, to in args:
        assert np.array_equal(ro.cpu().numpy(), want[0]) and np.array_equal(to.cpu().numpy(), want[1])


def test_fork_append_release_compact_together():
    # a prompt is filled, forked into three samples that each append their own tokens, one sample
    # ends, the pool is compacted: every request's attention stays what its own tokens give
    pages, L, steps = 40, 203, 11
    c, s = dsa.quant_cache(pages)
    table = np.full((4, 6), -1, np.int32)
    table[0, :4] = [31, 5, 17, 22]
    ref = np.zeros(pages, np.int32)
    ref[table[0, :4]] = 1
    r, t = cuda(ref), cuda(table)
    k, v = Q.rows((L, 4, 192), 11), Q.rows((L, 4, 192), 12)
    dsa.kv_append_quant(c, s, t, i32(list(range(L))), k.cuda(), v.cuda(), q_req=i32([0] * L))
    dsa.pages_fork(r, t, i32([0, 0, 0]), i32([1, 2, 3]), i32([L, L, 192]), [c, s])
    dsa.check_device()
    lengths = [L, L, L, 192]
    held = [(k, v), (k, v), (k, v), (k[:192], v[:192])]
    # request 3 begins a page of its own
    t[3, 3] = int((r == 0).nonzero()[0])
    r[t[3, 3].long()] = 1
    plain = []
    for b in range(4):
        pc, ps = np.zeros((6,) + tuple(c.shape[1:]), np.uint8), np.zeros((6,) + tuple(s.shape[1:]))
        n = lengths[b]
        plain.append(Q.append(pc, ps, [list(range(6))], [0] * n, list(range(n)), held[b][0].double().numpy(),
                              held[b][1].double().numpy()))
    for step in range(steps):
        nk, nv = Q.rows((4, 4, 192), 50 + step), Q.rows((4, 4, 192), 90 + step)
        pos = [n + step for n in lengths]
        dsa.kv_append_quant(c, s, t, i32(pos), nk.cuda(), nv.cuda())
        for b in range(4):
            plain[b] = Q.append(*plain[b], [list(range(6))], [0], [pos[b]], nk[b:b + 1].double().numpy(),
                                nv[b:b + 1].double().numpy())

    def check(rows):
        pos = [lengths[b] + steps - 1 for b in rows]
        q = Q.rows((len(rows), 64, 192), 13, 0.3)
        lse = torch.empty((len(rows), 64), dtype=torch.float32, device="cuda")
        out = dsa.window_attn_quant(q.cuda(), c, s, t, i32(pos), 150, q_req=i32(rows), lse=lse)
        dsa.check_device()
        pc, ps = np.concatenate([plain[b][0] for b in rows]), np.concatenate([plain[b][1] for b in rows])
        tab = np.arange(6 * len(rows)).reshape(len(rows), 6)
        Q.check_attention(out, lse, Q.attention(q.double().numpy(), pc, ps, tab, list(range(len(rows))), pos,
                                                Q.window_tokens(pos, 150)))

    check([0, 1, 2, 3])
    dsa.pages_release(r, t, i32([1, 0]), i32([0, 0]))
    ro, to, new, n_live = dsa.pages_compact(r, t, [c, s])
    dsa.check_device()
    assert int(n_live) == int((r > 0).sum()) and int(t.max()) < int(n_live) and (t[:2] == -1).all()
    assert int(r[t[2, 0].long()]) == 2                              # the prompt's pages have two holders left
    check([2, 3])

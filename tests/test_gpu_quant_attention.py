"""GPU attention over the 8-bit cache (dsa_sparse_attn_decode_quant, dsa_sparse_attn_prefill_quant,
dsa_window_attn_quant) against the same in 64 bits.  Tolerances: _quant.attention derives them."""
import numpy as np
import pytest
import torch

from sparse_long_context_dsa_b200 import dsa

import _quant as Q

pytestmark = pytest.mark.gpu


def to(x, dtype=torch.int32):
    return torch.tensor(np.asarray(x), dtype=dtype, device="cuda")


def sparse(cache, scale, table, q, req, pos, sel, cnt, prefill=True, check=True):
    nq = len(pos)
    lse = torch.empty((nq, 64), dtype=torch.float32, device="cuda")
    out = torch.full((nq, 64, 192), 7.0, dtype=torch.bfloat16, device="cuda")
    args = (q.cuda(), cache.cuda(), scale.cuda(), to(table))
    if prefill:
        dsa.sparse_attn_prefill_quant(*args, to(req), to(pos), to(sel), to(cnt), out=out, lse=lse)
    else:
        dsa.sparse_attn_decode_quant(*args, to(pos), to(sel), to(cnt), out=out, lse=lse)
    if check:
        dsa.check_device()
    return out, lse


def reference(cache, scale, table, q, req, pos, tokens):
    return Q.attention(q.double().numpy(), cache.numpy(), scale.numpy(), table, req, pos, tokens)


def sparse_case(lengths, k, seed, pos=None, req=None, prefill=False, spread=0.7):
    pages = sum((L + 63) // 64 for L in lengths) + 1
    table = Q.random_table(lengths, pages, seed)
    cache, scale = Q.filled_cache(pages, seed + 1, spread)
    pos = [L - 1 for L in lengths] if pos is None else pos
    req = list(range(len(lengths))) if req is None else req
    q = Q.rows((len(pos), 64, 192), seed + 2, 0.3)
    sel, cnt = Q.random_selection(pos, k, seed + 3)
    out, lse = sparse(cache, scale, table, q, req, pos, sel, cnt, prefill)
    Q.check_attention(out, lse, reference(cache, scale, table, q, req, pos, Q.sel_tokens(sel, cnt, pos)))


@pytest.mark.parametrize("k", [1, 2, 5, 8, 9, 64, 100, 512])
def test_decode_random_selections(k):
    sparse_case([5000, 9000 + 3, 600 + 7, 1], k, 30 + k)


@pytest.mark.parametrize("batch", [1, 2, 4, 5, 9, 18, 37])
def test_decode_batches(batch):
    sparse_case([1500 + 37 * b for b in range(batch)], 130, batch)


def test_decode_long_selection():
    sparse_case([20000], 2048, 60)


@pytest.mark.parametrize("length", [1, 2, 7, 8, 9, 63, 64, 65])
def test_short_contexts(length):
    sparse_case([length, length + 1], 512, 70 + length)


def test_prefill_queries_of_several_requests():
    rng = np.random.default_rng(80)
    lengths = [1000, 613, 2000]
    req = (np.arange(90) % 3).tolist()
    pos = [int(rng.integers(0, lengths[r])) for r in req]
    sparse_case(lengths, 60, 80, pos, req, prefill=True)


@pytest.mark.parametrize("n,k", [(75, 128), (90, 200), (110, 192)])
def test_rows_behind_the_last_full_round(n, k):
    # more rows than CTAs at once, the rest of them few enough to be split in a launch of its own
    lengths = [1700, 2100]
    pages = 80
    table = Q.random_table(lengths, pages, 151)
    cache, scale = Q.filled_cache(pages, 152)
    req = [i % 2 for i in range(n)]
    pos = [lengths[r] - 1 - 3 * i for i, r in enumerate(req)]
    q = Q.rows((n, 64, 192), 153, 0.3)
    sel, cnt = Q.random_selection(pos, k, 154)
    out, lse = sparse(cache, scale, table, q, req, pos, sel, cnt)
    Q.check_attention(out, lse, reference(cache, scale, table, q, req, pos, Q.sel_tokens(sel, cnt, pos)))


def test_every_offset_of_the_own_region():
    pos = list(range(160, 176))
    sparse_case([176], 1, 81, pos, [0] * 16, prefill=True)
    sparse_case([176], 4, 82, pos, [0] * 16, prefill=True)


def test_rows_with_nothing_to_attend():
    # no selection, a selection wholly behind the query, a query before position 0
    pages = 5
    cache, scale = Q.filled_cache(pages, 83)
    table = Q.random_table([300], pages, 84)
    pos = [299, 100, -1, 40]
    q = Q.rows((4, 64, 192), 85, 0.3)
    sel, cnt = Q.random_selection([299, 100, 0, 40], 6, 86)
    cnt[0, 1] = 0
    sel[0, 1] = -1
    sel[1, 2] = [13, 14, 15, 16, 17, 18]
    cnt[1, 2] = 6
    out, lse = sparse(cache, scale, table, q, [0] * 4, pos, sel, cnt)
    Q.check_attention(out, lse, reference(cache, scale, table, q, [0] * 4, pos, Q.sel_tokens(sel, cnt, pos)))
    assert not out[0, 16:32].any() and torch.isinf(lse[0, 16:32]).all()
    assert not out[2].any() and not out[1, 32:48].any()


def poison(cache, scale, table, keep):
    """NaN codes at every token of the cache that `keep` [request] does not list, NaN scales on blocks with none."""
    good = np.zeros(tuple(cache.shape[:1]) + (64,), bool)
    for b, toks in enumerate(keep):
        toks = np.asarray(toks)
        good[np.asarray(table)[b, toks // 64], toks % 64] = True
    good = torch.from_numpy(good).view(-1, 1, 8, 1, 8, 1)
    cache = torch.where(good, cache, torch.full_like(cache, 0x7F))
    scale = torch.where(good.any(4)[..., 0], scale, torch.full_like(scale, float("nan")))
    return cache.contiguous(), scale.contiguous()


def test_masked_tokens_may_hold_nan():
    lengths = [1003, 70]
    pages = 20
    table = Q.random_table(lengths, pages, 87)
    cache, scale = Q.filled_cache(pages, 88)
    pos = [1002, 69]
    q = Q.rows((2, 64, 192), 89, 0.3)
    sel, cnt = Q.random_selection(pos, 30, 90)
    sel[:, 1:] = sel[:, :1]                                        # one selection for all groups, so the rest is unread
    cnt[:, 1:] = cnt[:, :1]
    tok = Q.sel_tokens(sel, cnt, pos)
    ref = reference(cache, scale, table, q, [0, 1], pos, tok)
    pc, ps = poison(cache, scale, table, [tok(0, 0), tok(1, 0)])
    out, lse = sparse(pc, ps, table, q, [0, 1], pos, sel, cnt, prefill=False)
    Q.check_attention(out, lse, ref)
    # the window's both ends inside a region
    for w in (1, 5, 60, 100):
        tok = Q.window_tokens(pos, w)
        ref = reference(cache, scale, table, q, [0, 1], pos, tok)
        pc, ps = poison(cache, scale, table, [tok(0, 0), tok(1, 0)])
        out, lse = window(pc, ps, table, q, None, pos, w)
        Q.check_attention(out, lse, ref)


def window(cache, scale, table, q, req, pos, w, check=True):
    lse = torch.empty((len(pos), 64), dtype=torch.float32, device="cuda")
    out = dsa.window_attn_quant(q.cuda(), cache.cuda(), scale.cuda(), to(table), to(pos), w,
                                q_req=None if req is None else to(req), lse=lse)
    if check:
        dsa.check_device()
    return out, lse


@pytest.mark.parametrize("w", [1, 2, 7, 8, 9, 63, 64, 65, 100, 512, 1000, 4096])
def test_window_decode(w):
    lengths = [1, 8, 200, 511, 512, 513, 2500]
    pages = sum((L + 63) // 64 for L in lengths)
    table = Q.random_table(lengths, pages, w)
    cache, scale = Q.filled_cache(pages, 91 + w)
    pos = [L - 1 for L in lengths]
    q = Q.rows((len(pos), 64, 192), 92 + w, 0.3)
    out, lse = window(cache, scale, table, q, None, pos, w)
    Q.check_attention(out, lse, reference(cache, scale, table, q, range(len(pos)), pos, Q.window_tokens(pos, w)))


@pytest.mark.parametrize("batch,w", [(8, 512), (8, 520), (1, 9), (3, 64), (40, 100)])
def test_many_short_calls_in_a_row(batch, w):
    # calls of a few microseconds one behind another, their last tiles of one to four steps: every
    # one of them ends, and the last gives what the first gave
    pages = 12 * batch
    table = np.arange(pages).reshape(batch, 12)
    cache, scale = Q.filled_cache(pages, 301)
    pos = [700 + i % 9 for i in range(batch)]
    args = (Q.rows((batch, 64, 192), 302, 0.3).cuda(), cache.cuda(), scale.cuda(), to(table), to(pos), w)
    first = dsa.window_attn_quant(*args)
    out = torch.empty_like(first)
    for i in range(20000):
        dsa.window_attn_quant(*args, out=out)
        if i % 1000 == 999:
            torch.cuda.synchronize()
    dsa.check_device()
    assert torch.equal(out, first)


def test_window_chunk_of_one_request():
    pages = 12
    table = Q.random_table([700], pages, 93)
    cache, scale = Q.filled_cache(pages, 94)
    for n in (150, 203):                                            # row by row; shared
        pos = list(range(700 - n, 700))
        q = Q.rows((n, 64, 192), 95, 0.3)
        out, lse = window(cache, scale, table, q, [0] * n, pos, 512)
        Q.check_attention(out, lse, reference(cache, scale, table, q, [0] * n, pos, Q.window_tokens(pos, 512)))


def test_window_chunk_into_an_output_of_eight_byte_alignment():
    # (the C call takes it; 16-byte stores would fault or split rows)
    pages, n, w = 6, 200, 100
    table = Q.random_table([300], pages, 136)
    cache, scale = Q.filled_cache(pages, 137)
    pos = list(range(100, 300))
    q = Q.rows((n, 64, 192), 138, 0.3)
    want, _ = window(cache, scale, table, q, [0] * n, pos, w)
    raw = torch.zeros(n * 64 * 192 + 4, dtype=torch.bfloat16, device="cuda")
    c, s, bt, p, r, qq = cache.cuda(), scale.cuda(), to(table), to(pos), to([0] * n), q.cuda()
    st = dsa.lib().dsa_window_attn_quant(qq.data_ptr(), c.data_ptr(), s.data_ptr(), pages, bt.data_ptr(), table.shape[1],
                                         1, r.data_ptr(), p.data_ptr(), n, w, raw.data_ptr() + 8, None, dsa._stream())
    assert st == dsa.OK
    dsa.check_device()
    assert torch.equal(raw[4:].view(n, 64, 192), want) and not raw[:4].any()


@pytest.mark.parametrize("w", [1, 9, 64, 100, 512])
def test_window_chunks_of_several_requests(w):
    # lists whose neighbours share windows, or do not: two requests' chunks one behind the other
    # (ends inside a block of 8), far positions, a descending stretch, the same position twice, padding
    pages = 30
    table = Q.random_table([900, 400], pages, w)
    cache, scale = Q.filled_cache(pages, w + 1)
    pos = list(range(100)) + list(range(700, 741)) + list(range(260, 300)) + [5, 890, 5, 890, 300, 299, 298, 297, 64, 64, -1, 64, -1, -1, 399]
    req = [0] * 141 + [1] * 40 + [0, 0, 1, 0, 1, 1, 1, 1, 0, 0, 0, 0, 1, 1, 1]
    q = Q.rows((len(pos), 64, 192), w + 2, 0.3)
    out, lse = window(cache, scale, table, q, req, pos, w)
    ref = reference(cache, scale, table, q, req, pos, Q.window_tokens(pos, w))
    Q.check_attention(out, lse, ref)
    for i, p in enumerate(pos):
        if p < 0:
            assert not out[i].any() and torch.isinf(lse[i]).all()


def test_rows_without_tokens_between_others():
    # more rows than CTAs at once (each runs through several), one and two and none of them with tokens
    pages, n, w = 4, 185, 1
    table = Q.random_table([200], pages, 139)
    cache, scale = Q.filled_cache(pages, 140)
    pos = [-1 if i % 5 in (1, 2, 4) or 60 < i < 140 else i for i in range(n)]
    q = Q.rows((n, 64, 192), 141, 0.3)
    for _ in range(5):
        out, lse = window(cache, scale, table, q, [0] * n, pos, w)
        Q.check_attention(out, lse, reference(cache, scale, table, q, [0] * n, pos, Q.window_tokens(pos, w)))
    sel, cnt = Q.random_selection([max(p, 0) for p in pos], 3, 142)
    out, lse = sparse(cache, scale, table, q, [0] * n, pos, sel, cnt)
    Q.check_attention(out, lse, reference(cache, scale, table, q, [0] * n, pos, Q.sel_tokens(sel, cnt, pos)))


def test_nan_at_a_token_that_some_of_a_chunk_attend():
    # V of two tokens: the newest one (the last query alone attends it) and the oldest of the first
    # query's window; the rest of the 8 stay finite
    pages = 14
    table = Q.random_table([800], pages, 130)
    cache, scale = Q.filled_cache(pages, 131)
    n = 200
    pos = list(range(544, 744))
    q = Q.rows((n, 64, 192), 132, 0.3)
    for t, dim in ((743, 3), (544 - 511, 5)):
        cache[table[0, t // 64], :, t % 64 // 8, 1, t % 8, dim] = 0x7F
    out, lse = window(cache, scale, table, q, [0] * n, pos, 512)
    nan = torch.isnan(out)
    assert nan[n - 1, :, 3].all() and nan[0, :, 5].all() and int(nan.sum()) == 2 * 64
    # all else is what it is with a zero in their place
    for t, dim in ((743, 3), (544 - 511, 5)):
        cache[table[0, t // 64], :, t % 64 // 8, 1, t % 8, dim] = 0
    ref = reference(cache, scale, table, q, [0] * n, pos, Q.window_tokens(pos, 512))
    for i, dim in ((n - 1, 3), (0, 5)):
        out[i, :, dim] = torch.from_numpy(ref[0][i, :, dim]).to(out)
    Q.check_attention(out, lse, ref)


def test_bad_pages_and_requests_in_a_chunk():
    pages = 10
    table = Q.random_table([500], pages, 133)
    cache, scale = Q.filled_cache(pages, 134)
    pos = list(range(290, 490))
    req = [0] * 200
    q = Q.rows((200, 64, 192), 135, 0.3)
    bad = table.copy()
    bad[0, 5] = pages                                              # tokens 320 .. 383
    out, lse = window(cache, scale, bad, q, req, pos, 200, check=False)
    with pytest.raises(dsa.DsaError):
        dsa.check_device()
    tok = Q.window_tokens(pos, 200)
    Q.check_attention(out, lse, reference(cache, scale, table, q, req, pos,
                                          lambda i, g: tok(i, g)[tok(i, g) // 64 != 5]))
    req[11] = 1                                                    # no such request: that query alone
    out, lse = window(cache, scale, table, q, req, pos, 200, check=False)
    with pytest.raises(dsa.DsaError):
        dsa.check_device()
    Q.check_attention(out, lse, reference(cache, scale, table, q, [0] * 200, pos,
                                          lambda i, g: tok(i, g)[:0] if i == 11 else tok(i, g)))
    out, lse = window(cache, scale, table[:, :7], q, [0] * 200, pos, 200, check=False)       # the table ends at token 447
    with pytest.raises(dsa.DsaError):
        dsa.check_device()
    Q.check_attention(out, lse, reference(cache, scale, table, q, [0] * 200, pos, lambda i, g: tok(i, g)[tok(i, g) < 448]))


def test_window_over_a_ring():
    ring = 9
    table = (np.arange(2)[:, None] * ring + np.arange(2000)[None] % ring).astype(np.int32)
    cache, scale = Q.filled_cache(2 * ring, 96)
    pos = [100003, 577]
    q = Q.rows((2, 64, 192), 97, 0.3)
    out, lse = window(cache, scale, table, q, None, pos, 512)
    Q.check_attention(out, lse, reference(cache, scale, table, q, [0, 1], pos, Q.window_tokens(pos, 512)))


@pytest.mark.parametrize("kind", ["not powers", "spread", "v spread", "growing k", "zero v", "zero k", "zero q",
                                  "tiny", "huge v", "outlier q"])
def test_scales_and_values_of_every_kind(kind):
    lengths = [700, 333]
    pages = 18
    table = Q.random_table(lengths, pages, 98)
    cache, scale = Q.filled_cache(pages, 99)
    q = Q.rows((2, 64, 192), 100, 0.3)
    gen = torch.Generator().manual_seed(5)
    if kind == "not powers":
        scale = scale * (0.6 + 0.9 * torch.rand(scale.shape, generator=gen))
    elif kind == "spread":
        scale = scale * torch.exp2(torch.randint(-6, 3, scale.shape, generator=gen).float())
    elif kind == "v spread":
        scale[..., 1] *= torch.exp2(torch.randint(-40, 41, scale[..., 1].shape, generator=gen).float())
    elif kind == "growing k":
        order = torch.from_numpy(table[0]).long()
        scale[order, ..., 0] *= torch.linspace(0.2, 6.0, len(order)).view(-1, 1, 1)
    elif kind == "zero v":
        scale[..., 1] = 0
    elif kind == "zero k":
        cache[:, :, :, 0] = 0
        scale[..., 0] = 0
    elif kind == "zero q":
        q[:, ::2] = 0
    elif kind == "tiny":
        q = (q.float() * 1e-30).to(torch.bfloat16)
        scale[..., 1] = 2.0 ** -126
    elif kind == "huge v":
        scale[..., 1] = 2.0 ** 110
    elif kind == "outlier q":
        q[:, :, 3] *= 4096
        cache[:, :, :, 0, :, 3] = 0
    pos = [699, 332]
    sel, cnt = Q.random_selection(pos, 64, 101)
    out, lse = sparse(cache, scale, table, q, [0, 1], pos, sel, cnt, prefill=False)
    Q.check_attention(out, lse, reference(cache, scale, table, q, [0, 1], pos, Q.sel_tokens(sel, cnt, pos)))


def test_nan_of_an_attended_token_reaches_its_heads_alone():
    pages = 4
    table = Q.random_table([200], pages, 102)
    cache, scale = Q.filled_cache(pages, 103)
    pos = [199]
    q = Q.rows((1, 64, 192), 104, 0.3)
    sel, cnt = Q.random_selection(pos, 25, 105)
    clean, lse0 = sparse(cache, scale, table, q, [0], pos, sel, cnt)
    page, r = table[0, 199 // 64], 199 % 64 // 8
    cache[page, 1, r, 1, 7, 33] = 0x7F                             # V: one dim of group 1
    cache[page, 2, r, 0, 7, 50] = 0xFF                             # K: every dim of group 2
    out, lse = sparse(cache, scale, table, q, [0], pos, sel, cnt)
    nan = torch.isnan(out[0])
    assert nan[16:32, 33].all() and nan[32:48].all() and torch.isnan(lse[0, 32:48]).all()
    nan[16:32, 33] = False
    nan[32:48] = False
    assert not nan.any()
    assert torch.equal(out[0, :16], clean[0, :16]) and torch.equal(out[0, 48:], clean[0, 48:])


@pytest.mark.parametrize("what", ["region", "negative region", "page", "request", "count"])
def test_bad_indices_are_flagged_and_skipped(what):
    pages = 10
    table = Q.random_table([500], pages, 106)
    cache, scale = Q.filled_cache(pages, 107)
    pos = [499, 450]
    req = [0, 0]
    q = Q.rows((2, 64, 192), 108, 0.3)
    sel, cnt = Q.random_selection(pos, 20, 109)
    good_sel, good_cnt = sel.copy(), cnt.copy()
    if what == "region":
        sel[0, 1, 3] = 99999
    elif what == "negative region":
        sel[0, 1, 3] = -5
    elif what == "page":
        table = table.copy()
        bad = int(sel[0, 0, 5]) // 8
        table[0, bad] = pages
    elif what == "request":
        req = [1, 0]
    elif what == "count":
        cnt[0, 1] = 21
    out, lse = sparse(cache, scale, table, q, req, pos, sel, cnt, check=False)
    with pytest.raises(dsa.DsaError):
        dsa.check_device()

    def tokens(i, g):
        r = good_sel[i, g, :good_cnt[i, g]].astype(np.int64)
        if what in ("region", "negative region") and (i, g) == (0, 1):
            r = np.delete(r, 3)
        if what == "page":
            r = r[r // 8 != bad]
        if what == "request" and i == 0:
            r = r[:0]
        t = (r[:, None] * 8 + np.arange(8)).ravel()
        return t[t <= pos[i]]
    Q.check_attention(out, lse, reference(cache, scale, table, q, [0, 0], pos, tokens))


def test_pages_behind_four_gigabytes():
    pages = (1 << 32) // (4 * 8 * 2 * 8 * 192) + 40
    small, sscale = Q.filled_cache(6, 110)
    cache, scale = dsa.quant_cache(pages)
    cache[-6:] = small.cuda()
    scale[-6:] = sscale.cuda()
    table = Q.random_table([380], 6, 111)
    pos = [379]
    q = Q.rows((1, 64, 192), 112, 0.3)
    sel, cnt = Q.random_selection(pos, 40, 113)
    lse = torch.empty((1, 64), dtype=torch.float32, device="cuda")
    out = dsa.sparse_attn_decode_quant(q.cuda(), cache, scale, to(table + pages - 6), to(pos), to(sel), to(cnt), lse=lse)
    dsa.check_device()
    Q.check_attention(out, lse, Q.attention(q.double().numpy(), small.numpy(), sscale.numpy(), table, [0], pos,
                                            Q.sel_tokens(sel, cnt, pos)))


def test_rows_do_not_depend_on_the_rest_of_the_call():
    # the same query alone, in a small batch and in a large one: 2^-8 for each bf16 rounding (the
    # split of a row over CTAs may differ), and twice the same call bit for bit
    pages = 40
    table = Q.random_table([2500], pages, 114)
    cache, scale = Q.filled_cache(pages, 115)
    pos = (np.arange(200) * 12 + 100).tolist()
    q = Q.rows((200, 64, 192), 116, 0.3)
    sel, cnt = Q.random_selection(pos, 128, 117)
    full, lse = sparse(cache, scale, table, q, [0] * 200, pos, sel, cnt)
    again, lse2 = sparse(cache, scale, table, q, [0] * 200, pos, sel, cnt)
    assert torch.equal(full, again) and torch.equal(lse, lse2)
    for n in (1, 3, 20):
        part, l = sparse(cache, scale, table, q[-n:], [0] * n, pos[-n:], sel[-n:], cnt[-n:])
        ref = reference(cache, scale, table, q[-n:], [0] * n, pos[-n:], Q.sel_tokens(sel[-n:], cnt[-n:], pos[-n:]))
        Q.check_attention(part, l, ref)
        Q.check_attention(full[-n:], lse[-n:], ref)


def test_streams_and_graphs_at_once():
    # two captured graphs and an eager call, replayed on streams of their own at the same time
    lengths = [3000, 1777]
    pages = 80
    table = Q.random_table(lengths, pages, 118)
    cache, scale = Q.filled_cache(pages, 119)
    pos = [2999, 1776]
    q = Q.rows((2, 64, 192), 120, 0.3)
    sel, cnt = Q.random_selection(pos, 200, 121)
    want, wl = sparse(cache, scale, table, q, [0, 1], pos, sel, cnt, prefill=False)
    c, s, bt, p, qq, si, sc = cache.cuda(), scale.cuda(), to(table), to(pos), q.cuda(), to(sel), to(cnt)
    wwant = dsa.window_attn_quant(qq, c, s, bt, p, 512)
    torch.cuda.synchronize()
    outs, graphs = [], []
    for _ in range(2):
        o, l = torch.empty_like(want), torch.empty_like(wl)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            dsa.sparse_attn_decode_quant(qq, c, s, bt, p, si, sc, out=o, lse=l)
            w = dsa.window_attn_quant(qq, c, s, bt, p, 512)
        outs.append((o, l, w))
        graphs.append(gr)
    streams = [torch.cuda.Stream() for _ in range(3)]
    eager = torch.empty_like(want)
    torch.cuda.synchronize()
    for _ in range(5):
        for st, gr in zip(streams, graphs):
            with torch.cuda.stream(st):
                gr.replay()
        with torch.cuda.stream(streams[2]):
            dsa.sparse_attn_decode_quant(qq, c, s, bt, p, si, sc, out=eager)
    torch.cuda.synchronize()
    dsa.check_device()
    for o, l, w in outs:
        assert torch.equal(o, want) and torch.equal(l, wl) and torch.equal(w, wwant)
    assert torch.equal(eager, want)


def test_append_then_attend_as_a_decode_loop():
    # 12 steps of a ragged batch: append, sparse attention and window attention over what the
    # plain append holds
    lengths = [130, 64, 7]
    pages = 8
    table = Q.random_table(lengths, pages, 122, extra=12)
    c, s = dsa.quant_cache(pages)
    pc, ps = c.cpu().numpy(), s.cpu().double().numpy()
    req = [b for b, L in enumerate(lengths) for _ in range(L)]
    at = [t for L in lengths for t in range(L)]
    k, v = Q.rows((len(req), 4, 192), 123), Q.rows((len(req), 4, 192), 124)
    dsa.kv_append_quant(c, s, to(table), to(at), k.cuda(), v.cuda(), q_req=to(req))
    pc, ps = Q.append(pc, ps, table, req, at, k.double().numpy(), v.double().numpy())
    for step in range(12):
        pos = [L + step for L in lengths]
        k, v = Q.rows((3, 4, 192), 200 + step), Q.rows((3, 4, 192), 300 + step)
        q = Q.rows((3, 64, 192), 400 + step, 0.3)
        dsa.kv_append_quant(c, s, to(table), to(pos), k.cuda(), v.cuda())
        pc, ps = Q.append(pc, ps, table, [0, 1, 2], pos, k.double().numpy(), v.double().numpy())
        sel, cnt = Q.random_selection(pos, 10, step)
        lse = torch.empty((3, 64), dtype=torch.float32, device="cuda")
        out = dsa.sparse_attn_decode_quant(q.cuda(), c, s, to(table), to(pos), to(sel), to(cnt), lse=lse)
        Q.check_attention(out, lse, Q.attention(q.double().numpy(), pc, ps, table, [0, 1, 2], pos,
                                                Q.sel_tokens(sel, cnt, pos)))
        out = dsa.window_attn_quant(q.cuda(), c, s, to(table), to(pos), 50, lse=lse)
        Q.check_attention(out, lse, Q.attention(q.double().numpy(), pc, ps, table, [0, 1, 2], pos,
                                                Q.window_tokens(pos, 50)))
    dsa.check_device()
    assert np.array_equal(c.cpu().numpy(), pc) and np.array_equal(s.cpu().double().numpy(), ps)

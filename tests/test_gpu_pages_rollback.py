"""A request cut back inside a page that others hold too, and then appended to: by way of a fork, the
other holders' pages keep every byte and their attention every bit."""
import numpy as np
import pytest
import torch

from sparse_long_context_dsa_b200 import dsa

import _quant as Q

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def attend(c, s, t, row, length, seed=7):
    q = Q.rows((1, 64, 192), seed, 0.3)
    lse = torch.empty((1, 64), dtype=torch.float32, device="cuda")
    out = dsa.window_attn_quant(q.cuda(), c, s, t, i32([length - 1]), 400, q_req=i32([row]), lse=lse)
    return q, out, lse


@pytest.mark.parametrize("cut", ["child", "parent"])
@pytest.mark.parametrize("keep", [100, 64, 70, 255, 1])
def test_fork_cut_append(cut, keep):
    pages, L = 24, 256
    c, s = dsa.quant_cache(pages)
    table = np.full((4, 7), -1, np.int32)
    table[0, :4] = [9, 2, 17, 5]
    ref = np.zeros(pages, np.int32)
    ref[table[0, :4]] = 1
    r, t = i32(ref), i32(table)
    k, v = Q.rows((L, 4, 192), 1), Q.rows((L, 4, 192), 2)
    dsa.kv_append_quant(c, s, t, i32(range(L)), k.cuda(), v.cuda(), q_req=i32([0] * L))
    dsa.pages_fork(r, t, i32([0]), i32([1]), i32([L]), [c, s])      # all four pages shared
    held = table[0, :4].tolist()
    row, other = (1, 0) if cut == "child" else (0, 1)
    before = c[held].clone(), s[held].clone(), attend(c, s, t, other, L)
    # the row attends its first `keep` tokens as it is
    dsa.pages_release(r, t, i32([row]), i32([keep]))
    zero = np.zeros((4,) + tuple(c.shape[1:]), np.uint8), np.zeros((4,) + tuple(s.shape[1:]))
    plain = Q.append(*zero, [[0, 1, 2, 3]], [0] * L, list(range(L)), k.double().numpy(), v.double().numpy())
    q, out, lse = attend(c, s, t, row, keep)
    Q.check_attention(out, lse, Q.attention(q.double().numpy(), *plain, [[0, 1, 2, 3]], [0], [keep - 1],
                                            Q.window_tokens([keep - 1], 400)))
    # and goes on in a row of its own: 9 tokens, ten times as large (their blocks' scales rise)
    dsa.pages_fork(r, t, i32([row]), i32([2]), i32([keep]), [c, s])
    dsa.pages_release(r, t, i32([row]), i32([0]))
    dsa.check_device()
    nk, nv = Q.rows((9, 4, 192), 3) * 10, Q.rows((9, 4, 192), 4) * 10
    at = list(range(keep, keep + 9))
    for p in {x // 64 for x in at}:
        if int(t[2, p]) < 0:                                       # a page that begins with them
            free = int((r == 0).nonzero()[0])
            t[2, p], r[free] = free, 1
    dsa.kv_append_quant(c, s, t, i32(at), nk.cuda(), nv.cuda(), q_req=i32([2] * 9))
    dsa.check_device()
    assert torch.equal(c[held], before[0]) and torch.equal(s[held], before[1])
    _, out, lse = attend(c, s, t, other, L)
    assert torch.equal(out, before[2][1]) and torch.equal(lse, before[2][2])
    tab = [[0, 1, 2, 3, 4]]
    more = [np.concatenate([x, np.zeros((1,) + x.shape[1:], x.dtype)]) for x in plain]
    more = Q.append(*more, tab, [0] * 9, at, nk.double().numpy(), nv.double().numpy())
    q, out, lse = attend(c, s, t, 2, keep + 9)
    Q.check_attention(out, lse, Q.attention(q.double().numpy(), *more, tab, [0], [keep + 8], Q.window_tokens([keep + 8], 400)))
    dsa.check_device()
    counts = r.cpu().numpy()
    names = t.cpu().numpy()
    assert np.array_equal(np.bincount(names[names >= 0], minlength=pages), counts)

"""The bound on q's two e4m3 terms, reached: 2^-e q = hi + lo with e4m3's subnormal step 2^-9, the head's
largest of 2^-e q in (224, 448].  Its bf16 elements have 8 significant bits, of which hi takes 4 and lo
the rest exactly, unless they end below the step: lo is off by at most half a step, 2^-10, relative to a
largest above 224 2^-10 / 224 < 2^-17.  The row kernel's second term is 16 lo: 2^-14 / 224 < 2^-21."""
import numpy as np
import pytest
import torch

from sparse_long_context_dsa_b200 import dsa

import _quant as Q

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def case(small, n, off):
    """n queries of one request, each head 225 and 191 elements `small`, over keys of one sign (0 where
    the 225 is): every element's error adds up.  Returns the call's lse error and the bound's tolerance."""
    pages, L = 4, 200
    table = Q.random_table([L], pages, 1)
    cache, scale = Q.filled_cache(pages, 2, 0.0)
    cache[:, :, :, 0] = 0x7E                                       # K: 448 times the scale
    cache[:, :, :, 0, :, 0] = 0
    scale[..., 0] = 2.0 ** -9
    q = torch.full((n, 64, 192), small, dtype=torch.bfloat16)
    q[..., 0] = 225.0
    assert float(q[0, 0, 1]) == small
    pos = [L - 1 - i % 50 for i in range(n)]
    lse = torch.empty((n, 64), dtype=torch.float32, device="cuda")
    out = dsa.window_attn_quant(q.cuda(), cache.cuda(), scale.cuda(), i32(table), i32(pos), 150, q_req=i32([0] * n), lse=lse)
    dsa.check_device()
    ref = Q.attention(q.double().numpy(), cache.numpy(), scale.numpy(), table, [0] * n, pos, Q.window_tokens(pos, 150), off)
    Q.check_attention(out, lse, ref)
    return np.abs(lse.cpu().double().numpy() - ref[1]).max(), 191 * 448 * 2.0 ** -9 / np.sqrt(192)


def shared(n):
    return n * 4 > 2 * torch.cuda.get_device_properties(0).multi_processor_count


def test_shared_windows_of_a_chunk():
    # 2.5 steps: hi = 2 (ties to even), lo = 0: off by half a step, 2^-10
    n = 80
    assert shared(n)
    err, sum_k = case(2.5 * 2.0 ** -9, n, 2.0 ** -17)
    assert 0.99 * 2.0 ** -10 * sum_k < err < 1.01 * 2.0 ** -10 * sum_k
    # which is above 2^-18 of the largest
    assert err > 2.0 ** -18 * 225 * sum_k


def test_rows_by_themselves():
    n = 3
    assert not shared(n)
    err, sum_k = case(2.5 * 2.0 ** -9, n, 2.0 ** -21)              # exact: 16 lo = 8 steps
    err2, _ = case(2.5 * 2.0 ** -13, n, 2.0 ** -21)                # 16 lo = 2.5 steps: off by half of one, 2^-14
    assert 0.99 * 2.0 ** -14 * sum_k < err2 < 1.01 * 2.0 ** -14 * sum_k
    assert err < 2.0 ** -16 * sum_k


@pytest.mark.parametrize("k", [20, 130])
def test_random_queries_of_the_row_kernel_within_its_own_bound(k):
    lengths = [1100, 300]
    pages = 24
    table = Q.random_table(lengths, pages, 3)
    cache, scale = Q.filled_cache(pages, 4)
    pos = [1099, 299]
    q = Q.rows((2, 64, 192), 5, 0.3)
    sel, cnt = Q.random_selection(pos, k, 6)
    lse = torch.empty((2, 64), dtype=torch.float32, device="cuda")
    out = dsa.sparse_attn_decode_quant(q.cuda(), cache.cuda(), scale.cuda(), i32(table), i32(pos), i32(sel), i32(cnt), lse=lse)
    dsa.check_device()
    Q.check_attention(out, lse, Q.attention(q.double().numpy(), cache.numpy(), scale.numpy(), table, [0, 1], pos,
                                            Q.sel_tokens(sel, cnt, pos), 2.0 ** -21))

"""The 8-bit attention at the ends of the scales' range, against the same in 64 bits (tolerances:
_quant.attention)."""
import numpy as np
import pytest
import torch

from sparse_long_context_dsa_b200 import dsa

import _quant as Q

pytestmark = pytest.mark.gpu


def to(x, dtype=torch.int32):
    return torch.tensor(np.asarray(x), dtype=dtype, device="cuda")


def attend(cache, scale, table, q, pos, w=None, sel=None, cnt=None):
    """Every query of request 0: over its window, or over a selection."""
    n = len(pos)
    lse = torch.empty((n, 64), dtype=torch.float32, device="cuda")
    args = (q.cuda(), cache.cuda(), scale.cuda(), to(table))
    if w is not None:
        out = dsa.window_attn_quant(*args, to(pos), w, q_req=to([0] * n), lse=lse)
    else:
        out = dsa.sparse_attn_prefill_quant(*args, to([0] * n), to(pos), to(sel), to(cnt), lse=lse)
    dsa.check_device()
    return out, lse


@pytest.mark.parametrize("n", [1, 80])
@pytest.mark.parametrize("up,down", [("k", "q"), ("q", "k")])
def test_scales_whose_product_is_ordinary(n, up, down):
    # keys of 2^119 and queries of 2^-119, and the other way round: their products are of order 1
    pages, L = 6, 380
    table = Q.random_table([L], pages, 1)
    cache, scale = Q.filled_cache(pages, 2, 0.0)
    k_exp = 119.0 if up == "k" else -119.0
    scale[..., 0] = 2.0 ** (k_exp - 7)                             # codes are some 2^7
    q = (Q.rows((n, 64, 192), 3, 0.0).double() * 0.3 * 2.0 ** -k_exp).to(torch.bfloat16)
    pos = [L - 1 - i % 40 for i in range(n)]
    sel, cnt = Q.random_selection(pos, 40, 4)
    qd = q.double().numpy()
    out, lse = attend(cache, scale, table, q, pos, sel=sel, cnt=cnt)
    Q.check_attention(out, lse, Q.attention(qd, cache.numpy(), scale.numpy(), table, [0] * n, pos, Q.sel_tokens(sel, cnt, pos)))
    out, lse = attend(cache, scale, table, q, pos, w=200)
    Q.check_attention(out, lse, Q.attention(qd, cache.numpy(), scale.numpy(), table, [0] * n, pos, Q.window_tokens(pos, 200)))


def whole(n, pos):
    """Selections of every region up to the query's own."""
    sel = np.tile(np.arange(pos // 8 + 1, dtype=np.int32), (n, 4, 1))
    return sel, np.full((n, 4), pos // 8 + 1, np.int32)


@pytest.mark.parametrize("n", [1, 75])
@pytest.mark.parametrize("kind", ["selection", "window"])
def test_smallest_values_over_many_tokens(kind, n):
    # 15,887 tokens of equal weight, values at the smallest scale and of one sign: the weights' sum times
    # 2^126 passes the numbers' range, the outputs (some 2^-119) do not
    L = 15887
    pages = (L + 63) // 64
    table = Q.random_table([L], pages, 5)
    cache, scale = Q.filled_cache(pages, 6, 0.0)
    cache &= 0x7F
    scale[..., 1] = 2.0 ** -126
    q = torch.zeros((n, 64, 192), dtype=torch.bfloat16)
    pos = [L - 1] * n
    sel, cnt = whole(n, L - 1)
    out, lse = attend(cache, scale, table, q, pos, w=L) if kind == "window" else attend(cache, scale, table, q, pos, sel=sel, cnt=cnt)
    ref = Q.attention(q[:1].double().numpy(), cache.numpy(), scale.numpy(), table, [0], pos[:1], Q.sel_tokens(sel, cnt, pos))
    Q.check_attention(out[:1], lse[:1], ref)
    assert torch.equal(out, out[:1].expand_as(out)) and torch.equal(lse, lse[:1].expand_as(lse))

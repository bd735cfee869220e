"""The 8-bit cache's host side, without a GPU: the plain forms that the GPU tests compare with, and
the refusals of the calls and of the binding."""
import numpy as np
import pytest
import torch

from sparse_long_context_dsa_b200 import build as B
from sparse_long_context_dsa_b200 import dsa

import _quant as Q


@pytest.fixture(scope="module")
def lib():
    B.build()
    return dsa.lib()


def test_code_values_are_the_formats():
    v = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(v), np.isnan(Q.VALUE)) and np.array_equal(v[~np.isnan(v)], Q.VALUE[~np.isnan(v)])


def test_codes_round_to_nearest_even():
    x = np.concatenate([np.linspace(-448, 448, 20001), Q.VALUE[:0x7F], (Q.VALUE[:0x7E] + Q.VALUE[1:0x7F]) / 2])
    want = torch.from_numpy(x).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(Q.e4m3_codes(x.astype(np.float32).astype(np.float64)), want)


def test_block_scale_is_the_smallest_power():
    assert Q.block_scale(448.0) == 1.0 and Q.block_scale(448.001) == 2.0 and Q.block_scale(224.0) == 0.5
    assert Q.block_scale(1e-40) == 2.0 ** -126 and Q.block_scale(np.inf) == 2.0 ** 120 and Q.block_scale(0.0) == 0.0


def test_a_cache_filled_token_by_token_is_one_filled_at_once():
    # powers of two: raising a scale shifts exponents, so the codes are the same unless the
    # value is an e4m3 subnormal of the final scale (there, two roundings may differ by one step)
    x = Q.rows((REGION_TOKENS, Q.G, Q.D), 1).double().numpy()
    y = Q.rows((REGION_TOKENS, Q.G, Q.D), 2).double().numpy()
    empty = np.zeros((1, Q.G, 8, 2, 8, Q.D), np.uint8), np.zeros((1, Q.G, 8, 2))
    table = [[0]]
    at_once = Q.append(*empty, table, [0] * 8, list(range(8)), x, y)
    c, s = empty
    for t in range(8):
        c, s = Q.append(c, s, table, [0], [t], x[t:t + 1], y[t:t + 1])
    assert np.array_equal(s, at_once[1])
    a, b = Q.VALUE[c], Q.VALUE[at_once[0]]
    assert np.array_equal(a[np.abs(b) >= 2.0 ** -6], b[np.abs(b) >= 2.0 ** -6])
    assert np.abs(a - b).max() <= 2.0 ** -9


REGION_TOKENS = 8


def test_attention_plain_form_is_the_oracles_on_exact_values(oracle_lib):
    # code * scale is exactly bf16, so the oracle's bf16 attention is this one
    lengths = [200, 77]
    table = Q.random_table(lengths, 8, 3)
    cache, scale = Q.filled_cache(8, 4)
    val = cache.view(torch.float8_e4m3fn).float() * scale[..., None, None]      # [p][4][8][2][8][192]
    bits = val.to(torch.bfloat16)
    assert torch.equal(bits.float(), val)
    bits = bits.view(torch.int16).numpy().view(np.uint16)
    kc, vc = (np.ascontiguousarray(bits[:, :, :, t].reshape(8, 4, 64, Q.D)) for t in (0, 1))
    q = Q.rows((2, 64, Q.D), 5, 0.0)
    pos = np.array([199, 76], np.int32)
    sel, cnt = Q.random_selection(pos, 6, 6)
    o, l, o64 = oracle_lib.sparse_attention(q.view(torch.int16).numpy().view(np.uint16), kc, vc,
                                            np.maximum(table, 0), np.arange(2, dtype=np.int32), pos, sel, cnt,
                                            want_f64=True)
    out, lse, _, _ = Q.attention(q.double().numpy(), cache.numpy(), scale.numpy(), table, [0, 1], pos,
                                 Q.sel_tokens(sel, cnt, pos))
    np.testing.assert_allclose(out, o64, rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(lse, l, rtol=1e-6)


P = 1 << 20                        # an address that is never read: these calls return before any device access


@pytest.mark.parametrize("call,word", [
    (lambda L: L.dsa_kv_append_quant(P, P, 1, P, 1, 1, None, P, -1, P, P, None), "n must"),
    (lambda L: L.dsa_kv_append_quant(P, P, 0, P, 1, 1, None, P, 1, P, P, None), "n_pages"),
    (lambda L: L.dsa_kv_append_quant(P, P, 1 << 31, P, 1, 1, None, P, 1, P, P, None), "n_pages"),
    (lambda L: L.dsa_kv_append_quant(P, P, 1, P, 0, 1, None, P, 1, P, P, None), "max_pages"),
    (lambda L: L.dsa_kv_append_quant(P, P, 1, P, 1 << 25, 1, None, P, 1, P, P, None), "max_pages"),
    (lambda L: L.dsa_kv_append_quant(P, P, 1, P, 1, 0, P, P, 1, P, P, None), "n_req"),
    (lambda L: L.dsa_kv_append_quant(None, P, 1, P, 1, 1, None, P, 1, P, P, None), "NULL"),
    (lambda L: L.dsa_kv_append_quant(P, P, 1, P, 1, 1, None, P, 1, None, P, None), "NULL"),
    (lambda L: L.dsa_kv_append_quant(P + 8, P, 1, P, 1, 1, None, P, 1, P, P, None), "aligned"),
    (lambda L: L.dsa_kv_append_quant(P, P, 1, P, 1, 1, None, P, 1, P + 8, P, None), "aligned"),
    (lambda L: L.dsa_sparse_attn_decode_quant(P, P, P, 1, P, 1, P, -1, P, P, 8, P, None, None), "nq"),
    (lambda L: L.dsa_sparse_attn_decode_quant(P, P, P, 1, P, 1, P, (1 << 24) + 1, P, P, 8, P, None, None), "nq"),
    (lambda L: L.dsa_sparse_attn_decode_quant(P, P, P, 1, P, 1, P, 1, P, P, 0, P, None, None), "k out"),
    (lambda L: L.dsa_sparse_attn_decode_quant(P, P, P, 1, P, 1, P, 1, P, P, 2049, P, None, None), "k out"),
    (lambda L: L.dsa_sparse_attn_decode_quant(P, P, P, 1, P, 1, P, 1, None, P, 8, P, None, None), "NULL"),
    (lambda L: L.dsa_sparse_attn_decode_quant(P, P, P, 1, P, 1, P, 1, P, P, 8, P + 4, None, None), "aligned"),
    (lambda L: L.dsa_sparse_attn_prefill_quant(P, P, P, 1, P, 1, 1, None, P, 1, P, P, 8, P, None, None), "q_req"),
    (lambda L: L.dsa_sparse_attn_prefill_quant(P, P, P, 1, P, 1, 0, P, P, 1, P, P, 8, P, None, None), "n_req"),
    (lambda L: L.dsa_window_attn_quant(P, P, P, 1, P, 1, 1, None, P, 1, 0, P, None, None), "window"),
    (lambda L: L.dsa_window_attn_quant(P, P, P, 1, P, 1, 1, None, P, 1, (1 << 20) + 1, P, None, None), "window"),
    (lambda L: L.dsa_window_attn_quant(P, P, P + 4, 1, P, 1, 1, None, P, 1, 8, P, None, None), "aligned"),
])
def test_bad_arguments_are_rejected_on_the_host(lib, call, word):
    assert call(lib) == dsa.ERR_INVALID_ARG
    assert word in lib.dsa_last_error().decode()


def test_zero_sized_calls_are_noops(lib):
    assert lib.dsa_kv_append_quant(None, None, 1, None, 1, 0, None, None, 0, None, None, None) == dsa.OK
    assert lib.dsa_sparse_attn_decode_quant(None, None, None, 1, None, 1, None, 0, None, None, 8, None, None,
                                            None) == dsa.OK
    assert lib.dsa_window_attn_quant(None, None, None, 1, None, 1, 0, None, None, 0, 512, None, None, None) == dsa.OK


def test_host_tensors_are_refused():
    cache, scale = dsa.quant_cache(1, "cpu")
    bt = torch.zeros((1, 1), dtype=torch.int32)
    row = torch.zeros((1, 4, 192), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        dsa.kv_append_quant(cache, scale, bt, torch.zeros(1, dtype=torch.int32), row, row)

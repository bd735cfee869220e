"""Plain forms of the 8-bit cache and its attention in 64 bits, for the tests (numpy, CPU)."""
import math

import numpy as np
import torch

G, PAGE, REGION, D, HQ = 4, 64, 8, 192, 64


def e4m3_values():
    """The 256 code values (NaN for 0x7f, 0xff), from the format's definition."""
    v = np.empty(256)
    for c in range(256):
        s, e, m = -1.0 if c & 0x80 else 1.0, (c >> 3) & 15, c & 7
        v[c] = s * (math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10))
    v[0x7F] = v[0xFF] = np.nan
    return v


VALUE = e4m3_values()


def e4m3_codes(x):
    """Nearest e4m3 code of each x (float64, exact inputs), ties to even, saturating; NaN -> 0x7f."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(x), 448.0)
    pos = VALUE[:0x7F]                                            # ascending, code = index
    hi = np.searchsorted(pos, np.nan_to_num(a), side="left").clip(0, 0x7E)
    lo = np.maximum(hi - 1, 0)
    dl, dh = np.nan_to_num(a) - pos[lo], pos[hi] - np.nan_to_num(a)
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(np.isnan(x), 0x7F, code)
    return (code | np.where(np.signbit(x) & ~np.isnan(x), 0x80, 0)).astype(np.uint8)


def block_scale(a):
    """Smallest power of two s in [2^-126, 2^120] with a <= 448 s, 0 for a = 0, by search."""
    if a == 0:
        return 0.0
    for e in range(-126, 121):
        if a <= 448 * math.ldexp(1.0, e):
            return math.ldexp(1.0, e)
    return math.ldexp(1.0, 120)


def append(cache, scale, table, req, pos, new_k, new_v):
    """The call's effect on copies: cache uint8 and scale float64 arrays; new rows float64 [n][4][192].
    Entries are (req, pos) lists; runs as the call defines them."""
    cache, scale = cache.copy(), scale.copy()
    new = np.stack([new_k, new_v], 2)                             # [n][4][2][192]
    i, n = 0, len(pos)
    while i < n:
        j = i + 1
        while j < n and req[j] == req[i] and pos[j] // REGION == pos[i] // REGION:
            j += 1
        run = [i]                                                 # up to the first entry that does not ascend
        while run[-1] + 1 < j and pos[run[-1] + 1] > pos[run[-1]]:
            run.append(run[-1] + 1)
        page, r = table[req[i]][pos[i] // PAGE], pos[i] % PAGE // REGION
        first = pos[i] % REGION
        for g in range(G):
            for t in range(2):
                rows = new[run, g, t]
                fin = np.abs(rows[~np.isnan(rows)])
                old = float(scale[page, g, r, t]) if first else 0.0
                s = max(old, block_scale(fin.max() if fin.size else 0.0))
                if s > old and first:
                    cache[page, g, r, t, :first] = e4m3_codes(VALUE[cache[page, g, r, t, :first]] * (old / s))
                for x, e in zip(rows, run):
                    with np.errstate(invalid="ignore"):
                        y = x / s if s else np.where(np.isnan(x), x, x * 0.0)
                    cache[page, g, r, t, pos[e] % REGION] = e4m3_codes(y)
                scale[page, g, r, t] = s
        i = j
    return cache, scale


def attention(q, cache, scale, table, req, pos, tokens, q_off=2.0 ** -18):
    """Rows of 64-bit attention and the tolerances of the GPU's.  q float64 [nq][64][192]; tokens(i, g):
    positions attended by row (i, g).  Returns out, lse [nq][64], and out_tol, lse_tol.

    The tolerances count, per head: the score's error d (q as two e4m3 terms: off by at most q_off of the
    head's largest element, 2^-21 where the second term is 16 times finer and 2^-17 where it is not,
    as test_gpu_quant_bounds.py derives and checks; 192 fp32 sums; the scaled score and exp2's
    argument rounded), a weight's relative error 2 d (its own and the sum's), its rounding to fp16
    (2^-11) and from there to three e5m2 terms (of a weight in [1, 2) the first, cut off, leaves less
    than 2^-2, the second of that less than 2^-5, the third, rounded, at most 2^-9; all three end at the
    subnormal step 2^-16, half of which is 2^-22 of a largest weight that is at least 2^5), and the
    output's bf16 rounding (2^-8)."""
    nq = q.shape[0]
    out, lse = np.zeros((nq, HQ, D)), np.full((nq, HQ), -np.inf)
    out_tol, lse_tol = np.zeros((nq, HQ, D)), np.zeros((nq, HQ))
    for i in range(nq):
        for g in range(G):
            tok = np.asarray(tokens(i, g), np.int64)
            if tok.size == 0:
                continue
            page = np.asarray(table)[req[i], tok // PAGE]
            r, row = tok % PAGE // REGION, tok % REGION
            sc = scale[page, g, r].astype(np.float64)             # [T][2]
            k = VALUE[cache[page, g, r, 0, row]] * sc[:, :1]
            v = VALUE[cache[page, g, r, 1, row]] * sc[:, 1:]
            qq = q[i, 16 * g:16 * g + 16]
            s = qq @ k.T / math.sqrt(D)
            m = s.max(1, keepdims=True)
            w = np.exp(s - m)
            z = w.sum(1, keepdims=True)
            w = w / z
            h = slice(16 * g, 16 * g + 16)
            out[i, h] = w @ v
            lse[i, h] = (m + np.log(z))[:, 0]
            absqk = np.abs(qq) @ np.abs(k).T / math.sqrt(D)
            d = (q_off * np.abs(qq).max(1)[:, None] * np.abs(k).sum(1)[None] / math.sqrt(D) +
                 192 * 2.0 ** -24 * absqk).max(1) + 2.0 ** -20 * (np.abs(s).max(1) + 1)
            ws = w * sc[:, 1]                                     # weights of the codes
            rounding = (2.0 ** -9 + 2.0 ** -11) * ws + 2.0 ** -22 * ws.max(1, keepdims=True)
            spread = np.expm1(2 * d)[:, None] * (w @ np.abs(v)) + rounding @ np.abs(VALUE[cache[page, g, r, 1, row]])
            out_tol[i, h] = 2.0 ** -8 * np.abs(out[i, h]) + spread * (1 + 2.0 ** -7)
            lse_tol[i, h] = d + 2.0 ** -20 * (1 + np.abs(lse[i, h]))
    return out, lse, out_tol, lse_tol


def check_attention(got, lse_got, ref):
    out, lse, out_tol, lse_tol = ref
    o = got.float().cpu().numpy().astype(np.float64)
    l = lse_got.cpu().numpy().astype(np.float64)
    assert np.all(np.isfinite(o))
    err = np.abs(o - out)
    assert np.all(err <= out_tol), (err - out_tol).max()
    assert np.array_equal(np.isinf(l), np.isinf(lse))
    fin = np.isfinite(lse)
    e = np.abs(l[fin] - lse[fin])
    assert np.all(e <= lse_tol[fin]), (e - lse_tol[fin]).max()


def sel_tokens(sel, count, pos):
    def tokens(i, g):
        r = np.asarray(sel[i, g, :count[i, g]], np.int64)
        t = (r[:, None] * REGION + np.arange(REGION)).ravel()
        return t[t <= pos[i]]
    return tokens


def window_tokens(pos, window):
    return lambda i, g: np.arange(max(0, int(pos[i]) - window + 1), int(pos[i]) + 1)


def rows(shape, seed, spread=0.7):
    """bf16 rows N(0, 1), each with a gain exp(spread N(0, 1))."""
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=gen)
    return (x * torch.exp(spread * torch.randn(shape[:-1] + (1,), generator=gen))).to(torch.bfloat16)


def filled_cache(pages, seed, spread=0.7):
    """(cache uint8, scale float32) on the CPU: every block of rows() quantised by the definition."""
    x = rows((pages, G, PAGE // REGION, 2, REGION, D), seed, spread).float()
    a = x.abs().amax((-1, -2))
    m, e = torch.frexp(a)
    s = torch.ldexp(torch.ones_like(a), (e - 9 + (m > 0.875)).to(torch.int32))
    return (x / s[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8), s


def random_table(lengths, pages, seed, extra=0):
    rng = np.random.default_rng(seed)
    each = [(L + extra + PAGE - 1) // PAGE for L in lengths]
    order = rng.permutation(pages)
    table = np.full((len(lengths), max(each)), -1, np.int32)
    at = 0
    for b, n in enumerate(each):
        table[b, :n] = order[at:at + n]
        at += n
    return table


def random_selection(pos, k, seed):
    rng = np.random.default_rng(seed)
    nq = len(pos)
    idx = np.full((nq, G, k), -1, np.int32)
    cnt = np.zeros((nq, G), np.int32)
    for i, p in enumerate(pos):
        own = int(p) // REGION
        for g in range(G):
            n = min(k, own + 1)
            pick = rng.choice(own, size=n - 1, replace=False) if n > 1 else np.zeros(0, np.int64)
            idx[i, g, :n] = np.sort(np.concatenate([pick, [own]])).astype(np.int32)
            cnt[i, g] = n
    return idx, cnt

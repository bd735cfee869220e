"""Measured cases of the quantised K/V cache: appending to it, attending it, and moving its pages.

The cache holds K and V of one layer in 8 bits (e4m3) with one fp32 scale for every block of
8 tokens (a region), KV group and tensor:

  kv_cache     uint8 [pages][4][8][2][8][192]   page, group, region of the page, K|V, token, dim
  kv_scale     fp32  [pages][4][8][2]           value = e4m3(code) * scale
  block_table  int32 [requests][max_pages]      page of tokens 64 v .. 64 v + 63 of a request (-1: none)

A block's scale is the smallest power of two (in [2^-126, 2^120]) with max|x| <= 448 scale; 0
for a block of zeros.  Tokens that join a block later raise its scale if they need to, and the
codes already there are rounded again for the new scale.

Operators (`op` of a case):
  append   new tokens' K and V (bf16) quantised into the cache
  sparse   GQA (64 heads, 4 groups, d = 192) of each query over its selected regions
  window   GQA of each query over its last `window` tokens
  fork     requests forked: full pages shared (reference counts), the partly filled one copied
  compact  requests cut back to a length, their pages released, and the live pages moved together
"""
import math

import torch

own = False

REGION, G, HQ, D, PAGE = 8, 4, 64, 192, 64
RPP = PAGE // REGION                     # regions of a page
HPG = HQ // G                            # query heads of a group
DEV = "cuda"


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one decode step's new tokens of a small batch, in the window layers' rings
        dict(name="append_decode_b8", op="append", requests=8, tokens=8, ctx=131072, ring=9),
        # a prefill chunk that begins inside a region
        dict(name="append_chunk_2k", op="append", requests=1, tokens=2048, ctx=262141, ring=0),
        # a single request's decode step at a short context: latency
        dict(name="sparse_decode_b1_16k", op="sparse", requests=1, queries=1, lo=16384, hi=16384, k=512),
        # batched decode
        dict(name="sparse_decode_b8_128k", op="sparse", requests=8, queries=8, lo=131072, hi=131072, k=512),
        # ragged decode batch
        dict(name="sparse_decode_b32_ragged", op="sparse", requests=32, queries=32, lo=4096, hi=262144, k=512),
        # a prefill chunk's last queries, every one with its own selection
        dict(name="sparse_prefill_256_32k", op="sparse", requests=1, queries=256, lo=32768, hi=32768, k=512),
        # the window layers' decode step
        dict(name="window_decode_b8", op="window", requests=8, queries=8, lo=1000, hi=1000000, window=512),
        # the window layers' prefill chunk
        dict(name="window_chunk_512", op="window", requests=1, queries=512, lo=3500, hi=3500, window=512),
        # parallel samples of one prompt
        dict(name="fork_4_of_1", op="fork", requests=1, forks=4, lo=16421, hi=16421, pages=512),
        # beams of a batch
        dict(name="fork_64_of_8", op="fork", requests=8, forks=64, lo=20000, hi=60000, pages=7000),
        # a small pool after two of its requests ended
        dict(name="compact_512", op="compact", requests=6, lo=1000, hi=6000, pages=512),
        # a large pool after half of its requests ended
        dict(name="compact_8k", op="compact", requests=32, lo=4096, hi=24000, pages=8192),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append", "sparse", "sparse", "sparse", "window", "window", "fork", "compact"])
    if op == "append":
        requests = _log(rng, 1, 64)
        per = _log(rng, 1, max(1, 2048 // requests))
        # rings hold the window and one region more: 9 pages
        ring = 9 if per <= 64 and rng.random() < 0.5 else 0
        return dict(op=op, requests=requests, tokens=requests * per, ctx=_log(rng, 1, 262144), ring=ring)
    if op == "sparse":
        k = rng.choice([_log(rng, 1, 512), 512])
        if rng.random() < 0.6:
            requests = _log(rng, 1, 32)
            lo = _log(rng, 1, 100000)
            return dict(op=op, requests=requests, queries=requests, lo=lo, hi=_log(rng, lo, 131072), k=k)
        requests = _log(rng, 1, 4)
        lo = _log(rng, 300, 20000)
        return dict(op=op, requests=requests, queries=_log(rng, requests, 256), lo=lo, hi=_log(rng, lo, 32768), k=k)
    if op == "window":
        if rng.random() < 0.5:
            requests = _log(rng, 1, 32)
            lo = _log(rng, 1, 10000)
            return dict(op=op, requests=requests, queries=requests, lo=lo, hi=_log(rng, lo, 1000000),
                        window=rng.choice([512, _log(rng, 1, 1024)]))
        requests = _log(rng, 1, 4)
        return dict(op=op, requests=requests, queries=_log(rng, requests, 512), lo=600, hi=_log(rng, 600, 8000),
                    window=rng.choice([512, _log(rng, 1, 512)]))
    requests = _log(rng, 1, 16)
    hi = _log(rng, 200, 20000)
    lo = _log(rng, 64, hi)
    need = requests * (hi // PAGE + 2)
    if op == "fork":
        forks = _log(rng, 1, 64)
        return dict(op=op, requests=requests, forks=forks, lo=lo, hi=hi, pages=need + forks + _log(rng, 1, 500))
    return dict(op=op, requests=max(2, requests), lo=lo, hi=hi,
                pages=max(2, requests) * (hi // PAGE + 2) + _log(rng, 1, 500))


# ------------------------------------------------------------------ inputs

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _rows(shape, g):
    """Token rows: N(0, 1) with a gain of its own for every row (rows of a cache differ in size)."""
    x = torch.randn(shape, generator=g, device=DEV)
    return (x * torch.exp(0.7 * torch.randn(shape[:-1] + (1,), generator=g, device=DEV))).to(torch.bfloat16)


def _scale_of(amax):
    """The smallest power of two s with amax <= 448 s, in [2^-126, 2^120]; 0 for 0."""
    m, e = torch.frexp(amax)                                     # amax = m 2^e, m in [0.5, 1); 448 = 0.875 2^9
    e = (e - 9 + (m > 0.875)).clamp(-126, 120).to(torch.int32)
    return torch.where(amax > 0, ((e + 127) << 23).view(torch.float32), torch.zeros_like(amax))


def _codes_of(x, s):
    """x [..., 8, 192] with a scale for each block -> e4m3 codes."""
    y = torch.where(s[..., None, None] > 0, x / s[..., None, None], torch.zeros_like(x))
    return y.to(torch.float8_e4m3fn).view(torch.uint8)


def _pool(pages, g):
    """A filled cache: every block quantised from rows as _rows draws them."""
    cache = torch.empty((pages, G, RPP, 2, REGION, D), dtype=torch.uint8, device=DEV)
    scale = torch.empty((pages, G, RPP, 2), dtype=torch.float32, device=DEV)
    for p in range(0, pages, 512):
        x = _rows((min(512, pages - p), G, RPP, 2, REGION, D), g).float()
        s = _scale_of(x.abs().amax((-1, -2)))
        cache[p:p + 512], scale[p:p + 512] = _codes_of(x, s), s
    return cache, scale


def _lengths(case, g, n):
    lo, hi = math.log(case["lo"]), math.log(case["hi"])
    u = torch.rand(n, generator=g, device=DEV, dtype=torch.float64).tolist()
    return [min(case["hi"], max(case["lo"], int(round(math.exp(lo + x * (hi - lo)))))) for x in u]


def _tables(lengths, pages, g, columns=None):
    """Block table of requests of these lengths, pages taken in a random order; -1 behind the last."""
    each = [(L + PAGE - 1) // PAGE for L in lengths]
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(lengths), columns or max(each)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(each):
        table[b, :n] = order[at:at + n]
        at += n
    return table


def _int(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _query_positions(case, lengths, g):
    """(q_req, q_pos): the newest position of every request, or the last ones of each, request by request."""
    n, b = case["queries"], case["requests"]
    each = [n // b + (i < n % b) for i in range(b)]
    req = [i for i in range(b) for _ in range(each[i])]
    pos = [max(0, lengths[i] - each[i] + j) for i in range(b) for j in range(each[i])]
    return _int(req), _int(pos)


def _selection(q_pos, k, g):
    """Every query's own region and a random k - 1 of the regions before it, ascending; -1 behind them."""
    own_region = (q_pos // REGION).long()
    most = int(own_region.max()) + 1
    r = torch.arange(most, device=DEV)
    idx = torch.full((q_pos.shape[0], G, k), -1, dtype=torch.int32, device=DEV)
    take = min(k, most)
    for i in range(0, q_pos.shape[0], 64):
        o = own_region[i:i + 64, None, None]
        w = torch.rand((o.shape[0], G, most), generator=g, device=DEV)
        w = torch.where(r < o, w, torch.where(r == o, 2.0, -1.0))
        v, j = torch.topk(w, take, dim=-1)
        j = torch.where(v >= 0, j, most).sort(-1).values
        idx[i:i + 64, :, :take] = torch.where(j < most, j, -1).to(torch.int32)
    return idx, (idx >= 0).sum(-1).to(torch.int32)


def prepare(case, seed):
    g = _generator(seed)
    op, b = case["op"], case["requests"]
    s = {"case": case}
    if op == "append":
        per, ctx, ring = case["tokens"] // b, case["ctx"], case["ring"]
        start = [max(0, ctx - i * 3) for i in range(b)]           # every request at a place of its own
        columns = (max(start) + per + PAGE - 1) // PAGE
        first = [x // PAGE for x in start]
        last = [(x + per - 1) // PAGE for x in start]
        if ring:
            v = torch.arange(columns, device=DEV)[None]
            s["table"] = (torch.arange(b, device=DEV)[:, None] * ring + v % ring).to(torch.int32)
            pages = b * ring
        else:                                                     # the pages that the chunk touches
            pages = sum(y - x + 1 for x, y in zip(first, last))
            order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
            s["table"] = torch.full((b, columns), -1, dtype=torch.int32, device=DEV)
            at = 0
            for i in range(b):
                n = last[i] - first[i] + 1
                s["table"][i, first[i]:last[i] + 1] = order[at:at + n]
                at += n
        s["cache"], s["scale"] = _pool(pages, g)
        s["req"] = _int([i for i in range(b) for _ in range(per)])
        s["pos"] = _int([start[i] + j for i in range(b) for j in range(per)])
        s["new_k"] = _rows((b * per, G, D), g)
        s["new_v"] = _rows((b * per, G, D), g)
        return s
    lengths = _lengths(case, g, b)
    if op in ("sparse", "window"):
        if op == "window" and case["queries"] == b:               # decode: rings
            ring = (case["window"] + REGION - 2) // PAGE + 2
            v = torch.arange((max(lengths) + PAGE - 1) // PAGE, device=DEV)[None]
            s["table"] = (torch.arange(b, device=DEV)[:, None] * ring + v % ring).to(torch.int32)
            pages = b * ring
        else:
            pages = sum((L + PAGE - 1) // PAGE for L in lengths)
            s["table"] = _tables(lengths, pages, g)
        s["cache"], s["scale"] = _pool(pages, g)
        s["req"], s["pos"] = _query_positions(case, lengths, g)
        nq = case["queries"]
        s["q"] = torch.randn((nq, HQ, D), generator=g, device=DEV).to(torch.bfloat16)
        s["out"] = torch.empty((nq, HQ, D), dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty((nq, HQ), dtype=torch.float32, device=DEV)
        if op == "sparse":
            s["sel"], s["count"] = _selection(s["pos"], case["k"], g)
        return s
    pages = case["pages"]
    columns = case["hi"] // PAGE + 2
    live = _tables(lengths, pages, g, columns)
    forks = case.get("forks", 0)
    s["table"] = torch.full((b + forks, columns), -1, dtype=torch.int32, device=DEV)
    s["table"][:b] = live
    s["ref"] = torch.zeros(pages, dtype=torch.int32, device=DEV)
    s["ref"][live[live >= 0].long()] = 1
    s["cache"], s["scale"] = _pool(pages, g)
    if op == "fork":
        s["parent"] = _int([i % b for i in range(forks)])
        s["child"] = _int([b + i for i in range(forks)])
        s["length"] = _int([max(1, lengths[i % b] - (i * 5) % 130) for i in range(forks)])
    else:                                                         # every second request ends, the last keeps half
        s["cut"] = _int([i for i in range(b) if i % 2 == 0 or i == b - 1])
        s["keep"] = _int([lengths[i] // 2 if i == b - 1 else 0 for i in range(b) if i % 2 == 0 or i == b - 1])
        s["ref_mid"], s["table_mid"] = torch.empty_like(s["ref"]), torch.empty_like(s["table"])
        s["new_index"] = torch.empty_like(s["ref"])
        s["n_live"] = torch.empty(1, dtype=torch.int32, device=DEV)
    s["ref_out"], s["table_out"] = torch.empty_like(s["ref"]), torch.empty_like(s["table"])
    return s


# ------------------------------------------------------------------ the plain forms

def _values(codes, scale):
    """codes [..., 8, 192], a scale for each block -> fp32 values."""
    return codes.view(torch.float8_e4m3fn).float() * scale[..., None, None]


def _append(s):
    cache, scale, pos, req = s["cache"], s["scale"], s["pos"].long(), s["req"].long()
    page = s["table"][req, pos // PAGE].long()
    block, at = torch.unique(page * RPP + pos % PAGE // REGION, return_inverse=True)
    n = block.numel()
    pg, rg = block // RPP, block % RPP
    # the call's rows of every block, [blocks][4][2][8][192], and which of the 8 they are
    x = torch.zeros((n, G, 2, REGION, D), device=DEV)
    x[at, :, 0, pos % REGION] = s["new_k"].float()
    x[at, :, 1, pos % REGION] = s["new_v"].float()
    given = torch.zeros((n, REGION), dtype=torch.bool, device=DEV)
    given[at, pos % REGION] = True
    row = torch.arange(REGION, device=DEV)
    first = torch.where(given, row, REGION).amin(1, keepdim=True)
    kept = row < first                                            # rows that were there before
    old = torch.where(first[:, :, None] > 0, scale[pg, :, rg].flatten(1)[:, None], 0.0).view(n, G, 2)
    new = torch.maximum(old, _scale_of(x.abs().amax((-1, -2))))
    codes = cache[pg, :, rg]
    kept_x = _values(codes, old)
    rows = torch.where(kept[:, None, None, :, None], kept_x, x)
    touched = (kept | given)[:, None, None, :, None]
    cache[pg, :, rg] = torch.where(touched, _codes_of(rows, new), codes)
    scale[pg, :, rg] = new
    return {"codes": cache.view(torch.float8_e4m3fn), "scale": scale}


def _attention(q, k, v, ok):
    """q [n][4][16][192], k and v [n][4][T][192], ok [n][4][T] -> out bf16 [n][64][192], lse fp32 [n][64]."""
    x = torch.matmul(q, k.transpose(-1, -2)) / math.sqrt(D)
    x = torch.where(ok[:, :, None], x, -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(m > -math.inf, m, 0.0))
    z = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / torch.where(z > 0, z, 1.0)
    return out.flatten(1, 2).to(torch.bfloat16), (m + torch.log(z)).flatten(1)


def _regions_of(s, regions):
    """Values and tokens of regions [n][4][r] (-1: none): k, v [n][4][8 r][192], token [n][4][8 r]."""
    there = regions >= 0
    r = torch.where(there, regions, 0).long()
    n = r.shape[0]
    page = s["table"][s["req"].long()[:, None, None], r // RPP].long().clamp(min=0)
    group = torch.arange(G, device=DEV)[None, :, None]
    kv = _values(s["cache"][page, group, r % RPP], s["scale"][page, group, r % RPP])      # [n][4][r][2][8][192]
    token = r[..., None] * REGION + torch.arange(REGION, device=DEV)
    token = torch.where(there[..., None], token, 1 << 40)
    return kv[:, :, :, 0].reshape(n, G, -1, D), kv[:, :, :, 1].reshape(n, G, -1, D), token.flatten(2)


def _sparse(s):
    k, v, token = _regions_of(s, s["sel"])
    q = s["q"].float().view(-1, G, HPG, D)
    out, lse = _attention(q, k, v, token <= s["pos"][:, None, None])
    return {"out": out, "lse": lse}


def _window(s):
    w = s["case"]["window"]
    pos = s["pos"].long()
    lo = (pos - w + 1).clamp(min=0)
    r = lo[:, None] // REGION + torch.arange(w // REGION + 2, device=DEV)
    r = torch.where(r <= pos[:, None] // REGION, r, -1)
    k, v, token = _regions_of(s, r[:, None].expand(-1, G, -1))
    q = s["q"].float().view(-1, G, HPG, D)
    ok = (token <= pos[:, None, None]) & (token >= lo[:, None, None])
    out, lse = _attention(q, k, v, ok)
    return {"out": out, "lse": lse}


def _fork(s):
    ref, table = s["ref"].clone(), s["table"].clone()
    length, parent, child = s["length"].long(), s["parent"].long(), s["child"].long()
    full, part = length // PAGE, length % PAGE > 0
    rows = table[parent]
    column = torch.arange(table.shape[1], device=DEV)
    shared = column < full[:, None]
    ref += torch.bincount(torch.where(shared, rows, ref.numel()).flatten().long(), minlength=ref.numel() + 1)[:-1]
    free = torch.argsort((s["ref"] != 0).to(torch.int8), stable=True)[:len(full)]
    fresh = free[(part.long().cumsum(0) - 1).clamp(min=0)]
    source = rows.gather(1, full.clamp(max=table.shape[1] - 1)[:, None])[:, 0].long()
    rows = torch.where(shared, rows, -1)
    rows = torch.where(part[:, None] & (column == full[:, None]), fresh[:, None].to(torch.int32), rows)
    table[child] = rows
    ref[fresh[part]] = 1
    s["cache"][fresh[part]] = s["cache"][source[part]]
    s["scale"][fresh[part]] = s["scale"][source[part]]
    return {"ref": ref, "table": table, "cache": s["cache"], "scale": s["scale"]}


def _compact(s):
    ref, table = s["ref"].clone(), s["table"].clone()
    # the released pages
    column = torch.arange(table.shape[1], device=DEV)
    cut = s["cut"].long()
    gone = column >= ((s["keep"].long() + PAGE - 1) // PAGE)[:, None]
    rows = table[cut]
    dropped = torch.where(gone & (rows >= 0), rows, ref.numel()).flatten().long()
    ref -= torch.bincount(dropped, minlength=ref.numel() + 1)[:-1]
    table[cut] = torch.where(gone, -1, rows)
    # live pages behind the first n_live, from the last one, to the free pages among those, from the first one
    index = torch.arange(ref.numel(), device=DEV)
    live = ref > 0
    n_live = live.sum()
    source = torch.nonzero(live & (index >= n_live))[:, 0].flip(0)
    to = torch.nonzero(~live & (index < n_live))[:, 0]
    new_index = torch.where(live, index, -1)
    new_index[source] = to
    ref[to] = ref[source]
    ref[source] = 0
    s["cache"][to] = s["cache"][source]
    s["scale"][to] = s["scale"][source]
    table = torch.where(table >= 0, new_index[table.clamp(min=0).long()], -1).to(torch.int32)
    return {"ref": ref, "table": table, "cache": s["cache"], "scale": s["scale"],
            "new_index": new_index.to(torch.int32), "n_live": n_live.view(1).to(torch.int32)}


# ------------------------------------------------------------------ the framework's calls

def _own_append(s):
    from sparse_long_context_dsa_b200 import dsa
    dsa.kv_append_quant(s["cache"], s["scale"], s["table"], s["pos"], s["new_k"], s["new_v"], q_req=s["req"])
    return {"codes": s["cache"].view(torch.float8_e4m3fn), "scale": s["scale"]}


def _own_sparse(s):
    from sparse_long_context_dsa_b200 import dsa
    if s["case"]["queries"] == s["case"]["requests"]:             # decode: query i is request i's
        out = dsa.sparse_attn_decode_quant(s["q"], s["cache"], s["scale"], s["table"], s["pos"], s["sel"], s["count"],
                                           out=s["out"], lse=s["lse"])
    else:
        out = dsa.sparse_attn_prefill_quant(s["q"], s["cache"], s["scale"], s["table"], s["req"], s["pos"], s["sel"],
                                            s["count"], out=s["out"], lse=s["lse"])
    return {"out": out, "lse": s["lse"]}


def _own_window(s):
    from sparse_long_context_dsa_b200 import dsa
    out = dsa.window_attn_quant(s["q"], s["cache"], s["scale"], s["table"], s["pos"], s["case"]["window"],
                                q_req=s["req"], out=s["out"], lse=s["lse"])
    return {"out": out, "lse": s["lse"]}


def _own_fork(s):
    from sparse_long_context_dsa_b200 import dsa
    ref, table = dsa.pages_fork(s["ref"], s["table"], s["parent"], s["child"], s["length"], [s["cache"], s["scale"]],
                                ref_out=s["ref_out"], table_out=s["table_out"])
    return {"ref": ref, "table": table, "cache": s["cache"], "scale": s["scale"]}


def _own_compact(s):
    from sparse_long_context_dsa_b200 import dsa
    ref, table = dsa.pages_release(s["ref"], s["table"], s["cut"], s["keep"], ref_out=s["ref_mid"],
                                   table_out=s["table_mid"])
    ref, table, new_index, n_live = dsa.pages_compact(ref, table, [s["cache"], s["scale"]], ref_out=s["ref_out"],
                                                      table_out=s["table_out"], new_index=s["new_index"],
                                                      n_live=s["n_live"])
    return {"ref": ref, "table": table, "cache": s["cache"], "scale": s["scale"], "new_index": new_index,
            "n_live": n_live}


_PLAIN = {"append": _append, "sparse": _sparse, "window": _window, "fork": _fork, "compact": _compact}
_OWN = {"append": _own_append, "sparse": _own_sparse, "window": _own_window, "fork": _own_fork,
        "compact": _own_compact}


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


# ------------------------------------------------------------------ bytes and operations

def work(case):
    op, b = case["op"], case["requests"]
    block = 2 * REGION * D + 8                                    # K and V of a region and group, and their scales
    if op == "append":                                            # rows read, codes and scales written
        n = case["tokens"]
        return {"bytes": n * G * 2 * D * 3 + (n + REGION - 1) // REGION * G * 8 + n * 8, "flops": 2 * n * G * 2 * D}
    mean = case["lo"]
    if case["hi"] > case["lo"]:
        mean = (case["hi"] - case["lo"]) / math.log(case["hi"] / case["lo"])
    if op in ("sparse", "window"):
        nq = case["queries"]
        if op == "sparse":
            regions = min(case["k"], mean / REGION + 1)
            once = min(nq * regions, b * (mean / REGION + 1))     # regions that several queries select count once
        else:
            regions = min(case["window"] / REGION + 1, mean / REGION + 1)
            once = min(nq * regions, b * (regions + nq / b / REGION))
        return {"bytes": once * G * block + nq * HQ * (4 * D + 4), "flops": nq * regions * REGION * HQ * 4 * D}
    page = G * RPP * block
    if op == "fork":
        table = (b + case["forks"]) * (mean / PAGE + 2) * 4
        return {"bytes": 2 * case["forks"] * page + 2 * table + 8 * case["pages"], "flops": 0}
    # compaction: half of the requests' pages stay, in a random order over the pool
    live = b / 2 * mean / PAGE
    moved = live * max(0.0, 1 - live / case["pages"])
    return {"bytes": 2 * moved * page + 4 * b * (mean / PAGE + 2) * 4 + 20 * case["pages"], "flops": 0}


# ------------------------------------------------------------------ 64 bits

def _e4m3_value(x):
    """The e4m3 value nearest to x (ties to even), in 64 bits; |x| <= 448."""
    e = (torch.frexp(x).exponent.long() - 1).clamp(min=-6)        # |x| in [2^e, 2^(e+1)), or subnormal
    step = ((e - 3 + 1023) << 52).view(torch.float64)
    return torch.round(x / step) * step


def _exact_scale(a):
    if a == 0:
        return 0.0
    e = -126
    while 448.0 * 2.0 ** e < a and e < 120:
        e += 1
    return 2.0 ** e


def _exact_append(s):
    value = s["cache"].view(torch.float8_e4m3fn).double()
    scale = s["scale"].double().cpu()
    table, req, pos = s["table"].tolist(), s["req"].tolist(), s["pos"].tolist()
    blocks = {}
    for i, (b, p) in enumerate(zip(req, pos)):
        blocks.setdefault((table[b][p // PAGE], p % PAGE // REGION), []).append((p % REGION, i))
    new = torch.stack([s["new_k"], s["new_v"]], 2).double()       # [n][4][2][192]
    largest = new.abs().amax(-1).cpu()
    for (page, region), rows in blocks.items():
        first = rows[0][0]
        ratio = torch.zeros((G, 2), dtype=torch.float64)
        for g in range(G):
            for t in range(2):
                before = float(scale[page, g, region, t]) if first else 0.0
                now = max([before, _exact_scale(max(float(largest[i, g, t]) for _, i in rows))])
                ratio[g, t] = before / now if now else 0.0
                scale[page, g, region, t] = now
        ratio = ratio.to(DEV)[:, :, None, None]
        kept = value[page, :, region, :, :first]
        value[page, :, region, :, :first] = _e4m3_value(kept * ratio)
        inverse = scale[page, :, region].to(DEV)
        inverse = torch.where(inverse > 0, 1 / inverse, 0.0)[..., None]
        for row, i in rows:
            value[page, :, region, :, row] = _e4m3_value(new[i] * inverse)
    return {"codes": value, "scale": scale}


def _exact_attention(s, regions_of):
    n = s["q"].shape[0]
    out, lse = [], []
    for i in range(n):
        p, row = int(s["pos"][i]), s["table"][int(s["req"][i])].long()
        token = regions_of(i, p)                                  # [4][T], -1: none
        page = row[token.clamp(min=0) // PAGE].clamp(min=0)
        g = torch.arange(G, device=DEV)[:, None]
        region, t = token.clamp(min=0) % PAGE // REGION, token.clamp(min=0) % REGION
        rows = s["cache"][page, g, region, :, t].view(torch.float8_e4m3fn).double()       # [4][T][2][192]
        rows = rows * s["scale"][page, g, region].double()[..., None]
        k, v = rows[:, :, 0], rows[:, :, 1]
        x = s["q"][i].double().view(G, HPG, D) @ k.transpose(1, 2) / math.sqrt(D)
        x = x.masked_fill((token < 0)[:, None], -math.inf)
        z = torch.logsumexp(x, -1)
        w = torch.exp(x - torch.where(z.isinf(), 0.0, z)[..., None])
        out.append((w @ v).view(HQ, D))
        lse.append(z.view(HQ))
    return {"out": torch.stack(out), "lse": torch.stack(lse)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(s)
    if case["op"] == "sparse":
        def tokens(i, p):
            r = s["sel"][i].long()                                # [4][k]
            t = r[..., None] * REGION + torch.arange(REGION, device=DEV)
            return torch.where((r[..., None] >= 0) & (t <= p), t, -1).flatten(1)
        return _exact_attention(s, tokens)
    if case["op"] == "window":
        def tokens(i, p):
            return torch.arange(max(0, p - case["window"] + 1), p + 1, device=DEV).expand(G, -1)
        return _exact_attention(s, tokens)
    return None                                                   # pages and counts: whole numbers

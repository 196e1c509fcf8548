"""Cases of the paged serving operators: page tables, paged append, shared-prefix attention.

A serving program keeps the keys and values of its requests in pages of ``page`` tokens out of one
pool.  All requests of a batch share a long prefix (a system prompt, a document), whose pages are
stored once; each request then owns the pages of its own tokens.  A step of such a program is

    page_tables   grow (or free) each request's pages to its new length; slot of every new token
    paged_append  write the new tokens' keys and values to their slots
    prefix_attn   attention of the new tokens to the prefix, computed once for all requests, and
                  to their request's own tokens up to their position

``run`` passes once through one of the three.
"""
import random

import numpy as np
import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


def listed():
    def attn(name, dtype, B, heads, kv_heads, d, page, prefix, own_max, nq_max):
        return {"name": name, "op": "attn", "dtype": dtype, "B": B, "heads": heads,
                "kv_heads": kv_heads, "d": d, "page": page, "prefix": prefix, "own_max": own_max,
                "nq_max": nq_max}

    return [
        # one decode tick of 64 requests: most grow by a token, some finish, some are admitted
        {"name": "tables_tick", "op": "tables", "B": 64, "page": 64, "len_max": 4096,
         "admit_percent": 3, "prompt_max": 40},
        # a burst of admissions: a third of 1024 requests bring prompts, about a quarter million
        # tokens to place
        {"name": "tables_prompts", "op": "tables", "B": 1024, "page": 16, "len_max": 2048,
         "admit_percent": 33, "prompt_max": 1601},
        # the new tokens of one decode tick, slices of a fused projection
        {"name": "append_tick", "op": "append", "dtype": "bf16", "T": 64, "heads": 32,
         "kv_heads": 8, "d": 128, "page": 64},
        # a prompt of the gated training length written at once
        {"name": "append_prompts", "op": "append", "dtype": "bf16", "T": 16384, "heads": 32,
         "kv_heads": 8, "d": 128, "page": 64},
        # 32-bit cache, small pages, an odd number of tokens
        {"name": "append_f32", "op": "append", "dtype": "f32", "T": 1337, "heads": 16,
         "kv_heads": 16, "d": 64, "page": 16},
        # the smallest batch behind a short prompt: latency counts
        attn("attn_small", "bf16", 4, 32, 8, 128, 16, 1000, 130, 1),
        # one decode tick at the 32K context of the grouped-query decode workload
        attn("attn_tick", "bf16", 64, 32, 8, 128, 64, 32768, 1024, 1),
        # the same with a full batch and long answers: the requests' own tokens dominate
        attn("attn_tick_large", "bf16", 256, 32, 8, 128, 64, 32768, 2048, 1),
        # one key head per query head, d = 64, behind a 64K document
        attn("attn_tick_mha", "bf16", 32, 16, 16, 64, 32, 65536, 301, 1),
        # up to eight drafted tokens of each request checked at once, ragged
        attn("attn_verify", "bf16", 24, 32, 8, 128, 128, 8191, 700, 8),
        # prompts of very different lengths behind a system prompt
        attn("attn_prompts", "bf16", 12, 32, 8, 128, 64, 8192, 2000, 1400),
        # 32-bit cache
        attn("attn_tick_f32", "f32", 8, 16, 4, 64, 16, 4101, 513, 1),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["tables", "append", "attn", "attn", "attn", "attn"])
    if op == "tables":
        return {"op": op, "B": _log_int(rng, 1, 1024), "page": rng.choice([16, 32, 64, 128]),
                "len_max": _log_int(rng, 64, 4096), "admit_percent": rng.randint(0, 33),
                "prompt_max": _log_int(rng, 8, 1600)}
    heads, kv_heads = rng.choice([(32, 8), (16, 16), (16, 4), (8, 1), (8, 4), (32, 4)])
    d, page = rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "append":
        return {"op": op, "dtype": dtype, "T": _log_int(rng, 1, 8000), "heads": heads,
                "kv_heads": kv_heads, "d": d, "page": page}
    case = {"op": op, "dtype": dtype, "B": _log_int(rng, 1, 200), "heads": heads,
            "kv_heads": kv_heads, "d": d, "page": page, "prefix": _log_int(rng, 1, 65536),
            "own_max": _log_int(rng, 1, 2048), "nq_max": rng.choice([1, 1, 1, 4, 9, 0])}
    if case["nq_max"] == 0:  # prompts
        case["nq_max"] = _log_int(rng, 16, 1500)
        case["B"] = min(case["B"], 16)
        case["prefix"] = min(case["prefix"], 12000)
    case["own_max"] = max(case["own_max"], case["nq_max"])
    # no more than the largest listed cases cost, in bytes and in products
    while work(case)["flops"] > (1.0e12 if dtype == "bf16" else 5.0e10) \
            or work(case)["bytes"] > 1.0e9:
        if case["B"] > 1:
            case["B"] = max(1, case["B"] * 2 // 3)
        else:
            case["prefix"] = max(1, case["prefix"] * 2 // 3)
            case["nq_max"] = max(1, case["nq_max"] * 2 // 3)
    return case


# ---- sizes that a case alone decides (the order of the requests is the seed's) ----------------


def _spread(case):
    """A random.Random that depends on the case's values and nothing else."""
    return random.Random("/".join("%s=%s" % (k, case[k]) for k in sorted(case) if k != "name"))


def _attn_lengths(case):
    """(new tokens, own tokens with the new ones) of every request."""
    rng = _spread(case)
    pairs = []
    for b in range(case["B"]):
        nq = 1 if case["nq_max"] == 1 else rng.randint(1, case["nq_max"])
        pairs.append((nq, rng.randint(nq, max(nq, case["own_max"]))))
    pairs[-1] = (pairs[-1][0], max(pairs[-1][0], case["own_max"]))
    return pairs


def _table_lengths(case):
    """(tokens before, tokens after) of every request of a tick."""
    rng = _spread(case)
    pairs = []
    for b in range(case["B"]):
        x = rng.random() * 100
        if x < case["admit_percent"]:
            pairs.append((0, rng.randint(1, case["prompt_max"])))
        elif x < case["admit_percent"] + 4:
            pairs.append((rng.randint(1, case["len_max"] - 1), 0))  # finished: pages are freed
        else:
            before = rng.randint(1, case["len_max"] - 1)
            pairs.append((before, before + 1))
    return pairs


def _pages(n, page):
    return -(-n // page)


def work(case):
    if case["op"] == "tables":
        pairs = _table_lengths(case)
        page = case["page"]
        grown = sum(max(0, _pages(n, page) - _pages(o, page)) for o, n in pairs)
        freed = sum(max(0, _pages(o, page) - _pages(n, page)) for o, n in pairs)
        tokens = sum(max(0, n - o) for o, n in pairs)
        # both lengths read, the new one and the offset written; a page id read and written for
        # each page that moves; slot and position of each token
        return {"bytes": 16 * len(pairs) + 8 * (grown + freed) + 8 * tokens, "flops": 0}
    if case["op"] == "append":
        each = case["T"] * case["kv_heads"] * case["d"] * SIZE[case["dtype"]]
        return {"bytes": 4 * each + 4 * case["T"], "flops": 0}
    pairs = _attn_lengths(case)
    tokens = sum(nq for nq, _ in pairs)
    keys = case["prefix"] + sum(n for _, n in pairs)
    seen = sum(nq * case["prefix"] + nq * (n - nq) + nq * (nq + 1) // 2 for nq, n in pairs)
    size = SIZE[case["dtype"]]
    return {"bytes": 2 * keys * case["kv_heads"] * case["d"] * size
            + 2 * tokens * case["heads"] * case["d"] * size + 4 * tokens * case["heads"],
            "flops": 4 * seen * case["heads"] * case["d"]}


# ---- inputs -----------------------------------------------------------------------------------


def _int32(values):
    return torch.tensor(np.asarray(values, dtype=np.int32), device=DEV)


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device=DEV).manual_seed(int(seed))

    def normal(*shape, dtype):
        return torch.randn(*shape, device=DEV, dtype=dtype, generator=gen)

    if case["op"] == "tables":
        page = case["page"]
        pairs = _table_lengths(case)
        pairs = [pairs[i] for i in rng.permutation(len(pairs))]
        before, after = [list(x) for x in zip(*pairs)]
        ld = _pages(max(case["len_max"], case["prompt_max"]) + 1, page)
        held = [_pages(o, page) for o in before]
        grown = sum(max(0, _pages(n, page) - h) for n, h in zip(after, held))
        pool = sum(held) + grown + 37
        ids = rng.permutation(pool).astype(np.int32)
        table = np.full((len(pairs), ld), -1, np.int32)
        at = 0
        for b, h in enumerate(held):
            table[b, :h] = ids[at:at + h]
            at += h
        # the free pages lie in a ring, from a place that earlier steps have left
        free = ids[at:]
        head = int(rng.integers(0, pool))
        ring = np.full(pool, -1, np.int32)
        ring[(head + np.arange(len(free))) % pool] = free
        tokens = sum(max(0, n - o) for o, n in pairs)
        return {"op": "tables", "page": page, "lens": _int32(before), "new_lens": _int32(after),
                "table": _int32(table), "ring": _int32(ring), "free": _int32([head, len(free)]),
                "max_tokens": -(-tokens // 64) * 64 + 64, "pos_offset": 1000}

    dtype = TYPES[case["dtype"]]
    heads, kv_heads, d, page = case["heads"], case["kv_heads"], case["d"], case["page"]
    if case["op"] == "append":
        T = case["T"]
        # requests' tokens lie in order within pages that lie anywhere
        pool = _pages(T, page) + 23
        at = rng.permutation(pool)[np.arange(T) // page] * page + np.arange(T) % page
        return {"op": "append", "heads": heads, "kv_heads": kv_heads, "d": d,
                "qkv": normal(T, (heads + 2 * kv_heads) * d, dtype=dtype),
                "slots": _int32(at), "k_pages": normal(pool, kv_heads, page, d, dtype=dtype),
                "v_pages": normal(pool, kv_heads, page, d, dtype=dtype)}

    pairs = _attn_lengths(case)
    pairs = [pairs[i] for i in rng.permutation(len(pairs))]
    nq, lens = [list(x) for x in zip(*pairs)]
    T = sum(nq)
    prefix_pages = _pages(case["prefix"], page)
    ld = _pages(max(lens), page)
    held = [_pages(n, page) for n in lens]
    pool = prefix_pages + sum(held) + 11
    ids = rng.permutation(pool).astype(np.int32)
    table = np.full((len(pairs), ld), -1, np.int32)
    at = prefix_pages
    for b, h in enumerate(held):
        table[b, :h] = ids[at:at + h]
        at += h
    # queries of twice the keys' spread, so that some keys weigh much more than others
    qkv = normal(T, (heads + 2 * kv_heads) * d, dtype=dtype)
    qkv[:, :heads * d] *= 2
    return {"op": "attn", "heads": heads, "kv_heads": kv_heads, "d": d, "page": page, "qkv": qkv,
            "k_pages": normal(pool, kv_heads, page, d, dtype=dtype),
            "v_pages": normal(pool, kv_heads, page, d, dtype=dtype),
            "table": _int32(table), "lens": _int32(lens),
            "prefix_table": _int32(ids[:prefix_pages]), "prefix_len": case["prefix"],
            "cu_q": None if case["nq_max"] == 1 else _int32(np.concatenate([[0], np.cumsum(nq)])),
            "max_q": max(nq)}


# ---- one pass ---------------------------------------------------------------------------------


def run(state):
    if own:
        return _run_own(state)
    if state["op"] == "tables":
        return _tables_plain(state)
    if state["op"] == "append":
        return _append_plain(state)
    return _attn_plain(state)


def _split(state):
    """Query, key and value heads [T, heads, d] of a fused projection."""
    T, d = state["qkv"].shape[0], state["d"]
    q, k, v = state["qkv"].split(
        [state["heads"] * d, state["kv_heads"] * d, state["kv_heads"] * d], dim=1)
    return (q.view(T, state["heads"], d), k.view(T, state["kv_heads"], d),
            v.view(T, state["kv_heads"], d))


def _run_own(s):
    import block_sparse_attention_summaries_b200 as bsa

    if s["op"] == "tables":
        lens, free, cu_new, slots, positions = bsa.page_tables(
            s["lens"], s["new_lens"], s["table"], s["ring"], s["free"], s["page"],
            s["max_tokens"], pos_offset=s["pos_offset"])
        return {"lens": lens, "free": free, "cu_new": cu_new, "slots": slots,
                "positions": positions, "table": s["table"], "ring": s["ring"]}
    if s["op"] == "append":
        q, k, v = _split(s)
        bsa.paged_append(k, v, s["slots"], s["k_pages"], s["v_pages"])
        return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    q, k, v = _split(s)
    o, lse = bsa.prefix_attn(q, s["k_pages"], s["v_pages"], s["table"], s["lens"],
                             s["prefix_table"], s["prefix_len"], cu_q=s["cu_q"],
                             max_q=s["max_q"])
    return {"o": o, "lse": lse}


def _tables_plain(s):
    page, table, ring = s["page"], s["table"], s["ring"]
    B, ld = table.shape
    N = ring.shape[0]
    lens, new_lens = s["lens"].long(), s["new_lens"].long()
    head, avail = s["free"].long()
    have, want = (lens + page - 1) // page, (new_lens + page - 1) // page
    grow = (want - have).clamp(min=0)
    upto = grow.cumsum(0)
    served = (grow == 0) | (upto <= avail)
    first = upto - grow
    lens_out = torch.where(served, new_lens, lens)
    # pages that join, from the front of the ring
    c = torch.arange(ld, device=DEV)
    joins = (c >= have[:, None]) & (c < want[:, None]) & served[:, None]
    taken_at = (head + first[:, None] + c - have[:, None]) % N
    new_table = torch.where(joins, ring[taken_at], table)
    taken = torch.where(served, upto, 0).max() if B else 0
    # pages that leave, to its end
    drop = (have - want).clamp(min=0)
    after = drop.cumsum(0)
    leaves = (c >= want[:, None]) & (c < have[:, None])
    put_at = (head + avail + (after - drop)[:, None] + c - want[:, None]) % N
    pad = torch.cat([ring, ring[:1]])  # entry N takes what is not put
    pad.scatter_(0, torch.where(leaves, put_at, N).flatten(), table.flatten())
    table.copy_(new_table)
    ring.copy_(pad[:N])
    free = torch.stack([(head + taken) % N, avail - taken + after[-1]]).int()
    # the new tokens, packed request after request
    added = (new_lens - lens).clamp(min=0)
    cu_new = torch.cat([added.new_zeros(1), added.cumsum(0)])
    t = torch.arange(s["max_tokens"], device=DEV)
    b = torch.searchsorted(cu_new[1:], t, right=True).clamp(max=B - 1)
    pos = lens[b] + t - cu_new[b]
    live = (t < cu_new[-1]) & served[b]
    p = (pos // page).clamp(0, ld - 1)
    slots = torch.where(live, new_table[b, p].long() * page + pos % page, -1)
    positions = torch.where(live, pos + s["pos_offset"], -1)
    return {"lens": lens_out.int(), "free": free, "cu_new": cu_new.int(), "slots": slots.int(),
            "positions": positions.int(), "table": table, "ring": ring}


def _append_plain(s):
    q, k, v = _split(s)
    page = s["k_pages"].shape[2]
    at, row = (s["slots"] // page).long(), (s["slots"] % page).long()
    s["k_pages"][at, :, row] = k
    s["v_pages"][at, :, row] = v
    return {"k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _attn_plain(s):
    q, _, _ = _split(s)
    T, heads, d = q.shape
    kv_heads, page, n = s["kv_heads"], s["page"], s["prefix_len"]
    G = heads // kv_heads
    B, ld = s["table"].shape
    qf = q.float().view(T, kv_heads, G, d) * d ** -0.5

    def prefix(pages):  # [kv_heads, prefix, d]
        x = pages[s["prefix_table"].long()].transpose(0, 1).reshape(kv_heads, -1, d)
        return x[:, :n].float()

    def mine(pages):  # [B, kv_heads, ld * page, d]
        x = pages[s["table"].clamp(min=0).long()].transpose(1, 2)
        return x.reshape(B, kv_heads, ld * page, d).float()

    cu = torch.arange(B + 1, device=DEV) if s["cu_q"] is None else s["cu_q"].long()
    t = torch.arange(T, device=DEV)
    b = torch.searchsorted(cu[1:], t, right=True)
    i = t - cu[b]
    nq = cu[1:] - cu[:-1]
    pos = s["lens"].long()[b] - nq[b] + i  # own position of each token
    # [T, kv_heads, G, prefix] scores of the shared keys, [T, kv_heads, G, ld * page] of the own
    shared = torch.einsum("tkgd,knd->tkgn", qf, prefix(s["k_pages"]))
    padded = qf.new_zeros(B, s["max_q"], kv_heads, G, d)
    padded[b, i] = qf
    alone = torch.einsum("bikgd,bknd->bikgn", padded, mine(s["k_pages"]))[b, i]
    hidden = torch.arange(ld * page, device=DEV) > pos[:, None]
    alone = alone.masked_fill(hidden[:, None, None], float("-inf"))
    top = alone.amax(-1, keepdim=True)
    if n:
        top = torch.maximum(top, shared.amax(-1, keepdim=True))
    shared = torch.exp(shared - top)
    alone = torch.exp(alone - top)
    total = shared.sum(-1, keepdim=True) + alone.sum(-1, keepdim=True)
    o = torch.einsum("tkgn,knd->tkgd", shared, prefix(s["v_pages"]))
    weights = alone.new_zeros(B, s["max_q"], kv_heads, G, ld * page)
    weights[b, i] = alone
    o = o + torch.einsum("bikgn,bknd->bikgd", weights, mine(s["v_pages"]))[b, i]
    lse = (top + torch.log(total)).reshape(T, heads)
    return {"o": (o / total).reshape(T, heads, d).to(q.dtype), "lse": lse}


# ---- the definition in 64 bits ----------------------------------------------------------------


def exact(case, seed):
    if case["op"] == "tables":
        return None  # whole numbers
    s = prepare(case, seed)
    if case["op"] == "append":
        first = s["heads"] * s["d"]
        each = s["kv_heads"] * s["d"]

        def after(pages, new):  # pages as rows, one for each slot
            pool, kv_heads, page, d = pages.shape
            rows = pages.double().transpose(1, 2).reshape(pool * page, each)
            rows = rows.index_copy(0, s["slots"].long(), new.double())
            return rows.view(pool, page, kv_heads, d).transpose(1, 2).contiguous()

        return {"k_pages": after(s["k_pages"], s["qkv"][:, first:first + each]),
                "v_pages": after(s["v_pages"], s["qkv"][:, first + each:])}
    d, kv_heads, page, n = s["d"], s["kv_heads"], s["page"], s["prefix_len"]
    T = s["qkv"].shape[0]
    G = s["heads"] // kv_heads
    q = s["qkv"][:, :s["heads"] * d].double().reshape(T, kv_heads, G, d)
    cu = list(range(T + 1)) if s["cu_q"] is None else s["cu_q"].tolist()
    lens = s["lens"].tolist()

    def rows(pages, ids, count, head):
        return pages[ids.long(), head].reshape(-1, d)[:count].double()

    o = torch.empty(T, kv_heads, G, d, device=DEV, dtype=torch.float64)
    lse = torch.empty(T, kv_heads, G, device=DEV, dtype=torch.float64)
    for h in range(kv_heads):
        kp = rows(s["k_pages"], s["prefix_table"], n, h)
        vp = rows(s["v_pages"], s["prefix_table"], n, h)
        for b, length in enumerate(lens):
            mine = s["table"][b, :_pages(length, page)]
            k = torch.cat([kp, rows(s["k_pages"], mine, length, h)])
            v = torch.cat([vp, rows(s["v_pages"], mine, length, h)])
            nq = cu[b + 1] - cu[b]
            x = q[cu[b]:cu[b + 1], h].reshape(nq * G, d) @ k.T / d ** 0.5
            last = n + length - nq + torch.arange(nq, device=DEV).repeat_interleave(G)
            x[torch.arange(n + length, device=DEV)[None, :] > last[:, None]] = -float("inf")
            z = torch.logsumexp(x, dim=1)
            lse[cu[b]:cu[b + 1], h] = z.view(nq, G)
            o[cu[b]:cu[b + 1], h] = (torch.exp(x - z[:, None]) @ v).view(nq, G, d)
    return {"o": o.view(T, kv_heads * G, d), "lse": lse.view(T, kv_heads * G)}

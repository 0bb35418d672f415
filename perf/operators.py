"""Cases for the paged key/value cache: its page bookkeeping, its writes and the attention that reads it.

Operators: ``map`` (block tables and slot maps from request lengths), ``append`` (new rows into their slots), ``decode``
(one or a few query tokens per sequence, with or without a prefix that the whole batch shares) and ``prompt`` (ragged
prompt tokens, causal, over what the cache holds).  Pages are scattered over the pool in a random order, lengths are
ragged, and where a batch has eight sequences or more one of them is idle (length 0).
"""

import math

import torch

own = False


def listed():
    return [
        # One serving step of a full batch: every sequence grows by one token, a few cross into a new page.
        {"name": "map_step", "op": "map", "B": 64, "page": 16, "ctx": 8192, "new": 1},
        # A batch of long prompts enters an empty cache: every page and every slot is new.
        {"name": "map_prompts", "op": "map", "B": 37, "page": 64, "ctx": 0, "new": 32768},
        # The new token of every sequence of a batch.
        {"name": "append_step", "op": "append", "T": 64, "Hkv": 8, "D": 128, "page": 16, "f32": False, "token_major": True},
        # A prompt chunk whose rotary stage hands over 32-bit rows.
        {"name": "append_prompt_f32", "op": "append", "T": 40001, "Hkv": 8, "D": 64, "page": 64, "f32": True, "token_major": False},
        # A single user's chat: latency is what counts.
        {"name": "decode_one", "op": "decode", "B": 1, "Hq": 32, "Hkv": 8, "Nq": 1, "D": 128, "len": 2049, "page": 16,
         "prefix": 0, "token_major": True},
        # A full serving batch with ragged contexts.
        {"name": "decode_batch", "op": "decode", "B": 64, "Hq": 32, "Hkv": 8, "Nq": 1, "D": 128, "len": 8192, "page": 16,
         "prefix": 0, "token_major": True},
        # Long contexts, four drafted tokens each, one key/value head per query head.
        {"name": "decode_long_draft", "op": "decode", "B": 8, "Hq": 16, "Hkv": 16, "Nq": 4, "D": 64, "len": 131072, "page": 64,
         "prefix": 0, "token_major": False},
        # A system prompt shared by a small batch.
        {"name": "shared_small", "op": "decode", "B": 9, "Hq": 16, "Hkv": 4, "Nq": 1, "D": 64, "len": 200, "page": 32,
         "prefix": 4000, "token_major": True},
        # A long document that a whole batch asks about.
        {"name": "shared_long", "op": "decode", "B": 64, "Hq": 32, "Hkv": 8, "Nq": 1, "D": 128, "len": 2048, "page": 64,
         "prefix": 131072, "token_major": False},
        # Short prompts of several users in one call.
        {"name": "prompt_short", "op": "prompt", "B": 5, "Hq": 16, "Hkv": 16, "D": 64, "new": 301, "ctx": 0, "page": 16,
         "token_major": True},
        # One chunk of a chunked prefill far into a long document: few query rows, many keys.
        {"name": "prompt_chunk", "op": "prompt", "B": 1, "Hq": 32, "Hkv": 8, "D": 128, "new": 512, "ctx": 65536, "page": 64,
         "token_major": False},
        # A whole long prompt.
        {"name": "prompt_long", "op": "prompt", "B": 1, "Hq": 32, "Hkv": 8, "D": 128, "new": 12345, "ctx": 0, "page": 128,
         "token_major": True},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["map", "append", "decode", "decode", "shared", "prompt", "prompt"])
    page = rng.choice([16, 32, 64, 128, 256])
    hkv, group, d = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 5, 8]), rng.choice([64, 128])
    major = rng.random() < 0.5
    if op == "map":
        new = _log(rng, 1, 16384)
        return {"op": "map", "B": _log(rng, 1, 64 if new > 64 else 700), "page": page, "ctx": _log(rng, 1, 20000) if rng.random() < 0.7 else 0,
                "new": new}
    if op == "append":
        return {"op": "append", "T": _log(rng, 1, 40000), "Hkv": hkv, "D": d, "page": page, "f32": rng.random() < 0.4, "token_major": major}
    if op == "prompt":
        new = _log(rng, 2, 4000)
        b = _log(rng, 1, max(1, min(24, 8000 // new)))
        ctx = _log(rng, 1, 12000) if rng.random() < 0.6 else 0
        return {"op": "prompt", "B": b, "Hq": hkv * group, "Hkv": hkv, "D": d, "new": new, "ctx": ctx, "page": page, "token_major": major}
    b = _log(rng, 1, 96)
    most = max(1, 500000 // (b * hkv))
    case = {"op": "decode", "B": b, "Hq": hkv * group, "Hkv": hkv, "Nq": rng.choice([1, 1, 2, 3, 5]), "D": d,
            "len": _log(rng, 1, min(60000, 8 * most)), "page": page, "prefix": 0, "token_major": major}
    if op == "shared":
        case["len"], case["prefix"] = _log(rng, 1, min(3000, 8 * most)), _log(rng, 100, 60000)
    return case


def _ragged(count, most, least):
    """Lengths of a ragged batch: the first is the longest, the others spread between a tenth of it and all of it."""
    got = [max(least, int(most * (0.1 + 0.9 * ((i * 0.6180339887) % 1.0)))) if i else most for i in range(count)]
    if count >= 8:
        got[count // 2] = 0
    return got


def _lengths(case):
    """(context, new) tokens of every sequence."""
    b = case["B"]
    if case["op"] == "decode":
        kv = _ragged(b, case["len"], 1)
        return kv, [0] * b
    new = [1 if n else 0 for n in _ragged(b, 9, 1)] if case["new"] == 1 else _ragged(b, case["new"], 1)
    ctx = _ragged(b, case["ctx"], 0)[::-1] if case["ctx"] else [0] * b
    return ctx, new


def _pool(case, n_pages, gen):
    shape = (n_pages, case["page"], case["Hkv"], case["D"]) if case["token_major"] else (n_pages, case["Hkv"], case["page"], case["D"])
    pages = torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    return pages.transpose(1, 2) if case["token_major"] else pages


def _table(lens, page, order, width=0):
    """Block table [B, width] whose sequences take their pages from `order`, and how many were taken; -1 where there is none."""
    need = [-(-n // page) for n in lens]
    table = torch.full((len(lens), max(1, width, *need)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at : at + n]
        at += n
    return table, at


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    host = torch.Generator()
    host.manual_seed(seed)
    op, page = case["op"], case["page"]
    if op == "append":
        n_pages = -(-case["T"] // page) + 3
        slots = torch.randperm(n_pages * page, generator=host)[: case["T"]]
        slots[:: 29] = -1  # padding tokens have no slot
        rows = [torch.empty((case["T"], case["Hkv"], case["D"]), dtype=torch.float32 if case["f32"] else torch.bfloat16,
                            device="cuda").normal_(generator=gen).transpose(0, 1).unsqueeze(0) for _ in range(2)]
        return {"op": op, "k": rows[0], "v": rows[1], "k_pages": _pool(case, n_pages, gen), "v_pages": _pool(case, n_pages, gen),
                "slots": slots.cuda()}
    ctx, new = _lengths(case)
    total = [c + n for c, n in zip(ctx, new)]
    count = sum(-(-n // page) for n in total) + (-(-case.get("prefix", 0) // page)) + 5
    order = torch.randperm(count, generator=host).to(torch.int32)
    if op == "map":
        width = max(1, max(-(-n // page) for n in total))
        table, taken = _table(ctx, page, order, width)
        return {"op": op, "page": page, "table": table.cuda(), "ctx": _ints(ctx), "new": _ints(new), "free": order[taken:].contiguous().cuda(),
                "tokens": sum(new) + 7}
    table, taken = _table(total, page, order)
    state = {"op": op, "k_pages": _pool(case, count, gen), "v_pages": _pool(case, count, gen), "table": table.cuda(), "lens": _ints(total)}
    if op == "decode":
        state["q"] = torch.empty((case["B"], case["Nq"], case["Hq"], case["D"]), dtype=torch.bfloat16,
                                 device="cuda").normal_(generator=gen).transpose(1, 2)
        state["prefix_len"] = case["prefix"]
        state["prefix_table"] = order[taken : taken + -(-case["prefix"] // page)].cuda() if case["prefix"] else None
    else:
        state["q"] = torch.empty((sum(new), case["Hq"], case["D"]), dtype=torch.bfloat16,
                                 device="cuda").normal_(generator=gen).transpose(0, 1).unsqueeze(0)
        state["cu"] = _ints([sum(new[:b]) for b in range(len(new) + 1)])
        state["most_new"] = max(new)
    return state


# ------------------------------------------------------------------ plain forms
def _plain_map(s):
    page, table, ctx, new, free = s["page"], s["table"], s["ctx"], s["new"], s["free"]
    have, need = (ctx + page - 1) // page, (ctx + new + page - 1) // page
    take = need - have
    off = torch.cumsum(take, 0) - take
    col = torch.arange(table.shape[1], device=table.device)[None]
    at = off[:, None] + col - have[:, None]
    page_id = torch.where(at < free.shape[0], free[at.clamp(0, max(0, free.shape[0] - 1))], -1)
    table.copy_(torch.where((col >= have[:, None]) & (col < need[:, None]), page_id, table))
    ends = torch.cumsum(new, 0)
    cu = torch.cat([torch.zeros_like(ends[:1]), ends]).to(torch.int32)
    t = torch.arange(s["tokens"], device=table.device)
    seq = torch.searchsorted(ends, t, right=True).clamp(max=new.shape[0] - 1)
    pos = ctx[seq] + t - cu[seq]
    where = table[seq, (pos // page).clamp(0, table.shape[1] - 1)].to(torch.int64)
    slots = torch.where((t < ends[-1]) & (where >= 0), where * page + pos % page, -1)
    return [table, slots, cu, (ctx + new).to(torch.int32), take.sum().to(torch.int32).reshape(1)]


def _plain_append(s):
    slots, page = s["slots"], s["k_pages"].shape[2]
    live = torch.nonzero(slots >= 0)[:, 0]
    at = slots[live]
    s["k_pages"][at // page, :, at % page] = s["k"][0][:, live].transpose(0, 1).to(s["k_pages"].dtype)
    s["v_pages"][at // page, :, at % page] = s["v"][0][:, live].transpose(0, 1).to(s["v_pages"].dtype)
    return [s["k_pages"], s["v_pages"]]


def _dense(pages, table):
    """[..., pages] page numbers -> [..., Hkv, keys, D] in 32 bits."""
    got = pages[table.clamp(min=0).long()].transpose(-4, -3)  # [..., Hkv, pages, page, D]
    return got.reshape(*got.shape[:-3], -1, got.shape[-1]).float()


def _softmax(scores):
    """exp(scores - max), its sum and the log of the sum of exponentials; rows of -inf alone give zeros and -inf."""
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    return p, torch.where(total > 0, total, 1.0), (top + torch.log(total))[..., 0]


def _plain_decode(s):
    q = s["q"].float()
    b, hq, nq, d = q.shape
    k, v = _dense(s["k_pages"], s["table"]), _dense(s["v_pages"], s["table"])
    hkv, keys = k.shape[1], k.shape[2]
    rows = q.reshape(b, hkv, hq // hkv * nq, d) / math.sqrt(d)  # row = (head of the group, token)
    scores = rows @ k.transpose(-1, -2)
    last = (s["lens"][:, None] - nq + torch.arange(nq, device=q.device)).repeat(1, hq // hkv)
    scores = torch.where(torch.arange(keys, device=q.device) <= last[:, None, :, None], scores, -math.inf)
    if s["prefix_len"]:
        pk, pv = _dense(s["k_pages"], s["prefix_table"]), _dense(s["v_pages"], s["prefix_table"])
        shared = rows.transpose(0, 1).reshape(hkv, -1, d)
        more = (shared @ pk[:, : s["prefix_len"]].transpose(-1, -2)).reshape(hkv, b, -1, s["prefix_len"]).transpose(0, 1)
        p, total, lse = _softmax(torch.cat([more, scores], -1))
        first = p[..., : s["prefix_len"]].transpose(0, 1).reshape(hkv, -1, s["prefix_len"]) @ pv[:, : s["prefix_len"]]
        o = first.reshape(hkv, b, -1, d).transpose(0, 1) + p[..., s["prefix_len"] :] @ v
    else:
        p, total, lse = _softmax(scores)
        o = p @ v
    return [(o / total).reshape(b, hq, nq, d).to(s["q"].dtype), lse.reshape(b, hq, nq)]


def _plain_prompt(s):
    q, cu, lens = s["q"][0].float(), s["cu"].long(), s["lens"].long()
    hq, tokens, d = q.shape
    k, v = _dense(s["k_pages"], s["table"]), _dense(s["v_pages"], s["table"])
    hkv, keys = k.shape[1], k.shape[2]
    at = cu[:-1, None] + torch.arange(s["most_new"], device=q.device)  # padded [B, most_new] token numbers
    real = at < cu[1:, None]
    rows = q[:, at.clamp(max=tokens - 1)].transpose(0, 1) / math.sqrt(d)  # [B, Hq, most_new, D]
    b = rows.shape[0]
    scores = rows.reshape(b, hkv, -1, d) @ k.transpose(-1, -2)
    last = (lens - cu[1:])[:, None] + at
    seen = torch.arange(keys, device=q.device) <= torch.where(real, last, -1)[:, :, None]
    scores = torch.where(seen[:, None, None], scores.reshape(b, hkv, hq // hkv, -1, keys), -math.inf)
    p, total, lse = _softmax(scores)
    del scores
    o = (p.reshape(b, hkv, -1, keys) @ v).reshape(b, hkv, hq // hkv, -1, d) / total
    take = torch.nonzero(real.reshape(-1))[:, 0]  # padded rows in token order
    o = o.reshape(b, hq, -1, d).transpose(1, 2).reshape(-1, hq, d)[take].transpose(0, 1)
    lse = lse.reshape(b, hq, -1).transpose(1, 2).reshape(-1, hq)[take].transpose(0, 1)
    return [o[None].to(s["q"].dtype), lse[None]]


def run(s):
    if own:
        import long_sequence_exact_gb300 as lsx

        if s["op"] == "map":
            slots, cu, lens, taken = lsx.page_map(s["table"], s["ctx"], s["new"], s["free"], s["page"], s["tokens"])
            return [s["table"], slots, cu, lens, taken]
        if s["op"] == "append":
            lsx.page_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["slots"])
            return [s["k_pages"], s["v_pages"]]
        if s["op"] == "decode":
            return list(lsx.paged_decode(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"],
                                         prefix_table=s["prefix_table"], prefix_len=s["prefix_len"]))
        return list(lsx.paged_fwd(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], s["cu"]))
    return {"map": _plain_map, "append": _plain_append, "decode": _plain_decode, "prompt": _plain_prompt}[s["op"]](s)


def work(case):
    op = case["op"]
    if op == "append":
        live = case["T"] - -(-case["T"] // 29)
        row = case["Hkv"] * case["D"] * 2  # values of K and V
        return {"bytes": live * row * ((4 if case["f32"] else 2) + 2) + 8 * case["T"], "flops": 0}
    ctx, new = _lengths(case)
    b, page = case["B"], case["page"]
    if op == "map":
        take = sum(-(-(c + n) // page) - -(-c // page) for c, n in zip(ctx, new))
        # lengths in, pages taken read and written, slots, offsets and totals out
        return {"bytes": 8 * b + 8 * take + 8 * (sum(new) + 7) + 4 * (b + 1) + 4 * b + 4, "flops": 0}
    d, hq, hkv = case["D"], case["Hq"], case["Hkv"]
    row = 4 * hkv * d  # bytes of a key and its value
    if op == "decode":
        nq, prefix = case["Nq"], case["prefix"]
        pairs = sum(nq * prefix + sum(max(0, n - nq + i + 1) for i in range(nq)) for n in ctx)
        out = b * hq * nq * (2 * d + 2 * d + 4)
        pages = sum(-(-n // page) for n in ctx) + -(-prefix // page)
        return {"bytes": row * (sum(ctx) + prefix) + out + 4 * pages + 4 * b, "flops": 4 * d * hq * pairs}
    pairs = sum(n * c + n * (n + 1) // 2 for c, n in zip(ctx, new))
    total = sum(c + n for c, n in zip(ctx, new) if n)
    pages = sum(-(-(c + n) // page) for c, n in zip(ctx, new) if n)
    return {"bytes": row * total + sum(new) * hq * (4 * d + 4) + 4 * pages + 4 * (2 * b + 1), "flops": 4 * d * hq * pairs}


# ------------------------------------------------------------------ in 64 bits, from the definitions
def _exact_attention(q, k, v, last):
    """Queries q [R, D] over keys in order; row r sees keys 0..last[r]."""
    scores = (q @ k.T) * (q.shape[-1] ** -0.5)
    scores.masked_fill_(torch.arange(k.shape[0], device=q.device)[None] > last[:, None], -math.inf)
    lse = torch.logsumexp(scores, -1)
    weights = torch.exp(scores.sub_(lse[:, None])).nan_to_num_(nan=0.0)
    return weights @ v, lse


def _rows_of(pages, numbers, n):
    """Rows 0..n-1 of the sequence whose pages are `numbers`: [Hkv, n, D] in 64 bits."""
    page = pages.shape[2]
    numbers = numbers[: -(-n // page)].long()
    return pages[numbers].permute(1, 0, 2, 3).flatten(1, 2)[:, :n].double()


def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    if op == "map":
        return _exact_map(s)
    if op == "append":
        return _exact_append(s)
    q = s["q"].double()
    o = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.full(q.shape[:3], -math.inf, dtype=torch.float64, device="cuda")
    lens = s["lens"].tolist()
    group = case["Hq"] // case["Hkv"]
    prefix = case.get("prefix", 0)
    cu = s["cu"].tolist() if op == "prompt" else None
    if prefix:
        pk, pv = (_rows_of(s[x], s["prefix_table"], prefix) for x in ("k_pages", "v_pages"))
    for b, n in enumerate(lens):
        mine = (0, slice(cu[b], cu[b + 1])) if cu else (b, slice(0, q.shape[2]))
        count = mine[1].stop - mine[1].start
        if not count or not (n or prefix):
            continue
        k, v = (_rows_of(s[x], s["table"][b], n) for x in ("k_pages", "v_pages"))
        if prefix:
            k, v = torch.cat([pk, k], 1), torch.cat([pv, v], 1)
        last = prefix + n - count + torch.arange(count, device="cuda")
        last = torch.where(last < prefix, prefix - 1, last)  # a shared prefix is seen whole
        for h in range(case["Hq"]):
            o[mine[0], h, mine[1]], lse[mine[0], h, mine[1]] = _exact_attention(q[mine[0], h, mine[1]], k[h // group], v[h // group], last)
    return [o, lse]


def _exact_map(s):
    """Token by token, as a host program would keep its tables."""
    page, table, free = s["page"], s["table"].tolist(), s["free"].tolist()
    slots, cu, used = [], [0], 0
    for row, c, n in zip(table, s["ctx"].tolist(), s["new"].tolist()):
        for pos in range(c, c + n):
            if pos % page == 0:
                row[pos // page] = free[used] if used < len(free) else -1
                used += 1
            slots.append(row[pos // page] * page + pos % page if row[pos // page] >= 0 else -1)
        cu.append(cu[-1] + n)
    slots += [-1] * (s["tokens"] - len(slots))
    lens = [c + n for c, n in zip(s["ctx"].tolist(), s["new"].tolist())]
    return [torch.tensor(table, dtype=torch.int32), torch.tensor(slots), torch.tensor(cu, dtype=torch.int32),
            torch.tensor(lens, dtype=torch.int32), torch.tensor([used], dtype=torch.int32)]


def _exact_append(s):
    page, got = s["k_pages"].shape[2], []
    for rows, pages in ((s["k"], s["k_pages"]), (s["v"], s["v_pages"])):
        flat = pages.permute(0, 2, 1, 3).double().flatten(0, 1)  # [slots, Hkv, D]
        live = s["slots"] >= 0
        flat[s["slots"][live]] = rows[0].permute(1, 0, 2)[live].double()
        got.append(flat.unflatten(0, (-1, page)).permute(0, 2, 1, 3))
    return got

"""Cases of the paged cache's operators: what they take, their plain forms in elementary torch
operations, and their values from the definitions in 64 bits.

Five operators for the attention layers that stand between the recurrent ones of a hybrid model:
`kv_append` writes the keys and values of a batch of runs (prompt chunks, single tokens, drafted
runs) into the pages of their sequences, `attn_paged` is the causal attention of these runs over
the pages, and `pages_grow`, `pages_fork` and `pages_compact` give sequences pages, let sequences
share what they have in common, and move the pages in use to the front of the pool.  A page is in
use where a row of the table reaches it within its sequence's length; there are no other records.
"""
import math

import torch

own = False


def listed():
    return [
        # decode step of a handful of sequences, where latency counts: one has nothing but this token
        dict(name="attn_token_few", kind="attn", cached="300,0,5000", lengths="1,1,1", Hq=16, Hkv=2, D=128, page=16, window=0),
        # a decode step of 128 sequences of 1000 to 16000 tokens: the cache is read once
        dict(name="attn_token_many", kind="attn", n=128, run=1, lo=1000, hi=16000, Hq=32, Hkv=8, D=128, page=64, window=0),
        # a mixed batch under a window: prompt chunks, single tokens, drafted runs, an empty run, small heads
        dict(name="attn_mixed_window", kind="attn", cached="0,777,8000,4095,64,2000,31,6000,128,1023", lengths="512,1,300,1,5,3,129,1,0,7", Hq=24, Hkv=8, D=64, page=32, window=2048),
        # a chunk of a long prompt behind what earlier chunks left: bound by the products
        dict(name="attn_chunk_long", kind="attn", cached="28672", lengths="4096", Hq=32, Hkv=8, D=128, page=128, window=0),
        # keys and values of one decode step
        dict(name="append_token", kind="append", n=256, run=1, lo=1, hi=4000, Hkv=8, D=128, page=64),
        # those of a batch of prompt chunks, long and short ones
        dict(name="append_packed", kind="append", cached="0,777,4096,31,12000,0", lengths="9000,4096,12001,1,7000,670", Hkv=8, D=128, page=64),
        # a scheduler step of a few sequences
        dict(name="grow_few", kind="grow", slots=8, most=64, lo=1, hi=3000, more=5, page=64, n_pages=1024),
        # one of many sequences over a pool of small pages, some with whole prompts to come
        dict(name="grow_many", kind="grow", slots=512, most=2048, lo=1, hi=16000, more=3000, page=16, n_pages=524288),
        # four continuations of one prompt
        dict(name="fork_few", kind="fork", slots=8, most=64, lo=500, hi=2000, parents=1, children=4, layers=4, Hkv=2, D=128, page=64, n_pages=256),
        # beams of a large batch: the last page of 224 sequences in every layer
        dict(name="fork_many", kind="fork", slots=256, most=32, lo=60, hi=600, parents=32, children=7, layers=16, Hkv=8, D=128, page=64, n_pages=1600),
        # a small pool after some sequences ended
        dict(name="compact_few", kind="compact", slots=8, most=32, lo=200, hi=1000, layers=2, Hkv=2, D=64, page=32, n_pages=512),
        # a large pool, half of it in use
        dict(name="compact_many", kind="compact", slots=256, most=64, lo=60, hi=2000, layers=4, Hkv=8, D=128, page=64, n_pages=4300),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["attn", "attn", "attn", "attn", "append", "append", "grow", "fork", "compact"])
    Hkv, D, page = rng.choice([1, 2, 3, 4, 8]), rng.choice([64, 128, 128]), rng.choice([16, 32, 64, 128])
    c = dict(kind=kind, Hkv=Hkv, D=D, page=page)
    if kind == "attn":
        c["Hq"] = Hkv * rng.choice([1, 2, 3, 4, 5, 8, 16] if Hkv < 4 else [1, 2, 3, 4])
        c["window"] = rng.choice([0, 0, 0, 128, 1000, 4096])
        what = rng.choice(["tokens", "drafts", "mixed", "chunk"])
        if what in ("tokens", "drafts"):
            hi = _log(rng, 100, 12000)
            return dict(c, n=_log(rng, 1, 96), run=1 if what == "tokens" else rng.randint(2, 8), lo=rng.randint(0, hi // 2), hi=hi)
        n = rng.randint(3, 10) if what == "mixed" else 1
        cached = [rng.choice([0, _log(rng, 1, 6000)]) for _ in range(n)]
        new = [rng.choice([1, 1, rng.randint(2, 9), _log(rng, 1, 500), 0]) for _ in range(n)]
        if what == "chunk":
            cached, new = [_log(rng, 1, 24000)], [_log(rng, 16, 2000)]
        return dict(c, cached=",".join(map(str, cached)), lengths=",".join(map(str, new if any(new) else [1] * n)))
    if kind == "append":
        if rng.random() < 0.5:
            hi = _log(rng, 10, 4000)
            return dict(c, n=_log(rng, 1, 256), run=rng.choice([1, 1, 3, 6]), lo=0, hi=hi)
        n = rng.randint(1, 8)
        return dict(c, cached=",".join(str(rng.choice([0, _log(rng, 1, 8000)])) for _ in range(n)),
                    lengths=",".join(str(_log(rng, 1, 32000 // n)) for _ in range(n)))
    slots, hi = _log(rng, 2, 256), _log(rng, 20, 2000)
    most = -(-hi // page) + 8
    c = dict(c, slots=slots, most=most, lo=rng.randint(0, hi // 2), hi=hi)
    need = slots * -(-hi // page)
    if kind == "grow":
        used = sum(-(-v // page) for v in _spread(slots, c["lo"], hi))
        return dict(kind=kind, slots=slots, most=most, lo=c["lo"], hi=hi, more=rng.randint(1, 6 * page), page=page, n_pages=int(used * rng.uniform(1, 4)) + 8)
    layers = max(1, min(rng.randint(1, 8), (3 << 30) // (need * 8 * Hkv * page * D)))
    if kind == "fork":
        parents = rng.randint(1, max(1, slots // 3))
        return dict(c, layers=layers, parents=parents, children=rng.randint(1, max(1, slots // parents - 1)), n_pages=need + slots)
    return dict(c, layers=layers, n_pages=int(need * rng.uniform(1, 2)) + 8)


def _runs(case):
    """(tokens in the cache before each run, tokens of each run)"""
    if "lengths" in case:
        return [int(v) for v in case["cached"].split(",")], [int(v) for v in case["lengths"].split(",")]
    n, run, lo, hi = (case[k] for k in ("n", "run", "lo", "hi"))
    return _spread(n, lo, hi), [1 + (7919 * b + run - 1) % run for b in range(n)]


def _spread(n, lo, hi):
    """n lengths between lo and hi, in no order."""
    return [lo + (hi - lo) * ((b * 37 + 11) % n + 1) // n if n > 1 else hi for b in range(n)]


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen, device=dev, dtype=torch.bfloat16)  # noqa: E731
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    kind, page = case["kind"], case["page"]
    s = dict(case=case, kind=kind, page=page)
    if kind in ("attn", "append"):
        cached, new = _runs(case)
        n, Hkv, D = len(new), case["Hkv"], case["D"]
        cu = [0]
        for v in new:
            cu.append(cu[-1] + v)
        total = cu[-1]
        need = [-(-(a + b) // page) for a, b in zip(cached, new)]
        n_pages, n_slots = sum(need) + sum(need) // 8 + 2, n + n // 4 + 1
        # sequences' pages lie anywhere in the pool, their slots in no order
        at = torch.randperm(n_pages, generator=gen, device=dev).int()
        slots = torch.randperm(n_slots, generator=gen, device=dev)[:n]
        table = torch.full((n_slots, max(need) + 3), -1, dtype=torch.int32, device=dev)
        lens = torch.zeros(n_slots, dtype=torch.int32, device=dev)
        lens[slots] = ints(cached)
        i = torch.arange(table.shape[1], device=dev)
        first = torch.tensor([sum(need[:b]) for b in range(n)], device=dev)
        rows = first[:, None] + i
        table[slots] = torch.where(i < ints(need)[:, None], at[rows.clamp(max=n_pages - 1)], -1)
        s.update(table=table, lens=lens, slots=slots.int(), cu=ints(cu), cached=cached, new=new, total=total,
                 cu_arg=None if all(v == 1 for v in new) else ints(cu), cache=rnd(n_pages, 2, Hkv, page, D))
        # q, k and v are slices of one projection, as the layer makes them
        H = case.get("Hq", Hkv)
        qkv = rnd(total, (H + 2 * Hkv) * D)
        s["q"] = qkv[:, :H * D].view(total, H, D)
        s["k"] = qkv[:, H * D:(H + Hkv) * D].view(total, Hkv, D)
        s["v"] = qkv[:, (H + Hkv) * D:].view(total, Hkv, D)
        return s
    n_slots, most, n_pages = case["slots"], case["most"], case["n_pages"]
    lens = _spread(n_slots, case["lo"], case["hi"])
    if kind == "grow":
        # lengths jump about: by drafted runs, and by a whole prompt for some
        s["want"] = ints([v + (case["more"] if b % 3 == 0 else b % 7) for b, v in enumerate(lens)])
    if kind == "fork":
        P, C = case["parents"], case["children"]
        order = torch.randperm(n_slots, generator=gen, device=dev)
        s["src"] = order[:P].repeat_interleave(C).int()
        s["dst"] = order[P:P + P * C].int()
    if kind == "compact":
        # every other sequence has ended
        lens = [v if b % 2 == 0 else 0 for b, v in enumerate(lens)]
    order = torch.randperm(n_slots, generator=gen, device=dev)
    s["lens"] = ints(lens)[order]
    need = ((s["lens"] + page - 1) // page).long()
    first = need.cumsum(0) - need
    i = torch.arange(most, device=dev)
    at = torch.randperm(n_pages, generator=gen, device=dev).int()
    at = torch.cat([at, torch.full((1,), -1, dtype=torch.int32, device=dev)])
    rows = torch.where(i < need[:, None], (first[:, None] + i).clamp(max=n_pages), n_pages)
    s["table"] = at[rows]
    if kind != "grow":
        s["cache"] = rnd(case["layers"], n_pages, 2, case["Hkv"], page, case["D"])
    return s


def run(state):
    return (_own if own else _plain)(state)


def _own(s):
    import linear_attention_serving_chunk_gb300 as kda
    kind = s["kind"]
    if kind == "attn":
        return kda.attn_paged(s["q"], s["cache"], s["table"], s["lens"], slots=s["slots"], cu_seqlens=s["cu_arg"], window=s["case"]["window"])
    if kind == "append":
        kda.kv_append(s["k"], s["v"], s["cache"], s["table"], s["lens"], slots=s["slots"], cu_seqlens=s["cu_arg"])
        return s["cache"]
    if kind == "grow":
        left = kda.pages_grow(s["table"], s["lens"], s["want"], s["page"], s["case"]["n_pages"])
        return s["table"], left
    if kind == "fork":
        left = kda.pages_fork(s["cache"], s["table"], s["lens"], s["src"], s["dst"])
        return s["cache"], s["table"], s["lens"], left
    table, used = kda.pages_compact(s["cache"], s["table"], s["lens"])
    return s["cache"], table, used


def _plain(s):
    return {"attn": _plain_attn, "append": _plain_append, "grow": _plain_grow, "fork": _plain_fork, "compact": _plain_compact}[s["kind"]](s)


def _token_of(s):
    """(run, position in it) of every token."""
    t = torch.arange(s["total"], device=s["cu"].device)
    b = torch.searchsorted(s["cu"][1:].long(), t, right=True)
    return b, t - s["cu"].long()[b]


def _plain_attn(s):
    """All runs at once, padded to the longest run and the longest context."""
    c, q = s["case"], s["q"]
    Hq, Hkv, D, page = (c[k] for k in ("Hq", "Hkv", "D", "page"))
    G, n, longest = Hq // Hkv, len(s["new"]), max(s["new"])
    reach = max(a + b for a, b in zip(s["cached"], s["new"]))
    pages = -(-reach // page)
    slots = s["slots"].long()
    kv = s["cache"][s["table"][slots, :pages].long().clamp(min=0)]  # n, page, 2, head, token, D
    kv = kv.permute(2, 0, 3, 1, 4, 5).reshape(2, n, Hkv, pages * page, D)[:, :, :, :reach]
    b, pos = _token_of(s)
    qp = torch.zeros(n, longest, Hkv, G, D, device=q.device)
    qp[b, pos] = q.view(-1, Hkv, G, D).float()
    S = torch.matmul(qp.permute(0, 2, 1, 3, 4).reshape(n, Hkv, longest * G, D), kv[0].float().transpose(2, 3))
    S = S.view(n, Hkv, longest, G, reach)
    S *= 1 / math.sqrt(D)
    # token j of a run stands at position cached + j: it sees what is not behind it, under a
    # window the last `window` positions
    at = s["lens"][slots].long()[:, None] + torch.arange(longest, device=q.device)
    j = torch.arange(reach, device=q.device)
    hidden = j > at[:, :, None]
    if c["window"]:
        hidden |= j <= at[:, :, None] - c["window"]
    S.masked_fill_(hidden[:, None, :, None], -math.inf)
    S -= S.amax(-1, keepdim=True).clamp(min=-3e38)
    S = S.exp_()
    total = S.sum(-1, keepdim=True)
    # padded places hold what another sequence left there: they count as zero
    seen = j < (s["lens"][slots] + (s["cu"][1:] - s["cu"][:-1]))[:, None]
    v = kv[1].float().masked_fill(~seen[:, None, :, None], 0.0)
    o = torch.matmul(S.view(n, Hkv, longest * G, reach), v).view(n, Hkv, longest, G, D) / total
    return o.permute(0, 2, 1, 3, 4)[b, pos].reshape(-1, Hq, D).to(q.dtype)


def _plain_append(s):
    b, pos = _token_of(s)
    slot = s["slots"].long()[b]
    at = s["lens"].long()[slot] + pos
    pages, rows = s["table"][slot, at // s["page"]].long(), at % s["page"]
    s["cache"][pages, 0, :, rows] = s["k"]
    s["cache"][pages, 1, :, rows] = s["v"]
    return s["cache"]


def _marked(table, need, n_pages):
    """Whether each page is in use: reached by a row within its pages."""
    i = torch.arange(table.shape[1], device=table.device)
    mark = torch.zeros(n_pages + 1, dtype=torch.bool, device=table.device)
    mark[torch.where(i < need[:, None], table, n_pages).long()] = True
    return mark[:n_pages]


def _plain_grow(s):
    table, page, n_pages = s["table"], s["page"], s["case"]["n_pages"]
    have = (s["lens"].long() + page - 1) // page
    more = ((s["want"].long() + page - 1) // page - have).clamp(min=0)
    mark = _marked(table, have, n_pages)
    free = torch.argsort(mark.int(), stable=True)
    left = n_pages - mark.sum()
    end = more.cumsum(0)
    i = torch.arange(table.shape[1], device=table.device)
    rank = (end - more)[:, None] + i - have[:, None]
    # a row gets all of its pages or none; the first rows come first
    new = torch.where((end <= left)[:, None], free[rank.clamp(0, n_pages - 1)], -1).int()
    table.copy_(torch.where((i >= have[:, None]) & (i < (have + more)[:, None]), new, table))
    return table, (left - end[-1]).int().view(1)


def _plain_fork(s):
    cache, table, lens, page = s["cache"], s["table"], s["lens"], s["page"]
    n_pages = cache.shape[1]
    src, dst = s["src"].long(), s["dst"].long()
    have = (lens.long() + page - 1) // page
    alive = have.clone()
    alive[dst] = 0
    mark = _marked(table, alive, n_pages)
    free = torch.argsort(mark.int(), stable=True)
    left = n_pages - mark.sum()
    tail = lens[src].long() % page
    rank = (tail > 0).long().cumsum(0)
    i = torch.arange(table.shape[1], device=table.device)
    new = free[(rank - 1).clamp(0, n_pages - 1)].int()
    last = (tail > 0)[:, None] & (i == have[src][:, None] - 1)
    rows = torch.where(last, new[:, None], table[src])
    rows = torch.where(i < have[src][:, None], rows, -1)
    k = torch.nonzero(tail > 0)[:, 0]
    old = table[src[k], have[src[k]] - 1].long()
    keep = (torch.arange(page, device=table.device) < tail[k][:, None])[:, None, None, :, None]
    cache[:, new[k].long()] = torch.where(keep, cache[:, old], cache[:, new[k].long()])
    table[dst] = rows
    lens[dst] = lens[src]
    return cache, table, lens, (left - rank[-1]).int().view(1)


def _plain_compact(s):
    cache, table, page = s["cache"], s["table"], s["page"]
    n_pages = cache.shape[1]
    need = (s["lens"].long() + page - 1) // page
    mark = _marked(table, need, n_pages)
    used = mark.sum()
    p = torch.arange(n_pages, device=table.device)
    src, dst = torch.nonzero(mark & (p >= used))[:, 0], torch.nonzero(~mark & (p < used))[:, 0]
    cache[:, dst] = cache[:, src]
    now = p.int()
    now[src] = dst.int()
    i = torch.arange(table.shape[1], device=table.device)
    return cache, torch.where(i < need[:, None], now[table.clamp(min=0).long()], -1), used.int().view(1)


def work(case):
    kind, page = case["kind"], case["page"]
    if kind in ("attn", "append"):
        cached, new = _runs(case)
        Hkv, D, total = case["Hkv"], case["D"], sum(new)
        if kind == "append":
            return {"bytes": 8 * total * Hkv * D, "flops": 0}
        w, pairs, reach = case["window"], 0, 0
        for a, n in zip(cached, new):
            if n:
                pairs += sum(min(a + t + 1, w) for t in range(n)) if w else n * a + n * (n + 1) // 2
                reach += min(a + n, w + n - 1) if w else a + n
        return {"bytes": 4 * reach * Hkv * D + 4 * total * case["Hq"] * D, "flops": 4 * pairs * case["Hq"] * D}
    lens = _spread(case["slots"], case["lo"], case["hi"])
    if kind == "grow":
        more = sum(max(0, -(-(v + (case["more"] if b % 3 == 0 else b % 7)) // page) - -(-v // page)) for b, v in enumerate(lens))
        return {"bytes": 4 * (sum(-(-v // page) for v in lens) + more + 2 * len(lens)), "flops": 0}
    one = 4 * case["layers"] * case["Hkv"] * case["D"]  # bytes of a token in all layers
    if kind == "fork":
        m = case["parents"] * case["children"]
        tail = sum(v % page for v in lens) / len(lens)
        pages = sum(-(-v // page) for v in lens)
        return {"bytes": 2 * m * tail * one + 4 * (pages + m * (2 * pages / len(lens) + 4)), "flops": 0}
    pages = sum(-(-v // page) for b, v in enumerate(lens) if b % 2 == 0)
    moved = pages * max(0, case["n_pages"] - pages) / case["n_pages"]
    return {"bytes": 2 * moved * page * one + 4 * (pages + case["slots"] * (case["most"] + 1)), "flops": 0}


def exact(case, seed):
    if case["kind"] != "attn":
        return None  # whole numbers, and values that are moved
    s = prepare(case, seed)
    Hq, Hkv, D, page, w = (case[k] for k in ("Hq", "Hkv", "D", "page", "window"))
    G, at, out = Hq // Hkv, 0, torch.zeros(s["total"], Hq, D, dtype=torch.float64, device="cuda")
    slots = s["slots"].tolist()
    for b, (a, n) in enumerate(zip(s["cached"], s["new"])):
        reach = a + n
        pages = s["table"][slots[b], :-(-reach // page)].long()
        kv = s["cache"][pages].transpose(0, 1).transpose(1, 2)  # 2, head, page, token, D after the next line
        kv = kv.reshape(2, Hkv, -1, D)[:, :, :reach] if n else None
        for h in range(Hq if n else 0):
            k, v = kv[0, h // G].double(), kv[1, h // G].double()
            for t in range(0, n, 1024):
                m = min(1024, n - t)
                S = (s["q"][at + t:at + t + m, h].double() @ k.t()) / math.sqrt(D)
                row = torch.arange(a + t, a + t + m, device="cuda")[:, None]
                col = torch.arange(reach, device="cuda")
                see = (col <= row) & ((col > row - w) if w else (col >= 0))
                S = torch.where(see, torch.exp(S - torch.where(see, S, -math.inf).max(1, keepdim=True)[0]), 0.0)
                out[at + t:at + t + m, h] = (S @ v) / S.sum(1, keepdim=True)
        at += n
    return out

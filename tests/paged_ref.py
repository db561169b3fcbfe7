"""Plain forms of the paged cache's operators, token by token and page by page from their
descriptions in include/kda.h, and the inputs of their tests.  CPU tensors and lists in and out."""
import torch


def pages_of(tokens, page, most):
    """Pages of a sequence, None where its row cannot hold them."""
    n = -(-tokens // page)
    return None if tokens < 0 or n > most else n


def in_use(table, lens, page, n_pages, without=()):
    got = set()
    for b, row in enumerate(table.tolist()):
        if b not in without:
            got |= set(row[:pages_of(int(lens[b]), page, len(row)) or 0])
    return {p for p in got if 0 <= p < n_pages}


def grow(table, lens, want, page, n_pages):
    """(table, left)"""
    table, most = table.clone(), table.shape[1]
    used = in_use(table, lens, page, n_pages)
    free = [p for p in range(n_pages) if p not in used]
    at = 0
    for b in range(len(lens)):
        have, need = pages_of(int(lens[b]), page, most), pages_of(int(want[b]), page, most)
        if have is None or need is None or need <= have:
            continue
        more = need - have
        table[b, have:need] = torch.tensor(free[at:at + more] if at + more <= len(free) else [-1] * more)
        at += more
    return table, len(free) - at


def fork(cache, table, lens, src, dst, page):
    """(cache, table, lens, left); cache [layers, n_pages, 2, H, page, D]"""
    cache, table, lens = cache.clone(), table.clone(), lens.clone()
    n_slots, most = table.shape
    n_pages = cache.shape[1]
    ok = [0 <= s < n_slots and 0 <= d < n_slots for s, d in zip(src, dst)]
    taken = {}
    for i, d in enumerate(dst):
        if ok[i]:
            taken.setdefault(d, i)
    made = [i for i in range(len(src)) if ok[i] and taken[dst[i]] == i and src[i] not in taken
            and pages_of(int(lens[src[i]]), page, most) is not None]
    used = in_use(table, lens, page, n_pages, without={dst[i] for i in made})
    free = [p for p in range(n_pages) if p not in used]
    at = 0
    for i in made:
        tokens = int(lens[src[i]])
        n, tail = -(-tokens // page), tokens % page
        row = table[src[i], :n].tolist()
        if tail:
            if at < len(free):
                old, row[-1] = row[-1], free[at]
                if 0 <= old < n_pages:
                    cache[:, free[at], :, :, :tail] = cache[:, old, :, :, :tail]
            else:
                row, tokens = [], 0
            at += 1
        table[dst[i]] = torch.tensor(row + [-1] * (most - len(row)))
        lens[dst[i]] = tokens
    return cache, table, lens, len(free) - at


def compact(cache, table, lens, page):
    """(cache, table, used)"""
    cache, table = cache.clone(), table.clone()
    n_pages, most = cache.shape[1], table.shape[1]
    used = in_use(table, lens, page, n_pages)
    u = len(used)
    src = sorted(p for p in used if p >= u)
    now = dict(zip(src, sorted(p for p in range(u) if p not in used)))
    for p, q in now.items():
        cache[:, q] = cache[:, p]
    for b in range(len(lens)):
        n = pages_of(int(lens[b]), page, most) or 0
        row = table[b, :n].tolist()
        table[b] = torch.tensor([now.get(p, p) for p in row] + [-1] * (most - n))
    return cache, table, u


def append(k, v, cache, table, lens, slots, cu, page):
    cache = cache.clone()
    for b, s in enumerate(slots):
        for j in range(cu[b + 1] - cu[b]):
            at = int(lens[s]) + j
            p = int(table[s, at // page]) if at // page < table.shape[1] else -1
            if 0 <= p < cache.shape[0]:
                cache[p, 0, :, at % page] = k[cu[b] + j]
                cache[p, 1, :, at % page] = v[cu[b] + j]
    return cache


def gathered(cache, table, slot, reach):
    """Keys and values [2, H, reach, D] in float64 of the first `reach` tokens of a slot; pages
    outside the pool count as zeros."""
    n_pages, _, H, page, D = cache.shape
    out = torch.zeros(2, H, reach, D, dtype=torch.float64)
    for i in range(-(-reach // page)):
        p, n = int(table[slot, i]), min(page, reach - i * page)
        if 0 <= p < n_pages:
            out[:, :, i * page:i * page + n] = cache[p, :, :, :n].double()
    return out


def attention(q, cache, table, lens, slots, cu, window=0, scale=None):
    """(o, size): the attention in float64, and the same sums with the values' magnitudes."""
    total, Hq, D = q.shape
    G = Hq // cache.shape[2]
    scale = D ** -0.5 if scale is None else scale
    o, size = torch.zeros(total, Hq, D, dtype=torch.float64), torch.zeros(total, Hq, D, dtype=torch.float64)
    for b, s in enumerate(slots):
        n, before = cu[b + 1] - cu[b], int(lens[s])
        if n == 0:
            continue
        kv = gathered(cache, table, s, before + n)
        at = torch.arange(before, before + n)[:, None]
        j = torch.arange(before + n)
        see = (j <= at) & (j > at - window if window else j >= 0)
        for h in range(Hq):
            k, v = kv[0, h // G], kv[1, h // G]
            x = (q[cu[b]:cu[b + 1], h].double() @ k.t()) * scale
            w = torch.softmax(x.masked_fill(~see, float("-inf")), 1)
            o[cu[b]:cu[b + 1], h] = w @ v
            size[cu[b]:cu[b + 1], h] = w @ v.abs()
    return o, size


def offsets(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def sequences(reach, n_slots, page, seed, spare=2, most=None):
    """(table [n_slots, most], slots, n_pages): sequences of `reach` tokens at random pages of a
    pool and random slots."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-r // page) for r in reach]
    n_pages = sum(need) + spare
    at, slots = torch.randperm(n_pages, generator=g).tolist(), torch.randperm(n_slots, generator=g)[:len(reach)]
    table = torch.full((n_slots, (max(need) if need else 0) + 1 if most is None else most), -1, dtype=torch.int32)
    for s, n in zip(slots.tolist(), need):
        table[s, :n] = torch.tensor(at[:n], dtype=torch.int32)
        at = at[n:]
    return table, slots.int(), n_pages

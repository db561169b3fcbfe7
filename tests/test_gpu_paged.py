"""The paged cache on the GPU: appending to it and its pages, against plain forms
(tests/paged_ref.py).  Everything here is whole numbers and moved values: equal or wrong."""
import random

import pytest
import torch

import linear_attention_serving_chunk_gb300 as kda
import paged_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def clean_status():
    kda.device_status()
    yield
    assert kda.device_status() == 0  # (a test that expects a code has read it)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def noise(*shape, seed=0):
    """Random bits: every pattern of bf16, NaN among them; compared as integers."""
    g = torch.Generator().manual_seed(seed)
    return torch.randint(-2 ** 15, 2 ** 15, shape, generator=g, dtype=torch.int16).view(torch.bfloat16)


def same(a, b):
    return torch.equal(a.cpu().view(torch.int16), b.cpu().view(torch.int16))


# ---- kv_append ---------------------------------------------------------------------------------

@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("H,D", [(1, 64), (3, 64), (2, 128), (8, 128)])
@pytest.mark.parametrize("lens", [[1], [0], [1] * 9, [0, 1, 77, 0, 300, 5]])
def test_append(page, H, D, lens):
    cached = [(b * 53) % 200 for b in range(len(lens))]
    n_slots = len(lens) + 2
    table, slots, n_pages = ref.sequences([a + n for a, n in zip(cached, lens)], n_slots, page, page + H)
    held = torch.full((n_slots,), 7, dtype=torch.int32)
    held[slots.long()] = torch.tensor(cached, dtype=torch.int32)
    cu, total = ref.offsets(lens), sum(lens)
    rows = noise(total, 2 * H * D + 8, seed=1)  # k and v are slices
    k, v = rows[:, 8:8 + H * D].view(total, H, D), rows[:, 8 + H * D:].view(total, H, D)
    cache = noise(n_pages, 2, H, page, D, seed=2)
    want = ref.append(k, v, cache, table, held, slots.tolist(), cu, page)
    r, c = rows.cuda(), cache.cuda()
    args = (r[:, 8:8 + H * D].view(total, H, D), r[:, 8 + H * D:].view(total, H, D), c, table.cuda(), held.cuda())
    kda.kv_append(*args, slots=slots.cuda(), cu_seqlens=ints(cu))
    assert same(c, want)
    if all(n == 1 for n in lens):
        c.copy_(cache)
        kda.kv_append(*args, slots=slots.cuda())
        assert same(c, want)


def test_append_leaves_what_it_cannot_place():
    """A bad slot, a negative length, pages outside the pool, a row that ends: recorded, the other
    tokens stand; tokens behind the last run are not looked at."""
    page, H, D = 16, 2, 64
    lens = [3, 20, 2, 5, 4]
    cu, total = ref.offsets(lens), sum(lens) + 6
    k, v = noise(total, H, D, seed=1), noise(total, H, D, seed=2)
    cache = noise(8, 2, H, page, D, seed=3)
    table = torch.tensor([[0, 1], [2, 9], [3, -1], [4, 5], [6, 7]], dtype=torch.int32)
    held = torch.tensor([1, 14, 15, 30, -1], dtype=torch.int32)
    for slots in ([0, 1, 2, 3, 4], [0, 1, -1, 5, 2 ** 31 - 1]):
        c = cache.cuda()
        kda.kv_append(k.cuda(), v.cuda(), c, table.cuda(), held.cuda(), slots=ints(slots), cu_seqlens=ints(cu))
        assert kda.device_status() == kda.KDA_ERR_SHAPE
        good = [b for b, s in enumerate(slots) if 0 <= s < 5 and held[s] >= 0]
        want = cache
        for b in good:
            want = ref.append(k[cu[b]:cu[b + 1]], v[cu[b]:cu[b + 1]], want, table, held, [slots[b]], [0, lens[b]], page)
        assert same(c, want)
    c = cache.cuda()
    kda.kv_append(k.cuda(), v.cuda(), c, table.cuda(), held.cuda(), slots=ints([0]), cu_seqlens=ints([0, 4]))
    assert same(c, ref.append(k, v, cache, table, held, [0], [0, 4], page))
    for cu in ([5, 3], [-4, 3], [0, 1 << 30]):
        c = cache.cuda()
        kda.kv_append(k.cuda(), v.cuda(), c, table.cuda(), held.cuda(), slots=ints([0]), cu_seqlens=ints(cu))
        assert kda.device_status() == kda.KDA_ERR_SHAPE
        assert same(c, cache)


def test_append_of_runs_inside_the_rows():
    """Rows in front of the first run and behind the last are left out, and are no fault; so they are for
    the attention that follows."""
    page, H, D = 16, 2, 64
    cu, total, cached = [5, 8, 8, 45], 50, [3, 40, 0]
    table = torch.tensor([[4, 0, -1], [-1, -1, -1], [2, 5, 1]], dtype=torch.int32)
    table[1] = torch.tensor([3, 6, 7])
    k, v = torch.randn(total, H, D).bfloat16(), torch.randn(total, H, D).bfloat16()
    cache = torch.randn(8, 2, H, page, D).bfloat16()
    want = ref.append(k, v, cache, table, torch.tensor(cached), [0, 1, 2], cu, page)
    c = cache.cuda()
    kda.kv_append(k.cuda(), v.cuda(), c, table.cuda(), ints(cached), cu_seqlens=ints(cu))
    assert kda.device_status() == 0
    assert same(c, want)
    o = noise(total, H, D, seed=4)
    got = kda.attn_paged(k.cuda(), c, table.cuda(), ints(cached), cu_seqlens=ints(cu), o=o.cuda())
    assert kda.device_status() == 0
    assert same(got[:5], o[:5]) and same(got[45:], o[45:])
    assert bool(torch.isfinite(got[5:45].float()).all())


def test_append_beyond_32_bits():
    """Pages whose offsets pass 2^32 elements."""
    H, page, D = 8, 128, 128
    n_pages = (1 << 32) // (2 * H * page * D) + 40
    cache = torch.empty(n_pages, 2, H, page, D, dtype=torch.bfloat16, device="cuda")
    table, held = ints([[n_pages - 1, 0], [n_pages - 7, 1]]), ints([127, 5])
    k, v = noise(2, H, D, seed=1), noise(2, H, D, seed=2)
    kda.kv_append(k.cuda(), v.cuda(), cache, table, held)
    for b, (p, r) in enumerate([(n_pages - 1, 127), (n_pages - 7, 5)]):
        assert same(cache[p, 0, :, r], k[b]) and same(cache[p, 1, :, r], v[b])


# ---- pages -------------------------------------------------------------------------------------

def draw_sequences(rng, n_slots, most, page, n_pages, shared=True):
    """A table with sequences of all lengths, some sharing pages, and what lies behind them."""
    lens = [rng.choice([0, 1, page, page - 1, rng.randint(0, most * page), most * page]) for _ in range(n_slots)]
    table = torch.tensor([[rng.randint(-3, n_pages + 2) for _ in range(most)] for _ in range(n_slots)],
                         dtype=torch.int32).view(n_slots, most)
    free = rng.sample(range(n_pages), n_pages)
    for b in range(n_slots):
        need = -(-lens[b] // page)
        if need > len(free):
            lens[b] = need = 0
        got, free = free[:need], free[need:]
        if shared and b and rng.random() < 0.4:
            both = min(need, -(-lens[b - 1] // page)) // 2
            got[:both] = table[b - 1, :both].tolist()
        if need:
            table[b, :need] = torch.tensor(got, dtype=torch.int32)
    return table, torch.tensor(lens, dtype=torch.int32)


SHAPES = [(1, 1, 16, 1), (3, 4, 16, 33), (40, 9, 32, 200), (300, 20, 64, 2500), (7, 70, 128, 600), (1100, 3, 16, 4000)]


@pytest.mark.parametrize("n_slots,most,page,n_pages", SHAPES)
@pytest.mark.parametrize("full", [False, True])
def test_grow(n_slots, most, page, n_pages, full):
    rng = random.Random(n_slots + full)
    table, lens = draw_sequences(rng, n_slots, most, page, n_pages)
    # (full: more than there is, so that some rows get none)
    want = torch.tensor([rng.randint(0, most * page) if full or rng.random() < 0.3 else int(v) + rng.randint(0, 3)
                         for v in lens], dtype=torch.int32).clamp(max=most * page)
    expect, left = ref.grow(table, lens, want, page, n_pages)
    t = table.cuda()
    got = kda.pages_grow(t, lens.cuda(), want.cuda(), page, n_pages)
    assert got.tolist() == [left] and torch.equal(t.cpu(), expect)
    assert kda.pages_grow(t, lens.cuda(), want.cuda(), page, n_pages).tolist() == [left]
    assert torch.equal(t.cpu(), expect)  # lens has not changed: the same again


@pytest.mark.parametrize("n_pages", [1 << 20, (1 << 20) - 31, 70000])
def test_grow_of_a_large_pool(n_pages):
    """All of the pool goes to three rows, all but two pages of it in use before the fourth."""
    third = n_pages // 3
    table = torch.full((4, third + 9), -1, dtype=torch.int32, device="cuda")
    lens = ints([0, 0, 0, 0])
    want = ints([16 * third - 3, 16 * third, 16 * (n_pages - 2 - 2 * third), 17])
    assert kda.pages_grow(table, lens, want, 16, n_pages).tolist() == [0]
    rows = torch.cat([table[0, :third], table[1, :third], table[2, :n_pages - 2 - 2 * third], table[3, :2]])
    assert torch.equal(rows, torch.arange(n_pages, dtype=torch.int32, device="cuda"))
    more = want + ints([16, 0, 0, 0])
    assert kda.pages_grow(table, want, more, 16, n_pages).tolist() == [-1]
    assert table[0, third].item() == -1 and table[0, third - 1].item() == third - 1


def test_grow_leaves_what_is_malformed():
    table = torch.tensor([[0, 1], [5, 9], [2, 3], [4, 4]], dtype=torch.int32)
    for lens, want in (([16, -1, 40, 3], [32, 5, 32, 17]), ([16, 32, 0, 3], [1, 33, -5, 40])):
        t = table.cuda()
        expect, left = ref.grow(table, torch.tensor(lens), torch.tensor(want), 16, 8)
        assert kda.pages_grow(t, ints(lens), ints(want), 16, 8).tolist() == [left]
        assert kda.device_status() == kda.KDA_ERR_SHAPE and torch.equal(t.cpu(), expect)


@pytest.mark.parametrize("layers", [1, 3])
@pytest.mark.parametrize("n_slots,most,page,n_pages", SHAPES[1:])
def test_fork(n_slots, most, page, n_pages, layers):
    """Drawn forks, well-formed ones and others: rows taken twice, parents that are taken, indices
    outside the table, no page left."""
    rng = random.Random(n_slots * layers)
    table, lens = draw_sequences(rng, n_slots, most, page, n_pages, shared=False)
    cache = noise(layers, n_pages, 2, 1, page, 64, seed=n_slots)
    for wild in (False, True):
        if wild:
            n = n_slots
            src = [rng.randint(-1, n_slots) for _ in range(n)]
            dst = [rng.randint(-1, n_slots) for _ in range(n)]
        else:
            order = rng.sample(range(n_slots), n_slots)
            parents = order[:max(1, n_slots // 4)]
            dst = order[len(parents):]
            src = [rng.choice(parents) for _ in dst]
        want = ref.fork(cache, table, lens, src, dst, page)
        c, t, ln = cache.cuda(), table.cuda(), lens.cuda()
        left = kda.pages_fork(c, t, ln, ints(src), ints(dst))
        assert left.tolist() == [want[3]]
        assert torch.equal(t.cpu(), want[1]) and torch.equal(ln.cpu(), want[2]) and same(c, want[0])
        assert kda.device_status() == (kda.KDA_ERR_SHAPE if wild else 0)


def test_fork_without_pages_and_with_a_bad_tail():
    page = 16
    table = torch.tensor([[0, 1, 2], [7, 7, 7], [7, 7, 7], [3, 9, -1]], dtype=torch.int32)
    lens = torch.tensor([40, 0, 0, 20], dtype=torch.int32)
    cache = noise(1, 5, 2, 2, page, 64)
    for src, dst, status in (([0, 0, 3], [1, 2, 9], kda.KDA_ERR_SHAPE), ([0, 0], [1, 2], kda.KDA_ERR_SHAPE),
                             ([3], [1], kda.KDA_ERR_SHAPE)):
        want = ref.fork(cache, table, lens, src, dst, page)
        c, t, ln = cache.cuda(), table.cuda(), lens.cuda()
        assert kda.pages_fork(c, t, ln, ints(src), ints(dst)).tolist() == [want[3]]
        assert torch.equal(t.cpu(), want[1]) and torch.equal(ln.cpu(), want[2]) and same(c, want[0])
        assert kda.device_status() == status  # (page 9 is outside the pool)
    t, ln = table.cuda(), lens.cuda()
    assert kda.pages_fork(cache.cuda(), t, ln, ints([]), ints([])).tolist() == [1]
    assert kda.device_status() == kda.KDA_ERR_SHAPE and torch.equal(t.cpu(), table)


@pytest.mark.parametrize("layers", [1, 3])
@pytest.mark.parametrize("n_slots,most,page,n_pages", SHAPES)
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(n_slots, most, page, n_pages, layers, in_place):
    rng = random.Random(n_slots + layers)
    table, lens = draw_sequences(rng, n_slots, most, page, n_pages)
    for b in range(0, n_slots, 2):
        lens[b] = 0
    cache = noise(layers, n_pages, 2, 1, page, 64, seed=n_slots)
    want, renamed, used = ref.compact(cache, table, lens, page)
    c, t = cache.cuda(), table.cuda()
    if layers == 1:
        c = c[0]  # one layer's cache is taken as it is
    out, n = kda.pages_compact(c, t, lens.cuda(), table_out=t if in_place else None)
    assert n.tolist() == [used] and torch.equal(out.cpu(), renamed) and same(c.view(want.shape), want)
    assert torch.equal(t.cpu(), renamed if in_place else table)


def test_compact_leaves_what_is_malformed():
    """Entries outside the pool stay as they are; a row with a bad length holds no pages."""
    table = torch.tensor([[9, 12], [-4, 6], [7, 8], [1, 1]], dtype=torch.int32)
    lens = torch.tensor([20, 32, -1, 33], dtype=torch.int32)
    cache = noise(1, 10, 2, 1, 16, 64)
    want, renamed, used = ref.compact(cache, table, lens, 16)
    c = cache.cuda()
    out, n = kda.pages_compact(c, table.cuda(), lens.cuda())
    assert kda.device_status() == kda.KDA_ERR_SHAPE
    assert n.tolist() == [used] == [2] and torch.equal(out.cpu(), renamed) and same(c, want)
    with pytest.raises(ValueError):
        kda.pages_grow(table.cuda(), lens.cuda(), lens.cuda(), 16, 1 << 32)


def test_compact_of_a_large_pool():
    """2^20 pages of 4 KB: every third is in use, and each keeps its contents."""
    n_pages = 1 << 20
    cache = torch.empty(n_pages, 2, 1, 16, 64, dtype=torch.bfloat16, device="cuda")
    mark = torch.arange(n_pages, device="cuda", dtype=torch.int32)
    cache.view(torch.int32).view(n_pages, -1)[:] = mark[:, None]
    table = torch.stack([mark[0::3][:349525].flip(0), mark[0::3][:349525]])
    lens = ints([16 * 349525, 16])
    out, used = kda.pages_compact(cache, table, lens)
    assert used.tolist() == [349525]
    assert out[0].sort()[0].equal(torch.arange(349525, dtype=torch.int32, device="cuda"))
    held = cache.view(torch.int32).view(n_pages, -1)[out[0].long()]
    assert torch.equal(held, table[0][:, None].expand_as(held))
    assert out[1, 0].item() == 0 and (out[1, 1:] == -1).all()


def test_pages_captured_and_replayed_on_another_stream():
    """grow, append, fork and compact in one graph: replayed on other contents, as called in turn."""
    page, H, D, n_slots, most, n_pages = 16, 2, 64, 6, 8, 64
    s = torch.cuda.Stream()
    table, lens, cache = ints([[0] * most] * n_slots), ints([0] * n_slots), noise(2, n_pages, 2, H, page, D).cuda()
    want, src, dst = ints([0] * n_slots), ints([0, 1]), ints([4, 5])
    k, v = torch.empty(12, H, D, dtype=torch.bfloat16, device="cuda"), torch.empty(12, H, D, dtype=torch.bfloat16, device="cuda")
    cu = ints([0, 3, 6, 9, 12])

    def step():
        left = kda.pages_grow(table, lens, want, page, n_pages)
        for layer in range(2):
            kda.kv_append(k, v, cache[layer], table, lens, slots=ints_of, cu_seqlens=cu)
        lens.copy_(want)
        forked = kda.pages_fork(cache, table, lens, src, dst)
        _, used = kda.pages_compact(cache, table, lens, table_out=table)
        return left, forked, used

    ints_of = ints([0, 1, 2, 3])
    begin = [(torch.randint(0, 100, (n_slots,), generator=torch.Generator().manual_seed(i)), noise(12, H, D, seed=i),
              noise(12, H, D, seed=9 + i)) for i in range(3)]

    def fill(i):
        ln = begin[i][0].int()
        ln[4:] = 0
        t = torch.full((n_slots, most), -1, dtype=torch.int32)
        order, at = torch.randperm(n_pages, generator=torch.Generator().manual_seed(50 + i)).int(), 0
        for b in range(n_slots):
            need = -(-int(ln[b]) // page)
            t[b, :need] = order[at:at + need]
            at += need
        table.copy_(t), lens.copy_(ln), k.copy_(begin[i][1]), v.copy_(begin[i][2])
        want.copy_(ln + torch.tensor([3, 3, 3, 3, 0, 0], dtype=torch.int32))
        cache.copy_(noise(2, n_pages, 2, H, page, D, seed=i))

    def state():
        return [x.clone() for x in (table, lens, cache.view(torch.int16))]

    eager = []
    for i in range(3):
        fill(i)
        counts = [int(c) for c in step()]
        eager.append((counts, state()))
    fill(0)
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        outs = step()
    for i in (1, 0, 2):
        fill(i)
        g.replay()
        assert [int(c) for c in outs] == eager[i][0]
        assert all(torch.equal(a, b) for a, b in zip(state(), eager[i][1]))


@pytest.mark.parametrize("lens", [[5, -2, 5], [0, 8, -8, 3], [2, 2, 2, 2, -1, 1] + [0] * 400, [1] * 3000 + [-3000] + [1] * 3000])
def test_append_records_offsets_that_decrease(lens):
    """Between runs that are well-formed by themselves: recorded, and what is written stands where one of
    its token's runs puts it."""
    page, H, D = 16, 1, 64
    cu, n = ref.offsets(lens), len(lens)
    total = max(cu)
    k, v = noise(total, H, D, seed=1), noise(total, H, D, seed=2)
    table = torch.arange(n, dtype=torch.int32).view(n, 1)
    cache = noise(n, 2, H, page, D, seed=3)
    c = cache.cuda()
    kda.kv_append(k.cuda(), v.cuda(), c, table.cuda(), ints([0] * n), cu_seqlens=ints(cu))
    assert kda.device_status() == kda.KDA_ERR_SHAPE
    got = c.cpu().view(torch.int16)
    for b in range(n):
        for j in range(max(lens[b], 0)):
            for i, x in enumerate((k, v)):
                row = got[b, i, 0, j]
                assert torch.equal(row, x[cu[b] + j, 0].view(torch.int16)) or torch.equal(row, cache[b, i, 0, j].view(torch.int16))
        assert torch.equal(got[b, :, :, max(lens[b], 0):], cache[b, :, :, max(lens[b], 0):].view(torch.int16))


@pytest.mark.parametrize("layers", [1, 2])
@pytest.mark.parametrize("n_slots,most,page,n_pages", SHAPES[1:])
@pytest.mark.parametrize("spare", [0, 3, 10000])
def test_fork_of_rows_that_share_pages(n_slots, most, page, n_pages, layers, spare):
    """Parents and rows that are given up share pages with rows that go on: what those reach is not handed out.
    With a pool of few unused pages each of them counts."""
    rng = random.Random(n_slots * layers + spare)
    table, lens = draw_sequences(rng, n_slots, most, page, n_pages)
    used = ref.in_use(table, lens, page, n_pages)
    if spare < n_pages - len(used):  # the others belong to no pool
        now = {p: i for i, p in enumerate(sorted(used))}
        for b in range(n_slots):
            for i in range(-(-int(lens[b]) // page)):
                table[b, i] = now[int(table[b, i])]
        n_pages = len(used) + spare
    cache = noise(layers, n_pages, 2, 1, page, 64, seed=n_slots)
    order = rng.sample(range(n_slots), n_slots)
    parents = order[:max(1, n_slots // 3)]
    dst = order[len(parents):][:max(1, n_slots // 2)]
    src = [rng.choice(parents) for _ in dst]
    want = ref.fork(cache, table, lens, src, dst, page)
    c, t, ln = cache.cuda(), table.cuda(), lens.cuda()
    left = kda.pages_fork(c, t, ln, ints(src), ints(dst))
    assert left.tolist() == [want[3]]
    assert torch.equal(t.cpu(), want[1]) and torch.equal(ln.cpu(), want[2]) and same(c, want[0])
    # again, from the same parents: each row's own last page is given up, what it shares stays
    want = ref.fork(want[0], want[1], want[2], src, dst, page)
    left = kda.pages_fork(c, t, ln, ints(src), ints(dst))
    assert left.tolist() == [want[3]]
    assert torch.equal(t.cpu(), want[1]) and torch.equal(ln.cpu(), want[2]) and same(c, want[0])


def test_pages_replayed_on_two_other_streams():
    """One graph, captured on one stream and replayed on others in turn, on contents that change between."""
    page, H, D, n_slots, most, n_pages = 16, 1, 64, 4, 6, 40
    table, lens = ints([[-1] * most] * n_slots), ints([0] * n_slots)
    cache = torch.zeros(1, n_pages, 2, H, page, D, dtype=torch.bfloat16, device="cuda")
    want, src, dst, cu = ints([0] * n_slots), ints([0]), ints([3]), ints([0, 9, 30, 47])
    k, v = (torch.zeros(47, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))

    def step():
        left = kda.pages_grow(table, lens, want, page, n_pages)
        kda.kv_append(k, v, cache[0], table, lens, cu_seqlens=cu)
        lens.copy_(want)
        forked = kda.pages_fork(cache, table, lens, src, dst)
        _, used = kda.pages_compact(cache, table, lens, table_out=table)
        return left, forked, used

    captured = torch.cuda.Stream()
    captured.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=captured):
        outs = step()
    others = [torch.cuda.Stream(), torch.cuda.Stream()]
    for turn in range(6):
        now = [7 * turn, 30 - 4 * turn, 16, 50]
        rows, t = noise(2, 47, H, D, seed=turn), torch.full((n_slots, most), -1, dtype=torch.int32)
        at = 1
        for b, n in enumerate(now):
            need = -(-n // page)
            t[b, :need] = torch.arange(at, at + 3 * need, 3) % n_pages
            at += 3 * need
        full = noise(1, n_pages, 2, H, page, D, seed=20 + turn)
        ln, wt = torch.tensor(now, dtype=torch.int32), torch.tensor([now[0] + 9, now[1] + 21, now[2] + 17, now[3]], dtype=torch.int32)
        e_table, e_left = ref.grow(t, ln, wt, page, n_pages)
        e_cache = ref.append(rows[0], rows[1], full[0], e_table, ln, [0, 1, 2], cu.tolist(), page)[None]
        e_cache, e_table, e_lens, e_forked = ref.fork(e_cache, e_table, wt, [0], [3], page)
        e_cache, e_table, e_used = ref.compact(e_cache, e_table, e_lens, page)
        stream = others[turn % 2]
        with torch.cuda.stream(stream):  # all of it on that stream, which the other one's turn is waited for
            stream.wait_stream(others[(turn + 1) % 2])
            stream.wait_stream(captured)
            for x, y in ((table, t), (lens, ln), (want, wt), (k, rows[0]), (v, rows[1]), (cache, full)):
                x.copy_(y)
            g.replay()
            counts = [int(c) for c in outs]
        assert counts == [e_left, e_forked, e_used]
        stream.synchronize()
        assert torch.equal(table.cpu(), e_table) and torch.equal(lens.cpu(), e_lens) and same(cache, e_cache)

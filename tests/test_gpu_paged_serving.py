"""The paged cache's operators together, as a serving loop uses them: prompts in chunks, forked
sequences, drafted runs that draft verification cuts, compaction in between, all lengths on the GPU;
eagerly and with the step captured into a graph."""
import pytest
import torch

import linear_attention_serving_chunk_gb300 as kda
import paged_ref as ref

pytestmark = pytest.mark.gpu

PAGE, H, Hq, D, LAYERS, VOCAB, SLOTS, PAGES, MOST, DRAFTS = 16, 2, 6, 64, 2, 40, 6, 90, 12, 3


class Model:
    """Queries, keys, values of a token are rows of tables, so what the cache has to hold is known exactly."""

    def __init__(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.q = rnd(LAYERS, VOCAB, Hq, D).bfloat16()
        self.kv = rnd(2, LAYERS, VOCAB, H, D).bfloat16()
        self.head = (rnd(LAYERS * Hq * D, VOCAB) / (LAYERS * Hq * D) ** 0.5 * 6).bfloat16()
        self.cache = torch.full((LAYERS, PAGES, 2, H, PAGE, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.table = torch.full((SLOTS, MOST), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(SLOTS, dtype=torch.int32, device="cuda")

    def forward(self, tokens, slots, cu):
        """Probabilities after each token of the runs; their keys and values are in the cache then."""
        want = self.lens.clone()
        want[slots.long()] += cu[1:] - cu[:-1]
        left = kda.pages_grow(self.table, self.lens, want, PAGE, PAGES)
        out = []
        for i in range(LAYERS):
            t = tokens.long()
            kda.kv_append(self.kv[0, i][t], self.kv[1, i][t], self.cache[i], self.table, self.lens, slots, cu)
            out.append(kda.attn_paged(self.q[i][t], self.cache[i], self.table, self.lens, slots, cu))
        self.out = torch.cat([o.flatten(1) for o in out], 1)
        return torch.softmax((self.out @ self.head).float(), 1), left

    def step(self, tokens, slots, cu, u):
        """One run of a token and its drafts for each sequence: (emitted tokens, how many), lens moved on."""
        p, left = self.forward(tokens, slots, cu)
        out, n_out = kda.verify_draft(p, tokens, u, cu)
        self.lens[slots.long()] += n_out
        return out, n_out, left

    def check_cache(self, texts):
        """The pages of every sequence hold the keys and values of its tokens."""
        for s, text in texts.items():
            assert int(self.lens[s]) == len(text)
            t = torch.tensor(text, device="cuda")
            for i in range(LAYERS):
                held = ref.gathered(self.cache[i].cpu(), self.table.cpu(), s, len(text))
                assert torch.equal(held, self.kv[:, i][:, t].transpose(1, 2).double().cpu())


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def serve(graph):
    g = torch.Generator().manual_seed(5)
    m = Model(1)
    # three prompts in two chunks, the second one's first chunk all of it
    texts = {s: torch.randint(0, VOCAB, (n,), generator=g).tolist() for s, n in ((4, 37), (0, 16), (3, 50))}
    done = {s: 0 for s in texts}
    for cut in (16, 100):
        runs = {s: t[done[s]:cut] for s, t in texts.items()}
        cu = ints(ref.offsets([len(r) for r in runs.values()]))
        slots = ints(list(runs))
        m.forward(ints(sum(runs.values(), [])), slots, cu)
        m.lens[slots.long()] += cu[1:] - cu[:-1]
        for s, r in runs.items():
            done[s] += len(r)
    m.check_cache(texts)
    # two of them go on twice; what they share stays shared
    left = kda.pages_fork(m.cache, m.table, m.lens, ints([4, 3]), ints([1, 5]))
    texts[1], texts[5] = list(texts[4]), list(texts[3])
    m.check_cache(texts)
    # unused: all but 3 + 1 + 4 pages of the prompts and two copies of last ones
    assert left.tolist() == [PAGES - 10] and kda.device_status() == 0
    live = list(texts)
    slots, cu = ints(live), ints(ref.offsets([1 + DRAFTS] * len(live)))
    tokens, u = ints([0] * (len(live) * (1 + DRAFTS))), torch.zeros(len(live) * (1 + DRAFTS), device="cuda")
    replay = None
    if graph:
        lens = m.lens.clone()
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        replay = torch.cuda.CUDAGraph()
        with torch.cuda.graph(replay, stream=stream):
            outs = m.step(tokens, slots, cu, u)
        m.lens.copy_(lens)
    last = {s: int(torch.randint(0, VOCAB, (1,), generator=g)) for s in live}
    seen = []
    for turn in range(7):
        # drafts: the text's own words, so that some are accepted
        batch = [[last[s]] + torch.randint(0, VOCAB, (DRAFTS,), generator=g).tolist() for s in live]
        tokens.copy_(ints(sum(batch, [])))
        u.copy_(torch.rand(len(u), generator=g) * 0.05)  # (low: certain drafts pass at the rate of their weight)
        if graph:
            replay.replay()
        else:
            before = m.lens.clone()
            outs = m.step(tokens, slots, cu, u)
            for i in range(LAYERS):  # the attention of this step, against the plain form
                o, size = ref.attention(m.q[i][tokens.long()].cpu(), m.cache[i].cpu(), m.table.cpu(), before.cpu(), live, cu.tolist())
                err = (m.out[:, i * Hq * D:(i + 1) * Hq * D].view(-1, Hq, D).double().cpu() - o).abs()
                assert float((err - 2.0 ** -8 * o.abs() - (2.0 ** -8 + 2.0 ** -14) * size).max()) <= 0
        emitted, count = outs[0].view(len(live), -1).tolist(), outs[1].tolist()
        seen.append((emitted, count, outs[2].tolist()))
        for s, row, e, n in zip(live, batch, emitted, count):
            texts[s] += row[:1] + e[:n - 1]
            last[s] = e[n - 1]
        m.check_cache(texts)
        if turn == 3:
            table, used = kda.pages_compact(m.cache, m.table, m.lens)
            m.table.copy_(table)
            assert int(m.table.max()) == int(used) - 1
            m.check_cache(texts)
    assert kda.device_status() == 0
    return texts, seen


def test_serving_loop_eager_and_captured():
    """The same tokens either way; at least one draft in the run is accepted, at least one refused."""
    texts, seen = serve(False)
    counts = sum((c for _, c, _ in seen), [])
    assert min(counts) == 1 and max(counts) > 1
    again, seen_again = serve(True)
    assert again == texts and seen_again == seen


def test_two_captured_calls_with_workspaces_of_their_own():
    """Attention captured twice, on two streams, replayed at once: each as it is alone."""
    outs, graphs, want = [], [], []
    for seed in (1, 2):
        g = torch.Generator(device="cuda").manual_seed(seed)
        q = torch.randn(3, 8, 128, generator=g, device="cuda").bfloat16()
        cache = torch.randn(200, 2, 1, 64, 128, generator=g, device="cuda").bfloat16()
        table, lens = torch.randperm(200, generator=g, device="cuda").int().view(2, 100), ints([6000, 3000])
        args = (q, cache, table, lens, None, ints([0, 1, 3]))
        want.append(kda.attn_paged(*args))
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            outs.append(kda.attn_paged(*args))
        graphs.append((graph, s, args))
    torch.cuda.synchronize()
    for _ in range(20):
        for graph, s, _ in graphs:
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])
    assert kda.device_status() == 0


def test_pages_behind_a_window_are_given_up():
    """Sequences that only ever see the last positions give back the pages in front of them: the pool never holds
    more, other sequences take the pages, and no call records anything."""
    window, page, pages, slots_n = 40, 16, 16, 4
    g = torch.Generator().manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=g).bfloat16()  # noqa: E731
    cache = torch.full((1, pages, 2, H, page, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    table, lens = torch.full((slots_n, 28), -1, dtype=torch.int32, device="cuda"), ints([0] * slots_n)
    slots, history = ints([2, 0]), [[], []]
    for turn in range(34):
        n = (11, 6) if turn else (70, 5)
        cu, total = ref.offsets(n), sum(n)
        want = lens.clone()
        want[slots.long()] += ints(n)
        assert int(kda.pages_grow(table, lens, want, page, pages)) >= 0
        q, k, v = rnd(total, Hq, D), rnd(total, H, D), rnd(total, H, D)
        kda.kv_append(k.cuda(), v.cuda(), cache[0], table, lens, slots, ints(cu))
        o = kda.attn_paged(q.cuda(), cache[0], table, lens, slots, ints(cu), window=window).double().cpu()
        for b in range(2):  # against all keys and values that there were, in 64 bits
            history[b].append((k[cu[b]:cu[b + 1]], v[cu[b]:cu[b + 1]]))
            ks, vs = (torch.cat([h[i] for h in history[b]]).double() for i in (0, 1))
            before = len(ks) - n[b]
            i = torch.arange(before, len(ks))[:, None]
            see = (torch.arange(len(ks)) <= i) & (torch.arange(len(ks)) > i - window)
            for h in range(Hq):
                x = q[cu[b]:cu[b + 1], h].double() @ ks[:, h // (Hq // H)].t() * D ** -0.5
                w = torch.softmax(x.masked_fill(~see, float("-inf")), 1)
                exact, size = w @ vs[:, h // (Hq // H)], w @ vs[:, h // (Hq // H)].abs()
                err = (o[cu[b]:cu[b + 1], h] - exact).abs()
                assert float((err - 2.0 ** -8 * exact.abs() - (2.0 ** -8 + 2.0 ** -14) * size).max()) <= 0
        lens.copy_(want)
        gone = ((lens - window + 1).clamp(min=0) // page)[:, None]
        table.masked_fill_(torch.arange(table.shape[1], device="cuda") < gone, -1)
        if turn % 5 == 4:
            renamed, used = kda.pages_compact(cache, table, lens)
            assert int(used) <= 8 and torch.equal(renamed < 0, (table < 0) | (torch.arange(28, device="cuda") * page >= lens[:, None]))
            table.copy_(renamed)
        if turn == 20:  # a fork copies what is given up as it is, and may go on
            kda.pages_fork(cache, table, lens, ints([2]), ints([1]))
            last = (int(lens[2]) - 1) // page
            assert torch.equal(table[1, :last], table[2, :last]) and int(table[1, 0]) == -1 and int(lens[1]) == int(lens[2])
            lens[1] = 0
    assert int(lens[2]) > pages * page and kda.device_status() == 0
    # what a call needs is not there: a last page to copy, and an entry that is neither a page nor given up
    row = (int(lens[2]) - 1) // page
    assert int(lens[2]) % page
    for at, entry in ((row, -1), (0, -2), (1, pages)):
        t = table.clone()
        t[2, at] = entry
        kda.pages_fork(cache.clone(), t, lens.clone(), ints([2]), ints([1]))
        assert kda.device_status() == kda.KDA_ERR_SHAPE


@pytest.mark.parametrize("m", [16, 17, 40, 48, 5])
def test_a_sequence_goes_on_from_inside_a_shared_page(m):
    """By a fork from a slot that holds the first m tokens: another sequence, and the sequence itself, go on from
    there, and what the others hold stays."""
    page, pages, most = 16, 24, 6
    g = torch.Generator().manual_seed(m)
    cache = torch.randn(LAYERS, pages, 2, H, page, D, generator=g).bfloat16().cuda()
    table, lens = torch.full((5, most), -1, dtype=torch.int32, device="cuda"), ints([0] * 5)
    kda.pages_grow(table, lens, ints([55, 0, 0, 0, 0]), page, pages)
    lens[0] = 55
    kda.pages_fork(cache, table, lens, ints([0]), ints([1]))  # three full pages are shared

    def held(s):
        return [ref.gathered(cache[i].cpu(), table.cpu(), s, int(lens[s])) for i in range(LAYERS)]

    def same(a, b, n=None):
        return all(torch.equal(x[:, :, :n], y[:, :, :n]) for x, y in zip(a, b))

    def on(s, n):  # n more tokens of sequence s
        want = lens.clone()
        want[s] += n
        assert int(kda.pages_grow(table, lens, want, page, pages)) >= 0
        for i in range(LAYERS):
            k, v = torch.randn(2, n, H, D, generator=g).bfloat16().cuda()
            kda.kv_append(k, v, cache[i], table, lens, ints([s]), ints([0, n]))
        lens.copy_(want)

    first = held(0)
    for d in (2, 0):  # 4 is the free slot
        table[4], lens[4] = table[0], m
        assert int(kda.pages_fork(cache, table, lens, ints([4]), ints([d]))) >= 0
        lens[4] = 0
        assert int(lens[d]) == m and same(held(d), first, m)
        others = {s: held(s) for s in (0, 1, 2) if s != d}
        on(d, 20)
        assert same(held(d), first, m) and all(same(held(s), h) for s, h in others.items())
    assert same(held(1), first) and kda.device_status() == 0

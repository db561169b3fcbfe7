"""Attention over a paged cache on the GPU, against the plain form in 64 bits (tests/paged_ref.py)."""
import random

import pytest
import torch

import linear_attention_serving_chunk_gb300 as kda
import paged_ref as ref

pytestmark = pytest.mark.gpu

# Off by at most: the result's rounding to bf16 (2^-8 of it), the weights' (2^-8 of the sum of the
# values' magnitudes), and what fp32 leaves of scores and exponentials (scores up to 2^6 in base 2 with sums
# of 128 terms: 2^-24 x 2^6 x 2^4 relative in each weight).
HALF_STEP = 2.0 ** -8
WEIGHTS = 2.0 ** -8 + 2.0 ** -14


@pytest.fixture(autouse=True)
def clean_status():
    kda.device_status()
    yield
    assert kda.device_status() == 0  # (a test that expects a code has read it)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Batch:
    """Runs of `new` tokens behind `cached` ones, at random slots and pages; what the sequences do
    not reach is NaN."""

    def __init__(self, cached, new, Hq, H, D, page, seed=0, wide=0, loud=1.0):
        g = torch.Generator().manual_seed(seed)
        self.new, self.cu, total = new, ref.offsets(new), sum(new)
        self.reach = [a + b for a, b in zip(cached, new)]
        n_slots = len(new) + 2
        self.table, self.slots, n_pages = ref.sequences(self.reach, n_slots, page, seed)
        self.lens = torch.zeros(n_slots, dtype=torch.int32)
        self.lens[self.slots.long()] = torch.tensor(cached, dtype=torch.int32)
        self.cache = torch.full((n_pages, 2, H, page, D), float("nan"), dtype=torch.bfloat16)
        for s, reach in zip(self.slots.tolist(), self.reach):
            for i in range(-(-reach // page)):
                n = min(page, reach - i * page)
                self.cache[self.table[s, i], :, :, :n] = torch.randn(2, H, n, D, generator=g).bfloat16()
        rows = torch.randn(total, Hq * D + wide, generator=g) * loud
        self.rows, self.wide, self.shape = rows.bfloat16(), wide, (total, Hq, D)
        self.q = self.rows[:, wide:].view(self.shape)

    def want(self, window=0, scale=None, lens=None):
        return ref.attention(self.q, self.cache, self.table, self.lens, self.slots.tolist(), self.cu, window, scale)

    def call(self, cu=True, **kw):
        q = self.rows.cuda()[:, self.wide:].view(self.shape)
        return kda.attn_paged(q, self.cache.cuda(), self.table.cuda(), self.lens.cuda(), slots=self.slots.cuda(),
                              cu_seqlens=ints(self.cu) if cu else None, **kw)


def near(o, want):
    o, (exact, size) = o.double().cpu(), want
    err = (o - exact).abs()
    assert not torch.isnan(err).any()
    assert float((err - HALF_STEP * exact.abs() - WEIGHTS * size).max()) <= 0
    # no more than twice what independent roundings of both kinds leave
    spread = (HALF_STEP ** 2 / 3) ** 0.5 * 2
    assert float(err.norm()) <= 2 * spread * float(size.norm())


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,H", [(1, 1), (8, 2), (6, 2), (5, 1)])
@pytest.mark.parametrize("reach", [[0, 127, 128], [1, 255, 256, 700, 15, 16, 17]])
def test_single_tokens(page, D, Hq, H, reach):
    b = Batch(reach, [1] * len(reach), Hq, H, D, page, seed=page)
    near(b.call(cu=False), b.want())


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,H", [(2, 2), (8, 2), (3, 1), (16, 1)])
@pytest.mark.parametrize("window", [0, 1, 100, 128, 300])
def test_runs(page, D, Hq, H, window):
    """Prompt chunks, single tokens, drafted runs and empty ones, one run of a token too many for a tile."""
    b = Batch([0, 500, 130, 3, 640, 1, 0], [300, 1, 5, 0, 129, 43, 1], Hq, H, D, page, seed=window, wide=8)
    near(b.call(window=window), b.want(window))


@pytest.mark.parametrize("G", [1, 2, 7, 64, 100, 128, 129, 300])
def test_groups(G):
    """Groups that do not divide a tile, and those larger than one or two."""
    b = Batch([60, 0, 200], [9, 1, 3], G, 1, 64, 32, seed=G)
    near(b.call(), b.want())


@pytest.mark.parametrize("cached,new", [([20000], [1]), ([3000, 20], [2, 1]), ([0], [1500]), ([4000], [700]),
                                        ([100] * 300, [1] * 300), ([0] * 5 + [9000], [1, 0, 0, 2, 1, 3])])
@pytest.mark.parametrize("D", [64, 128])
def test_shared_out(cached, new, D):
    """Long sequences cut between many CTAs, and many short ones; without a workspace nothing is cut."""
    b = Batch(cached, new, 4, 1, D, 64, seed=len(new))
    want = b.want()
    near(b.call(), want)
    near(b.call(workspace=torch.empty(16, dtype=torch.uint8, device="cuda")), want)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,new", [(16, 1), (5, 7), (16, 6), (16, 11), (3, 60)])
def test_many_parts(G, new, D):
    """One head of keys over 110,000 positions: 152 shares for the rows of one item (16 to 180 of them)."""
    b = Batch([110000 - new], [new], G, 1, D, 128, seed=G)
    near(b.call(), b.want())


@pytest.mark.parametrize("H", [1, 3, 8])
def test_more_runs_than_threads(H):
    new = [(7 * i) % 4 for i in range(1000)]
    b = Batch([(13 * i) % 150 for i in range(1000)], new, 2 * H, H, 64, 16, seed=H)
    near(b.call(), b.want())


@pytest.mark.parametrize("scale", [1e-4, 0.125, 3.0])
@pytest.mark.parametrize("loud", [1e-3, 1.0, 20.0])
def test_scales(scale, loud):
    """Flat and peaked rows: weights that are all alike, and sums that one key decides."""
    b = Batch([900, 10], [3, 200], 4, 2, 128, 64, seed=3, loud=loud)
    o, size = b.want(scale=scale)
    got = b.call(scale=scale).double().cpu()
    # scores of `top` in base 2 carry 2^-24 of it and of their terms' sum
    top = float(b.q.double().abs().max()) * 128 * 4 * scale * 1.4427
    assert float(((got - o).abs() - HALF_STEP * o.abs() - (WEIGHTS + top * 2.0 ** -22) * size).max()) <= 0


def test_maxima_that_rise_and_fall():
    """Keys that grow along the sequence and shrink again: every tile brings a new maximum, or none."""
    b = Batch([2000, 2000], [1, 140], 4, 1, 64, 64, seed=1)
    for s, f in zip(b.slots.tolist(), (lambda i: 1 + i / 200, lambda i: 12 - i / 180)):
        for i in range(-(-2140 // 64)):
            p = int(b.table[s, i])
            if p >= 0:
                b.cache[p, 0] *= f(64 * i)
    b.q[:] = b.q.abs()  # (with keys of both signs the maximum is what grows)
    o, size = b.want()
    got = b.call().double().cpu()
    top = float(b.q.double().abs().max()) * 64 * 4 * 12 * 0.125 * 1.4427
    assert float(((got - o).abs() - HALF_STEP * o.abs() - (WEIGHTS + top * 2.0 ** -22) * size).max()) <= 0


def test_other_sequences_and_masked_keys_do_not_matter():
    """Inf and NaN in another sequence, in a run's later keys, behind the end and in front of the window."""
    b = Batch([100, 300], [5, 6], 4, 2, 64, 16, seed=5)
    want = b.call()[:5].clone()
    b.cache[b.table[b.slots[1].long(), :19].long()] = float("inf")
    assert torch.equal(b.call()[:5], want)
    # keys (not values) of the run's last token: the rows before it do not see them
    b = Batch([100], [5], 4, 2, 64, 16, seed=5)
    want = b.call()
    p = int(b.table[b.slots[0].long(), 104 // 16])
    b.cache[p, 0, :, 104 % 16] = float("nan")
    assert torch.equal(b.call()[:4], want[:4]) and torch.isnan(b.call()[4]).all()
    # pages in front of the window are given up: their entries may be anything
    b = Batch([300], [3], 4, 2, 64, 16, seed=6)
    near(b.call(window=70), b.want(70))
    want = b.call(window=70)
    b.table[b.slots[0].long(), :(300 - 69) // 16] = -5
    assert torch.equal(b.call(window=70), want)


def test_bad_entries():
    """A page outside the pool counts as zeros, a run without a valid slot or length or too long
    for its row is left out; all are recorded, and the other runs are as they were."""
    b = Batch([200, 40, 7, 90], [2, 3, 4, 1], 4, 2, 64, 16, seed=7)
    good = b.call()
    s = b.slots.long()
    b.table[s[0], 3], b.table[s[0], 12] = -1, b.cache.shape[0]
    o = b.call()
    assert kda.device_status() == kda.KDA_ERR_SHAPE
    near(o, b.want())
    assert torch.equal(o[2:], good[2:])
    for what in ("slot", "length", "long"):
        b = Batch([200, 40, 7, 90], [2, 3, 4, 1], 4, 2, 64, 16, seed=7)
        if what == "slot":
            b.slots[1] = 6
        else:
            b.lens[s[1]] = -3 if what == "length" else 16 * b.table.shape[1] - 2
        o = b.call()
        assert kda.device_status() == kda.KDA_ERR_SHAPE
        assert torch.equal(o[:2], good[:2]) and torch.equal(o[5:], good[5:])
    b = Batch([200, 40, 7, 90], [2, 3, 4, 1], 4, 2, 64, 16, seed=7)
    b.cu = [0, 2, 12, 9, 10]
    o = b.call()
    assert kda.device_status() == kda.KDA_ERR_SHAPE
    assert torch.equal(o[:2], good[:2]) and torch.equal(o[9:], good[9:])


@pytest.mark.parametrize("seed", range(24))
def test_drawn_batches(seed):
    """Random heads, pages, windows, contexts and runs, with and without a workspace."""
    rng = random.Random(seed)
    H, D, page = rng.choice([1, 2, 3, 5]), rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    n, G = rng.randint(1, 12), rng.choice([1, 2, 3, 4, 6, 8, 13, 33])
    new = [rng.choice([0, 1, 1, rng.randint(2, 8), rng.randint(1, 400)]) for _ in range(n)]
    cached = [rng.choice([0, rng.randint(1, 130), rng.randint(1, 3000)]) for _ in range(n)]
    if rng.random() < 0.3:
        new = [rng.randint(1, 3)] * n
    window = rng.choice([0, 0, 1, rng.randint(2, 300), rng.randint(100, 4000)])
    b = Batch(cached, new, G * H, H, D, page, seed=seed, wide=rng.choice([0, 8, 24]))
    kw = dict(workspace=torch.empty(0, dtype=torch.uint8, device="cuda")) if rng.random() < 0.3 else {}
    near(b.call(window=window, **kw), b.want(window))


def test_rows_outside_all_runs_and_in_place():
    b = Batch([50, 20], [3, 2], 4, 2, 64, 16, seed=8)
    want = b.call()
    q = torch.cat([b.q, torch.ones(4, 4, 64, dtype=torch.bfloat16)]).cuda()
    o = torch.full_like(q, 3.0)
    args = (b.cache.cuda(), b.table.cuda(), b.lens.cuda())
    kda.attn_paged(q, *args, slots=b.slots.cuda(), cu_seqlens=ints(b.cu), o=o)
    assert torch.equal(o[:5], want) and (o[5:] == 3).all()
    assert kda.attn_paged(q, *args, slots=b.slots.cuda(), cu_seqlens=ints(b.cu), o=q) is q
    assert torch.equal(q[:5], want) and (q[5:] == 1).all()
    # o as a slice of wider rows
    wide = torch.zeros(5, 4 * 64 + 24, dtype=torch.bfloat16, device="cuda")
    kda.attn_paged(b.q.cuda(), *args, slots=b.slots.cuda(), cu_seqlens=ints(b.cu), o=wide[:, 16:272].view(5, 4, 64))
    assert torch.equal(wide[:, 16:272].view(5, 4, 64), want) and (wide[:, :16] == 0).all() and (wide[:, 272:] == 0).all()


def test_the_same_bits_again_and_on_another_stream():
    b = Batch([5000, 100, 0], [4, 1, 600], 8, 2, 128, 64, seed=9)
    want = b.call()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        assert torch.equal(b.call(), want)
        s.wait_stream(torch.cuda.current_stream())
        o = b.call(stream=s)
        s.synchronize()
        assert torch.equal(o, want)


def test_cache_beyond_32_bits():
    """Pages whose offsets pass 2^32 elements."""
    H, page, D = 8, 128, 128
    n_pages = (1 << 32) // (2 * H * page * D) + 40
    cache = torch.empty(n_pages, 2, H, page, D, dtype=torch.bfloat16, device="cuda")
    small = Batch([500], [3], 16, H, D, page, seed=10)
    table = torch.full_like(small.table, -1)
    for i in range(4):
        p = int(small.table[small.slots[0].long(), i])
        table[small.slots[0].long(), i] = n_pages - 1 - 9 * i
        cache[n_pages - 1 - 9 * i] = small.cache[p].cuda()
    o = kda.attn_paged(small.q.cuda(), cache, table.cuda(), small.lens.cuda(), slots=small.slots.cuda(), cu_seqlens=ints(small.cu))
    assert torch.equal(o, small.call())


@pytest.mark.parametrize("D", [64, 128])
def test_what_a_wait_that_gave_up_leaves(D):
    """The hook makes one CTA give up before it begins: the rows that need its share keep what they held, whether
    it is a part of an item or has items of its own, the others are right, and so is the next call."""
    def stalled(b, **kw):
        o = torch.full(b.q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        b.call(window=kda.ATTN_TEST_STALL, o=o, **kw)
        assert kda.device_status() == kda.KDA_ERR_TIMEOUT
        return o

    # one item in 152 parts, with a workspace that holds parts of an earlier call and with a new one
    b = Batch([100000], [1], 4, 1, D, 64, seed=1)
    workspace = torch.empty(kda.attn_workspace_bytes(1, 1, 4, 1, D), dtype=torch.uint8, device="cuda")
    want = b.call(workspace=workspace)
    assert (stalled(b, workspace=workspace) == 7).all() and (stalled(b) == 7).all()
    assert torch.equal(b.call(workspace=workspace), want)
    # 400 sequences of a token behind 100: some of them are in the second share, and none in two at once
    b = Batch([100] * 400, [1] * 400, 4, 1, D, 64, seed=2)
    want = b.call()
    for kw in ({}, dict(workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))):
        o = stalled(b, **kw)
        kept = (o == 7).flatten(1).all(1)
        assert 1 <= int(kept.sum()) <= 8 and torch.equal(o[~kept], want[~kept])
        near(b.call(**kw), b.want())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cached,new", [([40, 3], [1, 9]), ([5000], [1]), ([300], [150])])
def test_scores_at_the_end_of_the_range(D, cached, new):
    """Scores of up to 2^30 decide for one key; a scale that takes them out of fp32 gives NaN, not zeros."""
    b = Batch(cached, new, 2, 1, D, 64, seed=4)
    # one key stands out in every row: the others' scores are closer than fp32 tells apart
    for s, reach in zip(b.slots.tolist(), b.reach):
        held = b.cache[b.table[s, 0].long()]
        b.cache[b.table[s, :-(-reach // 64)].long(), 0] = 0.25
        held[0, :, 0] = 0.5
    b.q[:] = 0.5  # scores 0.25 D or 0.125 D times the scale
    near(b.call(scale=2.0 ** 30 / (0.25 * D * 1.4427) * 0.99), b.want(scale=2.0 ** 30 / (0.25 * D * 1.4427) * 0.99))
    for scale in (1e38, 3e37):
        assert torch.isnan(b.call(scale=scale)).all()

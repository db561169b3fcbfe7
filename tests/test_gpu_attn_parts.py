"""Attention whose work is cut: joins of many parts, with values that tell where each weight went, and
runs of many items.  What the tolerances can see is shown on the CPU."""
import pytest
import torch

import linear_attention_serving_chunk_gb300 as kda
import paged_ref as ref
from test_gpu_attn import Batch, near

REACH, TILE, PARTS = 110000, 128, 152


@pytest.fixture
def clean_status():
    kda.device_status()
    yield
    assert kda.device_status() == 0


def marked(G, new, D, H=1):
    """A run behind a long sequence.  Column d of the values is 1 in the d-th of D pieces of the sequence and 0
    elsewhere: o is how the weight of a row lies along the sequence, and as large as the sum of magnitudes."""
    b = Batch([REACH - new], [new], G * H, H, D, 128, seed=G * D + new)
    row = b.table[b.slots[0].long()].tolist()
    for i in range(-(-REACH // 128)):
        at = torch.arange(128) + 128 * i
        b.cache[row[i], 1] = (at[:, None] * D // REACH == torch.arange(D)).bfloat16()
    return b


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,new,H", [(1, 1, 1), (16, 1, 1), (5, 7, 1), (16, 6, 1), (16, 11, 1), (3, 60, 1), (20, 12, 1), (16, 1, 2), (10, 13, 3)])
def test_every_part_counts_once(G, new, D, H, clean_status):
    b = marked(G, new, D, H)
    near(b.call(), b.want())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,new", [(16, 1), (16, 11)])
def test_what_the_tolerance_sees(G, new, D):
    """A part that is left out, counted twice, or weighted by a maximum that is not its own is found, wherever it is."""
    b = marked(G, new, D)
    kv = ref.gathered(b.cache, b.table, int(b.slots[0]), REACH)
    k, v = kv[0, 0], kv[1, 0]
    want = b.want()
    q = b.q.double().view(-1, D)
    x = torch.exp(q @ k.t() * D ** -0.5)
    see = torch.arange(REACH) <= (torch.arange(REACH - new, REACH).repeat_interleave(G))[:, None]
    x = torch.where(see, x, 0.0)

    def o(x):
        return ((x @ v) / x.sum(1, keepdim=True)).view(want[0].shape)

    near(o(x).bfloat16(), want)
    tiles = -(-REACH // TILE)
    for part in (0, 1, PARTS // 2, PARTS - 2, PARTS - 1):
        keys = slice(part * tiles // PARTS * TILE, (part + 1) * tiles // PARTS * TILE)
        for factor in (0.0, 2.0, 1.35):
            y = x.clone()
            y[:, keys] *= factor
            with pytest.raises(AssertionError):
                near(o(y).bfloat16(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [4, 7])
@pytest.mark.parametrize("window", [0, 1000])
def test_runs_of_many_items(G, window, D, clean_status):
    """More than 32 items of 256 rows in a run, over keys that grow along it: the share of a CTA begins at any of them."""
    b = Batch([30, 700, 5], [3, 2500, 1], G, 1, D, 64, seed=G + window)
    assert 2500 * G > 32 * 256
    near(b.call(window=window), b.want(window))


@pytest.mark.gpu
def test_a_run_of_a_thousand_items(clean_status):
    """Two rounds of the search among items: 32 ways, and 32 ways again."""
    b = Batch([100], [1300], 200, 1, 64, 128, seed=1)
    assert 1300 * 200 > 32 * 31 * 256
    near(b.call(window=90), b.want(90))

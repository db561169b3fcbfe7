"""What the paged cache's operators refuse before anything is launched (no GPU needed), the plain
forms that their GPU tests compare with, and how attention shares its work out."""
import ctypes
import os
import subprocess

import pytest
import torch

import linear_attention_serving_chunk_gb300 as kda
import paged_ref as ref

NULL, SHAPE, ALIGN, UNSUPPORTED, WORKSPACE = 1, 2, 3, 4, 5
at = ctypes.c_void_p  # never dereferenced: every call below is rejected first
GB = 1 << 30


@pytest.fixture(scope="module")
def L():
    kda.build()
    return kda.lib()


def call(fn, base, kw):
    a = dict(base)
    assert set(kw) <= set(a)
    a.update(kw)
    return fn(*a.values())


APPEND = dict(k=at(GB), ldk=128, v=at(2 * GB), ldv=128, cu=at(0x1000), n=2, total=8, H=2, D=64, cache=at(4 * GB),
              n_pages=10, page=16, table=at(0x2000), most=4, lens=at(0x3000), n_slots=3, slots=at(0x4000), stream=None)
RUNS_WRONG = [
    (dict(n=-1), SHAPE), (dict(total=-1), SHAPE), (dict(total=1 << 31), SHAPE), (dict(n=0), SHAPE),
    (dict(cu=None, n=3), SHAPE), (dict(cu=at(0x1002)), ALIGN), (dict(H=0), SHAPE), (dict(H=65536), SHAPE),
    (dict(D=96), UNSUPPORTED), (dict(page=8), UNSUPPORTED), (dict(page=256), UNSUPPORTED), (dict(page=48), UNSUPPORTED),
    (dict(n_pages=-1), SHAPE), (dict(n_pages=(1 << 20) + 1), UNSUPPORTED), (dict(most=-1), SHAPE),
    (dict(most=(1 << 20) + 1), UNSUPPORTED), (dict(n_slots=-1), SHAPE), (dict(slots=None, n_slots=1), SHAPE),
    (dict(cache=None), NULL), (dict(table=None), NULL), (dict(lens=None), NULL), (dict(cache=at(4 * GB + 8)), ALIGN),
    (dict(table=at(0x2001)), ALIGN), (dict(lens=at(0x3002)), ALIGN), (dict(slots=at(0x4002)), ALIGN),
    (dict(n=0, total=0), 0), (dict(total=0), 0)]


@pytest.mark.parametrize("kw,status", RUNS_WRONG + [
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(k=at(GB + 8)), ALIGN), (dict(v=at(GB + 2)), ALIGN),
    (dict(ldk=120), SHAPE), (dict(ldv=127), SHAPE), (dict(ldk=132), ALIGN), (dict(ldv=130), ALIGN),
    # rows in the cache, at its first and last places, and into it
    (dict(k=at(4 * GB)), SHAPE), (dict(v=at(4 * GB + 10 * 2 * 2 * 16 * 64 * 2 - 16)), SHAPE),
    (dict(k=at(4 * GB - 2048 + 16)), SHAPE)])
def test_append_refuses(L, kw, status):
    assert call(L.kda_kv_append, APPEND, kw) == status


ATTN = dict(q=at(GB), ldq=256, cu=at(0x1000), n=2, total=8, Hq=4, H=2, D=64, cache=at(4 * GB), n_pages=10, page=16,
            table=at(0x2000), most=4, lens=at(0x3000), n_slots=3, slots=at(0x4000), scale=0.125, window=0,
            o=at(3 * GB), ldo=256, ws=None, size=0, stream=None)


@pytest.mark.parametrize("kw,status", RUNS_WRONG + [
    (dict(q=None), NULL), (dict(o=None), NULL), (dict(q=at(GB + 8)), ALIGN), (dict(o=at(3 * GB + 4)), ALIGN),
    (dict(ldq=248), SHAPE), (dict(ldo=255), SHAPE), (dict(ldq=260), ALIGN), (dict(ldo=258), ALIGN),
    (dict(Hq=3), SHAPE), (dict(Hq=0), SHAPE), (dict(Hq=65536), SHAPE), (dict(window=-1), SHAPE), (dict(n_pages=0), SHAPE),
    (dict(scale=0.0), UNSUPPORTED), (dict(scale=-1.0), UNSUPPORTED), (dict(scale=float("nan")), UNSUPPORTED),
    (dict(scale=float("inf")), UNSUPPORTED), (dict(scale=3e38), UNSUPPORTED), (dict(ws=at(0x10008)), ALIGN),
    # o beside q but not over it, and in the cache
    (dict(o=at(GB + 16)), SHAPE), (dict(o=at(GB), ldo=264), SHAPE), (dict(o=at(4 * GB + 32)), SHAPE)])
def test_attention_refuses(L, kw, status):
    assert call(L.kda_attn_paged, ATTN, kw) == status


GROW = dict(table=at(0x100000), most=4, lens=at(0x3000), want=at(0x4000), n_slots=3, n_pages=10, page=16,
            left=at(0x5000), stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(most=-1), SHAPE), (dict(n_slots=-1), SHAPE), (dict(n_pages=-1), SHAPE), (dict(page=0), UNSUPPORTED),
    (dict(n_slots=(1 << 13) + 1), UNSUPPORTED), (dict(n_pages=(1 << 20) + 1), UNSUPPORTED), (dict(table=None), NULL),
    (dict(lens=None), NULL), (dict(want=None), NULL), (dict(left=None), NULL), (dict(want=at(0x4002)), ALIGN),
    (dict(left=at(0x5001)), ALIGN), (dict(table=at(0x3008)), SHAPE), (dict(table=at(0x4000)), SHAPE),
    (dict(left=at(0x100010)), SHAPE), (dict(left=at(0x3008)), SHAPE), (dict(left=at(0x4000)), SHAPE)])
def test_grow_refuses(L, kw, status):
    assert call(L.kda_pages_grow, GROW, kw) == status


FORK = dict(cache=at(4 * GB), layers=2, n_pages=10, H=2, page=16, D=64, table=at(0x100000), most=4, lens=at(0x3000),
            n_slots=3, src=at(0x4000), dst=at(0x5000), n=2, left=at(0x6000), ws=at(0x8000), size=4096, stream=None)
LAYERS_WRONG = [
    (dict(layers=0), SHAPE), (dict(H=0), SHAPE), (dict(D=32), UNSUPPORTED), (dict(page=24), UNSUPPORTED),
    (dict(layers=1 << 24, n_pages=1 << 20, H=64), UNSUPPORTED), (dict(cache=None), NULL), (dict(cache=at(8)), ALIGN),
    (dict(table=None), NULL), (dict(lens=None), NULL), (dict(ws=None), WORKSPACE), (dict(ws=at(0x8008)), ALIGN)]


@pytest.mark.parametrize("kw,status", LAYERS_WRONG + [
    (dict(n=-1), SHAPE), (dict(n=(1 << 20) + 1), UNSUPPORTED), (dict(n_slots=(1 << 13) + 1), UNSUPPORTED),
    (dict(src=None), NULL), (dict(dst=None), NULL), (dict(left=None), NULL), (dict(src=at(0x4001)), ALIGN),
    (dict(size=4 * (4 + 4 * 2) - 1), WORKSPACE), (dict(src=at(0x3008)), SHAPE), (dict(dst=at(0x100004)), SHAPE),
    (dict(left=at(0x5004)), SHAPE), (dict(ws=at(0x3000)), SHAPE), (dict(lens=at(0x100008)), SHAPE)])
def test_fork_refuses(L, kw, status):
    assert call(L.kda_pages_fork, FORK, kw) == status


COMPACT = dict(cache=at(4 * GB), layers=2, n_pages=10, H=2, page=16, D=64, table=at(0x100000), most=4,
               lens=at(0x3000), n_slots=3, out=at(0x200000), used=at(0x6000), ws=at(0x8000), size=4096, stream=None)


@pytest.mark.parametrize("kw,status", LAYERS_WRONG + [
    (dict(out=None), NULL), (dict(used=None), NULL), (dict(out=at(0x200002)), ALIGN), (dict(used=at(0x6003)), ALIGN),
    (dict(n_slots=(1 << 13) + 1), UNSUPPORTED), (dict(size=4 * (4 + 4 * 10) - 1), WORKSPACE),
    (dict(out=at(0x100004)), SHAPE), (dict(out=at(0x3000)), SHAPE), (dict(used=at(0x100000)), SHAPE),
    (dict(used=at(0x200010)), SHAPE), (dict(ws=at(0x100000)), SHAPE), (dict(ws=at(0x200000)), SHAPE)])
def test_compact_refuses(L, kw, status):
    assert call(L.kda_pages_compact, COMPACT, kw) == status


def test_workspace_sizes(L):
    assert kda.lib().kda_pages_workspace_bytes(-1) == 0
    assert kda.lib().kda_pages_workspace_bytes(10) == 4 * (4 + 4 * 10)
    assert kda.attn_workspace_bytes(1, 1, 4, 2, 128) > kda.attn_workspace_bytes(1, 1, 4, 2, 64) > 0
    for wrong in ((0, 0, 4, 2, 64), (1, 1, 3, 2, 64), (1, 1, 4, 2, 96), (1, 0, 4, 2, 64)):
        assert kda.attn_workspace_bytes(*wrong) == 0


def test_binding_refuses_wrong_tensors():
    q, i = torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    cache, table = torch.zeros(3, 2, 2, 16, 64, dtype=torch.bfloat16), torch.zeros(2, 4, dtype=torch.int32)
    for fn in (lambda: kda.attn_paged(q, cache, table, i), lambda: kda.kv_append(q[:, :2], q[:, :2], cache, table, i),
               lambda: kda.pages_grow(table, i, i, 16, 3), lambda: kda.pages_fork(cache, table, i, i, i),
               lambda: kda.pages_compact(cache, table, i)):
        with pytest.raises(ValueError):  # not on a GPU
            fn()
    for fn in (lambda: kda.attn_paged(None, cache, table, i), lambda: kda.pages_grow(None, i, i, 16, 3),
               lambda: kda.pages_compact([cache], table, i)):
        with pytest.raises(TypeError):
            fn()


def test_plain_attention_of_one_token_and_of_equal_keys():
    """One token alone gives its value; equal keys give the mean of the values that are seen."""
    cache = torch.randn(4, 2, 1, 16, 64).bfloat16()
    table, lens = torch.tensor([[2, 0], [1, 3]], dtype=torch.int32), torch.tensor([0, 20])
    q = torch.randn(3, 2, 64).bfloat16()
    o, _ = ref.attention(q, cache, table, lens, [0, 1], [0, 1, 3])
    assert torch.allclose(o[0], cache[2, 1, 0, 0].double().expand(2, 64))
    cache[:, 0] = 1.0
    v = torch.cat([cache[1, 1, 0], cache[3, 1, 0]]).double()
    o, _ = ref.attention(q, cache, table, lens, [0, 1], [0, 1, 3])
    assert torch.allclose(o[1], v[:21].mean(0).expand(2, 64)) and torch.allclose(o[2], v[:22].mean(0).expand(2, 64))
    o, _ = ref.attention(q, cache, table, lens, [0, 1], [0, 1, 3], window=5)
    assert torch.allclose(o[2], v[17:22].mean(0).expand(2, 64))


def test_plain_pages_of_a_worked_example():
    """Two sequences that share a page, one that ended: pages 1, 2 and 5 are in use."""
    table, lens = torch.tensor([[5, 2, 9], [5, 1, 0], [3, 4, 6]], dtype=torch.int32), torch.tensor([20, 17, 0])
    assert ref.in_use(table, lens, 16, 8) == {1, 2, 5}
    grown, left = ref.grow(table, lens, torch.tensor([33, 17, 16]), 16, 8)
    assert grown.tolist() == [[5, 2, 0], [5, 1, 0], [3, 4, 6]] and left == 3
    cache = torch.arange(8.0)[None, :, None, None, None, None].expand(1, 8, 2, 1, 16, 1)
    c, t, used = ref.compact(cache, table, lens, 16)
    assert used == 3 and t.tolist() == [[0, 2, -1], [0, 1, -1], [-1, -1, -1]]
    assert c[0, :, 0, 0, 0, 0].tolist() == [5, 1, 2, 3, 4, 5, 6, 7]
    c, t, n, left = ref.fork(cache, table, lens, [1], [2], 16)
    assert t[2].tolist() == [5, 0, -1] and n.tolist() == [20, 17, 17] and left == 4
    assert c[0, 0, 0, 0, :, 0].tolist() == [1.0] + [0.0] * 15


SHARES = r"""
#include <cstdio>
#include <cstdlib>
#include "kda_attn_plan.cuh"
using namespace kda::attn;
int main() {
  srand(1);
  for (int turn = 0; turn < 20000; ++turn) {
    Run r;
    r.G = 1 + rand() % (turn % 8 ? 20 : 300);
    r.before = rand() % (turn % 3 ? 20000 : 200);
    r.len = turn % 4 ? rand() % 1000 : 1;
    r.window = turn % 2 ? 1 + rand() % 5000 : 0;
    long long sum = 0;
    for (int i = 0; i <= r.items(); ++i) {
      if (r.units_before(i) != sum) return printf("units G %d before %d len %d window %d item %d\n", r.G, r.before, r.len, r.window, i), 1;
      if (i == r.items()) break;
      int lo = 1 << 30, hi = 0;  // the tiles that the item's rows see, row by row
      for (int q = i * kRows; q < (i + 1) * kRows && q < r.rows(); ++q) {
        const int p = r.before + q / r.G, f = r.window && p - r.window + 1 > 0 ? p - r.window + 1 : 0;
        if (f / kTile < lo) lo = f / kTile;
        if (p / kTile + 1 > hi) hi = p / kTile + 1;
      }
      if (lo != r.first(i) || hi != r.end(i)) return printf("tiles G %d before %d len %d window %d item %d\n", r.G, r.before, r.len, r.window, i), 1;
      sum += kItemUnits + (hi - lo) * ((r.rows() - i * kRows > 128) ? kWideTile : 1);
    }
  }
  Run far{(1 << 27) - 70000, 70000, 128, 0};  // the largest positions
  long long sum = 0;
  for (int i = 0; i < far.items(); ++i) sum += kItemUnits + static_cast<long long>(far.end(i)) * (far.rows() - i * kRows > 128 ? kWideTile : 1);
  if (sum != far.units()) return printf("far\n"), 1;
  // an item cut at any units: parts follow one another, none in the middle is empty, and the last one is known
  for (int turn = 0; turn < 20000; ++turn) {
    const int n = 1 + rand() % 60, weight = 1 + turn % kWideTile;
    const long long at = rand() % 500, units = kItemUnits + n * weight, each = kLeastUnits + rand() % 40;
    int done = 0;
    long long last = -1;
    for (long long c = at / each; c * each < at + units; ++c) {
      const int from = tiles_before(c * each - at, n, weight), to = tiles_before((c + 1) * each - at, n, weight);
      if (from != done || (from > 0 && from < n && to == from)) return printf("part\n"), 1;
      if (to > from) last = c;
      done = to;
    }
    if (done != n || last != quotient(at + kItemUnits + static_cast<long long>(n - 1) * weight, each)) return printf("parts\n"), 1;
  }
  return 0;
}
"""


def test_units_of_items_in_closed_form(tmp_path):
    """The sums by which attention cuts its work, against counting tile by tile."""
    src, exe = tmp_path / "shares.cpp", tmp_path / "shares"
    src.write_text(SHARES)
    csrc = os.path.join(os.path.dirname(kda.__file__), "csrc")
    subprocess.run(["g++", "-O2", "-std=c++17", "-I" + csrc, str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)], capture_output=True, text=True).stdout == ""
    assert subprocess.run([str(exe)]).returncode == 0


SCRATCH = 152 * 2 * 256 * (8 + 4 * 64)  # bytes of the attention's parts at least, heads of 64


@pytest.mark.parametrize("what", ["q", "o", "cache", "table", "lens", "slots", "cu"])
@pytest.mark.parametrize("end", ["first", "last"])
def test_attention_refuses_a_workspace_over_what_it_uses(L, what, end):
    """What the call reads or returns at the workspace's first bytes, or at its last ones."""
    ws, size = 64 * GB, kda.attn_workspace_bytes(2, 8, 4, 2, 64)
    assert size >= SCRATCH
    there = at(ws if end == "first" else ws + SCRATCH - 16)
    assert call(L.kda_attn_paged, ATTN, dict(ws=at(ws), size=size, **{what: there})) == SHAPE
    # where no part goes into it, or behind it, nothing is wrong but that there is no GPU
    assert call(L.kda_attn_paged, dict(ATTN, total=0), dict(ws=at(ws), size=size, **{what: there})) == 0


@pytest.mark.parametrize("what", ["table", "lens", "slots", "cu"])
def test_attention_refuses_an_output_over_its_tables(L, what):
    assert call(L.kda_attn_paged, ATTN, {what: at(3 * GB + 7 * 512 + 508)}) == SHAPE


@pytest.mark.parametrize("what", ["table", "lens", "slots", "cu"])
@pytest.mark.parametrize("end", [0, 10 * 2 * 2 * 16 * 64 * 2 - 4])
def test_append_refuses_tables_in_the_cache(L, what, end):
    assert call(L.kda_kv_append, APPEND, {what: at(4 * GB + end)}) == SHAPE


POOL = 2 * 10 * 2 * 2 * 16 * 64 * 2  # bytes of the cache of FORK and COMPACT: two layers


@pytest.mark.parametrize("end", [0, POOL - 16])
def test_pages_refuse_tables_in_the_cache(L, end):
    for what in ("table", "lens", "src", "dst", "left", "ws"):
        assert call(L.kda_pages_fork, FORK, {what: at(4 * GB + end)}) == SHAPE
    for what in ("table", "lens", "out", "used", "ws"):
        assert call(L.kda_pages_compact, COMPACT, {what: at(4 * GB + end)}) == SHAPE

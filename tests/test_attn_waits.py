"""The waits of paged attention's kernel that hang on more than one barrier, on the CPU: models of the
warps that signal and of those that wait, in random order, with signals that arrive as late as they
like and in any order between barriers.  The rules for barriers and phases are the kernel's own
(csrc/kda_attn_plan.cuh).  A wait that returns too early, or never, is found."""
import os
import subprocess

import linear_attention_serving_chunk_gb300 as kda

MODEL = r"""
#include <cstdio>
#include <cstdlib>
#include <deque>
#include <vector>
#include "kda_attn_plan.cuh"
using namespace kda::attn;

// A barrier that one signal completes: a wait for phase n returns where the current phase's parity is another.
struct Bar {
  unsigned done = 0, due = 0;  // phases completed; signals on their way
  bool test(unsigned phase) const { return ((done ^ phase) & 1) != 0; }
};
bool often(int n) { return rand() % n != 0; }
// One of the signals that are on their way arrives; those of the slow barrier when nothing else happens, mostly.
bool deliver(std::vector<Bar *> &bars, int slow, bool idle) {
  const int n = static_cast<int>(bars.size()), from = rand() % n;
  for (int i = 0; i < n; ++i) {
    Bar &b = *bars[(from + i) % n];
    if (!b.due || ((from + i) % n == slow && !idle && often(40))) continue;
    --b.due, ++b.done;
    return true;
  }
  return false;
}
"""

SUMS = MODEL + r"""
// Three places of scores, two warpgroups in turn; a sum of a warpgroup follows its weights, and its next scores may
// come before that.
int main() {
  for (int turn = 0; turn < 4000; ++turn) {
    srand(turn);
    std::vector<int> items(1 + rand() % 6);  // scores of each
    for (int &n : items) n = 1 + rand() % 12;
    Bar scores[2][2], sums[2][2];
    std::vector<Bar *> bars;
    for (int w = 0; w < 2; ++w)
      for (int i = 0; i < 2; ++i) bars.push_back(&scores[w][i]), bars.push_back(&sums[w][i]);
    const int slow = rand() % 8;
    unsigned summed[2] = {0, 0}, given[2] = {0, 0};  // sums that are made; weights that are there
    // the tensor core does one thing after another: a sum (w, none), or a signal
    struct Op { int w; Bar *signal; };
    std::deque<Op> queue;
    // the warp that issues
    size_t item = 0;
    int s = -1;
    unsigned announced[2] = {0, 0}, issued[2] = {0, 0};
    auto next_scores = [&](int w) { queue.push_back({w, &scores[w][turn_of(announced[w]++)]}); };
    auto issue = [&]() -> bool {
      if (item == items.size()) return false;
      const int all = items[item];
      if (s < 0) {
        for (s = 0; s < 3 && s < all; ++s) next_scores(s & 1);
        s = 0;
        return true;
      }
      const int w = s & 1;
      if (given[w] <= issued[w]) return false;
      queue.push_back({w, nullptr});
      queue.push_back({w, &sums[w][turn_of(issued[w]++)]});
      if (s + 3 < all) next_scores((s + 3) & 1);
      if (++s == all) ++item, s = -1;
      return true;
    };
    // the warpgroups
    struct Group { size_t item = 0; int j = 0, at = 0; unsigned n = 0; } group[2];
    auto step = [&](int w) -> int {
      Group &g = group[w];
      while (g.item < items.size() && g.j >= (items[g.item] + 1 - w) / 2) ++g.item, g.j = 0;
      if (g.item == items.size()) return 0;
      if (g.at == 0) {
        if (!scores[w][turn_of(g.n)].test(phase_of(g.n))) return 0;
        ++g.n, g.at = 1;
      } else if (g.at == 1) {
        if (g.n > 2) {
          if (!sums[w][turn_of(g.n - 3)].test(phase_of(g.n - 3))) return 0;
          if (summed[w] < g.n - 2) return -1;
        }
        g.at = g.j > 0 && rand() % 2 ? 2 : 3;
      } else if (g.at == 2) {  // O is scaled: the sum before has to be there
        if (!sums[w][turn_of(g.n - 2)].test(phase_of(g.n - 2))) return 0;
        if (summed[w] < g.n - 1) return -1;
        g.at = 3;
      } else {
        ++given[w], ++g.j, g.at = 0;
      }
      return 1;
    };
    for (int idle = 0; idle < 400;) {
      int did = 0;
      const int who = rand() % 5;
      if (who == 0) did = issue();
      else if (who <= 2) did = step(who - 1);
      else if (who == 3) did = deliver(bars, slow, idle > 60);
      else if (!queue.empty()) {
        if (queue.front().signal) ++queue.front().signal->due;
        else ++summed[queue.front().w];
        queue.pop_front();
        did = 1;
      }
      if (did < 0) return printf("turn %d: O is touched while a sum is being made\n", turn), 1;
      idle = did ? 0 : idle + 1;
    }
    if (item < items.size()) return printf("turn %d: everyone waits\n", turn), 1;
  }
  return 0;
}
"""

RING = MODEL + r"""
// Two warps that fill a ring with keys and values, and one that uses the tiles in order and releases them.
int main() {
  for (int turn = 0; turn < 4000; ++turn) {
    srand(turn);
    const int stages = turn % 2 ? 5 : 10, ahead = turn % 2 ? 2 : 2 + rand() % 2;
    std::vector<int> tiles;  // whose, in the order in which they are used
    for (int item = 1 + rand() % 8; item-- > 0;) {
      const int n = 1 + rand() % (rand() % 2 ? 3 : 20);
      for (int j = 0; j < ahead && j < n; ++j) tiles.push_back(0);
      for (int j = 0; j < n; ++j) {
        tiles.push_back(1);
        if (j + ahead < n) tiles.push_back(0);
      }
    }
    const int all = static_cast<int>(tiles.size());
    std::vector<Bar> empty(2 * stages);
    std::vector<Bar *> bars;
    for (Bar &b : empty) bars.push_back(&b);
    const int slow = rand() % (2 * stages);
    std::vector<int> filled(all, 0), released(all, 0);
    RingAt at[2], use;
    int fill[2] = {0, 0}, used = 0, freed = 0, lag = rand() % 4;
    auto load = [&](int w) -> int {
      if (fill[w] == all) return 0;
      RingAt &r = at[w];
      if (tiles[fill[w]] == w) {
        if (!empty[2 * r.stage + r.free()].test(r.free_phase())) return 0;
        if (fill[w] >= stages && !released[fill[w] - stages]) return -1;
        filled[fill[w]] = 1;
      }
      ++fill[w];
      r.next(stages);
      return 1;
    };
    for (int idle = 0; idle < 400;) {
      int did = 0;
      const int who = rand() % 4;
      if (who <= 1) did = load(who);
      else if (who == 2) did = deliver(bars, slow, idle > 60);
      else if (used < all && filled[used]) {
        ++used, did = 1;
        // released up to `lag` tiles later, in order
        while (freed < used && (used - freed > lag || used == all)) {
          released[freed++] = 1;
          ++empty[2 * use.stage + use.release()].due;
          use.next(stages);
        }
      }
      if (did < 0) return printf("turn %d: a tile is written over before it is released\n", turn), 1;
      idle = did ? 0 : idle + 1;
    }
    if (used < all) return printf("turn %d: everyone waits\n", turn), 1;
  }
  return 0;
}
"""


def run(tmp_path, text):
    src, exe = tmp_path / "waits.cpp", tmp_path / "waits"
    src.write_text(text)
    csrc = os.path.join(os.path.dirname(kda.__file__), "csrc")
    subprocess.run(["g++", "-O2", "-std=c++17", "-I" + csrc, str(src), "-o", str(exe)], check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True)
    assert (got.stdout, got.returncode) == ("", 0)


def test_a_sum_is_complete_before_it_is_scaled(tmp_path):
    run(tmp_path, SUMS)


def test_a_place_is_released_before_it_is_filled(tmp_path):
    run(tmp_path, RING)

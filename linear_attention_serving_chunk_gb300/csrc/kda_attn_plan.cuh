// How the work of paged attention is cut into tiles and shared out.  Host and device: no memory is
// touched here.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define KDA_HD __host__ __device__ __forceinline__
#else
#define KDA_HD inline
#endif

namespace kda {
namespace attn {

constexpr int kRows = 256;     // rows (token, head of the group) of an item, two tiles of 128
constexpr int kTile = 128;     // positions of a tile of keys
constexpr int kCtas = 152;     // one on each SM

// What things cost, in tiles of an item of at most 128 rows (each of its two chains takes every other tile).
constexpr int kWideTile = 2;   // a tile of an item with more rows
constexpr int kItemUnits = 7;  // an item, beside its tiles
constexpr int kLeastUnits = 4; // the least share of a CTA

// a / b for a >= 0, b > 0: 64-bit division takes several times as long.
KDA_HD int64_t quotient(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}
KDA_HD int64_t floor_div(int64_t a, int64_t b) { return a >= 0 ? quotient(a, b) : -quotient(b - 1 - a, b); }

// Sum of floor((2 k + b) / G) over k in [0, n), b >= 0.
//
// With b < G (the rest is n times b / G) the terms are the y in [1, m] with y G <= 2 k + b, where m
// is the last term: n m less, for each y, the ceil((y G - b) / 2) values of k that do not reach it.
KDA_HD int64_t floor_sum(int64_t n, int64_t G, int64_t b) {
  if (n <= 0) return 0;
  const int64_t q = quotient(b, G);
  int64_t sum = n * q;
  b -= q * G;
  if (G == 1) return sum + n * (n - 1);
  const int64_t m = quotient(2 * (n - 1) + b, G), odd = G & 1;
  // the sum of ceil(x / 2), x = y G - b: (x + 1) / 2 where x is odd
  const int64_t n_odd = odd ? (b & 1 ? m / 2 : (m + 1) / 2) : (b & 1 ? m : 0);
  return sum + n * m - (G * (m * (m + 1) / 2) - m * b + n_odd) / 2;
}

// One run: `len` tokens behind `before` ones, G heads a token, rows token by token.  Item i has rows
// [256 i, 256 i + 256) and the tiles that any of them sees.  Positions are under 2^27 and rows under 2^31.
struct Run {
  int before, len, G, window;  // window: the positions a token sees, 0 for all

  KDA_HD int rows() const { return len * G; }
  KDA_HD int items() const { return static_cast<int>((static_cast<unsigned>(rows()) + kRows - 1) / kRows); }
  // Tiles in front of the item's first and behind its last.
  KDA_HD int first(int i) const {
    if (!window) return 0;
    const int p = before + i * kRows / G - window + 1;
    return p > 0 ? p / kTile : 0;
  }
  KDA_HD int end(int i) const {
    const int last = static_cast<int>((static_cast<unsigned>(i + 1) * kRows - 1) / G);
    return (before + (last < len - 1 ? last : len - 1) + kTile) / kTile;
  }
  KDA_HD int rows_of(int i) const { return rows() - i * kRows < kRows ? rows() - i * kRows : kRows; }
  KDA_HD int weight(int i) const { return rows_of(i) > 128 ? kWideTile : 1; }
  KDA_HD int64_t units_of(int i) const { return kItemUnits + static_cast<int64_t>(weight(i)) * (end(i) - first(i)); }
  // Units of the items in front of item i: both ends grow by 256 / (128 G) tiles an item, rounded down.
  KDA_HD int64_t units_before(int i) const {
    const int n = items();
    const int64_t k = i < n ? i : n - 1;
    if (n == 0 || i == 0) return 0;
    const int64_t last = units_of(n - 1);
    if (n == 1) return last;
    int64_t tiles = floor_sum(k, G, (static_cast<int64_t>(G) * (before + kTile) + kRows - 1) / kTile);
    if (window) {
      const int64_t b = floor_div(static_cast<int64_t>(G) * (before - window + 1), kTile), skip = b < 0 ? (1 - b) / 2 : 0;
      if (k > skip) tiles -= floor_sum(k - skip, G, 2 * skip + b);
    }
    return k * kItemUnits + tiles * kWideTile + (i < n ? 0 : last);
  }
  KDA_HD int64_t units() const { return units_before(items()); }
};

// Tiles of an item that lie in front of unit u behind its beginning; a tile belongs to the share in which it
// begins.
KDA_HD int tiles_before(int64_t u, int n, int weight) {
  u -= kItemUnits;
  return u <= 0 ? 0 : u >= static_cast<int64_t>(n) * weight ? n : static_cast<int>((u + weight - 1) / weight);
}

// What happens k-th and is announced on two barriers in turn: the barrier, and the phase that it completes there.
// A wait tells a phase from the one before by its parity alone.  So who waits for the k-th has waited for the (k - 2)nd,
// and waits before the (k + 2)nd can happen: barriers are not signalled in the order of what completes them.
KDA_HD constexpr uint32_t turn_of(uint32_t k) { return k & 1; }
KDA_HD constexpr uint32_t phase_of(uint32_t k) { return k >> 1; }

// A place of a ring of `stages`, as a warp goes through them.  Two warps fill it, each the places of its own tiles, so
// neither waits for every release of a place: with one barrier for a place, a release that arrives late could be
// taken for the one two rounds before.  With two in turn, that would need one from four rounds before, whose
// place has not been filled again then.
struct RingAt {
  uint32_t stage = 0, round = 0;
  KDA_HD void next(uint32_t stages) {
    if (++stage == stages) stage = 0, ++round;
  }
  KDA_HD uint32_t release() const { return turn_of(round); }  // the barrier of this round's release
  // The release of the round before, which a fill waits for (in front of the first: the phase before a new barrier's).
  KDA_HD uint32_t free() const { return turn_of(round - 1); }
  KDA_HD uint32_t free_phase() const { return phase_of(round - 1); }
};

// Units of a CTA, at least two of the widest tiles, so that no share within an item is empty.
static_assert(kLeastUnits >= 2 * kWideTile, "shares");
KDA_HD int64_t share(int64_t units) {
  const int64_t each = (units + kCtas - 1) / kCtas;
  return each > kLeastUnits ? each : kLeastUnits;
}

}  // namespace attn
}  // namespace kda

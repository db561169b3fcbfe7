// Causal attention of a batch of runs over a paged cache, on tcgen05.
//
//   o_r = sum_j p_rj v_j / sum_j p_rj,   p_rj = exp(scale q_r . k_j - m_r),   j <= position of r
//
// in one pass over the keys, with the running maximum m and sum of each row (a tile that raises the
// maximum scales what was summed before).  A row is one token and one of the G heads that share a
// head of keys: rows are packed token by token, so a tile of 128 rows holds 128 / G tokens and
// every key that is read serves all of them.
//
// An item is a (run, head of keys, 256 rows) and its tiles of 128 keys; kda_attn_plan.cuh cuts the
// items of a call into equal shares of tiles, one for each of 152 CTAs, whatever the lengths: an
// item that is cut leaves (m, sum, o) of its parts in the workspace and a second kernel joins them.
// Nothing is taken in turn, so the same call gives the same bits.
//
// One CTA: two warpgroups, each with its 128 rows' scores, weights and sums in TMEM, a warp that
// issues the MMAs, one that works out the items, and two that look up pages and load tiles of K and of
// V by TMA into a ring of 160 KB.
//   S_w = Q_w K^T         128 x 128 x D, K-major tiles
//   P_w = exp(..) bf16    in the columns of S_w, read from there by the MMA
//   O_w += P_w V          128 x D x 128, V as it lies in the cache
// While one warpgroup turns its scores into weights the tensor core works for the other.  Items of
// more than 128 rows give each warpgroup 128 of them, with the same tiles.  Those of at most 128
// (tokens, drafted runs) give both the same rows and every other tile: then the keys are what counts,
// and two chains hide each other's latency; their sums meet in shared memory at the end.  With heads
// of 64 the sums leave room in TMEM for a third place of scores, which run ahead by one: their MMAs
// take half as long, and with two places a warpgroup waits for them (955 against 790 us for 4096 tokens
// behind 28,672, 32 heads of 64).
//
// Scores, maxima, sums and O are fp32.  The weights are rounded to bf16 for their product with V,
// which a row's sum does not see: by at most 2^-8 of each weight, in either direction.  A maximum is
// kept until a score is more than 2^8 above it in the exponent's base: weights up to 256 lose nothing, and
// most tiles then need no scaling of O.  The product with the scale is rounded in the maximum alone, which moves all
// weights of a row by the same factor; from scores of 2^31 on that factor may leave fp32's range, and a row whose
// sum is 0 then is NaN.  (A row sees itself: in range, its sum is not 0.)
//
// A warp whose rows are all beyond the item (three of four in a step of single tokens) computes
// nothing.  Keys behind a row's position, or behind the window, weigh nothing whatever they are; the
// rows of V behind the sequence are zeroed, for 0 times what lies there might not be 0.
//
// Prompt chunks are bound by the chain of each warpgroup, scores, weights, product, which the other one's hides in
// part: the tensor core is busy for 68 to 73 % of the time, and without the exponentials a call takes 5 % less, with half
// of the products 19 %.  4096 tokens behind 28,672, 32 heads of 128 over 8 of keys, take 1350 to 1390 us one
// after another for a second, at the clock that the power limit leaves (1.5 PFLOP/s; a large product of the library
// then keeps 1.74), and 1160 to 1190 in short bursts.  Single tokens are bound by memory: 646 us for 128
// sequences of 1000 to 16,000 tokens, 4.49 GB.  Short calls are bound by latency: about 5 us until the
// first scores, 1 us a tile (2 the first time, while its code comes), 3 us for the join.
//
// The MMAs are issued by an elected thread, with the warp's number and TMEM's address uniform for all: by lane 0, each
// waits for its operands to come into uniform registers (1694 us for those chunks in a burst).  Two warps load:
// with one, single tokens take 652, and heads of 64 in pages of 16 526 instead of 357.
#include <string.h>

#include <type_traits>

#include "kda_attn_plan.cuh"
#include "kda_paged.cuh"
#include "kda_pdl.cuh"
#include "kda_sm100.cuh"
#include "kda_tc_common.cuh"

namespace kda {

namespace {

using namespace sm100;
using attn::kCtas;
using attn::kRows;
using attn::kTile;
using attn::phase_of;
using attn::RingAt;
using attn::Run;
using attn::turn_of;

constexpr int kThreads = 384;
// Registers a thread: a launch of 384 threads gives 168 to each, 3 x 168 = 2 x 208 + 88.
constexpr int kRowRegs = 208, kOtherRegs = 88;
constexpr int kMmaWarp = 8, kLoadWarp = 9, kItemWarp = 10, kLoadVWarp = 11;
constexpr uint32_t kPolls = 1u << 20;
constexpr float kKeep = 8.f;  // log2

struct AttnArgs {
  const kda_bf16 *q;
  int64_t ldq;
  kda_bf16 *o;
  int64_t ldo;
  Runs runs;
  PagedSeqs seqs;
  int H, G, window;
  float scale2;   // scale times log2(e)
  uint8_t *ws;    // or NULL: no item is cut
  int *status;
  int test_stall;  // KDA_ATTN_TEST_STALL
};

// The workspace: for each CTA what the first item that it cuts off needs, and whether one of its waits gave up (then
// its parts may not be there), then the parts: 2 c is the end or the middle of an item that an earlier CTA
// began, 2 c + 1 the beginning of one that CTA c began.
struct Cut {
  int rows, row0, token0, head, last;  // last: the CTA of the last part; rows 0: nothing is cut
  int pad[3];
};
constexpr int kCutWords = sizeof(Cut) / 4, kFailed = kCutWords * kCtas;  // a word for each CTA from there on
constexpr size_t kCutBytes = (4 * (kCutWords + 1) * kCtas + 127) / 128 * 128;  // (lines of parts begin where the memory's do)
constexpr size_t kStatBytes = sizeof(float2) * kRows * 2 * kCtas;
constexpr size_t ws_bytes(int D) { return kCutBytes + kStatBytes + sizeof(float) * kRows * 2 * kCtas * D; }

struct Item {
  int rows;    // of the item; -1: there is none any more
  int row0;    // its first one in the run
  int token0;  // the run's first token
  int head;    // of keys
  int before;  // tokens in front of the run
  int reach;   // and with it
  int lo, n;   // tiles
  int slot;
  int part;    // of the workspace, -1: the whole item
};
constexpr int kItems = 4;

template <int D>
struct Smem {
  static constexpr uint32_t kRegion = kTile * 128;              // 64 columns of a tile
  static constexpr uint32_t kTileBytes = D / 64 * kRegion;
  static constexpr int kStages = D == 128 ? 5 : 10;
  static constexpr int kScores = D == 128 ? 2 : 3;              // places of scores and weights in TMEM
  static constexpr uint32_t kO = kScores * 128;                 // sums behind them
  // Of scores s of an item behind `turn` others: the warpgroup's own, or a third one in turn.
  __device__ static uint32_t place(uint32_t turn, uint32_t s) {
    return kScores == 2 ? s & 1 : (turn + s) % kScores;
  }
  static constexpr uint32_t Q = 0;
  static constexpr uint32_t MERGE = kTileBytes;                 // second Q tile, or 128 x 64 fp32
  static constexpr uint32_t STAGE = MERGE + 32 * 1024;
  static constexpr uint32_t BAR = STAGE + kStages * kTileBytes;
  static constexpr uint32_t FULL = BAR, EMPTY = FULL + 8 * kStages, SFULL = EMPTY + 16 * kStages,
                            PREADY = SFULL + 32, QREADY = PREADY + 8 * kScores, OFULL = QREADY + 16,
                            ODONE = OFULL + 16, IFULL = ODONE + 32, IEMPTY = IFULL + 8 * kItems,
                            MFULL = IEMPTY + 8 * kItems, MEMPTY = MFULL + 8, FIN = MEMPTY + 8;
  static constexpr uint32_t TMEM = FIN + 8;
  // int64: the first unit of the share's first run, the run's units for a head, its number; partial sums
  static constexpr uint32_t PLAN = TMEM + 8;
  static constexpr uint32_t FIRST = PLAN + 8 * 16;                // that run
  static constexpr uint32_t ITEM = FIRST + 32;
  static constexpr uint32_t STAT = ITEM + sizeof(Item) * kItems;
  static constexpr uint32_t BYTES = STAT + 128 * sizeof(float2);
  static_assert(BYTES <= 232448 && STAGE % 1024 == 0 && MERGE % 1024 == 0 && STAT % 8 == 0 &&
                    TMEM % 8 == 0,
                "shared memory");
};

template <int REGS, bool MORE>
__device__ __forceinline__ void set_registers() {
  if constexpr (MORE)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS));
  else
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS));
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void st_shared4(uint32_t at, float x, float y, float z, float w) {
  asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(x), "f"(y), "f"(z), "f"(w)
               : "memory");
}
__device__ __forceinline__ float4 ld_shared4(uint32_t at) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(at)
               : "memory");
  return v;
}
// Loads that stay in the order in which they stand.
__device__ __forceinline__ void ld_in_turn(float2 &v, const float2 *p) {
  asm volatile("ld.global.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "l"(p));
}
__device__ __forceinline__ void ld_in_turn(float4 &v, const float4 *p) {
  asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "l"(p));
}

__device__ __forceinline__ bool elect() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one != 0;
}

// D[tmem] (+)= A[tmem] * B[smem desc]^T: A is 128 rows of packed bf16 pairs, one column for two k.
__device__ __forceinline__ void mma_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Two values as bf16, the first in the lower half.
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Ones from bit n on: all for n <= 0, none for n >= 32.  (A mask's bit a score: two instructions, three with the
// bounds compared, which is 1.5 us of a mixed batch's 28.)
__device__ __forceinline__ uint32_t ones_from(int n) {
  uint32_t r;
  asm("shl.b32 %0, %1, %2;" : "=r"(r) : "r"(~0u), "r"(max(n, 0)));  // (a shift by 32 or more leaves nothing)
  return r;
}

// Run b as this call takes it: empty where an entry is malformed.
struct RunAt {
  int begin, slot;
  Run run;
};
static_assert(sizeof(RunAt) <= 32, "Smem::FIRST");
__device__ __forceinline__ RunAt run_at(const AttnArgs &a, int b, bool &bad) {
  int64_t begin = b * a.runs.fixed_len, end = begin + a.runs.fixed_len;
  // (the offsets and the slot are on their way at once: this is on every call's way to its first tile)
  const int slot = a.seqs.slots ? a.seqs.slots[b] : b;
  bool ok = true;
  if (a.runs.cu) ok = seq_range(a.runs.cu, b, a.runs.total, begin, end);
  const int64_t len = end - begin;
  int before = -1;
  if (slot >= 0 && slot < a.seqs.n_slots) before = a.seqs.lens[slot];
  ok = ok && before >= 0 &&
       before + len <= (static_cast<int64_t>(a.seqs.max_pages) << a.seqs.page_shift);
  if (!ok) {
    bad = true;
    return RunAt{0, 0, Run{0, 0, a.G, a.window}};
  }
  return RunAt{static_cast<int>(begin), slot, Run{before, static_cast<int>(len), a.G, a.window}};
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
attn_kernel(const __grid_constant__ CUtensorMap map, const AttnArgs a) {
  using M = Smem<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sb = smem_u32(smem);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31, cta = blockIdx.x;
  grid_launch_dependents();
  auto start_ws = [&]() {  // no item is cut yet, no wait has given up
    if (!a.ws || tid > kCutWords) return;
    reinterpret_cast<int *>(a.ws)[tid < kCutWords ? cta * kCutWords + tid : kFailed + cta] = 0;
  };
  if ((sb & 1023u) != 0) {  // the swizzled tiles need it
    grid_dependency_wait();
    start_ws();
    if (tid == 0) atomicOr(a.status, KDA_ERR_UNSUPPORTED);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < M::kStages; ++i) {
      mbar_init(sb + M::FULL + 8 * i, 1);
      mbar_init(sb + M::EMPTY + 16 * i, 1);
      mbar_init(sb + M::EMPTY + 16 * i + 8, 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(sb + M::SFULL + 8 * i, 1);
      mbar_init(sb + M::ODONE + 8 * i, 1);
    }
    for (int i = 0; i < M::kScores; ++i) mbar_init(sb + M::PREADY + 8 * i, 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(sb + M::QREADY + 8 * i, 4);
      mbar_init(sb + M::OFULL + 8 * i, 1);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(sb + M::IFULL + 8 * i, 1);
      mbar_init(sb + M::IEMPTY + 8 * i, 11);
    }
    mbar_init(sb + M::MFULL, 4);
    mbar_init(sb + M::MEMPTY, 4);
    mbar_init(sb + M::FIN, 1);
    fence_mbar_init();
  }
  if (warp == kLoadWarp && lane == 0) prefetch_tensormap(&map);
  if (warp == kMmaWarp) {
    tmem_alloc(sb + M::TMEM, 512);
    tmem_relinquish();
  }

  grid_dependency_wait();
  start_ws();

  // This CTA's share: all units, then the run in which the share begins.
  int64_t *const plan = reinterpret_cast<int64_t *>(smem + M::PLAN);
  bool bad = false;
  int64_t units = 0, whole = 0;  // whole: those of one head of this thread's run
  RunAt run{};
  for (int b = tid; b < a.runs.n; b += kThreads) {
    run = run_at(a, b, bad);
    whole = run.run.units();
    units += whole * a.H;
  }
  auto sum_up = [&](int64_t v, int64_t &before) {  // over the block; `before`: over the threads before
    int64_t x = v;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += y;
    }
    __syncthreads();
    if (lane == 31) plan[4 + warp] = x;
    __syncthreads();
    int64_t all = 0;
    before = x - v;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += plan[4 + w];
      all += plan[4 + w];
    }
    return all;
  };
  int64_t before;
  units = sum_up(units, before);
  const int64_t each = attn::share(units), start = each * cta, stop = min(start + each, units);
  auto found = [&](int b) {
    if (before <= start && start < before + whole * a.H) {
      plan[0] = before;
      plan[1] = whole;
      plan[2] = b;
      *reinterpret_cast<RunAt *>(smem + M::FIRST) = run;
    }
  };
  if (a.runs.n <= kThreads) {
    found(tid);
  } else if (start < stop) {
    int64_t carry = 0;
    for (int b0 = 0; b0 < a.runs.n && carry <= start; b0 += kThreads) {
      const int b = b0 + tid;
      whole = 0;
      if (b < a.runs.n) {
        run = run_at(a, b, bad);
        whole = run.run.units();
      }
      const int64_t all = sum_up(whole * a.H, before);
      before += carry;
      carry += all;
      found(b);
    }
  }
  if (bad) atomicOr(a.status, KDA_ERR_SHAPE);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t *>(smem + M::TMEM), 0);
  Item *const items = reinterpret_cast<Item *>(smem + M::ITEM);

  // Every wait is bounded.  A role whose wait gives up leaves its loop, and those that wait for it
  // give up in their turn.
  bool gave_up = false;
  auto wait = [&](uint32_t bar, uint32_t phase) -> bool {
    uint32_t left = kPolls;
#pragma unroll 1
    while (!mbar_try_wait(bar, phase & 1u))
      if (--left == 0) {
        gave_up = true;
        break;
      }
    gave_up = __any_sync(0xffffffffu, gave_up) != 0;  // a warp goes on or stops as one
    return !gave_up;
  };
  auto arrive = [&](uint32_t bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };

  // What follows a wait that gave up: the code, and for the join that parts may be missing.
  auto fail = [&]() {
    atomicOr(a.status, KDA_ERR_TIMEOUT);
    if (a.ws) reinterpret_cast<int *>(a.ws)[kFailed + cta] = 1;
  };
  // Test hook: a wait that nothing ends, before anything is issued.
  if (a.test_stall && cta == 1) {
    if (!mbar_wait_bounded(sb + M::FIN, 0, 1u << 10) && lane == 0) fail();
    __syncthreads();
    if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
    return;
  }

  if (warp >= 8) {
    set_registers<kOtherRegs, false>();
    if (warp == kItemWarp) {
      // ---- items -----------------------------------------------------------------------------
      uint32_t given = 0;
      auto give = [&](const Item &it) -> bool {
        const uint32_t s = given % kItems;
        if (!wait(sb + M::IEMPTY + 8 * s, given / kItems + 1)) return false;
        if (lane == 0) items[s] = it;
        arrive(sb + M::IFULL + 8 * s);
        ++given;
        return true;
      };
      if (start < stop) {
        int b = static_cast<int>(plan[2]), held = -32;
        bool none = false;
        RunAt r = *reinterpret_cast<const RunAt *>(smem + M::FIRST), lot{};
        auto take = [&]() {  // of 32 runs at a time, one in each lane
          if (b >= held + 32) {
            held = b;
            lot = run_at(a, min(b + lane, a.runs.n - 1), none);
          }
          const int from = b - held;
          auto of = [&](int v) { return __shfl_sync(0xffffffffu, v, from); };
          r = RunAt{of(lot.begin), of(lot.slot), Run{of(lot.run.before), of(lot.run.len), a.G, a.window}};
        };
        const int64_t whole = plan[1], x0 = start - plan[0], h0 = attn::quotient(x0, whole);
        const int64_t x = x0 - h0 * whole;
        int h = static_cast<int>(h0), i = 0, hi = r.run.items();
        while (hi - i > 32) {  // the items around unit x, 32 ways at a time
          const int step = (hi - i + 31) / 32, c = i + lane * step;
          const unsigned some = __ballot_sync(0xffffffffu, c < hi && r.run.units_before(c) <= x);
          i += (31 - __clz(some)) * step;
          hi = min(hi, i + step);
        }
        // and of these, each in a lane, the one that unit x is in
        const int64_t front = i ? r.run.units_before(i) : 0;
        const int mine = i + lane < hi ? static_cast<int>(r.run.units_of(i + lane)) : 0;
        int ends = mine;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
          const int y = __shfl_up_sync(0xffffffffu, ends, d);
          if (lane >= d) ends += y;
        }
        const int in = __ffs(__ballot_sync(0xffffffffu, front + ends > x)) - 1;
        i += in;
        int64_t at = plan[0] + h * whole + front + __shfl_sync(0xffffffffu, ends - mine, in);  // where it begins
        while (at < stop) {
          const int lo = r.run.first(i), n = r.run.end(i) - lo, weight = r.run.weight(i);
          // this share's part of the item, in tiles
          int from = attn::tiles_before(start - at, n, weight), to = attn::tiles_before(stop - at, n, weight);
          if (!a.ws) {  // an item belongs to the share in which it begins
            from = 0;
            to = at >= start ? n : 0;
          }
          if (from < to) {
            Item it;
            it.row0 = i * kRows;
            it.rows = r.run.rows_of(i);
            it.token0 = r.begin;
            it.head = h;
            it.before = r.run.before;
            it.reach = r.run.before + r.run.len;
            it.lo = lo + from;
            it.n = to - from;
            it.slot = r.slot;
            it.part = from > 0 ? 2 * cta : to < n ? 2 * cta + 1 : -1;
            if (from == 0 && to < n && lane == 0) {
              const int64_t last = at + attn::kItemUnits + static_cast<int64_t>(n - 1) * weight;
              reinterpret_cast<Cut *>(a.ws)[cta] =
                  Cut{it.rows, it.row0, it.token0, h, static_cast<int>(attn::quotient(last, each)), {}};
            }
            if (!give(it)) break;
          }
          at += attn::kItemUnits + static_cast<int64_t>(n) * weight;
          if (++i < r.run.items()) continue;
          i = 0;
          if (++h < a.H) continue;
          h = 0;
          do {
            if (++b == a.runs.n) break;
            take();
          } while (r.run.len == 0);
          if (b == a.runs.n) break;
        }
      }
      Item end{};
      end.rows = -1;
      if (!gave_up) give(end);
    } else if (warp != kMmaWarp) {
      // ---- pages and tiles: one warp loads the keys' and one the values' ------------------------
      const bool mine_is_v = warp == kLoadVWarp;
      RingAt ring;
      uint32_t taken = 0;
      bool wrong = false;
      const int per_tile = kTile >> a.seqs.page_shift;
      constexpr int halves = D / 64;
      // Tile t of keys (or values): pages that no row needs, and those outside the pool, come as zeros.
      auto load = [&](const Item &it, int t, int values, int first) -> bool {
        if ((values != 0) != mine_is_v) {  // the other's place in the ring
          ring.next(M::kStages);
          return true;
        }
        if (!wait(sb + M::EMPTY + 16 * ring.stage + 8 * ring.free(), ring.free_phase())) return false;
        const uint32_t bar = sb + M::FULL + 8 * ring.stage, to = sb + M::STAGE + ring.stage * M::kTileBytes;
        const int32_t *const row = a.seqs.table + static_cast<int64_t>(it.slot) * a.seqs.max_pages;
        if (lane == 0) {
          mbar_expect_tx(bar, M::kTileBytes);
          const int ahead = (t + 1) * per_tile + 31;  // the table's next line
          if (ahead < a.seqs.max_pages) asm volatile("prefetch.global.L1 [%0];" ::"l"(row + ahead));
        }
        __syncwarp();
        int plane = 0;
        if (lane < per_tile) {
          const int p = lane;
          const int i = t * per_tile + p, at = i << a.seqs.page_shift;
          int page = -1;
          if (at < it.reach && at + (1 << a.seqs.page_shift) > first) {
            page = row[i];
            if (page < 0 || page >= a.seqs.n_pages) {
              page = -1;
              wrong = true;
            }
          }
          plane = page < 0 ? a.seqs.n_pages * 2 * a.H : (page * 2 + values) * a.H + it.head;
        }
        for (int p = 0; p < per_tile; ++p) {
          const int at = __shfl_sync(0xffffffffu, plane, p);
          if (elect()) {
#pragma unroll
            for (int c = 0; c < halves; ++c)
              tma_load_3d(to + c * M::kRegion + (p << a.seqs.page_shift) * 128, &map, c * 64, 0, at, bar);
          }
        }
        __syncwarp();
        ring.next(M::kStages);
        return true;
      };
      auto load_item = [&](const Item &it) -> bool {
        const int first = a.window ? max(it.before + it.row0 / a.G - a.window + 1, 0) : 0;
        const int n = it.n, lo = it.lo;
        // in the order in which the MMAs want them: the scores run ahead of the sums
        const int ahead = it.rows > 128 ? (M::kScores + 1) / 2 : M::kScores;
        for (int j = 0; j < min(ahead, n); ++j)
          if (!load(it, lo + j, 0, first)) return false;
        for (int j = 0; j < n; ++j) {
          if (!load(it, lo + j, 1, first)) return false;
          if (j + ahead < n && !load(it, lo + j + ahead, 0, first)) return false;
        }
        return true;
      };

      for (;;) {
        const uint32_t s = taken % kItems;
        if (!wait(sb + M::IFULL + 8 * s, taken / kItems)) break;
        const Item it = items[s];
        arrive(sb + M::IEMPTY + 8 * s);
        ++taken;
        if (it.rows < 0 || !load_item(it)) break;
      }
      if (__any_sync(0xffffffffu, wrong) && lane == 0) atomicOr(a.status, KDA_ERR_SHAPE);
      if (gave_up) {  // the tiles on their way
        const uint32_t fills = ring.round * M::kStages + ring.stage, n = min(fills, static_cast<uint32_t>(M::kStages));
        for (uint32_t f = fills - n; f < fills; ++f)
          mbar_wait_bounded(sb + M::FULL + 8 * (f % M::kStages), (f / M::kStages) & 1u, kPolls);
      }
    } else {
      // ---- MMAs ------------------------------------------------------------------------------
      constexpr uint32_t ID_S = idesc_mma(128, kTile, kFmtBF16, kFmtBF16, 0, 0);
      constexpr uint32_t ID_O = idesc_mma(128, D, kFmtBF16, kFmtBF16, 0, 1);
      RingAt ring;
      uint32_t taken = 0, q_n[2] = {0, 0}, p_bits = 0;
      auto p_phase = [&](uint32_t place) {  // each place's phases of P, one after another
        const uint32_t phase = p_bits >> place;
        p_bits ^= 1u << place;
        return phase;
      };
      // Scores are announced to each warpgroup in turn on two barriers of its own: it waits for each of its
      // scores, and for no other's, and at most one more is there before it has taken the last.  (Descriptors
      // from an address that the compiler cannot see through: hoisted out of the loop, the sums of all steps
      // would take most of this warp's registers.)
      uint32_t announced[2] = {0, 0}, summed[2] = {0, 0};
      auto scores = [&](int place, int w, int q, uint32_t k) {
        const uint32_t full = sb + M::SFULL + 16 * w + 8 * turn_of(announced[w]++);
        if (elect()) {
          uint32_t qa = sb + M::Q + q * M::kTileBytes;
          asm volatile("" : "+r"(qa), "+r"(k));
          const uint64_t qd = sw128_desc(qa, 16, 1024), kd = sw128_desc(k, 16, 1024);
#pragma unroll
          for (int s = 0; s < D / 16; ++s) {
            const uint32_t off = ((s >> 2) * M::kRegion + (s & 3) * 32) >> 4;
            mma_f16(tmem + place * 128, qd + off, kd + off, ID_S, s > 0);
          }
          mma_commit(full);
        }
        __syncwarp();
      };
      auto weighted = [&](int place, int w, uint32_t v, bool add) {
        if (elect()) {
          uint32_t p = tmem + place * 128, o = tmem + M::kO + w * D;
          asm volatile("" : "+r"(p), "+r"(v));
          const uint64_t vd = sw128_desc(v, M::kRegion, 1024);
#pragma unroll
          for (int s = 0; s < kTile / 16; ++s)
            mma_ta(o, p + 8 * s, vd + ((s * 2048) >> 4), ID_O, add || s > 0);
        }
        __syncwarp();
      };
      auto commit = [&](uint32_t bar) {
        if (elect()) mma_commit(bar);
        __syncwarp();
      };
      auto tile = [&](uint32_t &at, uint32_t &free) -> bool {  // the next one in the ring
        at = sb + M::STAGE + ring.stage * M::kTileBytes;
        free = sb + M::EMPTY + 16 * ring.stage + 8 * ring.release();
        const bool ok = wait(sb + M::FULL + 8 * ring.stage, ring.round);
        ring.next(M::kStages);
        return ok;
      };
      auto run = [&]() {
        for (uint32_t turn = 0;;) {  // scores of the items before
          const uint32_t s = taken % kItems;
          if (!wait(sb + M::IFULL + 8 * s, taken / kItems)) return;
          const Item it = items[s];
          arrive(sb + M::IEMPTY + 8 * s);
          ++taken;
          if (it.rows < 0) return;
          const bool both = it.rows > 128;  // both warpgroups take every tile
          const int n = it.n;
          // the tile in which the sequence ends inside a page: V's rows from there on
          const int zero_tile = (it.reach & ((1 << a.seqs.page_shift) - 1)) ? it.reach / kTile - it.lo : -1;
          auto clear = [&](uint32_t v) {
            const int r0 = it.reach % kTile, r1 = (r0 | ((1 << a.seqs.page_shift) - 1)) + 1;
            for (int x = lane; x < (r1 - r0) * (D / 8); x += 32) {
              const int r = r0 + x / (D / 8), c = x % (D / 8);
              st_shared4(v + (c >> 3) * M::kRegion + r * 128 + (c & 7) * 16, 0.f, 0.f, 0.f, 0.f);
            }
            fence_proxy_async();
            __syncwarp();
          };
          // Scores s = 0, 1, ... of the item go to the warpgroups in turn, and to the places in TMEM: scores
          // s + kScores follow the sum that has read the weights s (MMAs are done in order).
          const int all = both ? 2 * n : n;
          uint32_t k = 0, v = 0, k_free = 0, v_free = 0;
          if (!wait(sb + M::QREADY, q_n[0]++)) return;
          if (both && !wait(sb + M::QREADY + 8, q_n[1]++)) return;
          tc_fence_after();
          // (twice in the code, for what it tests to be known, and two steps at a time, for the same reason)
          auto steps = [&](auto wide) -> bool {
            constexpr bool two = decltype(wide)::value;  // the tiles serve both warpgroups
            auto next_keys = [&](int s) -> bool { return (two && (s & 1)) || tile(k, k_free); };
            auto next_scores = [&](int s) {
              const bool second = s & 1;
              scores(M::place(turn, s), second, two && second, k);
              if (!two || second) commit(k_free);
            };
            for (int s = 0; s < min(M::kScores, all); ++s) {
              if (!next_keys(s)) return false;
              next_scores(s);
            }
#pragma unroll 2
            for (int s = 0; s < all; ++s) {
              const int w = s & 1, place = M::place(turn, s);
              if (!(two && w)) {
                if (!tile(v, v_free)) return false;
                if ((two ? s >> 1 : s) == zero_tile) clear(v);
              }
              const bool more = s + M::kScores < all;
              if (more && !next_keys(s + M::kScores)) return false;
              if (!wait(sb + M::PREADY + 8 * place, p_phase(place))) return false;
              tc_fence_after();
              weighted(place, w, v, s > 1);
              if (!two || w) commit(v_free);
              if (M::kScores > 2) commit(sb + M::ODONE + 16 * w + 8 * turn_of(summed[w]++));
              if (s + 2 >= all) commit(sb + M::OFULL + 8 * w);
              if (more) next_scores(s + M::kScores);
            }
            return true;
          };
          if (!(both ? steps(std::true_type{}) : steps(std::false_type{}))) return;
          turn += all;
        }
      };
      run();
      commit(sb + M::FIN);
      mbar_wait_bounded(sb + M::FIN, 0, kPolls);
    }
  } else {
    set_registers<kRowRegs, true>();
    // ---- weights and results ---------------------------------------------------------------
    const int w = warp >> 2, quad = warp & 3, r = quad * 32 + lane;  // row of the warpgroup's tile
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t to = tmem + M::kO + w * D + lanes;
    float2 *const stats = reinterpret_cast<float2 *>(smem + M::STAT);
    uint32_t taken = 0, turn = 0, s_n = 0, o_n = 0, m_n = 0;  // turn: scores of the items before
    // (an item stays in shared memory until its results are out: its fields would take registers)
    auto next_item = [&](const Item *&it) -> bool {
      const uint32_t is = taken % kItems;
      if (!wait(sb + M::IFULL + 8 * is, taken / kItems)) return false;
      it = items + is;
      ++taken;
      return true;
    };
    auto has_q = [&](const Item &it) { return it.rows > 128 || (w == 0 && it.rows >= 0); };
    // Q of an item, on its way while the last one's sums are still being made: 16 bytes a thread, eight
    // rows (16 where D = 64) at once
    auto fetch_q = [&](const Item &it) -> bool {
      if (w == 1 && !wait(sb + M::MEMPTY, m_n + 1)) return false;  // the second tile's place is shared
      constexpr int kAcross = D / 8, kAtOnce = 128 / kAcross;
      const int c = (tid & 127) % kAcross, row_of = it.rows > 128 ? w * 128 : 0;
      const uint32_t col = sb + M::Q + w * M::kTileBytes + (c >> 3) * M::kRegion;
      const kda_bf16 *const q = a.q + static_cast<int64_t>(it.token0) * a.ldq +
                                static_cast<int64_t>(it.head) * a.G * D + c * 8;
      const int i0 = (tid & 127) / kAcross, step_t = kAtOnce / a.G, step_g = kAtOnce - step_t * a.G;
      int t = (it.row0 + row_of + i0) / a.G, g = it.row0 + row_of + i0 - t * a.G;
      const int rows = min(it.rows - row_of, 128);
#pragma unroll 4
      for (int i = i0; i < rows; i += kAtOnce) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                         col + i * 128 + (((c & 7) ^ (i & 7)) << 4)),
                     "l"(__cvta_generic_to_global(q + t * a.ldq + g * D))
                     : "memory");
        t += step_t;
        if ((g += step_g) >= a.G) {
          g -= a.G;
          ++t;
        }
      }
      return true;
    };
    auto give_q = [&]() {
      asm volatile("cp.async.wait_all;" ::: "memory");
      fence_proxy_async();
      arrive(sb + M::QREADY + 8 * w);
    };
    // Writes o, or m, l and the sums of a part.
    auto results = [&](const Item &it, float m, float l) -> bool {
      const bool both = it.rows > 128;
      const int row_of = both ? w * 128 : 0, row = it.row0 + row_of + r, tok = row / a.G;
      const bool live = row_of + quad * 32 < it.rows, valid = row_of + r < it.rows;
      // parts: four columns of all rows, then the next four (a warp stores 512 bytes in a row)
      float4 *const part = it.part < 0 ? nullptr
                                       : reinterpret_cast<float4 *>(a.ws + kCutBytes + kStatBytes) +
                                             static_cast<int64_t>(it.part) * kRows * (D / 4) + row_of + r;
      kda_bf16 *const out = a.o + (static_cast<int64_t>(it.token0) + tok) * a.ldo +
                            (static_cast<int64_t>(it.head) * a.G + (row - tok * a.G)) * D;
      auto put = [&](const float (&o)[32], int c, float f) {  // columns [32 c, 32 c + 32) of this row
        if (!valid) return;
        if (part) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            part[(8 * c + i) * kRows] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = pack(o[8 * i + 2 * e] * f, o[8 * i + 2 * e + 1] * f);
            *reinterpret_cast<uint4 *>(out + 32 * c + 8 * i) = make_uint4(x[0], x[1], x[2], x[3]);
          }
        }
      };
      auto put_stats = [&]() {
        if (part && valid)
          reinterpret_cast<float2 *>(a.ws + kCutBytes)[it.part * kRows + row_of + r] = make_float2(m, l);
      };
      if (both || it.n == 1) {
        const float f = 1.f / l;
        if (live) {
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            float o[32];
            tmem_ld32(to + 32 * c, o);
            tmem_wait_ld();
            put(o, c, f);
          }
          put_stats();
        }
        tc_fence_before();
        return true;
      }
      // two chains of the same rows: the second one's sums come through shared memory, 64 columns at a
      // time, or all where 64 rows are enough, 16-byte words of a row XORed with the row
      const int across = it.rows <= 64 ? D / 32 : 2;
      const uint32_t at = sb + M::MERGE + r * across * 128;
      float mine = 1.f, other = 0.f, inv = 0.f;
#pragma unroll 1
      for (int c0 = 0; c0 < D / 32; c0 += across) {
        if (w == 1) {
          if (!wait(sb + M::MEMPTY, m_n + 1)) return false;
          ++m_n;
          if (live) {
            if (c0 == 0) stats[r] = make_float2(m, l);
#pragma unroll 1
            for (int c = 0; c < across; ++c) {
              float o[32];
              tmem_ld32(to + 32 * (c0 + c), o);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 8; ++i)
                st_shared4(at + (((c * 8 + i) ^ (r & 15)) << 4), o[4 * i], o[4 * i + 1], o[4 * i + 2],
                           o[4 * i + 3]);
            }
          }
          arrive(sb + M::MFULL);
        } else {
          if (!wait(sb + M::MFULL, m_n)) return false;
          ++m_n;
          if (live) {
            if (c0 == 0) {
              const float2 t = stats[r];
              const float top = fmaxf(m, t.x), base = top == -INFINITY ? 0.f : top;
              mine = ex2(m - base);
              other = ex2(t.x - base);
              l = l * mine + t.y * other;
              m = top;
              inv = 1.f / l;
              put_stats();
            }
#pragma unroll 1
            for (int c = 0; c < across; ++c) {
              float o[32];
              tmem_ld32(to + 32 * (c0 + c), o);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float4 x = ld_shared4(at + (((c * 8 + i) ^ (r & 15)) << 4));
                o[4 * i] = o[4 * i] * mine + x.x * other;
                o[4 * i + 1] = o[4 * i + 1] * mine + x.y * other;
                o[4 * i + 2] = o[4 * i + 2] * mine + x.z * other;
                o[4 * i + 3] = o[4 * i + 3] * mine + x.w * other;
              }
              put(o, c0 + c, inv);
            }
          }
          arrive(sb + M::MEMPTY);
        }
      }
      tc_fence_before();
      return true;
    };
    auto run = [&]() {
      const Item *at, *next;
      if (!next_item(at)) return;
      if (has_q(*at)) {
        if (!fetch_q(*at)) return;
        give_q();
      }
      for (; at->rows >= 0; at = next) {
        const Item &it = *at;
        const bool both = it.rows > 128;
        const int steps = both ? it.n : (it.n + 1 - w) >> 1;
        const int row_of = both ? w * 128 : 0;  // of the tile, in the item
        const bool live = row_of + quad * 32 < it.rows, valid = row_of + r < it.rows;
        const int row = it.row0 + row_of + r, tok = row / a.G;
        // the positions that the row sees: [see0, see1)
        const int see1 = it.before + tok + 1, see0 = a.window ? max(see1 - a.window, 0) : 0;
        float m = -INFINITY, l = 0.f;  // log2
        for (int j = 0; j < steps; ++j) {
          const uint32_t place = M::place(turn, 2 * j + w), ts = tmem + place * 128 + lanes;
          if (!wait(sb + M::SFULL + 16 * w + 8 * turn_of(s_n), phase_of(s_n))) return;
          ++s_n;
          // With two places, these scores came behind this warpgroup's last sum.  With three, behind the one before
          // it, which is waited for here so that each barrier of the sums is seen in all of its phases.
          auto summed = [&](uint32_t k) { return wait(sb + M::ODONE + 16 * w + 8 * turn_of(k), phase_of(k)); };
          if (M::kScores > 2 && s_n > 2 && !summed(s_n - 3)) return;
          if (live) {
            tc_fence_after();
            float s[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32(ts + 32 * c, s[c]);
            tmem_wait_ld();
            const int p0 = (it.lo + (both ? j : 2 * j + w)) * kTile;
            const int c1 = min(max(see1 - p0, 0), kTile), c0 = min(max(see0 - p0, 0), kTile);
            if (__any_sync(0xffffffffu, valid && (c0 > 0 || c1 < kTile))) {
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const uint32_t seen = ones_from(c0 - 32 * c) & ~ones_from(c1 - 32 * c);
#pragma unroll
                for (int i = 0; i < 32; ++i) s[c][i] = (seen >> i) & 1u ? s[c][i] : -INFINITY;
              }
            }
            float mx[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              mx[c] = s[c][0];
#pragma unroll
              for (int i = 1; i < 32; ++i) mx[c] = fmaxf(mx[c], s[c][i]);
            }
            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * a.scale2;
            const bool higher = valid && top > m + kKeep;  // (the first finite score is: m is -inf)
            if (__any_sync(0xffffffffu, higher)) {
              const float f = higher ? ex2(m - top) : 1.f;
              if (higher) m = top;
              l *= f;
              if (j > 0) {  // O of the tiles before: the next MMA waits for P
                if (M::kScores > 2) {
                  if (!summed(s_n - 2)) return;
                  tc_fence_after();
                }
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                  float o[32];
                  tmem_ld32(to + 32 * c, o);
                  tmem_wait_ld();
#pragma unroll
                  for (int i = 0; i < 32; ++i) o[i] *= f;
                  tmem_st32(to + 32 * c, o);
                }
              }
            }
            const float neg = m == -INFINITY ? 0.f : -m;  // (nothing seen yet: every weight is 2^-inf)
            const float2 scale = make_float2(a.scale2, a.scale2), shift = make_float2(neg, neg);
            float2 sum[2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float p[32];  // 64 weights as bf16
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const float *two = &s[2 * c + i / 16][2 * (i % 16)];
                float2 x = __ffma2_rn(make_float2(two[0], two[1]), scale, shift);
                x.x = ex2(x.x);
                x.y = ex2(x.y);
                sum[i & 1] = __fadd2_rn(sum[i & 1], x);
                p[i] = __uint_as_float(pack(x.x, x.y));
              }
              tmem_st32(ts + 32 * c, p);
            }
            l += sum[0].x + sum[0].y + (sum[1].x + sum[1].y);
            tmem_wait_st();
            tc_fence_before();
          }
          arrive(sb + M::PREADY + 8 * place);
        }
        turn += both ? 2 * it.n : it.n;
        // The next item's Q.  With 128 rows of its own the warpgroup has seen the last scores of this one;
        // else the other's may still be on their way, and are not when its last sum is there.  The second
        // tile's place takes sums below.
        if (!next_item(next)) return;
        const bool q = has_q(*next), q_later = q && !both && w == 1;
        if (q && both && !fetch_q(*next)) return;
        if (steps > 0) {
          if (!wait(sb + M::OFULL + 8 * w, o_n++)) return;
          tc_fence_after();
        }
        if (q && !q_later) {
          if (!both && !fetch_q(*next)) return;
          give_q();
        }
        if (steps > 0 && !results(it, m, l)) return;
        if (q_later) {
          if (!fetch_q(*next)) return;
          give_q();
        }
        arrive(sb + M::IEMPTY + 8 * static_cast<uint32_t>(at - items));
      }
    };
    run();
    asm volatile("cp.async.wait_all;" ::: "memory");  // (where a wait gave up)
  }
  if (gave_up && lane == 0) fail();
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of each item that was cut, o = sum 2^(m_p - m) o_p / sum 2^(m_p - m) l_p.  A lane takes a
// row and FOURS times four columns: what a warp reads lies in a row of memory.  Bound by latency, so the
// fewer rows an item has, the fewer columns a lane takes and the more parts are on their way at once: a
// sequence of a million keys in 152 parts.  An item of which a CTA gave up is left as it was.
constexpr int kJoinThreads = 512;
constexpr int kJoinWarps = kJoinThreads / 32;

template <int D, int FOURS, int kAtOnce>
__device__ void join_row(const AttnArgs &a, const Cut &cut, int r, int four) {
  const int cta = blockIdx.x, n = cut.last - cta + 1;  // parts: the first is 2 cta + 1, the others 2 c
  const float2 *stats = reinterpret_cast<const float2 *>(a.ws + kCutBytes) + r;
  const float4 *parts = reinterpret_cast<const float4 *>(a.ws + kCutBytes + kStatBytes) + four * kRows + r;
  float4 o[FOURS];
  float top = -INFINITY, l = 0.f;
#pragma unroll
  for (int c = 0; c < FOURS; ++c) o[c] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int p0 = 0; p0 < n; p0 += kAtOnce) {
    float2 s[kAtOnce];
    float4 v[kAtOnce][FOURS];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int p = min(p0 + i, n - 1);  // (behind the last one: the same again, without weight)
      const int64_t at = p ? 2 * (cta + p) : 2 * cta + 1;
      // (in this order, so that all are on their way before the first is used)
      ld_in_turn(s[i], stats + at * kRows);
#pragma unroll
      for (int c = 0; c < FOURS; ++c) ld_in_turn(v[i][c], parts + (at * (D / 4) + c) * kRows);
    }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i)
      if (p0 + i >= n) s[i] = make_float2(-INFINITY, 0.f);
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const float m = fmaxf(top, s[i].x), base = m == -INFINITY ? 0.f : m;
      const float mine = ex2(top - base), f = ex2(s[i].x - base);
      top = m;
      l = l * mine + s[i].y * f;
#pragma unroll
      for (int c = 0; c < FOURS; ++c) {
        o[c].x = o[c].x * mine + v[i][c].x * f, o[c].y = o[c].y * mine + v[i][c].y * f;
        o[c].z = o[c].z * mine + v[i][c].z * f, o[c].w = o[c].w * mine + v[i][c].w * f;
      }
    }
  }
  const float f = 1.f / l;
  const int row = cut.row0 + r, t = row / a.G, g = row - t * a.G;
  kda_bf16 *out = a.o + (static_cast<int64_t>(cut.token0) + t) * a.ldo +
                  (static_cast<int64_t>(cut.head) * a.G + g) * D + four * 4;
#pragma unroll
  for (int c = 0; c < FOURS; ++c)
    *reinterpret_cast<uint2 *>(out + 4 * c) =
        make_uint2(pack(o[c].x * f, o[c].y * f), pack(o[c].z * f, o[c].w * f));
}

// Block (cta, y): half y % 2 of the columns of every other 32 rows, from rows 32 (y / 2) on.
template <int D>
__global__ void __launch_bounds__(kJoinThreads, 1) attn_join_kernel(const AttnArgs a) {
  grid_dependency_wait();
  grid_launch_dependents();  // (the next call's start, which waits for this kernel's end)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Cut cut = reinterpret_cast<const Cut *>(a.ws)[blockIdx.x];
  constexpr int kHalf = D / 8;  // columns in fours
  int failed[(kCtas + 31) / 32];  // of all CTAs from this one on, on their way with the cut
#pragma unroll
  for (int i = 0; i < (kCtas + 31) / 32; ++i)
    failed[i] = reinterpret_cast<const int *>(a.ws)[kFailed + min(static_cast<int>(blockIdx.x) + 32 * i + lane, kCtas - 1)];
  const int half = blockIdx.y & 1, first = blockIdx.y >> 1, lots = ((cut.rows + 31) / 32 - first + 1) / 2;
  if (lots <= 0) return;
  int some = 0;
#pragma unroll
  for (int i = 0; i < (kCtas + 31) / 32; ++i)
    if (static_cast<int>(blockIdx.x) + 32 * i + lane <= cut.last) some |= failed[i];
  if (__any_sync(0xffffffffu, some)) return;
  const int each = lots == 1 ? kJoinWarps : lots == 2 ? kJoinWarps / 2 : kJoinWarps / 4;  // warps of 32 rows
  const int fours = kHalf > each ? kHalf / each : 1, lot = warp / each, four = (warp - lot * each) * fours;
  const int r = (first + 2 * lot) * 32 + lane;
  if (r >= cut.rows || four >= kHalf) return;
  const int at = half * kHalf + four;
  if (fours == 1 && cut.last - static_cast<int>(blockIdx.x) >= 4) join_row<D, 1, 16>(a, cut, r, at);
  else if (fours == 1) join_row<D, 1, 4>(a, cut, r, at);
  else if (fours == 2) join_row<D, 2, 4>(a, cut, r, at);
  else if constexpr (kHalf >= kJoinWarps) join_row<D, 4, 2>(a, cut, r, at);
}

template <int D>
cudaError_t run(const AttnArgs &a, const kda_bf16 *cache, cudaStream_t st) {
  const tcx::EncodeTiledFn encode = tcx::tensor_map_encoder();
  if (!encode) return cudaErrorInvalidValue;
  CUtensorMap map;
  memset(&map, 0, sizeof(map));
  const int page = 1 << a.seqs.page_shift;
  const cuuint64_t dims[3] = {D, static_cast<cuuint64_t>(page),
                              static_cast<cuuint64_t>(a.seqs.n_pages) * 2 * a.H};
  const cuuint64_t strides[2] = {2 * D, static_cast<cuuint64_t>(2) * D * page};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(page), 1};
  const cuuint32_t step[3] = {1, 1, 1};
  if (encode(&map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<kda_bf16 *>(cache), dims, strides, box, step,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  const auto kernel = attn_kernel<D>;
  if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D>::BYTES))
    return e;
  if (cudaError_t e = launch_pdl(kernel, dim3(kCtas), dim3(kThreads), Smem<D>::BYTES, st, map, a)) return e;
  if (!a.ws) return cudaSuccess;
  // (of runs of one length the host knows how many rows an item has at most)
  const int64_t rows = a.runs.cu ? kRows : a.runs.fixed_len * a.G;
  return launch_pdl(attn_join_kernel<D>, dim3(kCtas, rows > 32 ? 4 : 2), dim3(kJoinThreads), 0, st, a);
}

}  // namespace

size_t attn_workspace(int D) { return ws_bytes(D); }

cudaError_t attn_launch(const AttnCall &c, int D, cudaStream_t st) {
  AttnArgs a{c.q, c.ldq, c.o, c.ldo, c.runs, c.seqs, c.H, c.G, c.window,
             c.scale * 1.44269504088896340736f, static_cast<uint8_t *>(c.workspace), c.status, c.test_stall};
  return D == 64 ? run<64>(a, c.cache, st) : run<128>(a, c.cache, st);
}

}  // namespace kda

// Selective state space scan over packed prompts, in chunks of 128 tokens on the tensor cores.
//
// With l = the cumulative log decay inside a chunk (l_t includes token t) and S the state in front
// of it, per head:
//   o_t = e^{l_t} C_t S  +  sum_{s <= t} (C_t . B_s) e^{l_t - l_s} dt_s x_s  +  D x_t   (then the gate)
//   S  <- e^{l_end} S  +  sum_s B_s (e^{l_end - l_s} dt_s x_s)^T
//
// One CTA carries 128 state columns (two heads of 64 that share their B and C, or one head of 128)
// through the chunks of one segment of a sequence.  All products are tcgen05 MMAs of 128 rows:
//   G   [token x token]  = C B^T                       operands as they came by TMA
//   C S [token x column]
//   Y   [token x column] = M X                         M = G * e^{l_t - l_s} dt_s, causal, from TMEM;
//                                                      then e^{l_t} (C S) and D x are added
//   dS^T[column x n]     = X'^T B                      X' = e^{l_end - l_s} dt_s x_s
//
// Roundings.  x, B and C are bf16 and enter exactly.  X' is split into three bf16 planes that hold
// all 24 bits of its fp32 value, and the state itself stays in fp32 registers (S^T: a thread has one
// column and half of n), so S and S_final carry fp32 accuracy.  For the output, S enters as two
// planes (16 bits) and M as one (8 bits): the in-chunk weights are rounded once to the type of the
// result, which makes its error 1.1 times that of its own rounding (1.85e-3 against 1.66e-3 in the 2-norm).
// M in two planes leaves 1.66e-3, but its second plane has no columns of TMEM to itself: in those of C S, M
// can only be made once C S is there, which took 529 us where this takes 444 and 757 where this takes 720.
//
// Log decays are summed in blocks of 32 tokens from both ends (prefix for what is read at t, suffix
// for what is kept of s), so that an exponent is the difference of two sums inside a block alone.  There
// a token's log2 decay counts as -160 where it is below (its decay is 0 in fp32 either way), so that a
// token that forgets everything leaves the decays behind it as they are: its -160 in both sums costs them
// a few 2^-17, where a step of 1e5 would have cost them a third and an infinite sum made NaN of them.  A
// block pair (t-block > s-block) takes its decay as the product of e^{l_t - l_end(s-block)} and
// e^{l_end(s-block) - l_s}, both at most 1: one exponential per thread and block instead of 32.
//
// Long sequences are cut into segments that run side by side: a first pass takes the same steps for
// the state alone, from zero, over every segment but a sequence's last, and leaves N and the decay
// a of the whole segment; the second pass starts each segment from a_{j-1} (... (a_0 S0 + N_0) ...)
// + N_{j-1}.
//
// Roles, each at its own pace and with its own registers, joined by mbarriers:
//   state    (8 warps)  X', 32 tokens at a time; the state and its planes for the next chunk
//   token    (8 warps)  M; e^{l_t} C S + D x added to M X
//   output   (8 warps)  gate and store
//   one warp each       TMA loads; G, C S and M X; dS; the decays of the chunks ahead, and
//                       the rows behind a sequence's end cleared, so that nothing of the next
//                       sequence is multiplied, not even by zero
// X has two buffers, C and B have one.  M takes the columns of its G, 16 tokens at a time.  C S and M X
// have a place of their own in TMEM, so that the next chunk's C S need not wait for the result's warps
// (added up in one place, with G in two, 527 us where this took 487).  The gate and the result
// pass through the chunk's X tile once nothing reads it any more.  In the first pass the token warps
// build X' too, and the output warps keep the state.
//
// What bounds it (32768 packed tokens x 64 heads of 64, N = 128, gate: 444 us, of which the first pass
// 108; 131072 tokens x 16 heads of 128: 720 us, of which 196).  A chunk of 128 tokens x 128 columns takes
// 11,000 cycles in the second pass (9,000 without the gate) and 5,000 in the first.  Its products would
// take 3,600 at the tensor cores' rate, its tiles 1,200 at the memory's.  The element-wise work decides,
// each warp waiting for its own results (shared memory, TMEM, exponentials) most of the time: by the
// clock the state's warps are at work for 80 % of a chunk, the result's for 75, the token's for 60, the
// rest being the way from one role to the next.  In the first pass no part stands out: without the
// products 15 us less, without the second and third plane 30, without the state's sum 10.  So the roles
// run side by side instead of one after another (one group of 16 warps that did all of it in turn took
// 667 us when this form took 655), the loops are rolled where they can be (the code of the roles shares
// the instruction caches: with 206 KB of it a quarter of all stalls were for instructions) and a wait is
// a few instructions.
#include <string.h>

#include "kda_pdl.cuh"
#include "kda_serving.cuh"
#include "kda_tc_common.cuh"

namespace kda {

namespace {

using namespace tcx;

constexpr int kQ = 128;          // tokens of a chunk
// warps of the roles: whole warpgroups, since a warp reaches the 32 TMEM lanes of its number mod 4
constexpr int kStateWarps = 8, kTokenWarps = 8, kOutWarps = 8;
constexpr int kTokenWarp = kStateWarps, kOutWarp = kTokenWarp + kTokenWarps;
// (the token warps of the last 32 tokens have the most to do, and the loads the least: they share a
// scheduler, and so do the first 32 tokens and the decays)
constexpr int kDecayWarp = kOutWarp + kOutWarps, kTokenMma = kDecayWarp + 1, kStateMma = kDecayWarp + 2,
              kLoadWarp = kDecayWarp + 3;
constexpr int kOthers = 4;
constexpr int kThreads = 32 * (kDecayWarp + kOthers);
// registers a thread: 72 at launch, then in the second pass
constexpr int kLaunchRegs = 72, kStateRegs = 88, kTokenRegs = 64, kOutRegs = 72, kOtherRegs = 56;
static_assert(32 * (kStateWarps * kStateRegs + kTokenWarps * kTokenRegs + kOutWarps * kOutRegs +
                    kOthers * kOtherRegs) <= kThreads * kLaunchRegs,
              "a warpgroup would wait for registers that the block does not have");

// shared memory: tiles of [128 rows][2 regions of 64 columns], 128-byte swizzle
constexpr uint32_t TILE = 32 * KiB;
constexpr uint32_t SM_X = 0;                // X, two chunks
constexpr uint32_t SM_B = 2 * TILE;         // (first pass: two chunks)
constexpr uint32_t SM_C = 3 * TILE;
constexpr uint32_t SM_XP = 4 * TILE;        // X': 32 tokens (first pass: three of them)
constexpr uint32_t SM_SP = SM_XP + 24 * KiB;  // S^T: two planes of [128 columns][N / 64 regions]
constexpr uint32_t SP_PLANE = 32 * KiB;
constexpr uint32_t SM_DEC = SM_SP + 2 * SP_PLANE;  // decays: [2 chunks][2 heads] (first pass: 2 more)
constexpr uint32_t SM_DEC2 = SM_XP + 72 * KiB;
constexpr uint32_t DEC_BYTES = 5 * 512 + 32;
constexpr uint32_t SM_BAR = SM_DEC + 4 * DEC_BYTES;
constexpr uint32_t SM_MISC = SM_BAR + 336;
constexpr uint32_t SM_BYTES = SM_MISC + 64;
static_assert(SM_BYTES <= 232448 && SM_DEC2 + 4 * DEC_BYTES <= SM_DEC, "shared memory budget");

// X' of a round: [3 planes][2 regions of 64 columns][TOKENS rows].  In the second pass rounds 0 and 3 of
// a chunk share a buffer; 1 and 2 take the place of the state's planes, which C S has read by then (with
// the one buffer for all four, a quarter of the state warps' time went into waiting for it).
template <bool STATE_ONLY>
struct Weighted {
  static constexpr int TOKENS = 32, BUFS = STATE_ONLY ? 3 : 4;
  static constexpr int ROUNDS = kQ / TOKENS;
  static constexpr uint32_t REGION = TOKENS * 128, PLANE = 2 * REGION, BYTES = 3 * PLANE;
  static_assert(STATE_ONLY ? SM_XP + 3 * BYTES <= SM_DEC2
                           : SM_XP + BYTES <= SM_SP && SM_SP + 2 * BYTES <= SM_DEC, "X' buffers");
  static __device__ __forceinline__ uint32_t place(int i) {
    const uint32_t k = i % BUFS;
    if (STATE_ONLY) return SM_XP + k * BYTES;
    return k == 1 || k == 2 ? SM_SP + (k - 1) * BYTES : SM_XP;
  }
};

// Decays of one (chunk, head): offsets in bytes
constexpr uint32_t DC_L = 0;         // log2 decay from the 32-token block's start, token included
constexpr uint32_t DC_DT = 512;      // dt
constexpr uint32_t DC_F = 1024;      // decay to the block's end, times dt
constexpr uint32_t DC_E = 1536;      // decay from the chunk's start
constexpr uint32_t DC_W = 2048;      // decay to the chunk's end, times dt
constexpr uint32_t DC_T = 2560;      // log2 decays of the four blocks; then the chunk's decay

// mbarriers.  Two of each kind: of chunk c the one of its parity, in phase c / 2.  F: a tile has come;
// D: an MMA is done; A: warps have arrived (AM: M is there; AF: the result; AS: the state's planes; AY: Y has
// been read, in the first pass dS; AO: the result has left X's tile).  FIN is for a wait that has given up.
enum Bar : int { FX, FC, FB, DG, DCS, DDS, DY, AM, AF, AS, AY, AO, FIN, NBAR };
// One for each X' buffer (second pass: for each round of a chunk): filled, and read.
constexpr uint32_t BAR_AXP = SM_BAR + 16 * NBAR, BAR_DXP = BAR_AXP + 32;
// One for each buffer of decays: written, and no longer needed.
constexpr uint32_t BAR_PREP = BAR_DXP + 32, BAR_DFREE = BAR_PREP + 32;
static_assert(BAR_DFREE + 32 <= SM_MISC, "barriers");

// TMEM columns: G (later M), C S, Y, dS (the first pass: two of dS, and S)
constexpr uint32_t TM_CS = 128, TM_Y = 256, TM_DS = 384, TM_S = 256;
// M of head h in the columns of its G: tokens [16 k, 16 k + 16) in 8 of the 16 that held their G
__device__ __forceinline__ constexpr uint32_t tm_m(int h, int k) { return 16 * k + 8 * h; }

constexpr uint32_t kPolls = 1u << 20;

constexpr float kLeastDecay = -160.f;  // log2: below the smallest fp32 value, 2^-149

struct ChunkArgs {
  SsmArgs a;
  int64_t seg_len;   // tokens of a segment, a multiple of 128
  int blocks;        // column blocks: of a group, times G
  float *part;       // [segments, H, N, P]: what the first pass leaves
  float *part_decay; // [segments, H]
  int parts;         // segments that `part` has room for (0: no sequence is cut)
};

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap *map, int x, int y,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem desc]^T: A is 128 rows of packed bf16 pairs, one column for two k.
__device__ __forceinline__ void mma_f16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]),
      "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
      : "memory");
}

__device__ __forceinline__ bool elect() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one != 0;
}

template <int REGS, bool MORE, bool ON>
__device__ __forceinline__ void set_registers() {
  if constexpr (!ON)
    return;
  else if constexpr (MORE)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS));
  else
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS));
}

// The upper halves of two fp32 values: two truncated bf16.
__device__ __forceinline__ uint32_t upper(float lo, float hi) {
  return __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x7632);
}
__device__ __forceinline__ float truncated(float x) {
  return __uint_as_float(__float_as_uint(x) & 0xffff0000u);
}

struct Segment {
  int seq, index;    // sequence, and the segment's number in it
  int id0;           // id of the sequence's first segment (of the first ones, if it has several)
  int begin, len;    // tokens
  int last, bad;
};

// Segment `id` of the batch.  The segments in front of a sequence's last one are all seg_len long; ids
// [0, parts) are theirs, sequence after sequence (as many as the tokens have room for: the spare ones are
// none), and the last ones, one for each sequence, come behind.  So the full ones start first, and the
// shorter ones fill the end.  Called by a whole warp.  A segment in front is found by a walk over the
// sequences, 128 at a time; a last one is its sequence's number, and only one that has others in front sums
// up where they are.  (With the last ones behind the used ids alone every one of them took the walk:
// 32768 prompts of one token x 8 heads 191 ms, where this takes 8.3.)
__device__ __forceinline__ bool find_segment(const Runs &r, int64_t seg_len, int parts, int id,
                                             Segment &g) {
  const int lane = threadIdx.x & 31;
  auto front = [&](int s) -> int {  // segments in front of the last one
    int64_t b, n, u;
    if (s >= r.n) return 0;
    run_range(r, s, b, n, u);
    return n <= seg_len ? 0 : static_cast<int>((n - 1) / seg_len);
  };
  g.last = id >= parts;
  g.id0 = 0;
  if (g.last) {
    g.seq = id - parts;
    g.index = front(g.seq);
    if (g.index > 0) {  // where its others are: the sum over the sequences in front of it
      int sum = 0;
      for (int s = lane; s < g.seq; s += 32) {
        sum += front(s);
        sum = sum < parts ? sum : parts;  // (offsets that are not in order: no number to wrap around)
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      g.id0 = sum;
    }
  } else {
    int before = 0;
    g.seq = -1;
    for (int base = 0; base < r.n; base += 128) {
      int c[4], mine = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) mine += c[k] = front(base + 4 * lane + k);
      int x = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      const unsigned m = __ballot_sync(0xffffffffu, before + x > id);
      if (m) {
        const int l = __ffs(m) - 1;
        int s = base + 4 * lane, first = before + x - mine;
#pragma unroll
        for (int k = 0; k < 3; ++k)
          if (s == base + 4 * lane + k && first + c[k] <= id) {
            first += c[k];
            ++s;
          }
        g.seq = __shfl_sync(0xffffffffu, s, l);
        g.id0 = __shfl_sync(0xffffffffu, first, l);
        g.index = id - g.id0;
        break;
      }
      before += __shfl_sync(0xffffffffu, x, 31);
    }
    if (g.seq < 0) return false;
  }
  int64_t b, n, u;
  g.bad = !run_range(r, g.seq, b, n, u);
  g.begin = static_cast<int>(b + g.index * seg_len);
  g.len = static_cast<int>(g.last ? n - g.index * seg_len : seg_len);
  return true;
}

// STATE_ONLY: the first pass over the segments (no C, no output).
template <int N, int P, bool STATE_ONLY>
__global__ void __launch_bounds__(kThreads, 1)
ssm_chunk_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_b,
                 const __grid_constant__ CUtensorMap tm_c, const ChunkArgs p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  constexpr int HEADS = 128 / P;        // heads of a column block
  constexpr uint32_t BC_BYTES = 128 * N * 2;
  using XP = Weighted<STATE_ONLY>;
  constexpr int DECAY_WARPS = STATE_ONLY ? 2 : 1;  // (the first pass has no MMAs of Y)
  const SsmArgs &a = p.a;
  const uint32_t sb = smem_u32(smem);
  const Smem S{smem, sb};
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // The second pass may start on the SMs that the last segments of the first one leave idle; its state
  // warps wait for all of them.
  if (STATE_ONLY) grid_launch_dependents();
  if ((sb & 1023u) != 0) {  // the swizzled layouts need 1024-byte alignment
    if (tid == 0) atomicOr(a.status, KDA_ERR_UNSUPPORTED);
    return;
  }
  // One warp looks the segment up, the roles read of it what they need.
  const int id = blockIdx.x / p.blocks, block = blockIdx.x % p.blocks;
  Segment &seg = *reinterpret_cast<Segment *>(smem + SM_MISC + 16);
  if (warp == 0) {
    Segment found;
    if (!find_segment(a.runs, p.seg_len, p.parts, id, found)) {
      found.len = -1;
    } else {
      // offsets that are not in order can make more segments than the tokens have room for
      if (found.last && found.id0 + found.index > p.parts) found.bad = 1;
      if (found.bad && block == 0 && lane == 0) atomicOr(a.status, KDA_ERR_SHAPE);
      if (found.bad) found.len = -1;
    }
    if (lane == 0) seg = found;
  }
  __syncthreads();
  if (seg.len < 0) {
    grid_dependency_wait();  // (this grid does not end before the first pass does)
    return;
  }
  const int per_group = a.H / a.G, blocks_per_group = p.blocks / a.G;
  const int g = block / blocks_per_group;
  const int first_in_group = (block % blocks_per_group) * HEADS;
  const int h0 = g * per_group + first_in_group;
  const int heads = per_group - first_in_group < HEADS ? 1 : HEADS;
  const int n_chunks = (seg.len + kQ - 1) / kQ;

  auto bar = [&](int kind, int c) { return sb + SM_BAR + 16u * kind + 8u * (c & 1); };
  constexpr int DECS = STATE_ONLY ? 4 : 2;  // buffers of decays
  auto decays = [&](int c, int head) {
    const int k = c % DECS;
    return sb + (k < 2 ? SM_DEC : SM_DEC2) + ((k & 1) * 2 + head) * DEC_BYTES;
  };
  auto prepared = [&](int c) { return sb + BAR_PREP + 8u * (c % DECS); };
  auto dec_free = [&](int c) { return sb + BAR_DFREE + 8u * (c % DECS); };
  auto xp_full = [&](int i) { return sb + BAR_AXP + 8u * (i % XP::BUFS); };
  auto xp_read = [&](int i) { return sb + BAR_DXP + 8u * (i % XP::BUFS); };
  if (tid == 0) {
    for (int k = 0; k < NBAR; ++k) {
      uint32_t count = 1;
      if (k == AM || k == AF) count = kTokenWarps;
      if (k == AS) count = kStateWarps;
      if (k == AY || k == AO) count = kOutWarps;
      mbar_init(bar(k, 0), count);
      mbar_init(bar(k, 1), count);
    }
    for (int k = 0; k < DECS; ++k) {
      mbar_init(prepared(k), HEADS);
      mbar_init(dec_free(k), kStateWarps + kTokenWarps + (STATE_ONLY ? kOutWarps : 0));
    }
    for (int k = 0; k < XP::BUFS; ++k) {
      mbar_init(xp_full(k), kStateWarps);
      mbar_init(xp_read(k), 1);
    }
    fence_mbar_init();
  }
  if (warp == kStateMma) {
    tmem_alloc(sb + SM_MISC, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + SM_MISC);

  // Every wait is bounded.  A role whose wait gives up leaves its loop, so those that wait for it give
  // up too; the loop around a wait stays short, for the roles' code shares the instruction cache.
  bool gave_up = false;
  auto wait = [&](uint32_t b, uint32_t phase) -> bool {
    uint32_t left = kPolls;
#pragma unroll 1
    while (!mbar_try_wait(b, phase & 1u))
      if (--left == 0) {
        gave_up = true;
        return false;
      }
    return true;
  };
  auto wait_c = [&](int kind, int c) { return wait(bar(kind, c), static_cast<uint32_t>(c) >> 1); };
  // the same for a whole warp, which goes on or stops as one
  auto warp_wait = [&](uint32_t b, uint32_t phase) {
    return __all_sync(0xffffffffu, wait(b, phase)) != 0;
  };
  auto warp_wait_c = [&](int kind, int c) {
    return warp_wait(bar(kind, c), static_cast<uint32_t>(c) >> 1);
  };

  // tiles of chunk c
  auto tile_x = [&](int c) { return sb + SM_X + (c & 1) * TILE; };
  auto tile_b = [&](int c) { return sb + SM_B + (STATE_ONLY ? (c & 1) * TILE : 0u); };
  const uint32_t tile_c = sb + SM_C;

  auto arrive = [&](uint32_t b) {
    __syncwarp();
    if (lane == 0) mbar_arrive(b);
  };

  if (warp >= kDecayWarp) {
    set_registers<kOtherRegs, false, !STATE_ONLY>();
    if (warp == kLoadWarp) {
      if (lane == 0) {
        bool ok = true;
        int c = 0;
        for (; c < n_chunks; ++c) {
          const int t = seg.begin + c * kQ;
          auto load_bc = [&](const CUtensorMap *map, uint32_t to, uint32_t b) {
            mbar_expect_tx(b, BC_BYTES);
            for (int r = 0; r < N / 64; ++r)
              tma_load_2d(to + r * REG128, map, g * N + 64 * r, t, b);
          };
          if (c >= 2 && !(ok = wait_c(STATE_ONLY ? DDS : AO, c - 2))) break;
          mbar_expect_tx(bar(FX, c), TILE);
          for (int r = 0; r < 2; ++r)
            tma_load_2d(tile_x(c) + r * REG128, &tm_x, h0 * P + 64 * r, t, bar(FX, c));
          if (!STATE_ONLY && c > 0 && !(ok = wait_c(DDS, c - 1) && wait_c(DG, c - 1))) break;
          load_bc(&tm_b, tile_b(c), bar(FB, c));
          if constexpr (!STATE_ONLY) {
            if (c > 0 && !(ok = wait_c(DCS, c - 1))) break;
            load_bc(&tm_c, tile_c, bar(FC, c));
          }
        }
        if (!ok) {  // what is in flight lands before the shared memory goes
          for (int k = c > 1 ? c - 2 : 0; k <= c && k < n_chunks; ++k) {
            mbar_wait_bounded(bar(FX, k), (k >> 1) & 1, 1u << 16);
            mbar_wait_bounded(bar(FB, k), (k >> 1) & 1, 1u << 16);
            if (!STATE_ONLY) mbar_wait_bounded(bar(FC, k), (k >> 1) & 1, 1u << 16);
          }
        }
      }
    } else if (warp == kTokenMma && !STATE_ONLY) {
      // A whole warp goes through an MMA loop (so that addresses and descriptors stay in uniform
      // registers); one lane issues.
      constexpr uint32_t ID_G = idesc_mma(128, 128, kFmtBF16, kFmtBF16, 0, 0), ID_CS = ID_G;
      constexpr uint32_t ID_MX = idesc_mma(128, P, kFmtBF16, kFmtBF16, 0, 1);
      const uint64_t c_k = sw128_desc(tile_c, 16u, 1024u), s_k = sw128_desc(sb + SM_SP, 16u, 1024u);
      const bool one = elect();
      bool ok = true;
      for (int c = 0; c < n_chunks; ++c) {
        const uint64_t x_mn = sw128_desc(tile_x(c), REG128, 1024u);
        ok = warp_wait_c(FB, c) && warp_wait_c(FC, c) && (c == 0 || warp_wait_c(DY, c - 1));
        if (!ok) break;
        tc_fence_after();
        if (one) {
          const uint64_t b_k = sw128_desc(tile_b(c), 16u, 1024u);
#pragma unroll 1
          for (int r = 0; r < N / 64; ++r)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_f16(tmem, c_k + r * (REG128 >> 4) + 2 * k, b_k + r * (REG128 >> 4) + 2 * k, ID_G,
                      r + k > 0);
          mma_commit(bar(DG, c));
        }
        ok = warp_wait_c(AS, c) && (c == 0 || warp_wait_c(AF, c - 1));
        if (!ok) break;
        tc_fence_after();
        if (one) {
#pragma unroll 1
          for (int r = 0; r < 2 * (N / 64); ++r) {  // (plane, 64 of n); 16 of n in a step of 32 bytes
            const uint32_t at = (r % (N / 64)) * (REG128 >> 4);
            const uint64_t cd = c_k + at, sd = s_k + at + (r / (N / 64)) * (SP_PLANE >> 4);
#pragma unroll
            for (int k = 0; k < 4; ++k) mma_f16(tmem + TM_CS, cd + 2 * k, sd + 2 * k, ID_CS, r + k > 0);
          }
          mma_commit(bar(DCS, c));
        }
        ok = warp_wait_c(FX, c) && warp_wait_c(AM, c) && (c == 0 || warp_wait_c(AY, c - 1));
        if (!ok) break;
        tc_fence_after();
        if (one) {
#pragma unroll 1
          for (int r = 0; r < 2 * HEADS; ++r) {  // (head, 64 tokens); 16 tokens in a step
            const int h = r / 2, k0 = 4 * (r % 2);
            const uint32_t m = tmem + tm_m(h, k0);
            const uint64_t xd = x_mn + ((h * REG128 + k0 * 2048u) >> 4);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_f16_ta(tmem + TM_Y + 64 * h, m + tm_m(0, k), xd + 128 * k, ID_MX, k0 + k > 0);
          }
          mma_commit(bar(DY, c));
        }
      }
      if (!ok && one) {  // MMAs in flight finish before TMEM goes
        mma_commit(bar(FIN, 0));
        mbar_wait_bounded(bar(FIN, 0), 0, 1u << 16);
      }
    } else if (warp == kStateMma) {
      constexpr uint32_t ID_DS = idesc_mma(128, N, kFmtBF16, kFmtBF16, 1, 1);
      const bool one = elect();
      bool ok = true;
      for (int c = 0; c < n_chunks && ok; ++c) {
        ok = warp_wait_c(FB, c) && warp_wait(prepared(c), c / DECS);
        if constexpr (STATE_ONLY) {
          ok = ok && (c < 2 || warp_wait_c(AY, c - 2));
        }
        const uint64_t b_mn = sw128_desc(tile_b(c), REG128, 1024u);
        const uint32_t to = tmem + (STATE_ONLY ? 128u * (c & 1) : TM_DS);
#pragma unroll 1
        for (int r = 0; r < XP::ROUNDS && ok; ++r) {
          const int i = XP::ROUNDS * c + r;
          ok = warp_wait(xp_full(i), i / XP::BUFS);
          if (!ok) break;
          tc_fence_after();
          if (one) {
            const uint64_t xp =
                sw128_desc(sb + XP::place(i), XP::REGION, 1024u);
            constexpr int STEPS = XP::TOKENS / 16;
#pragma unroll
            for (int k = 0; k < 3 * STEPS; ++k)
              mma_f16(to, xp + (((k / STEPS) * XP::PLANE + (k % STEPS) * 2048u) >> 4),
                      b_mn + ((r * XP::TOKENS * 128u + (k % STEPS) * 2048u) >> 4), ID_DS, r + k > 0);
            mma_commit(xp_read(i));
            if (r == XP::ROUNDS - 1) mma_commit(bar(DDS, c));
          }
        }
      }
      if (!ok && one) {
        mma_commit(bar(FIN, 1));
        mbar_wait_bounded(bar(FIN, 1), 0, 1u << 16);
      }
    } else {
      // lane i has tokens 4 i .. 4 i + 3, eight lanes a block of 32.  One (chunk, head) after another; the
      // next one's steps are on their way (and widened only where they are used).
      uint32_t next[4];
      auto fetch = [&](int it) {
        const int at = it / HEADS * kQ + 4 * lane, left = seg.len - at;
        const kda_bf16 *from =
            a.dt + static_cast<int64_t>(seg.begin + at) * a.lddt + h0 + it % HEADS;
#pragma unroll
        for (int i = 0; i < 4; ++i, from += a.lddt) {
          next[i] = 0;
          if (it % HEADS < heads && i < left) next[i] = *from;
        }
      };
      const int first = warp == kDecayWarp ? 0 : 1;
      float A2s[HEADS], biases[HEADS];
#pragma unroll
      for (int h = 0; h < HEADS; ++h) {
        A2s[h] = h < heads ? a.A[h0 + h] * 1.44269504088896340736f : 0.f;
        biases[h] = h < heads && a.dt_bias ? a.dt_bias[h0 + h] : 0.f;
      }
      fetch(first);
#pragma unroll 1
      for (int it = first; it < n_chunks * HEADS; it += DECAY_WARPS) {
        const int c = it / HEADS, hh = it % HEADS;
        const int len = seg.len - c * kQ < kQ ? seg.len - c * kQ : kQ;
        uint32_t raw[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) raw[i] = next[i];
        fetch(it + DECAY_WARPS);
        if (c >= DECS && !warp_wait(dec_free(c), c / DECS - 1)) break;
        {
          const bool mine = hh < heads;
          const float A2 = hh ? A2s[HEADS - 1] : A2s[0];
          const float bias = hh ? biases[HEADS - 1] : biases[0];
          float dt[4], ld[4], pre[4], suf[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            dt[i] = mine && 4 * lane + i < len ? ssm_step(a, __uint_as_float(raw[i] << 16), bias) : 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            ld[i] = dt[i] * A2;
            ld[i] = ld[i] < kLeastDecay ? kLeastDecay : ld[i];  // (NaN stays)
          }
          pre[0] = ld[0];
#pragma unroll
          for (int i = 1; i < 4; ++i) pre[i] = pre[i - 1] + ld[i];
          suf[3] = 0.f;
#pragma unroll
          for (int i = 2; i >= 0; --i) suf[i] = suf[i + 1] + ld[i + 1];
          const float four = suf[0] + ld[0];
          float up = four, down = four;
#pragma unroll
          for (int o = 1; o < 8; o <<= 1) {
            const float u = __shfl_up_sync(0xffffffffu, up, o, 8);
            const float d = __shfl_down_sync(0xffffffffu, down, o, 8);
            if ((lane & 7) >= o) up += u;
            if ((lane & 7) + o < 8) down += d;
          }
          const float whole = __shfl_sync(0xffffffffu, up, 7, 8);
          // sums of the lanes before and after, without this one's
          float up_ex = __shfl_up_sync(0xffffffffu, up, 1, 8);
          float down_ex = __shfl_down_sync(0xffffffffu, down, 1, 8);
          if ((lane & 7) == 0) up_ex = 0.f;
          if ((lane & 7) == 7) down_ex = 0.f;
          float blocks[4], front = 0.f, behind = 0.f;
#pragma unroll
          for (int b = 0; b < 4; ++b) blocks[b] = __shfl_sync(0xffffffffu, whole, 8 * b);
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            if (b < lane / 8) front += blocks[b];
            if (3 - b > lane / 8) behind += blocks[3 - b];
          }
          const uint32_t at = decays(c, hh);
          float4 v;
          float *vp = &v.x;
          auto put = [&](uint32_t off) {
            *reinterpret_cast<float4 *>(S.ptr(at + off + 16 * lane)) = v;
          };
#pragma unroll
          for (int i = 0; i < 4; ++i) vp[i] = up_ex + pre[i];
          put(DC_L);
#pragma unroll
          for (int i = 0; i < 4; ++i) vp[i] = dt[i];
          put(DC_DT);
#pragma unroll
          for (int i = 0; i < 4; ++i) vp[i] = ex2(suf[i] + down_ex) * dt[i];
          put(DC_F);
#pragma unroll
          for (int i = 0; i < 4; ++i) vp[i] = ex2(front + (up_ex + pre[i]));
          put(DC_E);
#pragma unroll
          for (int i = 0; i < 4; ++i) vp[i] = ex2(behind + (suf[i] + down_ex)) * dt[i];
          put(DC_W);
#pragma unroll
          for (int b = 0; b < 4; ++b)
            if (lane == b) S.f32(at + DC_T + 4 * b) = blocks[b];
          if (lane == 4)
            S.f32(at + DC_T + 16) = exp2f((blocks[0] + blocks[1]) + (blocks[2] + blocks[3]));
        }
        // Clear what lies behind the sequence's end (the first pass has whole chunks only).  The tiles'
        // barriers are not a phase behind: their last users have freed this buffer of decays.
        if (!STATE_ONLY && len < kQ && hh == 0) {
          if (!warp_wait_c(FX, c) || !warp_wait_c(FB, c)) break;
          for (int i = lane; i < (kQ - len) * 8; i += 32) {
            const uint32_t off = static_cast<uint32_t>(len) * 128u + 16u * i;
            for (int r = 0; r < 2; ++r)
              S.u128(tile_x(c) + r * REG128 + off) = make_uint4(0, 0, 0, 0);
            for (int r = 0; r < N / 64; ++r)
              S.u128(tile_b(c) + r * REG128 + off) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async();
        }
        arrive(prepared(c));
      }
    }
    __syncwarp();
  } else if (warp >= kOutWarp) {
    set_registers<kOutRegs, false, !STATE_ONLY>();
    const int quad = warp & 3, half = (warp - kOutWarp) >> 2;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    if constexpr (!STATE_ONLY) {
      // columns [64 half, 64 half + 64): 32 rows of 128 bytes a warp.  In global memory 4 rows in one
      // instruction, in TMEM a row for each lane.
      const bool in = HEADS == 1 || half < heads;
      const int64_t cols = static_cast<int64_t>(h0) * P + 64 * half;
      const int r0 = lane >> 3, piece = lane & 7;
      const bool gate = a.z && in;
      // row r0 of this warp's 32, in the gate and in the result
      const int64_t row0 = seg.begin + quad * 32 + r0;
      const kda_bf16 *gate_at = a.z + row0 * a.ldz + cols + 8 * piece;
      kda_bf16 *out_at = a.o + row0 * a.ldo + cols + 8 * piece;
#pragma unroll 1
      for (int c = 0; c < n_chunks; ++c, gate_at += kQ * a.ldz, out_at += kQ * a.ldo) {
        const int left = seg.len - c * kQ - quad * 32;  // rows of this warp, if under 32
        const uint32_t stage = tile_x(c) + half * REG128 + quad * 4096u;
        uint4 z[8];
        if (gate) {
          const kda_bf16 *from = gate_at;
#pragma unroll
          for (int i = 0; i < 8; ++i, from += 4 * a.ldz)
            if (4 * i + r0 < left) z[i] = *reinterpret_cast<const uint4 *>(from);
          if (lane + kQ < left)  // the next chunk's lines
            asm volatile("prefetch.global.L2 [%0];" ::"l"(
                a.z + static_cast<int64_t>(seg.begin + (c + 1) * kQ + quad * 32 + lane) * a.ldz + cols));
        }
        // X is read by the state's warps until dS is done, by the others until Y is
        if (!warp_wait_c(DDS, c) || !warp_wait_c(AF, c)) break;
        tc_fence_after();
        if (gate) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = 4 * i + r0;
            S.u128(stage + r * 128u + ((piece ^ (r & 7)) << 4)) = z[i];
          }
          __syncwarp();
        }
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {
          float y[16];
          tmem_ld16(lanes + TM_Y + 64 * half + 16 * k, y);
          tmem_wait_ld();
          if (k == 3) {
            tc_fence_before();
            arrive(bar(AY, c));
          }
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t at = stage + lane * 128u + (((2 * k + j) ^ (lane & 7)) << 4);
            if (gate) {
              const uint4 raw = S.u128(at);
              const uint32_t in4[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const int i = 8 * j + 2 * q;
                const float2 f = unpack_bf16x2(in4[q]);
                const float2 l = __fmul2_rn(f, make_float2(-1.44269504f, -1.44269504f));
                const float2 d = __fadd2_rn(make_float2(ex2(l.x), ex2(l.y)), make_float2(1.f, 1.f));
                // (z times its sigmoid first: y times a gate near the type's lowest value is infinite)
                const float2 v = __fmul2_rn(make_float2(y[i], y[i + 1]),
                                            __fmul2_rn(f, make_float2(rcp(d.x), rcp(d.y))));
                y[i] = v.x;
                y[i + 1] = v.y;
              }
            }
            const int i = 8 * j;
            S.u128(at) =
                make_uint4(pack_bf16x2(y[i], y[i + 1]), pack_bf16x2(y[i + 2], y[i + 3]),
                           pack_bf16x2(y[i + 4], y[i + 5]), pack_bf16x2(y[i + 6], y[i + 7]));
          }
        }
        __syncwarp();
        if (in) {
          kda_bf16 *to = out_at;
#pragma unroll
          for (int i = 0; i < 8; ++i, to += 4 * a.ldo) {
            const int r = 4 * i + r0;
            if (r < left)
              *reinterpret_cast<uint4 *>(to) = S.u128(stage + r * 128u + ((piece ^ (r & 7)) << 4));
          }
        }
        fence_proxy_async();  // the tile goes back to the TMA
        arrive(bar(AO, c));
      }
    } else {
      // the state of the first pass: S^T in TMEM, a column for each lane and half of n a warp
      const int row = quad * 32 + lane, n0 = half * (N / 2);
      const int hcol = HEADS == 2 ? quad >> 1 : 0;
      const size_t at0 = (static_cast<size_t>(id) * a.H + h0 + hcol) * N * P +
                         static_cast<size_t>(n0) * P + row % P;
      float decay = 1.f;
      for (int c = 0; c < n_chunks; ++c) {
        if (!warp_wait(prepared(c), c / DECS)) break;
        const float keep = S.f32(decays(c, hcol) + DC_T + 16);
        decay *= keep;
        if (!warp_wait_c(DDS, c)) break;
        tc_fence_after();
#pragma unroll 1
        for (int k = 0; k < N / 2; k += 16) {
          float s[16], v[16];
          if (c > 0) tmem_ld16(lanes + TM_S + n0 + k, s);
          tmem_ld16(lanes + 128 * (c & 1) + n0 + k, v);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) s[i] = c > 0 ? fmaf(keep, s[i], v[i]) : v[i];
          if (c + 1 < n_chunks) {
            tmem_st16(lanes + TM_S + n0 + k, s);
          } else if (hcol < heads) {
#pragma unroll
            for (int i = 0; i < 16; ++i) p.part[at0 + static_cast<size_t>(k + i) * P] = s[i];
          }
        }
        tmem_wait_st();
        tc_fence_before();
        arrive(bar(AY, c));
        if (lane == 0) mbar_arrive(dec_free(c));
      }
      if (n0 == 0 && row % P == 0 && hcol < heads)
        p.part_decay[static_cast<size_t>(id) * a.H + h0 + hcol] = decay;
    }
  } else if (warp >= kTokenWarp && !STATE_ONLY) {
    set_registers<kTokenRegs, false, !STATE_ONLY>();
      const int half = (warp - kTokenWarp) >> 2;  // of the columns of Y; of the blocks of M
      const int quad = warp & 3, row = quad * 32 + lane;  // token of G, M and Y
      const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16);
      const int hout = HEADS == 2 ? half : 0;
      const float skip = a.D && hout < heads ? a.D[h0 + hout] : 0.f;
      for (int c = 0; c < n_chunks; ++c) {
        const uint32_t dec = decays(c, 0);
        if (!warp_wait(prepared(c), c / DECS) || !warp_wait_c(FX, c) || !warp_wait_c(DG, c)) break;
        tc_fence_after();
        // M, 32 tokens s at a time, of which a warp takes 16
#pragma unroll 1
        for (int b = 0; b < 4; ++b) {
          const int s0 = 32 * b + 16 * half;
          float m[16];
          if (b > quad) {
#pragma unroll
            for (int i = 0; i < 16; ++i) m[i] = 0.f;
            tmem_st16(lanes + s0, m);
            continue;
          }
          tmem_ld16(lanes + s0, m);
          tmem_wait_ld();
#pragma unroll
          for (int h = 0; h < HEADS; ++h) {
            const uint32_t d = dec + h * DEC_BYTES;
            const float lt = S.f32(d + DC_L + 4 * row);
            uint32_t words[8];
            if (b < quad) {
              float l = lt;  // from the block's end to t
              for (int q = b + 1; q < quad; ++q) l += S.f32(d + DC_T + 4 * q);
              const float e = ex2(l);
              const float2 e2 = make_float2(e, e);
#pragma unroll
              for (int i = 0; i < 16; i += 4) {
                const float4 f = *reinterpret_cast<const float4 *>(S.ptr(d + DC_F + 4 * (s0 + i)));
                const float2 u = __fmul2_rn(make_float2(m[i], m[i + 1]),
                                            __fmul2_rn(make_float2(f.x, f.y), e2));
                const float2 v = __fmul2_rn(make_float2(m[i + 2], m[i + 3]),
                                            __fmul2_rn(make_float2(f.z, f.w), e2));
                words[i / 2] = pack_bf16x2(u.x, u.y);
                words[i / 2 + 1] = pack_bf16x2(v.x, v.y);
              }
            } else {
              const int t = lane - 16 * half;
#pragma unroll
              for (int i = 0; i < 16; i += 4) {
                const float4 l = *reinterpret_cast<const float4 *>(S.ptr(d + DC_L + 4 * (s0 + i)));
                const float4 w = *reinterpret_cast<const float4 *>(S.ptr(d + DC_DT + 4 * (s0 + i)));
                const float2 d0 = __fadd2_rn(make_float2(lt, lt), make_float2(-l.x, -l.y));
                const float2 d1 = __fadd2_rn(make_float2(lt, lt), make_float2(-l.z, -l.w));
                const float2 u = __fmul2_rn(make_float2(m[i], m[i + 1]),
                                            __fmul2_rn(make_float2(ex2(d0.x), ex2(d0.y)),
                                                       make_float2(w.x, w.y)));
                const float2 v = __fmul2_rn(make_float2(m[i + 2], m[i + 3]),
                                            __fmul2_rn(make_float2(ex2(d1.x), ex2(d1.y)),
                                                       make_float2(w.z, w.w)));
                // (a choice, not a product: what lies in the future may be infinite)
                words[i / 2] = pack_bf16x2(i <= t ? u.x : 0.f, i + 1 <= t ? u.y : 0.f);
                words[i / 2 + 1] = pack_bf16x2(i + 2 <= t ? v.x : 0.f, i + 3 <= t ? v.y : 0.f);
              }
            }
            tmem_st8(lanes + s0 + 8 * h, words);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        arrive(bar(AM, c));
        if (!warp_wait_c(DCS, c) || !warp_wait_c(DY, c)) break;
        tc_fence_after();
        // C S, scaled to each token, and D x join M X
        const float e = S.f32(dec + hout * DEC_BYTES + DC_E + 4 * row);
        const float2 e2 = make_float2(e, e), skip2 = make_float2(skip, skip);
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {
          float y[16], cs[16];
          tmem_ld16(lanes + TM_CS + 64 * half + 16 * k, cs);
          tmem_ld16(lanes + TM_Y + 64 * half + 16 * k, y);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint4 raw = S.u128(tile_x(c) + half * REG128 + row * 128u +
                                     (static_cast<uint32_t>((2 * k + j) ^ (row & 7)) << 4));
            const uint32_t in[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int i = 8 * j + 2 * q;
              const float2 f = __ffma2_rn(e2, make_float2(cs[i], cs[i + 1]),
                                          __ffma2_rn(skip2, unpack_bf16x2(in[q]), make_float2(y[i], y[i + 1])));
              y[i] = f.x;
              y[i + 1] = f.y;
            }
          }
          tmem_st16(lanes + TM_Y + 64 * half + 16 * k, y);
        }
        tmem_wait_st();
        tc_fence_before();
        arrive(bar(AF, c));
        if (lane == 0) mbar_arrive(dec_free(c));
      }
  } else {
    // the state's warps; in the first pass the token's beside them, every other round each
    set_registers<kStateRegs, true, !STATE_ONLY>();
    // X' of the tokens of round r of chunk c: a thread takes 8 columns of a row in both regions
    auto put_weighted = [&](int c, int r) -> bool {
      const int i = XP::ROUNDS * c + r;
      if constexpr (STATE_ONLY) {
        if (i >= XP::BUFS && !warp_wait(xp_read(i), i / XP::BUFS - 1)) return false;
      } else {
        if (r == 1 && !warp_wait_c(DCS, c)) return false;
        if (r == 3 && !warp_wait(xp_read(0), c)) return false;
      }
      const int j = tid & 7, row = (tid >> 3) % XP::TOKENS, tok = XP::TOKENS * r + row;
      const uint32_t flip = static_cast<uint32_t>(j ^ (row & 7)) << 4;
      const uint32_t dec = decays(c, 0) + DC_W + 4 * tok;
#pragma unroll
      for (int region = 0; region < 2; ++region) {
        const float w = S.f32(dec + (HEADS == 2 ? region : 0) * DEC_BYTES);
        const uint4 raw = S.u128(tile_x(c) + region * REG128 + tok * 128u + flip);
        const uint32_t in4[4] = {raw.x, raw.y, raw.z, raw.w};
        const float2 w2 = make_float2(w, w);
        uint32_t out[3][4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float2 f = __fmul2_rn(unpack_bf16x2(in4[e]), w2);
          out[0][e] = upper(f.x, f.y);
          f = __fadd2_rn(f, make_float2(-truncated(f.x), -truncated(f.y)));
          out[1][e] = upper(f.x, f.y);
          f = __fadd2_rn(f, make_float2(-truncated(f.x), -truncated(f.y)));
          out[2][e] = upper(f.x, f.y);
        }
        const uint32_t to = sb + XP::place(i) + region * XP::REGION + row * 128u + flip;
#pragma unroll
        for (int k = 0; k < 3; ++k)
          S.u128(to + k * XP::PLANE) = make_uint4(out[k][0], out[k][1], out[k][2], out[k][3]);
      }
      fence_proxy_async();
      arrive(xp_full(i));
      return true;
    };
    if constexpr (STATE_ONLY) {
      for (int c = 0; c < n_chunks; ++c) {
        if (!warp_wait(prepared(c), c / DECS) || !warp_wait_c(FX, c)) break;
        bool ok = true;
#pragma unroll 1
        for (int r = warp / kTokenWarp; r < XP::ROUNDS && ok; r += 2) ok = put_weighted(c, r);
        if (!ok) break;
        if (lane == 0) mbar_arrive(dec_free(c));
      }
    } else {
      constexpr int NT = N / 2;                      // state entries of a thread
      const int n0 = (warp >> 2) * NT, quad = warp & 3;
      const int row = quad * 32 + lane;              // column of the state: TMEM lane of dS^T
      const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16);
      const int hcol = HEADS == 2 ? quad >> 1 : 0;   // its head
      const bool in = hcol < heads;
      const size_t at0 =
          static_cast<size_t>(h0 + hcol) * N * P + static_cast<size_t>(n0) * P + row % P;
      const size_t state = static_cast<size_t>(a.H) * N * P;
      float s[NT];
#pragma unroll
      for (int i = 0; i < NT; ++i) s[i] = 0.f;
      grid_dependency_wait();
      if (in) {
        if (a.S_in) {
          const float *from = a.S_in + seg.seq * state + at0;
#pragma unroll
          for (int i = 0; i < NT; ++i) s[i] = from[static_cast<size_t>(i) * P];
        }
        for (int j = 0; j < seg.index; ++j) {
          const float *from = p.part + (seg.id0 + j) * state + at0;
          const float d = p.part_decay[static_cast<size_t>(seg.id0 + j) * a.H + h0 + hcol];
#pragma unroll
          for (int i = 0; i < NT; ++i) s[i] = fmaf(d, s[i], from[static_cast<size_t>(i) * P]);
        }
      }
      // S^T as two bf16 planes, columns as rows of n
      auto put_state = [&](int c) {
#pragma unroll
        for (int j = 0; j < NT / 8; ++j) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 u = make_float2(s[8 * j + 2 * e], s[8 * j + 2 * e + 1]);
            hi[e] = pack_bf16x2(u.x, u.y);
            const float2 f = unpack_bf16x2(hi[e]);
            const float2 r = __fadd2_rn(u, make_float2(-f.x, -f.y));
            lo[e] = pack_bf16x2(r.x, r.y);
          }
          const int n = n0 + 8 * j;
          const uint32_t at = sb + SM_SP + (n / 64) * REG128 + row * 128u +
                              (static_cast<uint32_t>(((n % 64) / 8) ^ (row & 7)) << 4);
          S.u128(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          S.u128(at + SP_PLANE) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        fence_proxy_async();
        arrive(bar(AS, c));
      };
      put_state(0);
      bool ok = true;
      for (int c = 0; c < n_chunks; ++c) {
        ok = warp_wait(prepared(c), c / DECS) && warp_wait_c(FX, c);
#pragma unroll 1
        for (int r = 0; r < XP::ROUNDS && ok; ++r) ok = put_weighted(c, r);
        ok = ok && warp_wait_c(DDS, c);
        if (!ok) break;
        tc_fence_after();
        const float keep = S.f32(decays(c, hcol) + DC_T + 16);
#pragma unroll
        for (int k = 0; k < NT; k += 16) {
          float v[16];
          tmem_ld16(lanes + TM_DS + n0 + k, v);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) s[k + i] = fmaf(keep, s[k + i], v[i]);
        }
        tc_fence_before();
        arrive(dec_free(c));
        if (c + 1 < n_chunks) put_state(c + 1);
      }
      if (ok && in && seg.last && a.S_out) {
        float *to = a.S_out + seg.seq * state + at0;
#pragma unroll
        for (int i = 0; i < NT; ++i) to[static_cast<size_t>(i) * P] = s[i];
      }
    }
  }
  if (gave_up) atomicOr(a.status, KDA_ERR_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  if (warp == kStateMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

constexpr int kSMs = 152;

int column_blocks(int H, int P, int G) { return P == 128 ? H : G * ((H / G + 1) / 2); }

// Tokens of a segment (0: no sequence is cut).  The host knows the mean length alone.  Costs in chunks of
// the second pass, for sequences of the mean length cut into k segments each: a chunk of the first
// pass is 0.5 of one (2.5 us against 5), starting a CTA one.  Where whole sequences do best but the
// lengths may differ, long ones are still cut: one long prompt among short ones would keep its own few
// SMs busy long after the others are done.  Cut at an SM's share of all chunks, the segments in front
// are one wave at most; at half of it two, which leaves shorter pieces for the end but more for the first
// pass.  Half is taken where the share is long (48 chunks) and the whole sequences are two waves of CTAs at
// most, so that there is little else to fill the SMs with.  Measured on 48 ragged batches (3 to 32 prompts of
// 16 to 100,000 tokens, 16 to 128 heads), half against whole shares, us: up to two waves 452 / 491 (6 prompts
// of 1 to 12001 tokens x 64 heads of 64, a share of 54), 637 / 683 (x 96 heads, 81), 1001 / 1148 (6 of 143557
// tokens in all, 118), the others even; beyond that from 881 / 696 (the first one's prompts x 128 heads, 108)
// and 476 / 439 (30000 and nine times 500, 57) to 575 / 737, as often worse as better; under 48 chunks
// 281 / 251 (x 32 heads, 27), 369 / 340 (x 48 heads, 41), 316 / 284 (16000 and nine times 500, 34).
int64_t segment_tokens(int n_seq, int64_t total, int blocks, bool ragged) {
  const int64_t chunks = (total / n_seq + kQ) / kQ;
  auto waves = [&](int64_t tasks) { return (tasks + kSMs - 1) / kSMs; };
  int64_t best = 0;
  double least = 0.0;
  for (int64_t k = 1; k <= 64 && (k == 1 || chunks >= 4 * k); ++k) {
    const int64_t per = (chunks + k - 1) / k;
    const int64_t tasks = static_cast<int64_t>(n_seq) * blocks;
    const double cost =
        waves(tasks * k) * (per + 1.0) + (k > 1 ? waves(tasks * (k - 1)) * (0.5 * per + 1.0) : 0.0);
    if (k == 1 || cost < least) {
      least = cost;
      best = k == 1 ? 0 : per * kQ;
    }
  }
  if (best == 0 && ragged && n_seq > 1) {
    const int64_t share = waves(total / kQ * blocks);
    const bool half = share >= 48 && waves(static_cast<int64_t>(n_seq) * blocks) <= 2;
    const int64_t cut = half ? share / 2 : share > 12 ? share : 12;
    if (total >= 2 * cut * kQ) best = cut * kQ;
  }
  return best;
}

// Segments in front of the last ones, at most: each holds seg_len tokens of its own.
size_t front_most(int64_t total, int64_t seg_len) {
  return seg_len ? static_cast<size_t>(total / seg_len) : 0;
}

size_t segment_bytes(int64_t total, int64_t seg_len, int H, int P, int N) {
  return front_most(total, seg_len) * H * (static_cast<size_t>(N) * P + 4) * sizeof(float);
}

bool row_map(CUtensorMap *map, const kda_bf16 *base, int64_t cols, int64_t rows, int64_t ld) {
  const EncodeTiledFn encode = tensor_map_encoder();
  if (!encode) return false;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(rows > 1 ? ld : cols) * 2};
  const cuuint32_t box[2] = {64, kQ};
  const cuuint32_t step[2] = {1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<kda_bf16 *>(base), dims,
                strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int N, int P, bool STATE_ONLY>
cudaError_t launch(const ChunkArgs &p, const CUtensorMap (&maps)[3], unsigned grid, bool early,
                   cudaStream_t st) {
  const auto kernel = ssm_chunk_kernel<N, P, STATE_ONLY>;
  const cudaError_t err =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SM_BYTES);
  if (err != cudaSuccess) return err;
  if (early) return launch_pdl(kernel, dim3(grid), dim3(kThreads), SM_BYTES, st, maps[0], maps[1], maps[2], p);
  kernel<<<grid, kThreads, SM_BYTES, st>>>(maps[0], maps[1], maps[2], p);
  return cudaGetLastError();
}

template <int N, int P>
cudaError_t run(ChunkArgs p, int64_t seg_len, cudaStream_t st) {
  const SsmArgs &a = p.a;
  CUtensorMap maps[3];
  memset(maps, 0, sizeof(maps));
  if (a.runs.total > 0 &&
      (!row_map(&maps[0], a.x, static_cast<int64_t>(a.H) * P, a.runs.total, a.ldx) ||
       !row_map(&maps[1], a.B, static_cast<int64_t>(a.G) * N, a.runs.total, a.ldb) ||
       !row_map(&maps[2], a.C, static_cast<int64_t>(a.G) * N, a.runs.total, a.ldc)))
    return cudaErrorInvalidValue;
  p.seg_len = seg_len ? seg_len : (a.runs.total / kQ + 1) * kQ;
  p.parts = static_cast<int>(front_most(a.runs.total, seg_len));
  const size_t front = static_cast<size_t>(p.parts) * p.blocks;
  const size_t blocks = front + static_cast<size_t>(a.runs.n) * p.blocks;
  if (blocks > 0x7fffffffull) return cudaErrorInvalidValue;
  if (front > 0) {
    const cudaError_t err = launch<N, P, true>(p, maps, static_cast<unsigned>(front), false, st);
    if (err != cudaSuccess) return err;
  }
  return launch<N, P, false>(p, maps, static_cast<unsigned>(blocks), front > 0, st);
}

}  // namespace

size_t ssm_chunk_workspace(int n_seq, int64_t total, int H, int P, int G, int N) {
  const int64_t seg_len = segment_tokens(n_seq, total, column_blocks(H, P, G), true);
  return segment_bytes(total, seg_len, H, P, N);
}

// Without a workspace of that size no sequence is cut into segments.
cudaError_t ssm_chunk_launch(const SsmArgs &a, int P, int G, int N, void *workspace, size_t bytes,
                             cudaStream_t st) {
  ChunkArgs p{};
  p.a = a;
  p.blocks = column_blocks(a.H, P, G);
  int64_t seg_len = segment_tokens(a.runs.n, a.runs.total, p.blocks, a.runs.cu != nullptr);
  if (seg_len) {
    if (!workspace || bytes < segment_bytes(a.runs.total, seg_len, a.H, P, N)) {
      seg_len = 0;
    } else {
      p.part = static_cast<float *>(workspace);
      p.part_decay = p.part + front_most(a.runs.total, seg_len) * a.H * N * P;
    }
  }
  if (N == 64) return P == 64 ? run<64, 64>(p, seg_len, st) : run<64, 128>(p, seg_len, st);
  return P == 64 ? run<128, 64>(p, seg_len, st) : run<128, 128>(p, seg_len, st);
}

}  // namespace kda

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
//   Y   [token x column] = C S                         then scaled by e^{l_t}, D x added
//                       += M X                         M = G * e^{l_t - l_s} dt_s, causal, from TMEM
//   dS^T[column x n]     = X'^T B                      X' = e^{l_end - l_s} dt_s x_s
//
// Roundings.  x, B and C are bf16 and enter exactly.  X' is split into three bf16 planes that hold
// all 24 bits of its fp32 value, and the state itself lives in registers in fp32 (S^T: one thread
// per column and quarter of n), so S and S_final carry fp32 accuracy.  For the output, S enters as two
// planes (16 bits) and M as one (8 bits): the in-chunk weights are rounded once to the type of the
// result, which adds an error of the size of the result's own rounding.
//
// Log decays are summed in blocks of 32 tokens from both ends (prefix for what is read at t, suffix
// for what is kept of s), so that an exponent never comes from the difference of two long sums.  A
// block pair (t-block > s-block) takes its decay as the product of e^{l_t - l_end(s-block)} and
// e^{l_end(s-block) - l_s}, both at most 1: one exponential per thread and block instead of 32.
//
// Long sequences are cut into segments that run side by side: a first pass takes the same steps for
// the state alone, from zero, over every segment but a sequence's last, and leaves N and the decay
// a of the whole segment; the second pass starts each segment from a_{j-1} (... (a_0 S0 + N_0) ...)
// + N_{j-1}.
//
// Roles: warps 0-15 (four warpgroups, the workers) do the element-wise work, warp 16 issues the TMA
// loads, warp 17 the MMAs, warps 18 and 19 compute the decays of the chunks ahead (one head each)
// and clear the rows behind a sequence's end, so that nothing of the next sequence is multiplied,
// not even by zero.  X, C and B rotate through three buffers: the next X goes where C was (free
// first), the next C where B was, the next B where X was.
#include <string.h>

#include "kda_serving.cuh"
#include "kda_tc_common.cuh"

namespace kda {

namespace {

using namespace tcx;

constexpr int kQ = 128;          // tokens of a chunk
constexpr int kWorkerWarps = 16;
constexpr int kThreads = 32 * (kWorkerWarps + 4);
constexpr int kLoadWarp = kWorkerWarps, kMmaWarp = kWorkerWarps + 1, kDecayWarp = kWorkerWarps + 2;

// shared memory
constexpr uint32_t SM_BUF = 0;              // X, C, B: three buffers of [128 rows][2 regions of 64]
constexpr uint32_t BUF_BYTES = 32 * KiB;
constexpr uint32_t SM_XP = 96 * KiB;        // X': three planes of [64 tokens][2 regions of 64]
constexpr uint32_t XP_PLANE = 16 * KiB;
constexpr uint32_t SM_SP = 144 * KiB;       // S^T: two planes of [128 columns][N / 64 regions]
constexpr uint32_t SP_PLANE = 32 * KiB;
constexpr uint32_t SM_DEC = 208 * KiB;      // decays: [2 chunks][2 heads] of struct Decays
constexpr uint32_t DEC_BYTES = 5 * 512 + 32;
constexpr uint32_t SM_BAR = SM_DEC + 4 * DEC_BYTES;
constexpr uint32_t SM_MISC = SM_BAR + 256;
constexpr uint32_t SM_BYTES = SM_MISC + 64;
static_assert(SM_BYTES <= 232448, "shared memory budget");

// Decays of one (chunk, head): offsets in bytes
constexpr uint32_t DC_L = 0;         // log2 decay from the 32-token block's start, token included
constexpr uint32_t DC_DT = 512;      // dt
constexpr uint32_t DC_F = 1024;      // decay to the block's end, times dt
constexpr uint32_t DC_E = 1536;      // decay from the chunk's start
constexpr uint32_t DC_W = 2048;      // decay to the chunk's end, times dt
constexpr uint32_t DC_T = 2560;      // log2 decays of the four blocks; then the chunk's decay

// mbarriers, two of each kind: of chunk c the one of its parity, in phase c / 2 (for the two halves
// of X' the one of the half, in phase c)
enum Bar : int { FX, FC, FB, PREP, DFREE, DG, DCS, DXP, DDS, DY, AXP, AM, AS, AY, AO, NBAR };

// TMEM columns
constexpr uint32_t TM_G = 0, TM_Y = 128, TM_DS = 256, TM_M = 384;

constexpr uint32_t kPolls = 1u << 24;

struct ChunkArgs {
  SsmArgs a;
  int64_t seg_len;   // tokens of a segment, a multiple of 128
  int blocks;        // column blocks: of a group, times G
  float *part;       // [segments, H, N, P]: what the first pass leaves
  float *part_decay; // [segments, H]
  int single;        // no sequence is cut (one segment for each sequence)
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

__device__ __forceinline__ bool elect() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one != 0;
}

// K-step k of a K-major operand: 32 bytes inside a 128-byte row, then the next 64-column region.
__device__ __forceinline__ constexpr uint32_t k_step(int k) {
  return (static_cast<uint32_t>(k >> 2) * REG128 + static_cast<uint32_t>(k & 3) * 32u) >> 4;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() {
  asm volatile("cp.async.wait_all;" ::: "memory");
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
  int id0;           // id of the sequence's first segment
  int64_t begin;     // first token
  int64_t len;
  bool last, bad;
};

// Segment `id` of the batch: sequence after sequence, ceil(length / seg_len) of each and one for an
// empty one.  Called by a whole warp; false beyond the last.
__device__ __forceinline__ bool find_segment(const Runs &r, int64_t seg_len, int id, Segment &g) {
  const int lane = threadIdx.x & 31;
  auto count = [&](int s) -> int {
    int64_t b, n, u;
    if (s >= r.n) return 0;
    run_range(r, s, b, n, u);
    return n <= seg_len ? 1 : static_cast<int>((n + seg_len - 1) / seg_len);
  };
  int before = 0;
  for (int base = 0; base < r.n; base += 32) {
    const int c = count(base + lane);
    int x = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    const unsigned m = __ballot_sync(0xffffffffu, before + x > id);
    if (m) {
      const int l = __ffs(m) - 1;
      g.seq = base + l;
      g.id0 = before + __shfl_sync(0xffffffffu, x - c, l);
      g.index = id - g.id0;
      int64_t b, n, u;
      g.bad = !run_range(r, g.seq, b, n, u);
      g.begin = b + g.index * seg_len;
      g.last = (g.index + 1) * seg_len >= n;
      g.len = g.last ? n - g.index * seg_len : seg_len;
      return true;
    }
    before += __shfl_sync(0xffffffffu, x, 31);
  }
  return false;
}

// STATE_ONLY: the first pass over the segments (no C, no output).
template <int N, int P, bool STATE_ONLY>
__global__ void __launch_bounds__(kThreads, 1)
ssm_chunk_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_b,
                 const __grid_constant__ CUtensorMap tm_c, const ChunkArgs p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  constexpr int HEADS = 128 / P;        // heads of a column block
  constexpr int NT = N / 4;             // state entries of a worker thread
  constexpr uint32_t BC_BYTES = 128 * N * 2;
  const SsmArgs &a = p.a;
  const uint32_t sb = smem_u32(smem);
  const Smem S{smem, sb};
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if ((sb & 1023u) != 0) {  // the swizzled layouts need 1024-byte alignment
    if (tid == 0) atomicOr(a.status, KDA_ERR_UNSUPPORTED);
    return;
  }
  Segment seg;
  const int id = blockIdx.x / p.blocks, block = blockIdx.x % p.blocks;
  if (!find_segment(a.runs, p.seg_len, id, seg)) return;
  if (seg.bad && block == 0 && tid == 0) atomicOr(a.status, KDA_ERR_SHAPE);
  if (seg.bad || (STATE_ONLY && seg.last)) return;
  const int per_group = a.H / a.G, blocks_per_group = p.blocks / a.G;
  const int g = block / blocks_per_group;
  const int first_in_group = (block % blocks_per_group) * HEADS;
  const int h0 = g * per_group + first_in_group;
  const int heads = per_group - first_in_group < HEADS ? 1 : HEADS;
  const int n_chunks = static_cast<int>((seg.len + kQ - 1) / kQ);

  volatile int *s_abort = reinterpret_cast<volatile int *>(smem + SM_MISC + 8);
  auto bar = [&](int kind, int c) { return sb + SM_BAR + 16u * kind + 8u * (c & 1); };
  if (tid == 0) {
    *s_abort = 0;
    for (int k = 0; k < NBAR; ++k) {
      const uint32_t count = k == PREP ? 2u : k >= AXP || k == DFREE ? kWorkerWarps : 1u;
      mbar_init(bar(k, 0), count);
      mbar_init(bar(k, 1), count);
    }
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(sb + SM_MISC, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + SM_MISC);

  // Every wait is bounded; one that gives up ends them all.
  auto wait = [&](uint32_t b, uint32_t phase) -> bool {
    for (uint32_t i = 0; i < kPolls; ++i) {
      if (mbar_try_wait(b, phase & 1u)) return true;
      if (*s_abort) return false;
    }
    *s_abort = 1;
    atomicOr(a.status, KDA_ERR_TIMEOUT);
    return false;
  };
  auto wait_c = [&](int kind, int c) { return wait(bar(kind, c), static_cast<uint32_t>(c) >> 1); };
  // the same for a whole warp, which goes on or stops as one
  auto warp_wait = [&](uint32_t b, uint32_t phase) {
    return __all_sync(0xffffffffu, wait(b, phase)) != 0;
  };
  auto warp_wait_c = [&](int kind, int c) {
    return warp_wait(bar(kind, c), static_cast<uint32_t>(c) >> 1);
  };

  // buffers of chunk c
  auto buf = [&](int i) { return sb + SM_BUF + static_cast<uint32_t>(i % 3) * BUF_BYTES; };
  auto buf_x = [&](int c) { return STATE_ONLY ? sb + SM_BUF + (c & 1) * BUF_BYTES : buf(c); };
  auto buf_c = [&](int c) { return buf(c + 1); };
  auto buf_b = [&](int c) {
    return STATE_ONLY ? ((c & 1) ? sb + SM_SP : sb + SM_BUF + 2 * BUF_BYTES) : buf(c + 2);
  };

  if (warp == kLoadWarp) {
    if (lane == 0) {
      bool ok = true;
      int c = 0;
      for (; c < n_chunks && ok; ++c) {
        const int t = static_cast<int>(seg.begin + static_cast<int64_t>(c) * kQ);
        auto load_x = [&]() {
          mbar_expect_tx(bar(FX, c), BUF_BYTES);
          for (int r = 0; r < 2; ++r)
            tma_load_2d(buf_x(c) + r * REG128, &tm_x, h0 * P + 64 * r, t, bar(FX, c));
        };
        auto load_bc = [&](const CUtensorMap *map, uint32_t to, uint32_t b) {
          mbar_expect_tx(b, BC_BYTES);
          for (int r = 0; r < N / 64; ++r) tma_load_2d(to + r * REG128, map, g * N + 64 * r, t, b);
        };
        if constexpr (STATE_ONLY) {
          if (c >= 2) ok = wait_c(DDS, c - 2);
          if (!ok) break;
          load_x();
          load_bc(&tm_b, buf_b(c), bar(FB, c));
        } else {
          if (c > 0) ok = wait_c(DCS, c - 1);
          if (!ok) break;
          load_x();
          if (c > 0) ok = wait_c(DDS, c - 1);
          if (!ok) break;
          load_bc(&tm_c, buf_c(c), bar(FC, c));
          if (c > 0) ok = wait_c(DY, c - 1);
          if (!ok) break;
          load_bc(&tm_b, buf_b(c), bar(FB, c));
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
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // The whole warp goes through the loop (so that addresses and descriptors stay in uniform
    // registers); one lane issues.
    constexpr uint32_t ID_KK = idesc_mma(128, 128, kFmtBF16, kFmtBF16, 0, 0);
    constexpr uint32_t ID_MX = idesc_mma(128, P, kFmtBF16, kFmtBF16, 0, 1);
    constexpr uint32_t ID_DS = idesc_mma(128, N, kFmtBF16, kFmtBF16, 1, 1);
    const bool one = elect();
    bool ok = true;
    for (int c = 0; c < n_chunks; ++c) {
      const uint64_t b_k = sw128_desc(buf_b(c), 16u, 1024u);  // B by rows of n, and by rows of tokens
      const uint64_t b_mn = sw128_desc(buf_b(c), REG128, 1024u);
      if constexpr (!STATE_ONLY) {
        const uint64_t c_k = sw128_desc(buf_c(c), 16u, 1024u);
        const uint64_t s_k = sw128_desc(sb + SM_SP, 16u, 1024u);
        ok = warp_wait_c(FC, c) && warp_wait_c(FB, c) && warp_wait_c(PREP, c);
        if (!ok) break;
        tc_fence_after();
        if (one) {
#pragma unroll
          for (int k = 0; k < N / 16; ++k)
            mma_f16(tmem + TM_G, c_k + k_step(k), b_k + k_step(k), ID_KK, k > 0);
          mma_commit(bar(DG, c));
        }
        ok = warp_wait_c(AS, c) && (c == 0 || warp_wait_c(AY, c - 1));
        if (!ok) break;
        tc_fence_after();
        if (one) {
#pragma unroll
          for (int k = 0; k < 2 * (N / 16); ++k)
            mma_f16(tmem + TM_Y, c_k + k_step(k % (N / 16)),
                    s_k + k_step(k % (N / 16)) + (k / (N / 16)) * (SP_PLANE >> 4), ID_KK, k > 0);
          mma_commit(bar(DCS, c));
        }
      } else {
        ok = warp_wait_c(FB, c) && warp_wait_c(PREP, c) && warp_wait_c(AS, c);
        if (!ok) break;
      }
      const uint64_t xp_mn = sw128_desc(sb + SM_XP, REG64, 1024u);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        ok = ok && warp_wait(bar(AXP, half), c);
        if (ok) {
          tc_fence_after();
          if (one) {
#pragma unroll
            for (int k = 0; k < 12; ++k)
              mma_f16(tmem + TM_DS, xp_mn + (((k / 4) * XP_PLANE + (k % 4) * 2048u) >> 4),
                      b_mn + ((half * REG64 + (k % 4) * 2048u) >> 4), ID_DS, half + k > 0);
            mma_commit(half == 0 ? bar(DXP, 0) : bar(DDS, c));
          }
        }
      }
      if (!ok) break;
      if constexpr (!STATE_ONLY) {
        ok = warp_wait_c(FX, c) && warp_wait_c(AM, c);
        if (!ok) break;
        tc_fence_after();
        if (one) {
          const uint64_t x_mn = sw128_desc(buf_x(c), REG128, 1024u);
#pragma unroll
          for (int k = 0; k < 8 * HEADS; ++k)
            mma_f16_ta(tmem + TM_Y + 64 * (k / 8), tmem + TM_M + 64 * (k / 8) + 8 * (k % 8),
                       x_mn + (((k / 8) * REG128 + (k % 8) * 2048u) >> 4), ID_MX, 1);
          mma_commit(bar(DY, c));
        }
      }
    }
    if (!ok && one) {  // MMAs in flight finish before TMEM goes
      mma_commit(bar(DXP, 1));
      mbar_wait_bounded(bar(DXP, 1), 0, 1u << 16);
    }
    __syncwarp();
  } else if (warp >= kDecayWarp) {
    // decays: lane i has tokens 4 i .. 4 i + 3, eight lanes a block
    const int hh = warp - kDecayWarp;
    const bool mine = hh < heads;
    const float A2 = mine ? a.A[h0 + hh] * 1.44269504088896340736f : 0.f;
    for (int c = 0; c < n_chunks; ++c) {
      const int64_t t0 = seg.begin + static_cast<int64_t>(c) * kQ;
      const int len = seg.len - static_cast<int64_t>(c) * kQ < kQ
                          ? static_cast<int>(seg.len - static_cast<int64_t>(c) * kQ)
                          : kQ;
      float dt[4], pre[4], suf[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        dt[i] = mine && 4 * lane + i < len ? ssm_dt(a, t0 + 4 * lane + i, h0 + hh) : 0.f;
      pre[0] = dt[0] * A2;
#pragma unroll
      for (int i = 1; i < 4; ++i) pre[i] = pre[i - 1] + dt[i] * A2;
      suf[3] = 0.f;
#pragma unroll
      for (int i = 2; i >= 0; --i) suf[i] = suf[i + 1] + dt[i + 1] * A2;
      const float four = suf[0] + dt[0] * A2;
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
      for (int k = 0; k < 4; ++k) blocks[k] = __shfl_sync(0xffffffffu, whole, 8 * k);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (k < lane / 8) front += blocks[k];
        if (3 - k > lane / 8) behind += blocks[3 - k];
      }
      if (c >= 2 && !warp_wait(bar(DFREE, c), (c >> 1) - 1)) break;
      const uint32_t at = sb + SM_DEC + ((c & 1) * 2 + hh) * DEC_BYTES;
      float4 v;
      float *vp = &v.x;
      auto put = [&](uint32_t off) { *reinterpret_cast<float4 *>(S.ptr(at + off + 16 * lane)) = v; };
#pragma unroll
      for (int i = 0; i < 4; ++i) vp[i] = up_ex + pre[i];
      put(DC_L);
#pragma unroll
      for (int i = 0; i < 4; ++i) vp[i] = dt[i];
      put(DC_DT);
#pragma unroll
      for (int i = 0; i < 4; ++i) vp[i] = exp2f(suf[i] + down_ex) * dt[i];
      put(DC_F);
#pragma unroll
      for (int i = 0; i < 4; ++i) vp[i] = exp2f(front + (up_ex + pre[i]));
      put(DC_E);
#pragma unroll
      for (int i = 0; i < 4; ++i) vp[i] = exp2f(behind + (suf[i] + down_ex)) * dt[i];
      put(DC_W);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (lane == k) S.f32(at + DC_T + 4 * k) = blocks[k];
      if (lane == 4) S.f32(at + DC_T + 16) = exp2f((blocks[0] + blocks[1]) + (blocks[2] + blocks[3]));
      if (len < kQ) {  // clear what lies behind the sequence's end
        if (!warp_wait_c(FX, c) || !warp_wait_c(FB, c)) break;
        const int rows = kQ - len;
        for (int i = hh * 32 + lane; i < rows * 8; i += 64) {
          const uint32_t off = static_cast<uint32_t>(len) * 128u + 16u * i;
          for (int r = 0; r < 2; ++r) S.u128(buf_x(c) + r * REG128 + off) = make_uint4(0, 0, 0, 0);
          for (int r = 0; r < N / 64; ++r)
            S.u128(buf_b(c) + r * REG128 + off) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(PREP, c));
    }
  } else {
    // ---- the workers ----------------------------------------------------------------------
    const int wg = warp >> 2, quad = warp & 3;
    const int row = quad * 32 + lane;  // TMEM lane: token of G, M, Y; column of dS^T
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const int hcol = HEADS == 2 ? quad >> 1 : 0;   // head of this thread's state column
    const int hout = HEADS == 2 ? wg >> 1 : 0;     // head of its output columns [32 wg, 32 wg + 32)
    const bool col_in = hcol < heads, out_in = hout < heads;
    const int n0 = wg * NT;
    const size_t col_at = static_cast<size_t>(h0 + hcol) * N * P + static_cast<size_t>(n0) * P +
                          row % P;
    const size_t state = static_cast<size_t>(a.H) * N * P;
    auto arrive = [&](uint32_t b) {
      __syncwarp();
      if (lane == 0) mbar_arrive(b);
    };
    float s[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) s[i] = 0.f;
    if (!STATE_ONLY && col_in) {
      if (a.S_in) {
        const float *from = a.S_in + seg.seq * state + col_at;
#pragma unroll
        for (int i = 0; i < NT; ++i) s[i] = from[static_cast<size_t>(i) * P];
      }
      for (int j = 0; j < seg.index; ++j) {
        const float *from = p.part + (seg.id0 + j) * state + col_at;
        const float d = p.part_decay[static_cast<size_t>(seg.id0 + j) * a.H + h0 + hcol];
#pragma unroll
        for (int i = 0; i < NT; ++i) s[i] = fmaf(d, s[i], from[static_cast<size_t>(i) * P]);
      }
    }
    // S^T as two bf16 planes, columns as rows of n
    auto put_state = [&]() {
#pragma unroll
      for (int j = 0; j < NT / 8; ++j) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float u = s[8 * j + 2 * e], v = s[8 * j + 2 * e + 1];
          hi[e] = pack_bf16x2(u, v);
          const float2 f = unpack_bf16x2(hi[e]);
          lo[e] = pack_bf16x2(u - f.x, v - f.y);
        }
        const int n = n0 + 8 * j;
        const uint32_t at = sb + SM_SP + (n / 64) * REG128 + row * 128u +
                            (static_cast<uint32_t>(((n % 64) / 8) ^ (row & 7)) << 4);
        S.u128(at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        S.u128(at + SP_PLANE) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
      fence_proxy_async();
    };
    if constexpr (!STATE_ONLY) {
      put_state();
      // weights of later blocks of tokens: zero, once and for all
      float none[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) none[i] = 0.f;
      for (int b = quad + 1; b < 4; ++b)
        if (HEADS == 2 ? (wg & 1) == 0 : wg == 0) tmem_st16(lanes + TM_M + 64 * hout + 16 * b, none);
      tmem_wait_st();
    }
    arrive(bar(AS, 0));
    float decay = 1.f;
    const float skip = !STATE_ONLY && a.D && out_in ? a.D[h0 + hout] : 0.f;

    for (int c = 0; c < n_chunks; ++c) {
      const int64_t t0 = seg.begin + static_cast<int64_t>(c) * kQ;
      const uint32_t dec = sb + SM_DEC + (c & 1) * 2 * DEC_BYTES;
      if (!warp_wait_c(PREP, c) || !warp_wait_c(FX, c)) break;
      // X' overwrites what other warps staged of the last output
      if (!STATE_ONLY && c > 0 && !warp_wait_c(AO, c - 1)) break;
      bool ok = true;
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        if (half == 1 && !(ok = warp_wait(bar(DXP, 0), c))) break;
        // X' of tokens [64 half, 64 half + 64): a thread takes 8 columns of each region of a row
        const int j = tid & 7, tok = tid >> 3;
        const uint32_t off = tok * 128u + (static_cast<uint32_t>(j ^ (tok & 7)) << 4);
#pragma unroll
        for (int region = 0; region < 2; ++region) {
          const float w = S.f32(dec + (HEADS == 2 ? region : 0) * DEC_BYTES + DC_W +
                                4 * (64 * half + tok));
          const uint4 raw = S.u128(buf_x(c) + region * REG128 + half * REG64 + off);
          const uint32_t in[4] = {raw.x, raw.y, raw.z, raw.w};
          const float2 w2 = make_float2(w, w);
          uint32_t out[3][4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float2 f = __fmul2_rn(unpack_bf16x2(in[e]), w2);
            out[0][e] = upper(f.x, f.y);
            f = __fadd2_rn(f, make_float2(-truncated(f.x), -truncated(f.y)));
            out[1][e] = upper(f.x, f.y);
            f = __fadd2_rn(f, make_float2(-truncated(f.x), -truncated(f.y)));
            out[2][e] = upper(f.x, f.y);
          }
          const uint32_t to = sb + SM_XP + region * REG64 + off;
#pragma unroll
          for (int k = 0; k < 3; ++k)
            S.u128(to + k * XP_PLANE) = make_uint4(out[k][0], out[k][1], out[k][2], out[k][3]);
        }
        fence_proxy_async();
        arrive(bar(AXP, half));

        if constexpr (!STATE_ONLY) {
          if (half == 1) break;
          if (!(ok = warp_wait_c(DG, c))) break;
          tc_fence_after();
          // M: causal weights of the tokens, 32 at a time
          const uint32_t d = dec + hout * DEC_BYTES;
          const float lt = S.f32(d + DC_L + 4 * row);
#pragma unroll 1
          for (int k = 0; k < (HEADS == 2 ? 2 : 1); ++k) {
            const int b = HEADS == 1 ? wg : k == 0 ? wg & 1 : 3 - (wg & 1);  // block of s
            if (b > quad) continue;
            float m[32];
            tmem_ld32(lanes + TM_G + 32 * b, m);
            tmem_wait_ld();
            uint32_t packed[16];
            if (b < quad) {
              float l = lt;  // from the block's end to t
              for (int q = b + 1; q < quad; ++q) l += S.f32(d + DC_T + 4 * q);
              const float e = ex2(l);
              const float2 e2 = make_float2(e, e);
#pragma unroll
              for (int i = 0; i < 32; i += 4) {
                const float4 f = *reinterpret_cast<const float4 *>(S.ptr(d + DC_F + 4 * (32 * b + i)));
                const float2 u = __fmul2_rn(make_float2(m[i], m[i + 1]),
                                            __fmul2_rn(make_float2(f.x, f.y), e2));
                const float2 v = __fmul2_rn(make_float2(m[i + 2], m[i + 3]),
                                            __fmul2_rn(make_float2(f.z, f.w), e2));
                packed[i / 2] = pack_bf16x2(u.x, u.y);
                packed[i / 2 + 1] = pack_bf16x2(v.x, v.y);
              }
            } else {
#pragma unroll
              for (int i = 0; i < 32; i += 4) {
                const float4 l = *reinterpret_cast<const float4 *>(S.ptr(d + DC_L + 4 * (32 * b + i)));
                const float4 w = *reinterpret_cast<const float4 *>(S.ptr(d + DC_DT + 4 * (32 * b + i)));
                const float u0 = i <= lane ? m[i] * (ex2(lt - l.x) * w.x) : 0.f;
                const float u1 = i + 1 <= lane ? m[i + 1] * (ex2(lt - l.y) * w.y) : 0.f;
                const float u2 = i + 2 <= lane ? m[i + 2] * (ex2(lt - l.z) * w.z) : 0.f;
                const float u3 = i + 3 <= lane ? m[i + 3] * (ex2(lt - l.w) * w.w) : 0.f;
                packed[i / 2] = pack_bf16x2(u0, u1);
                packed[i / 2 + 1] = pack_bf16x2(u2, u3);
              }
            }
            float words[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) words[i] = __uint_as_float(packed[i]);
            tmem_st16(lanes + TM_M + 64 * hout + 16 * b, words);
          }
        }
      }
      if (!ok) break;

      if constexpr (!STATE_ONLY) {
        if (!warp_wait_c(DCS, c)) break;
        tc_fence_after();
        // C S, scaled to each token, and D x
        const float e = S.f32(dec + hout * DEC_BYTES + DC_E + 4 * row);
        const float2 e2 = make_float2(e, e), skip2 = make_float2(skip, skip);
        float y[32];
        tmem_ld32(lanes + TM_Y + 32 * wg, y);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint4 raw = S.u128(buf_x(c) + (wg >> 1) * REG128 + row * 128u +
                                   (static_cast<uint32_t>((4 * (wg & 1) + j) ^ (row & 7)) << 4));
          const uint32_t in[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int i = 8 * j + 2 * q;
            const float2 f = __ffma2_rn(e2, make_float2(y[i], y[i + 1]),
                                        __fmul2_rn(skip2, unpack_bf16x2(in[q])));
            y[i] = f.x;
            y[i + 1] = f.y;
          }
        }
        tmem_st32(lanes + TM_Y + 32 * wg, y);
        tmem_wait_st();
        tc_fence_before();
        arrive(bar(AM, c));
      }

      // the state behind this chunk
      if (!warp_wait_c(DDS, c)) break;
      tc_fence_after();
      // X' is free from here on: each warp stages 32 rows of 64 bytes of z, then of o, there
      const uint32_t stage = sb + SM_XP + warp * 2048u;
      const int64_t rows_left = seg.len - static_cast<int64_t>(c) * kQ - quad * 32;
      const int64_t first = t0 + quad * 32, cols = static_cast<int64_t>(h0) * P + 32 * wg;
      if (!STATE_ONLY && a.z && out_in) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 8 * i + (lane >> 2), j = lane & 3;
          if (r < rows_left)
            cp_async16(stage + r * 64u + ((j ^ ((r >> 1) & 3)) << 4),
                       a.z + (first + r) * a.ldz + cols + 8 * j);
        }
      }
      const float keep = S.f32(dec + hcol * DEC_BYTES + DC_T + 16);
      decay *= keep;
      {
        float v[NT];
        if constexpr (NT == 32)
          tmem_ld32(lanes + TM_DS + n0, v);
        else
          tmem_ld16(lanes + TM_DS + n0, v);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < NT; ++i) s[i] = fmaf(keep, s[i], v[i]);
      }
      tc_fence_before();
      if (!STATE_ONLY && c + 1 < n_chunks) put_state();
      arrive(bar(AS, c + 1));
      if (lane == 0) mbar_arrive(bar(DFREE, c));

      if constexpr (!STATE_ONLY) {
        if (a.z) {
          cp_async_wait_all();
          __syncwarp();
        }
        if (!warp_wait_c(DY, c)) break;
        tc_fence_after();
        float y[32];
        tmem_ld32(lanes + TM_Y + 32 * wg, y);
        tmem_wait_ld();
        tc_fence_before();
        arrive(bar(AY, c));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t at = stage + lane * 64u + ((j ^ ((lane >> 1) & 3)) << 4);
          if (a.z) {
            const uint4 raw = S.u128(at);
            const uint32_t in[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float2 f = unpack_bf16x2(in[q]);
              y[8 * j + 2 * q] *= silu(f.x);
              y[8 * j + 2 * q + 1] *= silu(f.y);
            }
          }
          S.u128(at) = make_uint4(
              pack_bf16x2(y[8 * j], y[8 * j + 1]), pack_bf16x2(y[8 * j + 2], y[8 * j + 3]),
              pack_bf16x2(y[8 * j + 4], y[8 * j + 5]), pack_bf16x2(y[8 * j + 6], y[8 * j + 7]));
        }
        __syncwarp();
        if (out_in) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = 8 * i + (lane >> 2), j = lane & 3;
            if (r < rows_left)
              *reinterpret_cast<uint4 *>(a.o + (first + r) * a.ldo + cols + 8 * j) =
                  S.u128(stage + r * 64u + ((j ^ ((r >> 1) & 3)) << 4));
          }
        }
        arrive(bar(AO, c));
      }
    }
    if (!*s_abort && col_in) {
      float *to = nullptr;
      if (STATE_ONLY)
        to = p.part + static_cast<size_t>(id) * state + col_at;
      else if (seg.last && a.S_out)
        to = a.S_out + seg.seq * state + col_at;
      if (to)
#pragma unroll
        for (int i = 0; i < NT; ++i) to[static_cast<size_t>(i) * P] = s[i];
      if (STATE_ONLY && wg == 0 && row % P == 0)
        p.part_decay[static_cast<size_t>(id) * a.H + h0 + hcol] = decay;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

constexpr int kSMs = 152;

int column_blocks(int H, int P, int G) { return P == 128 ? H : G * ((H / G + 1) / 2); }

// Tokens of a segment.  Costs in chunks of the second pass, for sequences of the mean length cut into
// k segments each: a chunk of the first pass is 0.45 of one, starting a CTA one.
int64_t segment_tokens(int n_seq, int64_t total, int blocks) {
  const int64_t chunks = (total / n_seq + kQ) / kQ;
  auto waves = [&](int64_t tasks) { return (tasks + kSMs - 1) / kSMs; };
  int64_t best = 0;
  double least = 0.0;
  for (int64_t k = 1; k <= 64 && (k == 1 || chunks >= 4 * k); ++k) {
    const int64_t per = (chunks + k - 1) / k;
    const int64_t tasks = static_cast<int64_t>(n_seq) * blocks;
    const double cost =
        waves(tasks * k) * (per + 1.0) + (k > 1 ? waves(tasks * (k - 1)) * (0.45 * per + 1.0) : 0.0);
    if (k == 1 || cost < least) {
      least = cost;
      best = k == 1 ? 0 : per * kQ;  // 0: not cut
    }
  }
  return best;
}

size_t segments_most(int n_seq, int64_t total, int64_t seg_len) {
  return seg_len ? static_cast<size_t>(total / seg_len + n_seq) : static_cast<size_t>(n_seq);
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
cudaError_t launch(const ChunkArgs &p, const CUtensorMap (&maps)[3], unsigned grid,
                   cudaStream_t st) {
  const cudaError_t err =
      cudaFuncSetAttribute(ssm_chunk_kernel<N, P, STATE_ONLY>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize, SM_BYTES);
  if (err != cudaSuccess) return err;
  ssm_chunk_kernel<N, P, STATE_ONLY><<<grid, kThreads, SM_BYTES, st>>>(maps[0], maps[1], maps[2], p);
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
  p.single = seg_len == 0;
  p.seg_len = seg_len ? seg_len : (a.runs.total / kQ + 1) * kQ;
  const size_t blocks = segments_most(a.runs.n, a.runs.total, seg_len) * p.blocks;
  if (blocks > 0x7fffffffull) return cudaErrorInvalidValue;
  const unsigned grid = static_cast<unsigned>(blocks);
  if (seg_len) {
    const cudaError_t err = launch<N, P, true>(p, maps, grid, st);
    if (err != cudaSuccess) return err;
  }
  return launch<N, P, false>(p, maps, grid, st);
}

}  // namespace

size_t ssm_chunk_workspace(int n_seq, int64_t total, int H, int P, int G, int N) {
  const int64_t seg_len = segment_tokens(n_seq, total, column_blocks(H, P, G));
  if (!seg_len) return 0;
  return segments_most(n_seq, total, seg_len) * H * (static_cast<size_t>(N) * P + 4) * sizeof(float);
}

// Without a workspace of that size no sequence is cut into segments.
cudaError_t ssm_chunk_launch(const SsmArgs &a, int P, int G, int N, void *workspace, size_t bytes,
                             cudaStream_t st) {
  ChunkArgs p{};
  p.a = a;
  p.blocks = column_blocks(a.H, P, G);
  int64_t seg_len = segment_tokens(a.runs.n, a.runs.total, p.blocks);
  if (seg_len) {
    if (!workspace || bytes < ssm_chunk_workspace(a.runs.n, a.runs.total, a.H, P, G, N)) {
      seg_len = 0;
    } else {
      p.part = static_cast<float *>(workspace);
      p.part_decay = p.part + segments_most(a.runs.n, a.runs.total, seg_len) * a.H * N * P;
    }
  }
  if (N == 64) return P == 64 ? run<64, 64>(p, seg_len, st) : run<64, 128>(p, seg_len, st);
  return P == 64 ? run<128, 64>(p, seg_len, st) : run<128, 128>(p, seg_len, st);
}

}  // namespace kda

// Short causal depthwise convolution over packed prompts, and over token runs on a pool of the
// sequences' last inputs.
//
//   o_t[c] = act(bias[c] + sum_{w < W} weight[c, w] x_{t - (W - 1) + w}[c]),  act = silu or identity
//
// with the W - 1 held rows (or zeros) in front of a sequence's first token.  Both kernels are bound
// by memory: x is read once and o written once.  A thread owns VEC neighbouring channels (one
// 16-byte vector where the layout allows it) and walks along the tokens with the last W - 1 rows in
// registers.  It takes AHEAD tokens at a time (4 of a prompt or a run, 1 alone); a prompt's next 4 rows
// are in flight while the present ones are worked on (without that: 110 us instead of 98 at 32768 x
// 4352), and each row is widened to fp32 once for the W outputs that it enters.  The arithmetic is
// packed fp32x2 over channel pairs.  At that size the kernel moves 5.8 TB/s, 0.86 of a plain copy; the
// exponential and the reciprocal of silu take 0.6 of its time on their pipe.
#include "kda_serving.cuh"

namespace kda {

namespace {

// One warp to a CTA: 20 CTAs of 32 threads took 98 us for 32768 x 4352 tokens x channels, 5 of 128 threads
// 105 us: the tiles of a long prompt end more evenly.  They leave 96 registers a thread, for which the form of
// vectors and 4 taps keeps 48 bytes on the stack (60 bytes of spill stores; 3 taps 16, 2 taps 32).
constexpr int kConvThreads = 32;

template <int VEC>
struct Row {  // VEC bf16 channels of one row, two to a word (one alone: the lower half)
  uint32_t w[VEC == 8 ? 4 : 1];
};

template <int VEC>
__device__ __forceinline__ Row<VEC> load_row(const kda_bf16 *p) {
  Row<VEC> r;
  if constexpr (VEC == 8)
    *reinterpret_cast<uint4 *>(r.w) = __ldg(reinterpret_cast<const uint4 *>(p));
  else
    r.w[0] = __ldg(p);
  return r;
}
// The same from memory that this launch writes (the pool).
template <int VEC>
__device__ __forceinline__ Row<VEC> load_held(const kda_bf16 *p) {
  Row<VEC> r;
  if constexpr (VEC == 8)
    *reinterpret_cast<uint4 *>(r.w) = *reinterpret_cast<const uint4 *>(p);
  else
    r.w[0] = *p;
  return r;
}

template <int VEC>
__device__ __forceinline__ void store_row(kda_bf16 *p, const Row<VEC> &r) {
  if constexpr (VEC == 8)
    *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<const uint4 *>(r.w);
  else
    *p = static_cast<kda_bf16>(r.w[0]);
}

template <int VEC>
__device__ __forceinline__ Row<VEC> zero_row() {
  Row<VEC> r;
#pragma unroll
  for (uint32_t &w : r.w) w = 0;
  return r;
}

__device__ __forceinline__ float2 widen(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

template <int W, int VEC>
struct Taps {
  static constexpr int PAIRS = VEC == 8 ? 4 : 1;
  float2 w[W][PAIRS], b[PAIRS];

  // weight [D, W]: the VEC x W values of channels c .. c + VEC - 1 lie together
  __device__ __forceinline__ void load(const ConvArgs &a, int c) {
    if constexpr (VEC == 8) {
      kda_bf16 v[8 * W], bias[8];
#pragma unroll
      for (int i = 0; i < W; ++i)
        reinterpret_cast<uint4 *>(v)[i] =
            __ldg(reinterpret_cast<const uint4 *>(a.weight + static_cast<size_t>(c) * W) + i);
      *reinterpret_cast<uint4 *>(bias) =
          a.bias ? __ldg(reinterpret_cast<const uint4 *>(a.bias + c)) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
#pragma unroll
        for (int k = 0; k < W; ++k)
          w[k][q] = make_float2(bf2f(v[2 * q * W + k]), bf2f(v[(2 * q + 1) * W + k]));
        b[q] = make_float2(bf2f(bias[2 * q]), bf2f(bias[2 * q + 1]));
      }
    } else {
#pragma unroll
      for (int k = 0; k < W; ++k)
        w[k][0] = make_float2(bf2f(a.weight[static_cast<size_t>(c) * W + k]), 0.f);
      b[0] = make_float2(a.bias ? bf2f(a.bias[c]) : 0.f, 0.f);
    }
  }

  // AHEAD rows in, their outputs in the same place; `held` becomes the last W - 1 rows.
  template <int AHEAD>
  __device__ __forceinline__ void apply(Row<VEC> (&held)[W - 1], Row<VEC> (&x)[AHEAD],
                                        int act) const {
    Row<VEC> last[W - 1];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
      constexpr int KEEP = AHEAD;  // rows of x behind the held ones
      last[k] = k + KEEP < W - 1 ? held[k + KEEP < W - 1 ? k + KEEP : 0]
                                 : x[k + KEEP < W - 1 ? 0 : k + KEEP - (W - 1)];
    }
#pragma unroll
    for (int q = 0; q < PAIRS; ++q) {
      float2 window[W];
#pragma unroll
      for (int k = 0; k < W - 1; ++k) window[k + 1] = widen(held[k].w[q]);
#pragma unroll
      for (int t = 0; t < AHEAD; ++t) {
#pragma unroll
        for (int k = 0; k < W - 1; ++k) window[k] = window[k + 1];
        window[W - 1] = widen(x[t].w[q]);
        float2 s = b[q];
#pragma unroll
        for (int k = 0; k < W; ++k) s = __ffma2_rn(w[k][q], window[k], s);
        if (act) {
          const float2 e = __fmul2_rn(s, make_float2(-1.44269504088896340736f, -1.44269504088896340736f));
          const float2 d = __fadd2_rn(make_float2(ex2(e.x), ex2(e.y)), make_float2(1.f, 1.f));
          s = __fmul2_rn(s, make_float2(rcp(d.x), rcp(d.y)));
        }
        const __nv_bfloat162 r = __floats2bfloat162_rn(s.x, s.y);
        x[t].w[q] = *reinterpret_cast<const uint32_t *>(&r);
      }
    }
#pragma unroll
    for (int k = 0; k < W - 1; ++k) held[k] = last[k];
  }
};

// Row pos - back of sequence s (pos: position of the current token, row t): x inside the sequence,
// a held row in front of it.
template <int W, int VEC>
__device__ __forceinline__ Row<VEC> earlier_row(const ConvArgs &a, int s, int64_t t, int64_t pos,
                                                int back, int c) {
  if (pos >= back) return load_row<VEC>(a.x + (t - back) * a.ldx + c);
  if (!a.state_in) return zero_row<VEC>();
  const int64_t j = static_cast<int64_t>(s) * (W - 1) + (W - 1) - back + pos;
  return load_row<VEC>(a.state_in + j * a.D + c);
}

// The number of sequences that end at or before token t: a 32-way search by the whole warp.
__device__ __forceinline__ int first_sequence(const Runs &r, int64_t t) {
  if (!r.cu) return static_cast<int>(t / r.fixed_len);
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = r.n;
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32, i = lo + lane * step;
    const int n = __popc(__ballot_sync(0xffffffffu, i < hi && r.cu[i + 1] <= t));
    if (n == 0) return lo;
    if (step == 1) return lo + n;
    const int next = lo + (n - 1) * step + 1;
    hi = lo + n * step < hi ? lo + n * step : hi;
    lo = next;
  }
  return lo;
}

// Packed prompts.  Block = (tile, channels), channels fastest: `tile_tokens` tokens from
// tile * tile_tokens on; the blocks behind the tiles write one sequence's final rows each.
template <int W, int VEC>
__global__ void __launch_bounds__(kConvThreads, 20)
conv_fwd_kernel(const ConvArgs a, int c_blocks, int64_t tiles, int tile_tokens) {
  constexpr int AHEAD = 4;
  const int64_t tile = blockIdx.x / c_blocks;
  const int c = (static_cast<int>(blockIdx.x % c_blocks) * kConvThreads + threadIdx.x) * VEC;
  if (tile >= tiles) {
    const int s = static_cast<int>(tile - tiles);
    int64_t begin, len, used;
    if (!run_range(a.runs, s, begin, len, used)) {
      if (c == 0) atomicOr(a.status, KDA_ERR_SHAPE);
      return;
    }
    if (c >= a.D || !a.state_out) return;
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
      const Row<VEC> r = earlier_row<W, VEC>(a, s, begin + len, len, W - 1 - k, c);
      store_row<VEC>(a.state_out + (static_cast<int64_t>(s) * (W - 1) + k) * a.D + c, r);
    }
    return;
  }
  int64_t t = tile * tile_tokens;
  const int64_t t_end = t + tile_tokens < a.runs.total ? t + tile_tokens : a.runs.total;
  int s = first_sequence(a.runs, t);
  if (c >= a.D) return;
  Taps<W, VEC> taps;
  taps.load(a, c);
  while (t < t_end && s < a.runs.n) {
    int64_t begin, len, used;
    if (!run_range(a.runs, s, begin, len, used) || begin > t || begin + len <= t) {
      // a malformed entry, or a gap between sequences: its rows are not written
      const int64_t next = begin > t ? begin : t;
      if (begin <= t) ++s;
      t = next;
      continue;
    }
    const int64_t end = begin + len < t_end ? begin + len : t_end;
    Row<VEC> held[W - 1], x[AHEAD], next[AHEAD];
#pragma unroll
    for (int k = 0; k < W - 1; ++k)
      held[k] = earlier_row<W, VEC>(a, s, t, t - begin, W - 1 - k, c);
    const kda_bf16 *in = a.x + t * a.ldx + c;
    kda_bf16 *out = a.o + t * a.ldo + c;
    int left = static_cast<int>(end - t);
    auto load = [&](Row<VEC> (&to)[AHEAD], int n) {
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) to[i] = i < n ? load_row<VEC>(in + i * a.ldx) : zero_row<VEC>();
      in += AHEAD * a.ldx;
    };
    load(x, left);
    for (; left > 0; left -= AHEAD, out += AHEAD * a.ldo) {
      load(next, left - AHEAD);
      taps.apply(held, x, a.act);  // (after a last, shorter step `held` is not used any more)
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        if (i < left) store_row<VEC>(out + i * a.ldo, x[i]);
        x[i] = next[i];
      }
    }
    t = end;
    if (t < t_end) ++s;
  }
}

// Token runs on the pool: block = (run, channels), channels fastest.
template <int W, int VEC, int AHEAD>
__global__ void __launch_bounds__(kConvThreads) conv_tokens_kernel(const ConvArgs a, int c_blocks) {
  const int b = blockIdx.x / c_blocks;
  const int c = (static_cast<int>(blockIdx.x % c_blocks) * kConvThreads + threadIdx.x) * VEC;
  if (c >= a.D) return;
  int64_t begin, len, used;
  const int64_t slot = a.slots ? a.slots[b] : b;
  if (!run_range(a.runs, b, begin, len, used) || slot < 0 || slot >= a.n_slots) {
    if (c == 0) atomicOr(a.status, KDA_ERR_SHAPE);
    return;
  }
  Taps<W, VEC> taps;
  Row<VEC> held[W - 1], last[W - 1];
#pragma unroll
  for (int k = 0; k < W - 1; ++k)
    last[k] = held[k] = load_held<VEC>(a.state_in + (slot * (W - 1) + k) * a.D + c);
  if (a.o) {
    taps.load(a, c);
    for (int64_t t = 0; t < used; t += AHEAD) {
      Row<VEC> x[AHEAD];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i)
        x[i] = t + i < used ? load_row<VEC>(a.x + (begin + t + i) * a.ldx + c) : zero_row<VEC>();
      taps.apply(held, x, a.act);
#pragma unroll
      for (int i = 0; i < AHEAD; ++i)
        if (t + i < used) store_row<VEC>(a.o + (begin + t + i) * a.ldo + c, x[i]);
    }
    for (int64_t t = used; t < len; ++t)
      store_row<VEC>(a.o + (begin + t) * a.ldo + c, zero_row<VEC>());
  }
  if (a.state_out && used > 0) {
    // the last W - 1 of [held rows ; used rows of x]
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
      const int64_t t = used - (W - 1) + k;
      Row<VEC> r;
      if (t >= 0) {
        r = load_row<VEC>(a.x + (begin + t) * a.ldx + c);
      } else {
        r = last[W - 2];
#pragma unroll
        for (int i = W - 3; i >= 0; --i)
#pragma unroll
          for (int q = 0; q < Taps<W, VEC>::PAIRS; ++q)
            r.w[q] = used + k <= i ? last[i].w[q] : r.w[q];
      }
      store_row<VEC>(a.state_out + (slot * (W - 1) + k) * a.D + c, r);
    }
  }
}

// Vectors of 8 channels where every row starts on a 16-byte boundary, single channels otherwise.
bool vector_rows(const ConvArgs &a) {
  return a.D % 8 == 0 && a.ldx % 8 == 0 && a.ldo % 8 == 0 && aligned16(a.x) && aligned16(a.o) &&
         aligned16(a.weight) && aligned16(a.bias) && aligned16(a.state_in) &&
         aligned16(a.state_out);
}

// Tokens of a tile, 8 to 64: as many as leave 1024 threads to every SM (a tile reads W - 1 rows in front
// of its own again).
constexpr int64_t kTargetThreads = 152 * 1024;

template <int W, int VEC>
cudaError_t conv_fwd_run(const ConvArgs &a, cudaStream_t st) {
  const int c_blocks = (a.D / VEC + kConvThreads - 1) / kConvThreads;
  int tile_tokens = 8;
  while (tile_tokens < 64 &&
         a.runs.total * c_blocks * kConvThreads >= 2 * tile_tokens * kTargetThreads)
    tile_tokens *= 2;
  const int64_t tiles = (a.runs.total + tile_tokens - 1) / tile_tokens;
  const int64_t blocks = (tiles + a.runs.n) * c_blocks;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  conv_fwd_kernel<W, VEC><<<static_cast<unsigned>(blocks), kConvThreads, 0, st>>>(a, c_blocks, tiles,
                                                                                tile_tokens);
  return cudaGetLastError();
}

template <int W, int VEC>
cudaError_t conv_tokens_run(const ConvArgs &a, cudaStream_t st) {
  const int c_blocks = (a.D / VEC + kConvThreads - 1) / kConvThreads;
  const int64_t blocks = static_cast<int64_t>(a.runs.n) * c_blocks;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  const unsigned grid = static_cast<unsigned>(blocks);
  if (a.runs.fixed_len == 1)
    conv_tokens_kernel<W, VEC, 1><<<grid, kConvThreads, 0, st>>>(a, c_blocks);
  else
    conv_tokens_kernel<W, VEC, 4><<<grid, kConvThreads, 0, st>>>(a, c_blocks);
  return cudaGetLastError();
}

}  // namespace

cudaError_t conv_fwd_launch(const ConvArgs &a, int W, cudaStream_t st) {
  const bool v = vector_rows(a);
  if (W == 2) return v ? conv_fwd_run<2, 8>(a, st) : conv_fwd_run<2, 1>(a, st);
  if (W == 3) return v ? conv_fwd_run<3, 8>(a, st) : conv_fwd_run<3, 1>(a, st);
  return v ? conv_fwd_run<4, 8>(a, st) : conv_fwd_run<4, 1>(a, st);
}

cudaError_t conv_tokens_launch(const ConvArgs &a, int W, cudaStream_t st) {
  const bool v = vector_rows(a);
  if (W == 2) return v ? conv_tokens_run<2, 8>(a, st) : conv_tokens_run<2, 1>(a, st);
  if (W == 3) return v ? conv_tokens_run<3, 8>(a, st) : conv_tokens_run<3, 1>(a, st);
  return v ? conv_tokens_run<4, 8>(a, st) : conv_tokens_run<4, 1>(a, st);
}

}  // namespace kda

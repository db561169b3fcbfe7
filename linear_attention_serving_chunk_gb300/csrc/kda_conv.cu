// Short causal depthwise convolution over packed prompts, and over token runs on a pool of the
// sequences' last inputs.
//
//   o_t[c] = act(bias[c] + sum_{w < W} weight[c, w] x_{t - (W - 1) + w}[c]),  act = silu or identity
//
// with the W - 1 held rows (or zeros) in front of a sequence's first token.  Both kernels are bound
// by memory: x is read once and o written once.  A thread owns VEC neighbouring channels and walks
// along the tokens with the last W - 1 rows in registers, so that a row is loaded once, as one
// 16-byte vector where the layout allows it.
#include "kda_serving.cuh"

namespace kda {

namespace {

constexpr int kConvThreads = 128;

template <int VEC>
struct Row {  // VEC bf16 channels of one row
  kda_bf16 v[VEC];
};

template <int VEC>
__device__ __forceinline__ Row<VEC> load_row(const kda_bf16 *p) {
  Row<VEC> r;
  if constexpr (VEC == 8) {
    *reinterpret_cast<uint4 *>(r.v) = *reinterpret_cast<const uint4 *>(p);
  } else {
    r.v[0] = *p;
  }
  return r;
}

template <int VEC>
__device__ __forceinline__ void store_row(kda_bf16 *p, const Row<VEC> &r) {
  if constexpr (VEC == 8)
    *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<const uint4 *>(r.v);
  else
    *p = r.v[0];
}

template <int VEC>
__device__ __forceinline__ Row<VEC> zero_row() {
  Row<VEC> r;
#pragma unroll
  for (int i = 0; i < VEC; ++i) r.v[i] = 0;
  return r;
}

template <int W, int VEC>
struct Taps {
  float w[W][VEC], b[VEC];

  __device__ __forceinline__ void load(const ConvArgs &a, int c) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
#pragma unroll
      for (int k = 0; k < W; ++k) w[k][i] = bf2f(a.weight[static_cast<size_t>(c + i) * W + k]);
      b[i] = a.bias ? bf2f(a.bias[c + i]) : 0.f;
    }
  }
  // one output row from the W - 1 rows before it (oldest first) and its own
  __device__ __forceinline__ Row<VEC> apply(const Row<VEC> (&held)[W - 1], const Row<VEC> &x,
                                            int act) const {
    Row<VEC> o;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      float s = b[i];
#pragma unroll
      for (int k = 0; k < W - 1; ++k) s = fmaf(w[k][i], bf2f(held[k].v[i]), s);
      s = fmaf(w[W - 1][i], bf2f(x.v[i]), s);
      o.v[i] = f2bf(act ? silu(s) : s);
    }
    return o;
  }
};

template <int W, int VEC>
__device__ __forceinline__ void shift(Row<VEC> (&held)[W - 1], const Row<VEC> &x) {
#pragma unroll
  for (int k = 0; k < W - 2; ++k) held[k] = held[k + 1];
  held[W - 2] = x;
}

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

// Packed prompts.  Block = (tile, channels), channels fastest: `tile_tokens` tokens from
// tile * tile_tokens on; the blocks behind the tiles write one sequence's final rows each.
template <int W, int VEC>
__global__ void __launch_bounds__(kConvThreads)
conv_fwd_kernel(const ConvArgs a, int c_blocks, int64_t tiles, int tile_tokens) {
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
  if (c >= a.D) return;
  int64_t t = tile * tile_tokens;
  const int64_t t_end = t + tile_tokens < a.runs.total ? t + tile_tokens : a.runs.total;
  // the tile's first sequence: the number of sequences that end at or before t
  int s;
  if (a.runs.cu) {
    int lo = 0, hi = a.runs.n;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (a.runs.cu[mid + 1] <= t)
        lo = mid + 1;
      else
        hi = mid;
    }
    s = lo;
  } else {
    s = static_cast<int>(t / a.runs.fixed_len);
  }
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
    Row<VEC> held[W - 1];
#pragma unroll
    for (int k = 0; k < W - 1; ++k)
      held[k] = earlier_row<W, VEC>(a, s, t, t - begin, W - 1 - k, c);
    const kda_bf16 *x = a.x + t * a.ldx + c;
    kda_bf16 *o = a.o + t * a.ldo + c;
    for (; t < end; ++t, x += a.ldx, o += a.ldo) {
      const Row<VEC> r = load_row<VEC>(x);
      store_row<VEC>(o, taps.apply(held, r, a.act));
      shift<W, VEC>(held, r);
    }
    if (t < t_end) ++s;
  }
}

// Token runs on the pool: block = (run, channels), channels fastest.
template <int W, int VEC>
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
  taps.load(a, c);
  Row<VEC> held[W - 1];
#pragma unroll
  for (int k = 0; k < W - 1; ++k)
    held[k] = load_row<VEC>(a.state_in + (slot * (W - 1) + k) * a.D + c);
  for (int64_t t = 0; t < used; ++t) {
    const Row<VEC> r = load_row<VEC>(a.x + (begin + t) * a.ldx + c);
    if (a.o) store_row<VEC>(a.o + (begin + t) * a.ldo + c, taps.apply(held, r, a.act));
    shift<W, VEC>(held, r);
  }
  if (a.o)
    for (int64_t t = used; t < len; ++t)
      store_row<VEC>(a.o + (begin + t) * a.ldo + c, zero_row<VEC>());
  if (a.state_out && used > 0)
#pragma unroll
    for (int k = 0; k < W - 1; ++k)
      store_row<VEC>(a.state_out + (slot * (W - 1) + k) * a.D + c, held[k]);
}

// Vectors of 8 channels where every row starts on a 16-byte boundary, single channels otherwise.
bool vector_rows(const ConvArgs &a) {
  return a.D % 8 == 0 && a.ldx % 8 == 0 && a.ldo % 8 == 0 && aligned16(a.x) && aligned16(a.o) &&
         aligned16(a.state_in) && aligned16(a.state_out);
}

template <int W, int VEC>
cudaError_t conv_fwd_run(const ConvArgs &a, cudaStream_t st) {
  const int tile_tokens = 32;
  const int64_t tiles = (a.runs.total + tile_tokens - 1) / tile_tokens;
  const int c_blocks = (a.D / VEC + kConvThreads - 1) / kConvThreads;
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
  conv_tokens_kernel<W, VEC><<<static_cast<unsigned>(blocks), kConvThreads, 0, st>>>(a, c_blocks);
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

// Writes the keys and values of a batch of runs into the pages of their sequences.
//
// Bound by memory: each row of k and v is read once and written once.  A block takes kVectors 16-byte
// vectors a thread of consecutive tokens; the run, slot and page of each of its tokens are looked up
// once, by one thread each, and the vectors are all in flight before the first is stored.  44 us for 32,768
// packed tokens of 8 heads of 128 (268 MB, 6.1 TB/s); with 8 vectors a thread 47, with 2 47, with blocks
// of 512 threads 51, with streaming loads or stores no change.
#include "kda_paged.cuh"
#include "kda_pdl.cuh"

namespace kda {

namespace {

constexpr int kThreads = 256;
constexpr int kVectors = 4;
constexpr int kTokens = kThreads * kVectors / 16 + 1;  // of a block: a token has 16 vectors at least

// Place of token t's first key in the cache, in elements: -1 where it has none.
__device__ int64_t place(const AppendArgs &a, int64_t t) {
  const Runs &r = a.runs;
  int64_t begin, end;
  int b;
  if (r.cu) {
    int lo = 0, hi = r.n;  // the last run that starts at or before t
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (r.cu[mid] <= t) lo = mid;
      else hi = mid - 1;
    }
    b = lo;
    if (b == r.n) {  // behind the last run, unless the offsets are malformed
      if (r.cu[b] > t || r.cu[b] < 0) atomicOr(a.status, KDA_ERR_SHAPE);
      return -1;
    }
    const bool ok = seq_range(r.cu, b, r.total, begin, end);
    if (!ok || t < begin || t >= end) {
      if (!(ok && b == 0 && t < begin)) atomicOr(a.status, KDA_ERR_SHAPE);  // (else: in front of the first run)
      return -1;
    }
  } else {
    b = static_cast<int>(t / r.fixed_len);
    begin = b * r.fixed_len;
  }
  const PagedSeqs &s = a.seqs;
  int slot;
  int64_t at;
  bool ok = run_slot(s, b, slot, at);
  at += t - begin;
  const int64_t i = at >> s.page_shift;
  ok = ok && i < s.max_pages;
  const int page = ok ? s.table[static_cast<int64_t>(slot) * s.max_pages + i] : -1;
  if (page < 0 || page >= s.n_pages) {
    atomicOr(a.status, KDA_ERR_SHAPE);
    return -1;
  }
  return (((static_cast<int64_t>(page) * 2 * a.H) << s.page_shift) + (at & ((1 << s.page_shift) - 1))) * a.D;
}

// per_token: vectors of a token, k's heads and then v's; inverse: 1 / per_token.
template <int D>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const AppendArgs a, int per_token, float inverse) {
  __shared__ int64_t where[kTokens];
  grid_launch_dependents();  // (the attention's start, which waits for this kernel's end)
  const int64_t v0 = static_cast<int64_t>(blockIdx.x) * (kThreads * kVectors), t0 = v0 / per_token;
  const int first = static_cast<int>(v0 - t0 * per_token);
  const int tokens = (first + kThreads * kVectors + per_token - 1) / per_token;
  for (int i = threadIdx.x; i < tokens; i += kThreads)
    where[i] = t0 + i < a.runs.total ? place(a, t0 + i) : -1;
  // the rows are read while the places are looked up
  uint4 v[kVectors];
  int token[kVectors];
  int64_t off[kVectors];
  const int half = per_token / 2;
  const int64_t plane = static_cast<int64_t>(D) << a.seqs.page_shift;
#pragma unroll
  for (int j = 0; j < kVectors; ++j) {
    const int x = first + j * kThreads + threadIdx.x;
    // x / per_token, by a product that is off by one at most (the integer division took 1.4 of 45 us)
    int n = static_cast<int>(static_cast<float>(x) * inverse);
    n -= n * per_token > x;
    n += (n + 1) * per_token <= x;
    token[j] = n;
    const int in = x - n * per_token, is_v = in >= half, row = in - (is_v ? half : 0);
    const int h = row / (D / 8), e = row % (D / 8) * 8;
    const int64_t t = t0 + token[j];
    off[j] = (static_cast<int64_t>(is_v ? a.H : 0) + h) * plane + e;
    if (t < a.runs.total)
      v[j] = *reinterpret_cast<const uint4 *>((is_v ? a.v + t * a.ldv : a.k + t * a.ldk) + row * 8);
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kVectors; ++j) {
    const int64_t at = where[token[j]];
    if (at >= 0) *reinterpret_cast<uint4 *>(a.cache + at + off[j]) = v[j];
  }
  // Offsets that decrease between runs that are well-formed by themselves: no look-up of a token sees them.  (In front
  // of the stores it costs 4 of 44 us, in the order of the loads.)
  if (a.runs.cu) {
    bool bad = false;
    for (int64_t b = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; b < a.runs.n;
         b += static_cast<int64_t>(gridDim.x) * kThreads) {
      int64_t begin, end;
      bad |= !seq_range(a.runs.cu, static_cast<int>(b), a.runs.total, begin, end);
    }
    if (bad) atomicOr(a.status, KDA_ERR_SHAPE);
  }
}

}  // namespace

cudaError_t kv_append_launch(const AppendArgs &a, cudaStream_t st) {
  const int per_token = 2 * a.H * a.D / 8;
  const int64_t blocks = (a.runs.total * per_token + kThreads * kVectors - 1) / (kThreads * kVectors);
  const dim3 grid(static_cast<unsigned>(blocks));
  if (a.D == 64) kv_append_kernel<64><<<grid, kThreads, 0, st>>>(a, per_token, 1.f / per_token);
  else kv_append_kernel<128><<<grid, kThreads, 0, st>>>(a, per_token, 1.f / per_token);
  return cudaGetLastError();
}

}  // namespace kda

// Verification of drafted tokens against the target's probabilities, from given random numbers.
//
// Run b is the last accepted token and k drafted ones; row j of the target judges token j + 1.
// Draft j is accepted while u_j q_j(x) < p_j(x).  At the first refusal the next token comes from
// max(p - q, 0) (from p where that is zero everywhere), after k acceptances from the target's last
// row, by the inverse distribution: the smallest i with w_0 + ... + w_i > u (sum of w).
//
// Bound by memory: one row of p (and of q) per run is read.  A cluster of CTAs shares a run's row.
// Which token a sum lands on must hardly depend on the order of the additions, so sums carry 43 bits
// at least: a lane adds its elements in fp32 together with what the roundings lost (double-precision
// adds run at 2 per SM and cycle here, below the rate at which elements arrive), everything above a
// lane is in double precision.  The row is cut into segments of kSeg elements whose sums stay in
// shared memory; the segment that the target falls into is read a second time, from L2, 32
// neighbouring elements a lane, and then the 32 of the lane that it falls into, one a lane.
//
// 256 runs over 131072 words in fp32: 43.0 us for the 190 MB of the rows that this batch needs, 4.4 TB/s
// (with what the roundings lost in one fp32 sum, right to 38 bits in the worst case, 42.5; with that sum
// kept exact element by element, 47 bits, 52).  A few runs over 32000 words take 11 us on the device, a chain of dependent reads (offsets, drafted tokens,
// their probabilities, the row, its two searches).  CTAs of 256 threads, two of them for a row at
// this size: four took 47 us, one of 512 threads 44; four vectors in flight a lane: two took 46, eight 51.
#include "kda_serving.cuh"

namespace kda {

namespace {

constexpr int kVThreads = 256;
constexpr int kVWarps = kVThreads / 32;
constexpr int kSeg = 1024;

__device__ __forceinline__ unsigned cluster_rank() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ unsigned cluster_size() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A double in the shared memory of CTA `rank` of this cluster, at this CTA's address `p`.
__device__ __forceinline__ double peer_load(const double *p, unsigned rank) {
  uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(p)), there;
  double v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(at), "r"(rank));
  asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(there) : "memory");
  return v;
}

__device__ __forceinline__ float prob(const float *p, int64_t i) { return p[i]; }
__device__ __forceinline__ float prob(const kda_bf16 *p, int64_t i) { return bf2f(p[i]); }

__device__ __forceinline__ float minus(float a, float b) { return a - b; }
__device__ __forceinline__ float2 minus(float2 a, float2 b) {
  return __ffma2_rn(b, make_float2(-1.f, -1.f), a);
}
__device__ __forceinline__ float plus(float a, float b) { return a + b; }
__device__ __forceinline__ float2 plus(float2 a, float2 b) { return __fadd2_rn(a, b); }
// a + b rounded, and what the rounding lost
template <typename V>
__device__ __forceinline__ V exact(V a, V b, V &lost) {
  const V s = plus(a, b), r = minus(s, a);
  lost = plus(minus(a, minus(s, r)), minus(b, r));
  return s;
}

// The row's weights: max(p - q, 0), p without one token, or p.  NaN counts as 0.
template <typename T>
struct Weights {
  const T *p, *q;
  int without;  // a token of the row, or -1: none

  // w = hi + lo: the rounded difference, and what its rounding lost
  static __device__ __forceinline__ void weight(float pv, float qv, float &hi, float &lo) {
    hi = fmaxf(pv - qv, 0.f);
    lo = hi > 0.f ? (pv - hi) - qv : 0.f;
  }
  static __device__ __forceinline__ void weight(float2 pv, float2 qv, float2 &hi, float2 &lo) {
    hi = minus(pv, qv);
    hi = make_float2(fmaxf(hi.x, 0.f), fmaxf(hi.y, 0.f));
    lo = minus(minus(pv, hi), qv);
    lo = make_float2(hi.x > 0.f ? lo.x : 0.f, hi.y > 0.f ? lo.y : 0.f);
  }
  __device__ __forceinline__ double one(int i) const {
    float hi, lo;
    weight(prob(p, i), q ? prob(q, i) : 0.f, hi, lo);
    return i == without ? 0.0 : static_cast<double>(hi) + static_cast<double>(lo);
  }
};

// Two sums side by side, hi + lo + tail each: the sum, what its roundings lost, and what the roundings of
// that lost.  With u = 2^-24: four elements of sum g lose 2 u g at most among themselves and u g in their
// differences; adding these seven terms plainly is off by 18 u^2 g, so a lane's sum is right to 18 u^2 = 2^-43.8.
struct Sum {
  float2 hi = {0.f, 0.f}, lo = {0.f, 0.f}, tail = {0.f, 0.f};

  // Four elements each, x with xl lost before: first among themselves, so that what their roundings lose is
  // small against the group and may be added as it is.
  __device__ __forceinline__ void add(const float2 (&x)[4], const float2 (&xl)[4]) {
    float2 a, b, c, d, again;
    const float2 four = exact(exact(x[0], x[1], a), exact(x[2], x[3], b), c);
    hi = exact(hi, four, d);
    a = plus(plus(plus(a, b), c), plus(plus(xl[0], xl[1]), plus(xl[2], xl[3])));
    lo = exact(lo, d, again);
    tail = plus(tail, again);
    lo = exact(lo, a, again);
    tail = plus(tail, again);
  }
  // both sums
  __device__ __forceinline__ double value() const {
    float a, b, c, d;
    const float top = exact(hi.x, hi.y, a), low = exact(exact(lo.x, lo.y, b), a, c);
    const float sum = exact(top, low, d);
    return static_cast<double>(sum) + static_cast<double>(d + ((tail.x + tail.y) + (b + c)));
  }
};

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// inclusive prefix sums over the lanes
__device__ __forceinline__ double warp_scan(double v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double w = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += w;
  }
  return v;
}

// One lane's elements of segment [i0, i0 + kSeg) of the row: SPREAD, vectors of the 32 lanes side by
// side; otherwise 32 neighbouring ones a lane.
template <typename T, bool VECTOR, bool SPREAD>
__device__ __forceinline__ double segment_sum(const Weights<T> &w, int i0, int V, int lane) {
  // The one segment that holds the token taken out is added element by element, without it (in double
  // precision: what is left of it may be far smaller than that token's weight).
  if (static_cast<unsigned>(w.without - i0) < kSeg) {
    double v = 0.0;
#pragma unroll 4
    for (int k = 0; k < kSeg / 32; ++k) {
      const int i = i0 + (SPREAD ? k * 32 + lane : lane * 32 + k);
      if (i < V) v += w.one(i);
    }
    return v;
  }
  Sum s;
  if constexpr (VECTOR) {
    constexpr int E = 16 / sizeof(T), STEPS = kSeg / (32 * E), AHEAD = STEPS < 4 ? STEPS : 4;
    const int first = i0 + lane * (SPREAD ? E : 32);
    constexpr int STEP = SPREAD ? 32 * E : E;
#pragma unroll
    for (int k0 = 0; k0 < STEPS; k0 += AHEAD) {
      uint4 pv[AHEAD], qv[AHEAD];
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        const int i = first + (k0 + k) * STEP;
        pv[k] = qv[k] = make_uint4(0, 0, 0, 0);
        if (i < V) {
          pv[k] = __ldg(reinterpret_cast<const uint4 *>(w.p + i));
          if (w.q) qv[k] = __ldg(reinterpret_cast<const uint4 *>(w.q + i));
        }
      }
#pragma unroll
      for (int g = 0; g < AHEAD * E; g += 8) {
        float2 hi[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const T *pe = reinterpret_cast<const T *>(pv) + g + 2 * e, *qe = reinterpret_cast<const T *>(qv) + g + 2 * e;
          Weights<T>::weight(make_float2(prob(pe, 0), prob(pe, 1)), make_float2(prob(qe, 0), prob(qe, 1)),
                             hi[e], lo[e]);
        }
        s.add(hi, lo);
      }
    }
  } else {
#pragma unroll 1
    for (int k = 0; k < kSeg / 32; k += 8) {
      float pv[8], qv[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int i = i0 + (SPREAD ? (k + e) * 32 + lane : lane * 32 + k + e);
        pv[e] = qv[e] = 0.f;
        if (i < V) {
          pv[e] = prob(w.p, i);
          if (w.q) qv[e] = prob(w.q, i);
        }
      }
      float2 hi[4], lo[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        Weights<T>::weight(make_float2(pv[2 * e], pv[2 * e + 1]), make_float2(qv[2 * e], qv[2 * e + 1]),
                           hi[e], lo[e]);
      s.add(hi, lo);
    }
  }
  return s.value();
}

template <typename T, bool VECTOR>
__global__ void __launch_bounds__(kVThreads) verify_kernel(const VerifyArgs a) {
  extern __shared__ double s_seg[];  // sums of this CTA's segments
  __shared__ double s_total;
  __shared__ int s_got;
  const unsigned rank = cluster_rank(), ranks = cluster_size();
  const int b = blockIdx.x / ranks;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const T *target = static_cast<const T *>(a.target), *draft = static_cast<const T *>(a.draft);
  int64_t t0, t1;
  // every run has its last accepted token; the whole cluster takes the same way out
  if (!seq_range(a.cu, b, a.total, t0, t1) || t1 == t0 || t0 < b ||
      t1 - b - 1 > a.total - a.n) {
    if (rank == 0 && tid == 0) {
      atomicOr(a.status, KDA_ERR_SHAPE);
      a.n_out[b] = 0;
    }
    return;
  }
  const int k = static_cast<int>(t1 - t0) - 1;
  if (warp == 0) {
    int got = k;
    for (int j0 = 0; j0 < k && got == k; j0 += 32) {
      const int j = j0 + lane;
      bool refused = false;
      if (j < k) {
        const int x = a.tokens[t0 + j + 1];
        refused = true;
        if (x >= 0 && x < a.V) {
          const double p = prob(target, (t0 + j) * a.V + x);
          const double q = draft ? prob(draft, (t0 - b + j) * a.V + x) : 1.0;
          refused = !(static_cast<double>(a.u[t0 + j]) * q < p);
        } else if (rank == 0) {
          atomicOr(a.status, KDA_ERR_SHAPE);
        }
      }
      const unsigned m = __ballot_sync(0xffffffffu, refused);
      if (m) got = j0 + __ffs(m) - 1;
    }
    if (lane == 0) s_got = got;
  }
  __syncthreads();
  const int got = s_got;
  const bool cut = got < k;
  if (rank == 0)
    for (int j = tid; j <= k; j += kVThreads)
      if (j != got) a.out_tokens[t0 + j] = j < got ? a.tokens[t0 + j + 1] : -1;

  Weights<T> w{target + (t0 + got) * a.V, cut && draft ? draft + (t0 - b + got) * a.V : nullptr, -1};
  if (cut && !draft) {
    const int x = a.tokens[t0 + got + 1];
    if (x >= 0 && x < a.V) w.without = x;  // (a token outside the row has no weight to take out)
  }
  const int segs = (a.V + kSeg - 1) / kSeg;
  const int seg0 = static_cast<int>(static_cast<int64_t>(segs) * rank / ranks);
  const int seg1 = static_cast<int>(static_cast<int64_t>(segs) * (rank + 1) / ranks);
  double total = 0.0, before = 0.0;
  for (int pass = 0; pass < 2; ++pass) {
    for (int s = seg0 + warp; s < seg1; s += kVWarps) {
      const double v = warp_sum(segment_sum<T, VECTOR, true>(w, s * kSeg, a.V, lane));
      if (lane == 0) s_seg[s - seg0] = v;
    }
    if (pass > 0) cluster_wait();  // every CTA has read the first totals
    __syncthreads();
    if (warp == 0) {
      double sum = 0.0;
      for (int s = 0; s < seg1 - seg0; s += 32)
        sum += __shfl_sync(0xffffffffu,
                           warp_scan(s + lane < seg1 - seg0 ? s_seg[s + lane] : 0.0, lane), 31);
      if (lane == 0) s_total = sum;
    }
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    total = before = 0.0;
    for (unsigned r = 0; r < ranks; ++r) {
      if (r == rank) before = total;
      total += peer_load(&s_total, r);
    }
    cluster_arrive();  // waited for before s_total goes
    if (total > 0.0 || (!w.q && w.without < 0)) break;
    w.q = nullptr;  // nothing is left of the row: the target's own weights
    w.without = -1;
  }
  if (!(total > 0.0 && total < 1e300)) {
    if (rank == 0 && tid == 0) {
      atomicOr(a.status, KDA_ERR_RANGE);
      a.out_tokens[t0 + got] = -1;
      a.n_out[b] = got;
    }
  } else if (warp == 0) {
    const float u = a.u[t1 - 1];
    const double want = static_cast<double>(u >= 0.f ? fminf(u, 0x1.fffffep-1f) : 0.f) * total;
    // the CTA whose part of the row holds it
    if (want >= before && want < before + s_total) {
      double sum = before;
      int seg = -1;
      for (int s = 0; s < seg1 - seg0 && seg < 0; s += 32) {
        const double c = warp_scan(s + lane < seg1 - seg0 ? s_seg[s + lane] : 0.0, lane);
        const unsigned m = __ballot_sync(0xffffffffu, sum + c > want);
        const int at = m ? __ffs(m) - 1 : 32;  // lanes in front of it count in full
        const double front = __shfl_sync(0xffffffffu, c, (at + 31) & 31);
        if (m) seg = s + at;
        if (at > 0) sum += front;
      }
      if (seg < 0) seg = seg1 - seg0 - 1;  // rounding of the sums alone
      const int i0 = (seg0 + seg) * kSeg;
      double mine = segment_sum<T, VECTOR, false>(w, i0, a.V, lane);
      double c = warp_scan(mine, lane);
      unsigned over = __ballot_sync(0xffffffffu, mine > 0.0 && sum + c > want);
      unsigned some = __ballot_sync(0xffffffffu, mine > 0.0);
      const int from = over ? __ffs(over) - 1 : some ? 31 - __clz(some) : 0;
      sum += __shfl_sync(0xffffffffu, c - mine, from);
      const int i = i0 + from * 32 + lane;
      mine = i < a.V ? w.one(i) : 0.0;
      c = warp_scan(mine, lane);
      over = __ballot_sync(0xffffffffu, mine > 0.0 && sum + c > want);
      some = __ballot_sync(0xffffffffu, mine > 0.0);
      if (lane == (over ? __ffs(over) - 1 : some ? 31 - __clz(some) : 0)) {
        a.out_tokens[t0 + got] = i;
        a.n_out[b] = got + 1;
      }
    }
  }
  __syncwarp();
  cluster_wait();
}

template <typename T, bool VECTOR>
cudaError_t run(const VerifyArgs &a, cudaStream_t st) {
  const int segs = (a.V + kSeg - 1) / kSeg;
  int ranks = 1;
  while (ranks < 8 && a.n * ranks < 2 * 152 && ranks * kVWarps < segs) ranks *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.n) * ranks);
  cfg.blockDim = dim3(kVThreads);
  cfg.dynamicSmemBytes = ((segs + ranks - 1) / ranks) * sizeof(double);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, verify_kernel<T, VECTOR>, a);
}

}  // namespace

cudaError_t verify_launch(const VerifyArgs &a, bool half, cudaStream_t st) {
  const size_t size = half ? 2 : 4;
  // 16-byte loads where every row starts on a 16-byte boundary
  const bool v = a.V * size % 16 == 0 && aligned16(a.target) && aligned16(a.draft);
  if (half) return v ? run<kda_bf16, true>(a, st) : run<kda_bf16, false>(a, st);
  return v ? run<float, true>(a, st) : run<float, false>(a, st);
}

}  // namespace kda

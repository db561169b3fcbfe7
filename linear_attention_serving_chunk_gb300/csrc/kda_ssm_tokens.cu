// Selective state space recurrence token by token, on states held in registers.
//
// Per (run, head), with an N x P fp32 state S, group g = h / (H / G):
//   dt = softplus(raw + dt_bias),  a = exp(dt A_h)
//   S <- a S + B (dt x)^T,   o = (S^T C + D_h x) silu(z)
//
// Bound by memory for short runs: a state is read once and, with commit, written once.  One CTA owns one
// state; TPR = P / 4 of its threads lie along a row (4 columns each) and its row groups along N, as in the
// KDA decode step.  The tokens of a run are staged TB at a time (B, C and x in fp32), a thread then takes
// its block of the state through all of them and leaves its part of S^T C per token in shared memory: two
// barriers per TB tokens.  The arithmetic is packed fp32x2 over column pairs.
//
// One token on 512 x 32 states of 128 x 128: 315 us, 6.85 TB/s, the rate of a plain copy.  Runs of 1 to 5
// tokens without commit on 256 x 32 states of 128 x 64: 60 us, 4.6 TB/s.  There a CTA's own chain counts
// (offsets, rows, a barrier, the tokens, a barrier, the result) against the states that an SM has on their
// way meanwhile; a quarter fewer instructions per token changed nothing.
//
// A decay near 1 is applied as S + ((a - 1) S + B dt x) with a - 1 from expm1: rounded to fp32, a itself
// is off by up to 2^-24 the same way at every token, which over the hundreds of tokens that such a
// state remembers adds up to several 1e-6.  Below 1/2, where a S loses nothing, a is used as it is.
#include "kda_serving.cuh"

namespace kda {

namespace {

// Threads of a CTA, and CTAs that an SM is to hold: 64 values of the state a thread and as many states on
// their way as the registers allow.  (Runs on 128 x 64 states: 5 CTAs of 128 threads 60 us, 4 of 256 threads
// 65, 4 of 128 threads 68, 6 spill; one token on 128 x 128 states: 2 of 256 threads 315, 128 threads 322.)
constexpr int threads_of(int state) { return state > 8192 ? 256 : 128; }
constexpr int ctas_of(int state) { return state > 8192 ? 2 : state > 4096 ? 5 : 8; }

template <int N, int P, int TB>
__global__ void __launch_bounds__(threads_of(N * P), ctas_of(N * P))
ssm_tokens_kernel(const SsmArgs a) {
  constexpr int kThreads = threads_of(N * P), kWarps = kThreads / 32;
  constexpr int TPR = P / 4;           // threads along a row
  constexpr int RG = kThreads / TPR;   // row groups
  constexpr int RPT = N / RG;          // rows per thread
  constexpr int RGW = 32 / TPR;        // row groups of one warp
  static_assert(RPT * RG == N && TPR * RG == kThreads, "state tiling");
  __shared__ float2 s_bc[TB][N];       // (B, C)
  __shared__ float4 s_x[TB][TPR];
  __shared__ float4 s_a[TB];           // S <- k S + (m S + B dt x): (k, m) = (1, a - 1) or (0, a); dt
  __shared__ float4 s_part[TB][kWarps][TPR];

  const int b = blockIdx.x / a.H, h = blockIdx.x % a.H, g = h / (a.H / a.G);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cg = tid % TPR, rg = tid / TPR;
  int64_t begin, len, used;
  const int64_t slot = a.slots ? a.slots[b] : b;
  if (!run_range(a.runs, b, begin, len, used) || slot < 0 || slot >= a.n_slots) {
    if (h == 0 && tid == 0) atomicOr(a.status, KDA_ERR_SHAPE);
    return;
  }
  const size_t at = (static_cast<size_t>(slot) * a.H + h) * (N * P) +
                    static_cast<size_t>(rg) * RPT * P + 4 * cg;
  float2 s[RPT][2];
#pragma unroll
  for (int r = 0; r < RPT; ++r) {
    const float4 v = __ldcs(reinterpret_cast<const float4 *>(a.S_in + at + r * P));
    s[r][0] = make_float2(v.x, v.y);
    s[r][1] = make_float2(v.z, v.w);
  }
  const float A = a.A[h], D = a.D ? a.D[h] : 0.f;

  for (int64_t t0 = 0; t0 < used; t0 += TB) {
    const int nt = used - t0 < TB ? static_cast<int>(used - t0) : TB;
    const int64_t row0 = begin + t0;
    if (t0 > 0) __syncthreads();
    const int mine = tid - kThreads / 2;  // (the ends of the block stage the rows of one token)
    if (mine >= 0 && mine < nt) {
      const float dt = ssm_dt(a, row0 + mine, h), m = expm1f(dt * A);
      s_a[mine] = m > -0.5f ? make_float4(1.f, m, dt, 0.f) : make_float4(0.f, expf(dt * A), dt, 0.f);
    }
    for (int i = tid; i < nt * (N / 2); i += kThreads) {
      const int t = i / (N / 2), n = 2 * (i % (N / 2));
      const uint32_t B = *reinterpret_cast<const uint32_t *>(a.B + (row0 + t) * a.ldb + g * N + n);
      const uint32_t C = *reinterpret_cast<const uint32_t *>(a.C + (row0 + t) * a.ldc + g * N + n);
      const float b0 = __uint_as_float(B << 16), b1 = __uint_as_float(B & 0xffff0000u);
      const float c0 = __uint_as_float(C << 16), c1 = __uint_as_float(C & 0xffff0000u);
      *reinterpret_cast<float4 *>(&s_bc[t][n]) = make_float4(b0, c0, b1, c1);
    }
    for (int i = kThreads - 1 - tid; i < nt * (P / 2); i += kThreads) {
      const int t = i / (P / 2), p = i % (P / 2);
      const uint32_t x =
          reinterpret_cast<const uint32_t *>(a.x + (row0 + t) * a.ldx + h * P)[p];
      reinterpret_cast<float2 *>(s_x[t])[p] =
          make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
    }
    __syncthreads();
    for (int t = 0; t < nt; ++t) {
      const float4 km = s_a[t], x = s_x[t][cg];
      const float2 k2 = make_float2(km.x, km.x), m2 = make_float2(km.y, km.y),
                   dt2 = make_float2(km.z, km.z);
      const float2 x0 = __fmul2_rn(dt2, make_float2(x.x, x.y)),
                   x1 = __fmul2_rn(dt2, make_float2(x.z, x.w));
      float2 y0 = make_float2(0.f, 0.f), y1 = y0;
#pragma unroll
      for (int r = 0; r < RPT; ++r) {
        const float2 bc = s_bc[t][rg * RPT + r];
        const float2 B2 = make_float2(bc.x, bc.x), C2 = make_float2(bc.y, bc.y);
        s[r][0] = __ffma2_rn(k2, s[r][0], __ffma2_rn(m2, s[r][0], __fmul2_rn(B2, x0)));
        s[r][1] = __ffma2_rn(k2, s[r][1], __ffma2_rn(m2, s[r][1], __fmul2_rn(B2, x1)));
        y0 = __ffma2_rn(C2, s[r][0], y0);
        y1 = __ffma2_rn(C2, s[r][1], y1);
      }
      if constexpr (RGW == 2) {
        y0.x += __shfl_xor_sync(0xffffffffu, y0.x, 16);
        y0.y += __shfl_xor_sync(0xffffffffu, y0.y, 16);
        y1.x += __shfl_xor_sync(0xffffffffu, y1.x, 16);
        y1.y += __shfl_xor_sync(0xffffffffu, y1.y, 16);
      }
      if (lane < TPR) s_part[t][warp][cg] = make_float4(y0.x, y0.y, y1.x, y1.y);
    }
    __syncthreads();
    if (a.o)
      for (int i = tid; i < nt * (P / 2); i += kThreads) {
        const int t = i / (P / 2), p = i % (P / 2);
        const float2 x = reinterpret_cast<const float2 *>(s_x[t])[p];
        float2 y = __fmul2_rn(make_float2(D, D), x);
#pragma unroll
        for (int w = 0; w < kWarps; ++w)
          y = __fadd2_rn(y, reinterpret_cast<const float2 *>(s_part[t][w])[p]);
        if (a.z) {
          const uint32_t z =
              reinterpret_cast<const uint32_t *>(a.z + (row0 + t) * a.ldz + h * P)[p];
          y.x *= silu(__uint_as_float(z << 16));
          y.y *= silu(__uint_as_float(z & 0xffff0000u));
        }
        const __nv_bfloat162 r = __floats2bfloat162_rn(y.x, y.y);
        reinterpret_cast<uint32_t *>(a.o + (row0 + t) * a.ldo + h * P)[p] =
            *reinterpret_cast<const uint32_t *>(&r);
      }
  }
  if (a.o)
    for (int64_t i = used * P + tid; i < len * P; i += kThreads)
      a.o[(begin + i / P) * a.ldo + h * P + i % P] = 0;
  if (a.S_out && used > 0)
#pragma unroll
    for (int r = 0; r < RPT; ++r)
      __stcs(reinterpret_cast<float4 *>(a.S_out + at + r * P),
             make_float4(s[r][0].x, s[r][0].y, s[r][1].x, s[r][1].y));
}

template <int N, int P>
cudaError_t run(const SsmArgs &a, bool single, cudaStream_t st) {
  const unsigned grid = static_cast<unsigned>(a.runs.n) * a.H;
  constexpr int threads = threads_of(N * P);
  if (single)
    ssm_tokens_kernel<N, P, 1><<<grid, threads, 0, st>>>(a);
  else
    ssm_tokens_kernel<N, P, N * P <= 8192 ? 8 : 4><<<grid, threads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t ssm_tokens_launch(const SsmArgs &a, int P, int N, bool single, cudaStream_t st) {
  if (N == 64) return P == 64 ? run<64, 64>(a, single, st) : run<64, 128>(a, single, st);
  return P == 64 ? run<128, 64>(a, single, st) : run<128, 128>(a, single, st);
}

}  // namespace kda

// Arguments that the kernels of the state space layer (short convolution, selective scan) and of
// draft verification take by value, and the small device functions that they share.
#pragma once

#include "kda_common.cuh"

namespace kda {

// A batch of token runs: rows [cu[b], cu[b + 1]) of packed tensors, or fixed_len tokens each
// where cu is NULL.  `used` (NULL: all) cuts every run to its first used[b] tokens.
struct Runs {
  const int32_t *cu;
  const int32_t *used;
  int n;
  int64_t total, fixed_len;
};

// Token range [b, b + len) of run s, and how many of them are used.  false for a malformed entry
// (an empty run; the caller records KDA_ERR_SHAPE).
__device__ __forceinline__ bool run_range(const Runs &r, int s, int64_t &begin, int64_t &len,
                                          int64_t &used) {
  int64_t end;
  bool ok = true;
  if (r.cu) {
    ok = seq_range(r.cu, s, r.total, begin, end);
  } else {
    begin = static_cast<int64_t>(s) * r.fixed_len;
    end = begin + r.fixed_len;
  }
  used = len = end - begin;
  if (r.used && ok) {
    const int64_t u = r.used[s];
    if (u < 0 || u > len) {
      begin = len = used = 0;
      return false;
    }
    used = u;
  }
  return ok;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 1 / (1 + exp(-x)): two approximations of 2^-22 and 2^-23 relative; exp overflows to +inf for
// x < -88, which gives 0.
__device__ __forceinline__ float sigmoid(float x) {
  return rcp(1.f + ex2(-1.44269504088896340736f * x));
}
__device__ __forceinline__ float silu(float x) { return x * sigmoid(x); }

// log(1 + exp(x)) = max(x, 0) + log(1 + v), v = exp(-|x|), to a few 1e-7 relative everywhere.
// log(1 + v) = 2 artanh(s) with s = v / (2 + v) <= 1/3, by its series in s^2 up to s^13 / 13 (the next
// term is under 2e-8 of the first).  The product |x| log2(e) is kept in two parts, since its rounding
// would come back as a relative error of v; |x| is held at 100, where v is 0 already, so that -inf
// gives 0 (a step that leaves the state as it is) and +inf itself.
__device__ __forceinline__ float softplus(float x) {
  const float m = -fminf(fabsf(x), 100.f), hi = m * 1.44269504f;
  // (the second factor: log2(e) less the fp32 value of the first)
  const float lo = fmaf(m, 1.44269504f, -hi) + m * 1.92596299e-8f;
  float v = ex2(hi);
  v = fmaf(v, 0.69314718f * lo, v);
  const float s = v * rcp(2.f + v), s2 = s * s;
  float q = fmaf(s2, 1.f / 13.f, 1.f / 11.f);
  q = fmaf(q, s2, 1.f / 9.f);
  q = fmaf(q, s2, 1.f / 7.f);
  q = fmaf(q, s2, 1.f / 5.f);
  q = fmaf(q, s2, 1.f / 3.f);
  q = fmaf(q * s2, s, s);
  return x != x ? x : fmaxf(x, 0.f) + (q + q);
}

struct ConvArgs {
  const kda_bf16 *x, *weight, *bias, *state_in;
  kda_bf16 *state_out, *o;
  int64_t ldx, ldo;
  int D, act;
  Runs runs;
  const int32_t *slots;
  int n_slots;
  int *status;
};

struct SsmArgs {
  const kda_bf16 *x, *dt, *B, *C, *z;
  const float *A, *D, *dt_bias;
  int64_t ldx, lddt, ldb, ldc, ldz, ldo;
  int H, G, softplus;
  Runs runs;
  const float *S_in;
  float *S_out;
  const int32_t *slots;
  int n_slots;
  kda_bf16 *o;
  int *status;
};

struct VerifyArgs {
  const void *target, *draft;
  const int32_t *tokens;
  const float *u;
  const int32_t *cu;
  int n, V;
  int64_t total;
  int32_t *out_tokens, *n_out;
  int *status;
};

// The step of one token: dt after bias and softplus.
__device__ __forceinline__ float ssm_step(const SsmArgs &a, float raw, float bias) {
  return a.softplus ? softplus(raw + bias) : raw + bias;
}
__device__ __forceinline__ float ssm_dt(const SsmArgs &a, int64_t t, int h) {
  return ssm_step(a, bf2f(a.dt[t * a.lddt + h]), a.dt_bias ? a.dt_bias[h] : 0.f);
}

int *status_word(cudaStream_t st);
bool aligned16(const void *p);

cudaError_t conv_fwd_launch(const ConvArgs &a, int W, cudaStream_t st);
cudaError_t conv_tokens_launch(const ConvArgs &a, int W, cudaStream_t st);
cudaError_t ssm_tokens_launch(const SsmArgs &a, int P, int N, bool single, cudaStream_t st);
size_t ssm_chunk_workspace(int n_seq, int64_t total, int H, int P, int G, int N);
cudaError_t ssm_chunk_launch(const SsmArgs &a, int P, int G, int N, void *workspace, size_t bytes,
                             cudaStream_t st);
cudaError_t verify_launch(const VerifyArgs &a, bool half, cudaStream_t st);

}  // namespace kda

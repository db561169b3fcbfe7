// C ABI of the state space layer's operators and of draft verification: host-side argument checks
// and launches, in the manner of kda_api.cu.
#include "kda_serving.cuh"

namespace kda {

namespace {

bool size_ok(int d) { return d == 64 || d == 128; }
bool aligned(const void *p, unsigned bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

int launched(cudaError_t err) { return err == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

// The batch arguments that the prompt and the token forms share: KDA_OK and the tokens of every
// run where they are all the same, or what is wrong.
int check_runs(const int32_t *cu_seqlens, int n, int64_t total, int64_t *fixed_len) {
  *fixed_len = 0;
  if (n < 0 || total < 0) return KDA_ERR_SHAPE;
  if (n == 0) return total == 0 ? KDA_OK : KDA_ERR_SHAPE;
  if (total > 0x7fffffffLL) return KDA_ERR_SHAPE;
  if (!cu_seqlens) {
    if (total % n != 0) return KDA_ERR_SHAPE;
    *fixed_len = total / n;
  }
  return aligned(cu_seqlens, 4) ? KDA_OK : KDA_ERR_ALIGN;
}

int check_conv(const ConvArgs &a, int W) {
  if (a.D <= 0) return KDA_ERR_SHAPE;
  if (W < 2 || W > 4 || (a.act != 0 && a.act != KDA_CONV_SILU)) return KDA_ERR_UNSUPPORTED;
  if (a.runs.total > 1 && (a.ldx < a.D || (a.o && a.ldo < a.D))) return KDA_ERR_SHAPE;
  if (!a.weight || (a.runs.total > 0 && !a.x)) return KDA_ERR_NULL;
  const void *ptrs[] = {a.x, a.weight, a.bias, a.state_in, a.state_out, a.o};
  for (const void *p : ptrs)
    if (!aligned(p, 2)) return KDA_ERR_ALIGN;
  return KDA_OK;
}

int check_ssm(const SsmArgs &a, int P, int N, unsigned flags) {
  if (a.H <= 0 || a.H > 65535 || a.G <= 0 || a.H % a.G != 0) return KDA_ERR_SHAPE;
  if (!size_ok(P) || !size_ok(N) || (flags & ~KDA_SSM_DT_SOFTPLUS)) return KDA_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(a.runs.n) * a.H > 0x7fffffffLL) return KDA_ERR_SHAPE;
  const int64_t cols = static_cast<int64_t>(a.H) * P, groups = static_cast<int64_t>(a.G) * N;
  if (a.runs.total > 1 &&
      (a.ldx < cols || a.lddt < a.H || a.ldb < groups || a.ldc < groups || (a.o && a.ldo < cols) ||
       (a.z && a.ldz < cols)))
    return KDA_ERR_SHAPE;
  if (!a.A || (a.runs.total > 0 && (!a.x || !a.dt || !a.B || !a.C))) return KDA_ERR_NULL;
  // rows of x, B, C, z and o start on 16-byte boundaries; dt's anywhere
  const void *rows[] = {a.x, a.B, a.C, a.z, a.o, a.S_in, a.S_out};
  for (const void *p : rows)
    if (!aligned16(p)) return KDA_ERR_ALIGN;
  if (a.runs.total > 1 && ((a.ldx | a.ldb | a.ldc | (a.o ? a.ldo : 0) | (a.z ? a.ldz : 0)) & 7))
    return KDA_ERR_ALIGN;
  if (!aligned(a.dt, 2) || !aligned(a.A, 4) || !aligned(a.D, 4) || !aligned(a.dt_bias, 4))
    return KDA_ERR_ALIGN;
  return KDA_OK;
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" {

int kda_conv_fwd(const kda_bf16 *x, int64_t ldx, const kda_bf16 *weight, const kda_bf16 *bias,
                 const int32_t *cu_seqlens, int n_seq, int64_t total_tokens, int D, int W,
                 unsigned flags, const kda_bf16 *conv0, kda_bf16 *conv_final, kda_bf16 *o,
                 int64_t ldo, kda_stream_t stream) {
  int64_t fixed_len;
  if (int e = check_runs(cu_seqlens, n_seq, total_tokens, &fixed_len)) return e;
  ConvArgs a{x, weight, bias, conv0, conv_final, o, ldx, ldo, D, static_cast<int>(flags),
             Runs{cu_seqlens, nullptr, n_seq, total_tokens, fixed_len}, nullptr, n_seq, nullptr};
  if (int e = check_conv(a, W)) return e;
  if (n_seq == 0) return KDA_OK;
  if (total_tokens > 0 && !o) return KDA_ERR_NULL;
  // read by blocks that run beside its writers
  if ((o && o == x) || (conv0 && conv0 == conv_final)) return KDA_ERR_SHAPE;
  if (total_tokens == 0 && !conv_final) return KDA_OK;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (!(a.status = status_word(st))) return KDA_ERR_CUDA;
  return launched(conv_fwd_launch(a, W, st));
}

int kda_conv_tokens(const kda_bf16 *x, int64_t ldx, const kda_bf16 *weight, const kda_bf16 *bias,
                    const int32_t *cu_seqlens, int n, int64_t total_tokens, int D, int W,
                    unsigned flags, kda_bf16 *conv_pool, int n_slots, const int32_t *slots,
                    const int32_t *used, int commit, kda_bf16 *o, int64_t ldo,
                    kda_stream_t stream) {
  int64_t fixed_len;
  if (int e = check_runs(cu_seqlens, n, total_tokens, &fixed_len)) return e;
  if (n_slots < 0 || (!slots && n > n_slots)) return KDA_ERR_SHAPE;
  ConvArgs a{x, weight, bias, conv_pool, commit ? conv_pool : nullptr, o, ldx, ldo, D,
             static_cast<int>(flags), Runs{cu_seqlens, used, n, total_tokens, fixed_len}, slots,
             n_slots, nullptr};
  if (int e = check_conv(a, W)) return e;
  if (!aligned(slots, 4) || !aligned(used, 4)) return KDA_ERR_ALIGN;
  if (total_tokens == 0) return KDA_OK;  // no token: every slot stays as it is
  if (!conv_pool || (!o && !commit)) return KDA_ERR_NULL;
  if (commit && o == x) return KDA_ERR_SHAPE;  // the last rows of x are read again behind the output
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (!(a.status = status_word(st))) return KDA_ERR_CUDA;
  return launched(conv_tokens_launch(a, W, st));
}

int kda_ssm_fwd(const kda_bf16 *x, int64_t ldx, const kda_bf16 *dt, int64_t lddt, const float *A,
                const kda_bf16 *B, int64_t ldb, const kda_bf16 *C, int64_t ldc, const float *D,
                const kda_bf16 *z, int64_t ldz, const float *dt_bias, unsigned flags,
                const int32_t *cu_seqlens, int n_seq, int64_t total_tokens, int H, int P, int G,
                int N, const float *S0, kda_bf16 *o, int64_t ldo, float *S_final, void *workspace,
                size_t workspace_bytes, kda_stream_t stream) {
  int64_t fixed_len;
  if (int e = check_runs(cu_seqlens, n_seq, total_tokens, &fixed_len)) return e;
  SsmArgs a{x, dt, B, C, z, A, D, dt_bias, ldx, lddt, ldb, ldc, ldz, ldo, H, G,
            (flags & KDA_SSM_DT_SOFTPLUS) != 0,
            Runs{cu_seqlens, nullptr, n_seq, total_tokens, fixed_len}, S0, S_final, nullptr, n_seq,
            o, nullptr};
  if (int e = check_ssm(a, P, N, flags)) return e;
  if (n_seq == 0) return KDA_OK;
  if (total_tokens > 0 && !o) return KDA_ERR_NULL;
  // read by blocks that run beside its writers (x by the first pass over long sequences)
  if ((S0 && S0 == S_final) || (o && (o == x || o == B || o == C || o == dt))) return KDA_ERR_SHAPE;
  if (!aligned16(workspace)) return KDA_ERR_ALIGN;
  if (total_tokens == 0 && !S_final) return KDA_OK;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (!(a.status = status_word(st))) return KDA_ERR_CUDA;
  return launched(ssm_chunk_launch(a, P, G, N, workspace, workspace_bytes, st));
}

size_t kda_ssm_fwd_workspace_bytes(int n_seq, int64_t total_tokens, int H, int P, int G, int N) {
  if (n_seq <= 0 || total_tokens <= 0 || H <= 0 || G <= 0 || H % G != 0 || !size_ok(P) ||
      !size_ok(N))
    return 0;
  return ssm_chunk_workspace(n_seq, total_tokens, H, P, G, N);
}

int kda_ssm_tokens(const kda_bf16 *x, int64_t ldx, const kda_bf16 *dt, int64_t lddt,
                   const float *A, const kda_bf16 *B, int64_t ldb, const kda_bf16 *C, int64_t ldc,
                   const float *D, const kda_bf16 *z, int64_t ldz, const float *dt_bias,
                   unsigned flags, const int32_t *cu_seqlens, int n, int64_t total_tokens, int H,
                   int P, int G, int N, float *state_pool, int n_slots, const int32_t *slots,
                   const int32_t *used, int commit, kda_bf16 *o, int64_t ldo,
                   kda_stream_t stream) {
  int64_t fixed_len;
  if (int e = check_runs(cu_seqlens, n, total_tokens, &fixed_len)) return e;
  if (n_slots < 0 || (!slots && n > n_slots)) return KDA_ERR_SHAPE;
  SsmArgs a{x, dt, B, C, z, A, D, dt_bias, ldx, lddt, ldb, ldc, ldz, ldo, H, G,
            (flags & KDA_SSM_DT_SOFTPLUS) != 0,
            Runs{cu_seqlens, used, n, total_tokens, fixed_len}, state_pool,
            commit ? state_pool : nullptr, slots, n_slots, o, nullptr};
  if (int e = check_ssm(a, P, N, flags)) return e;
  if (!aligned(slots, 4) || !aligned(used, 4)) return KDA_ERR_ALIGN;
  if (total_tokens == 0) return KDA_OK;  // no token: every state stays as it is
  if (!state_pool || (!o && !commit)) return KDA_ERR_NULL;
  if (o && (o == B || o == C || o == dt)) return KDA_ERR_SHAPE;  // read by the blocks of other heads
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (!(a.status = status_word(st))) return KDA_ERR_CUDA;
  return launched(ssm_tokens_launch(a, P, N, fixed_len == 1, st));
}

int kda_verify_draft(const void *target, const void *draft, int prob_bytes, int V,
                     const int32_t *tokens, const float *u, const int32_t *cu_seqlens, int n,
                     int64_t total_tokens, int32_t *out_tokens, int32_t *n_out,
                     kda_stream_t stream) {
  if (n < 0 || total_tokens < 0 || total_tokens > 0x7fffffffLL || V <= 0) return KDA_ERR_SHAPE;
  if ((prob_bytes != 2 && prob_bytes != 4) || V > (1 << 22)) return KDA_ERR_UNSUPPORTED;
  if (n == 0) return total_tokens == 0 ? KDA_OK : KDA_ERR_SHAPE;
  if (n > (1 << 24) || total_tokens < n) return KDA_ERR_SHAPE;  // a run has one token at least
  if (!target || !tokens || !u || !cu_seqlens || !out_tokens || !n_out) return KDA_ERR_NULL;
  const void *words[] = {tokens, u, cu_seqlens, out_tokens, n_out};
  for (const void *p : words)
    if (!aligned(p, 4)) return KDA_ERR_ALIGN;
  if (!aligned(target, prob_bytes) || !aligned(draft, prob_bytes)) return KDA_ERR_ALIGN;
  if (out_tokens == tokens) return KDA_ERR_SHAPE;  // read by the other blocks of the run's cluster
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  VerifyArgs a{target, draft, tokens, u, cu_seqlens, n, V, total_tokens, out_tokens, n_out,
               status_word(st)};
  if (!a.status) return KDA_ERR_CUDA;
  return launched(verify_launch(a, prob_bytes == 2, st));
}

}  // extern "C"

// Arguments that the kernels of the paged cache take by value, and what they share.
#pragma once

#include "kda_serving.cuh"

namespace kda {

// The sequences of a cache: slot s holds lens[s] tokens in the pages table[s][0 ...].
struct PagedSeqs {
  const int32_t *table;
  int max_pages;
  const int32_t *lens;
  const int32_t *slots;  // slot of each run, or NULL: slot b
  int n_slots;
  int n_pages;
  int page_shift;  // a page holds 1 << page_shift tokens
};

// Slot of run b and the tokens in front of the run; false for a slot outside the table or a
// length that is negative (the caller records KDA_ERR_SHAPE).
__device__ __forceinline__ bool run_slot(const PagedSeqs &s, int b, int &slot, int64_t &before) {
  slot = s.slots ? s.slots[b] : b;
  before = 0;
  if (slot < 0 || slot >= s.n_slots) return false;
  before = s.lens[slot];
  return before >= 0;
}

struct AppendArgs {
  const kda_bf16 *k, *v;
  int64_t ldk, ldv;
  Runs runs;
  PagedSeqs seqs;
  int H, D;
  kda_bf16 *cache;
  int *status;
};

struct AttnCall {
  const kda_bf16 *q;
  int64_t ldq;
  kda_bf16 *o;
  int64_t ldo;
  Runs runs;
  PagedSeqs seqs;
  const kda_bf16 *cache;
  int H, G, window;  // heads of keys, query heads for each
  float scale;
  void *workspace;   // attn_workspace(D) bytes, or NULL
  int *status;
  bool test_stall;   // KDA_ATTN_TEST_STALL
};

enum PagesOp { kPagesGrow, kPagesFork, kPagesCompact };

struct PagesArgs {
  int32_t *table;
  int32_t *table_out;  // compact
  int max_pages, n_slots;
  int32_t *lens;
  const int32_t *want;       // grow
  const int32_t *src, *dst;  // fork
  int m;
  int n_pages, page_shift;
  int32_t *count;  // pages left (grow, fork) or used (compact)
  int32_t *ws;     // fork, compact: PagesWs
  int ws_n;
  int *status;
};

// The moves that the planning kernel leaves for the copying one, in int32 words: how many, then
// ws_n sources, ws_n destinations, and of a fork the tokens in each page and the fresh pages.
constexpr int kPagesWsHead = 4;
constexpr int kPagesWsArrays = 4;
__host__ __device__ constexpr int64_t pages_ws_bytes(int64_t n) {
  return 4 * (kPagesWsHead + kPagesWsArrays * n);
}

constexpr int kMaxPages = 1 << 20;  // of a pool, and of a row of the table
constexpr int kMaxSlots = 1 << 13;

size_t attn_workspace(int D);
cudaError_t attn_launch(const AttnCall &c, int D, cudaStream_t st);
cudaError_t kv_append_launch(const AppendArgs &a, cudaStream_t st);
cudaError_t pages_launch(PagesOp op, const PagesArgs &a, cudaStream_t st);
// The moves of a plan: `layers` layers of n_pages pages of `planes` planes of row_bytes a token.
cudaError_t pages_move_launch(PagesOp op, const PagesArgs &a, kda_bf16 *cache, int layers,
                              int planes, int row_bytes, cudaStream_t st);

}  // namespace kda

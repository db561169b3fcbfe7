// C ABI of the paged cache's operators: host-side argument checks and launches, in the manner of
// kda_serving_api.cu.
#include <initializer_list>

#include "kda_paged.cuh"

namespace kda {

namespace {

bool size_ok(int d) { return d == 64 || d == 128; }
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }
int launched(cudaError_t err) { return err == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

// log2 of a page's tokens, -1 for a size that is not supported.
int page_shift(int page) {
  return page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : page == 128 ? 7 : -1;
}

// Whether [p, p + bytes) and [q, q + more) share anything.
bool overlap(const void *p, int64_t bytes, const void *q, int64_t more) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return p && q && bytes > 0 && more > 0 && a < b + static_cast<uintptr_t>(more) &&
         b < a + static_cast<uintptr_t>(bytes);
}

struct Range {
  const void *p;
  int64_t bytes;
};
bool overlaps_any(const Range &r, std::initializer_list<Range> others) {
  for (const Range &x : others)
    if (overlap(r.p, r.bytes, x.p, x.bytes)) return true;
  return false;
}

// The cache of all layers.  (check_layers keeps its pieces of 4 KB under 2^31.)
Range pool_of(const kda_bf16 *cache, int layers, int n_pages, int H, int page, int D) {
  return {cache, 4LL * H * page * D * n_pages * layers};
}

// Tokens of every run where they are all the same (0 with offsets), as in kda_serving_api.cu.
int check_runs(const int32_t *cu_seqlens, int n, int64_t total, int64_t *fixed_len) {
  *fixed_len = 0;
  if (n < 0 || total < 0 || total > 0x7fffffffLL) return KDA_ERR_SHAPE;
  if (n == 0) return total == 0 ? KDA_OK : KDA_ERR_SHAPE;
  if (!cu_seqlens) {
    if (total % n != 0) return KDA_ERR_SHAPE;
    *fixed_len = total / n;
  }
  return aligned4(cu_seqlens) ? KDA_OK : KDA_ERR_ALIGN;
}

int check_table(const int32_t *table, const int32_t *lens, int max_pages, int n_slots, int n_pages,
                int page) {
  if (max_pages < 0 || n_slots < 0 || n_pages < 0) return KDA_ERR_SHAPE;
  if (page_shift(page) < 0) return KDA_ERR_UNSUPPORTED;
  if (max_pages > kMaxPages || n_pages > kMaxPages) return KDA_ERR_UNSUPPORTED;
  if (n_slots > 0 && (!lens || (max_pages > 0 && !table))) return KDA_ERR_NULL;
  return aligned4(table) && aligned4(lens) ? KDA_OK : KDA_ERR_ALIGN;
}

// What the two operators on runs take alike; the caller has checked the runs.
int check_heads(int H, int D, const kda_bf16 *cache, int n_pages) {
  if (H <= 0 || H > 65535) return KDA_ERR_SHAPE;
  if (!size_ok(D)) return KDA_ERR_UNSUPPORTED;
  // planes of a head are counted in 31 bits
  if (static_cast<int64_t>(n_pages) * 2 * H > 0x7fffffffLL) return KDA_ERR_UNSUPPORTED;
  if (n_pages > 0 && !cache) return KDA_ERR_NULL;
  return aligned16(cache) ? KDA_OK : KDA_ERR_ALIGN;
}

// Pages of all layers as planes of a head: how many fit the moving kernel's counter.
int check_layers(const kda_bf16 *cache, int layers, int n_pages, int H, int page, int D) {
  if (layers <= 0) return KDA_ERR_SHAPE;
  if (int e = check_heads(H, D, cache, n_pages)) return e;
  const int64_t pieces = (static_cast<int64_t>(page) * D * 2 + 4095) / 4096 * 2 * H;
  return n_pages * (static_cast<double>(pieces) * layers) < 2147483648.0 ? KDA_OK : KDA_ERR_UNSUPPORTED;
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" {

int kda_kv_append(const kda_bf16 *k, int64_t ldk, const kda_bf16 *v, int64_t ldv,
                  const int32_t *cu_seqlens, int n, int64_t total_tokens, int H, int D,
                  kda_bf16 *cache, int n_pages, int page, const int32_t *table, int max_pages,
                  const int32_t *lens, int n_slots, const int32_t *slots, kda_stream_t stream) {
  int64_t fixed_len;
  if (int e = check_runs(cu_seqlens, n, total_tokens, &fixed_len)) return e;
  if (int e = check_table(table, lens, max_pages, n_slots, n_pages, page)) return e;
  if (int e = check_heads(H, D, cache, n_pages)) return e;
  if (!slots && n > n_slots) return KDA_ERR_SHAPE;
  const int64_t cols = static_cast<int64_t>(H) * D;
  if (total_tokens > 1 && (ldk < cols || ldv < cols)) return KDA_ERR_SHAPE;
  if (total_tokens > 0 && (!k || !v)) return KDA_ERR_NULL;
  if (!aligned16(k) || !aligned16(v) || !aligned4(slots)) return KDA_ERR_ALIGN;
  if (total_tokens > 1 && ((ldk | ldv) & 7)) return KDA_ERR_ALIGN;
  if (total_tokens == 0) return KDA_OK;
  if (total_tokens * cols / 4096 >= 0x7fffffffLL) return KDA_ERR_UNSUPPORTED;
  // rows or tables that lie in the cache would be read by one block and written by another
  const int64_t bytes = 2 * cols * 2 * n_pages * page;
  if (overlaps_any({cache, bytes}, {{k, 2 * ((total_tokens - 1) * ldk + cols)}, {v, 2 * ((total_tokens - 1) * ldv + cols)},
                                    {table, 4LL * n_slots * max_pages}, {lens, 4LL * n_slots}, {slots, 4LL * n},
                                    {cu_seqlens, 4LL * (n + 1)}}))
    return KDA_ERR_SHAPE;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  AppendArgs a{k, v, ldk, ldv, Runs{cu_seqlens, nullptr, n, total_tokens, fixed_len},
               PagedSeqs{table, max_pages, lens, slots, n_slots, n_pages, page_shift(page)}, H, D,
               cache, status_word(st)};
  if (!a.status) return KDA_ERR_CUDA;
  return launched(kv_append_launch(a, st));
}

int kda_attn_paged(const kda_bf16 *q, int64_t ldq, const int32_t *cu_seqlens, int n,
                   int64_t total_tokens, int Hq, int H, int D, const kda_bf16 *cache, int n_pages,
                   int page, const int32_t *table, int max_pages, const int32_t *lens, int n_slots,
                   const int32_t *slots, float scale, int window, kda_bf16 *o, int64_t ldo,
                   void *workspace, size_t workspace_bytes, kda_stream_t stream) {
  int64_t fixed_len;
  if (int e = check_runs(cu_seqlens, n, total_tokens, &fixed_len)) return e;
  if (int e = check_table(table, lens, max_pages, n_slots, n_pages, page)) return e;
  if (int e = check_heads(H, D, cache, n_pages)) return e;
  const bool test_stall = window == KDA_ATTN_TEST_STALL;
  if (test_stall) window = 0;
  if (Hq <= 0 || Hq % H != 0 || Hq > 65535 || window < 0) return KDA_ERR_SHAPE;
  if (!slots && n > n_slots) return KDA_ERR_SHAPE;
  // (also refuses NaN; the kernel multiplies it by log2(e))
  if (!(scale > 0.f && scale <= 1e38f)) return KDA_ERR_UNSUPPORTED;
  const int64_t cols = static_cast<int64_t>(Hq) * D;
  if (total_tokens > 1 && (ldq < cols || ldo < cols)) return KDA_ERR_SHAPE;
  if (total_tokens > 0 && (!q || !o)) return KDA_ERR_NULL;
  if (!aligned16(q) || !aligned16(o) || !aligned4(slots) || !aligned16(workspace))
    return KDA_ERR_ALIGN;
  if (total_tokens > 1 && ((ldq | ldo) & 7)) return KDA_ERR_ALIGN;
  if (total_tokens == 0) return KDA_OK;
  if (total_tokens * (Hq / H) > 0x7fffff00LL) return KDA_ERR_UNSUPPORTED;  // rows of a run, in 31 bits
  if (n_pages == 0) return KDA_ERR_SHAPE;  // no token can have a place
  const int64_t rows = 2 * ((total_tokens - 1) * ldo + cols);
  // q is read, and the cache, by blocks that run beside the writers of o; o may be q
  if ((o != q || ldo != ldq) && overlap(o, rows, q, 2 * ((total_tokens - 1) * ldq + cols)))
    return KDA_ERR_SHAPE;
  const bool cut = workspace && workspace_bytes >= attn_workspace(D);
  const Range held{cache, 4LL * H * D * page * n_pages}, pages{table, 4LL * n_slots * max_pages}, ends{lens, 4LL * n_slots},
      at{slots, 4LL * n}, offsets{cu_seqlens, 4LL * (n + 1)}, out{o, rows},
      scratch{workspace, cut ? static_cast<int64_t>(attn_workspace(D)) : 0};
  if (overlaps_any(out, {held, pages, ends, at, offsets})) return KDA_ERR_SHAPE;
  if (overlaps_any(scratch, {out, {q, 2 * ((total_tokens - 1) * ldq + cols)}, held, pages, ends, at, offsets}))
    return KDA_ERR_SHAPE;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  AttnCall c{q, ldq, o, ldo, Runs{cu_seqlens, nullptr, n, total_tokens, fixed_len},
             PagedSeqs{table, max_pages, lens, slots, n_slots, n_pages, page_shift(page)}, cache, H,
             Hq / H, window, scale, cut ? workspace : nullptr, status_word(st), test_stall};
  if (!c.status) return KDA_ERR_CUDA;
  return launched(attn_launch(c, D, st));
}

size_t kda_attn_paged_workspace_bytes(int n, int64_t total_tokens, int Hq, int H, int D) {
  if (n <= 0 || total_tokens <= 0 || H <= 0 || Hq <= 0 || Hq % H != 0 || !size_ok(D)) return 0;
  return attn_workspace(D);
}

int kda_pages_grow(int32_t *table, int max_pages, const int32_t *lens, const int32_t *want,
                   int n_slots, int n_pages, int page, int32_t *left, kda_stream_t stream) {
  if (int e = check_table(table, lens, max_pages, n_slots, n_pages, page)) return e;
  if (n_slots > kMaxSlots) return KDA_ERR_UNSUPPORTED;
  if (!left || (n_slots > 0 && !want)) return KDA_ERR_NULL;
  if (!aligned4(want) || !aligned4(left)) return KDA_ERR_ALIGN;
  const int64_t rows = 4LL * n_slots, all = rows * max_pages;
  // what one CTA writes while another reads
  if (overlap(table, all, lens, rows) || overlap(table, all, want, rows) ||
      overlap(left, 4, table, all) || overlap(left, 4, lens, rows) || overlap(left, 4, want, rows))
    return KDA_ERR_SHAPE;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  PagesArgs a{};
  a.table = table;
  a.max_pages = max_pages;
  a.n_slots = n_slots;
  a.lens = const_cast<int32_t *>(lens);  // (read only)
  a.want = want;
  a.n_pages = n_pages;
  a.page_shift = page_shift(page);
  a.count = left;
  if (!(a.status = status_word(st))) return KDA_ERR_CUDA;
  return launched(pages_launch(kPagesGrow, a, st));
}

size_t kda_pages_workspace_bytes(int n) {
  return n < 0 ? 0 : static_cast<size_t>(pages_ws_bytes(n));
}

int kda_pages_fork(kda_bf16 *cache, int layers, int n_pages, int H, int page, int D,
                   int32_t *table, int max_pages, int32_t *lens, int n_slots, const int32_t *src,
                   const int32_t *dst, int n, int32_t *left, void *workspace,
                   size_t workspace_bytes, kda_stream_t stream) {
  if (int e = check_table(table, lens, max_pages, n_slots, n_pages, page)) return e;
  if (int e = check_layers(cache, layers, n_pages, H, page, D)) return e;
  if (n < 0) return KDA_ERR_SHAPE;
  if (n_slots > kMaxSlots || n > kMaxPages) return KDA_ERR_UNSUPPORTED;
  if (!left || (n > 0 && (!src || !dst))) return KDA_ERR_NULL;
  if (!aligned4(src) || !aligned4(dst) || !aligned4(left) || !aligned16(workspace))
    return KDA_ERR_ALIGN;
  const int64_t need = pages_ws_bytes(n), rows = 4LL * n_slots, all = rows * max_pages;
  if (!workspace || workspace_bytes < static_cast<size_t>(need)) return KDA_ERR_WORKSPACE;
  // written by one CTA while another reads it, or written twice
  const Range out[] = {{table, all}, {lens, rows}, {left, 4}, {workspace, need}, pool_of(cache, layers, n_pages, H, page, D)};
  for (int i = 0; i < 5; ++i) {
    for (int j = 0; j < i; ++j)
      if (overlap(out[i].p, out[i].bytes, out[j].p, out[j].bytes)) return KDA_ERR_SHAPE;
    if (overlaps_any(out[i], {{src, 4LL * n}, {dst, 4LL * n}})) return KDA_ERR_SHAPE;
  }
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  PagesArgs a{};
  a.table = table;
  a.max_pages = max_pages;
  a.n_slots = n_slots;
  a.lens = lens;
  a.src = src;
  a.dst = dst;
  a.m = n;
  a.n_pages = n_pages;
  a.page_shift = page_shift(page);
  a.count = left;
  a.ws = static_cast<int32_t *>(workspace);
  a.ws_n = n;
  if (!(a.status = status_word(st))) return KDA_ERR_CUDA;
  if (cudaError_t e = pages_launch(kPagesFork, a, st)) return launched(e);
  if (n == 0 || n_pages == 0) return KDA_OK;
  return launched(pages_move_launch(kPagesFork, a, cache, layers, 2 * H, 2 * D, st));
}

int kda_pages_compact(kda_bf16 *cache, int layers, int n_pages, int H, int page, int D,
                      const int32_t *table, int max_pages, const int32_t *lens, int n_slots,
                      int32_t *table_out, int32_t *used, void *workspace, size_t workspace_bytes,
                      kda_stream_t stream) {
  if (int e = check_table(table, lens, max_pages, n_slots, n_pages, page)) return e;
  if (int e = check_layers(cache, layers, n_pages, H, page, D)) return e;
  if (n_slots > kMaxSlots) return KDA_ERR_UNSUPPORTED;
  if (!used || (n_slots > 0 && max_pages > 0 && !table_out)) return KDA_ERR_NULL;
  if (!aligned4(table_out) || !aligned4(used) || !aligned16(workspace)) return KDA_ERR_ALIGN;
  const int64_t need = pages_ws_bytes(n_pages), rows = 4LL * n_slots, all = rows * max_pages;
  if (!workspace || workspace_bytes < static_cast<size_t>(need)) return KDA_ERR_WORKSPACE;
  // the table's own place is fine: a row is read and written by one warp
  if ((table_out != table && overlap(table_out, all, table, all)) ||
      overlap(table_out, all, lens, rows) || overlap(used, 4, table_out, all) ||
      overlap(used, 4, table, all) || overlap(used, 4, lens, rows) ||
      overlap(workspace, need, table, all) || overlap(workspace, need, table_out, all) ||
      overlap(workspace, need, lens, rows) || overlap(workspace, need, used, 4))
    return KDA_ERR_SHAPE;
  if (overlaps_any(pool_of(cache, layers, n_pages, H, page, D),
                   {{table, all}, {table_out, all}, {lens, rows}, {used, 4}, {workspace, need}}))
    return KDA_ERR_SHAPE;
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  PagesArgs a{};
  a.table = const_cast<int32_t *>(table);  // (read only, unless it is the output)
  a.table_out = table_out;
  a.max_pages = max_pages;
  a.n_slots = n_slots;
  a.lens = const_cast<int32_t *>(lens);  // (read only)
  a.n_pages = n_pages;
  a.page_shift = page_shift(page);
  a.count = used;
  a.ws = static_cast<int32_t *>(workspace);
  a.ws_n = n_pages;
  if (!(a.status = status_word(st))) return KDA_ERR_CUDA;
  if (cudaError_t e = pages_launch(kPagesCompact, a, st)) return launched(e);
  if (n_pages == 0) return KDA_OK;
  return launched(pages_move_launch(kPagesCompact, a, cache, layers, 2 * H, 2 * D, st));
}

}  // extern "C"

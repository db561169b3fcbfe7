// Pages of a cache: giving them to sequences, sharing them, moving them together.
//
// A page is in use where a row of the table reaches it within its sequence's length.  There are no
// reference counts: every call marks the pages in use from the table itself, so a sequence is freed
// by its length alone and shared pages need no care.  One planning kernel does that and what
// follows from it; a second one moves what the plan says.
//
// Planning.  One cluster of 8 CTAs, so that nothing passes through global memory and no launch
// follows another:
//   1. mark: a warp takes a row and sets a bit for each of its pages, in a bitmap of its CTA's
//      shared memory (OR in any order gives the same bits; 128 KB for the largest pool, 2^20);
//   2. each CTA ORs an eighth of the eight bitmaps, counts the bits that are not set, and learns
//      from the others' counts the rank of its first unused page;
//   3. grow: the k-th unused page goes to the row whose demand covers rank k, found by bisection in
//      the prefix sums of the demands; fork: it goes to the k-th fork with a partial last page;
//      compact: with u pages in use, the k-th unused page below u takes the k-th used page from u on.
// What bounds it: the latency of a dozen dependent steps and five cluster barriers, and for large
// tables the loads of step 1, which 256 warps have in flight at once.  One CTA marks 512 rows of
// 500 entries eight times slower, and the whole GPU would need a grid-wide barrier.
//
// Moving.  A warp takes 4 KB pieces of (page, layer, K or V of a head), eight 16-byte loads in
// flight a lane; sources and destinations are disjoint, so pieces need no order.  Bound by memory.
#include "kda_paged.cuh"
#include "kda_pdl.cuh"
#include "kda_sm100.cuh"

namespace kda {

namespace {

constexpr int kPThreads = 1024;
constexpr int kPRanks = 8;
constexpr int kNone = 0x7fffffff;

__device__ __forceinline__ unsigned cluster_rank() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The word at this CTA's shared address `p`, of CTA `rank`.
__device__ __forceinline__ uint32_t remote(const void *p, unsigned rank) {
  uint32_t there, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(there)
               : "r"(sm100::smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(there) : "memory");
  return v;
}

// Sum of v over the threads before this one and, in `total`, over all of the block.
__device__ __forceinline__ int block_scan(int v, int &total) {
  __shared__ int sums[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  __syncthreads();  // (the last call's sums have been read)
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  int s = sums[lane];
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int y = __shfl_up_sync(0xffffffffu, s, d);
    if (lane >= d) s += y;
  }
  total = __shfl_sync(0xffffffffu, s, 31);
  const int before = warp ? __shfl_sync(0xffffffffu, s, warp - 1) : 0;
  return before + x - v;
}

struct Plan {
  const PagesArgs &a;
  int *rows;  // shared: grow, the prefix sums of the demands; fork, the fork that takes each row

  // Pages of `tokens` tokens, or -1 where the table's row cannot hold them.
  __device__ int pages_of(int tokens) const {
    const int64_t n = (static_cast<int64_t>(tokens) + (1 << a.page_shift) - 1) >> a.page_shift;
    return tokens < 0 || n > a.max_pages ? -1 : static_cast<int>(n);
  }
  __device__ bool fork_in_range(int i) const {
    const int s = a.src[i], d = a.dst[i];
    return s >= 0 && s < a.n_slots && d >= 0 && d < a.n_slots;
  }
  // Whether fork i is made: its row is its own, and its parent's row is nobody's.
  __device__ bool fork_made(int i) const {
    return fork_in_range(i) && rows[a.dst[i]] == i && rows[a.src[i]] == kNone &&
           pages_of(a.lens[a.src[i]]) >= 0;
  }
  __device__ int fork_tail(int i) const { return a.lens[a.src[i]] & ((1 << a.page_shift) - 1); }
};

template <PagesOp OP>
__global__ void __launch_bounds__(kPThreads, 1) pages_plan_kernel(const PagesArgs a) {
  extern __shared__ uint32_t bits[];
  __shared__ int s_total;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(cluster_rank());
  const int words = (a.n_pages + 31) / 32, share = (words + kPRanks - 1) / kPRanks;
  const Plan plan{a, reinterpret_cast<int *>(bits + words)};
  int *const rows = plan.rows;
  int bad = 0;
  if (OP != kPagesGrow) grid_launch_dependents();

  // 1. marks
  for (int w = tid; w < words; w += kPThreads)
    bits[w] = w == words - 1 && (a.n_pages & 31) ? ~0u << (a.n_pages & 31) : 0u;
  if (OP == kPagesFork) {
    for (int b = tid; b < a.n_slots; b += kPThreads) rows[b] = kNone;
    __syncthreads();
    for (int i = tid; i < a.m; i += kPThreads)
      if (plan.fork_in_range(i)) atomicMin(&rows[a.dst[i]], i);
  }
  __syncthreads();
  for (int b = rank * 32 + warp; b < a.n_slots; b += kPRanks * 32) {
    if (OP == kPagesFork && rows[b] != kNone && plan.fork_made(rows[b])) continue;
    const int need = plan.pages_of(a.lens[b]);
    if (need < 0) bad = 1;
    const int32_t *row = a.table + static_cast<int64_t>(b) * a.max_pages;
    for (int i = lane; i < need; i += 32 * 8) {
      int p[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) p[j] = i + 32 * j < need ? row[i + 32 * j] : kNone;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (p[j] >= 0 && p[j] < a.n_pages)
          atomicOr(&bits[p[j] >> 5], 1u << (p[j] & 31));
        else if (p[j] != kNone || i + 32 * j < need)
          bad = 1;
      }
    }
  }

  // 2. this CTA's share of all marks, and the unused pages before it
  cluster_sync();
  const int each = (share + kPThreads - 1) / kPThreads;  // words of a thread, one after another
  const int w0 = min(rank * share + tid * each, words), w1 = min(min(w0 + each, (rank + 1) * share), words);
  int unused = 0;
  for (int w = w0; w < w1; ++w) {
    uint32_t v = 0;
#pragma unroll
    for (unsigned q = 0; q < kPRanks; ++q) v |= remote(bits + w, q);
    bits[w] = v;  // (nobody else reads this CTA's share of this CTA's bitmap)
    unused += 32 - __popc(v);
  }
  int total, first = block_scan(unused, total);
  if (tid == 0) s_total = total;
  cluster_sync();
  int left = 0;
#pragma unroll
  for (int q = 0; q < kPRanks; ++q) {
    const int n = static_cast<int>(remote(&s_total, q));
    if (q < rank) first += n;
    left += n;
  }

  if (OP == kPagesGrow) {
    int64_t carry = 0;
    for (int b0 = 0; b0 < a.n_slots; b0 += kPThreads) {
      const int b = b0 + tid;
      int more = 0;
      if (b < a.n_slots) {
        const int have = plan.pages_of(a.lens[b]), want = plan.pages_of(a.want[b]);
        if (want < 0) bad = 1;
        if (have >= 0 && want > have) more = want - have;
      }
      int all, before = block_scan(more, all);
      if (b < a.n_slots) rows[b] = static_cast<int>(min(carry + before + more, int64_t(1) << 30));
      carry += all;
    }
    __syncthreads();
    const int n = a.n_slots;
    for (int w = w0; w < w1; ++w)
      for (uint32_t v = ~bits[w]; v; v &= v - 1, ++first) {
        if (n == 0 || first >= rows[n - 1]) break;
        int lo = 0, hi = n - 1;  // the first row whose demands end behind this rank
        while (lo < hi) {
          const int mid = (lo + hi) / 2;
          if (rows[mid] > first) hi = mid;
          else lo = mid + 1;
        }
        if (rows[lo] <= left)
          a.table[static_cast<int64_t>(lo) * a.max_pages + plan.pages_of(a.lens[lo]) + first -
                  (lo ? rows[lo - 1] : 0)] = w * 32 + __ffs(v) - 1;
      }
    for (int b = rank * 32 + warp; b < n; b += kPRanks * 32) {
      if (rows[b] <= left) continue;  // all of its pages, or none
      const int have = plan.pages_of(a.lens[b]), want = plan.pages_of(a.want[b]);
      if (have < 0) continue;
      for (int i = have + lane; i < want; i += 32)
        a.table[static_cast<int64_t>(b) * a.max_pages + i] = -1;
    }
    if (rank == 0 && tid == 0)
      *a.count = static_cast<int>(max(left - carry, -static_cast<int64_t>(kNone)));
  }

  if (OP == kPagesFork) {
    int32_t *src = a.ws + kPagesWsHead, *dst = src + a.ws_n, *len = dst + a.ws_n,
            *fresh = len + a.ws_n;
    int want = 0;  // forks with a partial last page
    for (int i0 = 0; i0 < a.m; i0 += kPThreads) {
      const int i = i0 + tid;
      want += __syncthreads_count(i < a.m && plan.fork_made(i) && plan.fork_tail(i));
    }
    for (int w = w0; w < w1; ++w)
      for (uint32_t v = ~bits[w]; v && first < want; v &= v - 1, ++first)
        fresh[first] = w * 32 + __ffs(v) - 1;
    cluster_sync();
    __shared__ int s_rank[kPThreads];  // of the fork's fresh page; -1: needs none, -2: not made
    int before = 0;
    for (int i0 = 0; i0 < a.m; i0 += kPThreads) {
      const int i = i0 + tid;
      const bool made = i < a.m && plan.fork_made(i), tail = made && plan.fork_tail(i);
      int all;
      const int at = block_scan(tail, all);
      s_rank[tid] = tail ? before + at : made ? -1 : -2;
      if (i < a.m && !made) bad = 1;
      before += all;
      __syncthreads();
      for (int j = rank * 32 + warp; j < min(kPThreads, a.m - i0); j += kPRanks * 32) {
        const int r = s_rank[j];
        if (r == -2) continue;
        const int s = a.src[i0 + j], d = a.dst[i0 + j], tokens = a.lens[s];
        const int32_t *from = a.table + static_cast<int64_t>(s) * a.max_pages;
        int32_t *to = a.table + static_cast<int64_t>(d) * a.max_pages;
        const bool none = r >= left;  // no page is left for it: an empty row
        const int need = none ? 0 : plan.pages_of(tokens);
        const int whole = need - (r >= 0 && !none);
        for (int e = lane; e < a.max_pages; e += 32) {
          if (e < whole) to[e] = from[e];
          else if (e >= need) to[e] = -1;
        }
        if (lane == 0) {
          a.lens[d] = none ? 0 : tokens;
          if (whole < need) {
            const int old = from[whole], page = __ldcg(fresh + r);
            const bool ok = old >= 0 && old < a.n_pages;
            to[whole] = page;
            src[r] = ok ? old : -1;
            dst[r] = page;
            len[r] = plan.fork_tail(i0 + j);
            if (!ok) bad = 1;
          }
        }
      }
      __syncthreads();
    }
    if (rank == 0 && tid == 0) {
      a.ws[0] = min(want, left);
      *a.count = left - want;
    }
  }

  if (OP == kPagesCompact) {
    int32_t *src = a.ws + kPagesWsHead, *dst = src + a.ws_n, *now = dst + a.ws_n;
    const int used = a.n_pages - left;
    // rank of an unused page: those before it; of a used one from `used` on: the used ones before
    // it, less the used ones below `used`, which are as many as the unused ones from there on
    // fewer than `left`.  Holes are the unused pages below `used`.
    __shared__ int s_below;  // unused pages below `used`, in this CTA's share
    if (tid == 0) s_below = 0;
    __syncthreads();
    int below = 0;
    for (int w = w0; w < w1; ++w) {
      const int n = used - w * 32;  // pages of this word below `used`
      if (n > 0) below += __popc(~bits[w] & (n >= 32 ? ~0u : (1u << n) - 1));
    }
    if (below) atomicAdd(&s_below, below);
    cluster_sync();
    int holes = 0;
#pragma unroll
    for (int q = 0; q < kPRanks; ++q) holes += static_cast<int>(remote(&s_below, q));
    // the used pages before this thread's words: the words' pages less the unused ones
    int k = first, u = w0 * 32 - first - (used - holes);
    for (int w = w0; w < w1; ++w)
      for (int j = 0; j < 32; ++j) {
        const int p = w * 32 + j;
        if (p >= a.n_pages) break;
        if (bits[w] >> j & 1) {
          if (p >= used) src[u] = p;
          ++u;
        } else {
          if (p < used) dst[k] = p;
          ++k;
        }
      }
    cluster_sync();
    u = w0 * 32 - first - (used - holes);
    for (int w = w0; w < w1; ++w)
      for (uint32_t v = bits[w]; v; v &= v - 1, ++u) {
        const int p = w * 32 + __ffs(v) - 1;
        if (p >= used && p < a.n_pages) now[p] = __ldcg(dst + u);
      }
    cluster_sync();
    for (int b = rank * 32 + warp; b < a.n_slots; b += kPRanks * 32) {
      const int need = plan.pages_of(a.lens[b]);
      const int32_t *row = a.table + static_cast<int64_t>(b) * a.max_pages;
      int32_t *out = a.table_out + static_cast<int64_t>(b) * a.max_pages;
      for (int i = lane; i < a.max_pages; i += 32) {
        int p = -1;
        if (i < need) {
          p = row[i];
          if (p >= used && p < a.n_pages) p = __ldcg(now + p);
        }
        out[i] = p;
      }
    }
    if (rank == 0 && tid == 0) {
      a.ws[0] = holes;
      *a.count = used;
    }
  }
  if (bad) atomicOr(a.status, KDA_ERR_SHAPE);
  cluster_sync();  // no CTA's shared memory goes while another may read it
}

constexpr int kMThreads = 256;
constexpr int kPiece = 4096;  // bytes: 32 lanes x 8 vectors

// FORK: the first len[m] tokens of each plane; else all of it.
template <bool FORK>
__global__ void __launch_bounds__(kMThreads) pages_move_kernel(const PagesArgs a, uint8_t *cache,
                                                               int layers, int planes,
                                                               int row_bytes) {
  grid_dependency_wait();
  const int moves = a.ws[0], lane = threadIdx.x & 31;
  const int32_t *src = a.ws + kPagesWsHead, *dst = src + a.ws_n, *len = dst + a.ws_n;
  const int plane_bytes = row_bytes << a.page_shift;
  const unsigned pieces = (plane_bytes + kPiece - 1) / kPiece, each = planes * pieces;
  const unsigned all = static_cast<unsigned>(moves) * layers * each;
  const int64_t page_bytes = static_cast<int64_t>(plane_bytes) * planes;
  for (unsigned x = blockIdx.x * (kMThreads / 32) + (threadIdx.x >> 5); x < all;
       x += gridDim.x * (kMThreads / 32)) {
    // (pieces of a page follow one another)
    const unsigned page = x / each, in = x - page * each, plane = in / pieces,
                   piece = in - plane * pieces, layer = page % layers, m = page / layers;
    const int from = src[m], to = dst[m];
    const int end = FORK ? len[m] * row_bytes : plane_bytes;
    if (from < 0) continue;
    const int at = piece * kPiece + lane * 16;
    const int64_t base = (static_cast<int64_t>(layer) * a.n_pages) * page_bytes + static_cast<int64_t>(plane) * plane_bytes + at;
    const uint8_t *s = cache + base + from * page_bytes;
    uint8_t *d = cache + base + to * page_bytes;
    uint4 v[kPiece / 512];
#pragma unroll
    for (int j = 0; j < kPiece / 512; ++j)
      if (at + j * 512 < end) v[j] = __ldcs(reinterpret_cast<const uint4 *>(s + j * 512));
#pragma unroll
    for (int j = 0; j < kPiece / 512; ++j)
      if (at + j * 512 < end) *reinterpret_cast<uint4 *>(d + j * 512) = v[j];
  }
}

template <PagesOp OP>
cudaError_t plan(const PagesArgs &a, cudaStream_t st) {
  const size_t bytes = 4 * (static_cast<size_t>(a.n_pages + 31) / 32 + (OP == kPagesCompact ? 0 : a.n_slots));
  if (bytes > 40 * 1024)  // (with the static arrays, more than any kernel gets unasked)
    if (cudaError_t e = cudaFuncSetAttribute(pages_plan_kernel<OP>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             4 * (kMaxPages / 32 + kMaxSlots)))
      return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kPRanks);
  cfg.blockDim = dim3(kPThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kPRanks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, pages_plan_kernel<OP>, a);
}

}  // namespace

cudaError_t pages_launch(PagesOp op, const PagesArgs &a, cudaStream_t st) {
  return op == kPagesGrow ? plan<kPagesGrow>(a, st)
         : op == kPagesFork ? plan<kPagesFork>(a, st)
                            : plan<kPagesCompact>(a, st);
}

cudaError_t pages_move_launch(PagesOp op, const PagesArgs &a, kda_bf16 *cache, int layers,
                              int planes, int row_bytes, cudaStream_t st) {
  // eight CTAs an SM fill its threads; fewer where there can be no more moves
  const int64_t pieces = ((static_cast<int64_t>(row_bytes) << a.page_shift) + kPiece - 1) / kPiece *
                         planes * layers * a.ws_n;
  const int64_t ctas = (pieces + kMThreads / 32 - 1) / (kMThreads / 32);
  const dim3 grid(static_cast<unsigned>(ctas < 152 * 8 ? ctas : 152 * 8));
  uint8_t *bytes = reinterpret_cast<uint8_t *>(cache);
  return op == kPagesFork
             ? launch_pdl(pages_move_kernel<true>, grid, dim3(kMThreads), 0, st, a, bytes, layers, planes, row_bytes)
             : launch_pdl(pages_move_kernel<false>, grid, dim3(kMThreads), 0, st, a, bytes, layers, planes, row_bytes);
}

}  // namespace kda

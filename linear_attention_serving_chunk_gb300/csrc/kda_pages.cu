// Pages of a cache: giving them to sequences, sharing them, moving them together.
//
// A page is in use where a row of the table reaches it within its sequence's length.  There are no
// reference counts: every call marks the pages in use from the table itself, so a sequence is freed
// by its length alone and shared pages need no care.  One planning kernel does that and what
// follows from it; a second one moves what the plan says.
//
// Planning.  One cluster of 8 CTAs, so that little passes through global memory and no launch follows
// another:
//   1. mark: a warp takes 256 entries of a row, by prefix sums over the rows' entries, so that long rows are
//      no one's alone, and sets a bit for each page in a bitmap of its CTA's shared memory (OR in any
//      order gives the same bits; 128 KB for the largest pool, 2^20);
//   2. each CTA ORs an eighth of the eight bitmaps, four words a thread, and leaves the words and how many
//      unused pages of its share lie before each;
//   3. a warp takes a word and a lane a page: from the word and the counts, read where they lie, follows
//      the page's rank among the unused (or the used) ones.  grow: the k-th unused page goes to the row
//      whose demand covers rank k, found by bisection in the prefix sums of the demands; fork: to the k-th
//      fork with a partial last page; compact: with u pages in use, the k-th unused page below u takes
//      the k-th used page from u on.
// What bounds it: the latency of a dozen dependent steps and three or four cluster barriers (1100 cycles
// each), and for large tables the loads of step 1, which 256 warps have in flight at once.  Us in a graph: 8.4
// for a few pages of 8 sequences, 25 for 107,000 pages of 512 sequences with 257,000 in use (53 where a
// thread took its words' pages in turn and a warp a row; 45 where all lanes of a warp read the same remote
// word, since those reads are served one after another).
//
// Moving.  A warp takes 4 KB pieces of (page, layer, K or V of a head), eight 16-byte loads in
// flight a lane; sources and destinations are disjoint, so pieces need no order.  Bound by memory: 130 us for
// the last pages of 224 forks in 16 layers (904 MB, 6.9 TB/s), 350 us for 2.2 GB of a compaction.
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
__device__ __forceinline__ uint4 remote4(const void *p, unsigned rank) {
  uint32_t there;
  uint4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(there)
               : "r"(sm100::smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(there)
               : "memory");
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

constexpr int kEntries = 256;  // entries of the table that a warp takes at once, eight a lane

struct Plan {
  const PagesArgs &a;
  int *pieces;  // shared: the prefix sums of the rows' entries in use, in pieces
  int *rows;    // shared: grow, the prefix sums of the demands; fork, the fork that takes each row

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

// Words of the bitmap that one CTA counts, and of the whole: a multiple of what a thread takes.
__host__ __device__ constexpr int share_of(int n_pages) {
  return ((n_pages + 31) / 32 + 4 * kPRanks - 1) / (4 * kPRanks) * 4;
}

template <PagesOp OP>
__global__ void __launch_bounds__(kPThreads, 1) pages_plan_kernel(const PagesArgs a) {
  extern __shared__ __align__(16) uint32_t bits[];
  __shared__ int s_total;
  __shared__ int s_rank[kPThreads];  // fork: of the fresh page; -1: needs none, -2: not made
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = static_cast<int>(cluster_rank());
  const int share = share_of(a.n_pages), words = share * kPRanks;
  int *const counts = reinterpret_cast<int *>(bits + words);  // unused pages of the share before each word
  const Plan plan{a, counts + share, counts + share + a.n_slots};
  int *const pieces = plan.pieces, *const rows = plan.rows;
  const int wid = warp * kPRanks + rank, all_warps = kPRanks * 32;
  int bad = 0;
  if (OP != kPagesGrow) grid_launch_dependents();

  // 1. marks; pages that there are not are in use
  for (int w = tid; w < words; w += kPThreads) {
    const int n = a.n_pages - w * 32;
    bits[w] = n >= 32 ? 0u : n <= 0 ? ~0u : ~0u << n;
  }
  int want = 0;  // fork: those with a partial last page
  if (OP == kPagesFork) {
    for (int b = tid; b < a.n_slots; b += kPThreads) rows[b] = kNone;
    __syncthreads();
    for (int i = tid; i < a.m; i += kPThreads)
      if (plan.fork_in_range(i)) atomicMin(&rows[a.dst[i]], i);
  }
  __syncthreads();
  // The entries in use of each row, and what grow's rows want, by all CTAs alike.
  int n_pieces = 0;
  int64_t demand = 0;
  for (int b0 = 0; b0 < a.n_slots; b0 += kPThreads) {
    const int b = b0 + tid;
    int have = 0, more = 0, all;
    if (b < a.n_slots && !(OP == kPagesFork && rows[b] != kNone && plan.fork_made(rows[b]))) {
      have = plan.pages_of(a.lens[b]);
      if (OP == kPagesGrow) {
        const int need = plan.pages_of(a.want[b]);
        if (need < 0) bad = 1;
        if (have >= 0 && need > have) more = need - have;
      }
      if (have < 0) {
        have = 0;
        bad = 1;
      }
    }
    const int mine = (have + kEntries - 1) / kEntries, before = block_scan(mine, all);
    if (b < a.n_slots) pieces[b] = n_pieces + before + mine;
    n_pieces += all;
    if (OP == kPagesGrow) {
      const int wanted = block_scan(more, all);
      if (b < a.n_slots) rows[b] = static_cast<int>(min(demand + wanted + more, int64_t(1) << 30));
      demand += all;
    }
  }
  __syncthreads();
  for (int x = wid; x < n_pieces; x += all_warps) {
    int b = 0;
    for (int hi = a.n_slots, step = hi; step > 1;) {  // the row of piece x, 32 ways at a time
      step = (hi - b + 31) / 32;
      const int f = __ffs(__ballot_sync(0xffffffffu, pieces[min(b + (lane + 1) * step, hi) - 1] > x)) - 1;
      b += f * step;
      hi = min(hi, b + step);
    }
    const int need = plan.pages_of(a.lens[b]), i0 = (x - (b ? pieces[b - 1] : 0)) * kEntries + lane;
    const int32_t *row = a.table + static_cast<int64_t>(b) * a.max_pages;
    int p[kEntries / 32];
#pragma unroll
    for (int j = 0; j < kEntries / 32; ++j) p[j] = i0 + 32 * j < need ? row[i0 + 32 * j] : 0;
#pragma unroll
    for (int j = 0; j < kEntries / 32; ++j) {
      if (i0 + 32 * j >= need) continue;
      if (p[j] >= 0 && p[j] < a.n_pages) atomicOr(&bits[p[j] >> 5], 1u << (p[j] & 31));
      else if (p[j] != -1) bad = 1;  // (-1: given up)
    }
  }

  // Forks i0 ..: their ranks in s_rank, `before` and what they want themselves in front of the next ones.
  auto fork_ranks = [&](int i0, int before) {
    const int i = i0 + tid;
    const bool made = i < a.m && plan.fork_made(i), tail = made && plan.fork_tail(i);
    int all;
    const int at = block_scan(tail, all);
    s_rank[tid] = tail ? before + at : made ? -1 : -2;
    if (i < a.m && !made) bad = 1;
    __syncthreads();
    return all;
  };
  if (OP == kPagesFork)
    for (int i0 = 0; i0 < a.m; i0 += kPThreads) want += fork_ranks(i0, want);

  // 2. this CTA's share of all marks, and the unused pages before each word
  cluster_sync();
  {
    const int w = rank * share + 4 * tid;
    uint4 v = make_uint4(0, 0, 0, 0);
    const bool some = 4 * tid < share;
    if (some) {
#pragma unroll
      for (unsigned q = 0; q < kPRanks; ++q) {
        const uint4 x = remote4(bits + w, q);
        v.x |= x.x, v.y |= x.y, v.z |= x.z, v.w |= x.w;
      }
      // (nobody else reads this CTA's share of this CTA's bitmap before the barrier)
      *reinterpret_cast<uint4 *>(bits + w) = v;
    }
    const int x = __popc(~v.x), y = __popc(~v.y), z = __popc(~v.z);
    int total;
    const int first = block_scan(some ? x + y + z + __popc(~v.w) : 0, total);
    if (some)
      *reinterpret_cast<int4 *>(counts + 4 * tid) =
          make_int4(first, first + x, first + x + y, first + x + y + z);
    if (tid == 0) s_total = total;
  }
  cluster_sync();
  int base[kPRanks], left = 0;  // unused pages in front of each share, and all
#pragma unroll
  for (int q = 0; q < kPRanks; ++q) {
    base[q] = left;
    left += static_cast<int>(remote(&s_total, q));
  }
  // A word of the marks, and the unused pages before it.
  auto word = [&](int w, int &before) -> uint32_t {
    const int q = w / share;
    before = static_cast<int>(remote(counts + (w - q * share), q));
#pragma unroll
    for (int r = 1; r < kPRanks; ++r)
      if (r == q) before += base[r];
    return remote(bits + w, q);
  };
  // Calls each(page, whether it is unused, unused pages before it) for a lane's pages, in ascending order,
  // until a word has `end` unused pages before it.  A warp has eight words in a row, and reads those of four
  // rounds at once, one in each lane: lanes that ask for the same remote word are served one after another.
  auto each_page = [&](int end, auto &&each) {
    for (int w0 = wid * 8; w0 < words; w0 += 32 * all_warps) {
      int k = end;
      const int mine = w0 + (lane / 8) * 8 * all_warps + lane % 8;
      const uint32_t v = mine < words ? ~word(mine, k) : 0u;
      for (int s = 0; s < 32; ++s) {
        const uint32_t u = __shfl_sync(0xffffffffu, v, s);
        const int before = __shfl_sync(0xffffffffu, k, s), w = __shfl_sync(0xffffffffu, mine, s);
        if (before >= end) {
          if (s % 8 == 0) return;  // (so have the words of later rounds)
          s |= 7;
          continue;
        }
        each(w * 32 + lane, u >> lane & 1, before + __popc(u & ((1u << lane) - 1)));
      }
    }
  };

  if (OP == kPagesGrow) {
    const int n = a.n_slots, given = n ? rows[n - 1] : 0;
    int begin = 0, end = 0;  // the ranks that the row of the warp's last page takes, and where
    int32_t *to = nullptr;
    each_page(given, [&](int p, bool unused, int k) {
      const bool mine = unused && k < given;
      if (__any_sync(0xffffffffu, mine && k >= end)) {
        int lo = 0, hi = n - 1;  // the first row whose demands end behind this rank
        while (lo < hi) {
          const int mid = (lo + hi) / 2;
          if (rows[mid] > k) hi = mid;
          else lo = mid + 1;
        }
        begin = lo ? rows[lo - 1] : 0;
        end = rows[lo];
        to = a.table + static_cast<int64_t>(lo) * a.max_pages + plan.pages_of(a.lens[lo]);
      }
      if (mine && end <= left) to[k - begin] = p;
      // ranks only rise: the last lane's row is where the next word goes on
      begin = __shfl_sync(0xffffffffu, begin, 31);
      end = __shfl_sync(0xffffffffu, end, 31);
      to = reinterpret_cast<int32_t *>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(to), 31));
    });
    if (given > left)  // a row gets all of its pages or none
      for (int b = wid; b < n; b += all_warps) {
        if (rows[b] <= left) continue;
        const int have = plan.pages_of(a.lens[b]), need = plan.pages_of(a.want[b]);
        if (have < 0) continue;
        for (int i = have + lane; i < need; i += 32)
          a.table[static_cast<int64_t>(b) * a.max_pages + i] = -1;
      }
    if (rank == 0 && tid == 0)
      *a.count = static_cast<int>(max(left - demand, -static_cast<int64_t>(kNone)));
  }

  if (OP == kPagesFork) {
    int32_t *src = a.ws + kPagesWsHead, *dst = src + a.ws_n, *len = dst + a.ws_n,
            *fresh = len + a.ws_n;
    each_page(want, [&](int p, bool unused, int k) {
      if (unused && k < want) fresh[k] = p;
    });
    cluster_sync();
    int before = 0;
    for (int i0 = 0; i0 < a.m; i0 += kPThreads) {
      if (a.m > kPThreads) before += fork_ranks(i0, before);  // (else they are there)
      const int across = max((a.max_pages + kEntries - 1) / kEntries, 1);
      const int64_t all = static_cast<int64_t>(min(kPThreads, a.m - i0)) * across;
      for (int64_t x = wid; x < all; x += all_warps) {
        const int j = static_cast<int>(x / across);
        const int e0 = static_cast<int>(x - static_cast<int64_t>(j) * across) * kEntries + lane;
        const int r = s_rank[j];
        if (r == -2) continue;
        const int s = a.src[i0 + j], d = a.dst[i0 + j], tokens = a.lens[s];
        const int32_t *from = a.table + static_cast<int64_t>(s) * a.max_pages;
        int32_t *to = a.table + static_cast<int64_t>(d) * a.max_pages;
        const bool none = r >= left;  // no page is left for it: an empty row
        const int need = none ? 0 : plan.pages_of(tokens);
        const int whole = need - (r >= 0 && !none), page = whole < need ? __ldcg(fresh + r) : -1;
#pragma unroll
        for (int e = e0; e < e0 + kEntries; e += 32)
          if (e < a.max_pages) to[e] = e < whole ? from[e] : e < need ? page : -1;
        if (e0 == 0) {
          a.lens[d] = none ? 0 : tokens;
          if (whole < need) {
            const int old = from[whole];
            const bool ok = old >= 0 && old < a.n_pages;
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
    int32_t *src = a.ws + kPagesWsHead, *dst = src + a.ws_n;
    const int used = a.n_pages - left;
    // the unused pages below `used`: as many as used ones lie from there on
    int holes = left;
    if (used < a.n_pages) {
      const uint32_t v = ~word(used / 32, holes);
      holes += __popc(v & ((1u << (used % 32)) - 1));
    }
    // rank of a used page among those from `used` on: the pages before it, less the unused ones and
    // the used ones below `used`
    each_page(kNone, [&](int p, bool unused, int k) {
      if (unused) {
        if (p < used) dst[k] = p;
      } else if (p >= used && p < a.n_pages) {
        src[p - k - (used - holes)] = p;
      }
    });
    cluster_sync();
    const int across = (a.max_pages + kEntries - 1) / kEntries;
    const int64_t all = static_cast<int64_t>(a.n_slots) * across;
    for (int64_t x = wid; x < all; x += all_warps) {
      const int b = static_cast<int>(x / across);
      const int i0 = static_cast<int>(x - static_cast<int64_t>(b) * across) * kEntries + lane;
      const int need = plan.pages_of(a.lens[b]);
      const int32_t *row = a.table + static_cast<int64_t>(b) * a.max_pages;
      int32_t *out = a.table_out + static_cast<int64_t>(b) * a.max_pages;
      int p[kEntries / 32];
#pragma unroll
      for (int j = 0; j < kEntries / 32; ++j) p[j] = i0 + 32 * j < need ? row[i0 + 32 * j] : -1;
#pragma unroll
      for (int j = 0; j < kEntries / 32; ++j) {
        if (p[j] >= used && p[j] < a.n_pages) {
          int k;
          const uint32_t v = ~word(p[j] / 32, k);
          k += __popc(v & ((1u << (p[j] % 32)) - 1));
          p[j] = __ldcg(dst + (p[j] - k - (used - holes)));
        }
        if (i0 + 32 * j < a.max_pages) out[i0 + 32 * j] = p[j];
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
    const int64_t base = static_cast<int64_t>(layer) * a.n_pages * page_bytes +
                         static_cast<int64_t>(plane) * plane_bytes + at;
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
  const size_t bytes = 4 * (static_cast<size_t>(share_of(a.n_pages)) * (kPRanks + 1) +
                            static_cast<size_t>(a.n_slots) * (OP == kPagesCompact ? 1 : 2));
  if (bytes > 40 * 1024)  // (with the static arrays, more than any kernel gets unasked)
    if (cudaError_t e = cudaFuncSetAttribute(pages_plan_kernel<OP>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             4 * (kMaxPages / 32 / kPRanks * (kPRanks + 1) + 2 * kMaxSlots)))
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
  const auto kernel = op == kPagesFork ? pages_move_kernel<true> : pages_move_kernel<false>;
  return launch_pdl(kernel, grid, dim3(kMThreads), 0, st, a, bytes, layers, planes, row_bytes);
}

}  // namespace kda

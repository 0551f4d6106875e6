// Page operations of paged pools: copying, forking, allocating, freeing and
// compacting 128-token pages that block tables map and reference counts own
// (0: free).  All bookkeeping stays on the device, so a serving step that
// forks or frees sequences can be enqueued without a round trip to the host.
//
// Every operation gives the same result whatever order its threads run in:
// counts change by integer atomics, table entries are claimed by exchanges,
// and pages are dealt by rank (the lowest free id first).  The bookkeeping is
// bound by launch latency, so each operation does all of it in one launch: one
// cluster of CTAs whose steps are separated by cluster barriers, and whose
// error words are joined at the end into the status (no clearing launch).
// Fork of 32 sequences of up to 4000 tokens, 16 MB of last pages moved: 14.4 us.
// Page contents move in 16-byte chunks, four per thread in flight, by a grid of
// their own; copying is bound by HBM, 2 bytes per byte moved (a
// compaction that moves 440 MB both ways counted: 77 us, 5.7 TB/s).
#include "msa_pages.h"
#include "msa_q8.cuh"
#include "msa_tma.h"

namespace msa {
namespace {

constexpr int kThreads = 512;
constexpr int kSeg = kThreads * 16 * 4;   // bytes of a page copied by one CTA step
constexpr int kBook = 1024;               // threads of a bookkeeping CTA
constexpr int kBookCtas = 8;              // CTAs of the bookkeeping cluster

// The workspace: status word; then per-page words: the free list (and fork's
// source and destination pages), or of a compaction the holes, the pages that
// fill them and each page's fate.
constexpr size_t kWsHead = 256;
struct PageWs {
  int* status;
  int32_t* count;   // pages that a compaction moves
  int32_t* x;       // free list, or holes
  int32_t* y;       // source pages, or movers
  int32_t* z;       // destination pages, or fates
};
PageWs carve(char* ws, int pages) {
  int32_t* w = reinterpret_cast<int32_t*>(ws);
  PageWs p;
  p.status = w;
  p.count = w + 1;
  p.x = w + kWsHead / 4;
  const int n = pages > kMaxBatch ? pages : kMaxBatch;
  p.y = p.x + n;
  p.z = p.y + n;
  return p;
}

// The worse of two codes (no page left before an invalid entry).
__device__ __forceinline__ int worse(int x, int y) { return max(x, y); }

// Joins every thread's code over the cluster and writes the status; a barrier
// over the cluster.
__device__ __forceinline__ void write_status(int code, int* status) {
  __shared__ int sm_code;
  if (threadIdx.x == 0) sm_code = 0;
  __syncthreads();
  if (code) atomicMax(&sm_code, code);
  cluster_sync();
  if (cluster_rank() == 0 && threadIdx.x == 0) {
    int c = 0;
    for (int r = 0; r < kBookCtas; ++r) c = worse(c, ld_cluster_int(&sm_code, r));
    *status = c;
  }
  cluster_sync();   // no CTA leaves while its word is read
}

// ---- page contents ---------------------------------------------------------
struct CopyPlan {
  PoolSet ps;
  int seg0[kMaxPools + 1];   // first segment of each pool; seg0[n]: segments of a page
};

CopyPlan copy_plan(const PoolSet& ps) {
  CopyPlan c;
  c.ps = ps;
  c.seg0[0] = 0;
  for (int i = 0; i < ps.n; ++i)
    c.seg0[i + 1] = c.seg0[i] + (int)((ps.pool[i].page_bytes + kSeg - 1) / kSeg);
  return c;
}

// Segment `seg` of page src -> page dst: all of it, or the first `rows` of 128
// token rows of the pools that hold rows.
__device__ __forceinline__ void copy_segment(const CopyPlan& c, int seg, int64_t src, int64_t dst,
                                             int rows) {
  int i = 0;
  while (c.seg0[i + 1] <= seg) ++i;
  const msa_pool& p = c.ps.pool[i];
  const int64_t pb = (int64_t)p.page_bytes;
  const int64_t end = p.per_token ? pb / kBlock * rows : pb;
  const int64_t o0 = (int64_t)(seg - c.seg0[i]) * kSeg;
  const int64_t o1 = min(end, o0 + kSeg);
  const char* s = static_cast<const char*>(p.base) + src * pb;
  char* d = static_cast<char*>(p.base) + dst * pb;
  if ((pb & 15) == 0 && (end & 15) == 0 && ((uintptr_t)p.base & 15) == 0) {
    uint4 v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t o = o0 + (int64_t)(u * kThreads + threadIdx.x) * 16;
      if (o < o1) v[u] = *reinterpret_cast<const uint4*>(s + o);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t o = o0 + (int64_t)(u * kThreads + threadIdx.x) * 16;
      if (o < o1) *reinterpret_cast<uint4*>(d + o) = v[u];
    }
  } else {
    for (int64_t o = o0 + threadIdx.x; o < o1; o += kThreads) d[o] = s[o];
  }
}

__global__ void __launch_bounds__(kThreads) pages_copy_kernel(const __grid_constant__ CopyPlan c,
                                                              int pages,
                                                              const int32_t* __restrict__ src,
                                                              const int32_t* __restrict__ dst,
                                                              int n, int* status) {
  auto bad = [&](int j) {
    const int s = src[j], d = dst[j];
    return s < 0 || s >= pages || d < 0 || d >= pages;
  };
  if (blockIdx.x == 0) {   // the first CTA looks all pairs over and writes the status
    bool any = false;
    for (int j = threadIdx.x; j < n; j += kThreads) any |= bad(j);
    any = __syncthreads_or(any);
    if (threadIdx.x == 0) *status = any ? kDevInvalid : 0;
  }
  const int segs = c.seg0[c.ps.n];
  for (int64_t w = blockIdx.x; w < (int64_t)n * segs; w += gridDim.x) {
    const int j = (int)(w / segs), seg = (int)(w % segs);
    if (!bad(j) && src[j] != dst[j]) copy_segment(c, seg, src[j], dst[j], kBlock);
  }
}

// ---- reference counts --------------------------------------------------------
// One mapping of page e less; a page that no entry mapped is reported and kept at 0.
__device__ __forceinline__ int release(const PageTable& pt, int e) {
  if (e == -1) return 0;
  if (e < 0 || e >= pt.pages) return kDevInvalid;
  if (atomicSub(pt.refs + e, 1) > 0) return 0;
  atomicAdd(pt.refs + e, 1);
  return kDevInvalid;
}

// Sum of v over the CTA (every thread gets it).
__device__ __forceinline__ int cta_sum(int v, int* sm) {
  v = __reduce_add_sync(0xffffffffu, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  int t = 0;
  for (int w = 0; w < (int)(blockDim.x >> 5); ++w) t += sm[w];
  return t;
}
// Exclusive prefix of a flag over the CTA, and its total.
__device__ __forceinline__ int cta_rank(bool f, int* sm, int* total) {
  const unsigned m = __ballot_sync(0xffffffffu, f);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __syncthreads();
  if (lane == 0) sm[warp] = __popc(m);
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < (int)(blockDim.x >> 5); ++w) {
    before += w < warp ? sm[w] : 0;
    all += sm[w];
  }
  *total = all;
  return before + __popc(m & ((1u << lane) - 1));
}
// Pages of [lo, hi) in use, counted by the CTA (past L1: the counts may have
// changed in this launch).
__device__ __forceinline__ int cta_live(const int32_t* refs, int lo, int hi, int* sm) {
  int n = 0;
  for (int i = lo + threadIdx.x; i < hi; i += blockDim.x) n += __ldcg(refs + i) > 0;
  return cta_sum(n, sm);
}

// This CTA's share of the cluster's pages.
__device__ __forceinline__ void page_range(int pages, int& lo, int& hi) {
  const int chunk = (pages + kBookCtas - 1) / kBookCtas;
  lo = min(pages, cluster_rank() * chunk);
  hi = min(pages, lo + chunk);
}

// The first `most` free pages in ascending order into list, by the cluster;
// returns how many there are.  A barrier over the cluster before and after.
__device__ __forceinline__ int list_free(const PageTable& pt, int most, int32_t* list, int* sm) {
  __shared__ int sm_free;
  int lo, hi;
  cluster_sync();
  page_range(pt.pages, lo, hi);
  const int live = cta_live(pt.refs, lo, hi, sm);
  if (threadIdx.x == 0) sm_free = hi - lo - live;
  cluster_sync();
  int r = 0, all = 0;
  for (int c = 0; c < kBookCtas; ++c) {
    const int f = ld_cluster_int(&sm_free, c);
    r += c < cluster_rank() ? f : 0;
    all += f;
  }
  for (int i0 = lo; i0 < hi && r < most; i0 += blockDim.x) {
    const int i = i0 + threadIdx.x;
    const bool f = i < hi && __ldcg(pt.refs + i) <= 0;
    int total;
    const int k = r + cta_rank(f, sm, &total);
    if (f && k < most) list[k] = i;
    r += total;
  }
  cluster_sync();
  return min(all, most);
}

// Unmaps ranges of blocks, range after range: one block of 64 rows 38 us, of 256
// rows 155 us, 4096 blocks of one row 3.3 us.
__global__ void __launch_bounds__(kBook) pages_free_kernel(PageTable pt,
                                                           const __grid_constant__ RowList rl,
                                                           PageWs w) {
  int code = 0;
  for (int j = 0; j < rl.n; ++j) {
    int32_t* row = pt.table + (int64_t)rl.a[j] * pt.max_blocks;
    for (int kb = rl.b[j] + blockIdx.x * kBook + threadIdx.x; kb < rl.c[j]; kb += kBookCtas * kBook)
      code = worse(code, release(pt, atomicExch(row + kb, -1)));
  }
  write_status(code, w.status);
}

// Fork: every destination row lets go of its pages and takes the source's
// complete ones; then the pairs with a partly filled last page take free pages
// in order.  Pair j's source and destination page go to w.y and w.z (-1: none).
__global__ void __launch_bounds__(kBook) pages_fork_kernel(PageTable pt,
                                                           const __grid_constant__ RowList rl,
                                                           PageWs w) {
  __shared__ int sm[32];
  int code = 0;
  const int64_t entries = (int64_t)rl.n * pt.max_blocks;
  for (int64_t x = (int64_t)blockIdx.x * kBook + threadIdx.x; x < entries; x += kBookCtas * kBook) {
    const int j = (int)(x / pt.max_blocks), kb = (int)(x % pt.max_blocks);
    int32_t* dst = pt.table + (int64_t)rl.b[j] * pt.max_blocks + kb;
    // both reads, then both counts in flight at once
    const bool share = kb < rl.c[j] / kBlock;
    int e = share ? pt.table[(int64_t)rl.a[j] * pt.max_blocks + kb] : -1;
    const int old = *dst;
    // A page that nobody counts is not shared: its count would then miss the
    // source's mapping for good.  So no thread adds to such a count, and the
    // source's own mapping keeps a counted page's above 0: what is read here does
    // not depend on the order of the threads.
    const bool counted = e >= 0 && e < pt.pages && __ldcg(pt.refs + e) > 0;
    if (share && !counted) code = worse(code, kDevInvalid);
    if (!counted) e = -1;
    if (counted) atomicAdd(pt.refs + e, 1);
    code = worse(code, release(pt, old));
    *dst = e;
  }
  // pair j of thread j: does its last page need a copy, and which free page is its
  const int j = threadIdx.x;
  const bool part = j < rl.n && rl.c[j] % kBlock != 0;
  int need;
  const int kb = part ? rl.c[j] / kBlock : 0;
  int from = part ? pt.table[(int64_t)rl.a[j] * pt.max_blocks + kb] : -1;   // no row of dst_rows
  const int f = cta_rank(part, sm, &need);
  const int got = need ? list_free(pt, need, w.x, sm) : 0;
  if (blockIdx.x == 0) {
    int to = -1;
    // a page that nobody counts is on the free list: another pair may write it
    if (part && (from < 0 || from >= pt.pages || __ldcg(pt.refs + from) <= 0)) {
      code = worse(code, kDevInvalid);
      from = -1;
    }
    __syncthreads();                 // every count is read before a page is handed out
    if (from >= 0) {
      if (f >= got) {
        code = worse(code, kDevNoPages);
        from = -1;
      } else {
        to = __ldcg(w.x + f);
        pt.table[(int64_t)rl.b[j] * pt.max_blocks + kb] = to;
        pt.refs[to] = 1;
      }
    }
    if (j < rl.n) {
      w.y[j] = from;
      w.z[j] = to;
    }
  }
  write_status(code, w.status);
}

// The used rows of the partly filled pages.
__global__ void __launch_bounds__(kThreads) pages_fork_copy_kernel(
    const __grid_constant__ CopyPlan c, const __grid_constant__ RowList rl, PageWs w) {
  const int j = blockIdx.y, rows = rl.c[j] % kBlock, to = w.z[j];
  if (to < 0) return;
  for (int seg = blockIdx.x; seg < c.seg0[c.ps.n]; seg += gridDim.x)
    copy_segment(c, seg, w.y[j], to, rows);
}

// Maps the unmapped blocks of the ranges, in order, to the lowest free pages.  One
// CTA takes range after range: one block of 64 rows 108 us, of 256 rows 414 us (1.6
// us a row: a table read and the rank of its result), 4096 blocks of one row 13.6 us.
__global__ void __launch_bounds__(kBook) pages_alloc_kernel(PageTable pt,
                                                            const __grid_constant__ RowList rl,
                                                            PageWs w) {
  __shared__ int sm[32];
  int code = 0;
  const int n = list_free(pt, pt.pages, w.x, sm);
  if (blockIdx.x == 0) {
    int r = 0;
    for (int j = 0; j < rl.n; ++j) {
      int32_t* row = pt.table + (int64_t)rl.a[j] * pt.max_blocks;
      for (int k0 = rl.b[j]; k0 < rl.c[j]; k0 += kBook) {
        const int kb = k0 + threadIdx.x;
        const int e = kb < rl.c[j] ? row[kb] : 0;
        if (e < -1 || e >= pt.pages) code = worse(code, kDevInvalid);
        int total;
        const int k = r + cta_rank(e == -1, sm, &total);
        if (e == -1) {
          if (k < n) {
            const int pg = __ldcg(w.x + k);
            row[kb] = pg;
            pt.refs[pg] = 1;
          } else {
            code = worse(code, kDevNoPages);
          }
        }
        r += total;
      }
    }
  }
  write_status(code, w.status);
}

// ---- compaction ------------------------------------------------------------
constexpr int kStays = -1, kDead = INT32_MIN;   // fates; a mover holds its rank, hole h holds -2 - h

__global__ void __launch_bounds__(kBook) pages_plan_kernel(PageTable pt, PageWs w, int32_t* live_out) {
  __shared__ int sm[32];
  __shared__ int sm_live, sm_low;
  int lo, hi;
  page_range(pt.pages, lo, hi);
  const int mine = cta_live(pt.refs, lo, hi, sm);
  if (threadIdx.x == 0) sm_live = mine;
  cluster_sync();
  int r = 0, live = 0;                            // live pages before lo, in all
  for (int c = 0; c < kBookCtas; ++c) {
    const int n = ld_cluster_int(&sm_live, c);
    r += c < cluster_rank() ? n : 0;
    live += n;
  }
  const int mylow = cta_live(pt.refs, lo, max(lo, min(hi, live)), sm);
  if (threadIdx.x == 0) sm_low = mylow;
  cluster_sync();
  int low = 0;                                    // live pages already below `live`
  for (int c = 0; c < kBookCtas; ++c) low += ld_cluster_int(&sm_low, c);
  for (int i0 = lo; i0 < hi; i0 += kBook) {
    const int i = i0 + threadIdx.x;
    const bool f = i < hi && pt.refs[i] > 0;
    int total;
    const int k = r + cta_rank(f, sm, &total);
    if (i < hi) {
      int fate = kStays;
      if (f && i >= live) {
        fate = k - low;
        w.y[fate] = i;
      } else if (!f) {
        fate = kDead;
        if (i < live) {
          w.x[i - k] = i;
          fate = -2 - (i - k);
        }
      }
      w.z[i] = fate;
    }
    r += total;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *w.status = 0;                                // for the next kernel's reports
    *w.count = live - low;
    *live_out = live;
  }
  cluster_sync();                                 // no CTA leaves while its words are read
}

__global__ void __launch_bounds__(kThreads) pages_move_kernel(const __grid_constant__ CopyPlan c,
                                                              PageTable pt, int32_t* table_out,
                                                              int32_t* refs_out, PageWs w) {
  const int moves = *w.count;
  const int64_t tid = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int64_t step = (int64_t)gridDim.x * blockDim.x;
  const int64_t entries = (int64_t)pt.rows * pt.max_blocks;
  for (int64_t i = tid; i < entries; i += step) {
    int e = pt.table[i];
    if (e >= 0 && e < pt.pages) {
      const int fate = w.z[e];
      if (fate >= 0) {
        e = w.x[fate];
      } else if (fate != kStays) {
        // a page nobody counts: another row's page may move there, and the
        // entry would pass for a counted mapping of it
        atomicMax(w.status, kDevInvalid);
        e = -1;
      }
    } else if (e != -1) {
      atomicMax(w.status, kDevInvalid);
      e = -1;
    }
    table_out[i] = e;
  }
  // a hole's thread moves the count of the page that fills it (refs_out may be refs)
  for (int64_t i = tid; i < pt.pages; i += step) {
    const int fate = w.z[i];
    if (fate == kStays) {
      refs_out[i] = pt.refs[i];
    } else if (fate == kDead) {
      refs_out[i] = 0;
    } else if (fate < 0) {
      const int from = w.y[-2 - fate];
      refs_out[i] = pt.refs[from];
      refs_out[from] = 0;
    }
  }
  const int segs = c.seg0[c.ps.n];
  for (int64_t s = blockIdx.x; s < (int64_t)moves * segs; s += gridDim.x) {
    const int j = (int)(s / segs);
    copy_segment(c, (int)(s % segs), w.y[j], w.x[j], kBlock);
  }
}

template <typename... A>
cudaError_t launch_book(void (*kernel)(A...), cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(kBookCtas);
  cfg.blockDim = dim3(kBook);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = kBookCtas;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  note_launches(1);
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

size_t pages_workspace_bytes(int pages) {
  // at least one word per row of a list (fork's pairs)
  const size_t n = pages > kMaxBatch ? pages : kMaxBatch;
  return kWsHead + n * 3 * sizeof(int32_t);
}

cudaError_t launch_pages_copy(const PoolSet& ps, int pages, const int32_t* src, const int32_t* dst,
                              int n, char* ws, cudaStream_t st) {
  const PageWs w = carve(ws, pages);
  const CopyPlan c = copy_plan(ps);
  const int64_t work = (int64_t)n * c.seg0[ps.n], most = sm_count() * 4;
  note_launches(1);
  pages_copy_kernel<<<(unsigned)(work < most ? work : most), kThreads, 0, st>>>(c, pages, src, dst, n,
                                                                              w.status);
  return cudaGetLastError();
}

cudaError_t launch_pages_fork(const PoolSet& ps, const PageTable& pt, const RowList& rows, char* ws,
                              cudaStream_t st) {
  const PageWs w = carve(ws, pt.pages);
  const CopyPlan c = copy_plan(ps);
  cudaError_t e = launch_book(pages_fork_kernel, st, pt, rows, w);
  if (e != cudaSuccess) return e;
  bool part = false;
  for (int j = 0; j < rows.n; ++j) part |= rows.c[j] % kBlock != 0;
  const int segs = c.seg0[ps.n];
  if (part && segs > 0) {
    note_launches(1);
    pages_fork_copy_kernel<<<dim3(segs < 64 ? segs : 64, rows.n), kThreads, 0, st>>>(c, rows, w);
  }
  return cudaGetLastError();
}

cudaError_t launch_pages_free(const PageTable& pt, const RowList& rows, char* ws, cudaStream_t st) {
  return launch_book(pages_free_kernel, st, pt, rows, carve(ws, pt.pages));
}

cudaError_t launch_pages_alloc(const PageTable& pt, const RowList& rows, char* ws, cudaStream_t st) {
  return launch_book(pages_alloc_kernel, st, pt, rows, carve(ws, pt.pages));
}

cudaError_t launch_pages_compact(const PoolSet& ps, const PageTable& pt, int32_t* table_out,
                                 int32_t* refs_out, int32_t* live, char* ws, cudaStream_t st) {
  const PageWs w = carve(ws, pt.pages);
  const CopyPlan c = copy_plan(ps);
  const cudaError_t e = launch_book(pages_plan_kernel, st, pt, w, live);
  if (e != cudaSuccess) return e;
  note_launches(1);
  pages_move_kernel<<<sm_count() * 4, kThreads, 0, st>>>(c, pt, table_out, refs_out, w);
  return cudaGetLastError();
}

}  // namespace msa

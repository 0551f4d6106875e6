// Page operations of paged pools: copying, forking, allocating, freeing and
// compacting 128-token pages that block tables map and reference counts own
// (0: free).  All bookkeeping stays on the device, so a serving step that
// forks or frees sequences can be enqueued without a round trip to the host.
//
// Every operation gives the same result whatever order its threads run in:
// counts change by integer atomics, table entries are claimed by exchanges,
// and pages are dealt by rank (the lowest free id first).  A list of free
// pages is made by CTAs that each count the free pages before their own chunk
// (reading the counts once more costs less than a second launch up to about
// a million pages).  Page contents move in 16-byte chunks, four per thread in
// flight; copying is bound by HBM, 2 bytes per byte moved, the rest by launch
// latency.
#include "msa_device.cuh"
#include "msa_pages.h"
#include "msa_tma.h"

namespace msa {
namespace {

constexpr int kThreads = 512;
constexpr int kSeg = kThreads * 16 * 4;   // bytes of a page copied by one CTA step
constexpr int kMaxListCtas = 128;
constexpr int kChunk = 1024;              // least pages of a free-list CTA

// The workspace: status word; then per-page words of the free list, or of a
// compaction the holes, the pages that fill them and each page's fate.
constexpr size_t kWsHead = 256;
struct PageWs {
  int* status;
  int32_t* count;   // pages listed (free list) or moved (compaction)
  int32_t* live;
  int32_t* x;       // free list, or holes
  int32_t* y;       // movers
  int32_t* z;       // fates
};
PageWs carve(char* ws, int pages) {
  int32_t* w = reinterpret_cast<int32_t*>(ws);
  PageWs p;
  p.status = w;
  p.count = w + 1;
  p.live = w + 2;
  p.x = w + kWsHead / 4;
  p.y = p.x + pages;
  p.z = p.y + pages;
  return p;
}

__device__ __forceinline__ void flag(int* status, int code) { atomicMax(status, code); }

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
  const int segs = c.seg0[c.ps.n];
  for (int64_t w = blockIdx.x; w < (int64_t)n * segs; w += gridDim.x) {
    const int j = (int)(w / segs), seg = (int)(w % segs);
    const int s = src[j], d = dst[j];
    if (s < 0 || s >= pages || d < 0 || d >= pages) {
      if (threadIdx.x == 0) flag(status, kDevInvalid);
      continue;
    }
    if (s != d) copy_segment(c, seg, s, d, kBlock);
  }
}

// ---- reference counts --------------------------------------------------------
// One mapping of page e less; a page that no entry mapped is flagged and kept at 0.
__device__ __forceinline__ void release(const PageTable& pt, int e, int* status) {
  if (e == -1) return;
  if (e < 0 || e >= pt.pages) {
    flag(status, kDevInvalid);
    return;
  }
  if (atomicSub(pt.refs + e, 1) <= 0) {
    atomicAdd(pt.refs + e, 1);
    flag(status, kDevInvalid);
  }
}

__global__ void __launch_bounds__(256) pages_free_kernel(PageTable pt,
                                                         const __grid_constant__ RowList rl,
                                                         int* status) {
  const int j = blockIdx.y;
  int32_t* row = pt.table + (int64_t)rl.a[j] * pt.max_blocks;
  for (int kb = rl.b[j] + blockIdx.x * blockDim.x + threadIdx.x; kb < rl.c[j];
       kb += gridDim.x * blockDim.x)
    release(pt, atomicExch(row + kb, -1), status);
}

// Fork, step 1: the destination row lets go of its pages and takes the
// source's complete ones.
__global__ void __launch_bounds__(256) pages_share_kernel(PageTable pt,
                                                          const __grid_constant__ RowList rl,
                                                          int* status) {
  const int j = blockIdx.y, whole = rl.c[j] / kBlock;
  const int32_t* src = pt.table + (int64_t)rl.a[j] * pt.max_blocks;
  int32_t* dst = pt.table + (int64_t)rl.b[j] * pt.max_blocks;
  for (int kb = blockIdx.x * blockDim.x + threadIdx.x; kb < pt.max_blocks;
       kb += gridDim.x * blockDim.x) {
    int e = -1;
    if (kb < whole) {
      e = src[kb];
      if (e < 0 || e >= pt.pages) {
        flag(status, kDevInvalid);
        e = -1;
      } else {
        atomicAdd(pt.refs + e, 1);
      }
    }
    release(pt, dst[kb], status);
    dst[kb] = e;
  }
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
// Pages of [lo, hi) in use, counted by the CTA.
__device__ __forceinline__ int cta_live(const int32_t* refs, int lo, int hi, int* sm) {
  int n = 0;
  for (int i = lo + threadIdx.x; i < hi; i += blockDim.x) n += refs[i] > 0;
  return cta_sum(n, sm);
}

// Free pages in ascending order; CTA c lists those of chunk c.
__global__ void __launch_bounds__(1024) pages_list_kernel(const int32_t* __restrict__ refs, int pages,
                                                          int chunk, PageWs w) {
  __shared__ int sm[32];
  const int lo = blockIdx.x * chunk, hi = min(pages, lo + chunk);
  int r = lo - cta_live(refs, 0, lo, sm);
  for (int i0 = lo; i0 < hi; i0 += blockDim.x) {
    const int i = i0 + threadIdx.x;
    const bool f = i < hi && refs[i] <= 0;
    int total;
    const int k = cta_rank(f, sm, &total);
    if (f) w.x[r + k] = i;
    r += total;
  }
  if (blockIdx.x == gridDim.x - 1 && threadIdx.x == 0) *w.count = r;
}

// Fork, step 3: pair j with a partly filled last page takes free page number
// (pairs with one before j) and the used rows of the source's page.
__global__ void __launch_bounds__(kThreads) pages_fork_copy_kernel(
    const __grid_constant__ CopyPlan c, PageTable pt, const __grid_constant__ RowList rl, PageWs w) {
  const int segs = c.seg0[c.ps.n];
  const int j = blockIdx.y, rows = rl.c[j] % kBlock, kb = rl.c[j] / kBlock;
  if (rows == 0) return;
  int f = 0;
  for (int k = 0; k < j; ++k) f += rl.c[k] % kBlock != 0;
  const int from = pt.table[(int64_t)rl.a[j] * pt.max_blocks + kb];
  const bool bad = from < 0 || from >= pt.pages, none = f >= *w.count;
  const int to = none ? -1 : w.x[f];
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    if (bad) flag(w.status, kDevInvalid);
    if (none) flag(w.status, kDevNoPages);
    if (!bad && !none) {
      pt.table[(int64_t)rl.b[j] * pt.max_blocks + kb] = to;
      pt.refs[to] = 1;
    }
  }
  if (bad || none) return;
  for (int seg = blockIdx.x; seg < segs; seg += gridDim.x) copy_segment(c, seg, from, to, rows);
}

// Maps the unmapped blocks of the ranges, in order, to the listed pages.
__global__ void __launch_bounds__(1024) pages_alloc_kernel(PageTable pt,
                                                           const __grid_constant__ RowList rl,
                                                           PageWs w) {
  __shared__ int sm[32];
  int r = 0;
  const int n = *w.count;
  for (int j = 0; j < rl.n; ++j) {
    int32_t* row = pt.table + (int64_t)rl.a[j] * pt.max_blocks;
    for (int k0 = rl.b[j]; k0 < rl.c[j]; k0 += blockDim.x) {
      const int kb = k0 + threadIdx.x;
      const int e = kb < rl.c[j] ? row[kb] : 0;
      if (e < -1 || e >= pt.pages) flag(w.status, kDevInvalid);
      int total;
      const int k = r + cta_rank(e == -1, sm, &total);
      if (e == -1) {
        if (k < n) {
          row[kb] = w.x[k];
          pt.refs[w.x[k]] = 1;
        } else {
          flag(w.status, kDevNoPages);
        }
      }
      r += total;
    }
  }
}

// ---- compaction ------------------------------------------------------------
constexpr int kStays = -1, kDead = INT32_MIN;   // fates; a mover holds its rank, hole h holds -2 - h

__global__ void __launch_bounds__(1024) pages_plan_kernel(const int32_t* __restrict__ refs, int pages,
                                                          int chunk, PageWs w, int32_t* live_out) {
  __shared__ int sm[32];
  const int lo = blockIdx.x * chunk, hi = min(pages, lo + chunk);
  const int live = cta_live(refs, 0, pages, sm);
  const int low = cta_live(refs, 0, live, sm);    // live pages already below `live`
  int r = cta_live(refs, 0, lo, sm);              // live pages before i
  for (int i0 = lo; i0 < hi; i0 += blockDim.x) {
    const int i = i0 + threadIdx.x;
    const bool f = i < hi && refs[i] > 0;
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
    *w.count = live - low;
    *w.live = live;
    *live_out = live;
  }
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
      if (fate >= 0) e = w.x[fate];
      else if (fate != kStays) flag(w.status, kDevInvalid);   // maps a page nobody counts
    } else if (e != -1) {
      flag(w.status, kDevInvalid);
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

int list_chunk(int pages) {
  const int c = (pages + kMaxListCtas - 1) / kMaxListCtas;
  return c < kChunk ? kChunk : c;
}

cudaError_t clear_status(const PageWs& w, cudaStream_t st) {
  return cudaMemsetAsync(w.status, 0, sizeof(int), st);
}

cudaError_t launch_list(const PageTable& pt, const PageWs& w, cudaStream_t st) {
  const int chunk = list_chunk(pt.pages);
  note_launches(1);
  pages_list_kernel<<<(pt.pages + chunk - 1) / chunk, 1024, 0, st>>>(pt.refs, pt.pages, chunk, w);
  return cudaGetLastError();
}

}  // namespace

size_t pages_workspace_bytes(int pages) { return kWsHead + (size_t)pages * 3 * sizeof(int32_t); }

cudaError_t launch_pages_copy(const PoolSet& ps, int pages, const int32_t* src, const int32_t* dst,
                              int n, char* ws, cudaStream_t st) {
  const PageWs w = carve(ws, pages);
  const CopyPlan c = copy_plan(ps);
  const int64_t work = (int64_t)n * c.seg0[ps.n], most = sm_count() * 4;
  cudaError_t e = clear_status(w, st);
  if (e != cudaSuccess) return e;
  note_launches(1);
  pages_copy_kernel<<<(unsigned)(work < most ? work : most), kThreads, 0, st>>>(c, pages, src, dst, n,
                                                                              w.status);
  return cudaGetLastError();
}

cudaError_t launch_pages_fork(const PoolSet& ps, const PageTable& pt, const RowList& rows, char* ws,
                              cudaStream_t st) {
  const PageWs w = carve(ws, pt.pages);
  const CopyPlan c = copy_plan(ps);
  cudaError_t e = clear_status(w, st);
  if (e != cudaSuccess) return e;
  const int cols = (pt.max_blocks + 255) / 256;
  note_launches(1);
  pages_share_kernel<<<dim3(cols < 8 ? cols : 8, rows.n), 256, 0, st>>>(pt, rows, w.status);
  bool part = false;
  for (int j = 0; j < rows.n; ++j) part |= rows.c[j] % kBlock != 0;
  if (part) {
    if ((e = launch_list(pt, w, st)) != cudaSuccess) return e;
    note_launches(1);
    const int segs = c.seg0[ps.n] > 0 ? c.seg0[ps.n] : 1;
    pages_fork_copy_kernel<<<dim3(segs < 64 ? segs : 64, rows.n), kThreads, 0, st>>>(c, pt, rows, w);
  }
  return cudaGetLastError();
}

cudaError_t launch_pages_free(const PageTable& pt, const RowList& rows, char* ws, cudaStream_t st) {
  const PageWs w = carve(ws, pt.pages);
  cudaError_t e = clear_status(w, st);
  if (e != cudaSuccess) return e;
  const int cols = (pt.max_blocks + 255) / 256;
  note_launches(1);
  pages_free_kernel<<<dim3(cols < 8 ? cols : 8, rows.n), 256, 0, st>>>(pt, rows, w.status);
  return cudaGetLastError();
}

cudaError_t launch_pages_alloc(const PageTable& pt, const RowList& rows, char* ws, cudaStream_t st) {
  const PageWs w = carve(ws, pt.pages);
  cudaError_t e = clear_status(w, st);
  if (e != cudaSuccess) return e;
  if ((e = launch_list(pt, w, st)) != cudaSuccess) return e;
  note_launches(1);
  pages_alloc_kernel<<<1, 1024, 0, st>>>(pt, rows, w);
  return cudaGetLastError();
}

cudaError_t launch_pages_compact(const PoolSet& ps, const PageTable& pt, int32_t* table_out,
                                 int32_t* refs_out, int32_t* live, char* ws, cudaStream_t st) {
  const PageWs w = carve(ws, pt.pages);
  const CopyPlan c = copy_plan(ps);
  cudaError_t e = clear_status(w, st);
  if (e != cudaSuccess) return e;
  const int chunk = list_chunk(pt.pages);
  note_launches(2);
  pages_plan_kernel<<<(pt.pages + chunk - 1) / chunk, 1024, 0, st>>>(pt.refs, pt.pages, chunk, w,
                                                                    live);
  pages_move_kernel<<<sm_count() * 4, kThreads, 0, st>>>(c, pt, table_out, refs_out, w);
  return cudaGetLastError();
}

}  // namespace msa

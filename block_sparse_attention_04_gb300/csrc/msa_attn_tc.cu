// KV-outer sparse attention on tensor cores (prefill): step 4 of "MiniMax
// 模型迭代与竞品分析" section 2 (exact softmax over the selected blocks only),
// organised around the KV blocks, the "KV-outer" order that "MiniMax：Text-01 /
// M1 → M2.7 → M3" section 5 names for MSA's sparse kernel.
//
// A query-outer tile would hold one query's heads of one group (6 rows),
// far below the 128 rows a tcgen05 MMA wants.  So the selections are inverted:
// for every (sequence b, KV block kb, group g) the (query, slot) entries that
// chose it.  One tile = one such block x up to R entries, an entry's H/G heads
// padded to rpe = 8 (or 16) rows, i.e. at most 128 query-head rows against
// the block's 128 tokens.  One persistent CTA per SM runs two tile chains
// (tile t on chain t & 1), so one chain's S = Q K^T runs while the other
// chain's softmax works:
//   warp 0        TMA of Q tiles (8-head x D boxes, one per 8-row group)
//                 through a 3-deep ring: the Q copy is the longest latency
//   warp 1        TMA of K and V blocks of KV head g (block-major cache: 128
//                 rows of D bf16 at stride G*D) through 2-deep rings, one load
//                 per list
//   warp 2        tcgen05.mma, S(t) then P.V(t-1): S into TMEM, O = P V with P
//                 read from TMEM and V an MN-major smem operand
//   warps 3-10    row softmax, one warpgroup per chain (block-local max m, sum
//                 l; causal mask on the local block), P as bf16 written over S
//   warps 11-18   O as an unnormalised bf16 partial, one warpgroup per chain
// Each (query, head, slot) partial (O, m, l) is combined by a log-sum-exp
// merge into the bf16 output.
//
// An 8-bit cache (kernels with Q8 set) has four more warps in place of warp 1:
// they read a list's codes, convert them (K to bf16, V to f16, both exact) and
// write them into the same rings.  A tile has one KV block, so its exponents
// are two numbers, which travel in the tile's descriptor: 2^ek scales the
// scores, 2^ev waits for the merge.  P is relative to the block's own maximum,
// so f16 holds it, as 2^15 p (2^-11, and 2^-40 of the maximum at the small
// end: a weight that small counts for nothing beside codes that span 2^18), and
// O = sum p code is below 128 * 448 < 2^16: the partials are f16 too.  Rows of
// V behind the call's last query are zeroed on the way.  2048 queries at the end
// of 32K tokens, 48/8 heads: 252 us with lists (27) and merge (66), against 52
// for the products at the burst rate; per tile the softmax, the partials and the
// conversion (11 %) share the SM's issue slots and tensor-memory reads.
#include <climits>

#include "msa_q8.cuh"
#include "msa_tc.h"
#include "msa_tma.h"

namespace msa {
namespace {

// warps: Q TMA, K/V TMA, MMA, 2 softmax warpgroups, 2 O-epilogue warpgroups
constexpr int kQWarp = 0, kKVWarp = 1, kMmaWarp = 2, kSoftWarp0 = 3, kEpiWarp0 = 11;
constexpr int kAttnThreads = 32 * 19;
constexpr int kConvWarp0 = 19, kConv = 128;  // converters of an 8-bit cache
template <bool Q8>
constexpr int attn_threads() { return kAttnThreads + (Q8 ? kConv : 0); }
constexpr int kPassRows = 8192;    // (sequence, query) rows per pass

struct AttnPass {
  Shape s;
  Positions pos;
  int t0, Tp;            // queries [t0, t0+Tp) of every sequence
  int nbl;               // key blocks per (sequence, group) in the list space
  int nlists;            // B * nbl * G
  int R;                 // entries per tile = 128 / rpe
  int rpe;               // tile rows per entry: H/G rounded up to 8 or 16
  const int32_t* sel;    // [B][T][G][16]
  int32_t* count;        // [nlists]
  int32_t* off;          // [nlists + 1]   entry offsets
  int32_t* tile_off;     // [nlists + 1]   tile offsets; tile_off[nlists] = total
  int32_t* entries;      // packed (i - t0) * 16 + slot
  int4* tile_desc;       // per tile: list, first entry, entries (| (ek + 128) << 8 |
                         // (ev + 128) << 16 for an 8-bit cache), kb | g << 15 | b << 18
  uint16_t* part_o;      // [B*Tp*H*16][D] bf16, O = sum 2^(s-m) v (unnormalised);
                         // 8-bit cache: f16, O = sum 2^(s-m) code
  float2* part_ml;       // [B*Tp*H*16] (m in log2 units, l)
  float4* part_mle;      // ... 8-bit cache, in its place: (m, l, ev)
  int* status;
  uint32_t wait_polls;   // poll cap of the pipeline waits (0: wall-clock bound only)
  const uint8_t* k8;     // an 8-bit cache's codes and exponents (null: bf16 cache)
  const uint8_t* v8;
  const int8_t* k_exp;
  const int8_t* v_exp;
};

// Lists are ordered group-major, list (b, kb, g) at index (g*B + b)*nbl + kb:
// the tiles of one KV group are contiguous, so CTAs dealt nearby tiles all
// work on one group at a time.

__device__ __forceinline__ bool slot_valid(const AttnPass& a, int b, int i, int kb) {
  const int64_t t = (int64_t)a.pos.q_start[b] + i;
  return kb >= 0 && kb <= (int)(t / kBlock) && kb < a.s.max_blocks;
}

// ---- inverted lists -------------------------------------------------------
// The count and fill kernels give each CTA a contiguous range of the lists of
// one KV group (list_of is contiguous in (b, kb) for a fixed g).  The CTA
// reads every selection of its group in the pass and keeps the counts (or
// fill cursors) of its own lists in shared memory, so no global atomics are
// needed: with one global atomic per (query, group, slot) the two kernels
// were bound by atomic throughput (43 and 38 us per 8192-query pass at 128K).
constexpr int kCsrThreads = 512;
constexpr int kCsrMaxLists = 16384;  // shared-memory counters per CTA

struct CsrGrid {
  int per_group;   // CTAs per group
  int span;        // lists per CTA (the last CTA of a group may hold fewer)
};

inline CsrGrid csr_grid(const Shape& s, int nbl) {
  const int64_t lists_pg = (int64_t)s.B * nbl;
  int per = (sm_count() + s.G - 1) / s.G;
  const int64_t need = (lists_pg + kCsrMaxLists - 1) / kCsrMaxLists;
  if (per < need) per = (int)need;
  if (per > lists_pg) per = (int)(lists_pg > 0 ? lists_pg : 1);
  return CsrGrid{per, (int)((lists_pg + per - 1) / per)};
}

// This CTA's group and list range [lo, hi) within the group's B * nbl lists.
__device__ __forceinline__ void csr_cta_range(const AttnPass& a, int span, int per_group, int& g,
                                              int& lo, int& hi) {
  g = (int)blockIdx.x / per_group;
  const int c = (int)blockIdx.x % per_group;
  const int lists_pg = a.s.B * a.nbl;
  lo = min(lists_pg, c * span);
  hi = min(lists_pg, lo + span);
}

// One (sequence, query) row of group g per thread and step: its 16 slots are
// one 64-byte read, validated against the query's local block.
__global__ void __launch_bounds__(kCsrThreads) csr_count_kernel(AttnPass a, int span,
                                                                int per_group) {
  extern __shared__ int32_t s_cnt[];
  int g, lo, hi;
  csr_cta_range(a, span, per_group, g, lo, hi);
  const int nl = hi - lo;
  for (int k = threadIdx.x; k < nl; k += blockDim.x) s_cnt[k] = 0;
  __syncthreads();
  const int rows = a.s.B * a.Tp;
  const bool first = blockIdx.x % per_group == 0;  // one CTA per group flags bad ids
  for (int r = threadIdx.x; r < rows; r += blockDim.x) {
    const int b = r / a.Tp, i = a.t0 + r % a.Tp;
    const int4* sr = reinterpret_cast<const int4*>(
        a.sel + (((size_t)b * a.s.T + i) * a.s.G + g) * kTopk);
    const int64_t t = (int64_t)a.pos.q_start[b] + i;
    const int64_t lb = t / kBlock;
    const int lim = (int)(lb < a.s.max_blocks - 1 ? lb : a.s.max_blocks - 1);
    const int base = b * a.nbl - lo;
#pragma unroll
    for (int v = 0; v < kTopk / 4; ++v) {
      const int4 q4 = sr[v];
      const int ks[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int kb = ks[u];
        if (kb < 0) continue;
        if (kb > lim) {
          if (first) flag_invalid(a.status);
          continue;
        }
        const int l = base + kb;
        if ((unsigned)l < (unsigned)nl) atomicAdd(&s_cnt[l], 1);
      }
    }
  }
  __syncthreads();
  int32_t* cnt = a.count + (size_t)g * a.s.B * a.nbl + lo;
  for (int k = threadIdx.x; k < nl; k += blockDim.x) cnt[k] = s_cnt[k];
}

// Exclusive scans of entry counts and of tile counts, one CTA of 1024 threads.
// Each thread owns a contiguous run of lists, read and written with 16-byte
// accesses where the run is aligned.
__global__ void __launch_bounds__(1024) csr_scan_kernel(AttnPass a) {
  __shared__ int64_t s_e[1024], s_t[1024];
  const int n = a.nlists;
  const int per = ((n + 1023) / 1024 + 3) & ~3;  // a multiple of 4
  const int lo = min(n, (int)threadIdx.x * per), hi = min(n, lo + per);
  int64_t se = 0, st = 0;
  int k = lo;
  for (; k + 4 <= hi; k += 4) {
    const int4 c = *reinterpret_cast<const int4*>(a.count + k);
    se += (int64_t)c.x + c.y + c.z + c.w;
    st += (c.x + a.R - 1) / a.R + (c.y + a.R - 1) / a.R + (c.z + a.R - 1) / a.R +
          (c.w + a.R - 1) / a.R;
  }
  for (; k < hi; ++k) {
    const int c = a.count[k];
    se += c;
    st += (c + a.R - 1) / a.R;
  }
  s_e[threadIdx.x] = se;
  s_t[threadIdx.x] = st;
  __syncthreads();
  for (int d = 1; d < 1024; d <<= 1) {
    int64_t ve = 0, vt = 0;
    if ((int)threadIdx.x >= d) {
      ve = s_e[threadIdx.x - d];
      vt = s_t[threadIdx.x - d];
    }
    __syncthreads();
    s_e[threadIdx.x] += ve;
    s_t[threadIdx.x] += vt;
    __syncthreads();
  }
  int64_t oe = s_e[threadIdx.x] - se, ot = s_t[threadIdx.x] - st;
  k = lo;
  for (; k + 4 <= hi; k += 4) {
    const int4 c = *reinterpret_cast<const int4*>(a.count + k);
    int4 o, t;
    o.x = (int)oe; t.x = (int)ot; oe += c.x; ot += (c.x + a.R - 1) / a.R;
    o.y = (int)oe; t.y = (int)ot; oe += c.y; ot += (c.y + a.R - 1) / a.R;
    o.z = (int)oe; t.z = (int)ot; oe += c.z; ot += (c.z + a.R - 1) / a.R;
    o.w = (int)oe; t.w = (int)ot; oe += c.w; ot += (c.w + a.R - 1) / a.R;
    *reinterpret_cast<int4*>(a.off + k) = o;
    *reinterpret_cast<int4*>(a.tile_off + k) = t;
  }
  for (; k < hi; ++k) {
    const int c = a.count[k];
    a.off[k] = (int32_t)oe;
    a.tile_off[k] = (int32_t)ot;
    oe += c;
    ot += (c + a.R - 1) / a.R;
  }
  if (threadIdx.x == 1023) {
    a.off[n] = (int32_t)s_e[1023];
    a.tile_off[n] = (int32_t)s_t[1023];
  }
}

__global__ void __launch_bounds__(kCsrThreads) csr_fill_kernel(AttnPass a, int span,
                                                               int per_group) {
  extern __shared__ int32_t s_cur[];
  int g, lo, hi;
  csr_cta_range(a, span, per_group, g, lo, hi);
  const int nl = hi - lo;
  for (int k = threadIdx.x; k < nl; k += blockDim.x) s_cur[k] = 0;
  __syncthreads();
  const size_t l0 = (size_t)g * a.s.B * a.nbl + lo;  // global index of this CTA's first list
  const int rows = a.s.B * a.Tp;
  for (int r = threadIdx.x; r < rows; r += blockDim.x) {
    const int b = r / a.Tp, il = r % a.Tp;
    const int4* sr = reinterpret_cast<const int4*>(
        a.sel + (((size_t)b * a.s.T + a.t0 + il) * a.s.G + g) * kTopk);
    const int64_t t = (int64_t)a.pos.q_start[b] + a.t0 + il;
    const int64_t lb = t / kBlock;
    const int lim = (int)(lb < a.s.max_blocks - 1 ? lb : a.s.max_blocks - 1);
    const int base = b * a.nbl - lo;
#pragma unroll
    for (int v = 0; v < kTopk / 4; ++v) {
      const int4 q4 = sr[v];
      const int ks[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int kb = ks[u];
        const int l = base + kb;
        if (kb < 0 || kb > lim || (unsigned)l >= (unsigned)nl) continue;
        const int p = atomicAdd(&s_cur[l], 1);
        a.entries[a.off[l0 + l] + p] = il * kTopk + v * 4 + u;
      }
    }
  }
  // tile table, thread per list: one 16-byte descriptor per tile, so the
  // attention kernel reads a tile's coordinates with a single load
  for (int k = threadIdx.x; k < nl; k += blockDim.x) {
    const size_t L = l0 + k;
    const int t0 = a.tile_off[L], t1 = a.tile_off[L + 1];
    if (t0 == t1) continue;
    const int kb = (lo + k) % a.nbl, b = (lo + k) / a.nbl;
    const int cnt = a.count[L], o = a.off[L];
    int exps = 0;
    if (a.k_exp) {
      // a table entry outside the pool is flagged where its block is read
      const int64_t pb = cache_block(a.s, b, kb, nullptr);
      const int ek = pb < 0 ? 0 : clamp_exp(a.k_exp[pb * a.s.G + g]);
      const int ev = pb < 0 ? 0 : clamp_exp(a.v_exp[pb * a.s.G + g]);
      exps = (ek + 128) << 8 | (ev + 128) << 16;
    }
    for (int t = t0; t < t1; ++t) {
      const int e0 = (t - t0) * a.R;
      a.tile_desc[t] =
          make_int4((int)L, o + e0, min(a.R, cnt - e0) | exps, kb | (g << 15) | (b << 18));
    }
  }
}

// ---- the attention tile kernel ---------------------------------------------
constexpr int kTileChunk = 4;   // consecutive tiles dealt to a CTA at a time

// Local tile i of this CTA -> its descriptor (see the chunked deal in
// attn_tc_kernel).
struct CtaTiles {
  const int4* all;
  __device__ __forceinline__ int4 operator[](int i) const {
    return all[((i / kTileChunk) * (int)gridDim.x + (int)blockIdx.x) * kTileChunk + i % kTileChunk];
  }
};
constexpr int kQStages = 3;   // Q tiles in flight (the Q copy is the longest latency)
constexpr int kKVStages = 2;  // K and V blocks in flight

template <int D>
struct AttnCfg {
  static constexpr int kHalf = 128 * 128;              // one [128 rows][64] bf16 SW128 box
  static constexpr int kNHalf = D / 64;                // 64-dim halves of a row
  static constexpr int kQGroup = kNHalf * 1024;        // one 8-row group of the Q tile
  static constexpr int kSmemQ = 16 * kQGroup;          // Q tile (128 rows)
  static constexpr int kSmemK = kNHalf * kHalf;        // one K (or V) block of one KV head
  static constexpr int kSmem = kQStages * kSmemQ + 2 * kKVStages * kSmemK + 256 + 1024;
  // two chains: S/P at [0,128) and [128,256), O at [256,384) and [384,512)
  static constexpr uint32_t kTmemCols = 512;
};

template <int D, bool Q8>
__global__ void __launch_bounds__(attn_threads<Q8>(), 1)
    attn_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v, const AttnPass a) {
  using C = AttnCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* sQ = smem;                                  // [kQStages] Q tiles
  uint8_t* sK = sQ + kQStages * C::kSmemQ;             // [kKVStages] K blocks
  uint8_t* sV = sK + kKVStages * C::kSmemK;            // [kKVStages] V blocks
  uint64_t* bars = reinterpret_cast<uint64_t*>(sV + kKVStages * C::kSmemK);
  uint64_t* q_full = bars;                        // kQStages
  uint64_t* q_empty = q_full + kQStages;          // kQStages
  uint64_t* k_full = q_empty + kQStages;          // kKVStages
  uint64_t* k_empty = k_full + kKVStages;
  uint64_t* v_full = k_empty + kKVStages;
  uint64_t* v_empty = v_full + kKVStages;
  uint64_t* s_full = v_empty + kKVStages;         // per chain: S of its tile is in TMEM
  uint64_t* p_full = s_full + 2;                  // per chain: P written over S
  uint64_t* o_full = p_full + 2;                  // per chain: O of its tile is in TMEM
  uint64_t* o_empty = o_full + 2;                 // per chain: O read out
  uint64_t* bar_fin = o_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar_fin + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kQStages; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
    }
    for (int i = 0; i < kKVStages; ++i) {
      mbar_init(&k_full[i], Q8 ? kConv : 1);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], Q8 ? kConv : 1);
      mbar_init(&v_empty[i], 1);
    }
    for (int c = 0; c < 2; ++c) {
      mbar_init(&s_full[c], 1);
      mbar_init(&p_full[c], 128);
      mbar_init(&o_full[c], 1);
      mbar_init(&o_empty[c], 128);
    }
    mbar_init(bar_fin, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_q);
    if constexpr (!Q8) {
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
  }
  if (warp == kMmaWarp) tmem_alloc(tmem_slot, C::kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const int H = a.s.H, hpg = H / a.s.G;
  const int rshift = a.rpe == 8 ? 3 : 4;  // tile row -> entry
  // This CTA's tiles: chunks of kTileChunk consecutive tiles (mostly of one
  // list, so the K/V block in shared memory is reused within a chunk), dealt
  // round-robin.  With group-major lists, all CTAs then work within a narrow
  // stretch of the tile order, i.e. on one KV group at a time, whose Q rows
  // and K/V blocks stay in L2; contiguous ranges per CTA had every CTA on a
  // different group, and each query's Q rows were fetched from DRAM for
  // most of its 16 blocks.
  const int ntiles = a.tile_off[a.nlists];
  const int nchunks = (ntiles + kTileChunk - 1) / kTileChunk;
  const int my_chunks =
      (int)blockIdx.x < nchunks ? (nchunks - 1 - (int)blockIdx.x) / (int)gridDim.x + 1 : 0;
  int n = my_chunks * kTileChunk;                          // tiles of this CTA
  if (my_chunks > 0 && (nchunks - 1) % (int)gridDim.x == (int)blockIdx.x)
    n -= nchunks * kTileChunk - ntiles;                    // it holds the partial last chunk
  const CtaTiles desc{a.tile_desc};

  if (warp == kQWarp) {
    // ---------------------------------------------------- Q TMA (warp 0)
    // Q tiles through a kQStages ring: the Q of tile t is loaded once S of
    // tile t - kQStages is done, i.e. well before S of t is due.  Entry e
    // fills tile rows [e*rpe, e*rpe + rpe) (its hpg heads, then heads of the
    // next group or token, or zero fill past the end: rows the softmax and
    // epilogue skip), one box of 8 rows x D dims per lane.  L2 policy: Q rows
    // are read again for each block their query selected (evict last).
    const uint64_t pol_q = l2_policy_evict_last();
    const int bpe = a.rpe >> 3;                   // boxes per entry
    const int box_e = lane / bpe;                 // this lane's entry
    const int box_r = (lane % bpe) * 8;           // its first row within the entry
    int q_last[kQStages];                         // last tile loaded into each slot
#pragma unroll
    for (int i = 0; i < kQStages; ++i) q_last[i] = -1;
    for (int t = 0; t < n; ++t) {
      if (__any_sync(0xffffffffu, *abort_flag != 0)) break;  // warp-uniform
      const int4 d = desc[t];
      const int ne = d.z & 0xFF;
      int qrow = 0;
      if (box_e < ne) {
        const int il = a.entries[d.y + box_e] >> 4;
        qrow = (int)(((int64_t)(d.w >> 18) * a.s.T + a.t0 + il) * H + ((d.w >> 15) & 7) * hpg +
                     box_r);
      }
      const int qs = t % kQStages;
      const uint32_t u = (uint32_t)(t / kQStages);
      if (!__all_sync(0xffffffffu, mbar_wait(&q_empty[qs], (u & 1) ^ 1, a.status, a.wait_polls))) {
        *abort_flag = 1;
        break;
      }
      if (lane == 0) mbar_arrive_expect_tx(&q_full[qs], (uint32_t)(ne * a.rpe * D * 2));
      __syncwarp();
      if (box_e < ne)
        tma_load_3d_hint(smem_u32(sQ + qs * C::kSmemQ + ((box_e * a.rpe + box_r) >> 3) * C::kQGroup),
                         &tm_q, &q_full[qs], 0, qrow, 0, pol_q);
      q_last[qs] = t;
    }
    // no copy may still be landing in shared memory when the CTA exits (after
    // a timeout elsewhere the tiles were not all consumed): wait, bounded, for
    // the last load of each slot
    if (lane == 0) {
#pragma unroll
      for (int i = 0; i < kQStages; ++i)
        if (q_last[i] >= 0) mbar_wait(&q_full[i], (uint32_t)(q_last[i] / kQStages) & 1, nullptr);
    }
  } else if (warp == kKVWarp) {
    // -------------------------------------------------- K/V TMA (warp 1)
    // One K and one V block per list change, through a kKVStages ring; a
    // buffer is refilled once the last tile of its previous list is through
    // S (K) or P.V (V).  L2 policy: evict first (used once, from smem).
    if (!Q8 && lane == 0) {
      const uint64_t pol_kv = l2_policy_evict_first();
      int kv = -1, prev = -1;
      int k_last[kKVStages], v_last[kKVStages];   // last list loaded into each slot
#pragma unroll
      for (int i = 0; i < kKVStages; ++i) k_last[i] = v_last[i] = -1;
      for (int t = 0; t < n && !*abort_flag; ++t) {
        const int4 d = desc[t];
        if (d.x == prev) continue;
        prev = d.x;
        ++kv;
        const int ks = kv % kKVStages;
        const uint32_t w = (uint32_t)(kv / kKVStages);
        const int kb = d.w & 0x7FFF, g = (d.w >> 15) & 7, b = d.w >> 18;
        // through the block table when the caches are paged; an entry outside
        // the pool (flagged) reads zeros from past the pool's end
        const int64_t pb = cache_block(a.s, b, kb, a.status);
        const int row = (int)((pb < 0 ? a.s.cache_blocks() : pb) * kBlock);
        if (!mbar_wait(&k_empty[ks], (w & 1) ^ 1, a.status, a.wait_polls)) { *abort_flag = 1; break; }
        mbar_arrive_expect_tx(&k_full[ks], C::kSmemK);
#pragma unroll
        for (int h = 0; h < C::kNHalf; ++h)
          tma_load_3d_hint(smem_u32(sK + ks * C::kSmemK + h * C::kHalf), &tm_k, &k_full[ks], h * 64, g,
                           row, pol_kv);
        k_last[ks] = kv;
        if (!mbar_wait(&v_empty[ks], (w & 1) ^ 1, a.status, a.wait_polls)) { *abort_flag = 1; break; }
        mbar_arrive_expect_tx(&v_full[ks], C::kSmemK);
#pragma unroll
        for (int h = 0; h < C::kNHalf; ++h)
          tma_load_3d_hint(smem_u32(sV + ks * C::kSmemK + h * C::kHalf), &tm_v, &v_full[ks], h * 64, g,
                           row, pol_kv);
        v_last[ks] = kv;
      }
      // as for Q: no copy may still be landing when the CTA exits
#pragma unroll
      for (int i = 0; i < kKVStages; ++i) {
        if (k_last[i] >= 0) mbar_wait(&k_full[i], (uint32_t)(k_last[i] / kKVStages) & 1, nullptr);
        if (v_last[i] >= 0) mbar_wait(&v_full[i], (uint32_t)(v_last[i] / kKVStages) & 1, nullptr);
      }
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------ MMA (warp 2)
    // Order S(0), S(1), P.V(0), S(2), P.V(1), ...: the S of one chain runs
    // while the other chain's softmax works.  Tile t uses chain c = t & 1:
    // S and P in TMEM columns [128c, 128c + 128), O in [256 + 128c, ...).
    // tcgen05.mma executes in issue order, so S(t + 2) cannot overwrite the P
    // that P.V(t), issued before it, still reads.
    // The whole warp runs the loop; one elected lane issues the MMAs and
    // commits, from descriptors formed once per ring and stepped by byte
    // offset / 16 (measured: half the issue time of a loop run by lane 0).
    {
      constexpr uint32_t idesc_s = idesc_bf16(128, 128, false, false);
      constexpr uint32_t idesc_o =
          Q8 ? idesc_f16(128, D, false, true) : idesc_bf16(128, D, false, true);
      const uint64_t qdesc0 = smem_desc(smem_u32(sQ), 16, C::kQGroup, kSwizzle128B);
      const uint64_t kdesc0 = smem_desc(smem_u32(sK), 16, 1024, kSwizzle128B);
      const uint64_t vdesc0 = smem_desc(smem_u32(sV), C::kHalf, 1024, kSwizzle128B);
      int kv = -1, prev = -1;
      int pv_ks = 0;
      uint32_t pv_w = 0;
      bool pv_last = false, pv_first = false;
      bool ok = true;
      // the lists of tiles t and t + 1, loaded two tiles ahead (a load takes
      // about as long as issuing a tile's MMAs)
      int l0 = n > 0 ? desc[0].x : -1, l1 = n > 1 ? desc[1].x : -1;
      for (int t = 0; t <= n && ok; ++t) {
        int ks = 0;
        uint32_t w = 0;
        bool last = false, first = false;
        const int lt = l0, ln = l1;
        l0 = l1;
        l1 = t + 2 < n ? desc[t + 2].x : -1;
        if (t < n) {
          // ---- S(t)
          first = lt != prev;  // K and V are waited for once per list
          if (first) { prev = lt; ++kv; }
          ks = kv % kKVStages;
          w = (uint32_t)(kv / kKVStages);
          last = (t + 1 == n) || ln != lt;
          const int c = t & 1, qs = t % kQStages;
          const bool okl =
              mbar_wait(&q_full[qs], (uint32_t)(t / kQStages) & 1, a.status, a.wait_polls) &&
              (!first || mbar_wait(&k_full[ks], w & 1, a.status, a.wait_polls));
          ok = __all_sync(0xffffffffu, okl);
          if (!ok) break;
          tc_fence_after();
          const uint64_t qd = qdesc0 + (uint64_t)((qs * C::kSmemQ) >> 4);
          const uint64_t kd = kdesc0 + (uint64_t)((ks * C::kSmemK) >> 4);
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k)  // 16 dims: (k & 3) * 32 bytes within a 64-dim half
              tc_mma_f16(tmem + c * 128, qd + (uint64_t)(((k >> 2) * 1024 + (k & 3) * 32) >> 4),
                         kd + (uint64_t)(((k >> 2) * C::kHalf + (k & 3) * 32) >> 4), idesc_s,
                         k > 0);
            tc_commit(&q_empty[qs]);
            tc_commit(&s_full[c]);
            if (last) tc_commit(&k_empty[ks]);
          }
          __syncwarp();
        }
        if (t >= 1) {
          // ---- P.V(t - 1)
          const int tp = t - 1, c = tp & 1;
          const uint32_t j = (uint32_t)(tp >> 1);
          const bool okl =
              mbar_wait(&p_full[c], j & 1, a.status, a.wait_polls) &&
              (!pv_first || mbar_wait(&v_full[pv_ks], pv_w & 1, a.status, a.wait_polls)) &&
              (j == 0 || mbar_wait(&o_empty[c], (j - 1) & 1, a.status, a.wait_polls));
          ok = __all_sync(0xffffffffu, okl);
          if (!ok) break;
          tc_fence_after();
          const uint64_t vd = vdesc0 + (uint64_t)((pv_ks * C::kSmemK) >> 4);
          // P (bf16, two per column) is in TMEM columns [128c, 128c + 64)
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              tc_mma_f16_ts(tmem + 256 + c * 128, tmem + c * 128 + k * 8,
                            vd + (uint64_t)((k * 2048) >> 4), idesc_o, k > 0);
            tc_commit(&o_full[c]);
            if (pv_last) tc_commit(&v_empty[pv_ks]);
          }
          __syncwarp();
        }
        pv_ks = ks;
        pv_w = w;
        pv_last = last;
        pv_first = first;
      }
      if (!ok && lane == 0) *abort_flag = 1;
      // all MMAs done before TMEM is released
      if (elect_one()) tc_commit(bar_fin);
      __syncwarp();
      mbar_wait(bar_fin, 0, nullptr);
    }
  } else if (warp < kEpiWarp0) {
    // ------------------------------------------ softmax (2 warpgroups, one per chain)
    const int c = (warp - kSoftWarp0) >> 2;
    const int quad = warp & 3;
    const int r = quad * 32 + lane;  // tile row = TMEM lane
    const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16) + c * 128;
    float sl = a.s.scale * kLog2e;
    const int e = r >> rshift, hh = r & (a.rpe - 1);
    // the next tile's descriptor and this row's entry of it are loaded a tile
    // ahead: the two loads depend on each other and would stand before every S
    int4 nd = c < n ? desc[c] : make_int4(0, 0, 0, 0);
    int nen = c < n && e < (nd.z & 0xFF) ? a.entries[nd.y + e] : 0;
    for (int t = c; t < n; t += 2) {
      if (__any_sync(0xffffffffu, *abort_flag != 0)) break;  // warp-uniform
      const int4 d = nd;
      const int en = nen;
      if (t + 2 < n) nd = desc[t + 2];
      const int kb = d.w & 0x7FFF, g = (d.w >> 15) & 7, b = d.w >> 18;
      const bool valid = e < (d.z & 0xFF) && hh < hpg;
      if constexpr (Q8) {
        sl = a.s.scale * kLog2e * pow2i((d.z >> 8 & 0xFF) - 128);
        sl = fminf(fmaxf(sl, -3e38f), 3e38f);
      }
      const int il = valid ? en >> 4 : 0, slot = valid ? en & 15 : 0;
      const int64_t tq = (int64_t)a.pos.q_start[b] + a.t0 + il;
      // tokens kb*128 + col with col > lim are masked (only in the local block)
      const int lim = (int)(tq - (int64_t)kb * kBlock);
      const bool masked = __any_sync(0xffffffffu, valid && lim < kBlock - 1);
      if (!__all_sync(0xffffffffu, mbar_wait(&s_full[c], (uint32_t)(t >> 1) & 1, a.status, a.wait_polls))) {
        *abort_flag = 1;
        break;
      }
      tc_fence_after();
      if (t + 2 < n && e < (nd.z & 0xFF)) nen = a.entries[nd.y + e];
      // TMEM is read in 16-column loads: small loads leave the MMAs of the other
      // chain more of tensor memory than larger ones (measured).  Pass 1 waits for
      // two of them at a time (128K prefill attention 16.40 ms with one, 15.44
      // with two, 15.63 with four), pass 2 for each (15.49 with two).
      // pass 1: row maximum of the scaled scores: the maximum of the raw
      // scores, or their minimum when the scale is negative
      const bool neg = sl < 0.f;
      float mx = neg ? INFINITY : -INFINITY;
      if (masked) {
#pragma unroll 1
        for (int cc = 0; cc < 8; ++cc) {
          uint32_t h[16];
          tmem_ld16(lane_base + cc * 16, h);
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float x = __uint_as_float(h[k]);
            const bool in = cc * 16 + k <= lim;
            mx = neg ? fminf(mx, in ? x : INFINITY) : fmaxf(mx, in ? x : -INFINITY);
          }
        }
      } else if (neg) {
#pragma unroll 1
        for (int cc = 0; cc < 8; cc += 2) {
          const float r0 = tmem_ld16_red<false>(lane_base + (cc + 0) * 16);
          const float r1 = tmem_ld16_red<false>(lane_base + (cc + 1) * 16);
          tmem_ld_wait();
          mx = fminf(mx, fminf(r0, r1));
        }
      } else {   // the loads reduce 16 scores each
#pragma unroll 1
        for (int cc = 0; cc < 8; cc += 2) {
          const float r0 = tmem_ld16_red<true>(lane_base + (cc + 0) * 16);
          const float r1 = tmem_ld16_red<true>(lane_base + (cc + 1) * 16);
          tmem_ld_wait();
          mx = fmaxf(mx, fmaxf(r0, r1));
        }
      }
      const float m = mx * sl;
      // pass 2: P = 2^(s*scale*log2e - m) as bf16, two per column, written
      // over S in TMEM: the 32 scores of columns [32cc, 32cc+32) are read (two
      // loads) before columns [16cc, 16cc+16) are written, and those belong to
      // chunks already read; row sum
      const float nm = Q8 ? kPUp - m : -m;
      float2 l2 = make_float2(0.f, 0.f);
#pragma unroll 1
      for (int cc = 0; cc < 4; ++cc) {
        uint32_t wv[16];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t h[16];
          tmem_ld16(lane_base + cc * 32 + hf * 16, h);
          tmem_ld_wait();
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const int k = 2 * u;
            const int uu = hf * 8 + u;
            const float2 x =
                ffma2(make_float2(__uint_as_float(h[k]), __uint_as_float(h[k + 1])),
                      make_float2(sl, sl), make_float2(nm, nm));
            // bf16 cache: 6 of 16 pairs on the FMA pipe, the rest on the MUFU unit
            constexpr unsigned kPolyPairs = Q8 ? 0u : 0x4925u;  // uu = 0, 2, 5, 8, 11, 14
            const bool poly = (kPolyPairs >> uu) & 1u;
            float2 pp = make_float2(poly ? exp2_poly(x.x) : ex2(x.x), poly ? exp2_poly(x.y) : ex2(x.y));
            if (masked) {
              pp.x = cc * 32 + hf * 16 + k <= lim ? pp.x : 0.f;
              pp.y = cc * 32 + hf * 16 + k + 1 <= lim ? pp.y : 0.f;
            }
            l2 = fadd2(l2, pp);
            wv[uu] = Q8 ? pack_f16(pp.x, pp.y) : pack_bf16(pp.x, pp.y);
          }
        }
        tmem_st16(lane_base + cc * 16, wv);
      }
      tmem_st_wait();
      tc_fence_before();
      mbar_arrive(&p_full[c]);
      if (valid) {
        const size_t prow = (((size_t)b * a.Tp + il) * H + (size_t)g * hpg + hh) * kTopk + slot;
        if constexpr (Q8)
          __stcs(a.part_mle + prow,
                 make_float4(m, (l2.x + l2.y) * kPDown, (float)((d.z >> 16 & 0xFF) - 128), 0.f));
        else
          __stcs(a.part_ml + prow, make_float2(m, l2.x + l2.y));
      }
    }
  } else if (!Q8 || warp < kConvWarp0) {
    // ------------------------------------ O epilogue (2 warpgroups, one per chain)
    // O = P.V (unnormalised) as a bf16 partial; the merge divides by the
    // combined sum.
    const int c = (warp - kEpiWarp0) >> 2;
    const int quad = warp & 3;
    const int r = quad * 32 + lane;
    const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16) + 256 + c * 128;
    const int e = r >> rshift, hh = r & (a.rpe - 1);
    int4 nd = c < n ? desc[c] : make_int4(0, 0, 0, 0);     // a tile ahead, as above
    int nen = c < n && e < (nd.z & 0xFF) ? a.entries[nd.y + e] : 0;
    for (int t = c; t < n; t += 2) {
      if (__any_sync(0xffffffffu, *abort_flag != 0)) break;  // warp-uniform
      const int4 d = nd;
      const int en = nen;
      if (t + 2 < n) nd = desc[t + 2];
      const int g = (d.w >> 15) & 7, b = d.w >> 18;
      const bool valid = e < (d.z & 0xFF) && hh < hpg;
      const size_t prow =
          valid ? (((size_t)b * a.Tp + (en >> 4)) * H + (size_t)g * hpg + hh) * kTopk + (en & 15) : 0;
      if (!__all_sync(0xffffffffu, mbar_wait(&o_full[c], (uint32_t)(t >> 1) & 1, a.status, a.wait_polls))) {
        *abort_flag = 1;
        break;
      }
      tc_fence_after();
      if (t + 2 < n && e < (nd.z & 0xFF)) nen = a.entries[nd.y + e];
      // 32 bytes of two rows per lane become 64 bytes of a row over two lanes, so
      // that a store touches 16 lines and eight stores do for a lane: with one row
      // per lane and 16-byte stores a tile took 2048 line accesses, which paced it
      // (128K prefill attention 17.46 ms, now 14.89; 2048 queries of 32K on an
      // 8-bit cache 300 and 252 us with the softmax's changes; 64-byte rows over
      // four lanes with 16-byte stores 15.29 ms, over two 15.01; 32-byte stores
      // of a lane's own row 14.84, but 4096 queries at 64/8 heads 815 us for 787)
      const int own = valid ? (int)prow : -1;
      const bool up = lane & 1;
      int at[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) at[j] = __shfl_sync(0xffffffffu, own, (lane & ~1) + j);
#pragma unroll 1
      for (int cc = 0; cc < D / 32; ++cc) {
        uint32_t w[2][8];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t h[16];
          tmem_ld16(lane_base + cc * 32 + hf * 16, h);
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float x = __uint_as_float(h[2 * k]), y = __uint_as_float(h[2 * k + 1]);
            w[hf][k] = Q8 ? pack_f16(x * kPDown, y * kPDown) : pack_bf16(x, y);
          }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? w[0][k] : w[1][k], 1);
          w[0][k] = up ? got : w[0][k];
          w[1][k] = up ? w[1][k] : got;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
          if (at[j] >= 0) stg256(a.part_o + (size_t)at[j] * D + cc * 32 + up * 16, w[j]);
      }
      tc_fence_before();
      mbar_arrive(&o_empty[c]);
    }
  } else if constexpr (Q8) {
    // -------------------------------- converters (four warps, 8-bit cache)
    // One K and one V block per list change, as the K/V warp of a bf16 cache.
    // Each warp looks at 32 descriptors at a time for the lists that begin.
    const int tid = threadIdx.x - kConvWarp0 * 32;
    constexpr int NL = D / 16;               // 16-byte chunks of codes per thread and block
    // chunk u of this thread: row tid / 4 + 32 (u % 4), chunk 4 (u / 4) + tid % 4
    const int row0 = tid >> 2, c4 = tid & 3;
    const int64_t pitch = (int64_t)a.s.G * D;
    uint4 reg[NL];
    auto load = [&](const uint8_t* base, int64_t off) {
#pragma unroll
      for (int u = 0; u < NL; ++u)
        reg[u] = off < 0 ? make_uint4(0, 0, 0, 0)
                         : __ldg(reinterpret_cast<const uint4*>(
                               base + off + (row0 + 32 * (u & 3)) * pitch + (4 * (u >> 2) + c4) * 16));
    };
    auto store = [&](const bool is_v, uint32_t tile, int last) {   // rows behind `last` as zeros
#pragma unroll
      for (int u = 0; u < NL; ++u) {
        const int row = row0 + 32 * (u & 3), ch = 4 * (u >> 2) + c4;
        const uint32_t w[4] = {reg[u].x, reg[u].y, reg[u].z, reg[u].w};
        uint32_t h[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (is_v) e4m3x4_to_f16(row > last ? 0u : w[j], h[2 * j], h[2 * j + 1]);
          else e4m3x4_to_bf16(w[j], h[2 * j], h[2 * j + 1]);
        }
        sts128(tile + tile_off(row, 2 * ch), make_uint4(h[0], h[1], h[2], h[3]));
        sts128(tile + tile_off(row, 2 * ch + 1), make_uint4(h[4], h[5], h[6], h[7]));
      }
    };
    int kv = -1, prev = -1;
    bool ok = true;
    for (int t0 = 0; t0 < n && ok; t0 += 32) {
      const bool in = t0 + lane < n;
      const int4 d = in ? desc[t0 + lane] : make_int4(-1, 0, 0, 0);
      int before = __shfl_up_sync(0xffffffffu, d.x, 1);
      if (lane == 0) before = prev;
      prev = __shfl_sync(0xffffffffu, d.x, min(31, n - 1 - t0));
      for (uint32_t m = __ballot_sync(0xffffffffu, in && d.x != before); m != 0; m &= m - 1) {
        if (__any_sync(0xffffffffu, *abort_flag != 0)) { ok = false; break; }
        const int w = __shfl_sync(0xffffffffu, d.w, __ffs(m) - 1);
        const int kb = w & 0x7FFF, g = (w >> 15) & 7, b = w >> 18;
        const int64_t pb = cache_block(a.s, b, kb, a.status);
        const int64_t off = pb < 0 ? -1 : (pb * kBlock * a.s.G + g) * D;
        ++kv;
        const int ks = kv % kKVStages;
        const uint32_t par = ((uint32_t)(kv / kKVStages) & 1) ^ 1;
        load(a.k8, off);
        ok = __all_sync(0xffffffffu, mbar_wait(&k_empty[ks], par, a.status, a.wait_polls));
        if (!ok) break;
        store(false, smem_u32(sK + ks * C::kSmemK), kBlock);
        fence_async();
        mbar_arrive(&k_full[ks]);
        load(a.v8, off);
        ok = __all_sync(0xffffffffu, mbar_wait(&v_empty[ks], par, a.status, a.wait_polls));
        if (!ok) break;
        const int64_t last = (int64_t)a.pos.q_start[b] + a.s.T - 1 - (int64_t)kb * kBlock;
        store(true, smem_u32(sV + ks * C::kSmemK), last < kBlock ? (int)last : kBlock);
        fence_async();
        mbar_arrive(&v_full[ks]);
      }
    }
    if (!ok) *abort_flag = 1;
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// ---- merge: one warp per (sequence, query, head) ----------------------------
template <int D, bool Q8>
__global__ void __launch_bounds__(256) attn_tc_merge_kernel(AttnPass a, uint16_t* __restrict__ out) {
  constexpr int PER = D / 32;
  const int64_t gw = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int H = a.s.H, hpg = H / a.s.G;
  if (gw >= (int64_t)a.s.B * a.Tp * H) return;
  const int h = (int)(gw % H);
  const int64_t r = gw / H;
  const int b = (int)(r / a.Tp), il = (int)(r % a.Tp);
  const int i = a.t0 + il, g = h / hpg;
  const size_t prow0 = (((size_t)b * a.Tp + il) * H + h) * kTopk;
  float m = -INFINITY, l = 0.f, ev = 0.f;
  if (lane < kTopk) {
    const int kb = a.sel[(((size_t)b * a.s.T + i) * a.s.G + g) * kTopk + lane];
    if (slot_valid(a, b, i, kb)) {
      if constexpr (Q8) {
        const float4 mle = __ldcs(a.part_mle + prow0 + lane);
        m = mle.x;
        l = mle.y;
        ev = mle.z;
      } else {
        const float2 ml = __ldcs(a.part_ml + prow0 + lane);
        m = ml.x;
        l = ml.y;
      }
    }
  }
  float M = m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  // partial j holds O_j = sum p v with p = 2^(s - m_j): weight 2^(m_j - M),
  // normaliser sum_j 2^(m_j - M) l_j
  float w = (m == -INFINITY) ? 0.f : ex2(m - M);
  float W = w * l;
  float back = 1.f;
  if constexpr (Q8) {
    // O's terms also carry 2^ev: their weights relative to their own maximum
    const float mo = m + ev;
    float MO = mo;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) MO = fmaxf(MO, __shfl_xor_sync(0xffffffffu, MO, o));
    w = (m == -INFINITY) ? 0.f : ex2(mo - MO);
    back = ex2(MO - M);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) W += __shfl_xor_sync(0xffffffffu, W, o);
  float acc[PER];
#pragma unroll
  for (int e = 0; e < PER; ++e) acc[e] = 0.f;
  for (int j = 0; j < kTopk; ++j) {
    const float wj = __shfl_sync(0xffffffffu, w, j);
    if (wj == 0.f) continue;
    const uint16_t* src = a.part_o + (prow0 + j) * D + lane * PER;
    if constexpr (Q8) {
      uint32_t u[PER / 2];
      if constexpr (PER == 4) {
        const uint2 v = __ldcs(reinterpret_cast<const uint2*>(src));
        u[0] = v.x;
        u[PER / 2 - 1] = v.y;
      } else {
        u[0] = __ldcs(reinterpret_cast<const unsigned int*>(src));
      }
#pragma unroll
      for (int e = 0; e < PER / 2; ++e) {
        const float2 v = unpack_f16(u[e]);
        acc[2 * e] = fmaf(wj, v.x, acc[2 * e]);
        acc[2 * e + 1] = fmaf(wj, v.y, acc[2 * e + 1]);
      }
    } else if constexpr (PER == 4) {
      const uint2 u = __ldcs(reinterpret_cast<const uint2*>(src));
      acc[0] += wj * bf16lo(u.x);
      acc[1] += wj * bf16hi(u.x);
      acc[2] += wj * bf16lo(u.y);
      acc[3] += wj * bf16hi(u.y);
    } else {
      const uint32_t u = __ldcs(reinterpret_cast<const unsigned int*>(src));
      acc[0] += wj * bf16lo(u);
      acc[1] += wj * bf16hi(u);
    }
  }
  uint16_t* dst = out + (((size_t)b * a.s.T + i) * H + h) * D + lane * PER;
  // a selection without a visible token: zeros (8-bit calls)
  const float inv = Q8 && W == 0.f ? 0.f : back / W;
#pragma unroll
  for (int e = 0; e < PER; e += 2)
    *reinterpret_cast<uint32_t*>(dst + e) = pack_bf16(acc[e] * inv, acc[e + 1] * inv);
}

struct AttnLayout {
  size_t lists, entries, count_off, off_off, toff_off, ent_off, tl_off, po_off, pml_off, total;
};

AttnLayout attn_layout(const Shape& s, bool q8) {
  AttnLayout L{};
  const int tp = pass_len(s);
  L.lists = (size_t)s.B * s.max_blocks * s.G;
  L.entries = (size_t)s.B * tp * s.G * kTopk;
  auto al = [](size_t x) { return (x + 255) / 256 * 256; };
  size_t o = 0;
  L.count_off = o;  o += al(L.lists * 4);
  L.off_off = o;    o += al((L.lists + 1) * 4);
  L.toff_off = o;   o += al((L.lists + 1) * 4);
  L.ent_off = o;    o += al(L.entries * 4);
  L.tl_off = o;     o += al(L.entries * 16);
  const size_t prows = (size_t)s.B * tp * s.H * kTopk;
  L.po_off = o;     o += al(prows * s.D * 2);
  L.pml_off = o;    o += al(prows * (q8 ? sizeof(float4) : sizeof(float2)));
  L.total = o;
  return L;
}

template <int D, bool Q8>
cudaError_t launch_attn_tc_impl(const Shape& s, const Positions& pos, const uint16_t* q,
                                const CacheView& cv, const int32_t* sel, uint16_t* out,
                                const Workspace& ws, cudaStream_t st) {
  using C = AttnCfg<D>;
  const AttnLayout lay = attn_layout(s, Q8);
  char* base = ws.tc_base;
  const int hpg = s.H / s.G;
  const int rpe = hpg <= 8 ? 8 : 16;
  CUtensorMap tm_q, tm_k, tm_v;
  {
    // q as (64 dims, B*T*H rows, D/64 halves): one box = 8 rows (heads) x all
    // D dims, written half after half, i.e. one 8-row group of the Q tile
    cuuint64_t dims[3] = {64, (cuuint64_t)s.B * s.T * s.H, (cuuint64_t)(D / 64)};
    cuuint64_t strides[2] = {(cuuint64_t)D * 2, 128};
    cuuint32_t box[3] = {64, 8, (cuuint32_t)(D / 64)};
    if (!encode_bf16_map(&tm_q, q, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
  }
  if constexpr (Q8) {
    tm_k = tm_v = tm_q;   // not used
  } else {
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)s.G, (cuuint64_t)(s.cache_blocks() * kBlock)};
    cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)s.G * D * 2};
    cuuint32_t box[3] = {64, 1, (cuuint32_t)kBlock};
    if (!encode_bf16_map(&tm_k, cv.k, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_bf16_map(&tm_v, cv.v, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
  }
  cudaError_t e = cudaFuncSetAttribute(attn_tc_kernel<D, Q8>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  // one CTA per SM: all 512 TMEM columns and ~225 KiB of shared memory
  cudaFuncSetAttribute(attn_tc_kernel<D, Q8>, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
  if ((e = cudaFuncSetAttribute(csr_count_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kCsrMaxLists * 4)) != cudaSuccess ||
      (e = cudaFuncSetAttribute(csr_fill_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kCsrMaxLists * 4)) != cudaSuccess)
    return e;
  const int grid = sm_count();
  const int tp_max = pass_len(s);
  for (int t0 = 0; t0 < s.T; t0 += tp_max) {
    AttnPass a;
    a.s = s;
    a.pos = pos;
    a.t0 = t0;
    a.Tp = min(tp_max, s.T - t0);
    const int max_lb = max_local_block(s, pos, t0, t0 + a.Tp);
    a.nbl = max_lb + 1;
    a.nlists = s.B * a.nbl * s.G;
    a.rpe = rpe;
    a.R = 128 / rpe;
    a.sel = sel;
    a.count = reinterpret_cast<int32_t*>(base + lay.count_off);
    a.off = reinterpret_cast<int32_t*>(base + lay.off_off);
    a.tile_off = reinterpret_cast<int32_t*>(base + lay.toff_off);
    a.entries = reinterpret_cast<int32_t*>(base + lay.ent_off);
    a.tile_desc = reinterpret_cast<int4*>(base + lay.tl_off);
    a.part_o = reinterpret_cast<uint16_t*>(base + lay.po_off);
    a.part_ml = reinterpret_cast<float2*>(base + lay.pml_off);
    a.part_mle = reinterpret_cast<float4*>(base + lay.pml_off);
    a.status = ws.status;
    a.wait_polls = debug_wait_polls();
    a.k8 = Q8 ? static_cast<const uint8_t*>(cv.k) : nullptr;
    a.v8 = Q8 ? static_cast<const uint8_t*>(cv.v) : nullptr;
    a.k_exp = cv.k_exp;
    a.v_exp = cv.v_exp;
    const CsrGrid cg = csr_grid(s, a.nbl);
    const unsigned csr_ctas = (unsigned)(s.G * cg.per_group);
    const size_t csr_smem = (size_t)cg.span * 4;
    note_launches(4);
    csr_count_kernel<<<csr_ctas, kCsrThreads, csr_smem, st>>>(a, cg.span, cg.per_group);
    csr_scan_kernel<<<1, 1024, 0, st>>>(a);
    csr_fill_kernel<<<csr_ctas, kCsrThreads, csr_smem, st>>>(a, cg.span, cg.per_group);
    attn_tc_kernel<D, Q8><<<grid, attn_threads<Q8>(), C::kSmem, st>>>(tm_q, tm_k, tm_v, a);
    const int64_t warps = (int64_t)s.B * a.Tp * s.H;
    note_launches(1);
    attn_tc_merge_kernel<D, Q8><<<(unsigned)((warps + 7) / 8), 256, 0, st>>>(a, out);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

int pass_len(const Shape& s) {
  int tp = kPassRows / s.B;
  if (tp < 1) tp = 1;
  return tp < s.T ? tp : (s.T > 0 ? s.T : 1);
}

size_t tc_attn_workspace_bytes(const Shape& s) { return attn_layout(s, false).total; }
size_t tc_attn_q8_workspace_bytes(const Shape& s) { return attn_layout(s, true).total; }

cudaError_t launch_attn_tc(const Shape& s, const Positions& pos, const uint16_t* q,
                           const uint16_t* k, const uint16_t* v, const int32_t* sel,
                           uint16_t* out, const Workspace& ws, cudaStream_t st) {
  const CacheView cv{k, v, nullptr, nullptr, false};
  if (s.D == 128) return launch_attn_tc_impl<128, false>(s, pos, q, cv, sel, out, ws, st);
  return launch_attn_tc_impl<64, false>(s, pos, q, cv, sel, out, ws, st);
}

cudaError_t launch_attn_tc_q8(const Shape& s, const Positions& pos, const uint16_t* q,
                              const CacheView& cv, const int32_t* sel, uint16_t* out, int* status,
                              char* base, cudaStream_t st) {
  Workspace ws{};
  ws.status = status;
  ws.tc_base = base;
  if (s.D == 128) return launch_attn_tc_impl<128, true>(s, pos, q, cv, sel, out, ws, st);
  return launch_attn_tc_impl<64, true>(s, pos, q, cv, sel, out, ws, st);
}

}  // namespace msa

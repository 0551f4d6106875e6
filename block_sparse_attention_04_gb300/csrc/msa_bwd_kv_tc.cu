// dK and dV of the attention's backward pass on tensor cores, and, for a selection,
// dQ's parts: organised around the KV blocks, each owned by one CTA at a time, so that
// the sums over queries and over the heads of a group stay in tensor memory and need
// no atomics.
//
// A unit is a KV block (b, kb, g) with a run of tiles of up to 128 query-head rows:
// 128 queries of one head (dense), or up to R list entries whose heads fill rpe = 8 or
// 16 rows each (sparse; heads past the group's are zero-filled by the copy).  With the
// block's tokens on the 128 lanes of tensor memory and the rows as columns, per tile
//     S^T = K Q^T     dP^T = V dO^T                   (D deep)
//     P^T = 2^(S^T scale log2e - lse log2e)   dS^T = P^T (dP^T - delta)
//     dV += P^T dO    dK += dS^T Q                    (as deep as the tile has rows)
//     dQ part = dS K                                  (sparse: 128 tokens deep)
// P^T and dS^T are written over S^T and dP^T as bf16 and are the products' A operands
// in tensor memory; Q and dO, MN-major, their B operands from the tiles that the first
// two products read K-major.  Sparse, dS^T goes to shared memory instead, whose
// [token][row] order is dK's A operand K-major and that of dQ's part MN-major.
//   warp 0       TMA of Q and dO (four tiles in use or ahead), the rows' statistics; takes
//                the units from a shared counter.  Sparse: of Q alone
//   warp 1       TMA of the unit's K and V; sparse: of dO
//   warp 2       tcgen05.mma; sparse: of S and dV
//   warp 3       sparse: tcgen05.mma of dP, dK and dQ's part; dense: waits for copies
//   warps 4-19   P and dS: four warpgroups, 32 columns of a tile each; a unit's dV, dK
//   warps 20-23  sparse: dQ's parts, bf16, one row of 16 slots x D per (query, head)
// dS(n) is worked out during dV(n) and S(n+1), P(n+1) during dK(n) and dP(n+1).  Sparse,
// D = 128: tensor memory holds S, dP, dV and dK (512 columns), so dQ's part takes dP's
// columns until it has been read out, during dV(n+1) and S(n+2).
//
// What is rounded: P and dS to bf16, as operands; dQ's parts, one for each of the 16
// selected blocks, to bf16 (within 2^-8, summed in fp32 afterwards): as fp32 they would be
// 1.4 GB more written and 1.9 more read for 8192 tokens of 48 heads, 490 us more for 1407.
//
// Shared memory's 128 bytes a cycle are the bound: of a dense tile at D = 128 the
// products read 192 KB (both operands of S and dP, one of dV and dK), the copies write
// 64, and a thread per token would read every row's two numbers, 1 KB a warp, whose way to
// the registers costs as much as 104 KB.  So these come in through the products: a step of
// S and of dP on top of the others multiplies ones with them, as three bf16 parts
// (4 x 2048 tokens, 48/8 heads: 293 us, 347 with the numbers read by the threads).  A
// sparse tile's products read 288 KB (dS, too, and K once more), 64 are copied and 32
// written: 3000 cycles of the 4600 that a tile takes (8192 tokens: 1001 us, the tensor
// pipe at 0.55 of its cycles).
//
// Tried for the sparse tiles, 8192 tokens: all MMAs from one warp in a fixed order, as for
// the dense ones, 1107 us (D = 64, 2 x 101 tokens: 40 for 44); the parts read out by the
// P and dS warps, 1059 (with warp 2's waits by another warp 1270); dS over dO's slot, with two sets of statistics, 1098; a group's
// units together, so that its Q and dO stay in L2, 1030 to 1090; rows prefetched into L2
// three tiles ahead, 1600.
#include <type_traits>

#include "msa_bwd.h"
#include "msa_bwd_q_tc.cuh"
#include "msa_q8.cuh"
#include "msa_tma.h"

namespace msa {
namespace {

// warps: MMA (sparse: of dV and S); dense: the MMA warp's waits, sparse: MMA of dP, dK and
// dQ's part; P and dS
constexpr int kAW = 2, kBW = 3, kSoftW = 4;
constexpr int kNG = 4;                    // warpgroups for P and dS ...
constexpr int kCols = 128 / kNG;          // ... and the columns of a tile that each has
constexpr int kOutW = kSoftW + 4 * kNG;
template <bool SP>
constexpr int kv_threads() { return 32 * (kOutW + (SP ? 4 : 0)); }
constexpr int kRing = 4;                  // unit numbers published by warp 0, ahead of use
template <bool SP>
constexpr int ring_readers() { return 3 + 4 * kNG + (SP ? 4 : 0); }

template <int D, bool SP>
struct KvCfg {
  static constexpr int kNHalf = D / 64;
  static constexpr int kHalf = 128 * 128;            // 128 rows x 64 dims
  static constexpr int kTile = kNHalf * kHalf;       // K, V, a Q or a dO tile
  // Dense, D = 64: tensor memory has room for a second S, so that S(n+2) is made on dS(n)
  // and no P waits for its S (3 chunks of 1000 queries, 64/4 heads: 922 -> 812 us
  // in all)
  static constexpr bool kTwoS = !SP && D == 64;
  static constexpr int kTiles = kTwoS ? 8 : 4;       // Q and dO tiles in shared memory
  static constexpr int kSS = SP ? 1 : kTwoS ? 4 : 2; // statistics of tiles
  static constexpr int kStat = 16 * kAugBytes;       // statistics of a tile
  static constexpr int kOnes = 2 * 256;              // their selectors, A operands
  static constexpr int kDs = SP ? 2 * kHalf : 0;     // dS^T [2 x 64 rows][128 tokens]
  static constexpr int kFills = 2 * kTiles + kSS;
  static constexpr int kBars = (2 * (kTiles + kSS) + 13 + 2 * kRing) * 8 + (kRing + kFills) * 4 + 8;
  static constexpr int kSmem =
      (2 + kTiles) * kTile + kDs + kOnes + kSS * kStat + 2 * 80 + kBars;
  // Slots of tile n's Q and dO, and the number of times that they were filled before.
  // dO(n) is free first (after dV(n); sparse dP(n)), Q(n) after dK(n), and what comes
  // next, Q(n+2) and dO(n+2), goes into them in that order.
  // (Eight slots: each its own.)
  __device__ static int q_slot(int n) { return kTwoS ? 2 * (n & 3) : 2 * (n & 1) + (n >> 1 & 1); }
  __device__ static int o_slot(int n) { return kTwoS ? 2 * (n & 3) + 1 : 2 * (n & 1) + (~n >> 1 & 1); }
  __device__ static uint32_t use(int n) { return (uint32_t)(kTwoS ? n >> 2 : n >> 1); }
  // S of tile n: its columns (the second behind all others), its barrier and its parity
  __device__ static uint32_t s_at(int n) { return kTwoS && (n & 1) ? 256 + 2 * D : 0; }
  __device__ static int s_bar(int n) { return kTwoS ? n & 1 : 0; }
  __device__ static uint32_t s_use(int n) { return (uint32_t)(kTwoS ? n >> 1 : n) & 1; }
  // byte offsets of a tile of rows: sparse tiles hold 8-row groups, half after half
  static constexpr int kGroup = SP ? kNHalf * 1024 : 1024;   // next 8 rows
  static constexpr int kNext = SP ? 1024 : kHalf;            // next 64 dims
  // tensor memory columns: S, dP, dV, dK, dQ's part (D = 128: in dP's place)
  static constexpr uint32_t kP = 128, kDV = 256, kDK = 256 + D;
  static constexpr uint32_t dq() { return D == 128 ? kP : 256 + 2 * D; }
  static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
};

struct KvUnit {
  int b, g, kb, first, size, slot, tiles;
};
template <bool SP>
__device__ __forceinline__ KvUnit kv_unit(const BwdArgs& a, int it) {
  const int4 d = a.units[it];
  KvUnit u;
  u.kb = d.x & 0x7FFF;
  u.g = d.x >> 15 & 7;
  u.b = d.x >> 18;
  u.first = d.y;
  u.size = d.z;
  u.slot = d.w;
  u.tiles = SP ? (d.z + a.R - 1) / a.R : d.z;
  return u;
}

__device__ __forceinline__ float2 pair(const uint32_t* x, int i) {
  return make_float2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]));
}

// Dense: tile of the unit -> head of the group and query tile.
__device__ __forceinline__ void dense_tile(const BwdArgs& a, const KvUnit& u, int q0, int t, int& h,
                                           int& qt) {
  const int n = a.nqt - q0;
  h = (u.first + t) / n;
  qt = q0 + (u.first + t) % n;
}

// Sparse: 16-row steps of tile t (the last tile of a list may be short).
__device__ __forceinline__ int sparse_steps(const BwdArgs& a, const KvUnit& u, int t) {
  const int ne = min(a.R, u.size - t * a.R);
  return (ne * a.rpe + 15) >> 4;
}

// Sparse: what a lane of a copying warp knows of its 8-row group of a tile.
struct SparseRows {
  int entry, il, z, box_r, boxes;    // entry: of the tile that was fetched
  int64_t row;
  bool real;
  __device__ __forceinline__ void fetch(const BwdArgs& a, const KvUnit& u, int t, int lane) {
    const int at = t * a.R + (lane & 15) / (a.rpe >> 3);
    if (at < u.size) entry = a.entries[u.first + at];
  }
  __device__ __forceinline__ void place(const BwdArgs& a, const KvUnit& u, int t, int lane) {
    const int bpe = a.rpe >> 3;
    boxes = 2 * sparse_steps(a, u, t);
    real = t * a.R + (lane & 15) / bpe < u.size;
    il = real ? entry >> 4 : 0;
    row = (int64_t)u.b * a.s.T + a.t0 + il;
    // past the end for rows without an entry: zeros
    z = real ? (int)(row * a.s.G + u.g) : a.s.B * a.s.T * a.s.G;
    box_r = (lane & 15) % bpe * 8;
  }
};

template <int D, bool SP>
__device__ __forceinline__ void kv_cta(const CUtensorMap& tm_q, const CUtensorMap& tm_o,
                                       const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                       const BwdArgs& a) {
  using C = KvCfg<D, SP>;
  extern __shared__ __align__(1024) uint8_t smem[];   // the swizzled tiles' alignment
  uint8_t* sK = smem;
  uint8_t* sV = sK + C::kTile;
  uint8_t* sT = sV + C::kTile;                     // [kTiles] Q and dO
  uint8_t* sDs = sT + C::kTiles * C::kTile;
  uint8_t* sOnes = sDs + C::kDs;                   // selectors of lse and of delta
  uint8_t* sStat = sOnes + C::kOnes;               // [kSS] statistics
  // [2] per 8-row group of a sparse tile: the last token of the block that its query
  // sees (-1: none), then whether any of them is below 127
  int* sLim = reinterpret_cast<int*>(sStat + C::kSS * C::kStat);
  uint64_t* t_full = reinterpret_cast<uint64_t*>(sLim + 2 * 20);
  uint64_t* t_empty = t_full + C::kTiles;
  uint64_t* st_full = t_empty + C::kTiles;
  uint64_t* st_empty = st_full + C::kSS;
  uint64_t* kv_full = st_empty + C::kSS;           // K and V of the unit landed
  uint64_t* kv_empty = kv_full + 1;                // its last product that reads them is done
  uint64_t* s_full = kv_empty + 1;                 // [2] S of the tile is in tensor memory
  // [2] dP of the tile: one for even and odd tiles, as the warp that issues S waits for it
  // too and may fall behind
  uint64_t* dp_full = s_full + 2;
  uint64_t* p_full = dp_full + 2;                  // P written over S
  uint64_t* ds_full = p_full + 1;                  // dS written over dP (and to shared memory)
  uint64_t* acc_full = ds_full + 1;                // the unit's dV and dK are complete
  uint64_t* acc_empty = acc_full + 1;              // ... and read out
  uint64_t* dq_full = acc_empty + 1;               // sparse: dQ's part is in tensor memory
  uint64_t* dq_empty = dq_full + 1;                // ... and read out
  uint64_t* bar_fin = dq_empty + 1;
  uint64_t* it_full = bar_fin + 1;                 // [kRing]
  uint64_t* it_empty = it_full + kRing;
  int* ring = reinterpret_cast<int*>(it_empty + kRing);   // unit numbers, -1: no more
  // the last fill of each tile slot by warp 0, then by warp 1, then of each statistics slot
  int* last_fill = ring + kRing;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(last_fill + C::kFills);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kTiles; ++i) {
      mbar_init(&t_full[i], 1);
      mbar_init(&t_empty[i], SP ? 2 : 1);    // sparse: both MMA warps are done with it
    }
    for (int i = 0; i < C::kSS; ++i) {
      mbar_init(&st_full[i], 1);
      mbar_init(&st_empty[i], SP ? 2 : 1);
    }
    mbar_init(kv_full, 1);
    mbar_init(kv_empty, SP ? 2 : 1);
    mbar_init(&s_full[0], SP ? 2 : 1);     // sparse: and the tile's limits are there
    mbar_init(&s_full[1], 1);
    mbar_init(&dp_full[0], 1);
    mbar_init(&dp_full[1], 1);
    // a warp arrives once (512 threads: see below); dense: and what comes next has landed
    mbar_init(p_full, 4 * kNG + (SP ? 0 : 1));
    mbar_init(ds_full, 4 * kNG + (SP ? 0 : 1));
    mbar_init(acc_full, SP ? 2 : 1);
    mbar_init(acc_empty, 4 * kNG);
    mbar_init(dq_full, 1);
    mbar_init(dq_empty, 4);
    mbar_init(bar_fin, SP ? 2 : 1);
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&it_full[i], 1);
      mbar_init(&it_empty[i], ring_readers<SP>());
    }
    *abort_flag = 0;
    for (int i = 0; i < C::kFills; ++i) last_fill[i] = -1;
    fence_mbar_init();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_o);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  // The statistics' rows are 8 bf16, K-major without a swizzle: -lse in three parts at 0..2,
  // -delta at 4..6 (see msa_bwd.h).  An MMA is 16 deep: the second 8 are the first again
  // (a stride of 0), and meet zeros.  The selectors have ones at 0..2 or 4..6; all their
  // 128 rows are the same 8
  if (threadIdx.x < C::kOnes / 16) {
    const int sel = threadIdx.x >> 4, second = threadIdx.x >> 3 & 1;   // of lse or delta; dims 8..
    const uint32_t one = second ? 0u : 0x3F80u, a0 = sel ? 0u : one, a1 = sel ? one : 0u;
    sts128(smem_u32(sOnes) + threadIdx.x * 16, make_uint4(a0 | a0 << 16, a0, a1 | a1 << 16, a1));
    fence_async();
  }
  if (warp == kAW) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int T = a.s.T, H = a.s.H;

  // A warp's next unit from the ring (every lane gets it); false: no more, or given up.
  int ki = 0;
  auto next_unit = [&](int& it, bool& ok) {
    const int slot = ki % kRing;
    ok = __all_sync(0xffffffffu, *abort_flag == 0 && mbar_wait(&it_full[slot], (ki / kRing) & 1,
                                                               a.status, a.wait_polls));
    if (!ok) return false;
    // read by every lane before the slot is handed back
    it = __shfl_sync(0xffffffffu, ring[slot], 0);
    if (lane == 0) mbar_arrive(&it_empty[slot]);
    ++ki;
    return it >= 0;
  };
  auto wait_all = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, a.status, a.wait_polls));
  };
  // One arrival for the lanes' work so far.
  auto warp_arrive = [&](uint64_t* bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };
  // Sparse: a tile's rows, 8 to a box.
  auto load_rows = [&](uint8_t* dst, const CUtensorMap* map, uint64_t* bar, const SparseRows& x,
                       uint64_t pol) {
    if (lane == 0) mbar_arrive_expect_tx(bar, (uint32_t)(x.boxes * C::kGroup));
    __syncwarp();
#pragma unroll 4
    for (int i = 0; i < x.boxes; ++i) {
      const int z = __shfl_sync(0xffffffffu, x.z, i), box_r = __shfl_sync(0xffffffffu, x.box_r, i);
      if (elect_one())
        tma_load_4d_hint(smem_u32(dst + i * C::kGroup), map, bar, 0, box_r, z, 0, pol);
    }
    __syncwarp();
  };

  if (warp == 0) {
    // ------------------------- Q and statistics, dense: dO too (warp 0); takes the units
    const uint64_t pol = l2_policy_evict_last();   // rows are read again by other units
    const int n_units = a.n_units[0];
    int cur = 0;
    if (lane == 0) {
      cur = atomicAdd(a.next_unit, 1);
      if (cur >= n_units) cur = -1;
      ring[0] = cur;
      mbar_arrive(&it_full[0]);
    }
    cur = __shfl_sync(0xffffffffu, cur, 0);
    int n = 0;                     // tiles issued
    bool ok = true;
    for (int k = 0; cur >= 0 && ok; ++k) {
      // publish the next unit before this one's tiles
      const int r = k + 1, slot = r % kRing;
      if (r >= kRing && !wait_all(&it_empty[slot], ((r / kRing) - 1) & 1)) { ok = false; break; }
      int nx = 0;
      if (lane == 0) {
        nx = *abort_flag ? n_units : atomicAdd(a.next_unit, 1);
        if (nx >= n_units) nx = -1;
        ring[slot] = nx;
        mbar_arrive(&it_full[slot]);
      }
      nx = __shfl_sync(0xffffffffu, nx, 0);
      const KvUnit u = kv_unit<SP>(a, cur);
      const int q0 = SP ? 0 : bwd_first_tile(a, u.b, u.kb);
      const int64_t t_last = (int64_t)a.pos.q_start[u.b] + T - 1;
      SparseRows rows{};
      if constexpr (SP) rows.fetch(a, u, 0, lane);
      for (int t = 0; t < u.tiles; ++t, ++n) {
        const int qs = C::q_slot(n), os = C::o_slot(n), ss = n % C::kSS;
        uint8_t* const dst = sT + qs * C::kTile;
        const uint32_t st = smem_u32(sStat + ss * C::kStat);
        if (__any_sync(0xffffffffu, *abort_flag != 0) || !wait_all(&t_empty[qs], (C::use(n) & 1) ^ 1)) {
          ok = false;
          break;
        }
        if constexpr (SP) {
          rows.place(a, u, t, lane);
          load_rows(dst, &tm_q, &t_full[qs], rows, pol);
          if (lane == 0) last_fill[qs] = (int)C::use(n);
          // a block that the sequence's last query does not reach the end of may hold
          // anything behind it: rows without an entry see none of it
          const int64_t seen = (int64_t)a.pos.q_start[u.b] + a.t0 + rows.il - (int64_t)u.kb * kBlock;
          const int lim = rows.real ? (int)(seen < 127 ? seen : 127)
                                    : (t_last - (int64_t)u.kb * kBlock < 127 ? -1 : 127);
          const bool any = __any_sync(0xffffffffu, (lane & 15) < rows.boxes && lim < 127);
          const int bpe = a.rpe >> 3, boxes = rows.boxes;
          const uint32_t sg = rows.real ? (uint32_t)(rows.row * a.s.G + u.g) * bpe + lane % bpe
                                        : a.stat_groups;
          // The statistics by way of registers: they are asked for before their slot is free,
          // which it is when S has to be issued (as bulk copies, 16 to a tile, they held S up
          // for 3000 cycles)
          uint4 x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t from = __shfl_sync(0xffffffffu, sg, i * 4 + (lane >> 3));
            x[i] = make_uint4(0, 0, 0, 0);
            if (i * 4 + (lane >> 3) < boxes)
              x[i] = __ldcg(reinterpret_cast<const uint4*>(a.stat + (size_t)from * kAugBytes) + (lane & 7));
          }
          rows.fetch(a, u, t + 1, lane);
          if (!wait_all(&st_empty[ss], ((uint32_t)(n / C::kSS) & 1) ^ 1)) { ok = false; break; }
          if (lane < 16) sLim[(n & 1) * 20 + lane] = lim;
          if (lane == 16) sLim[(n & 1) * 20 + 16] = any;
#pragma unroll
          for (int i = 0; i < 4; ++i) sts128(st + (i * 32 + lane) * 16, x[i]);
          fence_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(&st_full[ss]);
        } else {
          int h, qt;
          dense_tile(a, u, q0, t, h, qt);
          h += u.g * a.hpg;
          const size_t sg = (size_t)(u.b * H + h) * a.stat_groups + qt * 16;
          auto load_tile = [&](int slot, const CUtensorMap* map) {
            mbar_arrive_expect_tx(&t_full[slot], C::kTile);
#pragma unroll
            for (int hf = 0; hf < C::kNHalf; ++hf)
              tma_load_4d_hint(smem_u32(sT + slot * C::kTile + hf * C::kHalf), map, &t_full[slot],
                               hf * 64, h, qt * 128, u.b, pol);
            last_fill[slot] = (int)C::use(n);
          };
          if (lane == 0) load_tile(qs, &tm_q);
          __syncwarp();
          if (!wait_all(&st_empty[ss], ((uint32_t)(n / C::kSS) & 1) ^ 1)) { ok = false; break; }
          if (lane == 0) {
            mbar_arrive_expect_tx(&st_full[ss], C::kStat);
            bulk_load(st, a.stat + sg * kAugBytes, C::kStat, &st_full[ss]);
            last_fill[2 * C::kTiles + ss] = n / C::kSS;
          }
          __syncwarp();
          if (!wait_all(&t_empty[os], (C::use(n) & 1) ^ 1)) { ok = false; break; }
          if (lane == 0) load_tile(os, &tm_o);
          __syncwarp();
        }
      }
      cur = nx;
    }
    if (!ok && lane == 0) *abort_flag = 1;
  } else if (warp == 1) {
    // ------------------------------------------- K and V, sparse: dO too (warp 1)
    // (A box of 8 rows takes a warp some 70 cycles to issue, so that one warp with a tile's
    // 32 held up the rest: 8192 tokens 1093 us for 1011.)
    const uint64_t pol = l2_policy_evict_last();
    const int late = a.late_kv;
    int it, n = 0, nu = 0;
    bool ok;
    while (next_unit(it, ok)) {
      const KvUnit u = kv_unit<SP>(a, it);
      if (u.tiles == 0) continue;
      SparseRows rows{};
      if constexpr (SP) rows.fetch(a, u, 0, lane);
      if (nu > 0 && !wait_all(kv_empty, (uint32_t)(nu - 1) & 1)) { ok = false; break; }
      if (!SP && nu == late) copy_delay(a.late_ns);
      if (lane == 0) {
        const int row = (int)(((int64_t)u.b * a.s.max_blocks + u.kb) * kBlock);
        mbar_arrive_expect_tx(kv_full, 2 * C::kTile);
#pragma unroll
        for (int hf = 0; hf < C::kNHalf; ++hf) {
          tma_load_3d(smem_u32(sK + hf * C::kHalf), &tm_k, kv_full, hf * 64, u.g, row);
          tma_load_3d(smem_u32(sV + hf * C::kHalf), &tm_v, kv_full, hf * 64, u.g, row);
        }
      }
      __syncwarp();
      ++nu;
      if constexpr (SP) {
        for (int t = 0; t < u.tiles; ++t, ++n) {
          const int os = C::o_slot(n);
          if (__any_sync(0xffffffffu, *abort_flag != 0) || !wait_all(&t_empty[os], (C::use(n) & 1) ^ 1)) {
            ok = false;
            break;
          }
          if (n == late) copy_delay(a.late_ns);
          rows.place(a, u, t, lane);
          load_rows(sT + os * C::kTile, &tm_o, &t_full[os], rows, pol);
          if (lane == 0) last_fill[C::kTiles + os] = (int)C::use(n);
          rows.fetch(a, u, t + 1, lane);
        }
        if (!ok) break;
      }
    }
    if (!ok && lane == 0) *abort_flag = 1;
    if (nu > 0) mbar_wait(kv_full, (uint32_t)(nu - 1) & 1, nullptr);
  } else if (warp == kAW || (SP && warp == kBW)) {
    // ------------------------------------------------------- MMA (warps 2, 3)
    constexpr uint32_t idesc_n = idesc_bf16(128, D, false, true);     // dV, dK
    constexpr uint32_t idesc_q = idesc_bf16(128, D, true, true);      // dQ's part
    const uint64_t kd = smem_desc(smem_u32(sK), 16, 1024, kSwizzle128B);
    const uint64_t vd = smem_desc(smem_u32(sV), 16, 1024, kSwizzle128B);
    const uint64_t kmn = smem_desc(smem_u32(sK), C::kHalf, 1024, kSwizzle128B);
    const uint64_t dsmn = smem_desc(smem_u32(sDs), C::kHalf, 1024, kSwizzle128B);
    const uint64_t dsk = smem_desc(smem_u32(sDs), 16, 1024, kSwizzle128B);
    const uint64_t tk = smem_desc(smem_u32(sT), 16, C::kGroup, kSwizzle128B);
    const uint64_t tmn = smem_desc(smem_u32(sT), C::kNext, C::kGroup, kSwizzle128B);
    // A (128 x D, K-major) times a tile of rows, K-major: `steps` x 16 columns, on top of
    // the rows' statistics (sel 0: -lse, 1: -delta).  (An instruction descriptor that is
    // not a constant costs an MMA 40 cycles: full tiles have one.)
    const uint64_t onesd = smem_desc(smem_u32(sOnes), 128, 0, 0);
    const uint64_t augd = smem_desc(smem_u32(sStat), 0, kAugBytes, 0);
    auto rows_product = [&](uint32_t d, uint64_t ad, int slot, int steps, int sel, int ss) {
      const uint64_t bd = tk + (uint64_t)((slot * C::kTile) >> 4);
      auto all = [&](uint32_t idesc) {
        tc_mma_f16(tmem + d, onesd + (uint64_t)((sel * 256) >> 4),
                   augd + (uint64_t)((ss * C::kStat) >> 4), idesc, 0u);
        if (sel == 0 && a.no_scores) return;
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
          tc_mma_f16(tmem + d, ad + (uint64_t)(((j >> 2) * C::kHalf + (j & 3) * 32) >> 4),
                     bd + (uint64_t)(((j >> 2) * C::kNext + (j & 3) * 32) >> 4), idesc, 1u);
      };
      if (!SP || steps == 8) all(idesc_bf16(128, 128, false, false));
      else all(idesc_bf16(128, 0, false, false) | (uint32_t)(2 * steps) << 17);
    };
    // P^T or dS^T (TMEM at column p, kCols columns of a tile in half as many) times a tile
    auto sum_product = [&](uint32_t d, uint32_t p, int slot, int steps, bool add) {
      const uint64_t bd = tmn + (uint64_t)((slot * C::kTile) >> 4);
      auto step = [&](int j) {
        tc_mma_f16_ts(tmem + d, tmem + p + j * 16 / kCols * kCols + j * 16 % kCols / 2,
                      bd + (uint64_t)((j * 2 * C::kGroup) >> 4), idesc_n, add || j > 0 ? 1u : 0u);
      };
      if (!SP || steps == 8) {
#pragma unroll
        for (int j = 0; j < 8; ++j) step(j);
      } else {
        for (int j = 0; j < steps; ++j) step(j);
      }
    };
    int it, n = 0, nu = 0;       // tiles and units (with tiles) so far
    bool ok;
    if constexpr (!SP) {
      // -------------- S(0), dP(0); dV(n), S(n + 1) on P(n); dK(n), dP(n + 1) on dS(n)
      // One warp, in this order: S(n + 1), whose P takes longest, is not held up by the
      // others (two warps, as below: 4 x 2048 tokens 347 us for 302).  Few MMAs are
      // in flight behind an issue, and a wait takes 190 cycles even where it is over, so
      // that the next warp takes the waits for copies and this one two a tile
      while (next_unit(it, ok)) {
        const KvUnit u = kv_unit<SP>(a, it);
        if (u.tiles == 0) continue;
        auto issue_s = [&](int m) {
          rows_product(C::s_at(m), kd, C::q_slot(m), 8, 0, m % C::kSS);
          tc_commit(&s_full[C::s_bar(m)]);
        };
        auto issue_dp = [&](int m) {
          rows_product(C::kP, vd, C::o_slot(m), 8, 1, m % C::kSS);
          tc_commit(&dp_full[m & 1]);
          tc_commit(&st_empty[m % C::kSS]);
        };
        const bool two = C::kTwoS && u.tiles > 1;
        ok = wait_all(kv_full, (uint32_t)nu & 1);
        for (int m = n; m <= n + two && ok; ++m)
          ok = wait_all(&t_full[C::q_slot(m)], C::use(m) & 1) &&
               wait_all(&st_full[m % C::kSS], (uint32_t)(m / C::kSS) & 1);
        ok = ok && wait_all(&t_full[C::o_slot(n)], C::use(n) & 1);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          issue_s(n);
          issue_dp(n);
          if (two) issue_s(n + 1);
          if (u.tiles == 1) tc_commit(kv_empty);
        }
        __syncwarp();
        for (int t = 0; t < u.tiles; ++t, ++n) {
          const int qs = C::q_slot(n), os = C::o_slot(n);
          const bool more = t + 1 < u.tiles;
          ok = wait_all(p_full, (uint32_t)n & 1);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            sum_product(C::kDV, C::s_at(n), os, 8, t > 0);
            tc_commit(&t_empty[os]);
            if (!C::kTwoS && more) issue_s(n + 1);   // over P(n), which dV(n) reads
          }
          __syncwarp();
          ok = wait_all(ds_full, (uint32_t)n & 1);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            sum_product(C::kDK, C::kP, qs, 8, t > 0);
            tc_commit(&t_empty[qs]);
            if (more) {                              // over dS(n), which dK(n) reads
              issue_dp(n + 1);
              if (C::kTwoS && t + 2 < u.tiles) issue_s(n + 2);
              if (t + 2 == u.tiles) tc_commit(kv_empty);
            } else {
              tc_commit(acc_full);
            }
          }
          __syncwarp();
        }
        if (!ok) break;
        ++nu;
      }
    } else if (warp == kAW) {
      // ------------------------------------------------ S(0); dV(n), S(n + 1)
      // Two warps, as issuing takes long (a product, with its wait and commits, 500 to 800
      // cycles of a warp), and dQ's part with its readout is what is waited for
      while (next_unit(it, ok)) {
        const KvUnit u = kv_unit<SP>(a, it);
        if (u.tiles == 0) continue;
        ok = wait_all(kv_full, (uint32_t)nu & 1);
        if (!ok) break;
        const int64_t left = (int64_t)a.pos.q_start[u.b] + T - 1 - (int64_t)u.kb * kBlock;
        if (left < kBlock - 1) {
          // K rows behind the last query may hold anything; as terms of dQ's part they
          // are multiplied by zeros: cleared
          for (int e = lane; e < C::kNHalf * kBlock * 8; e += 32) {
            const int row = e >> 3 & 127;
            if (row > (int)left)
              sts128(smem_u32(sK) + (e >> 10) * C::kHalf + row * 128 + (e & 7) * 16,
                     make_uint4(0, 0, 0, 0));
          }
          fence_async();
          __syncwarp();
        }
        auto issue_s = [&](int m, int t) {         // S of tile m, the unit's t-th
          const int qs = C::q_slot(m), ss = m % C::kSS;
          if (!wait_all(&t_full[qs], C::use(m) & 1) ||
              !wait_all(&st_full[ss], (uint32_t)(m / C::kSS) & 1))
            return false;
          // hands on what warp 0 wrote: the limits.  (They are kept for two tiles: dP of the
          // tile between, which frees the statistics, is issued behind dS of the first)
          if (lane == 0) mbar_arrive(s_full);
          tc_fence_after();
          if (elect_one()) {
            rows_product(C::s_at(0), kd, qs, sparse_steps(a, u, t), 0, ss);
            tc_commit(s_full);
            tc_commit(&t_empty[qs]);
            tc_commit(&st_empty[ss]);
            if (t + 1 == u.tiles) tc_commit(kv_empty);
          }
          __syncwarp();
          return true;
        };
        ok = issue_s(n, 0);
        for (int t = 0; t < u.tiles && ok; ++t, ++n) {
          const int os = C::o_slot(n);
          ok = wait_all(p_full, (uint32_t)n & 1) &&
               (t > 0 || nu == 0 || wait_all(acc_empty, (uint32_t)(nu - 1) & 1)) &&
               wait_all(&t_full[os], C::use(n) & 1);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            sum_product(C::kDV, C::s_at(0), os, sparse_steps(a, u, t), t > 0);
            tc_commit(&t_empty[os]);
            if (t + 1 == u.tiles) tc_commit(acc_full);
          }
          __syncwarp();
          // S(n + 1) goes over P(n), which dV(n), issued before, reads, and behind dP(n), which
          // is waited for longer
          if (t + 1 < u.tiles)
            ok = wait_all(&dp_full[n & 1], (uint32_t)(n >> 1) & 1) && issue_s(n + 1, t + 1);
        }
        if (!ok) break;
        ++nu;
      }
    } else {
      // ------------------------------------------ dP(n); dQ's part(n), dK(n)
      while (next_unit(it, ok)) {
        const KvUnit u = kv_unit<SP>(a, it);
        if (u.tiles == 0) continue;
        ok = wait_all(kv_full, (uint32_t)nu & 1);
        if (!ok) break;
        for (int t = 0; t < u.tiles && ok; ++t, ++n) {
          const int qs = C::q_slot(n), os = C::o_slot(n), ss = n % C::kSS;
          const bool more = t + 1 < u.tiles;
          // D = 128: dQ's part of the tile before is in dP's place until it is read out
          ok = wait_all(&t_full[os], C::use(n) & 1) &&
               wait_all(&st_full[ss], (uint32_t)(n / C::kSS) & 1) &&
               (D != 128 || n == 0 || wait_all(dq_empty, (uint32_t)(n - 1) & 1));
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            rows_product(C::kP, vd, os, sparse_steps(a, u, t), 1, ss);
            tc_commit(&dp_full[n & 1]);
            tc_commit(&t_empty[os]);
            tc_commit(&st_empty[ss]);
          }
          __syncwarp();
          ok = wait_all(ds_full, (uint32_t)n & 1) &&
               (t > 0 || nu == 0 || wait_all(acc_empty, (uint32_t)(nu - 1) & 1));
          if (D != 128 && n > 0) ok = ok && wait_all(dq_empty, (uint32_t)(n - 1) & 1);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            // dQ's part = dS K: 128 tokens in 8 steps; read out during dK
#pragma unroll
            for (int j = 0; j < 8; ++j)
              tc_mma_f16(tmem + C::dq(), dsmn + (uint64_t)((j * 2048) >> 4),
                         kmn + (uint64_t)((j * 2048) >> 4), idesc_q, j > 0 ? 1u : 0u);
            tc_commit(dq_full);
            if (!more) tc_commit(kv_empty);
            const int steps = sparse_steps(a, u, t);
            const uint64_t bd = tmn + (uint64_t)((qs * C::kTile) >> 4);
            auto step = [&](int j) {
              tc_mma_f16(tmem + C::kDK, dsk + (uint64_t)(((j >> 2) * C::kHalf + (j & 3) * 32) >> 4),
                         bd + (uint64_t)((j * 2 * C::kGroup) >> 4), idesc_n,
                         t > 0 || j > 0 ? 1u : 0u);
            };
            if (steps == 8) {
#pragma unroll
              for (int j = 0; j < 8; ++j) step(j);
            } else {
              for (int j = 0; j < steps; ++j) step(j);
            }
            tc_commit(&t_empty[qs]);
            if (!more) tc_commit(acc_full);
          }
          __syncwarp();
        }
        if (!ok) break;
        ++nu;
      }
    }
    if (!ok && lane == 0) *abort_flag = 1;
    // all MMAs of both warps done before tensor memory is released
    if (elect_one()) tc_commit(bar_fin);
    __syncwarp();
    mbar_wait(bar_fin, 0, nullptr);
  } else if (!SP && warp == kBW) {
    // -------------------------------------- the MMA warp's waits (dense, warp 3)
    // Arrives with the softmax warps: at P(n) once the next tile's Q and statistics are in
    // shared memory (and the last unit's sums have been read out), at dS(n) once its dO is.
    int it, n = 0, nu = 0;
    bool ok;
    while (next_unit(it, ok)) {
      const KvUnit u = kv_unit<SP>(a, it);
      if (u.tiles == 0) continue;
      for (int t = 0; t < u.tiles; ++t, ++n) {
        const int m = n + 1;
        const bool more = t + 1 < u.tiles;
        auto wait_q = [&](int x) {
          return wait_all(&t_full[C::q_slot(x)], C::use(x) & 1) &&
                 wait_all(&st_full[x % C::kSS], (uint32_t)(x / C::kSS) & 1);
        };
        ok = __any_sync(0xffffffffu, *abort_flag != 0) == 0 && (C::kTwoS || !more || wait_q(m)) &&
             (t > 0 || nu == 0 || wait_all(acc_empty, (uint32_t)(nu - 1) & 1)) &&
             (n == 0 || wait_all(p_full, (uint32_t)(n - 1) & 1));   // not into the phase before
        if (!ok) break;
        if (lane == 0) mbar_arrive(p_full);
        ok = (!more || wait_all(&t_full[C::o_slot(m)], C::use(m) & 1)) &&
             (!C::kTwoS || t + 2 >= u.tiles || wait_q(n + 2)) &&
             (n == 0 || wait_all(ds_full, (uint32_t)(n - 1) & 1));
        if (!ok) break;
        if (lane == 0) mbar_arrive(ds_full);
      }
      if (!ok) break;
      ++nu;
    }
    if (!ok && lane == 0) *abort_flag = 1;
  } else if (warp >= kSoftW && warp < kOutW) {
    // ------------------------------------------ P, dS; dV and dK (warps 4-19)
    const int c = (warp - kSoftW) >> 2;           // columns kCols c .. of each tile
    const int quad = warp & 3;
    const int r = quad * 32 + lane;               // token of the block = TMEM lane
    const uint32_t base = tmem + ((uint32_t)(quad * 32) << 16);
    const float sl = a.no_scores ? 1.f : a.s.scale * kLog2e;
    const float2 sl2 = make_float2(sl, sl);
    int it, n = 0, nu = 0;
    bool ok;
    while (next_unit(it, ok)) {
      const KvUnit u = kv_unit<SP>(a, it);
      const int q0 = SP ? 0 : bwd_first_tile(a, u.b, u.kb);
      const int64_t t_key = (int64_t)u.kb * kBlock + r;
      const bool used = t_key <= (int64_t)a.pos.q_start[u.b] + T - 1;  // by the last query
      for (int t = 0; t < u.tiles; ++t, ++n) {
        int cols = kCols;                         // of this warpgroup's that the tile has
        int lim = 0;                              // dense: columns below see another token
        bool masked;
        ok = *abort_flag == 0 &&
             mbar_wait(&s_full[C::s_bar(n)], C::s_use(n), a.status, a.wait_polls);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const int* tl = sLim + (n & 1) * 20 + c * (kCols / 8);
        if constexpr (SP) {
          cols = sparse_steps(a, u, t) * 16 - c * kCols;
          masked = sLim[(n & 1) * 20 + 16] != 0;
        } else {
          int h, qt;
          dense_tile(a, u, q0, t, h, qt);
          const int64_t d = t_key - ((int64_t)a.pos.q_start[u.b] + qt * 128);
          lim = used ? (int)(d > 0 ? d : 0) - c * kCols : kCols;
          masked = __any_sync(0xffffffffu, lim > 0);
        }
        // zeros at columns col and col + 1 of this warpgroup, where they do not see token r
        auto hide = [&](float2& v, int col) {
          v.x = (SP ? r > tl[col >> 3] : col < lim) ? 0.f : v.x;
          v.y = (SP ? r > tl[col >> 3] : col + 1 < lim) ? 0.f : v.y;
        };
        tc_fence_after();
        float2 p[kCols / 2];
        // P of 16 columns, and dS of them, with the masks (few tiles have any) or without
        auto p_of = [&](auto mask, int q) {
          uint32_t x[16], w[8];
          tmem_ld16(base + C::s_at(n) + c * kCols + q * 16, x);
          tmem_ld_wait();
#pragma unroll
          for (int g4 = 0; g4 < 4; ++g4) {          // 4 columns
            const float2 y0 = fmul2(pair(x, 2 * g4), sl2), y1 = fmul2(pair(x, 2 * g4 + 1), sl2);
            float2 p0 = make_float2(ex2(y0.x), ex2(y0.y)), p1 = make_float2(ex2(y1.x), ex2(y1.y));
            if constexpr (mask.value) {
              hide(p0, q * 16 + 4 * g4);
              hide(p1, q * 16 + 4 * g4 + 2);
            }
            p[q * 8 + 2 * g4] = p0;
            p[q * 8 + 2 * g4 + 1] = p1;
            w[2 * g4] = pack_bf16(p0.x, p0.y);
            w[2 * g4 + 1] = pack_bf16(p1.x, p1.y);
          }
          // over columns that were read already
          tmem_st8(base + C::s_at(n) + c * kCols + q * 8, w);
        };
        auto ds_of = [&](auto mask, int q) {
          uint32_t x[16], w[8];
          tmem_ld16(base + C::kP + c * kCols + q * 16, x);
          tmem_ld_wait();
#pragma unroll
          for (int g4 = 0; g4 < 4; ++g4) {
            float2 d0 = fmul2(p[q * 8 + 2 * g4], pair(x, 2 * g4));
            float2 d1 = fmul2(p[q * 8 + 2 * g4 + 1], pair(x, 2 * g4 + 1));
            if constexpr (mask.value) {             // 0 even where dP is not finite
              hide(d0, q * 16 + 4 * g4);
              hide(d1, q * 16 + 4 * g4 + 2);
            }
            w[2 * g4] = pack_bf16(d0.x, d0.y);
            w[2 * g4 + 1] = pack_bf16(d1.x, d1.y);
          }
          if constexpr (SP) {
            // row r's 16-byte chunks of 8 columns, 128-byte swizzle.  The tile before has
            // been read: this tile's dP was issued behind its products
#pragma unroll
            for (int k = 0; k < 2; ++k)
              sts128(smem_u32(sDs) + tile_off(r, c * (kCols / 8) + q * 2 + k),
                     make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]));
          } else {
            tmem_st8(base + C::kP + c * kCols + q * 8, w);
          }
        };
#pragma unroll
        for (int q = 0; q < kCols / 16; ++q) {
          if (SP && q * 16 >= cols) continue;
          if (masked) p_of(std::true_type(), q);
          else p_of(std::false_type(), q);
        }
        tmem_st_wait();
        tc_fence_before();
        warp_arrive(p_full);
        ok = __all_sync(0xffffffffu, mbar_wait(&dp_full[n & 1], (uint32_t)(n >> 1) & 1, a.status,
                                               a.wait_polls));
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int q = 0; q < kCols / 16; ++q) {
          if (SP && q * 16 >= cols) continue;
          if (masked) ds_of(std::true_type(), q);
          else ds_of(std::false_type(), q);
        }
        if constexpr (SP) fence_async();
        else tmem_st_wait();
        tc_fence_before();
        warp_arrive(ds_full);
      }
      if (!ok) break;
      // ---- the unit's dV (the first half of the warpgroups) and dK, a token per thread
      // and a run of dims per warpgroup
      if (u.tiles > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(acc_full, (uint32_t)nu & 1, a.status, a.wait_polls));
        if (!ok) break;
        tc_fence_after();
      }
      constexpr int kDims = 2 * D / kNG;
      const bool is_k = c >= kNG / 2;
      const int dim0 = c % (kNG / 2) * kDims;
      const bool write = t_key < a.pos.kv_len[u.b];
      const size_t at = ((((size_t)u.b * a.s.max_blocks + u.kb) * kBlock + r) * a.s.G + u.g) * D + dim0;
      float* acc = a.acc + (is_k ? (size_t)a.s.cache_blocks() * kBlock * a.s.G * D : 0) + at;
      const float f = is_k ? a.s.scale : 1.f;
#pragma unroll 1
      for (int cc = 0; cc < kDims / 16; ++cc) {
        uint32_t x[16];
        if (u.tiles > 0) {
          tmem_ld16(base + (is_k ? C::kDK : C::kDV) + dim0 + cc * 16, x);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] = 0;
        }
        if (u.slot >= 0) {
          float* dst = a.part_kv +
                       ((((size_t)u.slot * 2 + is_k) * (D / 8) + (dim0 + cc * 16) / 8) * kBlock + r) * 8;
#pragma unroll
          for (int e = 0; e < 16; e += 8) {
            const uint32_t y[8] = {x[e], x[e + 1], x[e + 2], x[e + 3],
                                   x[e + 4], x[e + 5], x[e + 6], x[e + 7]};
            stg256(dst + e * kBlock, y);
          }
          continue;
        }
        if (!write) continue;
        if (!a.first) {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            x[e] = __float_as_uint(__uint_as_float(x[e]) + acc[cc * 16 + e]);
        }
        if (!a.last) {
#pragma unroll
          for (int e = 0; e < 16; ++e) acc[cc * 16 + e] = __uint_as_float(x[e]);
          continue;
        }
        uint4 y[2];
#pragma unroll
        for (int e = 0; e < 2; ++e)
          y[e] = make_uint4(
              pack_bf16(__uint_as_float(x[8 * e]) * f, __uint_as_float(x[8 * e + 1]) * f),
              pack_bf16(__uint_as_float(x[8 * e + 2]) * f, __uint_as_float(x[8 * e + 3]) * f),
              pack_bf16(__uint_as_float(x[8 * e + 4]) * f, __uint_as_float(x[8 * e + 5]) * f),
              pack_bf16(__uint_as_float(x[8 * e + 6]) * f, __uint_as_float(x[8 * e + 7]) * f));
        uint4* dst = reinterpret_cast<uint4*>((is_k ? a.dk : a.dv) + at + cc * 16);
        dst[0] = y[0];
        dst[1] = y[1];
      }
      if (u.tiles > 0) {
        tc_fence_before();
        warp_arrive(acc_empty);
        ++nu;
      }
    }
    if (!ok) *abort_flag = 1;
  } else if constexpr (SP) {
    // ------------------------------------------------ dQ's parts (warps 20-23)
    const int quad = warp & 3;
    const int r = quad * 32 + lane;               // row of the tile = TMEM lane
    const uint32_t base = tmem + ((uint32_t)(quad * 32) << 16) + C::dq();
    const int rshift = a.rpe == 8 ? 3 : 4;
    const int e = r >> rshift, hh = r & (a.rpe - 1);
    int it, n = 0;
    bool ok;
    while (next_unit(it, ok)) {
      const KvUnit u = kv_unit<SP>(a, it);
      for (int t = 0; t < u.tiles; ++t, ++n) {
        const bool valid = t * a.R + e < u.size && hh < a.hpg;
        ok = __all_sync(0xffffffffu, *abort_flag == 0 &&
                                         mbar_wait(dq_full, (uint32_t)n & 1, a.status, a.wait_polls));
        if (!ok) break;
        tc_fence_after();
        uint16_t* dst = a.part_dq + ((size_t)(u.first / a.R + t) * (D / 16) * kBlock + r) * 16;
#pragma unroll 1
        for (int cc = 0; cc < D / 32; ++cc) {
          uint32_t x[32];
          tmem_ld32(base + cc * 32, x);
          tmem_ld_wait();
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            uint32_t w[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
              w[k] = pack_bf16(__uint_as_float(x[16 * hf + 2 * k]),
                               __uint_as_float(x[16 * hf + 2 * k + 1]));
            if (valid) stg256(dst + (size_t)(2 * cc + hf) * kBlock * 16, w);
          }
        }
        tc_fence_before();
        warp_arrive(dq_empty);
      }
      if (!ok) break;
    }
    if (!ok) *abort_flag = 1;
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kAW) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  // no copy may still be landing when the CTA exits: the last one into each slot (not an
  // earlier one, whose phase may be two behind)
  if (threadIdx.x < C::kTiles + C::kSS) {
    const int i = threadIdx.x;
    const int last = i < C::kTiles ? max(last_fill[i], last_fill[i + C::kTiles])
                                   : last_fill[i + C::kTiles];
    if (last >= 0) mbar_wait(i < C::kTiles ? &t_full[i] : &st_full[i - C::kTiles],
                             (uint32_t)last & 1, nullptr);
  }
}

template <int D>
__global__ void __launch_bounds__(kv_threads<true>(), 1)
    bwd_sparse_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_o,
                      const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      const __grid_constant__ BwdArgs a) {
  after_previous();
  kv_cta<D, true>(tm_q, tm_o, tm_k, tm_v, a);
}

// Dense: dQ's CTAs are the last of the launch, so that they take the SMs as the KV-outer ones
// leave them (two launches, the second behind the end of the first: 4 x 2048 tokens 632 us for
// 603).  Neither kind waits for the other.
template <int D>
__global__ void __launch_bounds__(kv_threads<false>(), 1)
    bwd_dense_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_o,
                     const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const __grid_constant__ BwdArgs a) {
  static_assert(kv_threads<false>() == dq::kThreadsQ, "both kinds of CTA have the same threads");
  after_previous();
  if ((int)blockIdx.x < a.kv_ctas) kv_cta<D, false>(tm_q, tm_o, tm_k, tm_v, a);
  else dq::q_cta<D>(tm_o, tm_k, tm_v, a);
}

template <int D, bool SP>
cudaError_t launch_kv(const BwdArgs& args, const AttnBwd& t, cudaStream_t st) {
  BwdArgs a = args;
  const Shape& s = a.s;
  CUtensorMap tm_q, tm_o, tm_k, tm_v;
  if (SP) {
    // (64 dims, heads of a group, groups of all queries, 64-dim halves): one box is 8
    // heads of an entry, zeros past the group's heads
    cuuint64_t dims[4] = {64, (cuuint64_t)a.hpg, (cuuint64_t)s.B * s.T * s.G, (cuuint64_t)(D / 64)};
    cuuint64_t strides[3] = {(cuuint64_t)D * 2, (cuuint64_t)a.hpg * D * 2, 128};
    cuuint32_t box[4] = {64, 8, 1, (cuuint32_t)(D / 64)};
    if (!encode_bf16_map(&tm_q, t.q, 4, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_bf16_map(&tm_o, t.dout, 4, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
  } else {
    // (D dims, heads, queries, sequences): one box is 128 queries x 64 dims of a head,
    // zeros past the sequence's last query
    cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)s.H, (cuuint64_t)s.T, (cuuint64_t)s.B};
    cuuint64_t strides[3] = {(cuuint64_t)D * 2, (cuuint64_t)s.H * D * 2,
                             (cuuint64_t)s.T * s.H * D * 2};
    cuuint32_t box[4] = {64, 1, 128, 1};
    if (!encode_bf16_map(&tm_q, t.q, 4, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_bf16_map(&tm_o, t.dout, 4, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
  }
  cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)s.G, (cuuint64_t)(s.cache_blocks() * kBlock)};
  cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)s.G * D * 2};
  cuuint32_t box[3] = {64, 1, (cuuint32_t)kBlock};
  if (!encode_bf16_map(&tm_k, t.k, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_bf16_map(&tm_v, t.v, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  // one CTA per SM (it takes all of tensor memory, also where shared memory has room for two)
  const int ctas = sm_count();
  cudaError_t e;
  if constexpr (SP) {
    constexpr int smem = KvCfg<D, true>::kSmem;
    if ((e = cudaFuncSetAttribute(bwd_sparse_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  smem)) != cudaSuccess)
      return e;
    return launch_behind(bwd_sparse_kernel<D>, ctas, kv_threads<true>(), smem, st, tm_q, tm_o, tm_k,
                         tm_v, a);
  } else {
    constexpr int smem = KvCfg<D, false>::kSmem > dq::QCfg<D>::kSmem ? KvCfg<D, false>::kSmem
                                                                     : dq::QCfg<D>::kSmem;
    a.kv_ctas = ctas;
    const int64_t items = (int64_t)a.q_items * a.q_splits;
    const int q_ctas = (int)(items < ctas ? items : ctas);
    if ((e = cudaFuncSetAttribute(bwd_dense_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  smem)) != cudaSuccess ||
        (e = launch_behind(bwd_dense_kernel<D>, (unsigned)(ctas + q_ctas), kv_threads<false>(), smem, st,
                           tm_q, tm_o, tm_k, tm_v, a)) != cudaSuccess ||
        a.q_splits == 1)
      return e;
    return launch_behind(dq::bwd_q_join_kernel<D>,
                         (unsigned)(((int64_t)a.q_items * 128 * (D / 4) + 255) / 256), 256, 0, st, a);
  }
}

}  // namespace

cudaError_t launch_bwd_kv(const BwdArgs& a, const AttnBwd& t, cudaStream_t st) {
  if (a.sel) return a.s.D == 128 ? launch_kv<128, true>(a, t, st) : launch_kv<64, true>(a, t, st);
  return a.s.D == 128 ? launch_kv<128, false>(a, t, st) : launch_kv<64, false>(a, t, st);
}

}  // namespace msa

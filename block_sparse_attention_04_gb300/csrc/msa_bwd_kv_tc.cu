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
// two products read K-major.  For dQ's part dS^T also goes to shared memory, whose
// [token][row] order is an MN-major A operand.
//   warp 0       TMA of Q (3 stages; sparse 2) and dO (2 stages), bulk copies of the
//                rows' statistics; takes the units from a shared counter
//   warp 1       TMA of the unit's K and V
//   warp 2       tcgen05.mma
//   warps 3-10   P and dS: two warpgroups, 64 columns of a tile each; a unit's dV, dK
//   warps 11-14  sparse: dQ's parts, bf16, one row of 16 slots x D per (query, head)
// The dense order of the products is dV(n), S(n+1), dK(n), dP(n+1): dS(n) is worked out
// during the first two, P(n+1) during the last two.  Sparse, D = 128: tensor memory
// holds S, dP, dV and dK (512 columns), so dQ's part takes dP's columns until it has
// been read out, and the order is dV(n), dP(n), S(n+1), dK(n), dQ(n): the readout runs
// during dV(n+1).
#include "msa_bwd.h"
#include "msa_q8.cuh"
#include "msa_tma.h"

namespace msa {
namespace {

constexpr int kMmaW = 2, kSoftW = 3, kOutW = 11;
template <bool SP>
constexpr int kv_threads() { return 32 * (SP ? 15 : 11); }
constexpr int kRing = 4;                  // unit numbers published by warp 0, ahead of use
template <bool SP>
constexpr int ring_readers() { return 2 + 8 + (SP ? 4 : 0); }

template <int D, bool SP>
struct KvCfg {
  static constexpr int kNHalf = D / 64;
  static constexpr int kHalf = 128 * 128;            // 128 rows x 64 dims
  static constexpr int kTile = kNHalf * kHalf;       // K, V, a Q or a dO tile
  static constexpr int kQS = SP ? 2 : 3, kOS = 2;    // stages of Q and dO
  static constexpr int kSS = 2;                      // ... of the statistics: with Q (sparse), dO
  static constexpr int kStat = 16 * kStatBytes;      // statistics of a tile
  static constexpr int kDs = SP ? 2 * kHalf : 0;     // dS^T [2 x 64 rows][128 tokens]
  static constexpr int kSmem =
      2 * kTile + (kQS + kOS) * kTile + kDs + kSS * (kStat + 80) + 256;
  // byte offsets of a tile of rows: sparse tiles hold 8-row groups, half after half
  static constexpr int kGroup = SP ? kNHalf * 1024 : 1024;   // next 8 rows
  static constexpr int kNext = SP ? 1024 : kHalf;            // next 64 dims
  // tensor memory columns: S, dP, dV, dK, dQ's part (D = 128: in dP's place)
  static constexpr uint32_t kS = 0, kP = 128, kDV = 256, kDK = 256 + D;
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

template <int D, bool SP>
__global__ void __launch_bounds__(kv_threads<SP>(), 1)
    bwd_kv_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_o,
                  const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                  const __grid_constant__ BwdArgs a) {
  using C = KvCfg<D, SP>;
  extern __shared__ __align__(1024) uint8_t smem[];   // the swizzled tiles' alignment
  uint8_t* sK = smem;
  uint8_t* sV = sK + C::kTile;
  uint8_t* sQ = sV + C::kTile;                     // [kQS]
  uint8_t* sO = sQ + C::kQS * C::kTile;            // [kOS]
  uint8_t* sDs = sO + C::kOS * C::kTile;
  uint8_t* sStat = sDs + C::kDs;                   // [kSS] statistics
  // [kSS] per 8-row group of a sparse tile: the last token of the block that its query
  // sees (-1: none), then whether any of them is below 127
  int* sLim = reinterpret_cast<int*>(sStat + C::kSS * C::kStat);
  uint64_t* q_full = reinterpret_cast<uint64_t*>(sLim + C::kSS * 20);
  uint64_t* q_empty = q_full + C::kQS;
  uint64_t* o_full = q_empty + C::kQS;
  uint64_t* o_empty = o_full + C::kOS;
  uint64_t* kv_full = o_empty + C::kOS;            // K and V of the unit landed
  uint64_t* kv_empty = kv_full + 1;                // its last product that reads them is done
  uint64_t* s_full = kv_empty + 1;                 // S of the tile is in tensor memory
  uint64_t* dp_full = s_full + 1;                  // dP of the tile
  uint64_t* p_full = dp_full + 1;                  // P written over S
  uint64_t* ds_full = p_full + 1;                  // dS written over dP (and to shared memory)
  uint64_t* acc_full = ds_full + 1;                // the unit's dV and dK are complete
  uint64_t* acc_empty = acc_full + 1;              // ... and read out
  uint64_t* dq_full = acc_empty + 1;               // sparse: dQ's part is in tensor memory
  uint64_t* dq_empty = dq_full + 1;                // ... and read out
  uint64_t* bar_fin = dq_empty + 1;
  uint64_t* it_full = bar_fin + 1;                 // [kRing]
  uint64_t* it_empty = it_full + kRing;
  int* ring = reinterpret_cast<int*>(it_empty + kRing);   // unit numbers, -1: no more
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ring + kRing);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kQS; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
    }
    for (int i = 0; i < C::kOS; ++i) {
      mbar_init(&o_full[i], 1);
      mbar_init(&o_empty[i], 1);
    }
    mbar_init(kv_full, 1);
    mbar_init(kv_empty, 1);
    mbar_init(s_full, 1);
    mbar_init(dp_full, 1);
    mbar_init(p_full, 256);
    mbar_init(ds_full, 256);
    mbar_init(acc_full, 1);
    mbar_init(acc_empty, 256);
    mbar_init(dq_full, 1);
    mbar_init(dq_empty, 128);
    mbar_init(bar_fin, 1);
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&it_full[i], 1);
      mbar_init(&it_empty[i], ring_readers<SP>());
    }
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_o);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == kMmaW) tmem_alloc(tmem_slot, 512);
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

  if (warp == 0) {
    // ------------------------------------------------ Q, dO, statistics (warp 0)
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
    int n = 0;                     // tiles begun (Q and statistics issued)
    int no = 0;                    // dO tiles issued
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
      for (int t = 0; t < u.tiles; ++t, ++n, ++no) {
        if (__any_sync(0xffffffffu, *abort_flag != 0)) { ok = false; break; }
        const int qs = n % C::kQS, os = no % C::kOS;
        const uint32_t qw = (uint32_t)(n / C::kQS), ow = (uint32_t)(no / C::kOS);
        if constexpr (SP) {
          const int boxes = 2 * sparse_steps(a, u, t);     // 8-row groups of the tile
          const int bpe = a.rpe >> 3, e = (lane & 15) / bpe;
          const int at = t * a.R + e;
          const bool real = at < u.size;
          int il = 0;
          if (real) il = a.entries[u.first + at] >> 4;
          const int64_t row = (int64_t)u.b * T + a.t0 + il;
          // past the end for rows without an entry: zeros
          const int z = real ? (int)(row * a.s.G + u.g) : a.s.B * T * a.s.G;
          const int box_r = (lane & 15) % bpe * 8;
          // a block that the sequence's last query does not reach the end of may hold
          // anything behind it: rows without an entry see none of it
          const int64_t seen = (int64_t)a.pos.q_start[u.b] + a.t0 + il - (int64_t)u.kb * kBlock;
          const int lim = real ? (int)(seen < 127 ? seen : 127)
                               : (t_last - (int64_t)u.kb * kBlock < 127 ? -1 : 127);
          const bool any = __any_sync(0xffffffffu, (lane & 15) < boxes && lim < 127);
          if (!wait_all(&q_empty[qs], (qw & 1) ^ 1)) { ok = false; break; }
          if (lane < 16) sLim[qs * 20 + lane] = lim;
          if (lane == 16) sLim[qs * 20 + 16] = any;
          __syncwarp();
          if (lane == 0)
            mbar_arrive_expect_tx(&q_full[qs], (uint32_t)(boxes * (C::kGroup + kStatBytes)));
          __syncwarp();
          if (lane < boxes) {
            tma_load_4d_hint(smem_u32(sQ + qs * C::kTile + lane * C::kGroup), &tm_q, &q_full[qs], 0,
                             box_r, z, 0, pol);
            const size_t sg = real ? (size_t)(row * a.s.G + u.g) * bpe + lane % bpe : a.stat_groups;
            bulk_load(smem_u32(sStat + qs * C::kStat + lane * kStatBytes), a.stat + sg * kStatBytes,
                      kStatBytes, &q_full[qs]);
          }
          if (!wait_all(&o_empty[os], (ow & 1) ^ 1)) {
            ok = false;
            ++n;                   // Q of this tile is on its way, its dO is not
            break;
          }
          if (lane == 0) mbar_arrive_expect_tx(&o_full[os], (uint32_t)(boxes * C::kGroup));
          __syncwarp();
          if (lane < boxes)
            tma_load_4d_hint(smem_u32(sO + os * C::kTile + lane * C::kGroup), &tm_o, &o_full[os], 0,
                             box_r, z, 0, pol);
        } else {
          int h, qt;
          dense_tile(a, u, q0, t, h, qt);
          h += u.g * a.hpg;
          if (!wait_all(&q_empty[qs], (qw & 1) ^ 1)) { ok = false; break; }
          if (lane == 0) {
            mbar_arrive_expect_tx(&q_full[qs], C::kTile);
#pragma unroll
            for (int hf = 0; hf < C::kNHalf; ++hf)
              tma_load_4d_hint(smem_u32(sQ + qs * C::kTile + hf * C::kHalf), &tm_q, &q_full[qs],
                               hf * 64, h, qt * 128, u.b, pol);
          }
          __syncwarp();
          if (!wait_all(&o_empty[os], (ow & 1) ^ 1)) {
            ok = false;
            ++n;
            break;
          }
          if (lane == 0) {
            mbar_arrive_expect_tx(&o_full[os], C::kTile + C::kStat);
            bulk_load(smem_u32(sStat + os * C::kStat),
                      a.stat + ((size_t)(u.b * H + h) * a.stat_groups + qt * 16) * kStatBytes,
                      C::kStat, &o_full[os]);
#pragma unroll
            for (int hf = 0; hf < C::kNHalf; ++hf)
              tma_load_4d_hint(smem_u32(sO + os * C::kTile + hf * C::kHalf), &tm_o, &o_full[os],
                               hf * 64, h, qt * 128, u.b, pol);
          }
          __syncwarp();
        }
      }
      cur = nx;
    }
    if (!ok && lane == 0) *abort_flag = 1;
    // no copy may still be landing when the CTA exits: the last load of each stage
    if (lane == 0) {
      for (int m = n - 1; m >= 0 && m >= n - C::kQS; --m)
        mbar_wait(&q_full[m % C::kQS], (uint32_t)(m / C::kQS) & 1, nullptr);
      for (int m = no - 1; m >= 0 && m >= no - C::kOS; --m)
        mbar_wait(&o_full[m % C::kOS], (uint32_t)(m / C::kOS) & 1, nullptr);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------ K and V (warp 1)
    int it, n = 0;
    bool ok;
    while (next_unit(it, ok)) {
      const KvUnit u = kv_unit<SP>(a, it);
      if (u.tiles == 0) continue;
      if (n > 0 && !wait_all(kv_empty, (uint32_t)(n - 1) & 1)) { ok = false; break; }
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
      ++n;
    }
    if (!ok && lane == 0) *abort_flag = 1;
    if (n > 0) mbar_wait(kv_full, (uint32_t)(n - 1) & 1, nullptr);
  } else if (warp == kMmaW) {
    // ---------------------------------------------------------- MMA (warp 2)
    constexpr uint32_t idesc_n = idesc_bf16(128, D, false, true);     // dV, dK
    constexpr uint32_t idesc_q = idesc_bf16(128, D, true, true);      // dQ's part
    const uint64_t kd = smem_desc(smem_u32(sK), 16, 1024, kSwizzle128B);
    const uint64_t vd = smem_desc(smem_u32(sV), 16, 1024, kSwizzle128B);
    const uint64_t kmn = smem_desc(smem_u32(sK), C::kHalf, 1024, kSwizzle128B);
    const uint64_t dsmn = smem_desc(smem_u32(sDs), C::kHalf, 1024, kSwizzle128B);
    const uint64_t qk = smem_desc(smem_u32(sQ), 16, C::kGroup, kSwizzle128B);
    const uint64_t ok_ = smem_desc(smem_u32(sO), 16, C::kGroup, kSwizzle128B);
    const uint64_t qmn = smem_desc(smem_u32(sQ), C::kNext, C::kGroup, kSwizzle128B);
    const uint64_t omn = smem_desc(smem_u32(sO), C::kNext, C::kGroup, kSwizzle128B);
    // A (128 x D, K-major) times a tile of rows, K-major: `steps` x 16 columns
    auto rows_product = [&](uint32_t d, uint64_t ad, uint64_t bd, int steps) {
      const uint32_t idesc = idesc_bf16(128, 0, false, false) | (uint32_t)(2 * steps) << 17;
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
        tc_mma_f16(tmem + d, ad + (uint64_t)(((j >> 2) * C::kHalf + (j & 3) * 32) >> 4),
                   bd + (uint64_t)(((j >> 2) * C::kNext + (j & 3) * 32) >> 4), idesc, j > 0 ? 1u : 0u);
    };
    // P^T or dS^T (TMEM at column p, 64 columns of a tile in 32) times a tile of rows
    auto sum_product = [&](uint32_t d, uint32_t p, uint64_t bd, int steps, bool add) {
      for (int j = 0; j < steps; ++j)
        tc_mma_f16_ts(tmem + d, tmem + p + (j >> 2) * 64 + (j & 3) * 8,
                      bd + (uint64_t)((j * 2 * C::kGroup) >> 4), idesc_n, add || j > 0 ? 1u : 0u);
    };
    int it, n = 0, nu = 0;       // tiles and units (with tiles) so far
    bool ok;
    while (next_unit(it, ok)) {
      const KvUnit u = kv_unit<SP>(a, it);
      if (u.tiles == 0) continue;
      ok = wait_all(kv_full, (uint32_t)nu & 1);
      if (!ok) break;
      const int64_t left = (int64_t)a.pos.q_start[u.b] + T - 1 - (int64_t)u.kb * kBlock;
      if (SP && left < kBlock - 1) {
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
      auto issue_s = [&](int m, int t) {           // S of tile m, the unit's t-th
        const int qs = m % C::kQS;
        if (!wait_all(&q_full[qs], (uint32_t)(m / C::kQS) & 1)) return false;
        tc_fence_after();
        const int steps = SP ? sparse_steps(a, u, t) : 8;
        if (elect_one()) {
          rows_product(C::kS, kd, qk + (uint64_t)((qs * C::kTile) >> 4), steps);
          tc_commit(s_full);
        }
        __syncwarp();
        return true;
      };
      auto issue_dp = [&](int m, int t, bool release) {
        const int os = m % C::kOS;
        if (!wait_all(&o_full[os], (uint32_t)(m / C::kOS) & 1)) return false;
        tc_fence_after();
        const int steps = SP ? sparse_steps(a, u, t) : 8;
        if (elect_one()) {
          rows_product(C::kP, vd, ok_ + (uint64_t)((os * C::kTile) >> 4), steps);
          tc_commit(dp_full);
          if (release) tc_commit(SP ? &o_empty[os] : kv_empty);
        }
        __syncwarp();
        return true;
      };
      ok = issue_s(n, 0) && (SP || issue_dp(n, 0, u.tiles == 1));
      for (int t = 0; t < u.tiles && ok; ++t, ++n) {
        const int steps = SP ? sparse_steps(a, u, t) : 8;
        const int qs = n % C::kQS, os = n % C::kOS;
        const bool more = t + 1 < u.tiles;
        // ---- dV += P^T dO
        ok = wait_all(p_full, (uint32_t)n & 1) &&
             (t > 0 || nu == 0 || wait_all(acc_empty, (uint32_t)(nu - 1) & 1)) &&
             (!SP || wait_all(&o_full[os], (uint32_t)(n / C::kOS) & 1));
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          sum_product(C::kDV, C::kS, omn + (uint64_t)((os * C::kTile) >> 4), steps, t > 0);
        }
        __syncwarp();
        if constexpr (SP) {
          if (D == 128 && n > 0) ok = wait_all(dq_empty, (uint32_t)(n - 1) & 1);
          ok = ok && issue_dp(n, t, true);
        }
        if (ok && more) ok = issue_s(n + 1, t + 1);
        // ---- dK += dS^T Q
        ok = ok && wait_all(ds_full, (uint32_t)n & 1);
        if (SP && D != 128 && ok && n > 0) ok = wait_all(dq_empty, (uint32_t)(n - 1) & 1);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          sum_product(C::kDK, C::kP, qmn + (uint64_t)((qs * C::kTile) >> 4), steps, t > 0);
          tc_commit(&q_empty[qs]);
          if (!SP) tc_commit(&o_empty[os]);    // with the statistics, which dS has used
          if constexpr (SP) {
            // ---- dQ part = dS K: 128 tokens in 8 steps
#pragma unroll
            for (int j = 0; j < 8; ++j)
              tc_mma_f16(tmem + C::dq(), dsmn + (uint64_t)((j * 2048) >> 4),
                         kmn + (uint64_t)((j * 2048) >> 4), idesc_q, j > 0 ? 1u : 0u);
            tc_commit(dq_full);
            if (!more) tc_commit(kv_empty);
          }
          if (!more) tc_commit(acc_full);
        }
        __syncwarp();
        if (!SP && more) ok = issue_dp(n + 1, t + 1, t + 2 == u.tiles);
      }
      if (!ok) break;
      ++nu;
    }
    if (!ok && lane == 0) *abort_flag = 1;
    // all MMAs done before tensor memory is released
    if (elect_one()) tc_commit(bar_fin);
    __syncwarp();
    mbar_wait(bar_fin, 0, nullptr);
  } else if (warp < kOutW) {
    // ------------------------------------------ P, dS; dV and dK (warps 3-10)
    const int c = (warp - kSoftW) >> 2;           // columns 64 c .. 64 c + 63; dV or dK
    const int quad = warp & 3;
    const int r = quad * 32 + lane;               // token of the block = TMEM lane
    const uint32_t base = tmem + ((uint32_t)(quad * 32) << 16);
    const float sl = a.s.scale * kLog2e;
    const float2 sl2 = make_float2(sl, sl);
    int it, n = 0, nu = 0;
    bool ok;
    while (next_unit(it, ok)) {
      const KvUnit u = kv_unit<SP>(a, it);
      const int q0 = SP ? 0 : bwd_first_tile(a, u.b, u.kb);
      const int64_t t_key = (int64_t)u.kb * kBlock + r;
      const bool used = t_key <= (int64_t)a.pos.q_start[u.b] + T - 1;  // by the last query
      for (int t = 0; t < u.tiles; ++t, ++n) {
        const int ss = n % C::kSS;
        int cols = 64;                            // of this warpgroup's 64 that the tile has
        int lim = 0;                              // dense: columns below see another token
        bool masked;
        ok = *abort_flag == 0 &&
             mbar_wait(SP ? &q_full[ss] : &o_full[ss], (uint32_t)(n / C::kSS) & 1, a.status,
                       a.wait_polls) &&
             mbar_wait(s_full, (uint32_t)n & 1, a.status, a.wait_polls);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const int* tl = sLim + ss * 20 + c * 8;
        if constexpr (SP) {
          cols = min(64, max(0, sparse_steps(a, u, t) * 16 - c * 64));
          masked = sLim[ss * 20 + 16] != 0;
        } else {
          int h, qt;
          dense_tile(a, u, q0, t, h, qt);
          const int64_t d = t_key - ((int64_t)a.pos.q_start[u.b] + qt * 128);
          lim = used ? (int)(d > 0 ? d : 0) - c * 64 : 64;
          masked = __any_sync(0xffffffffu, lim > 0);
        }
        // column 32 hf + e of this warpgroup is seen by token r
        auto hidden = [&](int col) { return SP ? r > tl[col >> 3] : col < lim; };
        tc_fence_after();
        // statistics of 8 columns: 64 bytes, -lse log2e then -delta
        const float4* st = reinterpret_cast<const float4*>(sStat + ss * C::kStat + c * 8 * kStatBytes);
        float2 p[32];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          if (hf * 32 >= cols) continue;
          uint32_t x[32];
          tmem_ld32(base + C::kS + c * 64 + hf * 32, x);
          tmem_ld_wait();
          uint32_t w[16];
#pragma unroll
          for (int g4 = 0; g4 < 8; ++g4) {        // 4 columns
            const float4 nl = st[(hf * 4 + (g4 >> 1)) * 4 + (g4 & 1)];
            const float2 y0 = ffma2(make_float2(__uint_as_float(x[4 * g4]), __uint_as_float(x[4 * g4 + 1])),
                                    sl2, make_float2(nl.x, nl.y));
            const float2 y1 = ffma2(make_float2(__uint_as_float(x[4 * g4 + 2]), __uint_as_float(x[4 * g4 + 3])),
                                    sl2, make_float2(nl.z, nl.w));
            float2 p0 = make_float2(ex2(y0.x), ex2(y0.y)), p1 = make_float2(ex2(y1.x), ex2(y1.y));
            if (masked) {
              const int col = hf * 32 + 4 * g4;
              p0.x = hidden(col) ? 0.f : p0.x;
              p0.y = hidden(col + 1) ? 0.f : p0.y;
              p1.x = hidden(col + 2) ? 0.f : p1.x;
              p1.y = hidden(col + 3) ? 0.f : p1.y;
            }
            p[hf * 16 + 2 * g4] = p0;
            p[hf * 16 + 2 * g4 + 1] = p1;
            w[2 * g4] = pack_bf16(p0.x, p0.y);
            w[2 * g4 + 1] = pack_bf16(p1.x, p1.y);
          }
          // over columns that were read already
          tmem_st16(base + C::kS + c * 64 + hf * 16, w);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(p_full);
        ok = __all_sync(0xffffffffu, mbar_wait(dp_full, (uint32_t)n & 1, a.status, a.wait_polls));
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          if (hf * 32 >= cols) continue;
          uint32_t x[32];
          tmem_ld32(base + C::kP + c * 64 + hf * 32, x);
          tmem_ld_wait();
          uint32_t w[16];
#pragma unroll
          for (int g4 = 0; g4 < 8; ++g4) {
            const float4 nd = st[(hf * 4 + (g4 >> 1)) * 4 + 2 + (g4 & 1)];
            float2 d0 = fadd2(make_float2(__uint_as_float(x[4 * g4]), __uint_as_float(x[4 * g4 + 1])),
                              make_float2(nd.x, nd.y));
            float2 d1 = fadd2(make_float2(__uint_as_float(x[4 * g4 + 2]), __uint_as_float(x[4 * g4 + 3])),
                              make_float2(nd.z, nd.w));
            const float2 p0 = p[hf * 16 + 2 * g4], p1 = p[hf * 16 + 2 * g4 + 1];
            d0 = fmul2(p0, d0);
            d1 = fmul2(p1, d1);
            if (masked) {      // 0 even where dP is not finite
              const int col = hf * 32 + 4 * g4;
              d0.x = hidden(col) ? 0.f : d0.x;
              d0.y = hidden(col + 1) ? 0.f : d0.y;
              d1.x = hidden(col + 2) ? 0.f : d1.x;
              d1.y = hidden(col + 3) ? 0.f : d1.y;
            }
            w[2 * g4] = pack_bf16(d0.x, d0.y);
            w[2 * g4 + 1] = pack_bf16(d1.x, d1.y);
          }
          tmem_st16(base + C::kP + c * 64 + hf * 16, w);
          if constexpr (SP) {
            // [64 c + ..] of row r: four 16-byte chunks, 128-byte swizzle.  dQ's part of
            // the tile before has read the buffer: its products precede this tile's dP
#pragma unroll
            for (int k = 0; k < 4; ++k)
              sts128(smem_u32(sDs) + tile_off(r, c * 8 + hf * 4 + k),
                     make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]));
          }
        }
        tmem_st_wait();
        if constexpr (SP) fence_async();
        tc_fence_before();
        mbar_arrive(ds_full);
      }
      if (!ok) break;
      // ---- the unit's dV (c = 0) or dK (c = 1), a token per thread
      if (u.tiles > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(acc_full, (uint32_t)nu & 1, a.status, a.wait_polls));
        if (!ok) break;
        tc_fence_after();
      }
      const bool write = t_key < a.pos.kv_len[u.b];
      const size_t at = ((((size_t)u.b * a.s.max_blocks + u.kb) * kBlock + r) * a.s.G + u.g) * D;
      float* acc = a.acc + (c ? (size_t)a.s.cache_blocks() * kBlock * a.s.G * D : 0) + at;
      const float f = c ? a.s.scale : 1.f;
#pragma unroll 1
      for (int cc = 0; cc < D / 16; ++cc) {
        uint32_t x[16];
        if (u.tiles > 0) {
          tmem_ld16(base + (c ? C::kDK : C::kDV) + cc * 16, x);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] = 0;
        }
        if (u.slot >= 0) {
          float* dst = a.part_kv + (((size_t)u.slot * 2 + c) * kBlock + r) * D + cc * 16;
#pragma unroll
          for (int e = 0; e < 16; e += 8) {
            const uint32_t y[8] = {x[e], x[e + 1], x[e + 2], x[e + 3],
                                   x[e + 4], x[e + 5], x[e + 6], x[e + 7]};
            stg256(dst + e, y);
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
        uint4* dst = reinterpret_cast<uint4*>((c ? a.dk : a.dv) + at + cc * 16);
        dst[0] = y[0];
        dst[1] = y[1];
      }
      if (u.tiles > 0) {
        tc_fence_before();
        mbar_arrive(acc_empty);
        ++nu;
      }
    }
    if (!ok) *abort_flag = 1;
  } else if constexpr (SP) {
    // ------------------------------------------------ dQ's parts (warps 11-14)
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
        const int at = t * a.R + e;
        const bool valid = at < u.size && hh < a.hpg;
        int own = -1;
        if (valid) {
          const int en = a.entries[u.first + at];
          own = (int)((((int64_t)u.b * a.Tp + (en >> 4)) * H + u.g * a.hpg + hh) * kTopk + (en & 15));
        }
        ok = __all_sync(0xffffffffu, *abort_flag == 0 &&
                                         mbar_wait(dq_full, (uint32_t)n & 1, a.status, a.wait_polls));
        if (!ok) break;
        tc_fence_after();
        // 32 bytes of two rows per lane become 64 bytes of a row over two lanes: a store
        // then touches 16 lines, and 32-byte stores take half as many
        const bool up = lane & 1;
        int to[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) to[j] = __shfl_sync(0xffffffffu, own, (lane & ~1) + j);
#pragma unroll 1
        for (int cc = 0; cc < D / 32; ++cc) {
          uint32_t x[32], w[2][8];
          tmem_ld32(base + cc * 32, x);
          tmem_ld_wait();
#pragma unroll
          for (int hf = 0; hf < 2; ++hf)
#pragma unroll
            for (int k = 0; k < 8; ++k)
              w[hf][k] = pack_bf16(__uint_as_float(x[hf * 16 + 2 * k]),
                                   __uint_as_float(x[hf * 16 + 2 * k + 1]));
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? w[0][k] : w[1][k], 1);
            w[0][k] = up ? got : w[0][k];
            w[1][k] = up ? w[1][k] : got;
          }
#pragma unroll
          for (int j = 0; j < 2; ++j)
            if (to[j] >= 0) stg256(a.part_dq + (size_t)to[j] * D + cc * 32 + up * 16, w[j]);
        }
        tc_fence_before();
        mbar_arrive(dq_empty);
      }
      if (!ok) break;
    }
    if (!ok) *abort_flag = 1;
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaW) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool SP>
cudaError_t launch_kv(const BwdArgs& a, const AttnBwd& t, cudaStream_t st) {
  using C = KvCfg<D, SP>;
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
  cudaError_t e = cudaFuncSetAttribute(bwd_kv_kernel<D, SP>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  // one CTA per SM (it takes all of tensor memory, also where shared memory has room for two)
  note_launches(1);
  bwd_kv_kernel<D, SP><<<sm_count(), kv_threads<SP>(), C::kSmem, st>>>(tm_q, tm_o, tm_k, tm_v, a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_bwd_kv(const BwdArgs& a, const AttnBwd& t, cudaStream_t st) {
  if (a.sel) return a.s.D == 128 ? launch_kv<128, true>(a, t, st) : launch_kv<64, true>(a, t, st);
  return a.s.D == 128 ? launch_kv<128, false>(a, t, st) : launch_kv<64, false>(a, t, st);
}

}  // namespace msa

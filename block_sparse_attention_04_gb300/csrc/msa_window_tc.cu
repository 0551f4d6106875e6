// Sliding-window attention on tensor cores (msa_window_attn and
// msa_window_attn_q8 for prefill shapes): query t sees the tokens j <= t with
// j > t - window or j < sinks, on a bf16 or an 8-bit block-major cache.
//
// The rows of a tile are (query, head) pairs of one KV group: nq = 128 / (H/G)
// consecutive queries x H/G heads, so that even a few queries fill a tile.  A
// work item is two such tiles (2 nq queries of one sequence and group), run as
// two chains over the blocks that hold a token some query of the item sees
// (the sink blocks, then the window's); both chains read the same K and V
// block from shared memory.  S = Q K^T and O += P V on tcgen05; O stays in
// tensor memory across the blocks under an online softmax that rescales it
// only when a row's maximum grows by more than 2^8.  Per block and item:
// 2 x 2 x 128 x 128 x D multiply-adds against 2 x 128 x D cached values, i.e.
// bound by the tensor cores and, next to them, by the exponentials.
//   warp 0        takes items from a shared counter; TMA of the Q tiles
//   warp 1        bf16 cache: TMA of K and V blocks, 2-deep rings
//   warp 2        tcgen05.mma, per block n: P.V(c0, n-1), S(c0, n), P.V(c1, n-1),
//                 S(c1, n), also across items (each chain's Q tile is reloaded
//                 when its last S is done, so the next item's first S follows
//                 the last P.V); S and P share TMEM columns [128c, 128c + 128),
//                 O is at [256 + 128c, ...).  Rows of V that no query of the item
//                 sees (they may hold anything) are zeroed before their first
//                 use: a weight of 0 does not cancel a NaN.
//   warps 3-10    one warpgroup per chain, a row per thread: mask, maximum,
//                 P = 2^(x - m) over S, row sum; at the item's end O / l, written
//                 64 bytes of a row at a time by two lanes (16 bytes of 32 rows per
//                 store, as the rows lie in tensor memory, cost 4 % of the call;
//                 through shared memory the rows took 1 % more)
//   warps 11-14   8-bit cache, in place of warp 1: codes of the next block to
//                 registers, converted into the same rings: K to f16 and V to
//                 bf16 (both exact); Q tiles to f16 in place, each row scaled by
//                 a power of two to [2^13, 2^14) (exact but for elements 2^-27
//                 below the row's maximum).  f16 takes a third of the
//                 conversion's instructions; V needs bf16's range, because P
//                 (bf16, 2^-8) is relative to the largest p', which may belong
//                 to values that cancel or vanish.
// When the items are fewer than the SMs, each block list is split over several
// items, whose O, maxima and sums go to the workspace and are joined by
// window_join_kernel (64 queries of one sequence at 16K tokens, window 8000,
// 48/8 heads: 116 us in one part, 36 us).
// An 8-bit block's exponents: 2^ek scales the scores, 2^ev is folded into the
// exponential that multiplies V (p' = 2^(x + ev - m), m the maximum of x + ev),
// while the normaliser counts 2^(x - n) with its own maximum n.  p' gives the
// latter by one factor per row and block, 2^(m - ev - n), unless that factor is
// so large that p' may have vanished (blocks whose scale is 2^80 below the
// others', such as blocks of zeros): then it is summed by exponentials of its own.
//
// Measured (us; the MMAs' time at cuBLAS' burst rate beside it): 16K queries, 48/8
// heads, D 128, window 4096 and 64 sinks 1094 to 1141 on different machines (764 for
// the visible tokens), 8-bit cache 1449; 3 x 1000 queries, 64/4, D 64, window 1000,
// 8-bit cache 114 to 117 (26), bf16 98 to 100.  A block
// step of the two chains takes 1.5 us at D 64, 1.66 at D 128 (of which the MMAs
// 1.34), with an 8-bit cache 1.76 and 2.13: the chain S, maximum, P, P.V has few
// steps to overlap with, and power is at its limit.  An item costs 3-4 us beyond
// its steps: masked blocks, output, the first S.
#include "msa_q8.cuh"
#include "msa_serve.h"
#include "msa_tma.h"

namespace msa {
namespace {

constexpr int kQWarp = 0, kKVWarp = 1, kMmaWarp = 2, kSoftWarp0 = 3, kConvWarp0 = 11;
constexpr int kConv = 128;            // converter threads (8-bit cache)
constexpr int kStages = 2;            // K and V blocks in flight
constexpr float kLazy = 8.f;          // log2 growth of P tolerated before O is rescaled
constexpr float kFoldMax = 80.f;      // log2 of the largest factor from p' to the normaliser
constexpr int kItemRing = 4;          // item ids published by the Q warp, ahead of use
constexpr int kSplitItems = 152;      // most parts of split calls (an SM each)
constexpr int kMetaRing = 4;          // exponents of the blocks in flight

template <bool Q8>
constexpr int threads() { return 32 * (Q8 ? 15 : 11); }
// readers of a published item: the MMA warp, 8 softmax warps, and the K/V
// lane or the 4 converter warps
template <bool Q8>
constexpr int readers() { return Q8 ? 13 : 10; }

struct WinArgs {
  Shape s;
  Positions pos;
  int window, sinks;
  int nq;          // queries per tile: 128 / (H/G)
  int npair;       // items per (sequence, group): ceil(T / (2 nq))
  int splits;      // items that share a block list
  int nitems;      // npair * B * G * splits
  float* part_o;   // splits > 1: [item][chain][128][D] O relative to m
  float4* part_ml; // ... (m, n in log2 units, l)
  int* next_item;  // shared counter of taken items (zeroed with the status word)
  const uint8_t* k8;
  const uint8_t* v8;
  const int8_t* k_exp;
  const int8_t* v_exp;
  uint16_t* out;
  int* status;
  uint32_t wait_polls;
};

template <int D>
struct WinCfg {
  static constexpr int kNHalf = D / 64;
  static constexpr int kHalf = 128 * 128;       // 128 rows x 64 dims of 16 bits (16 KiB)
  static constexpr int kTile = kNHalf * kHalf;  // a Q tile, a K or a V block
  static constexpr int kSmem = 2 * kTile + 2 * kStages * kTile + 2048 + 512 + 1024;
  static constexpr uint32_t kTmemCols = 512;
};

// Item it: later query tiles first (their windows are the fuller ones).
struct Item {
  int b, g, i0;          // queries i0 ... i0 + 2 nq - 1 of sequence b (those below T)
  int t_first, t_last;   // their first and last position
  int lo;                // first token of the first query's window
  int p0, nblk;          // the item's blocks: list positions p0 ... p0 + nblk - 1
  int nsink, first;      // block p of the list is p (p < nsink) or first + p
};
__device__ __forceinline__ Item item_of(const WinArgs& a, int it) {
  Item d;
  const int per = a.s.B * a.s.G, split = it % a.splits;
  it /= a.splits;
  const int pair = a.npair - 1 - it / per, r = it % per;
  d.g = r % a.s.G;
  d.b = r / a.s.G;
  d.i0 = pair * 2 * a.nq;
  d.t_first = a.pos.q_start[d.b] + d.i0;
  d.t_last = a.pos.q_start[d.b] + min(a.s.T - 1, d.i0 + 2 * a.nq - 1);
  d.lo = max(0, d.t_first - a.window + 1);
  d.nsink = min((a.sinks + kBlock - 1) / kBlock, d.lo / kBlock);
  d.first = d.lo / kBlock - d.nsink;
  const int len = d.nsink + d.t_last / kBlock - d.lo / kBlock + 1;
  d.p0 = split * len / a.splits;
  d.nblk = (split + 1) * len / a.splits - d.p0;    // 0: a list shorter than the splits
  return d;
}
__device__ __forceinline__ int block_at(const Item& d, int p) {
  p += d.p0;
  return p < d.nsink ? p : d.first + p;
}

// Bits [0, n) of word w of a 128-bit mask.
__device__ __forceinline__ uint32_t below(int n, int w) {
  const int k = n - 32 * w;
  return k <= 0 ? 0u : k >= 32 ? 0xFFFFFFFFu : (1u << k) - 1u;
}

template <int D, bool Q8>
__global__ void __launch_bounds__(threads<Q8>(), 1)
    window_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ WinArgs a) {
  using C = WinCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* sQ = smem;                         // [chain] Q tiles
  uint8_t* sK = sQ + 2 * C::kTile;            // [kStages] K blocks
  uint8_t* sV = sK + kStages * C::kTile;      // [kStages] V blocks
  float* q_scale = reinterpret_cast<float*>(sV + kStages * C::kTile);   // [2][chain][128]
  uint64_t* bars = reinterpret_cast<uint64_t*>(q_scale + 2 * 2 * 128);
  uint64_t* q_full = bars;                    // per chain: the item's Q tile landed
  uint64_t* q_ready = q_full + 2;             // ... and is in f16 (8-bit cache)
  uint64_t* q_empty = q_ready + 2;            // per chain: the item's last S is done
  uint64_t* k_full = q_empty + 2;             // kStages
  uint64_t* k_empty = k_full + kStages;
  uint64_t* v_full = k_empty + kStages;
  uint64_t* v_empty = v_full + kStages;
  uint64_t* s_full = v_empty + kStages;       // per chain: S of the block is in TMEM
  uint64_t* p_full = s_full + 2;              // per chain: P written over S (O rescaled)
  uint64_t* o_full = p_full + 2;              // per chain: the item's last P.V is done
  uint64_t* bar_fin = o_full + 2;
  uint64_t* it_full = bar_fin + 1;            // kItemRing: an item id is published
  uint64_t* it_empty = it_full + kItemRing;   // kItemRing: every reader has it
  int* item_ring = reinterpret_cast<int*>(it_empty + kItemRing);  // ids, -1: no more
  int2* meta = reinterpret_cast<int2*>(item_ring + kItemRing);    // kMetaRing: (ek, ev)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(meta + kMetaRing);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int T = a.s.T, H = a.s.H, hpg = H / a.s.G, nq = a.nq;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&k_full[i], Q8 ? kConv : 1);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], Q8 ? kConv : 1);
      mbar_init(&v_empty[i], 1);
    }
    for (int c = 0; c < 2; ++c) {
      mbar_init(&q_full[c], 1);
      mbar_init(&q_ready[c], kConv);
      mbar_init(&q_empty[c], 1);
      mbar_init(&s_full[c], 1);
      mbar_init(&p_full[c], 128);
      mbar_init(&o_full[c], 1);
    }
    mbar_init(bar_fin, 1);
    for (int i = 0; i < kItemRing; ++i) {
      mbar_init(&it_full[i], 1);
      mbar_init(&it_empty[i], readers<Q8>());
    }
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

  // Item number k of this CTA from the ring (warp-collective; -1: no more, -2:
  // the wait ran out).  Every lane's read is consumed by the shuffle before
  // the slot is handed back.
  auto take_item = [&](int k) -> int {
    const int slot = k % kItemRing;
    if (!__all_sync(0xffffffffu,
                    mbar_wait(&it_full[slot], (k / kItemRing) & 1, a.status, a.wait_polls)))
      return -2;
    const int it = __shfl_sync(0xffffffffu, *(volatile int*)&item_ring[slot], 0);
    if (lane == 0) mbar_arrive(&it_empty[slot]);
    return it;
  };

  if (warp == kQWarp) {
    // ------------------------------------------------------- Q TMA (warp 0)
    if (lane == 0) {
      // publishes item k + 1's id (-1 once none is left, or after an abort)
      // before it loads item k's Q, so that the next item's blocks can start
      const uint64_t pol = l2_policy_evict_first();
      const uint32_t rows = (uint32_t)(nq * hpg);
      int cur = atomicAdd(a.next_item, 1);
      if (cur >= a.nitems) cur = -1;
      item_ring[0] = cur;
      mbar_arrive(&it_full[0]);
      int loads[2] = {0, 0};
      for (int k = 0; cur >= 0; ++k) {
        const int r = k + 1, slot = r % kItemRing;
        if (r >= kItemRing &&
            !mbar_wait(&it_empty[slot], ((r / kItemRing) - 1) & 1, a.status, a.wait_polls)) {
          *abort_flag = 1;
          break;
        }
        int nx = *abort_flag ? a.nitems : atomicAdd(a.next_item, 1);
        if (nx >= a.nitems) nx = -1;
        item_ring[slot] = nx;
        mbar_arrive(&it_full[slot]);
        const Item d = item_of(a, cur);
        // a tile that begins behind the last query is loaded from the first
        // one instead: its rows are computed and never written
        bool ok = true;
#pragma unroll
        for (int c = 0; c < 2 && d.nblk > 0; ++c) {
          if (loads[c] > 0 &&
              !mbar_wait(&q_empty[c], (loads[c] - 1) & 1, a.status, a.wait_polls)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&q_full[c], rows * D * 2);
          ++loads[c];
          const int i = d.i0 + c * nq;
          const int z = d.b * T + (i < T ? i : d.i0);
#pragma unroll
          for (int h = 0; h < C::kNHalf; ++h)
            tma_load_3d_hint(smem_u32(sQ + c * C::kTile + h * C::kHalf), &tm_q, &q_full[c], h * 64,
                             d.g * hpg, z, pol);
        }
        if (!ok) {
          *abort_flag = 1;
          break;
        }
        cur = nx;
      }
      // no copy may still be landing when the CTA exits
#pragma unroll
      for (int c = 0; c < 2; ++c)
        if (loads[c] > 0) mbar_wait(&q_full[c], (loads[c] - 1) & 1, nullptr);
    }
  } else if (warp == kKVWarp) {
    // ----------------------------------------------------- K/V TMA (warp 1)
    if (!Q8 && lane == 0) {
      int n = 0;
      bool ok = true, k_only = false;  // k_only: step n's K is loaded, its V is not
      for (int ki = 0; ok && !*abort_flag; ++ki) {
        const int slot = ki % kItemRing;
        if (!mbar_wait(&it_full[slot], (ki / kItemRing) & 1, a.status, a.wait_polls)) {
          ok = false;
          break;
        }
        const int it = *(volatile int*)&item_ring[slot];
        mbar_arrive(&it_empty[slot]);
        if (it < 0) break;
        const Item d = item_of(a, it);
        for (int p = 0; p < d.nblk; ++p, ++n) {
          const int ks = n % kStages;
          const uint32_t w = (uint32_t)(n / kStages);
          // an entry outside the pool (flagged) reads zeros from past its end
          const int64_t pb = cache_block(a.s, d.b, block_at(d, p), a.status);
          const int row = (int)((pb < 0 ? a.s.cache_blocks() : pb) * kBlock);
          if (!mbar_wait(&k_empty[ks], (w & 1) ^ 1, a.status, a.wait_polls)) { ok = false; break; }
          mbar_arrive_expect_tx(&k_full[ks], C::kTile);
#pragma unroll
          for (int h = 0; h < C::kNHalf; ++h)
            tma_load_3d(smem_u32(sK + ks * C::kTile + h * C::kHalf), &tm_k, &k_full[ks], h * 64, d.g,
                        row);
          if (!mbar_wait(&v_empty[ks], (w & 1) ^ 1, a.status, a.wait_polls)) {
            ok = false;
            k_only = true;
            break;
          }
          mbar_arrive_expect_tx(&v_full[ks], C::kTile);
#pragma unroll
          for (int h = 0; h < C::kNHalf; ++h)
            tma_load_3d(smem_u32(sV + ks * C::kTile + h * C::kHalf), &tm_v, &v_full[ks], h * 64, d.g,
                        row);
        }
      }
      if (!ok) *abort_flag = 1;
      // no copy may still be landing when the CTA exits: the last load of
      // each ring slot (a V load is issued only after its slot's K load)
      for (int m = n - 1; m >= 0 && m >= n - kStages; --m) {
        const int ks = m % kStages;
        const uint32_t ph = (uint32_t)(m / kStages) & 1;
        mbar_wait(&k_full[ks], ph, nullptr);
        mbar_wait(&v_full[ks], ph, nullptr);
      }
      if (k_only) mbar_wait(&k_full[n % kStages], (uint32_t)(n / kStages) & 1, nullptr);
    }
  } else if (warp == kMmaWarp) {
    // ---------------------------------------------------------- MMA (warp 2)
    // The whole warp runs the loop; one elected lane issues and commits.
    constexpr uint32_t idesc_s =
        Q8 ? idesc_f16(128, 128, false, false) : idesc_bf16(128, 128, false, false);
    constexpr uint32_t idesc_o = idesc_bf16(128, D, false, true);
    const uint64_t qdesc0 = smem_desc(smem_u32(sQ), 16, 1024, kSwizzle128B);
    const uint64_t kdesc0 = smem_desc(smem_u32(sK), 16, 1024, kSwizzle128B);
    const uint64_t vdesc0 = smem_desc(smem_u32(sV), C::kHalf, 1024, kSwizzle128B);
    // block steps issued, items taken, items begun (those with blocks), block of the item
    int n = 0, ki = 0, k = 0, p = 0;
    bool ok = true, has_s = true, has_pv = false;
    Item d;
    d.nblk = 0;
    // the block whose P.V is due: stage, wait parity, visible rows, first / last of its item
    int pks = 0, phi = 0, plo = 0, psk = 0;
    uint32_t pw = 0;
    bool pfirst = false, plast = false;
    while (ok) {
      if (__any_sync(0xffffffffu, *abort_flag != 0)) { ok = false; break; }
      if (has_s && p == d.nblk) {    // the next item
        int it;
        do {
          it = take_item(ki++);
          if (it >= 0) d = item_of(a, it);
        } while (it >= 0 && d.nblk == 0);
        if (it == -2) { ok = false; break; }
        has_s = it >= 0;
        if (has_s) {
          p = 0;
          ++k;
        }
      }
      if (!has_s && !has_pv) break;
      const int ks = n % kStages;
      const uint32_t w = (uint32_t)(n / kStages);
      if (has_pv) {
        ok = __all_sync(0xffffffffu, mbar_wait(&v_full[pks], pw & 1, a.status, a.wait_polls));
        if (!ok) break;
        if (!Q8 && (phi < kBlock - 1 || (plo > 0 && psk < kBlock))) {
          // rows of V that no query of the item sees
          const uint32_t v = smem_u32(sV + pks * C::kTile);
          auto clear = [&](int r0, int r1) {
            for (int e = lane + r0 * (D / 8); e < r1 * (D / 8); e += 32)
              sts128(v + tile_off(e / (D / 8), e % (D / 8)), make_uint4(0, 0, 0, 0));
          };
          clear(max(psk, 0), min(plo, kBlock));
          clear(phi + 1, kBlock);
          fence_async();
          __syncwarp();
        }
      }
      for (int c = 0; c < 2; ++c) {
        if (has_pv) {
          // ---- P.V(c, n - 1): P in TMEM columns [128c, 128c + 64)
          ok = __all_sync(0xffffffffu,
                          mbar_wait(&p_full[c], (uint32_t)(n - 1) & 1, a.status, a.wait_polls));
          if (!ok) break;
          tc_fence_after();
          const uint64_t vd = vdesc0 + (uint64_t)((pks * C::kTile) >> 4);
          if (elect_one()) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              tc_mma_f16_ts(tmem + 256 + c * 128, tmem + c * 128 + j * 8,
                            vd + (uint64_t)((j * 2048) >> 4), idesc_o, (!pfirst || j > 0) ? 1u : 0u);
            if (plast) tc_commit(&o_full[c]);
            if (c == 1) tc_commit(&v_empty[pks]);
          }
          __syncwarp();
        }
        if (has_s) {
          // ---- S(c, n) = Q_c K^T
          bool okl = true;
          if (p == 0)
            okl = mbar_wait(Q8 ? &q_ready[c] : &q_full[c], (k - 1) & 1, a.status, a.wait_polls);
          if (c == 0) okl = okl && mbar_wait(&k_full[ks], w & 1, a.status, a.wait_polls);
          ok = __all_sync(0xffffffffu, okl);
          if (!ok) break;
          tc_fence_after();
          const uint64_t qd = qdesc0 + (uint64_t)((c * C::kTile) >> 4);
          const uint64_t kd = kdesc0 + (uint64_t)((ks * C::kTile) >> 4);
          if (elect_one()) {
#pragma unroll
            for (int j = 0; j < D / 16; ++j)  // 16 dims: (j & 3) * 32 bytes within a 64-dim half
              tc_mma_f16(tmem + c * 128,
                         qd + (uint64_t)(((j >> 2) * C::kHalf + (j & 3) * 32) >> 4),
                         kd + (uint64_t)(((j >> 2) * C::kHalf + (j & 3) * 32) >> 4), idesc_s,
                         j > 0 ? 1u : 0u);
            tc_commit(&s_full[c]);
            if (c == 1) tc_commit(&k_empty[ks]);
            if (p + 1 == d.nblk) tc_commit(&q_empty[c]);
          }
          __syncwarp();
        }
      }
      if (!ok) break;
      has_pv = has_s;
      if (has_s) {
        const int tok0 = block_at(d, p) * kBlock;
        pks = ks;
        pw = w;
        phi = d.t_last - tok0;
        plo = d.lo - tok0;
        psk = a.sinks - tok0;
        pfirst = p == 0;
        plast = p + 1 == d.nblk;
        ++p;
        ++n;
      }
    }
    if (!ok && lane == 0) *abort_flag = 1;
    // all MMAs done before TMEM is released
    if (elect_one()) tc_commit(bar_fin);
    __syncwarp();
    mbar_wait(bar_fin, 0, nullptr);
  } else if (warp < kConvWarp0) {
    // ------------------------------------- softmax + output (warps 3-10)
    const int c = (warp - kSoftWarp0) >> 2;
    const int quad = warp & 3;
    const int r = quad * 32 + lane;  // row of the tile = TMEM lane
    const uint32_t s_base = tmem + ((uint32_t)(quad * 32) << 16) + c * 128;
    const uint32_t o_base = tmem + ((uint32_t)(quad * 32) << 16) + 256 + c * 128;
    const float sl = a.s.scale * kLog2e;
    const int rq = r / hpg, rh = r - rq * hpg;
    int n = 0, k = 0;                // block steps, items with blocks
    bool ok = true;
    for (int ki = 0; ok; ++ki) {
      const int it = take_item(ki);
      if (it < 0) {
        ok = it == -1;
        break;
      }
      const Item d = item_of(a, it);
      const int i = d.i0 + c * nq + rq;
      const bool valid = rq < nq && i < T;
      if (d.nblk == 0) {
        a.part_ml[(it * 2 + c) * 128 + r] = make_float4(-INFINITY, -INFINITY, 0.f, 0.f);
        continue;
      }
      const int tq = a.pos.q_start[d.b] + i;
      const int tlo = max(0, tq - a.window + 1);
      float fr = sl;                   // score factor of the row
      // O is in units of 2^m (m: maximum of x + ev), l in units of 2^n_ref
      // (maximum of x); without exponents they are the same
      float m_ref = -INFINITY, n_ref = -INFINITY, l = 0.f;
      for (int p = 0; p < d.nblk; ++p, ++n) {
        if (__any_sync(0xffffffffu, *abort_flag != 0) ||
            !__all_sync(0xffffffffu, mbar_wait(&s_full[c], (uint32_t)n & 1, a.status, a.wait_polls))) {
          ok = false;
          break;
        }
        tc_fence_after();
        float f = fr, ev = 0.f;
        if constexpr (Q8) {
          if (p == 0) fr *= q_scale[((k & 1) * 2 + c) * 128 + r];
          const int2 e = meta[n % kMetaRing];
          f = fminf(fmaxf(fr * pow2i(e.x), -3e38f), 3e38f);
          ev = (float)e.y;
        }
        // visible columns: [lo, hi] and [0, sk).  Of a masked block's four
        // chunks of 32 columns, those that all rows of the warp see take the
        // unmasked path and those that none sees are skipped.
        const int tok0 = block_at(d, p) * kBlock;
        const int hi = tq - tok0, lo = tlo - tok0, sk = a.sinks - tok0;
        const bool masked =
            __any_sync(0xffffffffu, hi < kBlock - 1 || (lo > 0 && sk < kBlock));
        uint32_t vis[4];
        int full = 0xF, empty = 0;       // chunks that all rows, no row sees
        if (masked) {
          full = 0;
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            vis[w] = below(hi + 1, w) & (~below(lo, w) | below(sk, w));
            full |= (__all_sync(0xffffffffu, vis[w] == 0xFFFFFFFFu) ? 1 : 0) << w;
            empty |= (__all_sync(0xffffffffu, vis[w] == 0u) ? 1 : 0) << w;
          }
        }
        // pass 1: row maximum of x = f s; whole chunks are reduced by the
        // loads (to the smallest s when f < 0)
        const bool up = __all_sync(0xffffffffu, f >= 0.f);
        float mx = -INFINITY;
        if (!masked) {
          if (up) {
            float s = -INFINITY;
#pragma unroll 1
            for (int cc = 0; cc < 8; cc += 2) {
              const float r0 = tmem_ld16_red<true>(s_base + cc * 16);
              const float r1 = tmem_ld16_red<true>(s_base + cc * 16 + 16);
              tmem_ld_wait();
              s = fmax3(s, r0, r1);
            }
            mx = s * f;
          } else {
            float s = INFINITY;
#pragma unroll 1
            for (int cc = 0; cc < 8; cc += 2) {
              const float r0 = tmem_ld16_red<false>(s_base + cc * 16);
              const float r1 = tmem_ld16_red<false>(s_base + cc * 16 + 16);
              tmem_ld_wait();
              s = fmin3(s, r0, r1);
            }
            mx = s * f;
          }
        } else {
#pragma unroll 1
          for (int cc = 0; cc < 4; ++cc) {
            if (empty >> cc & 1) continue;
            if (full >> cc & 1) {
              const float r0 = up ? tmem_ld16_red<true>(s_base + cc * 32)
                                  : tmem_ld16_red<false>(s_base + cc * 32);
              const float r1 = up ? tmem_ld16_red<true>(s_base + cc * 32 + 16)
                                  : tmem_ld16_red<false>(s_base + cc * 32 + 16);
              tmem_ld_wait();
              mx = fmaxf(mx, fmaxf(r0 * f, r1 * f));
            } else {
              const uint32_t vw = cc == 0 ? vis[0] : cc == 1 ? vis[1] : cc == 2 ? vis[2] : vis[3];
#pragma unroll
              for (int hf = 0; hf < 2; ++hf) {
                uint32_t h[16];
                tmem_ld16(s_base + cc * 32 + hf * 16, h);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e)
                  mx = fmaxf(mx, vw >> (hf * 16 + e) & 1 ? __uint_as_float(h[e]) * f : -INFINITY);
              }
            }
          }
        }
        // lazy rescale: a new reference only when the maximum grew by more
        // than kLazy (always at the row's first visible token)
        const bool grow = mx + ev > m_ref + kLazy;
        float alpha = 1.f;
        if (grow) {
          alpha = m_ref == -INFINITY ? 0.f : ex2(m_ref - (mx + ev));
          m_ref = mx + ev;
          if constexpr (!Q8) l *= alpha;
        }
        if constexpr (Q8) {
          if (mx > n_ref + kLazy) {
            l *= n_ref == -INFINITY ? 0.f : ex2(n_ref - mx);
            n_ref = mx;
          }
        }
        // O of the earlier blocks times alpha, in TMEM (their P.V are done:
        // this block's S was issued after them)
        if (p > 0 && __any_sync(0xffffffffu, grow)) {
#pragma unroll 1
          for (int cc = 0; cc < D / 16; ++cc) {
            uint32_t h[16];
            tmem_ld16(o_base + cc * 16, h);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) h[e] = __float_as_uint(__uint_as_float(h[e]) * alpha);
            tmem_st16(o_base + cc * 16, h);
          }
        }
        // the normaliser's terms from p', or (rarely) by themselves
        const float mn = m_ref == -INFINITY ? 0.f : m_ref - ev;
        const float nn = n_ref == -INFINITY ? 0.f : n_ref;
        bool apart = false;
        if constexpr (Q8) {
          apart = __any_sync(0xffffffffu, mn - nn > kFoldMax);
          if (apart) {
            float ls = 0.f;
#pragma unroll 1
            for (int cc = 0; cc < 8; ++cc) {
              if (empty >> (cc >> 1) & 1) continue;
              uint32_t h[16];
              tmem_ld16(s_base + cc * 16, h);
              tmem_ld_wait();
              uint32_t vw = 0xFFFFFFFFu;
              if (!(full >> (cc >> 1) & 1))
                vw = (cc < 2 ? vis[0] : cc < 4 ? vis[1] : cc < 6 ? vis[2] : vis[3]) >> ((cc & 1) * 16);
#pragma unroll
              for (int e = 0; e < 16; ++e)
                ls += vw >> e & 1 ? ex2(fmaf(__uint_as_float(h[e]), f, -nn)) : 0.f;
            }
            l += ls;
          }
        }
        // pass 2: P = 2^(x - mn) in 16 bits, two per column, written over S
        // (the 32 scores of columns [32cc, 32cc + 32) are read before columns
        // [16cc, 16cc + 16), already read, are written); row sum
        const float2 f2 = make_float2(f, f), nm2 = make_float2(-mn, -mn);
        float2 lsum = make_float2(0.f, 0.f);
        // columns [32cc, 32cc + 32) that every row sees
        auto whole_chunk = [&](int cc, uint32_t (&wv)[16]) {
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            uint32_t h[16];
            tmem_ld16(s_base + cc * 32 + hf * 16, h);
            tmem_ld_wait();
#pragma unroll
            for (int u = 0; u < 8; ++u) {
              const float2 x = ffma2(
                  make_float2(__uint_as_float(h[2 * u]), __uint_as_float(h[2 * u + 1])), f2, nm2);
              const float2 pp = make_float2(ex2(x.x), ex2(x.y));
              lsum = fadd2(lsum, pp);
              wv[hf * 8 + u] = pack_bf16(pp.x, pp.y);
            }
          }
        };
        if (!masked) {
#pragma unroll 1
          for (int cc = 0; cc < 4; ++cc) {
            uint32_t wv[16];
            whole_chunk(cc, wv);
            tmem_st16(s_base + cc * 16, wv);
          }
        } else {
#pragma unroll 1
          for (int cc = 0; cc < 4; ++cc) {
            uint32_t wv[16];
            if (empty >> cc & 1) {
#pragma unroll
              for (int u = 0; u < 16; ++u) wv[u] = 0u;
            } else if (full >> cc & 1) {
              whole_chunk(cc, wv);
            } else {
              const uint32_t vw = cc == 0 ? vis[0] : cc == 1 ? vis[1] : cc == 2 ? vis[2] : vis[3];
#pragma unroll
              for (int hf = 0; hf < 2; ++hf) {
                uint32_t h[16];
                tmem_ld16(s_base + cc * 32 + hf * 16, h);
                tmem_ld_wait();
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                  const float2 x = ffma2(
                      make_float2(__uint_as_float(h[2 * u]), __uint_as_float(h[2 * u + 1])), f2, nm2);
                  float2 pp;
                  pp.x = vw >> (hf * 16 + 2 * u) & 1 ? ex2(x.x) : 0.f;
                  pp.y = vw >> (hf * 16 + 2 * u + 1) & 1 ? ex2(x.y) : 0.f;
                  lsum = fadd2(lsum, pp);
                  wv[hf * 8 + u] = pack_bf16(pp.x, pp.y);
                }
              }
            }
            tmem_st16(s_base + cc * 16, wv);
          }
        }
        const float ls = lsum.x + lsum.y;
        if constexpr (Q8) {
          if (!apart) l = fmaf(ls, ex2(mn - nn), l);
        } else {
          l += ls;
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&p_full[c]);
      }
      if (!ok) break;
      // output: O / l after the item's last P.V
      if (!__all_sync(0xffffffffu, mbar_wait(&o_full[c], (uint32_t)k & 1, a.status, a.wait_polls))) {
        ok = false;
        break;
      }
      tc_fence_after();
      ++k;
      if (a.splits > 1) {
        const int prow = (it * 2 + c) * 128 + r;     // below 2^16: at most kSplitItems items
        if (valid) a.part_ml[prow] = make_float4(m_ref, Q8 ? n_ref : m_ref, l, 0.f);
#pragma unroll 1
        for (int cc = 0; cc < D / 16; ++cc) {
          uint32_t h[16];
          tmem_ld16(o_base + cc * 16, h);
          tmem_ld_wait();
          if (valid) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              *reinterpret_cast<uint4*>(a.part_o + (int64_t)prow * D + cc * 16 + e * 4) =
                  make_uint4(h[e * 4], h[e * 4 + 1], h[e * 4 + 2], h[e * 4 + 3]);
          }
        }
        continue;
      }
      const float inv = l == 0.f ? 0.f : (Q8 ? ex2(m_ref - n_ref) : 1.f) / l;
      // two lanes' rows, 32 bytes each, become 64 bytes of a row over both lanes
      uint16_t* dst =
          a.out + (((int64_t)d.b * T + d.i0 + c * nq) * H + (int64_t)d.g * hpg) * D;
      const int rel = valid ? (rq * H + rh) * D : -1;
      const bool up = lane & 1, wide = ((uintptr_t)a.out & 31) == 0;
      int at[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) at[j] = __shfl_sync(0xffffffffu, rel, (lane & ~1) + j);
#pragma unroll 1
      for (int cc = 0; cc < D / 32; ++cc) {
        uint32_t w[2][8];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t h[16];
          tmem_ld16(o_base + cc * 32 + hf * 16, h);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 8; ++j)
            w[hf][j] = pack_bf16(__uint_as_float(h[2 * j]) * inv, __uint_as_float(h[2 * j + 1]) * inv);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? w[0][j] : w[1][j], 1);
          w[0][j] = up ? got : w[0][j];
          w[1][j] = up ? w[1][j] : got;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
          if (at[j] >= 0) {
            uint16_t* p = dst + at[j] + cc * 32 + up * 16;
            if (wide) {
              stg256(p, w[j]);
            } else {                     // an output aligned to 16 bytes only
              *reinterpret_cast<uint4*>(p) = make_uint4(w[j][0], w[j][1], w[j][2], w[j][3]);
              *reinterpret_cast<uint4*>(p + 8) = make_uint4(w[j][4], w[j][5], w[j][6], w[j][7]);
            }
          }
      }
    }
    if (!ok) *abort_flag = 1;
  } else if constexpr (Q8) {
    // ------------------------------------------- converters (warps 11-14)
    const int tid = threadIdx.x - kConvWarp0 * 32;
    constexpr int NC = D / 16;               // 16-byte chunks of codes in a row
    constexpr int NL = NC;                   // chunks per thread and block (128 NC / 128)
    // chunk u of this thread: row tid / 4 + 32 (u % 4), chunk 4 (u / 4) + tid % 4
    const int row0 = tid >> 2, c4 = tid & 3;
    const int64_t pitch = (int64_t)a.s.G * D;
    struct Step {
      int64_t off;      // byte offset of the block's codes of the KV head, -1: none
      int ek, ev;
      int tok0;
    };
    // the block of list position p of item d
    auto resolve = [&](const Item& d, int p) {
      Step x;
      const int kb = block_at(d, p);
      x.tok0 = kb * kBlock;
      const int64_t pb = cache_block(a.s, d.b, kb, a.status);
      x.off = pb < 0 ? -1 : (pb * kBlock * a.s.G + d.g) * D;
      x.ek = pb < 0 ? 0 : clamp_exp(a.k_exp[pb * a.s.G + d.g]);
      x.ev = pb < 0 ? 0 : clamp_exp(a.v_exp[pb * a.s.G + d.g]);
      return x;
    };
    auto load = [&](const uint8_t* base, const Step& x, uint4 (&v)[NL]) {
#pragma unroll
      for (int u = 0; u < NL; ++u) {
        const int r = row0 + 32 * (u & 3), ch = 4 * (u >> 2) + c4;
        v[u] = x.off < 0 ? make_uint4(0, 0, 0, 0)
                         : __ldg(reinterpret_cast<const uint4*>(base + x.off + r * pitch + ch * 16));
      }
    };
    auto store = [&](const bool is_v, uint32_t tile, const uint4 (&v)[NL], int hi, int lo,
                     int sk) {
#pragma unroll
      for (int u = 0; u < NL; ++u) {
        const int r = row0 + 32 * (u & 3), ch = 4 * (u >> 2) + c4;
        const bool dead = r > hi || (r < lo && r >= sk);
        const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
        uint32_t h[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (is_v) e4m3x4_to_bf16(dead ? 0u : w[j], h[2 * j], h[2 * j + 1]);
          else e4m3x4_to_f16(w[j], h[2 * j], h[2 * j + 1]);
        }
        sts128(tile + tile_off(r, 2 * ch), make_uint4(h[0], h[1], h[2], h[3]));
        sts128(tile + tile_off(r, 2 * ch + 1), make_uint4(h[4], h[5], h[6], h[7]));
      }
    };
    // Q tiles of item k to f16, each row scaled to a maximum in [2^13, 2^14)
    auto convert_q = [&](int k) -> bool {
#pragma unroll 1
      for (int c = 0; c < 2; ++c) {
        if (!__all_sync(0xffffffffu, mbar_wait(&q_full[c], (uint32_t)k & 1, a.status, a.wait_polls)))
          return false;
        const uint32_t tile = smem_u32(sQ + c * C::kTile);
        uint32_t mx = 0;
#pragma unroll 4
        for (int ch = 0; ch < D / 8; ++ch) {
          const uint4 v = lds128(tile + tile_off(tid, ch));
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) mx = max(max(mx, w[j] & 0x7FFFu), w[j] >> 16 & 0x7FFFu);
        }
        int e = (int)(mx >> 7) - 127;                  // floor(log2 max); inf, NaN: 128
        e = mx == 0 || e == 128 ? 0 : max(e, -100);
        const float f = pow2i(13 - e);
#pragma unroll 4
        for (int ch = 0; ch < D / 8; ++ch) {
          const uint4 v = lds128(tile + tile_off(tid, ch));
          sts128(tile + tile_off(tid, ch),
                 make_uint4(pack_f16(bf16lo(v.x) * f, bf16hi(v.x) * f),
                            pack_f16(bf16lo(v.y) * f, bf16hi(v.y) * f),
                            pack_f16(bf16lo(v.z) * f, bf16hi(v.z) * f),
                            pack_f16(bf16lo(v.w) * f, bf16hi(v.w) * f)));
        }
        q_scale[((k & 1) * 2 + c) * 128 + tid] = pow2i(e - 13);
        fence_async();
        mbar_arrive(&q_ready[c]);
      }
      return true;
    };
    int n = 0, ki = 0, k = 0;        // block steps, items taken, items with blocks
    // the next item that has blocks
    auto next_item = [&](Item& d) -> int {
      int it;
      do {
        it = take_item(ki++);
        if (it >= 0) d = item_of(a, it);
      } while (it >= 0 && d.nblk == 0);
      return it;
    };
    uint4 kreg[NL], vreg[NL];
    Item d;
    Step cur;
    int it = next_item(d);
    bool ok = it != -2;
    if (it >= 0) {
      cur = resolve(d, 0);
      load(a.k8, cur, kreg);
    }
    while (ok && it >= 0) {
      int nit = -1;
      for (int p = 0; p < d.nblk && ok; ++p, ++n) {
        if (__any_sync(0xffffffffu, *abort_flag != 0)) { ok = false; break; }
        load(a.v8, cur, vreg);
        // the step after this one: its block and exponents early
        Step nxt = cur;
        Item nd = d;
        bool more = true;
        if (p + 1 < d.nblk) {
          nxt = resolve(d, p + 1);
        } else {
          nit = next_item(nd);
          if (nit == -2) { ok = false; break; }
          more = nit >= 0;
          if (more) nxt = resolve(nd, 0);
        }
        const int ks = n % kStages;
        const uint32_t w = (uint32_t)(n / kStages);
        ok = __all_sync(0xffffffffu, mbar_wait(&k_empty[ks], (w & 1) ^ 1, a.status, a.wait_polls));
        if (!ok) break;
        if (tid == 0) meta[n % kMetaRing] = make_int2(cur.ek, cur.ev);
        store(false, smem_u32(sK + ks * C::kTile), kreg, kBlock, 0, 0);
        fence_async();
        mbar_arrive(&k_full[ks]);
        if (p == 0 && !convert_q(k)) { ok = false; break; }
        if (more) load(a.k8, nxt, kreg);
        ok = __all_sync(0xffffffffu, mbar_wait(&v_empty[ks], (w & 1) ^ 1, a.status, a.wait_polls));
        if (!ok) break;
        store(true, smem_u32(sV + ks * C::kTile), vreg, d.t_last - cur.tok0, d.lo - cur.tok0,
              a.sinks - cur.tok0);
        fence_async();
        mbar_arrive(&v_full[ks]);
        cur = nxt;
        if (p + 1 == d.nblk) {
          it = nit;
          d = nd;
          ++n;
          break;
        }
      }
      ++k;
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

// Joins the parts of split block lists: one warp per (sequence, query, head).
template <int D>
__global__ void __launch_bounds__(256) window_join_kernel(const __grid_constant__ WinArgs a) {
  constexpr int PER = D / 32;
  const Shape& s = a.s;
  const int lane = threadIdx.x & 31, hpg = s.H / s.G;
  const int64_t gw = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (gw >= (int64_t)s.B * s.T * s.H) return;
  const int h = (int)(gw % s.H), g = h / hpg;
  const int i = (int)(gw / s.H % s.T), b = (int)(gw / s.H / s.T);
  const int pair = i / (2 * a.nq), j = i % (2 * a.nq);           // item, query in it
  const int64_t item = ((int64_t)(a.npair - 1 - pair) * s.B * s.G + b * s.G + g) * a.splits;
  const int row = (j / a.nq) * 128 + j % a.nq * hpg + h % hpg;   // chain, tile row
  float M = -INFINITY, N = -INFINITY;
  for (int p = lane; p < a.splits; p += 32) {
    const float4 v = a.part_ml[(item + p) * 256 + row];
    M = fmaxf(M, v.x);
    N = fmaxf(N, v.y);
  }
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) {
    M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
    N = fmaxf(N, __shfl_xor_sync(0xffffffffu, N, x));
  }
  float L = 0.f, acc[PER];
#pragma unroll
  for (int e = 0; e < PER; ++e) acc[e] = 0.f;
#pragma unroll 4
  for (int p = 0; p < a.splits; ++p) {
    const float4 v = a.part_ml[(item + p) * 256 + row];
    if (v.z == 0.f) continue;        // no visible token (or no block): nothing written
    const float w = v.x == -INFINITY ? 0.f : ex2(v.x - M);
    L = fmaf(v.y == -INFINITY ? 0.f : ex2(v.y - N), v.z, L);
    const float* o = a.part_o + ((item + p) * 256 + row) * D + lane * PER;
#pragma unroll
    for (int e = 0; e < PER; ++e) acc[e] = fmaf(w, o[e], acc[e]);
  }
  const float inv = L == 0.f ? 0.f : ex2(M - N) / L;
  uint16_t* dst = a.out + gw * D + lane * PER;
#pragma unroll
  for (int e = 0; e < PER; e += 2)
    *reinterpret_cast<uint32_t*>(dst + e) = pack_bf16(acc[e] * inv, acc[e + 1] * inv);
}

template <int D, bool Q8>
cudaError_t launch_impl(const Shape& s, const Positions& pos, const CacheView& c, int window,
                        int sinks, const uint16_t* q, uint16_t* out, int* status, char* base,
                        cudaStream_t st) {
  using C = WinCfg<D>;
  // the item counter sits in the word after the status word; both are zeroed
  if (cudaMemsetAsync(status, 0, 2 * sizeof(int), st) != cudaSuccess) return cudaErrorUnknown;
  const int hpg = s.H / s.G;
  WinArgs a;
  a.s = s;
  a.pos = pos;
  a.window = window;
  a.sinks = sinks;
  a.nq = 128 / hpg;
  a.npair = (s.T + 2 * a.nq - 1) / (2 * a.nq);
  a.splits = window_splits(s, pos, window, sinks);
  a.nitems = a.npair * s.B * s.G * a.splits;
  a.part_ml = reinterpret_cast<float4*>(base);
  a.part_o = reinterpret_cast<float*>(base + (size_t)kSplitItems * 256 * sizeof(float4));
  a.next_item = status + 1;
  a.k8 = static_cast<const uint8_t*>(c.k);
  a.v8 = static_cast<const uint8_t*>(c.v);
  a.k_exp = c.k_exp;
  a.v_exp = c.v_exp;
  a.out = out;
  a.status = status;
  a.wait_polls = debug_wait_polls();
  CUtensorMap tm_q, tm_k, tm_v;
  {
    // q as (D dims, H heads, B*T queries): one box = 64 dims of the H/G heads
    // of nq queries, rows in (query, head) order
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)s.H, (cuuint64_t)s.B * s.T};
    cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)s.H * D * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)hpg, (cuuint32_t)a.nq};
    if (!encode_bf16_map(&tm_q, q, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
  }
  if constexpr (!Q8) {
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)s.G, (cuuint64_t)(s.cache_blocks() * kBlock)};
    cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)s.G * D * 2};
    cuuint32_t box[3] = {64, 1, (cuuint32_t)kBlock};
    if (!encode_bf16_map(&tm_k, c.k, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_bf16_map(&tm_v, c.v, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
  } else {
    tm_k = tm_v = tm_q;   // not used
  }
  cudaError_t e = cudaFuncSetAttribute(window_tc_kernel<D, Q8>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  const int ctas = sm_count();
  note_launches(1);
  window_tc_kernel<D, Q8><<<a.nitems < ctas ? a.nitems : ctas, threads<Q8>(), C::kSmem, st>>>(
      tm_q, tm_k, tm_v, a);
  if (a.splits > 1) {
    const int64_t warps = (int64_t)s.B * s.T * s.H;
    note_launches(1);
    window_join_kernel<D><<<(unsigned)((warps + 7) / 8), 256, 0, st>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace

// Items of at most kSplitItems parts in all: no workspace grows with the call.
// A part keeps at least kMinBlocks blocks of the longest list (a part costs
// about 3 us of its own: Q, the output, the join).
size_t window_tc_scratch_bytes(const Shape& s) {
  const int nq = 128 / (s.H / s.G);
  const int64_t items = (int64_t)((s.T + 2 * nq - 1) / (2 * nq)) * s.B * s.G;
  if (items * 2 > kSplitItems) return 0;
  return (size_t)kSplitItems * 256 * (sizeof(float4) + s.D * sizeof(float));
}

int window_splits(const Shape& s, const Positions& pos, int window, int sinks) {
  constexpr int kMinBlocks = 4;
  const int nq = 128 / (s.H / s.G);
  const int64_t items = (int64_t)((s.T + 2 * nq - 1) / (2 * nq)) * s.B * s.G;
  if (items * 2 > kSplitItems) return 1;
  const int longest = window_list_len(s, pos, window, sinks);
  int n = (int)(kSplitItems / items);
  if (n > longest / kMinBlocks) n = longest / kMinBlocks;
  return n < 1 ? 1 : n;
}

int window_list_len(const Shape& s, const Positions& pos, int window, int sinks) {
  const int nq = 128 / (s.H / s.G);
  int longest = 1;
  for (int b = 0; b < s.B; ++b) {
    // the last item's queries see the longest list, or one block less
    const int t1 = pos.q_start[b] + s.T - 1;
    const int t0 = pos.q_start[b] + (s.T - 1) / (2 * nq) * (2 * nq);
    const int lo = (t0 - window + 1 > 0 ? t0 - window + 1 : 0) / kBlock;
    const int sb = (sinks + kBlock - 1) / kBlock;
    const int n = (sb < lo ? sb : lo) + t1 / kBlock - lo + 1;
    longest = n > longest ? n : longest;
  }
  return longest;
}

cudaError_t launch_window_tc(const Shape& s, const Positions& pos, const CacheView& c, int window,
                             int sinks, const uint16_t* q, uint16_t* out, int* status, char* base,
                             cudaStream_t st) {
  if (s.D == 128)
    return c.kv8 ? launch_impl<128, true>(s, pos, c, window, sinks, q, out, status, base, st)
                 : launch_impl<128, false>(s, pos, c, window, sinks, q, out, status, base, st);
  return c.kv8 ? launch_impl<64, true>(s, pos, c, window, sinks, q, out, status, base, st)
               : launch_impl<64, false>(s, pos, c, window, sinks, q, out, status, base, st);
}

}  // namespace msa

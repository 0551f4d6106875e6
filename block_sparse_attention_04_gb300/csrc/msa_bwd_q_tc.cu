// dQ of the dense attention's backward pass on tensor cores, query-outer: an item is a
// 128-query tile of one head (or a split of its key blocks, where there are few items),
// whose dQ stays in tensor memory over the key blocks,
//     S = Q K^T   dP = dO V^T   dS = 2^(S scale log2e - lse log2e) (dP - delta)
//     dQ += dS K
// with the queries on the 128 lanes.  dS is written over S as bf16, the A operand of the
// last product; K is read K-major by the first product and MN-major by the last.
//   warp 0       TMA of the item's Q and dO; takes the items from a shared counter
//   warp 1       TMA of K (3 stages: a block is read until its dQ product) and V (2)
//   warp 2       tcgen05.mma of dQ and S, S in two buffers
//   warp 3       tcgen05.mma of dP
//   warps 4-19   dS: four warpgroups, 32 keys of a block each; an item's dQ
// The two numbers of a row (lse, delta) stay in registers over an item.
#include "msa_bwd.h"
#include "msa_q8.cuh"
#include "msa_tma.h"

namespace msa {
namespace {

constexpr int kAW = 2, kBW = 3, kSoftW = 4;   // warps: MMA of S and dQ, of dP; dS
constexpr int kNG = 4;                    // warpgroups for dS ...
constexpr int kCols = 128 / kNG;          // ... and the keys of a block that each has
constexpr int kThreadsQ = 32 * (kSoftW + 4 * kNG);
constexpr int kRing = 4, kReaders = 3 + 4 * kNG;

template <int D>
struct QCfg {
  static constexpr int kNHalf = D / 64;
  static constexpr int kHalf = 128 * 128;
  static constexpr int kTile = kNHalf * kHalf;
  static constexpr int kKS = 3, kVS = 2;             // stages of K and V
  static constexpr int kSmem = (2 + kKS + kVS) * kTile + 512;
  // tensor memory columns: S in two buffers, dP, dQ
  static constexpr uint32_t kS = 0, kP = 256, kDQ = 384;
  static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
};

// Items heaviest first: query tiles from the last down; the heads of a group together.
struct QItem {
  int b, h, g, qt, kb0, kb1;     // key blocks [kb0, kb1)
};
__device__ __forceinline__ QItem q_item(const BwdQArgs& a, int it) {
  QItem d;
  const int split = it % a.splits;
  int r = it / a.splits;
  const int per = a.s.B * a.s.H;
  d.qt = a.nqt - 1 - r / per;
  r %= per;
  d.b = r / a.s.H;
  d.h = r % a.s.H;
  d.g = d.h / (a.s.H / a.s.G);
  const int i_last = min(a.s.T - 1, d.qt * 128 + 127);
  const int n = (int)(((int64_t)a.pos.q_start[d.b] + i_last) / kBlock) + 1;
  d.kb0 = (int)((int64_t)n * split / a.splits);
  d.kb1 = (int)((int64_t)n * (split + 1) / a.splits);
  return d;
}

template <int D>
__global__ void __launch_bounds__(kThreadsQ, 1)
    bwd_q_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_o,
                 const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                 const __grid_constant__ BwdQArgs a) {
  using C = QCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sQ = smem;
  uint8_t* sO = sQ + C::kTile;
  uint8_t* sK = sO + C::kTile;                     // [kKS]
  uint8_t* sV = sK + C::kKS * C::kTile;            // [kVS]
  uint64_t* q_full = reinterpret_cast<uint64_t*>(sV + C::kVS * C::kTile);
  uint64_t* q_empty = q_full + 1;
  uint64_t* k_full = q_empty + 1;                  // [kKS]
  uint64_t* k_empty = k_full + C::kKS;
  uint64_t* v_full = k_empty + C::kKS;             // [kVS]
  uint64_t* v_empty = v_full + C::kVS;
  uint64_t* s_full = v_empty + C::kVS;                // [2] S of the block is in its buffer
  uint64_t* dp_full = s_full + 2;
  // [2] dS written over S: one per buffer, as the warp that waits for both (dQ) may fall
  // behind the one that lets the next dS be made (dP)
  uint64_t* ds_full = dp_full + 1;
  uint64_t* acc_full = ds_full + 2;                // the item's dQ is complete
  uint64_t* acc_empty = acc_full + 1;              // ... and read out
  uint64_t* bar_fin = acc_empty + 1;
  uint64_t* it_full = bar_fin + 1;                 // [kRing]
  uint64_t* it_empty = it_full + kRing;
  int* ring = reinterpret_cast<int*>(it_empty + kRing);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ring + kRing);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 2);
    for (int i = 0; i < C::kKS; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < C::kVS; ++i) {
      mbar_init(&v_full[i], 1);
      mbar_init(&v_empty[i], 1);
    }
    mbar_init(&s_full[0], 1);
    mbar_init(&s_full[1], 1);
    mbar_init(dp_full, 1);
    mbar_init(&ds_full[0], 128 * kNG);
    mbar_init(&ds_full[1], 128 * kNG);
    mbar_init(acc_full, 1);
    mbar_init(acc_empty, 128 * kNG);
    mbar_init(bar_fin, 2);
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&it_full[i], 1);
      mbar_init(&it_empty[i], kReaders);
    }
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_o);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == kAW) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int T = a.s.T;

  // A warp's next item from the ring (every lane gets it); false: no more, or given up.
  int ki = 0;
  auto next_item = [&](int& it, bool& ok) {
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
    // ----------------------------------------------------- Q and dO (warp 0)
    if (lane == 0) {
      const uint64_t pol = l2_policy_evict_first();
      int cur = atomicAdd(a.next_item, 1);
      if (cur >= a.nitems * a.splits) cur = -1;
      ring[0] = cur;
      mbar_arrive(&it_full[0]);
      int n = 0;                 // items with key blocks, loaded
      bool ok = true;
      for (int k = 0; cur >= 0; ++k) {
        // publish the next item before this one's tiles, so that its K and V can start
        const int r = k + 1, slot = r % kRing;
        if (r >= kRing && !mbar_wait(&it_empty[slot], ((r / kRing) - 1) & 1, a.status, a.wait_polls)) {
          ok = false;
          break;
        }
        int nx = *abort_flag ? a.nitems * a.splits : atomicAdd(a.next_item, 1);
        if (nx >= a.nitems * a.splits) nx = -1;
        ring[slot] = nx;
        mbar_arrive(&it_full[slot]);
        const QItem d = q_item(a, cur);
        if (d.kb0 < d.kb1) {
          if (n > 0 && !mbar_wait(q_empty, (uint32_t)(n - 1) & 1, a.status, a.wait_polls)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(q_full, 2 * C::kTile);
#pragma unroll
          for (int hf = 0; hf < C::kNHalf; ++hf) {
            tma_load_4d_hint(smem_u32(sQ + hf * C::kHalf), &tm_q, q_full, hf * 64, d.h, d.qt * 128,
                             d.b, pol);
            tma_load_4d_hint(smem_u32(sO + hf * C::kHalf), &tm_o, q_full, hf * 64, d.h, d.qt * 128,
                             d.b, pol);
          }
          ++n;
        }
        cur = nx;
      }
      if (!ok) *abort_flag = 1;
      // no copy may still be landing when the CTA exits
      if (n > 0) mbar_wait(q_full, (uint32_t)(n - 1) & 1, nullptr);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------- K and V (warp 1)
    int it, n = 0;
    bool ok, k_only = false;     // k_only: block n's K is on its way, its V is not
    while (next_item(it, ok)) {
      const QItem d = q_item(a, it);
      for (int kb = d.kb0; kb < d.kb1; ++kb, ++n) {
        const int ks = n % C::kKS, vs = n % C::kVS;
        const int row = (int)(((int64_t)d.b * a.s.max_blocks + kb) * kBlock);
        ok = __any_sync(0xffffffffu, *abort_flag != 0) == 0 &&
             wait_all(&k_empty[ks], ((n / C::kKS) & 1) ^ 1);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&k_full[ks], C::kTile);
#pragma unroll
          for (int hf = 0; hf < C::kNHalf; ++hf)
            tma_load_3d(smem_u32(sK + ks * C::kTile + hf * C::kHalf), &tm_k, &k_full[ks], hf * 64, d.g,
                        row);
        }
        __syncwarp();
        ok = wait_all(&v_empty[vs], ((n / C::kVS) & 1) ^ 1);
        if (!ok) {
          k_only = true;
          break;
        }
        if (lane == 0) {
          mbar_arrive_expect_tx(&v_full[vs], C::kTile);
#pragma unroll
          for (int hf = 0; hf < C::kNHalf; ++hf)
            tma_load_3d(smem_u32(sV + vs * C::kTile + hf * C::kHalf), &tm_v, &v_full[vs], hf * 64, d.g,
                        row);
        }
        __syncwarp();
      }
      if (!ok) break;
    }
    if (!ok && lane == 0) *abort_flag = 1;
    const int nk = k_only ? n + 1 : n;
    for (int m = nk - 1; m >= 0 && m >= nk - C::kKS; --m)
      mbar_wait(&k_full[m % C::kKS], (uint32_t)(m / C::kKS) & 1, nullptr);
    for (int m = n - 1; m >= 0 && m >= n - C::kVS; --m)
      mbar_wait(&v_full[m % C::kVS], (uint32_t)(m / C::kVS) & 1, nullptr);
  } else if (warp == kAW || warp == kBW) {
    // ------------------------------------------------------- MMA (warps 2, 3)
    // Two warps, as issuing takes longer than the products: with one for all three a step
    // took 2650 cycles, 1536 of them MMAs.
    constexpr uint32_t idesc_s = idesc_bf16(128, 128, false, false);
    constexpr uint32_t idesc_q = idesc_bf16(128, D, false, true);
    const uint64_t qd = smem_desc(smem_u32(sQ), 16, 1024, kSwizzle128B);
    const uint64_t od = smem_desc(smem_u32(sO), 16, 1024, kSwizzle128B);
    const uint64_t kd = smem_desc(smem_u32(sK), 16, 1024, kSwizzle128B);
    const uint64_t vd = smem_desc(smem_u32(sV), 16, 1024, kSwizzle128B);
    const uint64_t kmn = smem_desc(smem_u32(sK), C::kHalf, 1024, kSwizzle128B);
    auto product = [&](uint32_t d, uint64_t ad, uint64_t bd) {
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {
        const uint64_t o = (uint64_t)(((j >> 2) * C::kHalf + (j & 3) * 32) >> 4);
        tc_mma_f16(tmem + d, ad + o, bd + o, idesc_s, j > 0 ? 1u : 0u);
      }
    };
    int it, n = 0, nu = 0;       // blocks and items (with blocks) so far
    bool ok;
    if (warp == kAW) {
      // ---------------------------------------- S(0), S(1); dQ(n), S(n + 2)
      while (next_item(it, ok)) {
        const QItem d = q_item(a, it);
        const int nt = d.kb1 - d.kb0;
        if (nt == 0) continue;
        const int64_t t_last = (int64_t)a.pos.q_start[d.b] + T - 1;
        ok = wait_all(q_full, (uint32_t)nu & 1);
        if (!ok) break;
        auto issue_s = [&](int m, int t) {         // of block m, the item's t-th
          const int ks = m % C::kKS;
          if (!wait_all(&k_full[ks], (uint32_t)(m / C::kKS) & 1)) return false;
          const int64_t left = t_last - (int64_t)(d.kb0 + t) * kBlock;
          if (left < kBlock - 1) {
            // rows behind the sequence's last query may hold anything; in dQ's product
            // they are multiplied by zeros: cleared
            for (int e = lane; e < C::kNHalf * kBlock * 8; e += 32) {
              const int row = e >> 3 & 127;
              if (row > (int)left)
                sts128(smem_u32(sK) + ks * C::kTile + (e >> 10) * C::kHalf + row * 128 + (e & 7) * 16,
                       make_uint4(0, 0, 0, 0));
            }
            fence_async();
            __syncwarp();
          }
          tc_fence_after();
          if (elect_one()) {
            product(C::kS + (m & 1) * 128, qd, kd + (uint64_t)((ks * C::kTile) >> 4));
            tc_commit(&s_full[m & 1]);
            if (t + 1 == nt) tc_commit(q_empty);
          }
          __syncwarp();
          return true;
        };
        ok = issue_s(n, 0) && (nt == 1 || issue_s(n + 1, 1));
        for (int t = 0; t < nt && ok; ++t, ++n) {
          const int ks = n % C::kKS;
          ok = wait_all(&ds_full[n & 1], (uint32_t)(n >> 1) & 1) &&
               (t > 0 || nu == 0 || wait_all(acc_empty, (uint32_t)(nu - 1) & 1));
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            // dS: a warpgroup's keys at the start of its columns of S, two in each
#pragma unroll
            for (int j = 0; j < 8; ++j)
              tc_mma_f16_ts(tmem + C::kDQ,
                            tmem + C::kS + (n & 1) * 128 + j * 16 / kCols * kCols + j * 16 % kCols / 2,
                            kmn + (uint64_t)((ks * C::kTile + j * 2048) >> 4), idesc_q,
                            t > 0 || j > 0 ? 1u : 0u);
            tc_commit(&k_empty[ks]);
            if (t + 1 == nt) tc_commit(acc_full);
          }
          __syncwarp();
          // over dS(n), which dQ(n), issued before, reads
          if (t + 2 < nt) ok = issue_s(n + 2, t + 2);
        }
        if (!ok) break;
        ++nu;
      }
    } else {
      // ------------------------------------------------------------ dP(n)
      while (next_item(it, ok)) {
        const QItem d = q_item(a, it);
        const int nt = d.kb1 - d.kb0;
        if (nt == 0) continue;
        ok = wait_all(q_full, (uint32_t)nu & 1);
        for (int t = 0; t < nt && ok; ++t, ++n) {
          const int vs = n % C::kVS;
          // dP(n - 1) has been read
          ok = wait_all(&v_full[vs], (uint32_t)(n / C::kVS) & 1) &&
               (n == 0 || wait_all(&ds_full[(n - 1) & 1], (uint32_t)((n - 1) >> 1) & 1));
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            product(C::kP, od, vd + (uint64_t)((vs * C::kTile) >> 4));
            tc_commit(dp_full);
            tc_commit(&v_empty[vs]);
            if (t + 1 == nt) tc_commit(q_empty);
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
  } else {
    // ------------------------------------------------- dS, dQ (warps 4-19)
    const int c = (warp - kSoftW) >> 2;           // keys kCols c ..; dims c D/kNG .. of dQ
    const int quad = warp & 3;
    const int r = quad * 32 + lane;               // query of the tile = TMEM lane
    const uint32_t base = tmem + ((uint32_t)(quad * 32) << 16);
    const float sl = a.s.scale * kLog2e;
    const float2 sl2 = make_float2(sl, sl);
    int it, n = 0, nu = 0;
    bool ok;
    while (next_item(it, ok)) {
      const QItem d = q_item(a, it);
      const int i = d.qt * 128 + r;
      const int64_t tq = (int64_t)a.pos.q_start[d.b] + i;
      const float* st = reinterpret_cast<const float*>(
                            a.stat + ((size_t)(d.b * a.s.H + d.h) * a.stat_groups + (i >> 3)) * kStatBytes) +
                        (i & 7);
      const float nl = st[0], nd = st[8];
      const float2 nl2 = make_float2(nl, nl), nd2 = make_float2(nd, nd);
      for (int kb = d.kb0; kb < d.kb1; ++kb, ++n) {
        // keys past the query, and rows past the last query, whatever they hold
        const int64_t l64 = min(tq, (int64_t)a.pos.q_start[d.b] + T - 1) - (int64_t)kb * kBlock;
        const int lim = (int)(l64 < kBlock ? l64 : kBlock) - c * kCols;
        const bool masked = __any_sync(0xffffffffu, lim < kCols - 1);
        ok = __all_sync(0xffffffffu,
                        *abort_flag == 0 &&
                            mbar_wait(&s_full[n & 1], (uint32_t)(n >> 1) & 1, a.status, a.wait_polls));
        if (!ok) break;
        tc_fence_after();
        const uint32_t s_at = base + C::kS + (n & 1) * 128 + c * kCols;
        float2 p[kCols / 2];
        {
          uint32_t x[32];
          tmem_ld32(s_at, x);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 y = ffma2(make_float2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])),
                                   sl2, nl2);
            p[e] = make_float2(ex2(y.x), ex2(y.y));
          }
        }
        ok = __all_sync(0xffffffffu, mbar_wait(dp_full, (uint32_t)n & 1, a.status, a.wait_polls));
        if (!ok) break;
        tc_fence_after();
        uint32_t x[32], w[16];
        tmem_ld32(base + C::kP + c * kCols, x);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float2 y = fadd2(make_float2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), nd2);
          y = fmul2(p[e], y);
          if (masked) {
            y.x = 2 * e <= lim ? y.x : 0.f;
            y.y = 2 * e + 1 <= lim ? y.y : 0.f;
          }
          w[e] = pack_bf16(y.x, y.y);
        }
        tmem_st16(s_at, w);              // over scores that were read already
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&ds_full[n & 1]);
      }
      if (!ok) break;
      // ---- the item's dQ: a query per thread, a run of dims per warpgroup
      const bool any = d.kb0 < d.kb1;
      if (any) {
        ok = __all_sync(0xffffffffu, mbar_wait(acc_full, (uint32_t)nu & 1, a.status, a.wait_polls));
        if (!ok) break;
        tc_fence_after();
      }
#pragma unroll 1
      for (int cc = 0; cc < D / kNG / 16; ++cc) {
        uint32_t x[16];
        const int dim = c * (D / kNG) + cc * 16;
        if (any) {
          tmem_ld16(base + C::kDQ + dim, x);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] = 0;
        }
        if (i >= T) continue;
        if (a.splits > 1) {
          float* dst = a.part + ((size_t)it * 128 + r) * D + dim;
#pragma unroll
          for (int e = 0; e < 16; e += 8) {
            const uint32_t y[8] = {x[e], x[e + 1], x[e + 2], x[e + 3],
                                   x[e + 4], x[e + 5], x[e + 6], x[e + 7]};
            stg256(dst + e, y);
          }
          continue;
        }
        uint4* dst = reinterpret_cast<uint4*>(
            a.dq + (((size_t)d.b * T + i) * a.s.H + d.h) * D + dim);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float f[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) f[k] = __uint_as_float(x[8 * e + k]) * a.s.scale;
          dst[e] = make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                              pack_bf16(f[6], f[7]));
        }
      }
      if (any) {
        tc_fence_before();
        mbar_arrive(acc_empty);
        ++nu;
      }
    }
    if (!ok) *abort_flag = 1;
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kAW) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// dQ of items in several splits: their sums in order.  A thread per 4 dims of a row.
template <int D>
__global__ void __launch_bounds__(256) bwd_q_join_kernel(const __grid_constant__ BwdQArgs a) {
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = e / (D / 4);
  if (row >= (int64_t)a.nitems * 128) return;
  const int item = (int)(row / 128), r = (int)(row % 128), dim = (int)(e % (D / 4)) * 4;
  const QItem d = q_item(a, item * a.splits);
  const int i = d.qt * 128 + r;
  if (i >= a.s.T) return;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int k = 0; k < a.splits; ++k) {
    const float4 y = __ldcs(reinterpret_cast<const float4*>(
        a.part + (((size_t)item * a.splits + k) * 128 + r) * D + dim));
    x.x += y.x;
    x.y += y.y;
    x.z += y.z;
    x.w += y.w;
  }
  const float f = a.s.scale;
  *reinterpret_cast<uint2*>(a.dq + (((size_t)d.b * a.s.T + i) * a.s.H + d.h) * D + dim) =
      make_uint2(pack_bf16(x.x * f, x.y * f), pack_bf16(x.z * f, x.w * f));
}

template <int D>
cudaError_t launch_q(const BwdQArgs& a, const AttnBwd& t, cudaStream_t st) {
  using C = QCfg<D>;
  const Shape& s = a.s;
  CUtensorMap tm_q, tm_o, tm_k, tm_v;
  {
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
  cudaError_t e = cudaFuncSetAttribute(bwd_q_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       C::kSmem);
  if (e != cudaSuccess) return e;
  const int ctas = sm_count();
  const int64_t items = (int64_t)a.nitems * a.splits;
  note_launches(1);
  bwd_q_kernel<D><<<(unsigned)(items < ctas ? items : ctas), kThreadsQ, C::kSmem, st>>>(
      tm_q, tm_o, tm_k, tm_v, a);
  if (a.splits > 1) {
    note_launches(1);
    bwd_q_join_kernel<D><<<(unsigned)(((int64_t)a.nitems * 128 * (D / 4) + 255) / 256), 256, 0, st>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_bwd_q(const BwdQArgs& a, const AttnBwd& t, cudaStream_t st) {
  return a.s.D == 128 ? launch_q<128>(a, t, st) : launch_q<64>(a, t, st);
}

}  // namespace msa

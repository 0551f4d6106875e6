// dQ of the dense attention's backward pass on tensor cores, query-outer (the CTAs of
// msa_bwd_kv_tc.cu's dense kernel that are not KV-outer ones): an item is a
// 128-query tile of one head (or a split of its key blocks, where there are few items),
// whose dQ stays in tensor memory over the key blocks,
//     S = Q K^T   dP = dO V^T   dS = 2^(S scale log2e - lse log2e) (dP - delta)
//     dQ += dS K
// with the queries on the 128 lanes.  Q and dS are A operands in tensor memory, so that of
// the products' operands only dO, and K and V as they stream by, are read from shared
// memory: 128 KB a block at D = 128 and 64 written, as many cycles as the MMAs take (with
// Q in shared memory too and dS over S one sequence of 16K tokens took 4 % longer).  K is
// read K-major by S and MN-major by dQ.  4 x 2048 tokens, 48/8 heads: 282 us alone, the tensor
// pipe at 0.50 of its cycles; what it waits for is the softmax of a block, as a second S
// does not fit into tensor memory at D = 128.
//   warp 0       TMA of the item's dO; takes the items from a shared counter
//   warp 1       TMA of K (four stages at D = 128: a block is read from S, two blocks ahead,
//                to dQ) and V (two)
//   warp 2       tcgen05.mma: once dS(n) is made dP(n+1), dQ(n), and S(n+2), as S(n+1) has
//                been read by then
//   warp 3       waits for the copies in the MMA warp's place
//   warps 4-19   Q into tensor memory; dS: four warpgroups, 32 keys of a block each; an
//                item's dQ
// The two numbers of a row (lse, delta) stay in registers over an item.
#pragma once
#include <type_traits>

#include "msa_bwd.h"
#include "msa_q8.cuh"
#include "msa_tma.h"

namespace msa {
namespace {
namespace dq {

constexpr int kMmaW = 2, kWaitW = 3, kSoftW = 4;
constexpr int kNG = 4;                    // warpgroups for dS ...
constexpr int kCols = 128 / kNG;          // ... and the keys of a block that each has
constexpr int kThreadsQ = 32 * (kSoftW + 4 * kNG);
constexpr int kRing = 4, kReaders = 3 + 4 * kNG;

template <int D>
struct QCfg {
  static constexpr int kNHalf = D / 64;
  static constexpr int kHalf = 128 * 128;
  static constexpr int kTile = kNHalf * kHalf;
  static constexpr int kKS = D == 128 ? 4 : 8, kVS = D == 128 ? 2 : 4;   // stages of K and V
  static constexpr int kSmem = (1 + kKS + kVS) * kTile + 512;
  // tensor memory columns: S, dP, dQ; two bf16 a column: dS, Q
  static constexpr uint32_t kS = 0, kP = 128, kDQ = 256, kDS = 384, kQ = 448;
  static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
};

// Items heaviest first: query tiles from the last down; the heads of a group together.
struct QItem {
  int b, h, g, qt, kb0, kb1;     // key blocks [kb0, kb1)
};
__device__ __forceinline__ QItem q_item(const BwdArgs& a, int it) {
  QItem d;
  const int split = it % a.q_splits;
  int r = it / a.q_splits;
  const int per = a.s.B * a.s.H;
  d.qt = a.nqt - 1 - r / per;
  r %= per;
  d.b = r / a.s.H;
  d.h = r % a.s.H;
  d.g = d.h / (a.s.H / a.s.G);
  const int i_last = min(a.s.T - 1, d.qt * 128 + 127);
  const int n = (int)(((int64_t)a.pos.q_start[d.b] + i_last) / kBlock) + 1;
  d.kb0 = (int)((int64_t)n * split / a.q_splits);
  d.kb1 = (int)((int64_t)n * (split + 1) / a.q_splits);
  return d;
}

template <int D>
__device__ __forceinline__ void q_cta(const CUtensorMap& tm_o, const CUtensorMap& tm_k,
                                      const CUtensorMap& tm_v, const BwdArgs& a) {
  using C = QCfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sO = smem;
  uint8_t* sK = sO + C::kTile;                     // [kKS]
  uint8_t* sV = sK + C::kKS * C::kTile;            // [kVS]
  uint64_t* o_full = reinterpret_cast<uint64_t*>(sV + C::kVS * C::kTile);
  uint64_t* o_empty = o_full + 1;
  uint64_t* k_full = o_empty + 1;                  // [kKS]
  uint64_t* k_empty = k_full + C::kKS;
  uint64_t* v_full = k_empty + C::kKS;             // [kVS]
  uint64_t* v_empty = v_full + C::kVS;
  uint64_t* q_full = v_empty + C::kVS;             // the item's Q is in tensor memory
  uint64_t* s_full = q_full + 1;                   // S of the block
  uint64_t* s_read = s_full + 1;
  uint64_t* dp_full = s_read + 1;                  // dP of the block
  uint64_t* ds_full = dp_full + 1;                 // dP read, dS written; next K and V landed
  uint64_t* ds_read = ds_full + 1;                 // its dQ product is done
  uint64_t* first = ds_read + 1;                   // the item's first copies landed
  uint64_t* acc_full = first + 1;                // the item's dQ is complete
  uint64_t* acc_empty = acc_full + 1;              // ... and read out
  uint64_t* bar_fin = acc_empty + 1;
  uint64_t* it_full = bar_fin + 1;                 // [kRing]
  uint64_t* it_empty = it_full + kRing;
  int* ring = reinterpret_cast<int*>(it_empty + kRing);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ring + kRing);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(o_full, 1);
    mbar_init(o_empty, 1);
    for (int i = 0; i < C::kKS; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < C::kVS; ++i) {
      mbar_init(&v_full[i], 1);
      mbar_init(&v_empty[i], 1);
    }
    mbar_init(q_full, 4 * kNG);     // one arrival a warp
    mbar_init(s_full, 1);
    mbar_init(s_read, 4 * kNG);
    mbar_init(dp_full, 1);
    mbar_init(ds_full, 4 * kNG + 1);
    mbar_init(first, 1);
    mbar_init(ds_read, 1);
    mbar_init(acc_full, 1);
    mbar_init(acc_empty, 4 * kNG);
    mbar_init(bar_fin, 1);
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&it_full[i], 1);
      mbar_init(&it_empty[i], kReaders);
    }
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_o);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == kMmaW) tmem_alloc(tmem_slot, 512);
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
                                                               a.status, a.q_wait_polls));
    if (!ok) return false;
    // read by every lane before the slot is handed back
    it = __shfl_sync(0xffffffffu, ring[slot], 0);
    if (lane == 0) mbar_arrive(&it_empty[slot]);
    ++ki;
    return it >= 0;
  };
  auto wait_all = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, a.status, a.q_wait_polls));
  };
  // One arrival for the lanes' work so far.
  auto warp_arrive = [&](uint64_t* bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };

  if (warp == 0) {
    // ----------------------------------------------------------- dO (warp 0)
    if (lane == 0) {
      const uint64_t pol = l2_policy_evict_first();
      int cur = atomicAdd(a.next_item, 1);
      if (cur >= a.q_items * a.q_splits) cur = -1;
      ring[0] = cur;
      mbar_arrive(&it_full[0]);
      int n = 0;                 // items with key blocks, loaded
      bool ok = true;
      for (int k = 0; cur >= 0; ++k) {
        // publish the next item before this one's tiles, so that its K and V can start
        const int r = k + 1, slot = r % kRing;
        if (r >= kRing && !mbar_wait(&it_empty[slot], ((r / kRing) - 1) & 1, a.status, a.q_wait_polls)) {
          ok = false;
          break;
        }
        int nx = *abort_flag ? a.q_items * a.q_splits : atomicAdd(a.next_item, 1);
        if (nx >= a.q_items * a.q_splits) nx = -1;
        ring[slot] = nx;
        mbar_arrive(&it_full[slot]);
        const QItem d = q_item(a, cur);
        if (d.kb0 < d.kb1) {
          if (n > 0 && !mbar_wait(o_empty, (uint32_t)(n - 1) & 1, a.status, a.q_wait_polls)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(o_full, C::kTile);
#pragma unroll
          for (int hf = 0; hf < C::kNHalf; ++hf)
            tma_load_4d_hint(smem_u32(sO + hf * C::kHalf), &tm_o, o_full, hf * 64, d.h, d.qt * 128,
                             d.b, pol);
          ++n;
        }
        cur = nx;
      }
      if (!ok) *abort_flag = 1;
      // no copy may still be landing when the CTA exits
      if (n > 0) mbar_wait(o_full, (uint32_t)(n - 1) & 1, nullptr);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------- K and V (warp 1)
    int it, n = 0;
    const int late = a.late_q;
    bool ok, k_only = false;     // k_only: block n's K is on its way, its V is not
    while (next_item(it, ok)) {
      const QItem d = q_item(a, it);
      for (int kb = d.kb0; kb < d.kb1; ++kb, ++n) {
        const int ks = n % C::kKS, vs = n % C::kVS;
        const int row = (int)(((int64_t)d.b * a.s.max_blocks + kb) * kBlock);
        ok = __any_sync(0xffffffffu, *abort_flag != 0) == 0 &&
             wait_all(&k_empty[ks], ((n / C::kKS) & 1) ^ 1);
        if (!ok) break;
        if (n == late) copy_delay(a.late_ns);
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
  } else if (warp == kMmaW) {
    // ---------------------------------------------------------- MMA (warp 2)
    constexpr uint32_t idesc_s = idesc_bf16(128, 128, false, false);
    constexpr uint32_t idesc_q = idesc_bf16(128, D, false, true);
    const uint64_t od = smem_desc(smem_u32(sO), 16, 1024, kSwizzle128B);
    const uint64_t kd = smem_desc(smem_u32(sK), 16, 1024, kSwizzle128B);
    const uint64_t vd = smem_desc(smem_u32(sV), 16, 1024, kSwizzle128B);
    const uint64_t kmn = smem_desc(smem_u32(sK), C::kHalf, 1024, kSwizzle128B);
    // 16 dims: (j & 3) * 32 bytes within a 64-dim half
    auto dims = [](int j) { return (uint64_t)(((j >> 2) * C::kHalf + (j & 3) * 32) >> 4); };
    auto stage = [](int i) { return (uint64_t)((i * C::kTile) >> 4); };
    // (inside an elected branch)
    auto issue_s = [&](int m) {
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
        tc_mma_f16_ts(tmem + C::kS, tmem + C::kQ + j * 8, kd + stage(m % C::kKS) + dims(j), idesc_s,
                      j > 0 ? 1u : 0u);
      tc_commit(s_full);
    };
    auto issue_dp = [&](int m, bool last) {
      const int vs = m % C::kVS;
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
        tc_mma_f16(tmem + C::kP, od + dims(j), vd + stage(vs) + dims(j), idesc_s, j > 0 ? 1u : 0u);
      tc_commit(dp_full);
      tc_commit(&v_empty[vs]);
      if (last) tc_commit(o_empty);
    };
    int it, n = 0, nu = 0;       // blocks and items (with blocks) so far
    bool ok;
    while (next_item(it, ok)) {
      const QItem d = q_item(a, it);
      const int nt = d.kb1 - d.kb0;
      if (nt == 0) continue;
      // (S and dP of the item before have been read: its last dQ product waited for that)
      ok = wait_all(first, (uint32_t)nu & 1);
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
        issue_s(n);
        issue_dp(n, nt == 1);
      }
      __syncwarp();
      if (nt > 1) {
        ok = wait_all(s_read, (uint32_t)n & 1);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) issue_s(n + 1);
        __syncwarp();
      }
      for (int t = 0; t < nt; ++t, ++n) {
        const int ks = n % C::kKS;
        ok = wait_all(ds_full, (uint32_t)n & 1);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          if (t + 1 < nt) issue_dp(n + 1, t + 2 == nt);    // first: dS(n + 1) waits for it
#pragma unroll
          for (int j = 0; j < 8; ++j)
            tc_mma_f16_ts(tmem + C::kDQ, tmem + C::kDS + j * 8, kmn + stage(ks) + (uint64_t)(j * 128),
                          idesc_q, t > 0 || j > 0 ? 1u : 0u);
          tc_commit(ds_read);
          tc_commit(&k_empty[ks]);
          if (t + 1 == nt) tc_commit(acc_full);
        }
        __syncwarp();
        if (t + 2 < nt) {
          ok = wait_all(s_read, (uint32_t)(n + 1) & 1);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) issue_s(n + 2);
          __syncwarp();
        }
      }
      if (!ok) break;
      ++nu;
    }
    if (!ok && lane == 0) *abort_flag = 1;
    // all MMAs done before tensor memory is released
    if (elect_one()) tc_commit(bar_fin);
    __syncwarp();
    mbar_wait(bar_fin, 0, nullptr);
  } else if (warp == kWaitW) {
    // ---------------------------------------------- the MMA warp's waits (warp 3)
    // A wait takes a warp 190 cycles even where it is over, and few MMAs are in flight
    // behind an issue: this warp waits for the copies, and arrives with the softmax warps.
    int it, n = 0, nu = 0;
    bool ok;
    while (next_item(it, ok)) {
      const QItem d = q_item(a, it);
      const int nt = d.kb1 - d.kb0;
      if (nt == 0) continue;
      const int64_t t_last = (int64_t)a.pos.q_start[d.b] + T - 1;
      auto wait_k = [&](int m, int t) {          // K of block m, the item's t-th
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
        return true;
      };
      auto wait_v = [&](int m) {
        return wait_all(&v_full[m % C::kVS], (uint32_t)(m / C::kVS) & 1);
      };
      ok = wait_all(o_full, (uint32_t)nu & 1) && wait_k(n, 0) && (nt == 1 || wait_k(n + 1, 1)) &&
           wait_v(n) && wait_all(q_full, (uint32_t)nu & 1);
      if (!ok) break;
      if (lane == 0) mbar_arrive(first);
      for (int t = 0; t < nt; ++t, ++n) {
        // an arrival must not count for the phase before
        ok = __any_sync(0xffffffffu, *abort_flag != 0) == 0 && (t + 1 >= nt || wait_v(n + 1)) &&
             (t + 2 >= nt || wait_k(n + 2, t + 2)) &&
             (t > 0 || nu == 0 || wait_all(acc_empty, (uint32_t)(nu - 1) & 1)) &&
             (n == 0 || wait_all(ds_full, (uint32_t)(n - 1) & 1));
        if (!ok) break;
        if (lane == 0) mbar_arrive(ds_full);
      }
      if (!ok) break;
      ++nu;
    }
    if (!ok && lane == 0) *abort_flag = 1;
  } else if (warp >= kSoftW) {
    // -------------------------------------------- Q, dS, dQ (warps 4-19)
    // keys kCols c ..; dims c D/kNG .. of Q and dQ
    const int c = (warp - kSoftW) >> 2;
    constexpr int kDims = D / kNG;
    const int quad = warp & 3;
    const int r = quad * 32 + lane;               // query of the tile = TMEM lane
    const uint32_t base = tmem + ((uint32_t)(quad * 32) << 16);
    const float sl = a.s.scale * kLog2e;
    const float2 sl2 = make_float2(sl, sl);
    // An item's Q (this thread's dims of its query) and its row's two numbers are read, and Q
    // is put into tensor memory, before the item ahead is written out: every S of that one
    // is done, as this thread has read the last, and the next item's first products run
    // meanwhile.
    float nl = 0.f, nd = 0.f;
    auto begin = [&](const QItem& d) {
      const int i = d.qt * 128 + r;
      const uint4* src = reinterpret_cast<const uint4*>(
          a.q + (((size_t)d.b * T + (i < T ? i : 0)) * a.s.H + d.h) * D + c * kDims);
      uint4 q[kDims / 8];
#pragma unroll
      for (int k = 0; k < kDims / 8; ++k) q[k] = i < T ? __ldg(src + k) : make_uint4(0, 0, 0, 0);
      const float* st = reinterpret_cast<const float*>(
                            a.nums + ((size_t)(d.b * a.s.H + d.h) * a.stat_groups + (i >> 3)) * kStatBytes) +
                        (i & 7);
      // (past L1: the kernels that write them may still run when this one is launched)
      nl = __ldcg(st);
      nd = __ldcg(st + 8);
      if (d.kb0 == d.kb1) return;
      if constexpr (kDims == 32) {
        const uint32_t w[16] = {q[0].x, q[0].y, q[0].z, q[0].w, q[1].x, q[1].y, q[1].z, q[1].w,
                                q[2].x, q[2].y, q[2].z, q[2].w, q[3].x, q[3].y, q[3].z, q[3].w};
        tmem_st16(base + C::kQ + c * 16, w);
      } else {
        const uint32_t w[8] = {q[0].x, q[0].y, q[0].z, q[0].w, q[1].x, q[1].y, q[1].z, q[1].w};
        tmem_st8(base + C::kQ + c * 8, w);
      }
      tmem_st_wait();
      tc_fence_before();
      warp_arrive(q_full);
    };
    int it, n = 0, nu = 0;
    bool ok, some = next_item(it, ok);
    if (some) begin(q_item(a, it));
    while (some) {
      const QItem d = q_item(a, it);
      const int i = d.qt * 128 + r;
      const int64_t tq = (int64_t)a.pos.q_start[d.b] + i;
      const float2 nl2 = make_float2(nl, nl), nd2 = make_float2(nd, nd);
      const bool any = d.kb0 < d.kb1;
      for (int kb = d.kb0; kb < d.kb1; ++kb, ++n) {
        // keys past the query, and rows past the last query, whatever they hold
        const int64_t l64 = min(tq, (int64_t)a.pos.q_start[d.b] + T - 1) - (int64_t)kb * kBlock;
        const int lim = (int)(l64 < kBlock ? l64 : kBlock) - c * kCols;
        const bool masked = __any_sync(0xffffffffu, lim < kCols - 1);
        ok = __all_sync(0xffffffffu, *abort_flag == 0 && mbar_wait(s_full, (uint32_t)n & 1, a.status,
                                                                   a.q_wait_polls));
        if (!ok) break;
        tc_fence_after();
        float2 p[kCols / 2];
        {
          uint32_t x[32];
          tmem_ld32(base + C::kS + c * kCols, x);
          tmem_ld_wait();
          tc_fence_before();
          warp_arrive(s_read);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 y = ffma2(make_float2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])),
                                   sl2, nl2);
            p[e] = make_float2(ex2(y.x), ex2(y.y));
          }
        }
        ok = __all_sync(0xffffffffu, mbar_wait(dp_full, (uint32_t)n & 1, a.status, a.q_wait_polls));
        if (!ok) break;
        tc_fence_after();
        uint32_t w[16];
        auto ds_of = [&](auto mask) {
          uint32_t x[32];
          tmem_ld32(base + C::kP + c * kCols, x);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float2 y = fadd2(make_float2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), nd2);
            y = fmul2(p[e], y);
            if constexpr (mask.value) {
              y.x = 2 * e <= lim ? y.x : 0.f;
              y.y = 2 * e + 1 <= lim ? y.y : 0.f;
            }
            w[e] = pack_bf16(y.x, y.y);
          }
        };
        if (masked) ds_of(std::true_type());
        else ds_of(std::false_type());
        ok = __all_sync(0xffffffffu, n == 0 || mbar_wait(ds_read, (uint32_t)(n - 1) & 1, a.status,
                                                         a.q_wait_polls));
        if (!ok) break;
        tmem_st16(base + C::kDS + c * (kCols / 2), w);
        tmem_st_wait();
        tc_fence_before();
        warp_arrive(ds_full);
      }
      if (!ok) break;
      const int done = it;
      some = next_item(it, ok);
      if (!ok) break;
      if (some) begin(q_item(a, it));
      // ---- the item's dQ: a query per thread, a run of dims per warpgroup
      if (any) {
        ok = __all_sync(0xffffffffu, mbar_wait(acc_full, (uint32_t)nu & 1, a.status, a.q_wait_polls));
        if (!ok) break;
        tc_fence_after();
      }
#pragma unroll 1
      for (int cc = 0; cc < kDims / 16; ++cc) {
        uint32_t x[16];
        const int dim = c * kDims + cc * 16;
        if (any) {
          tmem_ld16(base + C::kDQ + dim, x);
          tmem_ld_wait();
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] = 0;
        }
        if (i >= T) continue;
        if (a.q_splits > 1) {
          float* dst = a.part_q + ((size_t)done * 128 + r) * D + dim;
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
        warp_arrive(acc_empty);
        ++nu;
      }
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

// dQ of items in several splits: their sums in order.  A thread per 4 dims of a row.
template <int D>
__global__ void __launch_bounds__(256) bwd_q_join_kernel(const __grid_constant__ BwdArgs a) {
  after_previous();
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = e / (D / 4);
  if (row >= (int64_t)a.q_items * 128) return;
  const int item = (int)(row / 128), r = (int)(row % 128), dim = (int)(e % (D / 4)) * 4;
  const QItem d = q_item(a, item * a.q_splits);
  const int i = d.qt * 128 + r;
  if (i >= a.s.T) return;
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int k = 0; k < a.q_splits; ++k) {
    const float4 y = __ldcs(reinterpret_cast<const float4*>(
        a.part_q + (((size_t)item * a.q_splits + k) * 128 + r) * D + dim));
    x.x += y.x;
    x.y += y.y;
    x.z += y.z;
    x.w += y.w;
  }
  const float f = a.s.scale;
  *reinterpret_cast<uint2*>(a.dq + (((size_t)d.b * a.s.T + i) * a.s.H + d.h) * D + dim) =
      make_uint2(pack_bf16(x.x * f, x.y * f), pack_bf16(x.z * f, x.w * f));
}

}  // namespace dq
}  // namespace
}  // namespace msa

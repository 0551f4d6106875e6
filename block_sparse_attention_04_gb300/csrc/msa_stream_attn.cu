// Streaming attention over cached blocks: a caller's selection on an 8-bit
// cache (msa_sparse_attn_q8) and a sliding window with sinks on either cache
// (msa_window_attn, msa_window_attn_q8), for decode-sized calls; any shape.
//
// Mathematics: for query (b, t) and head h of KV group g, over the visible
// tokens j of the unit's blocks, s_j = scale q.k_j, o = sum 2^(x_j - m) v_j /
// sum 2^(x_j - m) with x = s log2(e).  An 8-bit cache holds k = ck 2^ek and
// v = cv 2^ev (ck, cv e4m3 codes, one exponent per block and KV head): ek
// scales the block's scores, and 2^ev is folded into the exponential that
// multiplies V, p'_j = 2^(x_j + ev - m') with m' the running maximum of x + ev.
// The normaliser keeps its own exponentials and maximum, l = sum 2^(x_j - n):
// a block of zeros has the smallest ev, and p' of it would vanish beside other
// blocks while its weights count.  The result is O / l * 2^(m' - n).
//
// The call's work is one sequence of (query, block) steps, query (b, t) after
// query, cut into equal runs; G CTAs take a run, one KV head each, and a run's
// share of one query is a segment.  The last warp copies K and V of each block
// (128 tokens of one KV head) into a ring of stages by TMA and runs ahead by its depth.  A team of eight warps
// takes a block, 16 tokens each, and its warps never wait for one another inside
// a segment:
// S^T = K Q^T (tokens x heads) with mma.sync m16n8k16, softmax in registers,
// P^T transposed inside the warp into the B operand of O^T += V^T P^T.  The
// order of the contraction's terms is free, so dims are dealt to threads such
// that every thread reads whole 16-byte chunks of the swizzled rows; pairs of
// tokens of V are put together with byte permutes.  e4m3 codes of K become f16
// (exact), Q is scaled by a power of two per row to fit f16 (exact but for
// elements 2^-27 below the row's maximum, which round at 2^-38 of it).  Codes
// of V become bf16 (exact), like P (2^-8): the largest p' may belong to values
// that cancel or vanish, so the others need bf16's range.
// At a segment's end all warps' (O, m, l) are joined in shared memory; a
// whole unit is written out directly, a cut one leaves a partial per CTA (at
// most two: the unit its run begins inside, the one it ends inside) that
// stream_finish_kernel joins.  Small calls, where a launch counts, give every
// unit a cluster of CTAs instead, which joins its parts through distributed
// shared memory.
//
// Bound by HBM for decode: 64 sequences, a bf16 window of 4096 tokens and 4
// sinks, G 8, D 128: 161 us against 155 for its bytes at the 6.78 TB/s of a plain
// copy (167 us when the heads of a block, whose rows lie side by side, were read
// by CTAs at different times).  An 8-bit cache needs as long
// for its arithmetic as for its bytes: 4 sequences of 64K tokens 79 us (copies
// alone 71, arithmetic alone 68, bytes 65); 64 selections of 16 blocks, of which
// every group has its own, in pieces of 128 bytes 1 KB apart, 60 us (55, 56 and
// 40).  f16 weights and values, whose conversion takes fewer instructions but
// whose weights need a maximum per 16 tokens, took 83 and 66 us; three teams of
// four warps with 32 tokens each 90 and 68 us.
#include "msa_q8.cuh"
#include "msa_tma.h"

namespace msa {
namespace {

constexpr int kTeam = 8;             // consumer warps that share a block, 16 tokens each
// Teams: the blocks of an 8-bit cache take more instructions per byte, and two
// teams on alternate blocks hide their latency (measured, 4 x 64K tokens, before
// the heads of a run went together: one team 116 us, two 108 us); a bf16 cache keeps HBM busy with one.
template <bool Q8, int NTH>
constexpr int teams() { return Q8 && NTH == 1 ? 2 : 1; }
constexpr int kQBufs = 2;
constexpr int kMaxStages = 8;
constexpr int kMaxCtas = kMaxStatusWords;        // partials and error words in the workspace
constexpr int kPassRows = 2048;      // (sequence, query) rows per pass
constexpr float kLazy = 8.f;         // log2 growth of p tolerated before O is rescaled
// Most dynamic shared memory of a CTA: 227 KiB but for the static part (barriers,
// row statistics: under 2 KiB).
constexpr int kSmemMax = 227 * 1024 - 2048;

struct StreamArgs {
  Shape s;
  int32_t q_start[kMaxBatch];
  int32_t step0[kMaxBatch + 1];   // first step of each sequence; [B]: all steps
  int t0, Tp, nruns, stages;
  int window, sinks;
  const int32_t* sel;
  const uint16_t* q;
  const int8_t* k_exp;
  const int8_t* v_exp;
  float* part_o;                  // [2 * CTA + slot][H/G][D], O relative to m
  float4* part_ml;                // [2 * CTA + slot][H/G] (m, n in log2 units, l)
  uint16_t* out;
  int* errs;                      // [nctas]
  int* status;
  bool first_pass;
  int parts;                      // > 0: a cluster of this many CTAs per unit
  uint32_t wait_polls;
};

// Run r begins at step floor(r * steps / nruns); CTA r * G + g takes its KV head g.
__host__ __device__ __forceinline__ int run_begin(int steps, int nruns, int r) {
  return (int)((int64_t)r * steps / nruns);
}
__device__ __forceinline__ int run_of(int steps, int nruns, int step) {
  return (int)((((int64_t)step + 1) * nruns - 1) / steps);
}

// A unit: a query and a KV head; the query's first step and its steps (the
// longest list of its sequence in this pass).
struct Unit {
  int b, i, g, t, first, len;
};

__device__ __forceinline__ Unit unit_of(const StreamArgs& a, int step, int g) {
  int lo = 0, hi = a.s.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.step0[mid] <= step) lo = mid; else hi = mid;
  }
  Unit u;
  u.b = lo;
  u.len = (a.step0[lo + 1] - a.step0[lo]) / a.Tp;
  const int i = (step - a.step0[lo]) / u.len;
  u.first = a.step0[lo] + i * u.len;
  u.g = g;
  u.i = a.t0 + i;
  u.t = a.q_start[lo] + u.i;
  return u;
}

// The segment of a CTA in cluster form: part `rank` of unit blockIdx.x / parts
// (units in order of sequence, query, group), list positions [p0, p1).
__device__ __forceinline__ Unit unit_of_cluster(const StreamArgs& a) {
  Unit u;
  const int unit = (int)blockIdx.x / a.parts;
  u.g = unit % a.s.G;
  u.i = unit / a.s.G % a.Tp;
  u.b = unit / a.s.G / a.Tp;
  u.t = a.q_start[u.b] + u.i;
  return u;
}

// The blocks of a unit's list: all 16 slots of a selection, or the blocks
// that hold a visible token (sink blocks first).
struct BlockList {
  int len, nsink, first;          // window: list position p is block p (p < nsink) or first + p
};
__device__ __forceinline__ BlockList list_of(const StreamArgs& a, int t) {
  if (a.sel) return BlockList{kTopk, 0, 0};
  const int lo = max(0, t - a.window + 1) / kBlock;
  const int ns = min((a.sinks + kBlock - 1) / kBlock, lo);
  return BlockList{ns + t / kBlock - lo + 1, ns, lo - ns};
}

template <int D, bool Q8, int NTH>
struct Cfg {
  static constexpr int kTeams = teams<Q8, NTH>();
  static constexpr int kWarps = kTeam * kTeams;
  static constexpr int kConsumers = 32 * kWarps;
  static constexpr int kThreads = kConsumers + 32;          // and the producer warp
  static constexpr int kTile = kBlock * D * (Q8 ? 1 : 2);   // K (or V) of one block and head
  static constexpr int kStage = 2 * kTile;
  static constexpr int kRedRow = D + 4;                     // padded row of the join buffer (floats)
};

template <int D, bool Q8, int NTH>
__global__ void __launch_bounds__(Cfg<D, Q8, NTH>::kThreads, 1) stream_attn_kernel(
    const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
    const __grid_constant__ StreamArgs a) {
  using C = Cfg<D, Q8, NTH>;
  constexpr int kWarps = C::kWarps, kConsumers = C::kConsumers;
  constexpr int NS = D / 16;       // k-steps of S
  constexpr int MT = D / 16;       // m-tiles of O^T
  extern __shared__ uint8_t dsm_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(dsm_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], q_full[kQBufs], q_empty[kQBufs];
  __shared__ int2 meta[kMaxStages];       // block (-1: none), exponents ek and ev * 2^16
  __shared__ float sm_m[kWarps][NTH * 8], sm_n[kWarps][NTH * 8], sm_l[kWarps][NTH * 8];
  __shared__ int err;
  const Shape& s = a.s;
  const int H = s.H, G = s.G, hpg = H / G, S = a.stages;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint16_t* qbuf = reinterpret_cast<uint16_t*>(sm + S * C::kStage);       // [kQBufs][hpg][D]
  const uint32_t red = smem_u32(qbuf + kQBufs * hpg * D);                 // [kWarps][hpg][kRedRow] float
  const int steps = a.step0[s.B];
  // steps of this CTA; in cluster form one segment, numbered from 0
  const int run = (int)blockIdx.x / G;
  const int run0 = a.parts ? 0 : run_begin(steps, a.nruns, run);
  const int run1 = a.parts ? 1 : run_begin(steps, a.nruns, run + 1);
  // the segment that begins at `step`: its unit and list positions; the next step
  auto segment = [&](int step, Unit& u, BlockList& bl, int& p0, int& p1) -> int {
    if (a.parts) {
      u = unit_of_cluster(a);
      bl = list_of(a, u.t);
      const int rank = (int)blockIdx.x % a.parts;
      p0 = rank * bl.len / a.parts;
      p1 = (rank + 1) * bl.len / a.parts;
      return 1;
    }
    u = unit_of(a, step, (int)blockIdx.x % G);
    bl = list_of(a, u.t);
    const int next = min(run1, u.first + u.len);
    p0 = step - u.first;
    p1 = min(next - u.first, bl.len);
    return next;
  };

  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kTeam);
    }
    for (int i = 0; i < kQBufs; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], kWarps);
    }
    err = 0;
    fence_mbar_init();
  }
  __syncthreads();

  if (warp == kWarps) {
    // ------------------------------------------------------------ producer
    const uint64_t pol = l2_policy_evict_first();
    const uint32_t qbytes = (uint32_t)(hpg * D * 2);
    int st = 0, k = 0;              // next stage, segments begun
    uint32_t ph = 1;                // phase parity that frees the stage (first lap: free)
    uint32_t used = 0, loaded = 0;  // stages ever loaded / parity of each stage's last load
    int nq = 0;
    bool ok = true;
    for (int step = run0, next; step < run1 && ok; step = next, ++k) {
      Unit u;
      BlockList bl;
      int p0, p1;
      next = segment(step, u, bl, p0, p1);
      const int qs = k % kQBufs;
      ok = __all_sync(0xffffffffu, k < kQBufs || mbar_wait(&q_empty[qs], ((k / kQBufs) - 1) & 1,
                                                           &err, a.wait_polls));
      if (!ok) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&q_full[qs], qbytes);
        bulk_load(smem_u32(qbuf + qs * hpg * D),
                  a.q + (((int64_t)u.b * s.T + u.i) * H + (int64_t)u.g * hpg) * D, qbytes,
                  &q_full[qs]);
      }
      ++nq;
      const int32_t* srow =
          a.sel ? a.sel + (((int64_t)u.b * s.T + u.i) * G + u.g) * kTopk : nullptr;
      for (int pc = p0; pc < p1 && ok; pc += 32) {
        // one list position per lane: its block, cache block and exponents
        int kb = -1, ex = 0, row = 0;
        const int p = pc + lane;
        if (p < p1) {
          kb = srow ? srow[p] : (p < bl.nsink ? p : bl.first + p);
          if (srow && kb >= 0 && (kb > u.t / kBlock || kb >= s.max_blocks)) {
            flag_invalid(&err);
            kb = -1;
          }
          if (kb >= 0) {
            const int64_t pb = cache_block(s, u.b, kb, &err);
            // an entry outside the pool (flagged) reads zeros from past its end
            row = (int)((pb < 0 ? s.cache_blocks() : pb) * kBlock);
            if (Q8 && pb >= 0) {
              ex = (clamp_exp(a.k_exp[pb * G + u.g]) & 0xFFFF) |
                   clamp_exp(a.v_exp[pb * G + u.g]) * 65536;
            }
          }
        }
        const int n = min(32, p1 - pc);
        for (int j = 0; j < n; ++j) {
          const int kbj = __shfl_sync(0xffffffffu, kb, j), rowj = __shfl_sync(0xffffffffu, row, j);
          const int exj = __shfl_sync(0xffffffffu, ex, j);
          ok = __all_sync(0xffffffffu, mbar_wait(&empty[st], ph, &err, a.wait_polls));
          if (!ok) break;
          if (lane == 0) {
            meta[st] = make_int2(kbj, exj);
            if (kbj < 0) {
              mbar_arrive(&full[st]);
            } else {
              mbar_arrive_expect_tx(&full[st], C::kStage);
              const uint32_t kd = smem_u32(sm + st * C::kStage), vd = kd + C::kTile;
              if constexpr (Q8) {
                tma_load_3d_hint(kd, &tm_k, &full[st], 0, u.g, rowj, pol);
                tma_load_3d_hint(vd, &tm_v, &full[st], 0, u.g, rowj, pol);
              } else {
#pragma unroll
                for (int h = 0; h < D / 64; ++h) {
                  tma_load_3d_hint(kd + h * 16384, &tm_k, &full[st], h * 64, u.g, rowj, pol);
                  tma_load_3d_hint(vd + h * 16384, &tm_v, &full[st], h * 64, u.g, rowj, pol);
                }
              }
            }
          }
          used |= 1u << st;
          loaded = (loaded & ~(1u << st)) | ((ph ^ 1u) << st);
          if (++st == S) {
            st = 0;
            ph ^= 1;
          }
        }
      }
    }
    // no copy may still be landing when the CTA exits (wall-clock bound only)
    if (lane == 0) {
      for (int i = 0; i < S; ++i)
        if (used >> i & 1) mbar_wait(&full[i], (loaded >> i) & 1, nullptr);
      for (int m = nq - 1; m >= 0 && m >= nq - kQBufs; --m)
        mbar_wait(&q_full[m % kQBufs], (m / kQBufs) & 1, nullptr);
    }
    __syncwarp();
  } else {
    // ----------------------------------------------------------- consumers
    // S^T = K Q^T (tokens x heads) and O^T += V^T P^T (dims x heads)
    const int g4 = lane >> 2, t4 = lane & 3;   // row group and column pair of a fragment
    const float qk = s.scale * kLog2e;
    const int wt = warp % kTeam;               // this warp's 16 tokens of a block
    int st = warp / kTeam, k = 0;              // the team's next stage
    int turn = st;                             // blocks before its next one
    uint32_t ph = 0;
    bool ok = true;
    for (int step = run0, next; step < run1; step = next, ++k) {
      Unit u;
      BlockList bl;
      int p0, p1;
      next = segment(step, u, bl, p0, p1);
      const int nblk = max(0, p1 - p0);   // 0: a run past the end of a shorter list
      const int lo = a.sel ? 0 : max(0, u.t - a.window + 1);   // visible: j <= t and
      const int sinks = a.sel ? 0 : a.sinks;                   // (j >= lo or j < sinks)
      const int qs = k % kQBufs;
      ok = __all_sync(0xffffffffu,
                      ok && mbar_wait(&q_full[qs], (k / kQBufs) & 1, &err, a.wait_polls));
      // Q^T fragments: head nt * 8 + g4, per k-step the four dims that this
      // thread's 16-byte chunks of a K row hold (see the reads of K below)
      uint32_t qb[NTH][NS][2];
      float fq[NTH][2];                // score factors of heads nt * 8 + 2 t4 + {0, 1}
#pragma unroll
      for (int nt = 0; nt < NTH; ++nt) {
        const int h = nt * 8 + g4;
        const uint32_t qrow = smem_u32(qbuf + (qs * hpg + min(h, hpg - 1)) * D);
#pragma unroll
        for (int ks = 0; ks < NS; ++ks) {
          int dim;
          if constexpr (Q8)
            dim = D == 128 ? (2 * t4 + (ks >> 2)) * 16 + (ks & 3) * 4 : t4 * 16 + ks * 4;
          else
            dim = (ks >> 2) * 64 + (2 * t4 + ((ks >> 1) & 1)) * 8 + (ks & 1) * 4;
          const uint2 w = h < hpg && ok ? lds64(qrow + dim * 2) : make_uint2(0, 0);
          qb[nt][ks][0] = w.x;
          qb[nt][ks][1] = w.y;
        }
        float f = qk;
        if constexpr (Q8) {
          // scale the row by a power of two: its largest magnitude to [2^13, 2^14)
          uint32_t mx = 0;
#pragma unroll
          for (int ks = 0; ks < NS; ++ks)
#pragma unroll
            for (int x = 0; x < 2; ++x)
              mx = max(max(mx, qb[nt][ks][x] & 0x7FFFu), qb[nt][ks][x] >> 16 & 0x7FFFu);
          mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          int e = (int)(mx >> 7) - 127;                   // floor(log2 max); inf, NaN: 128
          e = mx == 0 || e == 128 ? 0 : max(e, -100);
          const float up = pow2i(13 - e);
          f = qk * pow2i(e - 13);
#pragma unroll
          for (int ks = 0; ks < NS; ++ks)
#pragma unroll
            for (int x = 0; x < 2; ++x)
              qb[nt][ks][x] = pack_f16(bf16lo(qb[nt][ks][x]) * up, bf16hi(qb[nt][ks][x]) * up);
        }
        fq[nt][0] = __shfl_sync(0xffffffffu, f, 8 * t4);       // a lane of head 2 t4
        fq[nt][1] = __shfl_sync(0xffffffffu, f, 8 * t4 + 4);
      }
      // O^T: rows (dims) 2j and 2j + 1 of this thread's chunk of V, heads 2 t4 + {0, 1}
      float o[NTH][MT][4];
#pragma unroll
      for (int nt = 0; nt < NTH; ++nt)
#pragma unroll
        for (int j = 0; j < MT; ++j)
#pragma unroll
          for (int c = 0; c < 4; ++c) o[nt][j][c] = 0.f;
      // per head, the same in all lanes of a column: running maxima of x + ev
      // (of O's terms) and x (of l's; the same without ev); l: this thread's tokens
      float m[NTH][2], n[NTH][2], l[NTH][2];
#pragma unroll
      for (int nt = 0; nt < NTH; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          m[nt][e] = n[nt][e] = -INFINITY;
          l[nt][e] = 0.f;
        }

      for (; turn < nblk; turn += C::kTeams) {
        ok = __all_sync(0xffffffffu, ok && mbar_wait(&full[st], ph, &err, a.wait_polls));
        if (!ok) break;
        const int2 mt = meta[st];
        const int kb = mt.x;
        if (kb >= 0) {
          const int tok0 = kb * kBlock;
          const int w0 = tok0 + wt * 16;              // this warp's first token
          const bool whole = tok0 + kBlock - 1 <= u.t && (tok0 >= lo || tok0 + kBlock - 1 < sinks);
          const bool any = w0 <= u.t && (w0 + 15 >= lo || w0 < sinks);
          if (any) {
            const uint32_t kbase = smem_u32(sm + st * C::kStage), vbase = kbase + C::kTile;
            // ---- S^T of 16 tokens: rows g4 and g4 + 8
            const int r0 = wt * 16 + g4;                // r0 & 7 == (r0 + 8) & 7
            float sc[NTH][4];
#pragma unroll
            for (int nt = 0; nt < NTH; ++nt)
#pragma unroll
              for (int c = 0; c < 4; ++c) sc[nt][c] = 0.f;
            if constexpr (Q8) {
#pragma unroll
              for (int j = 0; j < D / 64; ++j) {
                const uint32_t at = D == 128 ? kbase + r0 * 128 + (((2 * t4 + j) ^ (r0 & 7)) << 4)
                                             : kbase + r0 * 64 + ((t4 ^ ((r0 >> 1) & 3)) << 4);
                const uint4 x0 = lds128(at), x1 = lds128(at + 8 * D);
                const uint32_t ya[4] = {x0.x, x0.y, x0.z, x0.w}, yb[4] = {x1.x, x1.y, x1.z, x1.w};
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                  uint32_t a0, a1, a2, a3;
                  e4m3x4_to_f16(ya[x], a0, a2);
                  e4m3x4_to_f16(yb[x], a1, a3);
#pragma unroll
                  for (int nt = 0; nt < NTH; ++nt)
                    mma_f16_16816(sc[nt], a0, a1, a2, a3, qb[nt][j * 4 + x][0], qb[nt][j * 4 + x][1]);
                }
              }
            } else {
#pragma unroll
              for (int hj = 0; hj < D / 32; ++hj) {      // 64-dim half, chunk of it
                const uint32_t at = kbase + (hj >> 1) * 16384 + r0 * 128 +
                                    (((2 * t4 + (hj & 1)) ^ (r0 & 7)) << 4);
                const uint4 x0 = lds128(at), x1 = lds128(at + 1024);
#pragma unroll
                for (int nt = 0; nt < NTH; ++nt) {
                  mma_bf16_16816(sc[nt], x0.x, x1.x, x0.y, x1.y, qb[nt][hj * 2][0], qb[nt][hj * 2][1]);
                  mma_bf16_16816(sc[nt], x0.z, x1.z, x0.w, x1.w, qb[nt][hj * 2 + 1][0],
                                 qb[nt][hj * 2 + 1][1]);
                }
              }
            }
            // ---- x = s log2(e), masked; the maxima move only when one grew
            float fk = 1.f, ev = 0.f;
            if constexpr (Q8) {
              fk = pow2i((int16_t)mt.y);
              ev = (float)(mt.y >> 16);
            }
            float mx[NTH][2];
            bool grow = false;
#pragma unroll
            for (int nt = 0; nt < NTH; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float f = Q8 ? fminf(fmaxf(fq[nt][e] * fk, -3e38f), 3e38f) : fq[nt][e];
                sc[nt][e] *= f;
                sc[nt][2 + e] *= f;
                if (!whole) {                             // tokens w0 + g4, w0 + g4 + 8
                  const int tok = w0 + g4;
                  if (!(tok <= u.t && (tok >= lo || tok < sinks))) sc[nt][e] = -INFINITY;
                  if (!(tok + 8 <= u.t && (tok + 8 >= lo || tok + 8 < sinks)))
                    sc[nt][2 + e] = -INFINITY;
                }
                mx[nt][e] = fmaxf(sc[nt][e], sc[nt][2 + e]);
                grow |= mx[nt][e] + ev > m[nt][e] + kLazy || (Q8 && mx[nt][e] > n[nt][e] + kLazy);
              }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
              for (int nt = 0; nt < NTH; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  float x = mx[nt][e];
#pragma unroll
                  for (int w = 4; w < 32; w <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, w));
                  const float mn = fmaxf(m[nt][e], x + ev);
                  const float al = m[nt][e] == -INFINITY ? 0.f : ex2(m[nt][e] - mn);
                  m[nt][e] = mn;
                  if constexpr (Q8) {
                    const float nn = fmaxf(n[nt][e], x);
                    l[nt][e] *= n[nt][e] == -INFINITY ? 0.f : ex2(n[nt][e] - nn);
                    n[nt][e] = nn;
                  } else {
                    l[nt][e] *= al;
                  }
#pragma unroll
                  for (int j = 0; j < MT; ++j) {
                    o[nt][j][e] *= al;
                    o[nt][j][2 + e] *= al;
                  }
                }
            }
            // ---- P^T: p' = 2^(x + ev - m) as bf16, transposed into B fragments
            // (tokens 2 t4, 2 t4 + 1 and 8 + ... of head g4)
            uint32_t pb[NTH][2];
#pragma unroll
            for (int nt = 0; nt < NTH; ++nt) {
              float p[4];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float mr = m[nt][e] == -INFINITY ? 0.f : m[nt][e] - ev;
                p[e] = ex2(sc[nt][e] - mr);
                p[2 + e] = ex2(sc[nt][2 + e] - mr);
                if constexpr (Q8) {
                  const float nr = n[nt][e] == -INFINITY ? 0.f : n[nt][e];
                  l[nt][e] += ex2(sc[nt][e] - nr) + ex2(sc[nt][2 + e] - nr);
                } else {
                  l[nt][e] += p[e] + p[2 + e];
                }
              }
              pb[nt][0] = movmatrix_trans(pack_bf16(p[0], p[1]));
              pb[nt][1] = movmatrix_trans(pack_bf16(p[2], p[3]));
            }
            // ---- V^T: tokens w0 + {2 t4, 2 t4 + 1, 8 + 2 t4, 9 + 2 t4}, the
            // dims of this thread's chunks; rows that the query does not see
            // (they may hold anything) as zeros
            const int v0 = wt * 16 + 2 * t4;
            bool dead[4] = {false, false, false, false};
            if (!whole) {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const int tok = tok0 + v0 + (j >> 1) * 8 + (j & 1);
                dead[j] = !(tok <= u.t && (tok >= lo || tok < sinks));
              }
            }
#pragma unroll
            for (int hb = 0; hb < (Q8 ? 1 : D / 64); ++hb) {    // boxes of a row
              constexpr int W = Q8 ? D / 32 : 4;          // words per token and box
              uint32_t vw[4][W];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const int r = v0 + (j >> 1) * 8 + (j & 1);
                if constexpr (Q8 && D == 64) {
                  const uint2 w = lds64(vbase + r * 64 + (((g4 >> 1) ^ ((r >> 1) & 3)) << 4) +
                                        (g4 & 1) * 8);
                  vw[j][0] = w.x;
                  vw[j][1] = w.y;
                } else {
                  const uint4 w = lds128(vbase + hb * 16384 + r * 128 + ((g4 ^ (r & 7)) << 4));
                  vw[j][0] = w.x;
                  vw[j][1] = w.y;
                  vw[j][W > 2 ? 2 : 0] = w.z;
                  vw[j][W > 2 ? 3 : 0] = w.w;
                }
                if (!whole && dead[j]) {
#pragma unroll
                  for (int x = 0; x < W; ++x) vw[j][x] = 0u;
                }
              }
#pragma unroll
              for (int x = 0; x < W; ++x) {
                if constexpr (Q8) {
#pragma unroll
                  for (int y = 0; y < 2; ++y) {           // dims 4x + 2y, 4x + 2y + 1: m-tile 2x + y
                    const uint32_t pick = y ? 0x7362u : 0x5140u;
                    uint32_t a0, a1, a2, a3;
                    e4m3x4_to_bf16(__byte_perm(vw[0][x], vw[1][x], pick), a0, a1);
                    e4m3x4_to_bf16(__byte_perm(vw[2][x], vw[3][x], pick), a2, a3);
#pragma unroll
                    for (int nt = 0; nt < NTH; ++nt)
                      mma_bf16_16816(o[nt][2 * x + y], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
                  }
                } else {                                  // dims 2x, 2x + 1 of the box's chunk
                  const uint32_t a0 = __byte_perm(vw[0][x], vw[1][x], 0x5410);
                  const uint32_t a1 = __byte_perm(vw[0][x], vw[1][x], 0x7632);
                  const uint32_t a2 = __byte_perm(vw[2][x], vw[3][x], 0x5410);
                  const uint32_t a3 = __byte_perm(vw[2][x], vw[3][x], 0x7632);
#pragma unroll
                  for (int nt = 0; nt < NTH; ++nt)
                    mma_bf16_16816(o[nt][hb * 4 + x], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
                }
              }
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[st]);
        if ((st += C::kTeams) >= S) {
          st -= S;
          ph ^= 1;
        }
      }
      turn -= nblk;
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_empty[qs]);

      // ---- join the warps: O relative to each warp's own m
#pragma unroll
      for (int nt = 0; nt < NTH; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int w = 4; w < 32; w <<= 1)
            l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], w);
      if (!named_bar_and(1, kConsumers, ok)) {   // also: the last segment's sums have been read
        ok = false;
        break;
      }
#pragma unroll
      for (int nt = 0; nt < NTH; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int h = nt * 8 + 2 * t4 + e;
          if (g4 == 0) {
            sm_m[warp][h] = m[nt][e];
            sm_n[warp][h] = Q8 ? n[nt][e] : m[nt][e];
            sm_l[warp][h] = l[nt][e];
          }
          // pairs of dims in fragment order: m-tile j, row group g4
          if (h < hpg) {
            const uint32_t row = red + ((warp * hpg + h) * C::kRedRow + 2 * g4) * 4;
#pragma unroll
            for (int j = 0; j < MT; ++j) sts_f2(row + j * 64, o[nt][j][e], o[nt][j][2 + e]);
          }
        }
      named_bar_sync(1, kConsumers);
      const bool whole_unit = a.parts ? a.parts == 1 : step == u.first && next == u.first + u.len;
      const int64_t slot = 2 * blockIdx.x + (step == u.first);
      for (int e = threadIdx.x; e < hpg * (D / 2); e += kConsumers) {
        const int h = e / (D / 2), pr = e % (D / 2);       // one head per warp and step
        float M = -INFINITY, N = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          M = fmaxf(M, sm_m[w][h]);
          N = fmaxf(N, sm_n[w][h]);
        }
        float L = 0.f, x = 0.f, y = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float mw = sm_m[w][h];
          const float f = mw == -INFINITY ? 0.f : ex2(mw - M);
          const float2 v = lds_f2(red + ((w * hpg + h) * C::kRedRow + pr * 2) * 4);
          const float nw = sm_n[w][h];
          L = fmaf(sm_l[w][h], nw == -INFINITY ? 0.f : ex2(nw - N), L);
          x = fmaf(v.x, f, x);
          y = fmaf(v.y, f, y);
        }
        const int j = pr >> 3, c = pr & 7;                 // m-tile, chunk of V
        const int dim = Q8 ? c * (D / 8) + 2 * j : (j >> 2) * 64 + c * 8 + 2 * (j & 3);
        if (whole_unit) {
          const float inv = L == 0.f ? 0.f : ex2(M - N) / L;      // nothing visible: zeros
          uint16_t* dst = a.out + (((int64_t)u.b * s.T + u.i) * H + (int64_t)u.g * hpg + h) * D + dim;
          *reinterpret_cast<uint32_t*>(dst) = pack_bf16(x * inv, y * inv);
        } else if (a.parts) {
          // over the ring, whose blocks are all consumed
          sts_f2(smem_u32(sm) + (h * D + dim) * 4, x, y);
          if (pr == 0) sts128(smem_u32(sm) + (hpg * D + h * 4) * 4,
                              make_uint4(__float_as_uint(M), __float_as_uint(N), __float_as_uint(L), 0));
        } else {
          *reinterpret_cast<float2*>(a.part_o + (slot * hpg + h) * D + dim) = make_float2(x, y);
          if (pr == 0) a.part_ml[slot * hpg + h] = make_float4(M, N, L, 0.f);
        }
      }
    }
  }
  __syncthreads();
  if (a.parts > 1) {
    // join the unit's parts: every CTA of the cluster takes a share of the
    // outputs and reads all parts' sums from their shared memory
    cluster_sync();
    const Unit u = unit_of_cluster(a);
    const int rank = (int)blockIdx.x % a.parts;
    const uint32_t base = smem_u32(sm);
    for (int e = rank * C::kThreads + threadIdx.x; e < hpg * (D / 2); e += a.parts * C::kThreads) {
      const int h = e / (D / 2);
      float M = -INFINITY, N = -INFINITY;
      for (int r = 0; r < a.parts; ++r) {
        const float2 mn = ld_cluster_f2(base + (hpg * D + h * 4) * 4, r);
        M = fmaxf(M, mn.x);
        N = fmaxf(N, mn.y);
      }
      float L = 0.f, x = 0.f, y = 0.f;
#pragma unroll 4
      for (int r = 0; r < a.parts; ++r) {
        const float2 mn = ld_cluster_f2(base + (hpg * D + h * 4) * 4, r);
        const float2 l = ld_cluster_f2(base + (hpg * D + h * 4 + 2) * 4, r);
        const float2 v = ld_cluster_f2(base + e * 8, r);
        const float f = mn.x == -INFINITY ? 0.f : ex2(mn.x - M);
        L = fmaf(l.x, mn.y == -INFINITY ? 0.f : ex2(mn.y - N), L);
        x = fmaf(v.x, f, x);
        y = fmaf(v.y, f, y);
      }
      const float inv = L == 0.f ? 0.f : ex2(M - N) / L;
      uint16_t* dst = a.out + (((int64_t)u.b * s.T + u.i) * H + (int64_t)u.g * hpg) * D + e * 2;
      *reinterpret_cast<uint32_t*>(dst) = pack_bf16(x * inv, y * inv);
    }
    cluster_sync();   // no CTA leaves while its sums are read
  }
  if (threadIdx.x == 0) {
    a.errs[blockIdx.x] = err;
    // cluster form: no kernel follows that joins the words; the reader does
    if (a.parts && blockIdx.x == 0) *a.status = kDevWords | (int)gridDim.x;
  }
}

// The worse of two error words (a timeout before an invalid block).
__device__ __forceinline__ int worse(int x, int y) {
  if (x == kDevTimeout || y == kDevTimeout) return kDevTimeout;
  return max(x, y);
}

// Joins the partials of the units that a run's end cuts: one warp per (run,
// query head), for the first run that begins inside a unit.  The first CTA also
// turns the CTAs' error words into the status.
template <int D>
__global__ void __launch_bounds__(256) stream_finish_kernel(const __grid_constant__ StreamArgs a) {
  constexpr int PER = D / 32;
  const Shape& s = a.s;
  const int lane = threadIdx.x & 31;
  if (blockIdx.x == 0 && threadIdx.x < 32) {
    int e = 0;
    for (int c = lane; c < a.nruns * s.G; c += 32) e = worse(e, a.errs[c]);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) e = worse(e, __shfl_xor_sync(0xffffffffu, e, x));
    if (lane == 0) *a.status = a.first_pass ? e : worse(e, *a.status);
  }
  const int hpg = s.H / s.G;
  const int gw = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int run = gw / s.H + 1, g = gw % s.H / hpg, h = gw % hpg, steps = a.step0[s.B];
  if (run >= a.nruns) return;
  const int begin = run_begin(steps, a.nruns, run);
  const Unit u = unit_of(a, begin, g);
  const int r0 = run_of(steps, a.nruns, u.first);
  if (begin == u.first || run != r0 + 1) return;
  const int r1 = run_of(steps, a.nruns, u.first + u.len - 1);
  // run r0 ends inside the unit (its slot 1), runs r0 + 1 ... r1 begin inside it (slot 0)
  float M = -INFINITY, N = -INFINITY;
  for (int r = r0 + lane; r <= r1; r += 32) {
    const float4 v = a.part_ml[(int64_t)(2 * (r * s.G + g) + (r == r0)) * hpg + h];
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
  for (int r = r0; r <= r1; ++r) {
    const int64_t p = (int64_t)(2 * (r * s.G + g) + (r == r0)) * hpg + h;
    const float4 v = a.part_ml[p];
    const float w = v.x == -INFINITY ? 0.f : ex2(v.x - M);
    float x[PER];
#pragma unroll
    for (int e = 0; e < PER; ++e) x[e] = a.part_o[p * D + lane * PER + e];
    L = fmaf(v.y == -INFINITY ? 0.f : ex2(v.y - N), v.z, L);
#pragma unroll
    for (int e = 0; e < PER; ++e) acc[e] = fmaf(w, x[e], acc[e]);
  }
  const float inv = L == 0.f ? 0.f : ex2(M - N) / L;
  uint16_t* dst =
      a.out + (((int64_t)u.b * s.T + u.i) * s.H + (int64_t)u.g * hpg + h) * D + lane * PER;
#pragma unroll
  for (int e = 0; e < PER; e += 2)
    *reinterpret_cast<uint32_t*>(dst + e) = pack_bf16(acc[e] * inv, acc[e + 1] * inv);
}

// CTAs per unit in cluster form, 0: runs.  A cluster joins its parts itself,
// which saves the second launch (about 3 us, the time of kSpare blocks), but
// gives a CTA ceil(longest list / parts) blocks where runs give it the average.
// A cluster's CTAs (one per SM) share one of the 8 GPCs, of at least 16 SMs.
constexpr int kMaxCluster = 8, kSpare = 4, kGpcs = 8, kGpcSms = 16;
int cluster_parts(int units, int longest, int64_t steps, int ctas) {
  int parts = longest < kMaxCluster ? longest : kMaxCluster;
  while (parts > 0 && units > kGpcs * (kGpcSms / parts)) --parts;
  if (parts == 0) return 0;
  return (longest + parts - 1) / parts <= steps / ctas + kSpare ? parts : 0;
}

int list_len(const Visible& vis, int t) {
  if (vis.sel) return kTopk;
  const int lo = (t - vis.window + 1 > 0 ? t - vis.window + 1 : 0) / kBlock;
  const int sb = (vis.sinks + kBlock - 1) / kBlock;
  return (sb < lo ? sb : lo) + t / kBlock - lo + 1;
}

bool encode_codes_map(CUtensorMap* map, const void* base, const Shape& s) {
  auto fn = tensor_map_encoder();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)s.D, (cuuint64_t)s.G, (cuuint64_t)(s.cache_blocks() * kBlock)};
  cuuint64_t strides[2] = {(cuuint64_t)s.D, (cuuint64_t)s.G * s.D};
  cuuint32_t box[3] = {(cuuint32_t)s.D, 1, (cuuint32_t)kBlock};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE,
            s.D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_bf16_cache_map(CUtensorMap* map, const void* base, const Shape& s) {
  cuuint64_t dims[3] = {(cuuint64_t)s.D, (cuuint64_t)s.G, (cuuint64_t)(s.cache_blocks() * kBlock)};
  cuuint64_t strides[2] = {(cuuint64_t)s.D * 2, (cuuint64_t)s.G * s.D * 2};
  cuuint32_t box[3] = {64, 1, (cuuint32_t)kBlock};
  return encode_bf16_map(map, base, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int D, bool Q8, int NTH>
cudaError_t launch_impl(const CacheView& c, StreamArgs& a, cudaStream_t st) {
  using C = Cfg<D, Q8, NTH>;
  const int hpg = a.s.H / a.s.G;
  CUtensorMap tm_k, tm_v;
  if constexpr (Q8) {
    if (!encode_codes_map(&tm_k, c.k, a.s) || !encode_codes_map(&tm_v, c.v, a.s))
      return cudaErrorInvalidValue;
  } else {
    if (!encode_bf16_cache_map(&tm_k, c.k, a.s) || !encode_bf16_cache_map(&tm_v, c.v, a.s))
      return cudaErrorInvalidValue;
  }
  const int fixed = 1024 + kQBufs * hpg * D * 2 + C::kWarps * hpg * C::kRedRow * 4;
  a.stages = (kSmemMax - fixed) / C::kStage;
  if (a.stages > kMaxStages) a.stages = kMaxStages;
  // a stage always serves the same team, whose waits on it then alternate in
  // parity (a team that met a stage every other lap would take the phase
  // before last for its own)
  a.stages -= a.stages % C::kTeams;
  const int smem = fixed + a.stages * C::kStage;
  // The limit belongs to the kernel, which calls of all threads share: always the
  // same value.  This call's own size, which depends on H/G, would let another
  // thread lower the limit between this thread's setting and its launch.
  cudaError_t e = cudaFuncSetAttribute(stream_attn_kernel<D, Q8, NTH>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
  if (e != cudaSuccess) return e;
  if (a.parts) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(a.s.B * a.Tp * a.s.G * a.parts);
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = a.parts;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    note_launches(1);
    return cudaLaunchKernelEx(&cfg, stream_attn_kernel<D, Q8, NTH>, tm_k, tm_v, a);
  }
  note_launches(2);
  stream_attn_kernel<D, Q8, NTH><<<a.nruns * a.s.G, C::kThreads, smem, st>>>(tm_k, tm_v, a);
  const int warps = (a.nruns - 1) * a.s.H;
  stream_finish_kernel<D><<<warps > 0 ? (warps + 7) / 8 : 1, 256, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

int stream_pass_rows(const Shape& s) {
  int tp = kPassRows / s.B;
  if (tp < 1) tp = 1;
  return tp < s.T ? tp : (s.T > 0 ? s.T : 1);
}

StreamPlan stream_plan(const Shape& s) {
  StreamPlan p{};
  auto al = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t rows = (size_t)2 * kMaxCtas * (s.H / s.G);
  size_t o = 0;
  p.errs_off = o;     o += al(kMaxCtas * sizeof(int));
  p.part_ml_off = o;  o += al(rows * sizeof(float4));
  p.part_o_off = o;   o += al(rows * s.D * sizeof(float));
  p.total = o;
  return p;
}

cudaError_t launch_stream_attn(const Shape& s, const Positions& pos, const CacheView& c,
                               const Visible& vis, const uint16_t* q, uint16_t* out, int* status,
                               bool join_status, char* base, cudaStream_t st) {
  const StreamPlan pl = stream_plan(s);
  const int tp = stream_pass_rows(s);
  const int ctas = sm_count() < kMaxCtas ? sm_count() : kMaxCtas;
  StreamArgs a;
  a.s = s;
  for (int b = 0; b < s.B; ++b) a.q_start[b] = pos.q_start[b];
  a.window = vis.window;
  a.sinks = vis.sinks;
  a.sel = vis.sel;
  a.q = q;
  a.k_exp = c.k_exp;
  a.v_exp = c.v_exp;
  a.part_o = reinterpret_cast<float*>(base + pl.part_o_off);
  a.part_ml = reinterpret_cast<float4*>(base + pl.part_ml_off);
  a.errs = reinterpret_cast<int*>(base + pl.errs_off);
  a.out = out;
  a.status = status;
  a.wait_polls = debug_wait_polls();
  for (int t0 = 0; t0 < s.T; t0 += tp) {
    a.t0 = t0;
    a.Tp = tp < s.T - t0 ? tp : s.T - t0;
    a.first_pass = t0 == 0 && !join_status;
    int len[kMaxBatch];
    for (int b = 0; b < s.B; ++b) {
      // the longest list of the pass: of the last query, or (a window that
      // ends inside a block) of one of the 128 before it
      len[b] = 1;
      const int last = pos.q_start[b] + t0 + a.Tp - 1;
      const int from = a.Tp > kBlock ? last - kBlock + 1 : last - a.Tp + 1;
      for (int t = from; t <= last; ++t) {
        const int n = list_len(vis, t);
        len[b] = n > len[b] ? n : len[b];
        if (vis.sel) break;
      }
    }
    a.step0[0] = 0;
    for (int b = 0; b < s.B; ++b) a.step0[b + 1] = a.step0[b] + a.Tp * len[b];
    const int steps = a.step0[s.B];
    a.nruns = steps < ctas / s.G ? steps : ctas / s.G;
    a.parts = 0;
    if (a.Tp == s.T && !join_status) {
      int longest = 1;
      for (int b = 0; b < s.B; ++b) longest = len[b] > longest ? len[b] : longest;
      a.parts = cluster_parts(s.B * a.Tp * s.G, longest, (int64_t)steps * s.G, ctas);
    }
    const bool wide = s.H / s.G > 8;    // heads of a group in one or two n-tiles of 8
    cudaError_t e;
    if (s.D == 128 && c.kv8)
      e = wide ? launch_impl<128, true, 2>(c, a, st) : launch_impl<128, true, 1>(c, a, st);
    else if (s.D == 128)
      e = wide ? launch_impl<128, false, 2>(c, a, st) : launch_impl<128, false, 1>(c, a, st);
    else if (c.kv8)
      e = wide ? launch_impl<64, true, 2>(c, a, st) : launch_impl<64, true, 1>(c, a, st);
    else
      e = wide ? launch_impl<64, false, 2>(c, a, st) : launch_impl<64, false, 1>(c, a, st);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace msa

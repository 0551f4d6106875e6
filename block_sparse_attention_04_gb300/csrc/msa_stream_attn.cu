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
// The call's work is one sequence of (unit, block) steps, unit (b, t, g) after
// unit, cut into equal runs, one per CTA and SM; a run's share of one unit is a
// segment.  Warp 8 copies K and V of each block (128 tokens of one KV head)
// into a ring of stages by TMA and runs ahead by its depth.  Warps 0-7 take 16
// tokens of every block each and never wait for one another inside a segment: S = Q K^T with mma.sync m16n8k16 (rows: the
// group's heads), softmax in registers, P straight from the accumulator
// layout into the A operand of O += P V.  The order of the contraction's
// terms is free, so dims (for S) and output columns (for O) are dealt to
// threads such that every thread reads whole 16-byte chunks of the swizzled
// rows; pairs of tokens of V are put together with byte permutes.  e4m3 codes
// become f16 (exact) by one conversion per pair; Q is scaled by a power of two
// per row to fit f16 (exact but for elements 2^-27 below the row's maximum,
// which round at 2^-38 of it), and P rounds to f16 (2^-11).  With a bf16 cache
// the products are bf16 and P rounds to bf16 (2^-8).
// At a segment's end the eight warps' (O, m, l) are joined in shared memory; a
// whole unit is written out directly, a cut one leaves a partial per CTA (at
// most two: the unit its run begins inside, the one it ends inside) that
// stream_finish_kernel joins.
#include "msa_q8.cuh"
#include "msa_tma.h"

namespace msa {
namespace {

constexpr int kConsWarps = 8;
constexpr int kConsumers = 32 * kConsWarps;
constexpr int kThreads = kConsumers + 32;
constexpr int kQBufs = 2;
constexpr int kMaxStages = 8;
constexpr int kMaxCtas = 512;        // partials and error words in the workspace
constexpr int kPassRows = 2048;      // (sequence, query) rows per pass
constexpr float kLazy = 8.f;         // log2 growth of p tolerated before O is rescaled
constexpr int kSmemMax = 227 * 1024;

struct StreamArgs {
  Shape s;
  int32_t q_start[kMaxBatch];
  int32_t step0[kMaxBatch + 1];   // first step of each sequence; [B]: all steps
  int t0, Tp, nctas, stages;
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
  uint32_t wait_polls;
};

// CTA c's run of steps begins at floor(c * steps / nctas).
__host__ __device__ __forceinline__ int run_begin(int steps, int nctas, int c) {
  return (int)((int64_t)c * steps / nctas);
}
__device__ __forceinline__ int run_of(int steps, int nctas, int step) {
  return (int)((((int64_t)step + 1) * nctas - 1) / steps);
}

// The unit that a step belongs to: its first step, its steps (the longest
// list of its sequence in this pass) and its query.
struct Unit {
  int b, i, g, t, first, len;
};

__device__ __forceinline__ Unit unit_of(const StreamArgs& a, int step) {
  int lo = 0, hi = a.s.B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.step0[mid] <= step) lo = mid; else hi = mid;
  }
  Unit u;
  u.b = lo;
  u.len = (a.step0[lo + 1] - a.step0[lo]) / (a.Tp * a.s.G);
  const int ig = (step - a.step0[lo]) / u.len;
  u.first = a.step0[lo] + ig * u.len;
  u.g = ig % a.s.G;
  u.i = a.t0 + ig / a.s.G;
  u.t = a.q_start[lo] + u.i;
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

template <int D, bool Q8>
struct Cfg {
  static constexpr int kTile = kBlock * D * (Q8 ? 1 : 2);   // K (or V) of one block and head
  static constexpr int kStage = 2 * kTile;
  static constexpr int kRedRow = D + 8;                     // padded row of the join buffer (floats)
};

template <int D, bool Q8>
__global__ void __launch_bounds__(kThreads, 1) stream_attn_kernel(
    const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
    const __grid_constant__ StreamArgs a) {
  using C = Cfg<D, Q8>;
  constexpr int NS = D / 16;       // k-steps of S
  constexpr int NO = D / 8;        // n-tiles of O
  extern __shared__ uint8_t dsm_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(dsm_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages], q_full[kQBufs], q_empty[kQBufs];
  __shared__ int meta_kb[kMaxStages], meta_ke[kMaxStages], meta_ve[kMaxStages];
  __shared__ float sm_m[kConsWarps][16], sm_n[kConsWarps][16], sm_l[kConsWarps][16];
  __shared__ int err;
  const Shape& s = a.s;
  const int H = s.H, G = s.G, hpg = H / G, S = a.stages;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint16_t* qbuf = reinterpret_cast<uint16_t*>(sm + S * C::kStage);       // [kQBufs][hpg][D]
  const uint32_t red = smem_u32(qbuf + kQBufs * hpg * D);                 // [8][hpg][kRedRow] float
  const int steps = a.step0[s.B];
  const int run0 = run_begin(steps, a.nctas, blockIdx.x);
  const int run1 = run_begin(steps, a.nctas, blockIdx.x + 1);

  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], kConsWarps);
    }
    for (int i = 0; i < kQBufs; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], kConsWarps);
    }
    err = 0;
    fence_mbar_init();
  }
  __syncthreads();

  if (warp == kConsWarps) {
    // ------------------------------------------------------------ producer
    const uint64_t pol = l2_policy_evict_first();
    const uint32_t qbytes = (uint32_t)(hpg * D * 2);
    int st = 0, k = 0;              // next stage, segments begun
    uint32_t ph = 1;                // phase parity that frees the stage (first lap: free)
    uint32_t used = 0, loaded = 0;  // stages ever loaded / parity of each stage's last load
    int nq = 0;
    bool ok = true;
    for (int step = run0, next; step < run1 && ok; step = next, ++k) {
      const Unit u = unit_of(a, step);
      next = min(run1, u.first + u.len);
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
      const BlockList bl = list_of(a, u.t);
      const int p0 = step - u.first, p1 = min(next - u.first, bl.len);
      const int32_t* srow =
          a.sel ? a.sel + (((int64_t)u.b * s.T + u.i) * G + u.g) * kTopk : nullptr;
      for (int pc = p0; pc < p1 && ok; pc += 32) {
        // one list position per lane: its block, cache block and exponents
        int kb = -1, ke = 0, ve = 0, row = 0;
        const int p = pc + lane;
        if (p < p1) {
          kb = srow ? srow[p] : (p < bl.nsink ? p : bl.first + p);
          if (srow && kb >= 0 && (kb > u.t / kBlock || kb >= s.max_blocks)) {
            flag_invalid(&err);
            kb = -1;
          }
          if (kb >= 0) {
            const int64_t pb = cache_block(s, u.b, kb, &err);
            if (pb < 0) {
              kb = -1;
            } else {
              row = (int)(pb * kBlock);
              if (Q8) {
                ke = clamp_exp(a.k_exp[pb * G + u.g]);
                ve = clamp_exp(a.v_exp[pb * G + u.g]);
              }
            }
          }
        }
        const int n = min(32, p1 - pc);
        for (int j = 0; j < n; ++j) {
          const int kbj = __shfl_sync(0xffffffffu, kb, j), rowj = __shfl_sync(0xffffffffu, row, j);
          const int kej = __shfl_sync(0xffffffffu, ke, j), vej = __shfl_sync(0xffffffffu, ve, j);
          ok = __all_sync(0xffffffffu, mbar_wait(&empty[st], ph, &err, a.wait_polls));
          if (!ok) break;
          if (lane == 0) {
            meta_kb[st] = kbj;
            meta_ke[st] = kej;
            meta_ve[st] = vej;
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
    const int g4 = lane >> 2, t4 = lane & 3;   // row (head or token) and column quad of a fragment
    const float qk = s.scale * kLog2e;
    int st = 0, k = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int step = run0, next; step < run1; step = next, ++k) {
      const Unit u = unit_of(a, step);
      next = min(run1, u.first + u.len);
      const BlockList bl = list_of(a, u.t);
      const int nblk = min(next - u.first, bl.len) - (step - u.first);
      const int lo = a.sel ? 0 : max(0, u.t - a.window + 1);   // visible: j <= t and
      const int sinks = a.sel ? 0 : a.sinks;                   // (j >= lo or j < sinks)
      const int qs = k % kQBufs;
      ok = __all_sync(0xffffffffu,
                      ok && mbar_wait(&q_full[qs], (k / kQBufs) & 1, &err, a.wait_polls));
      // Q fragments: rows g4 and g4 + 8, the four dims per k-step that this
      // thread's 16-byte chunks of a K row hold (see the reads of K below)
      uint32_t qa[NS][4];
      float fq[2] = {qk, qk};          // score factor of the two rows
#pragma unroll
      for (int rr = 0; rr < 2; ++rr) {
        const int h = g4 + 8 * rr;
        const uint32_t qrow = smem_u32(qbuf + (qs * hpg + min(h, hpg - 1)) * D);
        uint2 w[NS];
#pragma unroll
        for (int ks = 0; ks < NS; ++ks) {
          int dim;
          if constexpr (Q8)
            dim = D == 128 ? (2 * t4 + (ks >> 2)) * 16 + (ks & 3) * 4 : t4 * 16 + ks * 4;
          else
            dim = (ks >> 2) * 64 + (2 * t4 + ((ks >> 1) & 1)) * 8 + (ks & 1) * 4;
          w[ks] = h < hpg && ok ? lds64(qrow + dim * 2) : make_uint2(0, 0);
        }
        if constexpr (Q8) {
          // scale the row by a power of two: its largest magnitude to [2^13, 2^14)
          uint32_t mx = 0;
#pragma unroll
          for (int ks = 0; ks < NS; ++ks) {
            mx = max(max(mx, w[ks].x & 0x7FFFu), max(w[ks].x >> 16 & 0x7FFFu, w[ks].y & 0x7FFFu));
            mx = max(mx, w[ks].y >> 16 & 0x7FFFu);
          }
          mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
          int e = (int)(mx >> 7) - 127;                   // floor(log2 max); inf, NaN: 128
          e = mx == 0 || e == 128 ? 0 : max(e, -100);
          const float f = pow2i(13 - e);
          fq[rr] = qk * pow2i(e - 13);
#pragma unroll
          for (int ks = 0; ks < NS; ++ks) {
            qa[ks][rr] = pack_f16(bf16lo(w[ks].x) * f, bf16hi(w[ks].x) * f);
            qa[ks][2 + rr] = pack_f16(bf16lo(w[ks].y) * f, bf16hi(w[ks].y) * f);
          }
        } else {
#pragma unroll
          for (int ks = 0; ks < NS; ++ks) {
            qa[ks][rr] = w[ks].x;
            qa[ks][2 + rr] = w[ks].y;
          }
        }
      }
      float o[NO][4];
#pragma unroll
      for (int j = 0; j < NO; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[j][c] = 0.f;
      // running maxima of x + ev (of O's terms) and x (of l's; the same without ev)
      float m[2] = {-INFINITY, -INFINITY}, n[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

      for (int blk = 0; blk < nblk; ++blk) {
        ok = __all_sync(0xffffffffu, ok && mbar_wait(&full[st], ph, &err, a.wait_polls));
        if (!ok) break;
        const int kb = meta_kb[st];
        if (kb >= 0) {
          const int tok0 = kb * kBlock;
          const int w0 = tok0 + warp * 16;              // this warp's first token
          const bool whole = tok0 + kBlock - 1 <= u.t && (tok0 >= lo || tok0 + kBlock - 1 < sinks);
          const bool any = w0 <= u.t && (w0 + 15 >= lo || w0 < sinks);
          if (any) {
            const uint32_t kbase = smem_u32(sm + st * C::kStage), vbase = kbase + C::kTile;
            // ---- S = Q K^T of 16 tokens (two n-tiles of 8)
            float sc[2][4];
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
              const int r = warp * 16 + nt * 8 + g4;
#pragma unroll
              for (int c = 0; c < 4; ++c) sc[nt][c] = 0.f;
              if constexpr (Q8) {
#pragma unroll
                for (int j = 0; j < D / 64; ++j) {
                  const uint4 w = D == 128
                                      ? lds128(kbase + r * 128 + (((2 * t4 + j) ^ (r & 7)) << 4))
                                      : lds128(kbase + r * 64 + ((t4 ^ ((r >> 1) & 3)) << 4));
                  const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                  for (int x = 0; x < 4; ++x) {
                    const int ks = j * 4 + x;
                    mma_f16_16816(sc[nt], qa[ks][0], qa[ks][1], qa[ks][2], qa[ks][3],
                                  e4m3x2_to_f16x2(ww[x] & 0xFFFFu), e4m3x2_to_f16x2(ww[x] >> 16));
                  }
                }
              } else {
#pragma unroll
                for (int hj = 0; hj < D / 32; ++hj) {    // 64-dim half, chunk of it
                  const uint4 w = lds128(kbase + (hj >> 1) * 16384 + r * 128 +
                                         (((2 * t4 + (hj & 1)) ^ (r & 7)) << 4));
                  const int ks = hj * 2;
                  mma_bf16_16816(sc[nt], qa[ks][0], qa[ks][1], qa[ks][2], qa[ks][3], w.x, w.y);
                  mma_bf16_16816(sc[nt], qa[ks + 1][0], qa[ks + 1][1], qa[ks + 1][2],
                                 qa[ks + 1][3], w.z, w.w);
                }
              }
            }
            // ---- x = s log2(e), masked; row maxima
            float f[2] = {fq[0], fq[1]}, ev = 0.f;
            if constexpr (Q8) {
              const float fk = pow2i(meta_ke[st]);
              f[0] = fminf(fmaxf(fq[0] * fk, -3e38f), 3e38f);
              f[1] = fminf(fmaxf(fq[1] * fk, -3e38f), 3e38f);
              ev = (float)meta_ve[st];
            }
            bool vis[4] = {true, true, true, true};      // tokens (nt, e) = w0 + nt*8 + 2*t4 + e
            if (!whole) {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const int tok = w0 + (j >> 1) * 8 + 2 * t4 + (j & 1);
                vis[j] = tok <= u.t && (tok >= lo || tok < sinks);
              }
            }
            float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const float x = sc[nt][c] * f[c >> 1];
                sc[nt][c] = vis[nt * 2 + (c & 1)] ? x : -INFINITY;
                mx[c >> 1] = fmaxf(mx[c >> 1], sc[nt][c]);
              }
            bool grow = false;
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
              mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
              grow |= mx[r] + ev > m[r] + kLazy || (Q8 && mx[r] > n[r] + kLazy);
            }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                const float mn = fmaxf(m[r], mx[r] + ev);
                const float al = m[r] == -INFINITY ? 0.f : ex2(m[r] - mn);
                m[r] = mn;
                if constexpr (Q8) {
                  const float nn = fmaxf(n[r], mx[r]);
                  l[r] *= n[r] == -INFINITY ? 0.f : ex2(n[r] - nn);
                  n[r] = nn;
                } else {
                  l[r] *= al;
                }
#pragma unroll
                for (int j = 0; j < NO; ++j) {
                  o[j][2 * r] *= al;
                  o[j][2 * r + 1] *= al;
                }
              }
            }
            // ---- p' = 2^(x - m): A fragment of O += P V
            uint32_t pa[4];
            float sum[2] = {0.f, 0.f};
#pragma unroll
            for (int nt = 0; nt < 2; ++nt)
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                const float mr = m[r] == -INFINITY ? 0.f : m[r] - ev;
                const float p0 = ex2(sc[nt][2 * r] - mr), p1 = ex2(sc[nt][2 * r + 1] - mr);
                pa[nt * 2 + r] = Q8 ? pack_f16(p0, p1) : pack_bf16(p0, p1);
                if constexpr (Q8) {
                  const float nr = n[r] == -INFINITY ? 0.f : n[r];
                  sum[r] += ex2(sc[nt][2 * r] - nr) + ex2(sc[nt][2 * r + 1] - nr);
                } else {
                  sum[r] += p0 + p1;
                }
              }
            l[0] += sum[0];
            l[1] += sum[1];
            // ---- V: tokens w0 + {2 t4, 2 t4 + 1, 8 + 2 t4, 9 + 2 t4}, the
            // dims of this thread's chunks; rows that the query does not see
            // (they may hold anything) as zeros
            const int r0 = warp * 16 + 2 * t4;
            constexpr int kHalves = Q8 ? 1 : D / 64;      // boxes of a row
            constexpr int kDimsPer = Q8 ? D / 8 : 8;      // dims of this thread in a box
#pragma unroll
            for (int hb = 0; hb < kHalves; ++hb) {
              constexpr int W = Q8 ? D / 32 : 4;          // words per token
              uint32_t vw[4][W];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const int r = r0 + (j >> 1) * 8 + (j & 1);
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
                if (!whole && !vis[j]) {
#pragma unroll
                  for (int x = 0; x < W; ++x) vw[j][x] = 0u;
                }
              }
#pragma unroll
              for (int x = 0; x < W; ++x) {
                if constexpr (Q8) {
#pragma unroll
                  for (int y = 0; y < 2; ++y) {           // dims 4x + 2y, 4x + 2y + 1
                    const uint32_t sel = y ? 0x7362u : 0x5140u;
                    const uint32_t c0 = __byte_perm(vw[0][x], vw[1][x], sel);
                    const uint32_t c1 = __byte_perm(vw[2][x], vw[3][x], sel);
                    const int j = 4 * x + 2 * y;
                    mma_f16_16816(o[j], pa[0], pa[1], pa[2], pa[3], e4m3x2_to_f16x2(c0 & 0xFFFFu),
                                  e4m3x2_to_f16x2(c1 & 0xFFFFu));
                    mma_f16_16816(o[j + 1], pa[0], pa[1], pa[2], pa[3], e4m3x2_to_f16x2(c0 >> 16),
                                  e4m3x2_to_f16x2(c1 >> 16));
                  }
                } else {                                  // dims 2x, 2x + 1 of the box's chunk
                  const int j = hb * kDimsPer + 2 * x;
                  mma_bf16_16816(o[j], pa[0], pa[1], pa[2], pa[3],
                                 __byte_perm(vw[0][x], vw[1][x], 0x5410),
                                 __byte_perm(vw[2][x], vw[3][x], 0x5410));
                  mma_bf16_16816(o[j + 1], pa[0], pa[1], pa[2], pa[3],
                                 __byte_perm(vw[0][x], vw[1][x], 0x7632),
                                 __byte_perm(vw[2][x], vw[3][x], 0x7632));
                }
              }
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[st]);
        if (++st == S) {
          st = 0;
          ph ^= 1;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_empty[qs]);

      // ---- join the warps: O relative to each warp's own m
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      }
      if (!named_bar_and(1, kConsumers, ok)) {   // also: the last segment's sums have been read
        ok = false;
        break;
      }
      if (t4 == 0) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          sm_m[warp][g4 + 8 * r] = m[r];
          sm_n[warp][g4 + 8 * r] = Q8 ? n[r] : m[r];
          sm_l[warp][g4 + 8 * r] = l[r];
        }
      }
      // fragment order: columns 2 t4, 2 t4 + 1 of n-tile j side by side
#pragma unroll
      for (int r = 0; r < 2; ++r)
        if (g4 + 8 * r < hpg) {
          const uint32_t row = red + ((warp * hpg + g4 + 8 * r) * C::kRedRow + 2 * t4) * 4;
#pragma unroll
          for (int j = 0; j < NO; ++j) sts_f2(row + j * 32, o[j][2 * r], o[j][2 * r + 1]);
        }
      named_bar_sync(1, kConsumers);
      const bool whole_unit = step == u.first && next == u.first + u.len;
      const int64_t slot = 2 * blockIdx.x + (step == u.first);
      for (int e = threadIdx.x; e < hpg * NO * 4; e += kConsumers) {
        const int h = e / (NO * 4), j = e / 4 % NO;        // one head per warp and step
        float M = -INFINITY, N = -INFINITY;
#pragma unroll
        for (int w = 0; w < kConsWarps; ++w) {
          M = fmaxf(M, sm_m[w][h]);
          N = fmaxf(N, sm_n[w][h]);
        }
        float L = 0.f, x = 0.f, y = 0.f;
#pragma unroll
        for (int w = 0; w < kConsWarps; ++w) {
          const float mw = sm_m[w][h];
          const float f = mw == -INFINITY ? 0.f : ex2(mw - M);
          const float2 v = lds_f2(red + ((w * hpg + h) * C::kRedRow + (e % (NO * 4)) * 2) * 4);
          const float nw = sm_n[w][h];
          L = fmaf(sm_l[w][h], nw == -INFINITY ? 0.f : ex2(nw - N), L);
          x = fmaf(v.x, f, x);
          y = fmaf(v.y, f, y);
        }
        // dims j, j + 1 of one column: the lane of the other j holds the pair's other half
        const bool odd = j & 1;
        const float other = __shfl_xor_sync(0xffffffffu, odd ? x : y, 4);
        const float d0 = odd ? other : x, d1 = odd ? y : other;
        const int n = 2 * (e & 3) + odd, je = j & ~1;
        const int dim = Q8 ? n * (D / 8) + je : (je >> 3) * 64 + n * 8 + (je & 7);
        if (whole_unit) {
          const float inv = L == 0.f ? 0.f : ex2(M - N) / L;      // nothing visible: zeros
          uint16_t* dst = a.out + (((int64_t)u.b * s.T + u.i) * H + (int64_t)u.g * hpg + h) * D + dim;
          *reinterpret_cast<uint32_t*>(dst) = pack_bf16(d0 * inv, d1 * inv);
        } else {
          *reinterpret_cast<float2*>(a.part_o + (slot * hpg + h) * D + dim) = make_float2(d0, d1);
          if (e % (NO * 4) == 0) a.part_ml[slot * hpg + h] = make_float4(M, N, L, 0.f);
        }
      }
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) a.errs[blockIdx.x] = err;
}

// The worse of two error words (a timeout before an invalid block).
__device__ __forceinline__ int worse(int x, int y) {
  if (x == kDevTimeout || y == kDevTimeout) return kDevTimeout;
  return max(x, y);
}

// Joins the partials of the units that a run's end cuts: one warp per (run,
// head), for the first run that begins inside a unit.  The first CTA also
// turns the CTAs' error words into the status.
template <int D>
__global__ void __launch_bounds__(256) stream_finish_kernel(const __grid_constant__ StreamArgs a) {
  constexpr int PER = D / 32;
  const Shape& s = a.s;
  const int lane = threadIdx.x & 31;
  if (blockIdx.x == 0 && threadIdx.x < 32) {
    int e = 0;
    for (int c = lane; c < a.nctas; c += 32) e = worse(e, a.errs[c]);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) e = worse(e, __shfl_xor_sync(0xffffffffu, e, x));
    if (lane == 0) *a.status = a.first_pass ? e : worse(e, *a.status);
  }
  const int hpg = s.H / s.G;
  const int gw = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int run = gw / hpg + 1, h = gw % hpg, steps = a.step0[s.B];
  if (run >= a.nctas) return;
  const int begin = run_begin(steps, a.nctas, run);
  const Unit u = unit_of(a, begin);
  const int r0 = run_of(steps, a.nctas, u.first);
  if (begin == u.first || run != r0 + 1) return;
  const int r1 = run_of(steps, a.nctas, u.first + u.len - 1);
  // run r0 ends inside the unit (its slot 1), runs r0 + 1 ... r1 begin inside it (slot 0)
  float M = -INFINITY, N = -INFINITY;
  for (int r = r0 + lane; r <= r1; r += 32) {
    const float4 v = a.part_ml[(int64_t)(2 * r + (r == r0)) * hpg + h];
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
    const int64_t p = (int64_t)(2 * r + (r == r0)) * hpg + h;
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
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool encode_bf16_cache_map(CUtensorMap* map, const void* base, const Shape& s) {
  cuuint64_t dims[3] = {(cuuint64_t)s.D, (cuuint64_t)s.G, (cuuint64_t)(s.cache_blocks() * kBlock)};
  cuuint64_t strides[2] = {(cuuint64_t)s.D * 2, (cuuint64_t)s.G * s.D * 2};
  cuuint32_t box[3] = {64, 1, (cuuint32_t)kBlock};
  return encode_bf16_map(map, base, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int D, bool Q8>
cudaError_t launch_impl(const CacheView& c, StreamArgs& a, cudaStream_t st) {
  using C = Cfg<D, Q8>;
  const int hpg = a.s.H / a.s.G;
  CUtensorMap tm_k, tm_v;
  if constexpr (Q8) {
    if (!encode_codes_map(&tm_k, c.k, a.s) || !encode_codes_map(&tm_v, c.v, a.s))
      return cudaErrorInvalidValue;
  } else {
    if (!encode_bf16_cache_map(&tm_k, c.k, a.s) || !encode_bf16_cache_map(&tm_v, c.v, a.s))
      return cudaErrorInvalidValue;
  }
  const int fixed = 1024 + kQBufs * hpg * D * 2 + kConsWarps * hpg * C::kRedRow * 4;
  // static shared memory (barriers, row statistics) takes under 2 KiB
  a.stages = (kSmemMax - 2048 - fixed) / C::kStage;
  if (a.stages > kMaxStages) a.stages = kMaxStages;
  const int smem = fixed + a.stages * C::kStage;
  cudaError_t e = cudaFuncSetAttribute(stream_attn_kernel<D, Q8>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  note_launches(2);
  stream_attn_kernel<D, Q8><<<a.nctas, kThreads, smem, st>>>(tm_k, tm_v, a);
  const int warps = (a.nctas - 1) * hpg;
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
    for (int b = 0; b < s.B; ++b) a.step0[b + 1] = a.step0[b] + a.Tp * s.G * len[b];
    const int steps = a.step0[s.B];
    a.nctas = steps < ctas ? steps : ctas;
    cudaError_t e;
    if (s.D == 128)
      e = c.kv8 ? launch_impl<128, true>(c, a, st) : launch_impl<128, false>(c, a, st);
    else
      e = c.kv8 ? launch_impl<64, true>(c, a, st) : launch_impl<64, false>(c, a, st);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace msa

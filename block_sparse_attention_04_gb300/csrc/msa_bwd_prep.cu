// The attention's backward pass, its small kernels: row statistics, the inverted
// lists of a selection, the units of work, and the joins of partial sums.
#include <climits>

#include "msa_bwd.h"
#include "msa_device.cuh"

namespace msa {
namespace {

// ---- row statistics -----------------------------------------------------------
// Groups of rows: -lse log2e, and -delta = -dout.out.  A row whose whole context lies in
// block 0 (t < 128) leaves delta to a second kernel, which takes it from the probabilities, delta = sum P dP / sum P over its
// keys: with few tokens dS is a small difference of dP and delta, and out carries
// rounding of 2^-9 (8 tokens, scores of two units: dq 0.35 % off, now 0.25, what
// rounding dS leaves).  There a CTA takes a head, and a warp 16 of its queries against 8
// keys at a time on mma.sync, from K and V of block 0 in shared memory; the order of the
// dims in the products is permuted so that a lane's fragments of two steps are 16
// contiguous bytes.  (Fragments read from global memory: 45 us for four sequences.)
struct StatArgs {
  Shape s;
  Positions pos;
  const uint16_t *q, *k, *v, *out, *dout;
  const float* lse;
  uint8_t* stat;         // dense: the groups as numbers
  uint8_t* aug;          // the groups as operands
  float to_score;        // 1 / (scale log2e), or 1
  uint32_t groups;
  int rpe;               // 0: dense
  int* status;
};
constexpr int kStatThreads = 256;
// Writes x at its row of an operand group (0: lse, 1: delta): three bf16 parts.
__device__ __forceinline__ void put_aug(uint8_t* group, int which, int row, float x) {
  const float hi = __uint_as_float(pack_bf16(x, 0.f) << 16);
  float mid = 0.f, lo = 0.f;
  if (fabsf(hi) < INFINITY) {              // (a NaN goes on in hi)
    mid = __uint_as_float(pack_bf16(x - hi, 0.f) << 16);
    lo = x - hi - mid;
  }
  *reinterpret_cast<uint2*>(group + row * 16 + which * 8) =
      make_uint2(pack_bf16(hi, mid), pack_bf16(lo, 0.f));
}

// -delta of row (b, query i, head h).
__device__ __forceinline__ void put_delta(const StatArgs& a, int b, int i, int h, float x) {
  const int hpg = a.s.H / a.s.G;
  if (a.rpe == 0) {
    const size_t g = (size_t)(b * a.s.H + h) * a.groups + (i >> 3);
    reinterpret_cast<float*>(a.stat + g * kStatBytes)[8 + (i & 7)] = x;
    put_aug(a.aug + g * kAugBytes, 1, i & 7, x);
  } else {
    const size_t g =
        (((size_t)b * a.s.T + i) * a.s.G + h / hpg) * (a.rpe >> 3) + (h % hpg >> 3);
    put_aug(a.aug + g * kAugBytes, 1, h % hpg & 7, x);
  }
}

template <int D>
__device__ __forceinline__ void stat_first(const StatArgs& a) {
  extern __shared__ __align__(16) uint8_t kv[];      // K, then V: rows of D bf16 and 16 bytes
  constexpr int PITCH = 2 * D + 16;
  const int lane = threadIdx.x & 31, H = a.s.H, G = a.s.G;
  const int b = blockIdx.x / H, h = blockIdx.x % H, g = h / (H / G);
  const int n = min(a.s.T, kBlock - a.pos.q_start[b]);   // rows with t < 128
  if (n <= 0) return;
  {
    // rows behind the last query's hold anything: they are masked below
    const int rows = min(kBlock, (a.pos.q_start[b] + n + 7) & ~7);
    for (int e = threadIdx.x; e < 2 * rows * (D / 8); e += 256) {
      const int ch = e % (D / 8), row = e / (D / 8) % rows;
      const bool v = e >= rows * (D / 8);
      const uint16_t* src = (v ? a.v : a.k) + (((size_t)b * a.s.max_blocks * kBlock + row) * G + g) * D;
      *reinterpret_cast<uint4*>(kv + (v ? kBlock * PITCH : 0) + row * PITCH + ch * 16) =
          *reinterpret_cast<const uint4*>(src + 8 * ch);
    }
    __syncthreads();
  }
  const int i0 = (threadIdx.x >> 5) * 16;
  if (i0 >= n) return;
  const int r = lane >> 2, c = lane & 3;
  constexpr int NC = D / 32;
  uint4 fq[2][NC], fo[2][NC];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int i = min(i0 + r + 8 * u, n - 1);
    const size_t at = (((size_t)b * a.s.T + i) * H + h) * D + 8 * c;
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      fq[u][k] = *reinterpret_cast<const uint4*>(a.q + at + 32 * k);
      fo[u][k] = *reinterpret_cast<const uint4*>(a.dout + at + 32 * k);
    }
  }
  float sp[2] = {0.f, 0.f}, sd[2] = {0.f, 0.f}, nl[2];
  int t[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int i = min(i0 + r + 8 * u, n - 1);
    t[u] = a.pos.q_start[b] + i;
    nl[u] = -kLog2e * a.lse[((size_t)b * a.s.T + i) * H + h];
  }
  const float sl = a.s.scale * kLog2e;
  const int t_last = a.pos.q_start[b] + min(i0 + 15, n - 1);
  for (int j0 = 0; j0 <= t_last; j0 += 8) {
    const uint8_t* at = kv + (j0 + r) * PITCH + 16 * c;
    float x[4] = {0.f, 0.f, 0.f, 0.f}, y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const uint4 fk = *reinterpret_cast<const uint4*>(at + 64 * k);
      const uint4 fv = *reinterpret_cast<const uint4*>(at + kBlock * PITCH + 64 * k);
      mma_bf16_16816(x, fq[0][k].x, fq[1][k].x, fq[0][k].y, fq[1][k].y, fk.x, fk.y);
      mma_bf16_16816(x, fq[0][k].z, fq[1][k].z, fq[0][k].w, fq[1][k].w, fk.z, fk.w);
      mma_bf16_16816(y, fo[0][k].x, fo[1][k].x, fo[0][k].y, fo[1][k].y, fv.x, fv.y);
      mma_bf16_16816(y, fo[0][k].z, fo[1][k].z, fo[0][k].w, fo[1][k].w, fv.z, fv.w);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int u = e >> 1;
      if (j0 + 2 * c + (e & 1) > t[u]) continue;
      const float p = ex2(fmaf(x[e], sl, nl[u]));
      sp[u] += p;
      sd[u] = fmaf(p, y[e], sd[u]);
    }
  }
#pragma unroll
  for (int u = 0; u < 2; ++u) {
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      sp[u] += __shfl_xor_sync(0xffffffffu, sp[u], o);
      sd[u] += __shfl_xor_sync(0xffffffffu, sd[u], o);
    }
    // (a NaN in a row goes on into its delta)
    if (c == 0 && i0 + r + 8 * u < n) {
      const float nd = sp[u] == 0.f ? 0.f : -sd[u] / sp[u];
      const int i = i0 + r + 8 * u;
      put_delta(a, b, i, h, nd);
    }
  }
}

// It reads nothing that the kernel before it writes, and writes other words: it runs beside
// that and waits for it in the end, as the kernel behind waits for this one alone.
template <int D>
__global__ void __launch_bounds__(256) bwd_stat_first_kernel(const __grid_constant__ StatArgs a) {
  let_next();
  stat_first<D>(a);
  after_previous();
}

// A group of 8 rows per D/8 lanes: its 16 row reads are in flight together, and it is
// written whole.  (One row at a time, with its two numbers stored singly: 438 us for 16K
// queries of 48 heads, 403 MB.)
template <int D>
__global__ void __launch_bounds__(kStatThreads) bwd_stat_kernel(const __grid_constant__ StatArgs a) {
  if (threadIdx.x == 0) {
    if (blockIdx.x == 0) *a.status = 0;    // (a kernel that may report waits for this one first)
    let_next();
  }
  constexpr int LPR = D / 8;
  const int H = a.s.H, G = a.s.G, hpg = H / G;
  const int l = threadIdx.x % LPR;
  const int64_t grp = (int64_t)blockIdx.x * (kStatThreads / LPR) + threadIdx.x / LPR;
  // dense: groups in order (b, 8 queries, h); sparse: (b, query, g, 8 heads)
  int b, i0, h0, n;
  int64_t row;                       // the first row, of rows [B][T][H]
  const int step = a.rpe ? 1 : H;    // to the next
  bool in;
  size_t dst;                        // group
  if (a.rpe) {
    const int sub = a.rpe >> 3;
    in = grp < (int64_t)a.s.B * a.s.T * G * sub;
    const int64_t q = grp / (G * sub);
    const int x = (int)(grp - q * (G * sub));
    b = (int)(q / a.s.T);
    i0 = (int)(q - (int64_t)b * a.s.T);
    h0 = x / sub * hpg + x % sub * 8;
    n = min(8, hpg - x % sub * 8);
    row = q * H + h0;
    dst = (size_t)grp;
  } else {
    const int64_t q = grp / H;
    h0 = (int)(grp - q * H);
    in = q < (int64_t)a.s.B * a.groups;
    b = (int)(q / a.groups);
    i0 = (int)(q - (int64_t)b * a.groups) * 8;
    n = min(8, a.s.T - i0);
    row = ((int64_t)b * a.s.T + i0) * H + h0;
    dst = (size_t)(b * H + h0) * a.groups + (i0 >> 3);
  }
  if (!in) n = 0;
  uint4 o[8], g[8];
  const size_t at = row * D + 8 * l, next = (size_t)step * D;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    o[k] = g[k] = make_uint4(0, 0, 0, 0);
    if (k < n) {
      o[k] = __ldcs(reinterpret_cast<const uint4*>(a.out + at + k * next));
      g[k] = *reinterpret_cast<const uint4*>(a.dout + at + k * next);
    }
  }
  float lse = INFINITY;
  if ((l & 7) < n) lse = a.lse[row + (l & 7) * step];
  float mine = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint32_t ow[4] = {o[k].x, o[k].y, o[k].z, o[k].w}, gw[4] = {g[k].x, g[k].y, g[k].z, g[k].w};
    float d = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      d = fmaf(bf16lo(ow[e]), bf16lo(gw[e]), d);
      d = fmaf(bf16hi(ow[e]), bf16hi(gw[e]), d);
    }
#pragma unroll
    for (int e = LPR / 2; e > 0; e >>= 1) d += __shfl_xor_sync(0xffffffffu, d, e);
    if ((l & 7) == k) mine = d;
  }
  if (in) {
    // rows of the second kernel leave delta alone
    const int64_t t = (int64_t)a.pos.q_start[b] + i0 + (a.rpe ? 0 : l & 7);
    const bool lse_lane = l < 8, delta_lane = (LPR == 8 || l >= 8) && ((l & 7) >= n || t >= kBlock);
    if (!a.rpe) {
      float* st = reinterpret_cast<float*>(a.stat + dst * kStatBytes) + (l & 7);
      if (lse_lane) st[0] = -kLog2e * lse;
      if (delta_lane) st[8] = -mine;
    }
    // rows that there are none of: P = 2^-16384 = 0 (and no infinity, which the other
    // selector's zeros would make NaN)
    uint8_t* ag = a.aug + dst * kAugBytes;
    if (lse_lane) put_aug(ag, 0, l & 7, ((l & 7) < n ? -kLog2e * lse : -16384.f) * a.to_score);
    if (delta_lane) put_aug(ag, 1, l & 7, -mine);
  }
  if (a.rpe && blockIdx.x == 0 && threadIdx.x < 16)
    put_aug(a.aug + (size_t)a.groups * kAugBytes, threadIdx.x >> 3, threadIdx.x & 7,
            threadIdx.x < 8 ? -16384.f * a.to_score : 0.f);
}

// ---- inverted lists -------------------------------------------------------------
// For every (sequence, KV block, group) the (query, slot) entries that chose it, in an
// order that the selection alone decides, since sums over a list are not the same in
// every order: a warp walks a chunk of 64 queries slot by slot, and the lanes that
// meet in a list take their places in lane order.  Counts per chunk, then the entries
// of the chunks before, come from a first pass.

// The 16 ids of lane's row of a chunk of 32, -1 where they are not to be used.  Whether one
// is past the local block.
__device__ __forceinline__ bool chunk_ids(const BwdArgs& a, int b, int il, int g, int (&id)[kTopk]) {
  const bool in = il < a.Tp;
  const int i = a.t0 + (in ? il : 0);
  const int4* sr =
      reinterpret_cast<const int4*>(a.sel + (((size_t)b * a.s.T + i) * a.s.G + g) * kTopk);
  const int lb = (int)(((int64_t)a.pos.q_start[b] + i) / kBlock);
  bool bad = false;
#pragma unroll
  for (int v = 0; v < kTopk / 4; ++v) {
    const int4 q4 = sr[v];
    const int x[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      id[4 * v + u] = in && x[u] >= 0 && x[u] <= lb ? x[u] : -1;
      bad |= in && x[u] > lb;
    }
  }
  return bad;
}

// CTA (one warp): chunk, group; FILL false: counts, true: entries.
template <bool FILL>
__global__ void __launch_bounds__(32) bwd_lists_kernel(const __grid_constant__ BwdArgs a) {
  let_next();
  // the first pass's counts need nothing of the call: beside the statistics (see above)
  if (FILL || !a.first) after_previous();
  extern __shared__ int32_t s_cnt[];
  const int lane = threadIdx.x, g = blockIdx.x % a.s.G;
  const int ch = blockIdx.x / a.s.G % a.chunks, b = blockIdx.x / a.s.G / a.chunks;
  int32_t* cnt = a.cnt + (((size_t)b * a.chunks + ch) * a.s.G + g) * a.nbl;
  const int32_t* off = a.off + ((size_t)g * a.s.B + b) * a.nbl;
  // (off and cnt are not used yet where a list is empty: any value will do)
  for (int k = lane; k < a.nbl; k += 32) s_cnt[k] = FILL ? off[k] + cnt[k] : 0;
  __syncwarp();
  bool bad = false;
  for (int r0 = ch * kChunkRows; r0 < min(a.Tp, (ch + 1) * kChunkRows); r0 += 32) {
    const int il = r0 + lane;
    int id[kTopk];
    bad |= chunk_ids(a, b, il, g, id);
    int place[kTopk];
#pragma unroll
    for (int j = 0; j < kTopk; ++j) {
      if (!FILL) {
        if (id[j] >= 0) atomicAdd(&s_cnt[id[j]], 1);
      } else {
        const uint32_t same = __match_any_sync(0xffffffffu, id[j]);
        int at = 0;
        if (id[j] >= 0) at = s_cnt[id[j]] + __popc(same & ((1u << lane) - 1));
        __syncwarp();
        place[j] = id[j] >= 0 ? at : -1;
        if (id[j] >= 0) {
          a.entries[at] = il * kTopk + j;
          if ((same >> lane) == 1) s_cnt[id[j]] = at + 1;   // the last lane of the list
        }
        __syncwarp();
      }
    }
    if (FILL && il < a.Tp) {
      int4* w = reinterpret_cast<int4*>(a.where + (((size_t)b * a.Tp + il) * a.s.G + g) * kTopk);
#pragma unroll
      for (int v = 0; v < kTopk / 4; ++v)
        w[v] = make_int4(place[4 * v], place[4 * v + 1], place[4 * v + 2], place[4 * v + 3]);
    }
  }
  __syncwarp();
  if (!FILL) {
    for (int k = lane; k < a.nbl; k += 32) cnt[k] = s_cnt[k];
    after_previous();
    if (bad) flag_invalid(a.status);       // behind the kernel that clears it
  }
}

// Thread per list: its entries, and for each chunk those of the chunks before.
__global__ void __launch_bounds__(128) bwd_prefix_kernel(const __grid_constant__ BwdArgs a) {
  let_next();
  after_previous();
  const int64_t L = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (L >= (int64_t)a.s.G * a.s.B * a.nbl) return;
  const int kb = (int)(L % a.nbl), b = (int)(L / a.nbl % a.s.B), g = (int)(L / a.nbl / a.s.B);
  const size_t step = (size_t)a.s.G * a.nbl;
  int32_t* c = a.cnt + ((size_t)b * a.chunks * a.s.G + g) * a.nbl + kb;
  int32_t n = 0;
  int k = 0;
  for (; k + 8 <= a.chunks; k += 8) {
    int32_t v[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = c[(k + u) * step];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      c[(k + u) * step] = n;
      n += v[u];
    }
  }
  for (; k < a.chunks; ++k) {
    const int32_t v = c[k * step];
    c[k * step] = n;
    n += v;
  }
  a.count[L] = n;
}

// ---- units ------------------------------------------------------------------
// One CTA: every item (g, b, kb) below kv_len as one unit, or as several of at most
// `piece` tiles, whose sums are joined in their order afterwards.  The units are handed
// out as CTAs become free, so the large ones come first (with a group's large ones together, whose rows
// would stay in L2, 8192 sparse queries take 3 to 5 % longer).
constexpr int kClasses = 64;               // of sizes, the largest first
__device__ __forceinline__ int item_tiles(const BwdArgs& a, int64_t L, int* n) {
  const int kb = (int)(L % a.nbl), b = (int)(L / a.nbl % a.s.B);
  if ((int64_t)kb * kBlock >= a.pos.kv_len[b]) return -1;
  if (a.sel) {
    *n = a.count[L];
    return (*n + a.R - 1) / a.R;
  }
  return *n = (a.nqt - bwd_first_tile(a, b, kb)) * a.hpg;
}
__device__ __forceinline__ int item_class(const BwdArgs& a, int tiles) {
  return kClasses - 1 - (int)((int64_t)min(tiles, a.piece) * (kClasses - 1) / a.piece);
}

__global__ void __launch_bounds__(1024) bwd_units_kernel(const __grid_constant__ BwdArgs a) {
  let_next();
  if (a.sel) after_previous();             // dense units come from the shape: as above
  __shared__ int s_s[32], s_e[32];
  __shared__ int s_class[kClasses];    // units of a class, then the next one's place
  const int64_t n = (int64_t)a.s.G * a.s.B * a.nbl;
  const int64_t per = (n + 1023) / 1024;
  const int64_t lo = min(n, (int64_t)threadIdx.x * per), hi = min(n, lo + per);
  for (int k = threadIdx.x; k < kClasses; k += 1024) s_class[k] = 0;
  __syncthreads();
  int sl = 0, en = 0;
  for (int64_t L = lo; L < hi; ++L) {
    int cnt = 0;
    const int t = item_tiles(a, L, &cnt);
    if (t < 0) continue;
    en += t * a.R;
    const int pieces = t > a.piece ? (t + a.piece - 1) / a.piece : 1;
    atomicAdd(&s_class[item_class(a, t)], pieces);
    if (pieces > 1) sl += pieces;
  }
  // exclusive sums over the threads: in each warp, then of the warps'
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int sl_in = sl, en_in = en;
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, sl_in, o), z = __shfl_up_sync(0xffffffffu, en_in, o);
    if (lane >= o) {
      sl_in += y;
      en_in += z;
    }
  }
  if (lane == 31) {
    s_s[warp] = sl_in;
    s_e[warp] = en_in;
  }
  __syncthreads();
  int sl_all = s_s[lane], en_all = s_e[lane];
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, sl_all, o), z = __shfl_up_sync(0xffffffffu, en_all, o);
    if (lane >= o) {
      sl_all += y;
      en_all += z;
    }
  }
  const int slots = __shfl_sync(0xffffffffu, sl_all, 31);
  const int sl_before = __shfl_sync(0xffffffffu, sl_all, max(warp - 1, 0));
  const int en_before = __shfl_sync(0xffffffffu, en_all, max(warp - 1, 0));
  sl = (warp > 0 ? sl_before : 0) + sl_in - sl;
  en = (warp > 0 ? en_before : 0) + en_in - en;
  if (threadIdx.x < 32) {                  // exclusive scan of the classes, two a lane
    const int v0 = s_class[2 * threadIdx.x], v1 = s_class[2 * threadIdx.x + 1];
    int x = v0 + v1;
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if ((int)threadIdx.x >= o) x += y;
    }
    if (threadIdx.x == 31) a.n_units[0] = x;
    s_class[2 * threadIdx.x] = x - v0 - v1;
    s_class[2 * threadIdx.x + 1] = x - v1;
  }
  if (threadIdx.x == 1023) {
    a.n_units[1] = slots;
    *a.next_unit = *a.next_item = 0;
  }
  __syncthreads();
  for (int64_t L = lo; L < hi; ++L) {
    int cnt = 0;
    const int t = item_tiles(a, L, &cnt);
    if (a.sel) a.off[L] = en;
    if (t < 0) continue;
    const int e0 = en;
    en += t * a.R;
    const int kb = (int)(L % a.nbl), b = (int)(L / a.nbl % a.s.B), g = (int)(L / a.nbl / a.s.B);
    const int x = kb | g << 15 | b << 18;
    const int pieces = t > a.piece ? (t + a.piece - 1) / a.piece : 1;
    // (the order within a class is the run's own: the units do not depend on one another)
    int at = atomicAdd(&s_class[item_class(a, t)], pieces);
    for (int k = 0; k < pieces; ++k) {
      // pieces of nearly the same size
      const int t0 = (int)((int64_t)t * k / pieces), t1 = (int)((int64_t)t * (k + 1) / pieces);
      int first = t0, size = t1 - t0, slot = -1;
      if (a.sel) {
        first = e0 + t0 * a.R;
        size = min(cnt, t1 * a.R) - t0 * a.R;
      }
      if (pieces > 1) {
        slot = sl++;
        a.slots[slot] = make_int4(x, k == 0 ? pieces : 0, 0, 0);
      }
      a.units[at++] = make_int4(x, first, size, slot);
    }
  }
  after_previous();
}

// ---- joins --------------------------------------------------------------------
// dQ of a (query, group): its selected blocks' parts, times the scale.  A warp for N of the
// reads that cover an entry's rows, which are rpe x 32 contiguous bytes per 16 dims; the
// reads of four slots are in flight together.
template <int D, int RPE>
__global__ void __launch_bounds__(256) bwd_join_q_kernel(const __grid_constant__ BwdArgs a) {
  let_next();
  after_previous();
  constexpr int PER = 16 / RPE, R = 128 / RPE;   // 16-dim chunks that a warp's read covers
  constexpr int ALL = D / 16 / PER, N = ALL < 2 ? ALL : 2, U = 4;
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int64_t qg = w / (ALL / N);
  if (qg >= (int64_t)a.s.B * a.Tp * a.s.G) return;
  const int g = (int)(qg % a.s.G);
  const int64_t r = qg / a.s.G;
  const int b = (int)(r / a.Tp), i = a.t0 + (int)(r % a.Tp);
  const int hh = (lane >> 1) % RPE, d0 = (lane & 1) * 8;
  const int ch0 = (int)(w % (ALL / N)) * N * PER + (lane >> 1) / RPE;
  int e = -1;
  if (lane < kTopk) e = a.where[qg * kTopk + lane];
  const uint16_t* part = a.part_dq + (size_t)ch0 * 2048 + hh * 16 + d0;
  float acc[N][8];
#pragma unroll
  for (int k = 0; k < N; ++k)
#pragma unroll
    for (int x = 0; x < 8; ++x) acc[k][x] = 0.f;
#pragma unroll
  for (int j0 = 0; j0 < kTopk; j0 += U) {
    uint4 v[U][N];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int ej = __shfl_sync(0xffffffffu, e, j0 + u);
      const uint16_t* src = part + (size_t)(ej / R) * (D / 16 * 2048) + ej % R * RPE * 16;
#pragma unroll
      for (int k = 0; k < N; ++k) {
        v[u][k] = make_uint4(0, 0, 0, 0);
        if (ej >= 0 && hh < a.hpg) v[u][k] = __ldcs(reinterpret_cast<const uint4*>(src + k * PER * 2048));
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const uint32_t y[4] = {v[u][k].x, v[u][k].y, v[u][k].z, v[u][k].w};
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          acc[k][2 * x] += bf16lo(y[x]);
          acc[k][2 * x + 1] += bf16hi(y[x]);
        }
      }
  }
  if (hh >= a.hpg) return;
  const float f = a.s.scale;
  uint16_t* dst = a.dq + (((size_t)b * a.s.T + i) * a.s.H + g * a.hpg + hh) * D + ch0 * 16 + d0;
#pragma unroll
  for (int k = 0; k < N; ++k)
    *reinterpret_cast<uint4*>(dst + k * PER * 16) =
        make_uint4(pack_bf16(acc[k][0] * f, acc[k][1] * f), pack_bf16(acc[k][2] * f, acc[k][3] * f),
                   pack_bf16(acc[k][4] * f, acc[k][5] * f), pack_bf16(acc[k][6] * f, acc[k][7] * f));
}

// dK, dV of a block in several pieces: CTA (slot, part of the rows); the first slot's
// CTAs add the pieces up in order.
constexpr int kJoinParts = 8;
template <int D>
__global__ void __launch_bounds__(256) bwd_join_kv_kernel(const __grid_constant__ BwdArgs a) {
  let_next();
  after_previous();
  constexpr int ROWS = 2 * kBlock / kJoinParts;
  const int slot = blockIdx.x, part = blockIdx.y;
  if (slot >= a.n_units[1]) return;
  const int4 d = a.slots[slot];
  if (d.y == 0) return;
  const int kb = d.x & 0x7FFF, g = d.x >> 15 & 7, b = d.x >> 18;
  for (int e = threadIdx.x; e < ROWS * (D / 4); e += 256) {
    // dv's 128 rows, then dk's
    const int row = part * ROWS + e / 2 % ROWS, c = (e / 2 / ROWS * 2 + e % 2) * 4;
    const int tok = row % kBlock;
    const bool is_k = row >= kBlock;
    if ((int64_t)kb * kBlock + tok >= a.pos.kv_len[b]) continue;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = 0; k < d.y; ++k) {
      const float4 y = __ldcs(reinterpret_cast<const float4*>(
          a.part_kv + ((((size_t)(slot + k) * 2 + is_k) * (D / 8) + c / 8) * kBlock + tok) * 8 + c % 8));
      x.x += y.x;
      x.y += y.y;
      x.z += y.z;
      x.w += y.w;
    }
    const size_t at = ((((size_t)b * a.s.max_blocks + kb) * kBlock + tok) * a.s.G + g) * D + c;
    float4* acc = reinterpret_cast<float4*>(
        a.acc + (is_k ? (size_t)a.s.cache_blocks() * kBlock * a.s.G * D : 0) + at);
    if (!a.first) {
      const float4 y = *acc;
      x.x += y.x;
      x.y += y.y;
      x.z += y.z;
      x.w += y.w;
    }
    if (!a.last) {
      *acc = x;
      continue;
    }
    const float f = is_k ? a.s.scale : 1.f;
    *reinterpret_cast<uint2*>((is_k ? a.dk : a.dv) + at) =
        make_uint2(pack_bf16(x.x * f, x.y * f), pack_bf16(x.z * f, x.w * f));
  }
}

}  // namespace

cudaError_t launch_bwd_stats(const Shape& s, const Positions& pos, const AttnBwd& t, int rpe,
                             uint8_t* stat, uint8_t* aug, uint32_t stat_groups, int* status,
                             cudaStream_t st) {
  const float to_score = bwd_no_scores(s) ? 1.f : 1.f / (s.scale * kLog2e);
  StatArgs a{s, pos, t.q, t.k, t.v, t.out, t.dout, t.lse, stat, aug, to_score, stat_groups, rpe,
             status};
  const int per_cta = kStatThreads / (s.D / 8);
  const int64_t grps = rpe ? (int64_t)stat_groups : (int64_t)s.B * stat_groups * s.H;
  const unsigned ctas = (unsigned)((grps + per_cta - 1) / per_cta);
  note_launches(1);
  if (s.D == 128) bwd_stat_kernel<128><<<ctas, kStatThreads, 0, st>>>(a);
  else bwd_stat_kernel<64><<<ctas, kStatThreads, 0, st>>>(a);
  if (const cudaError_t e = cudaGetLastError(); e != cudaSuccess) return e;
  bool early = false;
  for (int b = 0; b < s.B; ++b) early |= pos.q_start[b] < kBlock;
  if (early) {
    const int smem = 2 * kBlock * (2 * s.D + 16);
    const cudaError_t e =
        s.D == 128 ? cudaFuncSetAttribute(bwd_stat_first_kernel<128>,
                                          cudaFuncAttributeMaxDynamicSharedMemorySize, smem)
                   : cudaSuccess;
    if (e != cudaSuccess) return e;
    return launch_behind(s.D == 128 ? bwd_stat_first_kernel<128> : bwd_stat_first_kernel<64>,
                         s.B * s.H, 256, smem, st, a);
  }
  return cudaSuccess;
}

cudaError_t launch_bwd_lists(const BwdArgs& a, cudaStream_t st) {
  const size_t smem = (size_t)a.nbl * sizeof(int32_t);       // at most 32768 blocks: 128 KiB
  cudaError_t e;
  if ((e = cudaFuncSetAttribute(bwd_lists_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)(32768 * sizeof(int32_t)))) != cudaSuccess ||
      (e = cudaFuncSetAttribute(bwd_lists_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)(32768 * sizeof(int32_t)))) != cudaSuccess)
    return e;
  const unsigned ctas = (unsigned)((int64_t)a.s.B * a.chunks * a.s.G);
  const int64_t lists = (int64_t)a.s.G * a.s.B * a.nbl;
  if ((e = launch_behind(bwd_lists_kernel<false>, ctas, 32, smem, st, a)) != cudaSuccess ||
      (e = launch_behind(bwd_prefix_kernel, (unsigned)((lists + 127) / 128), 128, 0, st, a)) !=
          cudaSuccess ||
      (e = launch_bwd_units(a, st)) != cudaSuccess)
    return e;
  return launch_behind(bwd_lists_kernel<true>, ctas, 32, smem, st, a);
}

cudaError_t launch_bwd_units(const BwdArgs& a, cudaStream_t st) {
  return launch_behind(bwd_units_kernel, 1, 1024, 0, st, a);
}

cudaError_t launch_bwd_join_q(const BwdArgs& a, cudaStream_t st) {
  const int reads = a.s.D / 16 * a.rpe / 16;               // of an entry's rows, two a warp
  const unsigned ctas = (unsigned)(((int64_t)a.s.B * a.Tp * a.s.G * (reads < 2 ? 1 : reads / 2) + 7) / 8);
  return launch_behind(a.s.D == 128
                           ? (a.rpe == 8 ? bwd_join_q_kernel<128, 8> : bwd_join_q_kernel<128, 16>)
                           : (a.rpe == 8 ? bwd_join_q_kernel<64, 8> : bwd_join_q_kernel<64, 16>),
                       ctas, 256, 0, st, a);
}

cudaError_t launch_bwd_join_kv(const BwdArgs& a, cudaStream_t st) {
  if (a.max_slots == 0) return cudaSuccess;
  const dim3 grid((unsigned)a.max_slots, kJoinParts);
  return launch_behind(a.s.D == 128 ? bwd_join_kv_kernel<128> : bwd_join_kv_kernel<64>, grid, 256, 0,
                       st, a);
}

}  // namespace msa

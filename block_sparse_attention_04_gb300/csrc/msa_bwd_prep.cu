// The attention's backward pass, its small kernels: row statistics, the inverted
// lists of a selection, the units of work, and the joins of partial sums.
#include <climits>

#include "msa_bwd.h"
#include "msa_device.cuh"

namespace msa {
namespace {

// ---- row statistics -----------------------------------------------------------
// Rows by CTAs of the first kind, D/8 lanes each: -lse log2e, and -delta = -dout.out.
// A row whose whole context lies in block 0 (t < 128) leaves delta to CTAs of the
// second kind, which take it from the probabilities, delta = sum P dP / sum P over its
// keys: with few tokens dS is a small difference of dP and delta, and out carries
// rounding of 2^-9 (8 tokens, scores of two units: dq 0.35 % off, now 0.25, what
// rounding dS leaves).  There a warp takes 16 queries of a head against 8 keys at a
// time on mma.sync; the order of the dims in the products is permuted so that a
// lane's fragments of two steps are 16 contiguous bytes.
struct StatArgs {
  Shape s;
  Positions pos;
  const uint16_t *q, *k, *v, *out, *dout;
  const float* lse;
  uint8_t* stat;
  uint32_t groups;
  int rpe;               // 0: dense
  int row_ctas;          // CTAs of the first kind
};
constexpr int kStatThreads = 256;

__device__ __forceinline__ float* stat_row(const StatArgs& a, int b, int i, int h) {
  const int hpg = a.s.H / a.s.G;
  size_t g;
  int r;
  if (a.rpe == 0) {
    g = (size_t)(b * a.s.H + h) * a.groups + (i >> 3);
    r = i & 7;
  } else {
    g = (((size_t)b * a.s.T + i) * a.s.G + h / hpg) * (a.rpe >> 3) + (h % hpg >> 3);
    r = h % hpg & 7;
  }
  return reinterpret_cast<float*>(a.stat + g * kStatBytes) + r;
}

template <int D>
__device__ __forceinline__ void stat_first(const StatArgs& a, int64_t task) {
  // (b, h, 16 queries): the first 128 positions of a sequence are at most 8 such
  const int lane = threadIdx.x & 31, H = a.s.H, G = a.s.G, g = (int)(task / 8 % H) / (H / G);
  const int b = (int)(task / 8 / H), h = (int)(task / 8 % H), i0 = (int)(task % 8) * 16;
  if (b >= a.s.B) return;
  const int n = min(a.s.T, kBlock - a.pos.q_start[b]);   // rows with t < 128
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
    // rows behind the last query's hold anything: they are masked below
    const size_t at = (((size_t)b * a.s.max_blocks * kBlock + j0 + r) * G + g) * D + 8 * c;
    float x[4] = {0.f, 0.f, 0.f, 0.f}, y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < NC; ++k) {
      const uint4 fk = *reinterpret_cast<const uint4*>(a.k + at + 32 * k);
      const uint4 fv = *reinterpret_cast<const uint4*>(a.v + at + 32 * k);
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
    if (c == 0 && i0 + r + 8 * u < n)
      stat_row(a, b, i0 + r + 8 * u, h)[8] = sp[u] == 0.f ? 0.f : -sd[u] / sp[u];
  }
}

template <int D>
__global__ void __launch_bounds__(kStatThreads) bwd_stat_kernel(const __grid_constant__ StatArgs a) {
  constexpr int LPR = D / 8;
  const int H = a.s.H, G = a.s.G, hpg = H / G;
  if ((int)blockIdx.x >= a.row_ctas) {
    stat_first<D>(a, (int64_t)(blockIdx.x - a.row_ctas) * (kStatThreads / 32) + (threadIdx.x >> 5));
    return;
  }
  const int l = threadIdx.x % LPR;
  const int per_row = a.rpe ? G * a.rpe : H;              // rows of a query
  const int Tn = a.rpe ? a.s.T : (int)a.groups * 8;
  const int64_t n = (int64_t)a.s.B * Tn * per_row;
  const int64_t step = (int64_t)a.row_ctas * (kStatThreads / LPR);
  for (int64_t e0 = (int64_t)blockIdx.x * (kStatThreads / LPR); e0 < n; e0 += step) {
    const int64_t e = e0 + threadIdx.x / LPR;
    const bool in = e < n;
    const int64_t r = (in ? e : n - 1) / per_row;
    const int hr = (int)((in ? e : n - 1) - r * per_row);
    const int b = (int)(r / Tn), i = (int)(r - (int64_t)b * Tn);
    const int hh = a.rpe ? hr % a.rpe : 0;
    const int h = a.rpe ? hr / a.rpe * hpg + hh : hr;
    const bool real = in && i < a.s.T && hh < hpg;
    float d = 0.f;
    if (real) {
      const size_t at = (((size_t)b * a.s.T + i) * H + h) * D + 8 * l;
      const uint4 o = *reinterpret_cast<const uint4*>(a.out + at);
      const uint4 g = *reinterpret_cast<const uint4*>(a.dout + at);
      const uint32_t ow[4] = {o.x, o.y, o.z, o.w}, gw[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        d = fmaf(bf16lo(ow[k]), bf16lo(gw[k]), d);
        d = fmaf(bf16hi(ow[k]), bf16hi(gw[k]), d);
      }
    }
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    if (!in || l != 0) continue;
    if (real) {
      float* st = stat_row(a, b, i, h);
      st[0] = -kLog2e * a.lse[((size_t)b * a.s.T + i) * H + h];
      if (a.pos.q_start[b] + (int64_t)i >= kBlock) st[8] = -d;
    } else if (a.rpe) {
      float* st = reinterpret_cast<float*>(
          a.stat + (((r * G + hr / a.rpe) * (a.rpe >> 3)) + (hh >> 3)) * kStatBytes) + (hh & 7);
      st[0] = -INFINITY;
      st[8] = 0.f;
    } else {
      float* st = stat_row(a, b, i, h);
      st[0] = -INFINITY;
      st[8] = 0.f;
    }
  }
  if (a.rpe && blockIdx.x == 0 && threadIdx.x < 16)
    reinterpret_cast<float*>(a.stat + (size_t)a.groups * kStatBytes)[threadIdx.x] =
        threadIdx.x < 8 ? -INFINITY : 0.f;
}

// ---- inverted lists -------------------------------------------------------------
// For every (sequence, KV block, group) the (query, slot) entries that chose it, in an
// order that the selection alone decides, since sums over a list are not the same in
// every order: a warp walks a chunk of 64 queries slot by slot, and the lanes that
// meet in a list take their places in lane order.  Counts per chunk, then the entries
// of the chunks before, come from a first pass.

// The 16 ids of lane's row of a chunk of 32, -1 where they are not to be used.
__device__ __forceinline__ void chunk_ids(const BwdArgs& a, int b, int il, int g, bool flag,
                                          int (&id)[kTopk]) {
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
  if (flag && bad) flag_invalid(a.status);
}

// CTA (one warp): chunk, group; FILL false: counts, true: entries.
template <bool FILL>
__global__ void __launch_bounds__(32) bwd_lists_kernel(const __grid_constant__ BwdArgs a) {
  extern __shared__ int32_t s_cnt[];
  const int lane = threadIdx.x, g = blockIdx.x % a.s.G;
  const int ch = blockIdx.x / a.s.G % a.chunks, b = blockIdx.x / a.s.G / a.chunks;
  int32_t* cnt = a.cnt + (((size_t)b * a.chunks + ch) * a.s.G + g) * a.nbl;
  const int32_t* off = a.off + ((size_t)g * a.s.B + b) * a.nbl;
  // (off and cnt are not used yet where a list is empty: any value will do)
  for (int k = lane; k < a.nbl; k += 32) s_cnt[k] = FILL ? off[k] + cnt[k] : 0;
  __syncwarp();
  for (int r0 = ch * kChunkRows; r0 < min(a.Tp, (ch + 1) * kChunkRows); r0 += 32) {
    const int il = r0 + lane;
    int id[kTopk];
    chunk_ids(a, b, il, g, !FILL, id);
#pragma unroll
    for (int j = 0; j < kTopk; ++j) {
      if (!FILL) {
        if (id[j] >= 0) atomicAdd(&s_cnt[id[j]], 1);
      } else {
        const uint32_t same = __match_any_sync(0xffffffffu, id[j]);
        int at = 0;
        if (id[j] >= 0) at = s_cnt[id[j]] + __popc(same & ((1u << lane) - 1));
        __syncwarp();
        if (id[j] >= 0) {
          a.entries[at] = il * kTopk + j;
          if ((same >> lane) == 1) s_cnt[id[j]] = at + 1;   // the last lane of the list
        }
        __syncwarp();
      }
    }
  }
  __syncwarp();
  if (!FILL)
    for (int k = lane; k < a.nbl; k += 32) cnt[k] = s_cnt[k];
}

// Thread per list: its entries, and for each chunk those of the chunks before.
__global__ void __launch_bounds__(128) bwd_prefix_kernel(const __grid_constant__ BwdArgs a) {
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
// `piece` tiles, whose sums are joined in their order afterwards.
__device__ __forceinline__ int item_tiles(const BwdArgs& a, int64_t L, int* n) {
  const int kb = (int)(L % a.nbl), b = (int)(L / a.nbl % a.s.B);
  if ((int64_t)kb * kBlock >= a.pos.kv_len[b]) return -1;
  if (a.sel) {
    *n = a.count[L];
    return (*n + a.R - 1) / a.R;
  }
  return *n = (a.nqt - bwd_first_tile(a, b, kb)) * a.hpg;
}

__global__ void __launch_bounds__(1024) bwd_units_kernel(const __grid_constant__ BwdArgs a) {
  __shared__ int s_u[1024], s_s[1024], s_e[1024];
  const int64_t n = (int64_t)a.s.G * a.s.B * a.nbl;
  const int64_t per = (n + 1023) / 1024;
  const int64_t lo = min(n, (int64_t)threadIdx.x * per), hi = min(n, lo + per);
  int u = 0, sl = 0, en = 0;
  for (int64_t L = lo; L < hi; ++L) {
    int cnt = 0;
    const int t = item_tiles(a, L, &cnt);
    if (a.sel) en += a.count[L];
    if (t < 0) continue;
    const int pieces = t > a.piece ? (t + a.piece - 1) / a.piece : 1;
    u += pieces;
    if (pieces > 1) sl += pieces;
  }
  s_u[threadIdx.x] = u;
  s_s[threadIdx.x] = sl;
  s_e[threadIdx.x] = en;
  __syncthreads();
  for (int d = 1; d < 1024; d <<= 1) {
    int x = 0, y = 0, z = 0;
    if ((int)threadIdx.x >= d) {
      x = s_u[threadIdx.x - d];
      y = s_s[threadIdx.x - d];
      z = s_e[threadIdx.x - d];
    }
    __syncthreads();
    s_u[threadIdx.x] += x;
    s_s[threadIdx.x] += y;
    s_e[threadIdx.x] += z;
    __syncthreads();
  }
  u = s_u[threadIdx.x] - u;
  sl = s_s[threadIdx.x] - sl;
  en = s_e[threadIdx.x] - en;
  for (int64_t L = lo; L < hi; ++L) {
    int cnt = 0;
    const int t = item_tiles(a, L, &cnt);
    const int e0 = en;
    if (a.sel) {
      a.off[L] = e0;
      en += a.count[L];
    }
    if (t < 0) continue;
    const int kb = (int)(L % a.nbl), b = (int)(L / a.nbl % a.s.B), g = (int)(L / a.nbl / a.s.B);
    const int x = kb | g << 15 | b << 18;
    const int pieces = t > a.piece ? (t + a.piece - 1) / a.piece : 1;
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
      a.units[u++] = make_int4(x, first, size, slot);
    }
  }
  if (threadIdx.x == 1023) {
    a.n_units[0] = u;
    a.n_units[1] = sl;
  }
}

// ---- joins --------------------------------------------------------------------
// dQ of a (query, head): its selected blocks' parts, times the scale.  A warp each.
template <int D>
__global__ void __launch_bounds__(256) bwd_join_q_kernel(const __grid_constant__ BwdArgs a) {
  constexpr int PER = D / 32;
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31, H = a.s.H;
  if (w >= (int64_t)a.s.B * a.Tp * H) return;
  const int h = (int)(w % H), g = h / a.hpg;
  const int64_t r = w / H;
  const int b = (int)(r / a.Tp), i = a.t0 + (int)(r % a.Tp);
  const int lb = (int)(((int64_t)a.pos.q_start[b] + i) / kBlock);
  bool ok = false;
  if (lane < kTopk) {
    const int kb = a.sel[(((size_t)b * a.s.T + i) * a.s.G + g) * kTopk + lane];
    ok = kb >= 0 && kb <= lb;
  }
  const uint32_t m = __ballot_sync(0xffffffffu, ok);
  float acc[PER];
#pragma unroll
  for (int e = 0; e < PER; ++e) acc[e] = 0.f;
  const uint16_t* src = a.part_dq + (size_t)w * kTopk * D + lane * PER;
#pragma unroll
  for (int j = 0; j < kTopk; ++j) {
    if (!(m >> j & 1)) continue;
    if constexpr (PER == 4) {
      const uint2 u = __ldcs(reinterpret_cast<const uint2*>(src + j * D));
      acc[0] += bf16lo(u.x);
      acc[1] += bf16hi(u.x);
      acc[2] += bf16lo(u.y);
      acc[3] += bf16hi(u.y);
    } else {
      const uint32_t u = __ldcs(reinterpret_cast<const unsigned int*>(src + j * D));
      acc[0] += bf16lo(u);
      acc[1] += bf16hi(u);
    }
  }
  uint16_t* dst = a.dq + (((size_t)b * a.s.T + i) * H + h) * D + lane * PER;
#pragma unroll
  for (int e = 0; e < PER; e += 2)
    *reinterpret_cast<uint32_t*>(dst + e) = pack_bf16(acc[e] * a.s.scale, acc[e + 1] * a.s.scale);
}

// dK, dV of a block in several pieces: CTA (slot, part of the rows); the first slot's
// CTAs add the pieces up in order.
constexpr int kJoinParts = 8;
template <int D>
__global__ void __launch_bounds__(256) bwd_join_kv_kernel(const __grid_constant__ BwdArgs a) {
  const int slot = blockIdx.x;
  if (slot >= a.n_units[1]) return;
  const int4 d = a.slots[slot];
  if (d.y == 0) return;
  const int kb = d.x & 0x7FFF, g = d.x >> 15 & 7, b = d.x >> 18;
  constexpr int ROWS = 2 * kBlock / kJoinParts, C4 = D / 4;
  for (int e = threadIdx.x; e < ROWS * C4; e += 256) {
    const int row = blockIdx.y * ROWS + e / C4, c = e % C4 * 4;     // dv's 128 rows, then dk's
    const int tok = row % kBlock;
    const bool is_k = row >= kBlock;
    if ((int64_t)kb * kBlock + tok >= a.pos.kv_len[b]) continue;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = 0; k < d.y; ++k) {
      const float4 y = __ldcs(reinterpret_cast<const float4*>(
          a.part_kv + ((size_t)(slot + k) * 2 * kBlock + row) * D + c));
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
                             uint8_t* stat, uint32_t stat_groups, cudaStream_t st) {
  StatArgs a{s, pos, t.q, t.k, t.v, t.out, t.dout, t.lse, stat, stat_groups, rpe, 0};
  const int lpr = s.D / 8, per_cta = kStatThreads / lpr;
  const int64_t rows = (int64_t)s.B * (rpe ? (int64_t)s.T * s.G * rpe : (int64_t)stat_groups * 8 * s.H);
  const int64_t ctas = (rows + per_cta - 1) / per_cta;
  a.row_ctas = (int)(ctas < 8 * kBwdSms ? ctas : 8 * kBwdSms);
  bool early = false;
  for (int b = 0; b < s.B; ++b) early |= pos.q_start[b] < kBlock;
  const int64_t tasks = early ? (int64_t)s.B * s.H * 8 : 0;   // a warp each
  const unsigned grid = (unsigned)(a.row_ctas + (tasks + kStatThreads / 32 - 1) / (kStatThreads / 32));
  note_launches(1);
  if (s.D == 128) bwd_stat_kernel<128><<<grid, kStatThreads, 0, st>>>(a);
  else bwd_stat_kernel<64><<<grid, kStatThreads, 0, st>>>(a);
  return cudaGetLastError();
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
  note_launches(3);
  bwd_lists_kernel<false><<<ctas, 32, smem, st>>>(a);
  bwd_prefix_kernel<<<(unsigned)((lists + 127) / 128), 128, 0, st>>>(a);
  if ((e = launch_bwd_units(a, st)) != cudaSuccess) return e;
  bwd_lists_kernel<true><<<ctas, 32, smem, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_bwd_units(const BwdArgs& a, cudaStream_t st) {
  note_launches(1);
  bwd_units_kernel<<<1, 1024, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_bwd_join_q(const BwdArgs& a, cudaStream_t st) {
  const unsigned ctas = (unsigned)(((int64_t)a.s.B * a.Tp * a.s.H + 7) / 8);
  note_launches(1);
  if (a.s.D == 128) bwd_join_q_kernel<128><<<ctas, 256, 0, st>>>(a);
  else bwd_join_q_kernel<64><<<ctas, 256, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_bwd_join_kv(const BwdArgs& a, cudaStream_t st) {
  if (a.max_slots == 0) return cudaSuccess;
  const dim3 grid((unsigned)a.max_slots, kJoinParts);
  note_launches(1);
  if (a.s.D == 128) bwd_join_kv_kernel<128><<<grid, 256, 0, st>>>(a);
  else bwd_join_kv_kernel<64><<<grid, 256, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace msa

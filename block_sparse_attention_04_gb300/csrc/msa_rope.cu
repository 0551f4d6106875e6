// The step in front of the attention (msa_rope_append) and its backward pass:
// the RMS norm of each query and key head, the rotation of its first dims by the
// token's position, and the rows of K, V and K_idx written into the block-major
// caches, in one pass over the projections.
//
//   forward   n = x w / sqrt(mean(x^2) + eps);  (a, b) -> (a c - b s, b c + a s)
//   backward  with dn the rotation of dy by the opposite angle, r = 1 / sqrt(...):
//             dw = sum dn x r;  g = dn w;  dx = r (g - x r mean(g x r))
//
// Bound by HBM: a token's rows are read once and written once.  A row (one head of
// a token) is spread over D/8 lanes of 8 dims: 16-byte accesses, the norm's sum by
// log2(D/8) shuffles, and with halves rotated (i with i + rot/2) the partner's 8
// values from the lane rot/16 away.  The angles of a token are made once per
// CTA for all of its heads: t * inv_freq in turns and its fraction in fp64 (fp32
// would leave 2^-24 * t turns of error: a third of a radian at t = 1M), sine and
// cosine of the fraction in fp32.
//
// What holds it up is the arithmetic of a row, so a row is C x + S y, y its partners, with
// the norm's weights inside C and S (one table per token for the queries, one for K), in
// packed fp32; a thread has the same rows of each token, and the next token's come by
// cp.async while one is worked on.  Many small CTAs, as each waits at a barrier per token.
// 8192 tokens, 48/8 heads of 128, half rotated: 47.5 us (270 MB, 0.84 of the copy rate; rows
// in registers, index arithmetic per row and tables of angles: 84).  Backward, 8192 tokens:
// 70 us and 3 for the weights' join (386 MB; 168 before).
#include <algorithm>
#include <type_traits>

#include "msa_device.cuh"
#include "msa_tma.h"
#include "msa_train.h"

namespace msa {
namespace {

constexpr int kStages = 2;                  // tokens in shared memory
constexpr int kRopeThreads = 128;           // (256: 46 and 87 us; 3 x 1000 tokens 15 for 11)
constexpr int kRows = 5;                    // rows of a token that a thread has, at most
constexpr int kFwdCtas = 8, kBwdCtas = 4;   // of an SM
constexpr int kBwdMaxCtas = 1024;
constexpr int kHalfRot = MSA_MAX_ROT / 2;

struct RopeArgs {
  Shape s;
  Positions pos;
  int rot;
  float eps, mscale;
  double turns[kHalfRot];      // inv_freq / 2 pi
  RopeIn in;
  RopeGrads g;
  uint16_t *q_out, *k_cache, *v_cache, *kidx_cache;
  int* status;
  int parts;                   // CTAs that share a run of tokens (each a part of its rows)
  float* part_w;               // backward: [CTAs][2][D] sums of the weights' gradients
};

// Sum over the LPR lanes of a row (LPR a power of two, rows aligned in the warp).
template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

template <int LPR>
__device__ __forceinline__ float2 row_sum(float2 x) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1)
    x = fadd2(x, make_float2(__shfl_xor_sync(0xffffffffu, x.x, o),
                             __shfl_xor_sync(0xffffffffu, x.y, o)));
  return x;
}

// What the rows of one token need: the turn of a row as out = C x + S y, y the partners'
// values, as float4s of C and S by lane (the lanes side by side, so that a warp's 16-byte
// reads meet no bank twice), and its cache row (block * 128 + token within it), or -1.
// With the norms' weights in C and S there is one table for the queries and one for K.
template <int D, int TYPES>
struct TokenTable {
  float4 cs[TYPES][4][D / 8];
  int64_t slot;
  __device__ __forceinline__ float* at(int type, int is_s, int d) {
    return reinterpret_cast<float*>(&cs[type][2 * is_s + d % 8 / 4][d / 8]) + d % 4;
  }
};
// A lane's C and S, or its 8 weights, as pairs.
template <int N>
struct Pairs {
  float2 v[N];
  __device__ __forceinline__ void set4(int j, const float4& f) {
    v[2 * j] = make_float2(f.x, f.y);
    v[2 * j + 1] = make_float2(f.z, f.w);
  }
};

// A walk over the call's tokens in steps of `step`, without a division per token.
struct TokenWalk {
  int64_t tok;
  int b, i, step_b, step_i, T;
  __device__ TokenWalk(int64_t first, int step, int T_) : tok(first), T(T_) {
    b = (int)(first / T);
    i = (int)(first - (int64_t)b * T);
    step_b = step / T;
    step_i = step % T;
  }
  __device__ void next(int step) {
    tok += step;
    b += step_b;
    i += step_i;
    if (i >= T) {
      i -= T;
      ++b;
    }
  }
};

// The pair of dims whose angle a thread makes: the last threads', whose warps have the
// fewest rows.
__device__ __forceinline__ int pair_of_thread() { return kRopeThreads - 1 - (int)threadIdx.x; }
// A thread's pair of dims: 2 p and 2 p + 1, or p and p + rot / 2.
template <bool INTER>
__device__ __forceinline__ int2 pair_dims(const RopeArgs& a) {
  const int p = pair_of_thread();
  return INTER ? make_int2(2 * p, 2 * p + 1) : make_int2(p, p + (a.rot >> 1));
}
// cosine and sine of the thread's pair for the walk's token, times mscale.
__device__ __forceinline__ float2 pair_angle(const RopeArgs& a, const TokenWalk& w) {
  const double u = (double)((int64_t)a.pos.q_start[w.b] + w.i) * a.turns[pair_of_thread()];
  float sn, c;
  sincospif(2.f * (float)(u - rint(u)), &sn, &c);
  return make_float2(c * a.mscale, sn * a.mscale);
}
__device__ __forceinline__ float weight_of(const uint16_t* w, int d) {
  return w ? bf16lo(w[d]) : 1.f;
}
// The partners of a lane's dims, as bf16: the other of each two, or with halves rotated the
// dims of the lane rot/16 away, at `other`.  Dims that are not rotated have zeros (S is zero
// there too, and an infinity stays what it is).
template <bool INTER>
__device__ __forceinline__ uint4 partners(const uint4& v, const uint4* other, bool rotated) {
  if (!rotated) return make_uint4(0, 0, 0, 0);
  if (!INTER) return *other;
  return make_uint4(__byte_perm(v.x, 0, 0x1032), __byte_perm(v.y, 0, 0x1032),
                    __byte_perm(v.z, 0, 0x1032), __byte_perm(v.w, 0, 0x1032));
}
template <int LPR>
__device__ __forceinline__ int partner_thread(int rot, int l) {
  const int h = rot >> 4;
  return (int)threadIdx.x - l + (l < h ? l + h : (l < 2 * h ? l - h : l));
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ void unpack4(const uint4& u, float2 (&x)[4]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = make_float2(bf16lo(w[i]), bf16hi(w[i]));
}
__device__ __forceinline__ uint4 pack4(const float2 (&x)[4]) {
  return make_uint4(pack_bf16(x[0].x, x[0].y), pack_bf16(x[1].x, x[1].y),
                    pack_bf16(x[2].x, x[2].y), pack_bf16(x[3].x, x[3].y));
}
// The rows u of the thread's warp that are anything but V.
template <int ROWS, int U>
__device__ __forceinline__ unsigned rows_with_work(int row, int n_rows, int n_qk) {
  unsigned m = 0;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int r = u * ROWS + row;
    if (__any_sync(0xffffffffu, r < n_rows && r < n_qk)) m |= 1u << u;
  }
  return m;
}

// CTA (run, part): every `gridDim.x / parts`-th token, of its H + 2 G rows (query heads, K,
// V) the part's.  A thread has the same rows of each token, so that types and offsets are
// worked out once; a token's rows are loaded, and its table made, while the one before it
// is worked on.
template <int D, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, kFwdCtas) rope_append_kernel(
    const __grid_constant__ RopeArgs a) {
  constexpr int LPR = D / 8, ROWS = kRopeThreads / LPR, U = kRows;
  __shared__ TokenTable<D, 2> ts[2];
  const int n_tok = (int)((int64_t)a.s.B * a.s.T);
  const int step = gridDim.x / a.parts, part = blockIdx.x % a.parts;
  const int H = a.s.H, G = a.s.G, heads = H + 2 * G;
  const int per = (heads + a.parts - 1) / a.parts;
  const int r0 = part * per, n_rows = min(heads, r0 + per) - r0;
  const int l = threadIdx.x % LPR, row = threadIdx.x / LPR;
  const int n_q = H - r0, n_qk = H + G - r0;  // rows below: queries, queries and K
  const int q_rows = min(n_q, n_rows);
  const unsigned work = rows_with_work<ROWS, U>(row, n_rows, n_qk);
  const int other = partner_thread<LPR>(a.rot, l);
  const bool rotated = 8 * l < a.rot;
  const int idx_at = part == a.parts - 1 && a.in.k_idx && (int)threadIdx.x < a.s.Di / 8
                         ? (int)threadIdx.x * 8 : -1;
  const int at = (r0 + row) * D + 8 * l;     // of the thread's first row
  extern __shared__ uint4 stage[];           // [kStages][U][threads], then K_idx [kStages][16]
  uint4* idx_stage = stage + kStages * U * kRopeThreads;
  TokenWalk tw(blockIdx.x / a.parts, step, a.s.T);
  const uint16_t* q = a.in.q + tw.tok * a.in.q_stride + at;
  const uint16_t* k = a.in.k + tw.tok * a.in.k_stride + at - H * D;
  const uint16_t* v = a.in.v + tw.tok * a.in.v_stride + at - (H + G) * D;
  const uint16_t* ki = idx_at >= 0 ? a.in.k_idx + tw.tok * a.s.Di + idx_at : nullptr;
  int64_t load_tok = tw.tok;                 // the token that q, k, v, ki point to
  auto load = [&](int st) {
    if (load_tok < n_tok) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = u * ROWS + row;
        uint4* dst = stage + (st * U + u) * kRopeThreads + threadIdx.x;
        if ((u + 1) * ROWS <= q_rows) cp_async_16(smem_u32(dst), q + u * ROWS * D);
        else if (r < n_rows) cp_async_16(smem_u32(dst), (r < n_q ? q : r < n_qk ? k : v) + u * ROWS * D);
      }
      if (ki) cp_async_16(smem_u32(idx_stage + st * 16 + threadIdx.x), ki);
      q += step * a.in.q_stride;
      k += step * a.in.k_stride;
      v += step * a.in.v_stride;
      if (ki) ki += (int64_t)step * a.s.Di;
      load_tok += step;
    }
    cp_async_commit();
  };
  const int2 pd = pair_dims<INTER>(a);
  float pw[2][2] = {};
  auto fill = [&](TokenTable<D, 2>& t) {
    if (pair_of_thread() < a.rot >> 1) {
      const float2 cs = pair_angle(a, tw);
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        *t.at(y, 0, pd.x) = cs.x * pw[y][0];
        *t.at(y, 1, pd.x) = -cs.y * pw[y][1];
        *t.at(y, 0, pd.y) = cs.x * pw[y][1];
        *t.at(y, 1, pd.y) = cs.y * pw[y][0];
      }
    }
    if (threadIdx.x == kRopeThreads - 65) {  // of a warp without angles
      const int64_t pos = (int64_t)a.pos.q_start[tw.b] + tw.i;
      const int64_t pb = cache_block(a.s, tw.b, (int)(pos / kBlock), nullptr);
      t.slot = pb < 0 ? -1 : pb * kBlock + pos % kBlock;   // outside the pool: not written
    }
  };
#pragma unroll
  for (int st = 0; st < kStages - 1; ++st) load(st);
  if (pair_of_thread() < a.rot >> 1) {
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      pw[y][0] = weight_of(y ? a.in.k_weight : a.in.q_weight, pd.x);
      pw[y][1] = weight_of(y ? a.in.k_weight : a.in.q_weight, pd.y);
    }
  }
  for (int e = a.rot + threadIdx.x; e < 2 * D; e += kRopeThreads) {
    const int y = e / D, d = e % D;          // dims that are not rotated
    if (d < a.rot) continue;
    const float wt = weight_of(y ? a.in.k_weight : a.in.q_weight, d);
#pragma unroll
    for (int buf = 0; buf < 2; ++buf) {
      *ts[buf].at(y, 0, d) = wt;
      *ts[buf].at(y, 1, d) = 0.f;
    }
  }
  fill(ts[0]);
  // The first CTA looks through the call's table entries and writes the status, so that
  // nothing has to clear it before the launch (a memset: 3 us of 15).
  bool outside = false;
  if (blockIdx.x == 0 && a.s.bt) {
    const int blocks = (a.s.T + kBlock - 1) / kBlock + 1;      // of a sequence, at most
    for (int64_t e = threadIdx.x; e < (int64_t)a.s.B * blocks; e += kRopeThreads) {
      const int b = (int)(e / blocks);
      const int64_t kb = a.pos.q_start[b] / kBlock + e % blocks;
      if (kb * kBlock < (int64_t)a.pos.q_start[b] + a.s.T)
        outside |= cache_block(a.s, b, (int)kb, nullptr) < 0;
    }
  }
  outside = __syncthreads_or(outside);
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = outside ? kDevInvalid : 0;
  for (int buf = 0, st = 0;; buf ^= 1, st = st + 1 == kStages ? 0 : st + 1) {
    const int64_t tok = tw.tok;
    load(st == 0 ? kStages - 1 : st - 1);    // read by every thread before the last barrier
    cp_async_wait<kStages - 1>();            // for all but the newest token's
    __syncwarp();                            // a row's copies are its warp's
    tw.next(step);
    const bool more = tw.tok < n_tok;
    if (more) fill(ts[buf ^ 1]);
    const int64_t slot = ts[buf].slot;
    uint16_t* q_out = a.q_out + tok * H * D + at;
    uint16_t* k_out = a.k_cache + slot * G * D + at - H * D;
    uint16_t* v_out = a.v_cache + slot * G * D + at - (H + G) * D;
    Pairs<8> t;
    // Row u, of queries only (`qs`) or any.
    auto do_row = [&](int u, auto qs) {
      constexpr bool QS = decltype(qs)::value;
      const int r = u * ROWS + row;
      const bool is_q = QS || r < n_q;
      if (u == 0 || is_q != (r - ROWS < n_q)) {
#pragma unroll
        for (int j = 0; j < 4; ++j) t.set4(j, ts[buf].cs[is_q ? 0 : 1][j][l]);
      }
      const uint4* in = stage + (st * U + u) * kRopeThreads;
      uint4 out = in[threadIdx.x];
      if (QS || (work >> u & 1)) {            // the same in every lane
        float2 x[4], y[4], sq = make_float2(0.f, 0.f);
        unpack4(out, x);
        unpack4(partners<INTER>(out, in + other, rotated), y);
#pragma unroll
        for (int i = 0; i < 4; ++i) sq = ffma2(x[i], x[i], sq);
        const float ss = row_sum<LPR>(sq.x + sq.y);
        float rs = 1.f;
        if (is_q ? a.in.q_weight != nullptr : a.in.k_weight != nullptr)
          rs = rsqrtf(ss * (1.f / D) + a.eps);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          x[i] = ffma2(fmul2(y[i], both(rs)), t.v[4 + i], fmul2(fmul2(x[i], both(rs)), t.v[i]));
        if (QS || r < n_qk) out = pack4(x);
      }
      if (QS) *reinterpret_cast<uint4*>(q_out + u * ROWS * D) = out;
      else if (r < n_rows && (is_q || slot >= 0))
        *reinterpret_cast<uint4*>((is_q ? q_out : r < n_qk ? k_out : v_out) + u * ROWS * D) = out;
    };
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // the same in every lane; a part's rows are queries first
      if ((u + 1) * ROWS <= q_rows) do_row(u, std::true_type());
      else if (u * ROWS < n_rows) do_row(u, std::false_type());
    }
    if (ki && slot >= 0)
      *reinterpret_cast<uint4*>(a.kidx_cache + slot * a.s.Di + idx_at) =
          idx_stage[st * 16 + threadIdx.x];
    if (!more) return;
    __syncthreads();
  }
}

// ---- backward ---------------------------------------------------------------
// The same walk over the tokens.  A thread sums the weights' gradients of its 8 dims over
// all its rows; the CTA's sums go to part_w, which a second kernel adds up, in fixed orders.
template <int D, bool INTER>
__global__ void __launch_bounds__(kRopeThreads, kBwdCtas) rope_append_bwd_kernel(
    const __grid_constant__ RopeArgs a) {
  constexpr int LPR = D / 8, ROWS = kRopeThreads / LPR, U = kRows;
  __shared__ TokenTable<D, 1> ts[2];
  __shared__ float4 w[2][2][LPR];
  const int n_tok = (int)((int64_t)a.s.B * a.s.T);
  const int step = gridDim.x / a.parts, part = blockIdx.x % a.parts;
  const int H = a.s.H, G = a.s.G, heads = H + 2 * G;
  const int per = (heads + a.parts - 1) / a.parts;
  const int r0 = part * per, n_rows = min(heads, r0 + per) - r0;
  const int l = threadIdx.x % LPR, row = threadIdx.x / LPR;
  const int n_q = H - r0, n_qk = H + G - r0;
  const int q_rows = min(n_q, n_rows);
  const unsigned work = rows_with_work<ROWS, U>(row, n_rows, n_qk);
  const int other = partner_thread<LPR>(a.rot, l);
  const bool rotated = 8 * l < a.rot;
  const bool q_norm = a.in.q_weight != nullptr, k_norm = a.in.k_weight != nullptr;
  const int at = (r0 + row) * D + 8 * l;
  TokenWalk tw(blockIdx.x / a.parts, step, a.s.T);
  extern __shared__ uint4 stage[];           // [kStages][gradients, inputs][U][threads]
  let_next();
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0;
  TokenWalk lw = tw;                         // the token to load next
  const uint16_t* q = a.in.q + lw.tok * a.in.q_stride + at;
  const uint16_t* k = a.in.k + lw.tok * a.in.k_stride + at - H * D;
  const uint16_t* gq = a.g.dq_out + lw.tok * H * D + at;
  auto load = [&](int st) {
    if (lw.tok < n_tok) {
      const int64_t slot =
          (int64_t)lw.b * a.s.max_blocks * kBlock + a.pos.q_start[lw.b] + lw.i;
      const uint16_t* gk = a.g.dk_cache + slot * G * D + at - H * D;
      const uint16_t* gv = a.g.dv_cache + slot * G * D + at - (H + G) * D;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = u * ROWS + row;
        uint4* dst = stage + (st * 2 * U + u) * kRopeThreads + threadIdx.x;
        if ((u + 1) * ROWS <= q_rows) {
          cp_async_16(smem_u32(dst), gq + u * ROWS * D);
          if (q_norm) cp_async_16(smem_u32(dst + U * kRopeThreads), q + u * ROWS * D);
        } else if (r < n_rows) {
          cp_async_16(smem_u32(dst), (r < n_q ? gq : r < n_qk ? gk : gv) + u * ROWS * D);
          if (r < n_q ? q_norm : r < n_qk && k_norm)
            cp_async_16(smem_u32(dst + U * kRopeThreads), (r < n_q ? q : k) + u * ROWS * D);
        }
      }
      q += step * a.in.q_stride;
      k += step * a.in.k_stride;
      gq += (int64_t)step * H * D;
      lw.next(step);
    }
    cp_async_commit();
  };
  const int2 pd = pair_dims<INTER>(a);
  auto fill = [&](TokenTable<D, 1>& t) {
    if (pair_of_thread() < a.rot >> 1) {
      const float2 cs = pair_angle(a, tw);
      *t.at(0, 0, pd.x) = *t.at(0, 0, pd.y) = cs.x;
      *t.at(0, 1, pd.x) = cs.y;
      *t.at(0, 1, pd.y) = -cs.y;
    }
  };
#pragma unroll
  for (int st = 0; st < kStages - 1; ++st) load(st);
  for (int e = threadIdx.x; e < 2 * D; e += kRopeThreads)
    reinterpret_cast<float*>(&w[e / D][e % 8 / 4][e % D / 8])[e % 4] =
        weight_of(e < D ? a.in.q_weight : a.in.k_weight, e % D);
  for (int d = a.rot + threadIdx.x; d < D; d += kRopeThreads) {
#pragma unroll
    for (int buf = 0; buf < 2; ++buf) {
      *ts[buf].at(0, 0, d) = 1.f;
      *ts[buf].at(0, 1, d) = 0.f;
    }
  }
  fill(ts[0]);
  float2 dw[2][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) dw[0][i] = dw[1][i] = make_float2(0.f, 0.f);
  __syncthreads();
  for (int buf = 0, st = 0;; buf ^= 1, st = st + 1 == kStages ? 0 : st + 1) {
    const int64_t tok = tw.tok;
    load(st == 0 ? kStages - 1 : st - 1);
    cp_async_wait<kStages - 1>();            // for all but the newest token's
    __syncwarp();
    tw.next(step);
    const bool more = tw.tok < n_tok;
    if (more) fill(ts[buf ^ 1]);
    uint16_t* dq = a.g.dq + tok * a.g.dq_stride + at;
    uint16_t* dk = a.g.dk + tok * a.g.dk_stride + at - H * D;
    uint16_t* dv = a.g.dv + tok * a.g.dv_stride + at - (H + G) * D;
    Pairs<8> t;
    Pairs<4> wt;
#pragma unroll
    for (int j = 0; j < 4; ++j) t.set4(j, ts[buf].cs[0][j][l]);
    auto do_row = [&](int u, auto qs) {
      constexpr bool QS = decltype(qs)::value;
      const int r = u * ROWS + row;
      const bool is_q = QS || r < n_q, is_k = !is_q && r < n_qk;
      if (u == 0 || is_q != (r - ROWS < n_q)) {
#pragma unroll
        for (int j = 0; j < 2; ++j) wt.set4(j, w[is_q ? 0 : 1][j][l]);
      }
      const uint4* in = stage + (st * 2 * U + u) * kRopeThreads;
      uint4 out = in[threadIdx.x];
      if (QS || (work >> u & 1)) {            // the same in every lane
        const bool norm = is_q ? q_norm : is_k && k_norm;
        float2 x[4], g[4], y[4];
        unpack4(out, g);
        unpack4(partners<INTER>(out, in + other, rotated), y);
        unpack4(norm && r < n_rows ? in[U * kRopeThreads + threadIdx.x] : make_uint4(0, 0, 0, 0), x);
        float2 sq = make_float2(0.f, 0.f), sm = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          g[i] = ffma2(y[i], t.v[4 + i], fmul2(g[i], t.v[i]));
          sq = ffma2(x[i], x[i], sq);
          sm = ffma2(fmul2(g[i], wt.v[i]), x[i], sm);
        }
        const float2 sums = row_sum<LPR>(make_float2(sq.x + sq.y, sm.x + sm.y));
        if (norm && (QS || r < n_rows)) {
          const float rs = rsqrtf(sums.x * (1.f / D) + a.eps);
          const float mean = -sums.y * rs * rs * (1.f / D);   // -mean(g w x r), times r
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 xr = fmul2(x[i], both(rs));
            if (is_q) dw[0][i] = ffma2(g[i], xr, dw[0][i]);
            else dw[1][i] = ffma2(g[i], xr, dw[1][i]);
            g[i] = fmul2(both(rs), ffma2(x[i], both(mean), fmul2(g[i], wt.v[i])));
          }
        }
        if (QS || r < n_qk) out = pack4(g);
      }
      if (QS || r < n_rows)
        *reinterpret_cast<uint4*>((is_q ? dq : is_k ? dk : dv) + u * ROWS * D) = out;
    };
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if ((u + 1) * ROWS <= q_rows) do_row(u, std::true_type());
      else if (u * ROWS < n_rows) do_row(u, std::false_type());
    }
    if (!more) break;
    __syncthreads();
  }
  if (!a.in.q_weight && !a.in.k_weight) return;
  // the rows of a warp, then its CTA's warps
  auto red = reinterpret_cast<float (*)[2][D]>(stage);   // [warps]: the rows are done with
  __syncthreads();
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float x = i % 2 ? dw[j][i / 2].y : dw[j][i / 2].x;
#pragma unroll
      for (int o = 16; o >= LPR; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
      if ((threadIdx.x & 31) < LPR) red[threadIdx.x >> 5][j][8 * l + i] = x;
    }
  __syncthreads();
  for (int d = threadIdx.x; d < 2 * D; d += kRopeThreads) {
    float x = 0.f;
    for (int wp = 0; wp < kRopeThreads / 32; ++wp) x += red[wp][d / D][d % D];
    a.part_w[(size_t)blockIdx.x * 2 * D + d] = x;
  }
}

// The CTAs' sums of 32 columns (q's D, then k's): each warp every 32nd CTA's, then the warps.
template <int D>
__global__ void __launch_bounds__(1024) rope_join_weights_kernel(const __grid_constant__ RopeArgs a,
                                                                 int ctas) {
  __shared__ float sum[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int d = blockIdx.x * 32 + lane;
  after_previous();
  float x = 0.f;
#pragma unroll 8
  for (int c = warp; c < ctas; c += 32) x += __ldcg(a.part_w + (size_t)c * 2 * D + d);
  sum[warp][lane] = x;
  __syncthreads();
  if (warp > 0) return;
  x = 0.f;
#pragma unroll
  for (int w = 0; w < 32; ++w) x += sum[w][lane];
  if (d < D ? a.in.q_weight != nullptr : a.in.k_weight != nullptr)
    (d < D ? a.g.dq_weight : a.g.dk_weight)[d % D] = x;
}

RopeArgs rope_args(const Shape& s, const Positions& pos, const msa_rope& r, const RopeIn& in) {
  RopeArgs a{};
  a.s = s;
  a.pos = pos;
  a.rot = r.rot;
  a.eps = r.eps;
  a.mscale = r.mscale;
  for (int i = 0; i < r.rot / 2; ++i) a.turns[i] = r.inv_freq[i] / 6.283185307179586476925;
  a.in = in;
  return a;
}

// CTAs of a call, `resident` at most unless a token alone takes more: a token's rows over as
// many CTAs as its threads' rows ask for, or more where there are fewer tokens than CTAs.
unsigned rope_grid(RopeArgs& a, int64_t resident, int threads, int rows_each) {
  const int64_t n = (int64_t)a.s.B * a.s.T;
  const int heads = a.s.H + 2 * a.s.G, rows = threads / (a.s.D / 8);
  const int least = (heads + rows * rows_each - 1) / (rows * rows_each);
  const int most = (heads + rows - 1) / rows;
  int64_t parts = n < resident ? resident / n : 1;
  if (parts > most) parts = most;
  if (parts < least) parts = least;
  a.parts = (int)parts;
  int64_t runs = resident / parts > 0 ? resident / parts : 1;
  if (runs > n) runs = n;
  return (unsigned)(runs * parts);
}

template <typename K>
cudaError_t launch_rows(K kernel, unsigned ctas, int threads, int smem, const RopeArgs& a,
                        cudaStream_t st) {
  if (cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           smem);
      e != cudaSuccess)
    return e;
  note_launches(1);
  kernel<<<ctas, threads, smem, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope_append(const Shape& s, const Positions& pos, const msa_rope& r,
                               const RopeIn& in, uint16_t* q_out, uint16_t* k_cache,
                               uint16_t* v_cache, uint16_t* kidx_cache, int* status,
                               cudaStream_t st) {
  RopeArgs a = rope_args(s, pos, r, in);
  a.q_out = q_out;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.kidx_cache = kidx_cache;
  a.status = status;
  const unsigned ctas = rope_grid(a, (int64_t)sm_count() * kFwdCtas, kRopeThreads, kRows);
  constexpr int smem = kStages * (kRows * kRopeThreads + 16) * (int)sizeof(uint4);
  if (s.D == 128)
    return r.interleaved ? launch_rows(rope_append_kernel<128, true>, ctas, kRopeThreads, smem, a, st)
                         : launch_rows(rope_append_kernel<128, false>, ctas, kRopeThreads, smem, a, st);
  return r.interleaved ? launch_rows(rope_append_kernel<64, true>, ctas, kRopeThreads, smem, a, st)
                       : launch_rows(rope_append_kernel<64, false>, ctas, kRopeThreads, smem, a, st);
}

size_t rope_bwd_scratch_bytes() { return (size_t)kBwdMaxCtas * 2 * 128 * sizeof(float); }

cudaError_t launch_rope_append_bwd(const Shape& s, const Positions& pos, const msa_rope& r,
                                   const RopeIn& in, const RopeGrads& g, int* status,
                                   char* base, cudaStream_t st) {
  RopeArgs a = rope_args(s, pos, r, in);
  a.g = g;
  a.status = status;
  a.part_w = reinterpret_cast<float*>(base);
  const unsigned ctas = rope_grid(a, std::min<int64_t>((int64_t)sm_count() * kBwdCtas, kBwdMaxCtas), kRopeThreads, kRows);
  constexpr int smem = kStages * 2 * kRows * kRopeThreads * (int)sizeof(uint4);
  const cudaError_t e =
      s.D == 128
          ? (r.interleaved
                 ? launch_rows(rope_append_bwd_kernel<128, true>, ctas, kRopeThreads, smem, a, st)
                 : launch_rows(rope_append_bwd_kernel<128, false>, ctas, kRopeThreads, smem, a, st))
          : (r.interleaved
                 ? launch_rows(rope_append_bwd_kernel<64, true>, ctas, kRopeThreads, smem, a, st)
                 : launch_rows(rope_append_bwd_kernel<64, false>, ctas, kRopeThreads, smem, a, st));
  if (e != cudaSuccess || (!in.q_weight && !in.k_weight)) return e;
  return s.D == 128
             ? launch_behind(rope_join_weights_kernel<128>, 8, 1024, 0, st, a, (int)ctas)
             : launch_behind(rope_join_weights_kernel<64>, 4, 1024, 0, st, a, (int)ctas);
}

}  // namespace msa

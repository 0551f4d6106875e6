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
// values come from the lane rot/16 away.  The angles of a token are made once per
// CTA for all of its heads: t * inv_freq in turns and its fraction in fp64 (fp32
// would leave 2^-24 * t turns of error: a third of a radian at t = 1M), sine and
// cosine of the fraction in fp32.
#include "msa_device.cuh"
#include "msa_tma.h"
#include "msa_train.h"

namespace msa {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kHalfRot = MSA_MAX_ROT / 2;

struct RopeArgs {
  Shape s;
  Positions pos;
  int rot, interleaved;
  float eps, mscale;
  double turns[kHalfRot];      // inv_freq / 2 pi
  RopeIn in;
  RopeGrads g;
  uint16_t *q_out, *k_cache, *v_cache, *kidx_cache;
  int* status;
  int parts;                   // CTAs that share a run of tokens (each a part of its rows)
  float* part_w;               // backward: [CTAs][2][D] sums of the weights' gradients
  unsigned* counter;
};

__device__ __forceinline__ uint4 ldg16(const uint16_t* p) {
  return *reinterpret_cast<const uint4*>(p);
}
__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16lo(w[i]);
    x[2 * i + 1] = bf16hi(w[i]);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                    pack_bf16(x[6], x[7]));
}
// Sum over the LPR lanes of a row (LPR a power of two, rows aligned in the warp).
template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Sines and cosines of tokens tok0 .. tok0 + n - 1 into cs[n][rot/2].
__device__ __forceinline__ void fill_angles(const RopeArgs& a, int64_t tok0, int n, float2* cs) {
  const int half = a.rot >> 1;
  for (int e = threadIdx.x; e < n * half; e += blockDim.x) {
    const int64_t tok = tok0 + e / half;
    const int b = (int)(tok / a.s.T), i = (int)(tok - (int64_t)b * a.s.T);
    const double u = (double)((int64_t)a.pos.q_start[b] + i) * a.turns[e % half];
    float sn, c;
    sincospif(2.f * (float)(u - rint(u)), &sn, &c);
    cs[e] = make_float2(c * a.mscale, sn * a.mscale);
  }
}

// Rotates the 8 dims of lane l of a row; `sign` -1 turns back.  Every lane of the
// warp calls this (the halves layout exchanges values by shuffles).
template <int LPR>
__device__ __forceinline__ void rotate8(const RopeArgs& a, const float2* cs, int l, float sign,
                                        float (&x)[8]) {
  if (a.interleaved) {
    if (8 * l < a.rot) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 t = cs[4 * l + i];
        const float u = x[2 * i], v = x[2 * i + 1], sn = sign * t.y;
        x[2 * i] = u * t.x - v * sn;
        x[2 * i + 1] = v * t.x + u * sn;
      }
    }
    return;
  }
  const int h = a.rot >> 4;                 // lanes of each half
  const int other = l < h ? l + h : (l < 2 * h ? l - h : l);
  const int src = (threadIdx.x & 31 & ~(LPR - 1)) + other;
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(0xffffffffu, x[i], src);
  if (l < 2 * h) {
    const float2* t = cs + 8 * (l < h ? l : l - h);
    const float sg = l < h ? -sign : sign;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] * t[i].x + sg * y[i] * t[i].y;
  }
}

constexpr int kFwdTokens = 4;               // tokens per CTA (at most)

// grid: runs of `tokens` tokens x parts.  Rows of a run in order (token, head): the
// H query heads, then G of K and G of V.
template <int D>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(
    const __grid_constant__ RopeArgs a, int tokens) {
  constexpr int LPR = D / 8, ROWS = kRopeThreads / LPR, U = 4;
  __shared__ float2 cs[kFwdTokens * kHalfRot];
  __shared__ float w[2][D];
  const int64_t n_tok = (int64_t)a.s.B * a.s.T;
  const int64_t tok0 = (int64_t)(blockIdx.x / a.parts) * tokens;
  const int part = blockIdx.x % a.parts;
  const int n = (int)(n_tok - tok0 < tokens ? n_tok - tok0 : tokens);
  const int H = a.s.H, G = a.s.G, heads = H + 2 * G;
  const int nrows = n * heads, per = (nrows + a.parts - 1) / a.parts;
  const int r0 = part * per, r1 = min(nrows, r0 + per);
  const int l = threadIdx.x % LPR, row = threadIdx.x / LPR;
  fill_angles(a, tok0, n, cs);
  for (int d = threadIdx.x; d < 2 * D; d += kRopeThreads) {
    const uint16_t* src = d < D ? a.in.q_weight : a.in.k_weight;
    w[d / D][d % D] = src ? bf16lo(src[d % D]) : 1.f;
  }
  __syncthreads();
  for (int base = r0; base < r1; base += ROWS * U) {
    uint4 raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = base + u * ROWS + row;
      raw[u] = make_uint4(0, 0, 0, 0);
      if (r < r1) {
        const int64_t tok = tok0 + r / heads;
        const int h = r % heads;
        const uint16_t* p = h < H       ? a.in.q + tok * a.in.q_stride + h * D
                            : h < H + G ? a.in.k + tok * a.in.k_stride + (h - H) * D
                                        : a.in.v + tok * a.in.v_stride + (h - H - G) * D;
        raw[u] = ldg16(p + 8 * l);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = base + u * ROWS + row;
      if (base + u * ROWS >= r1) break;     // the same in every lane
      const int rr = min(r, r1 - 1);
      const int tl = rr / heads, h = rr % heads;
      const bool is_q = h < H, is_v = h >= H + G;
      float x[8];
      unpack8(raw[u], x);
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
      ss = row_sum<LPR>(ss);
      if (is_q ? a.in.q_weight != nullptr : a.in.k_weight != nullptr) {
        const float rs = rsqrtf(ss * (1.f / D) + a.eps);
        const float* wr = w[is_q ? 0 : 1] + 8 * l;
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = x[i] * rs * wr[i];
      }
      rotate8<LPR>(a, cs + tl * (a.rot >> 1), l, 1.f, x);
      const uint4 y = is_v ? raw[u] : pack8(x);
      if (r >= r1) continue;
      const int64_t tok = tok0 + tl;
      if (is_q) {
        *reinterpret_cast<uint4*>(a.q_out + (tok * H + h) * D + 8 * l) = y;
      } else {
        const int b = (int)(tok / a.s.T);
        const int64_t t = (int64_t)a.pos.q_start[b] + (tok - (int64_t)b * a.s.T);
        const int64_t pb = cache_block(a.s, b, (int)(t / kBlock), a.status);
        if (pb < 0) continue;               // flagged: nothing written
        const int64_t slot = (pb * kBlock + t % kBlock) * G;
        uint16_t* dst = is_v ? a.v_cache + (slot + h - H - G) * D : a.k_cache + (slot + h - H) * D;
        *reinterpret_cast<uint4*>(dst + 8 * l) = y;
      }
    }
  }
  if (a.in.k_idx && part == a.parts - 1) {
    const int per_tok = a.s.Di / 8;
    for (int e = threadIdx.x; e < n * per_tok; e += kRopeThreads) {
      const int64_t tok = tok0 + e / per_tok;
      const int b = (int)(tok / a.s.T);
      const int64_t t = (int64_t)a.pos.q_start[b] + (tok - (int64_t)b * a.s.T);
      const int64_t pb = cache_block(a.s, b, (int)(t / kBlock), a.status);
      if (pb < 0) continue;
      const int c = e % per_tok;
      *reinterpret_cast<uint4*>(a.kidx_cache + (pb * kBlock + t % kBlock) * a.s.Di + 8 * c) =
          ldg16(a.in.k_idx + tok * a.s.Di + 8 * c);
    }
  }
}

// ---- backward ---------------------------------------------------------------
constexpr int kBwdThreads = 512;
constexpr int kBwdTokens = 4;
constexpr int kBwdMaxCtas = 1024;

// Persistent CTAs over runs of `tokens` tokens.  A thread sums the weights'
// gradients of its 8 dims over all its rows; the CTA's sums go to part_w in a fixed
// order, and the last CTA to finish adds the CTAs' up, again in a fixed order.
template <int D>
__global__ void __launch_bounds__(kBwdThreads, 2) rope_append_bwd_kernel(
    const __grid_constant__ RopeArgs a, int tokens) {
  constexpr int LPR = D / 8, ROWS = kBwdThreads / LPR, U = 2;
  __shared__ float2 cs[kBwdTokens * kHalfRot];
  __shared__ float w[2][D];
  __shared__ float red[kBwdThreads / 32][2][D];
  __shared__ bool last;
  const int64_t n_tok = (int64_t)a.s.B * a.s.T;
  const int H = a.s.H, G = a.s.G, heads = H + 2 * G;
  const int l = threadIdx.x % LPR, row = threadIdx.x / LPR;
  for (int d = threadIdx.x; d < 2 * D; d += kBwdThreads) {
    const uint16_t* src = d < D ? a.in.q_weight : a.in.k_weight;
    w[d / D][d % D] = src ? bf16lo(src[d % D]) : 1.f;
  }
  float dw[2][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) dw[0][i] = dw[1][i] = 0.f;
  for (int64_t tok0 = (int64_t)blockIdx.x * tokens; tok0 < n_tok;
       tok0 += (int64_t)gridDim.x * tokens) {
    const int n = (int)(n_tok - tok0 < tokens ? n_tok - tok0 : tokens);
    const int nrows = n * heads;
    __syncthreads();                         // the last run's angles are used up
    fill_angles(a, tok0, n, cs);
    __syncthreads();
    for (int base = 0; base < nrows; base += ROWS * U) {
      uint4 rx[U], rg[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = base + u * ROWS + row;
        rx[u] = rg[u] = make_uint4(0, 0, 0, 0);
        if (r < nrows) {
          const int64_t tok = tok0 + r / heads;
          const int h = r % heads;
          if (h < H) {
            rg[u] = ldg16(a.g.dq_out + (tok * H + h) * D + 8 * l);
            if (a.in.q_weight) rx[u] = ldg16(a.in.q + tok * a.in.q_stride + h * D + 8 * l);
          } else {
            const int b = (int)(tok / a.s.T);
            const int64_t t = (int64_t)a.pos.q_start[b] + (tok - (int64_t)b * a.s.T);
            const int64_t slot = ((int64_t)b * a.s.max_blocks * kBlock + t) * G;
            if (h < H + G) {
              rg[u] = ldg16(a.g.dk_cache + (slot + h - H) * D + 8 * l);
              if (a.in.k_weight) rx[u] = ldg16(a.in.k + tok * a.in.k_stride + (h - H) * D + 8 * l);
            } else {
              rg[u] = ldg16(a.g.dv_cache + (slot + h - H - G) * D + 8 * l);
            }
          }
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int r = base + u * ROWS + row;
        if (base + u * ROWS >= nrows) break;  // the same in every lane
        const int rr = min(r, nrows - 1);
        const int tl = rr / heads, h = rr % heads;
        const bool is_q = h < H, is_v = h >= H + G;
        float x[8], g[8];
        unpack8(rx[u], x);
        unpack8(rg[u], g);
        rotate8<LPR>(a, cs + tl * (a.rot >> 1), l, -1.f, g);
        float ss = 0.f, sg = 0.f;
        const float* wr = w[is_q ? 0 : 1] + 8 * l;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          ss = fmaf(x[i], x[i], ss);
          sg = fmaf(g[i] * wr[i], x[i], sg);
        }
        ss = row_sum<LPR>(ss);
        sg = row_sum<LPR>(sg);
        if (!is_v && (is_q ? a.in.q_weight != nullptr : a.in.k_weight != nullptr)) {
          const float rs = rsqrtf(ss * (1.f / D) + a.eps);
          const float mean = sg * rs * rs * (1.f / D);   // mean(g x r), times r
          if (r < nrows) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float c = g[i] * x[i] * rs;
              if (is_q) dw[0][i] += c;
              else dw[1][i] += c;
            }
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) g[i] = rs * (g[i] * wr[i] - x[i] * mean);
        }
        if (r >= nrows) continue;
        const int64_t tok = tok0 + tl;
        const uint4 y = is_v ? rg[u] : pack8(g);
        uint16_t* dst = is_q    ? a.g.dq + tok * a.g.dq_stride + h * D
                        : !is_v ? a.g.dk + tok * a.g.dk_stride + (h - H) * D
                                : a.g.dv + tok * a.g.dv_stride + (h - H - G) * D;
        *reinterpret_cast<uint4*>(dst + 8 * l) = y;
      }
    }
  }
  if (!a.in.q_weight && !a.in.k_weight) return;
  // the rows of a warp, then its CTA's warps
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float x = dw[j][i];
#pragma unroll
      for (int o = 16; o >= LPR; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
      if ((threadIdx.x & 31) < LPR) red[threadIdx.x >> 5][j][8 * l + i] = x;
    }
  __syncthreads();
  for (int d = threadIdx.x; d < 2 * D; d += kBwdThreads) {
    float x = 0.f;
    for (int wp = 0; wp < kBwdThreads / 32; ++wp) x += red[wp][d / D][d % D];
    a.part_w[(size_t)blockIdx.x * 2 * D + d] = x;
  }
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) last = atomicAdd(a.counter, 1u) == gridDim.x - 1;
  __syncthreads();
  if (!last) return;
  __threadfence();
  // 512 / 2D threads per column, each every so-many-th CTA, then their sums
  constexpr int S = kBwdThreads / (2 * D);
  const int d = threadIdx.x % (2 * D), k = threadIdx.x / (2 * D);
  float x = 0.f;
#pragma unroll 8
  for (int c = k; c < (int)gridDim.x; c += S) x += __ldcg(a.part_w + (size_t)c * 2 * D + d);
  float* sum = &red[0][0][0];
  __syncthreads();
  sum[threadIdx.x] = x;
  __syncthreads();
  if (k == 0) {
    for (int j = 1; j < S; ++j) x += sum[j * 2 * D + d];
    float* dst = d < D ? a.g.dq_weight : a.g.dk_weight;
    if (d < D ? a.in.q_weight != nullptr : a.in.k_weight != nullptr) dst[d % D] = x;
  }
}

RopeArgs rope_args(const Shape& s, const Positions& pos, const msa_rope& r, const RopeIn& in) {
  RopeArgs a{};
  a.s = s;
  a.pos = pos;
  a.rot = r.rot;
  a.interleaved = r.interleaved;
  a.eps = r.eps;
  a.mscale = r.mscale;
  for (int i = 0; i < r.rot / 2; ++i) a.turns[i] = r.inv_freq[i] / 6.283185307179586476925;
  a.in = in;
  return a;
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
  const int64_t n = (int64_t)s.B * s.T;
  // a few CTAs per SM: runs of tokens where there are enough of them, else a token's
  // rows over several CTAs
  const int64_t want = (int64_t)sm_count() * 4;
  int tokens = n >= want * kFwdTokens ? kFwdTokens : (n >= want * 2 ? 2 : 1);
  const int64_t runs = (n + tokens - 1) / tokens;
  const int rows = tokens * (s.H + 2 * s.G), per_cta = kRopeThreads / (s.D / 8);
  int64_t parts = runs < want ? want / runs : 1;
  if (parts > (rows + per_cta - 1) / per_cta) parts = (rows + per_cta - 1) / per_cta;
  a.parts = (int)parts;
  note_launches(1);
  if (s.D == 128)
    rope_append_kernel<128><<<(unsigned)(runs * parts), kRopeThreads, 0, st>>>(a, tokens);
  else
    rope_append_kernel<64><<<(unsigned)(runs * parts), kRopeThreads, 0, st>>>(a, tokens);
  return cudaGetLastError();
}

size_t rope_bwd_scratch_bytes() { return (size_t)kBwdMaxCtas * 2 * 128 * sizeof(float); }

cudaError_t launch_rope_append_bwd(const Shape& s, const Positions& pos, const msa_rope& r,
                                   const RopeIn& in, const RopeGrads& g, unsigned* counter,
                                   char* base, cudaStream_t st) {
  RopeArgs a = rope_args(s, pos, r, in);
  a.g = g;
  a.counter = counter;
  a.part_w = reinterpret_cast<float*>(base);
  const int64_t n = (int64_t)s.B * s.T;
  int64_t ctas = (int64_t)sm_count() * 2;
  if (ctas > kBwdMaxCtas) ctas = kBwdMaxCtas;
  const int tokens = n >= ctas * kBwdTokens ? kBwdTokens : (n >= ctas * 2 ? 2 : 1);
  const int64_t runs = (n + tokens - 1) / tokens;
  if (ctas > runs) ctas = runs;
  note_launches(1);
  if (s.D == 128)
    rope_append_bwd_kernel<128><<<(unsigned)ctas, kBwdThreads, 0, st>>>(a, tokens);
  else
    rope_append_bwd_kernel<64><<<(unsigned)ctas, kBwdThreads, 0, st>>>(a, tokens);
  return cudaGetLastError();
}

}  // namespace msa

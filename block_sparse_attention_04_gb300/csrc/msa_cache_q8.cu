// Writer of the 8-bit cache.  A cached value is code * 2^e: an e4m3 code and
// one exponent e per (cache block, KV head), for K and for V.  The exponent is
// the smallest with max |x| <= 448 * 2^e over the block's finite values, so
// no value saturates; a power of two keeps every code's mantissa when a later,
// larger token raises the exponent (only codes that become subnormal round
// again) and makes the dequantised value exact in bf16 and f16 arithmetic.
//
// One CTA per (sequence, touched block, KV head, K or V): it reads its new
// rows once into registers, reduces their maximum, joins it with the stored
// exponent if the block was begun by an earlier call, rounds the earlier rows
// to the new exponent when it grew, and writes the codes.  Bound by HBM for
// chunks (2 bytes read and 1 written per value), by launch latency for decode
// steps.  K_idx rows stay bf16; the CTA of head 0's K copies them.
#include "msa_q8.cuh"

namespace msa {
namespace {

constexpr int kAppThreads = 256;

// The smallest e with amax <= 448 * 2^e (448 = 0.875 * 2^9), from amax's bf16
// bits (finite, >= 0); subnormal and zero maxima give kMinExp.
__device__ __forceinline__ int need_exp(uint32_t bits) {
  const int ex = (int)(bits >> 7) - 126;             // amax = m * 2^ex, m in [0.5, 1)
  const int e = (bits & 0x7F) <= 0x60 ? ex - 9 : ex - 8;
  return bits < 0x80 ? kMinExp : clamp_exp(e);
}

template <int D>
__global__ void __launch_bounds__(kAppThreads) cache_append_q8_kernel(
    Shape s, Positions pos, int nbt, const uint16_t* __restrict__ k_new,
    const uint16_t* __restrict__ v_new, const uint4* __restrict__ kidx_new, uint8_t* __restrict__ k,
    uint8_t* __restrict__ v, int8_t* __restrict__ k_exp, int8_t* __restrict__ v_exp,
    uint4* __restrict__ kidx, int* __restrict__ status) {
  constexpr int CPR = D / 8;                          // 16-byte chunks of a new row
  constexpr int RPP = kAppThreads / CPR;              // rows per pass of the CTA
  constexpr int NP = kBlock / RPP;                    // passes over a block
  __shared__ uint32_t warp_max[kAppThreads / 32];
  const int g = blockIdx.x >> 1;
  const bool is_v = blockIdx.x & 1;
  const int b = blockIdx.z;
  const int q0 = pos.q_start[b];
  const int kb = q0 / kBlock + blockIdx.y;
  const int64_t base = (int64_t)kb * kBlock - q0;     // new row i sits at block row i - base
  const int r0 = base < 0 ? (int)-base : 0;           // first new block row
  const int r1 = (int)min((int64_t)kBlock, (int64_t)s.T - base);
  if (r0 >= r1) return;                               // the sequence does not reach this block
  const int64_t pb = cache_block(s, b, kb, status);
  if (pb < 0) return;                                 // flagged: nothing written
  const int tid = threadIdx.x, col = tid % CPR, rr = tid / CPR;
  const uint16_t* src = (is_v ? v_new : k_new) +
                        (((int64_t)b * s.T + base) * s.G + g) * D + col * 8;
  const int64_t rstride = (int64_t)s.G * D;

  uint4 x[NP];
  uint32_t amax = 0;                                  // largest finite |x| as bf16 bits
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int r = p * RPP + rr;
    x[p] = make_uint4(0, 0, 0, 0);
    if (r >= r0 && r < r1) x[p] = ldg_stream(src + r * rstride);
  }
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const uint32_t w[4] = {x[p].x, x[p].y, x[p].z, x[p].w};
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t lo = w[u] & 0x7FFFu, hi = (w[u] >> 16) & 0x7FFFu;
      amax = max(amax, lo < 0x7F80u ? lo : 0u);
      amax = max(amax, hi < 0x7F80u ? hi : 0u);
    }
  }
  amax = __reduce_max_sync(0xffffffffu, amax);
  if ((tid & 31) == 0) warp_max[tid >> 5] = amax;
  int8_t* exps = (is_v ? v_exp : k_exp) + pb * s.G + g;
  const int before = r0 > 0 ? clamp_exp(*exps) : kMinExp;
  __syncthreads();                                    // also: every thread has read *exps
#pragma unroll
  for (int w = 0; w < kAppThreads / 32; ++w) amax = max(amax, warp_max[w]);
  const int e = max(need_exp(amax), before);
  if (tid == 0) *exps = (int8_t)e;

  uint8_t* dst = (is_v ? v : k) + (pb * kBlock * s.G + g) * D + col * 8;
  if (r0 > 0 && e > before) {
    // earlier rows to the larger scale: exact but for codes that turn subnormal
    const float f = e - before > 126 ? 0.f : pow2i(before - e);
    for (int r = rr; r < r0; r += RPP) {
      uint2* c = reinterpret_cast<uint2*>(dst + r * rstride);
      const uint2 w = *c;
      uint2 o;
      const uint32_t in[2] = {w.x, w.y};
      uint32_t res[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint32_t hl, hh;
        e4m3x4_to_f16(in[u], hl, hh);
        const float2 lo = unpack_f16(hl), hi = unpack_f16(hh);
        res[u] = f32x2_to_e4m3x2(lo.x * f, lo.y * f) | f32x2_to_e4m3x2(hi.x * f, hi.y * f) << 16;
      }
      o.x = res[0];
      o.y = res[1];
      *c = o;
    }
  }
  // x * 2^-e, exact in fp32 (or below half the smallest code); infinities as NaN
  const float f = pow2i(-e);
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int r = p * RPP + rr;
    if (r < r0 || r >= r1) continue;
    const uint32_t w[4] = {x[p].x, x[p].y, x[p].z, x[p].w};
    uint32_t c[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      float lo = bf16lo(w[u]), hi = bf16hi(w[u]);
      lo = fabsf(lo) == INFINITY ? NAN : lo * f;
      hi = fabsf(hi) == INFINITY ? NAN : hi * f;
      c[u] = f32x2_to_e4m3x2(lo, hi);
    }
    *reinterpret_cast<uint2*>(dst + r * rstride) = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
  }
  if (g == 0 && !is_v) {
    const int ci = s.Di / 8;                          // 16-byte chunks of a K_idx row
    const uint4* si = kidx_new + ((int64_t)b * s.T + base) * ci;
    uint4* di = kidx + pb * kBlock * ci;
    for (int c = r0 * ci + tid; c < r1 * ci; c += kAppThreads) di[c] = si[c];
  }
}

}  // namespace

cudaError_t launch_cache_append_q8(const Shape& s, const Positions& pos, const uint16_t* k_new,
                                   const uint16_t* v_new, const uint16_t* kidx_new, uint8_t* k,
                                   uint8_t* v, int8_t* k_exp, int8_t* v_exp, uint16_t* kidx,
                                   int* status, cudaStream_t st) {
  int nbt = 0;                                        // most blocks a sequence touches
  for (int b = 0; b < s.B; ++b) {
    const int n = (int)((pos.q_start[b] % kBlock + (int64_t)s.T + kBlock - 1) / kBlock);
    nbt = n > nbt ? n : nbt;
  }
  const dim3 grid(2 * s.G, nbt, s.B);                 // nbt <= max_blocks + 1, within grid limits
  note_launches(1);
  const auto* kn = reinterpret_cast<const uint4*>(kidx_new);
  auto* kc = reinterpret_cast<uint4*>(kidx);
  if (s.D == 128)
    cache_append_q8_kernel<128><<<grid, kAppThreads, 0, st>>>(s, pos, nbt, k_new, v_new, kn, k, v,
                                                              k_exp, v_exp, kc, status);
  else
    cache_append_q8_kernel<64><<<grid, kAppThreads, 0, st>>>(s, pos, nbt, k_new, v_new, kn, k, v,
                                                             k_exp, v_exp, kc, status);
  return cudaGetLastError();
}

}  // namespace msa

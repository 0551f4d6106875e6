// Writer of the 8-bit cache.  A cached value is code * 2^e: an e4m3 code and
// one exponent e per (cache block, KV head), for K and for V.  The exponent is
// the smallest with max |x| <= 448 * 2^e over the block's finite values, so
// no value saturates; a power of two keeps every code's mantissa when a later,
// larger token raises the exponent (only codes that become subnormal round
// again) and makes the dequantised value exact in bf16 and f16 arithmetic.
//
// A task is one (sequence, touched block, KV head, K or V): its threads read
// their new rows once into registers, reduce their maximum, join it with the
// stored exponent if the block was begun by an earlier call, round the earlier
// rows to the new exponent when it grew, and write the codes.  The K_idx rows
// of a (sequence, block), which stay bf16, are one more task.  Chunks give a
// task a CTA, a few tokens per sequence (decode) give it a warp: a CTA per
// task made 64 sequences x 1 token 10.3 us of GPU time, against 2.9 us.
// Bound by HBM for chunks (2 bytes read and 1 written per value; 8192 tokens of
// 8 x 128 move 52 MB, 7.7 us at 6.78 TB/s, and take 12.8 us,
// with 512 or 128 threads per CTA 15.4 and 12.9), by launch
// latency for decode steps.  The first CTA checks every table entry of the call
// and writes the status word, so no clearing launch goes before.
#include "msa_q8.cuh"

namespace msa {
namespace {

constexpr int kAppThreads = 256;
constexpr int kFewTokens = 8;          // most tokens per sequence of the warp-per-task form

// The smallest e with amax <= 448 * 2^e (448 = 0.875 * 2^9), from amax's bf16
// bits (finite, >= 0); subnormal and zero maxima give kMinExp.
__device__ __forceinline__ int need_exp(uint32_t bits) {
  const int ex = (int)(bits >> 7) - 126;             // amax = m * 2^ex, m in [0.5, 1)
  const int e = (bits & 0x7F) <= 0x60 ? ex - 9 : ex - 8;
  return bits < 0x80 ? kMinExp : clamp_exp(e);
}

struct AppendArgs {
  Shape s;
  Positions pos;
  int nbt;                             // most blocks that a sequence's rows touch
  const uint16_t* k_new;
  const uint16_t* v_new;
  const uint4* kidx_new;
  uint8_t* k;
  uint8_t* v;
  int8_t* k_exp;
  int8_t* v_exp;
  uint4* kidx;
  int* status;
};

// W warps per task; NP 16-byte pieces of new rows per thread.
template <int D, int W, int NP>
__global__ void __launch_bounds__(kAppThreads) cache_append_q8_kernel(
    const __grid_constant__ AppendArgs a) {
  constexpr int TPT = 32 * W;                         // threads of a task
  constexpr int CPR = D / 8;                          // 16-byte pieces of a new row
  constexpr int RPP = TPT / CPR;                      // rows per pass
  __shared__ uint32_t warp_max[kAppThreads / 32];
  const Shape& s = a.s;
  if (blockIdx.x == 0) {
    // the status word: every entry that the call's rows go through
    bool bad = false;
    for (int i = threadIdx.x; i < s.B * a.nbt; i += kAppThreads) {
      const int b = i / a.nbt, kb = a.pos.q_start[b] / kBlock + i % a.nbt;
      if (s.bt && (int64_t)kb * kBlock < (int64_t)a.pos.q_start[b] + s.T) {
        const int pb = __ldg(s.bt + (int64_t)b * s.max_blocks + kb);
        bad |= pb < 0 || pb >= s.pool_blocks;
      }
    }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) *a.status = bad ? kDevInvalid : 0;
  }
  const int per = 2 * s.G + 1;                        // tasks of a (sequence, block)
  const int64_t task = (int64_t)blockIdx.x * (kAppThreads / TPT) + threadIdx.x / TPT;
  const int x = (int)(task % per), b = (int)(task / per / a.nbt);
  if (b >= s.B) return;                               // whole tasks only: W == 8 or single warps
  const int q0 = a.pos.q_start[b];
  const int kb = q0 / kBlock + (int)(task / per % a.nbt);
  const int64_t base = (int64_t)kb * kBlock - q0;     // new row i sits at block row i - base
  const int r0 = base < 0 ? (int)-base : 0;           // first new block row
  const int r1 = (int)min((int64_t)kBlock, (int64_t)s.T - base);
  if (r0 >= r1) return;                               // the sequence does not reach this block
  const int tid = threadIdx.x % TPT;
  if (x == 2 * s.G) {
    const int64_t pb = cache_block(s, b, kb, nullptr);
    if (pb < 0) return;                               // flagged above: nothing written
    const int ci = s.Di / 8;                          // 16-byte pieces of a K_idx row
    const uint4* si = a.kidx_new + ((int64_t)b * s.T + base) * ci;
    uint4* di = a.kidx + pb * kBlock * ci;
    for (int c = r0 * ci + tid; c < r1 * ci; c += TPT) di[c] = si[c];
    return;
  }
  const int g = x >> 1;
  const bool is_v = x & 1;
  const int col = tid % CPR, rr = tid / CPR;
  const int64_t rstride = (int64_t)s.G * D;
  const uint16_t* src =
      (is_v ? a.v_new : a.k_new) + (((int64_t)b * s.T + base) * s.G + g) * D + col * 8;
  uint4 v[NP];
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int r = r0 + p * RPP + rr;
    v[p] = r < r1 ? ldg_stream(src + r * rstride) : make_uint4(0, 0, 0, 0);
  }
  const int64_t pb = cache_block(s, b, kb, nullptr);
  int8_t* exps = (is_v ? a.v_exp : a.k_exp) + pb * s.G + g;
  const int before = r0 > 0 && pb >= 0 ? clamp_exp(*exps) : kMinExp;
  uint32_t amax = 0;                                  // largest finite |x| as bf16 bits
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const uint32_t w[4] = {v[p].x, v[p].y, v[p].z, v[p].w};
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t lo = w[u] & 0x7FFFu, hi = (w[u] >> 16) & 0x7FFFu;
      amax = max(amax, lo < 0x7F80u ? lo : 0u);
      amax = max(amax, hi < 0x7F80u ? hi : 0u);
    }
  }
  amax = __reduce_max_sync(0xffffffffu, amax);
  if constexpr (W > 1) {
    static_assert(W == kAppThreads / 32, "a task of several warps is a CTA");
    if ((tid & 31) == 0) warp_max[tid >> 5] = amax;
    __syncthreads();                                  // also: every thread has read *exps
#pragma unroll
    for (int w = 0; w < W; ++w) amax = max(amax, warp_max[w]);
  } else {
    __syncwarp();
  }
  if (pb < 0) return;                                 // flagged above: nothing written
  const int e = max(need_exp(amax), before);
  if (tid == 0) *exps = (int8_t)e;

  uint8_t* dst = (is_v ? a.v : a.k) + (pb * kBlock * s.G + g) * D + col * 8;
  if (r0 > 0 && e > before) {
    // earlier rows to the larger scale: exact but for codes that turn subnormal
    const float f = e - before > 126 ? 0.f : pow2i(before - e);
#pragma unroll 4
    for (int r = rr; r < r0; r += RPP) {
      uint2* c = reinterpret_cast<uint2*>(dst + r * rstride);
      const uint2 w = *c;
      const uint32_t in[2] = {w.x, w.y};
      uint32_t res[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint32_t hl, hh;
        e4m3x4_to_f16(in[u], hl, hh);
        const float2 lo = unpack_f16(hl), hi = unpack_f16(hh);
        res[u] = f32x2_to_e4m3x2(lo.x * f, lo.y * f) | f32x2_to_e4m3x2(hi.x * f, hi.y * f) << 16;
      }
      *c = make_uint2(res[0], res[1]);
    }
  }
  // x * 2^-e, exact in fp32 (or below half the smallest code); infinities as NaN
  const float f = pow2i(-e);
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int r = r0 + p * RPP + rr;
    if (r >= r1) continue;
    const uint32_t w[4] = {v[p].x, v[p].y, v[p].z, v[p].w};
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
}

template <int D>
cudaError_t launch_impl(const AppendArgs& a, cudaStream_t st) {
  const int64_t tasks = (int64_t)a.s.B * a.nbt * (2 * a.s.G + 1);
  note_launches(1);
  if (a.s.T <= kFewTokens) {
    constexpr int per_cta = kAppThreads / 32, rows_per_pass = 32 / (D / 8);
    cache_append_q8_kernel<D, 1, kFewTokens / rows_per_pass>
        <<<(unsigned)((tasks + per_cta - 1) / per_cta), kAppThreads, 0, st>>>(a);
  } else {
    constexpr int rows_per_pass = kAppThreads / (D / 8);
    cache_append_q8_kernel<D, kAppThreads / 32, kBlock / rows_per_pass>
        <<<(unsigned)tasks, kAppThreads, 0, st>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_append_q8(const Shape& s, const Positions& pos, const uint16_t* k_new,
                                   const uint16_t* v_new, const uint16_t* kidx_new, uint8_t* k,
                                   uint8_t* v, int8_t* k_exp, int8_t* v_exp, uint16_t* kidx,
                                   int* status, cudaStream_t st) {
  AppendArgs a;
  a.s = s;
  a.pos = pos;
  a.nbt = 1;
  for (int b = 0; b < s.B; ++b) {
    const int n = (int)((pos.q_start[b] % kBlock + (int64_t)s.T + kBlock - 1) / kBlock);
    a.nbt = n > a.nbt ? n : a.nbt;
  }
  a.k_new = k_new;
  a.v_new = v_new;
  a.kidx_new = reinterpret_cast<const uint4*>(kidx_new);
  a.k = k;
  a.v = v;
  a.k_exp = k_exp;
  a.v_exp = v_exp;
  a.kidx = reinterpret_cast<uint4*>(kidx);
  a.status = status;
  return s.D == 128 ? launch_impl<128>(a, st) : launch_impl<64>(a, st);
}

}  // namespace msa

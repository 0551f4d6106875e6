// The attention's backward pass (msa_sparse_attn_bwd, msa_dense_attn_bwd).
#include "msa_device.cuh"
#include "msa_train.h"

namespace msa {
namespace {

// How often query row r (of [B*T]) attends to block kb of group g.
__device__ __forceinline__ int listed(const Shape& s, const int32_t* sel, int64_t r, int g, int kb) {
  if (!sel) return 1;
  int n = 0;
  for (int j = 0; j < kTopk; ++j) n += sel[(r * s.G + g) * kTopk + j] == kb;
  return n;
}

template <int PER>
__device__ __forceinline__ void load(const uint16_t* p, float (&x)[PER]) {
#pragma unroll
  for (int e = 0; e < PER; ++e) x[e] = bf16lo(p[e]);
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
template <int PER>
__device__ __forceinline__ float dot(const float (&x)[PER], const float (&y)[PER]) {
  float r = 0.f;
#pragma unroll
  for (int e = 0; e < PER; ++e) r = fmaf(x[e], y[e], r);
  return warp_sum(r);
}

// One warp per (query, head): delta = sum P dP / sum P, then dq.
template <int D>
__global__ void __launch_bounds__(256) bwd_dq_kernel(Shape s, const __grid_constant__ Positions pos,
                                                     AttnBwd a, float* delta, int* status) {
  constexpr int PER = D / 32;
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (w >= (int64_t)s.B * s.T * s.H) return;
  const int h = (int)(w % s.H), g = h / (s.H / s.G);
  const int64_t r = w / s.H;
  const int b = (int)(r / s.T);
  const int t = pos.q_start[b] + (int)(r % s.T);
  float q[PER], go[PER], x[PER], acc[PER];
  load(a.q + w * D + lane * PER, q);
  load(a.dout + w * D + lane * PER, go);
#pragma unroll
  for (int e = 0; e < PER; ++e) acc[e] = 0.f;
  const float lse = a.lse[w];
  float sp = 0.f, spd = 0.f, dl = 0.f;
  for (int pass = 0; pass < 2; ++pass) {
    for (int kb = 0; kb <= t / kBlock; ++kb) {
      const int mult = listed(s, a.sel, r, g, kb);
      if (mult == 0) continue;
      const int last = min(t, kb * kBlock + kBlock - 1);
      for (int j = kb * kBlock; j <= last; ++j) {
        const int64_t row = (((int64_t)b * s.max_blocks * kBlock + j) * s.G + g) * D + lane * PER;
        float k[PER];
        load(a.k + row, k);
        load(a.v + row, x);
        const float p = __expf(dot(q, k) * s.scale - lse) * mult, dp = dot(go, x);
        if (pass == 0) {
          sp += p;
          spd = fmaf(p, dp, spd);
        } else {
          const float ds = p * (dp - dl);
#pragma unroll
          for (int e = 0; e < PER; ++e) acc[e] = fmaf(ds, k[e], acc[e]);
        }
      }
    }
    if (pass == 0) dl = sp > 0.f ? spd / sp : 0.f;
  }
  if (lane == 0) delta[w] = dl;
  if (a.sel && h % (s.H / s.G) == 0 && lane < kTopk)
    if (a.sel[(r * s.G + g) * kTopk + lane] > t / kBlock) flag_invalid(status);
#pragma unroll
  for (int e = 0; e < PER; ++e)
    a.dq[w * D + lane * PER + e] = (uint16_t)pack_bf16(acc[e] * s.scale, 0.f);
}

// One warp per (token, group): dk and dv.
template <int D>
__global__ void __launch_bounds__(256) bwd_dkv_kernel(Shape s, const __grid_constant__ Positions pos,
                                                      AttnBwd a, const float* delta) {
  constexpr int PER = D / 32;
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int rows = s.max_blocks * kBlock, hpg = s.H / s.G;
  if (w >= (int64_t)s.B * rows * s.G) return;
  const int g = (int)(w % s.G);
  const int b = (int)(w / s.G / rows), j = (int)(w / s.G % rows);
  if (j >= pos.kv_len[b]) return;
  float k[PER], v[PER], q[PER], go[PER], dk[PER], dv[PER];
  load(a.k + w * D + lane * PER, k);
  load(a.v + w * D + lane * PER, v);
#pragma unroll
  for (int e = 0; e < PER; ++e) dk[e] = dv[e] = 0.f;
  for (int i = max(0, j - pos.q_start[b]); i < s.T; ++i) {
    const int64_t r = (int64_t)b * s.T + i;
    const int mult = listed(s, a.sel, r, g, j / kBlock);
    if (mult == 0) continue;
    for (int h = g * hpg; h < (g + 1) * hpg; ++h) {
      const int64_t at = r * s.H + h;
      load(a.q + at * D + lane * PER, q);
      load(a.dout + at * D + lane * PER, go);
      const float p = __expf(dot(q, k) * s.scale - a.lse[at]) * mult;
      const float ds = p * (dot(go, v) - delta[at]);
#pragma unroll
      for (int e = 0; e < PER; ++e) {
        dv[e] = fmaf(p, go[e], dv[e]);
        dk[e] = fmaf(ds, q[e], dk[e]);
      }
    }
  }
#pragma unroll
  for (int e = 0; e < PER; ++e) {
    a.dk[w * D + lane * PER + e] = (uint16_t)pack_bf16(dk[e] * s.scale, 0.f);
    a.dv[w * D + lane * PER + e] = (uint16_t)pack_bf16(dv[e], 0.f);
  }
}

template <int D>
void launch(const Shape& s, const Positions& pos, const AttnBwd& a, int* status, float* delta,
            cudaStream_t st) {
  const int64_t rows = (int64_t)s.B * s.T * s.H;
  const int64_t toks = (int64_t)s.B * s.max_blocks * kBlock * s.G;
  note_launches(2);
  bwd_dq_kernel<D><<<(unsigned)((rows + 7) / 8), 256, 0, st>>>(s, pos, a, delta, status);
  bwd_dkv_kernel<D><<<(unsigned)((toks + 7) / 8), 256, 0, st>>>(s, pos, a, delta);
}

}  // namespace

size_t attn_bwd_scratch_bytes(const Shape& s, bool) {
  return (size_t)s.B * s.T * s.H * sizeof(float);
}

cudaError_t launch_attn_bwd(const Shape& s, const Positions& pos, const AttnBwd& a, int* status,
                            char* base, cudaStream_t st) {
  if (s.D == 128) launch<128>(s, pos, a, status, reinterpret_cast<float*>(base), st);
  else launch<64>(s, pos, a, status, reinterpret_cast<float*>(base), st);
  return cudaGetLastError();
}

}  // namespace msa

// Device helpers of the 8-bit cache: e4m3 codes with power-of-two scales.
#pragma once
#include "msa_device.cuh"
#include "msa_serve.h"

namespace msa {

// 2^e for e in [-126, 127].
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

// Weights in f16 are held as 2^15 p: p <= 1 then has f16's whole range.
constexpr float kPUp = 15.f, kPDown = 1.f / 32768;

// A stored exponent as the readers use it: any byte is defined.
__device__ __forceinline__ int clamp_exp(int e) { return min(max(e, kMinExp), kMaxExp); }

// Four e4m3 codes (low byte first) -> two pairs of f16, exact.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n"
      " cvt.rn.f16x2.e4m3x2 %1, h;\n}"
      : "=r"(lo), "=r"(hi)
      : "r"(codes));
}

// Four e4m3 codes (low byte first) -> two pairs of bf16, exact; NaN stays NaN.
__device__ __forceinline__ void e4m3x4_to_bf16(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  float a, b, c, d;
  asm("{\n .reg .b16 l, h;\n .reg .b32 x, y;\n mov.b32 {l, h}, %4;\n"
      " cvt.rn.f16x2.e4m3x2 x, l;\n cvt.rn.f16x2.e4m3x2 y, h;\n"
      " mov.b32 {l, h}, x;\n cvt.f32.f16 %0, l;\n cvt.f32.f16 %1, h;\n"
      " mov.b32 {l, h}, y;\n cvt.f32.f16 %2, l;\n cvt.f32.f16 %3, h;\n}"
      : "=f"(a), "=f"(b), "=f"(c), "=f"(d)
      : "r"(codes));
  lo = pack_bf16(a, b);
  hi = pack_bf16(c, d);
}

// Two fp32 -> two e4m3 codes (round to nearest even, saturating; NaN stays
// NaN): `lo` in bits 0-7, `hi` in bits 8-15.
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 unpack_f16(uint32_t h) {
  float2 f;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.f32.f16 %0, l;\n cvt.f32.f16 %1, h;\n}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}

// Instruction descriptor of kind::f16 with f16 A and B (format 0), f32 D.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool a_mn, bool b_mn) {
  return idesc_bf16(M, N, a_mn, b_mn) & ~((1u << 7) | (1u << 10));
}

// D = A(16x16 f16, row) * B(16x8 f16, col) + D, fp32 accumulate.
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The transpose of an 8x8 matrix of 16-bit values spread over the warp (lane
// 4 r + c holds columns 2c, 2c + 1 of row r).
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ uint4 lds128(uint32_t saddr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(saddr));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t saddr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(saddr));
  return v;
}
// Barrier over the cluster's CTAs (all threads), ordering their memory accesses.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
// Two floats at `saddr` in the shared memory of the cluster's CTA `rank`.
__device__ __forceinline__ float2 ld_cluster_f2(uint32_t saddr, int rank) {
  float2 v;
  asm volatile(
      "{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %2, %3;\n"
      " ld.shared::cluster.v2.f32 {%0, %1}, [a];\n}"
      : "=f"(v.x), "=f"(v.y)
      : "r"(saddr), "r"(rank));
  return v;
}
__device__ __forceinline__ int cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return (int)r;
}
// The int at this CTA's shared address `p` in the shared memory of CTA `rank`.
__device__ __forceinline__ int ld_cluster_int(const int* p, int rank) {
  int v;
  asm volatile(
      "{\n .reg .b32 a;\n mapa.shared::cluster.u32 a, %1, %2;\n ld.shared::cluster.b32 %0, [a];\n}"
      : "=r"(v)
      : "r"(smem_u32(p)), "r"(rank)
      : "memory");
  return v;
}
__device__ __forceinline__ void sts128(uint32_t saddr, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(saddr), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}
// Shared-memory writes of this thread before later accesses of the async proxy.
__device__ __forceinline__ void fence_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
// Byte offset of 16-byte chunk c (8 dims of 16 bits) of row r in a tile of
// 64-dim halves of 128 rows, 128-byte swizzle.
__device__ __forceinline__ uint32_t tile_off(int r, int c) {
  return (uint32_t)((c >> 3) * 16384 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}
__device__ __forceinline__ float2 lds_f2(uint32_t saddr) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(saddr));
  return v;
}
__device__ __forceinline__ void sts_f2(uint32_t saddr, float x, float y) {
  asm volatile("st.shared.v2.f32 [%0], {%1,%2};" ::"r"(saddr), "f"(x), "f"(y) : "memory");
}

}  // namespace msa

// The training pass of an attention layer: norm, rotation and cache write in
// one pass, its backward, and the attention's backward (internal interface).
#pragma once
#include "msa_internal.h"

namespace msa {

// Launches a kernel that begins with after_previous() behind another of the same call, so
// that its launch overlaps that one: a call has three to nine kernels, and where they are
// short the gaps between them count (dense, 77 tokens: 41 -> 32 us; sparse, 2 x 101: 90 ->
// 78).  The short ones let the next in when they start; behind the sparse KV-outer kernel,
// the waiting CTAs of a join would cost 100 us of 1410.  A kernel that needs nothing of the
// one before it waits in its end instead (dense, 77 tokens: 30 -> 25.5; 4 x 2048: 642 -> 632):
// it then reads only what the caller gave, and writes what no kernel before it reads.
template <typename... P, typename... A>
cudaError_t launch_behind(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem,
                          cudaStream_t st, const A&... args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  note_launches(1);
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// What msa_rope_append reads: rows of the projections, `stride` elements apart.
struct RopeIn {
  const uint16_t *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  const uint16_t *q_weight, *k_weight, *k_idx;   // or null
};
// *status is written.
cudaError_t launch_rope_append(const Shape& s, const Positions& pos, const msa_rope& r,
                               const RopeIn& in, uint16_t* q_out, uint16_t* k_cache,
                               uint16_t* v_cache, uint16_t* kidx_cache, int* status,
                               cudaStream_t st);

struct RopeGrads {
  const uint16_t *dq_out, *dk_cache, *dv_cache;
  uint16_t *dq, *dk, *dv;
  int64_t dq_stride, dk_stride, dv_stride;
  float *dq_weight, *dk_weight;
};
// base: scratch of rope_bwd_scratch_bytes().  *status is written.
size_t rope_bwd_scratch_bytes();
cudaError_t launch_rope_append_bwd(const Shape& s, const Positions& pos, const msa_rope& r,
                                   const RopeIn& in, const RopeGrads& g, int* status,
                                   char* base, cudaStream_t st);

// The attention's backward pass.  sel null: dense causal.  base: scratch of
// attn_bwd_scratch_bytes(s, sel != null) bytes; *status is written.
struct AttnBwd {
  const uint16_t *q, *k, *v, *out, *dout;
  const float* lse;
  const int32_t* sel;
  uint16_t *dq, *dk, *dv;
};
size_t attn_bwd_scratch_bytes(const Shape& s, bool sparse);
cudaError_t launch_attn_bwd(const Shape& s, const Positions& pos, const AttnBwd& a, int* status,
                            char* base, cudaStream_t st);

}  // namespace msa

// The training pass of an attention layer: norm, rotation and cache write in
// one pass, its backward, and the attention's backward (internal interface).
#pragma once
#include "msa_internal.h"

namespace msa {

// What msa_rope_append reads: rows of the projections, `stride` elements apart.
struct RopeIn {
  const uint16_t *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  const uint16_t *q_weight, *k_weight, *k_idx;   // or null
};
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
// base: scratch of rope_bwd_scratch_bytes(); counters: kRopeBwdCounters zeroed
// words.
constexpr int kRopeBwdCounters = 33;
size_t rope_bwd_scratch_bytes();
cudaError_t launch_rope_append_bwd(const Shape& s, const Positions& pos, const msa_rope& r,
                                   const RopeIn& in, const RopeGrads& g, unsigned* counters,
                                   char* base, cudaStream_t st);

// The attention's backward pass.  sel null: dense causal.  base: scratch of
// attn_bwd_scratch_bytes(s, sel != null) bytes; *status is cleared by the caller.
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

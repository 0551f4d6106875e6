// libmsa C ABI, training pass (include/msa.h): the step in front of the attention
// with its backward, and the attention's backward.  Argument checks and workspace
// layout; nothing is enqueued before every check has passed.
#include <cmath>
#include <cstring>

#include "msa_serve.h"
#include "msa_train.h"

namespace msa {
namespace {

constexpr size_t kAlign = 256;

size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
bool bad(const void* p) { return !p || ((uintptr_t)p & 15u) != 0; }
bool bad_or_null(const void* p) { return ((uintptr_t)p & 15u) != 0; }
int cuda_status(cudaError_t e) { return e == cudaSuccess ? MSA_OK : MSA_ERR_CUDA; }

int check_ws(const void* ws, size_t ws_bytes, size_t need) {
  if (!ws || ((uintptr_t)ws & (kAlign - 1)) != 0) return MSA_ERR_INVALID_ARG;
  return ws_bytes < need ? MSA_ERR_WORKSPACE : MSA_OK;
}

int check_rope(const msa_params* p, const msa_rope* r) {
  if (!r) return MSA_ERR_INVALID_ARG;
  if (r->rot < 0 || r->rot > p->D || (r->interleaved != 0 && r->interleaved != 1))
    return MSA_ERR_INVALID_ARG;
  if (r->rot % 16 != 0) return MSA_ERR_UNSUPPORTED;
  if (!std::isfinite(r->eps) || r->eps < 0.f || !std::isfinite(r->mscale))
    return MSA_ERR_INVALID_ARG;
  for (int i = 0; i < r->rot / 2; ++i)
    if (!std::isfinite(r->inv_freq[i])) return MSA_ERR_INVALID_ARG;
  return MSA_OK;
}

// A token's row of n elements, `stride` elements from the next.
bool bad_stride(int64_t stride, int n) { return stride < n || stride % 8 != 0; }

// First positions only (the cache's rows [q_start, q_start + T) are what counts).
int check_starts(const msa_params* p, const int32_t* q_start, Positions* pos) {
  if (!q_start) return MSA_ERR_INVALID_ARG;
  std::memset(pos, 0, sizeof(*pos));
  const int64_t cap = (int64_t)p->max_blocks * MSA_BLOCK;
  for (int b = 0; b < p->B; ++b) {
    if (q_start[b] < 0 || (int64_t)q_start[b] + p->T > cap) return MSA_ERR_INVALID_ARG;
    pos->q_start[b] = q_start[b];
    pos->kv_len[b] = q_start[b] + p->T;
  }
  return MSA_OK;
}

size_t bwd_bytes(const msa_params* p, bool sparse) {
  return kAlign + align_up(attn_bwd_scratch_bytes(shape_of(p), sparse));
}

int attn_bwd(const msa_params* p, const AttnBwd& a, bool sparse, const int32_t* q_start,
             const int32_t* kv_len, void* ws, size_t ws_bytes, cudaStream_t stream) {
  int rc = validate_params(p);
  if (rc) return rc;
  Positions pos;
  if ((rc = validate_positions(p, q_start, kv_len, &pos))) return rc;
  if (bad(a.q) || bad(a.k) || bad(a.v) || bad(a.out) || bad(a.lse) || bad(a.dout) || bad(a.dq) ||
      bad(a.dk) || bad(a.dv) || (sparse && bad(a.sel)))
    return MSA_ERR_INVALID_ARG;
  if ((rc = check_ws(ws, ws_bytes, bwd_bytes(p, sparse)))) return rc;
  if (p->T == 0) return MSA_OK;
  return cuda_status(launch_attn_bwd(shape_of(p), pos, a, static_cast<int*>(ws),
                                     static_cast<char*>(ws) + kAlign, stream));
}

}  // namespace
}  // namespace msa

using namespace msa;

extern "C" {

int msa_rope_append(const msa_params* p, const msa_rope* r, const int32_t* block_table,
                    int num_pool_blocks, const uint16_t* q, const uint16_t* k, const uint16_t* v,
                    int64_t q_stride, int64_t k_stride, int64_t v_stride,
                    const uint16_t* q_weight, const uint16_t* k_weight, const uint16_t* k_idx_new,
                    const int32_t* q_start, uint16_t* q_out, uint16_t* k_cache, uint16_t* v_cache,
                    uint16_t* k_idx_cache, void* ws, size_t ws_bytes, cudaStream_t stream) {
  int rc = validate_params(p);
  if (rc) return rc;
  if ((rc = check_rope(p, r))) return rc;
  if (block_table && (rc = validate_pool(block_table, num_pool_blocks))) return rc;
  Positions pos;
  if ((rc = check_starts(p, q_start, &pos))) return rc;
  if (bad(q) || bad(k) || bad(v) || bad(q_out) || bad(k_cache) || bad(v_cache) ||
      bad_or_null(q_weight) || bad_or_null(k_weight) || bad_or_null(k_idx_new) ||
      (k_idx_new && bad(k_idx_cache)))
    return MSA_ERR_INVALID_ARG;
  if (bad_stride(q_stride, p->H * p->D) || bad_stride(k_stride, p->G * p->D) ||
      bad_stride(v_stride, p->G * p->D))
    return MSA_ERR_INVALID_ARG;
  if ((rc = check_ws(ws, ws_bytes, kAlign))) return rc;
  if (p->T == 0) return MSA_OK;
  const RopeIn in{q, k, v, q_stride, k_stride, v_stride, q_weight, k_weight, k_idx_new};
  return cuda_status(launch_rope_append(shape_of(p, block_table, num_pool_blocks), pos, *r, in,
                                        q_out, k_cache, v_cache, k_idx_cache, static_cast<int*>(ws), stream));
}

size_t msa_rope_append_bwd_workspace_bytes(const msa_params* p) {
  if (validate_params(p) != MSA_OK) return 0;
  return kAlign + align_up(rope_bwd_scratch_bytes());
}

int msa_rope_append_bwd(const msa_params* p, const msa_rope* r, const uint16_t* q,
                        const uint16_t* k, int64_t q_stride, int64_t k_stride,
                        const uint16_t* q_weight, const uint16_t* k_weight,
                        const int32_t* q_start, const uint16_t* dq_out, const uint16_t* dk_cache,
                        const uint16_t* dv_cache, uint16_t* dq, uint16_t* dk, uint16_t* dv,
                        int64_t dq_stride, int64_t dk_stride, int64_t dv_stride, float* dq_weight,
                        float* dk_weight, void* ws, size_t ws_bytes, cudaStream_t stream) {
  int rc = validate_params(p);
  if (rc) return rc;
  if ((rc = check_rope(p, r))) return rc;
  Positions pos;
  if ((rc = check_starts(p, q_start, &pos))) return rc;
  if (bad(dq_out) || bad(dk_cache) || bad(dv_cache) || bad(dq) || bad(dk) || bad(dv) ||
      bad_or_null(q_weight) || bad_or_null(k_weight) || (q_weight && (bad(q) || bad(dq_weight))) ||
      (k_weight && (bad(k) || bad(dk_weight))))
    return MSA_ERR_INVALID_ARG;
  const int nq = p->H * p->D, nk = p->G * p->D;
  if ((q_weight && bad_stride(q_stride, nq)) || (k_weight && bad_stride(k_stride, nk)) ||
      bad_stride(dq_stride, nq) || bad_stride(dk_stride, nk) || bad_stride(dv_stride, nk))
    return MSA_ERR_INVALID_ARG;
  if ((rc = check_ws(ws, ws_bytes, msa_rope_append_bwd_workspace_bytes(p)))) return rc;
  if (p->T == 0) return MSA_OK;
  const RopeIn in{q, k, nullptr, q_stride, k_stride, 0, q_weight, k_weight, nullptr};
  const RopeGrads g{dq_out, dk_cache, dv_cache, dq, dk, dv, dq_stride, dk_stride, dv_stride,
                    dq_weight, dk_weight};
  return cuda_status(launch_rope_append_bwd(shape_of(p), pos, *r, in, g,
                                            static_cast<int*>(ws),
                                            static_cast<char*>(ws) + kAlign, stream));
}

size_t msa_sparse_bwd_workspace_bytes(const msa_params* p) {
  return validate_params(p) == MSA_OK ? bwd_bytes(p, true) : 0;
}

int msa_sparse_attn_bwd(const msa_params* p, const uint16_t* q, const uint16_t* k_cache,
                        const uint16_t* v_cache, const int32_t* sel, const uint16_t* out,
                        const float* lse, const uint16_t* dout, const int32_t* q_start,
                        const int32_t* kv_len, uint16_t* dq, uint16_t* dk, uint16_t* dv, void* ws,
                        size_t ws_bytes, cudaStream_t stream) {
  const AttnBwd a{q, k_cache, v_cache, out, dout, lse, sel, dq, dk, dv};
  return attn_bwd(p, a, true, q_start, kv_len, ws, ws_bytes, stream);
}

size_t msa_dense_bwd_workspace_bytes(const msa_params* p) {
  return validate_params(p) == MSA_OK ? bwd_bytes(p, false) : 0;
}

int msa_dense_attn_bwd(const msa_params* p, const uint16_t* q, const uint16_t* k_cache,
                       const uint16_t* v_cache, const uint16_t* out, const float* lse,
                       const uint16_t* dout, const int32_t* q_start, const int32_t* kv_len,
                       uint16_t* dq, uint16_t* dk, uint16_t* dv, void* ws, size_t ws_bytes,
                       cudaStream_t stream) {
  const AttnBwd a{q, k_cache, v_cache, out, dout, lse, nullptr, dq, dk, dv};
  return attn_bwd(p, a, false, q_start, kv_len, ws, ws_bytes, stream);
}

}  // extern "C"

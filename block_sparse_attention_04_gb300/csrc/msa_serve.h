// Serving operators beside the MSA forward pass: the 8-bit cache, sliding-
// window attention and the page operations (internal interface).
#pragma once
#include "msa_internal.h"

namespace msa {

constexpr int kMinExp = MSA_Q8_MIN_EXP, kMaxExp = MSA_Q8_MAX_EXP;

// A cache as the attention kernels read it: bf16 (kv8 false, exps null) or
// e4m3 codes with one power-of-two exponent per (cache block, KV head).
struct CacheView {
  const void* k;
  const void* v;
  const int8_t* k_exp;   // [blocks][G]
  const int8_t* v_exp;
  bool kv8;
};

// What a query sees: the blocks of a caller's selection (sel not null), or
// the tokens j <= t with j > t - window or j < sinks.
struct Visible {
  const int32_t* sel;    // [B][T][G][16] or null
  int window, sinks;
};

// Scratch of the streaming attention: two partials and one error word per CTA.
struct StreamPlan {
  size_t part_o_off, part_ml_off, errs_off, total;
};
StreamPlan stream_plan(const Shape& s);
int stream_pass_rows(const Shape& s);

// Attention of every query of the call by the streaming kernel (any shape).
// base: scratch of stream_plan(s).total bytes; *status receives the call's
// status word (no clearing needed beforehand), joined with what it holds when
// `join_status` is set.
cudaError_t launch_stream_attn(const Shape& s, const Positions& pos, const CacheView& c,
                               const Visible& vis, const uint16_t* q, uint16_t* out, int* status,
                               bool join_status, char* base, cudaStream_t st);

// Step 4 of an 8-bit call on tensor cores (prefill shapes).  base: scratch of
// tc_attn_q8_workspace_bytes(s) bytes; *status is cleared by the caller.
size_t tc_attn_q8_workspace_bytes(const Shape& s);
cudaError_t launch_attn_tc_q8(const Shape& s, const Positions& pos, const uint16_t* q,
                              const CacheView& c, const int32_t* sel, uint16_t* out, int* status,
                              char* base, cudaStream_t st);

// Sliding-window attention of every query of the call on tensor cores
// (prefill shapes).  status: the status word and the word after it; base:
// scratch of window_tc_scratch_bytes(s) bytes.
size_t window_tc_scratch_bytes(const Shape& s);
int window_splits(const Shape& s, const Positions& pos, int window, int sinks);
int window_list_len(const Shape& s, const Positions& pos, int window, int sinks);
cudaError_t launch_window_tc(const Shape& s, const Positions& pos, const CacheView& c, int window,
                             int sinks, const uint16_t* q, uint16_t* out, int* status, char* base,
                             cudaStream_t st);

// Appends tokens to an 8-bit cache (layouts of msa_cache_append_q8) and writes
// the status word.
cudaError_t launch_cache_append_q8(const Shape& s, const Positions& pos, const uint16_t* k_new,
                                   const uint16_t* v_new, const uint16_t* kidx_new, uint8_t* k,
                                   uint8_t* v, int8_t* k_exp, int8_t* v_exp, uint16_t* kidx,
                                   int* status, cudaStream_t st);

// Steps 1-3 into sel on the workspace of msa_workspace_bytes(p) (shared with
// msa_index_topk); positions and pointers are validated by the caller.
int run_index_in(const msa_params* p, const Shape& s, const Positions& pos, const uint16_t* q_idx,
                 const uint16_t* k_idx, int32_t* sel, void* ws, cudaStream_t st);
int validate_pool(const int32_t* block_table, int num_pool_blocks);

}  // namespace msa

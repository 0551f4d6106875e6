// libmsa C ABI, serving operators (include/msa.h): 8-bit caches, sliding-window
// attention and page operations.  Argument checks, workspace layout and the
// choice of kernels; nothing is enqueued before every check has passed.
#include <cmath>
#include <cstring>

#include "msa_pages.h"
#include "msa_serve.h"

namespace msa {
namespace {

constexpr size_t kAlign = 256;

size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
bool bad(const void* p) { return !p || ((uintptr_t)p & 15u) != 0; }
int cuda_status(cudaError_t e) { return e == cudaSuccess ? MSA_OK : MSA_ERR_CUDA; }

int check_ws(const void* ws, size_t ws_bytes, size_t need) {
  if (!ws || ((uintptr_t)ws & (kAlign - 1)) != 0) return MSA_ERR_INVALID_ARG;
  return ws_bytes < need ? MSA_ERR_WORKSPACE : MSA_OK;
}

// Parameters, the optional pool and the positions of an attention call.
int check_call(const msa_params* p, const int32_t* block_table, int num_pool_blocks,
               const int32_t* q_start, const int32_t* kv_len, Positions* pos) {
  int rc = validate_params(p);
  if (rc) return rc;
  if (block_table && (rc = validate_pool(block_table, num_pool_blocks))) return rc;
  return validate_positions(p, q_start, kv_len, pos);
}

// Workspace of the attention calls: the status word, then their scratch.
size_t stream_scratch(const msa_params* p) { return align_up(stream_plan(shape_of(p)).total); }
size_t sparse_scratch(const msa_params* p) {
  const size_t tc = tc_attn_q8_workspace_bytes(shape_of(p)), stream = stream_scratch(p);
  return align_up(tc > stream ? tc : stream);
}

// ---- which kernels run an attention call (MSA_KERNELS_AUTO) ---------------
// The time of both families in microseconds, from what a step of each took on
// GB300 (graph replays, 152 SMs, contexts of 16K, 1 and 16 sequences of 1 to 256
// queries, both head layouts; the estimates are within about 25 % of the
// measurements behind them).
constexpr double kSms = 152;

// Streaming: a time per (unit, block) step and CTA and 1.6 us per unit (the
// join of its warps), or the blocks' bytes where they do not stay in L2 between
// the queries that read them.
double stream_us(double units, double steps, double step_bytes, double distinct_bytes,
                 double step = 0.8) {
  const double compute = steps / kSms * step + units / kSms * 1.6;
  const double memory = distinct_bytes > 64e6 ? steps * step_bytes / 6.6e6 : 0.0;
  return 6.0 + (compute > memory ? compute : memory);
}

// Window on tensor cores: a step is one block for two tiles.  16 x 8 queries of
// a 512-token window, 48/8 heads: 44 us streaming, 22 us here; one decode token
// of 16 sequences, window 8000: 84 us streaming, 116 us here.
bool window_on_tc(const msa_params* p, const Shape& s, const Positions& pos, const Visible& vis,
                  bool kv8) {
  if (p->kernels != MSA_KERNELS_AUTO) return p->kernels == MSA_KERNELS_TENSORCORE;
  double blocks = 0;
  for (int b = 0; b < s.B; ++b) {
    const int t = pos.q_start[b] + s.T - 1;
    const int lo = (t - vis.window + 1 > 0 ? t - vis.window + 1 : 0) / kBlock;
    const int sb = (vis.sinks + kBlock - 1) / kBlock;
    blocks += (sb < lo ? sb : lo) + t / kBlock - lo + 1;
  }
  const double block_bytes = 2.0 * kBlock * s.D * (kv8 ? 1 : 2);
  const double steps = blocks * s.G;
  const double stream = stream_us((double)s.B * s.T * s.G, steps * s.T, block_bytes, steps * block_bytes);
  const int nq = 128 / (s.H / s.G);
  const double items = (double)((s.T + 2 * nq - 1) / (2 * nq)) * s.B * s.G;
  const int splits = window_splits(s, pos, vis.window, vis.sinks);
  const double longest = window_list_len(s, pos, vis.window, vis.sinks);
  const double step = s.D == 128 ? (kv8 ? 2.2 : 1.65) : (kv8 ? 1.8 : 1.55);
  const double tc = 10.0 + std::ceil(items * splits / kSms) * std::ceil(longest / splits) * step +
                    (splits > 1 ? 6.0 : 0.0);
  return tc < stream;
}

// Selected blocks of an 8-bit cache: the streaming kernel reads 16 blocks per
// (query, group); the KV-outer kernels read a block once per list and work in
// tiles of 128 query-head rows, of which a list has at least one: 96 queries of
// one sequence at 16K, 48/8 heads, 77 us streaming, 47 us KV-outer; 16 x 16
// queries 193 and 259 us.
bool sparse_on_tc(const msa_params* p, const Shape& s, const Positions& pos) {
  if (p->kernels != MSA_KERNELS_AUTO) return p->kernels == MSA_KERNELS_TENSORCORE;
  const double entries = (double)s.B * s.T * s.G * MSA_TOPK;
  double lists = 0;
  for (int b = 0; b < s.B; ++b) lists += (pos.q_start[b] + s.T - 1) / kBlock + 1;
  lists *= s.G;
  const double block_bytes = 2.0 * kBlock * s.D;
  const int rows = s.H / s.G <= 8 ? 8 : 16;
  const double stream = stream_us(entries / MSA_TOPK, entries, block_bytes, lists * block_bytes,
                                  s.D == 128 && rows > 8 ? 1.25 : 0.8);
  // lists that at least one of `entries` random choices meets, and full tiles
  const double tiles = lists * (1.0 - std::exp(-entries / lists)) + entries / (128 / rows);
  const double tc = 27.0 + tiles / kSms * (s.D == 128 ? 2.1 : 1.45);
  return tc < stream;
}

// ... of an 8-bit call: msa_forward's index scratch follows msa_workspace_bytes'
// own layout in the same bytes (the steps run in order), then the selection.
size_t q8_sel_off(const msa_params* p) {
  const size_t idx = msa_workspace_bytes(p), att = kAlign + sparse_scratch(p);
  return align_up(idx > att ? idx : att);
}

int run_attn_q8(const msa_params* p, const Shape& s, const Positions& pos, const uint16_t* q,
                const CacheView& c, const int32_t* sel, uint16_t* out, bool join_status, void* ws,
                cudaStream_t st) {
  char* base = static_cast<char*>(ws);
  if (sparse_on_tc(p, s, pos)) {
    if (!join_status && cudaMemsetAsync(ws, 0, sizeof(int), st) != cudaSuccess) return MSA_ERR_CUDA;
    return cuda_status(launch_attn_tc_q8(s, pos, q, c, sel, out, reinterpret_cast<int*>(base),
                                         base + kAlign, st));
  }
  return cuda_status(launch_stream_attn(s, pos, c, Visible{sel, 0, 0}, q, out,
                                        reinterpret_cast<int*>(base), join_status, base + kAlign, st));
}

int run_window(const msa_params* p, const int32_t* block_table, int num_pool_blocks, int window,
               int sinks, const uint16_t* q, const CacheView& c, const int32_t* q_start,
               const int32_t* kv_len, uint16_t* out, void* ws, size_t ws_bytes, cudaStream_t st) {
  Positions pos;
  int rc = check_call(p, block_table, num_pool_blocks, q_start, kv_len, &pos);
  if (rc) return rc;
  if (window < 1 || sinks < 0) return MSA_ERR_INVALID_ARG;
  if (bad(q) || bad(c.k) || bad(c.v) || bad(out)) return MSA_ERR_INVALID_ARG;
  if (c.kv8 && (bad(c.k_exp) || bad(c.v_exp))) return MSA_ERR_INVALID_ARG;
  if ((rc = check_ws(ws, ws_bytes, msa_window_workspace_bytes(p)))) return rc;
  if (p->T == 0) return MSA_OK;
  // no context is longer than the caches: sums of positions stay in 32 bits
  const int cap = p->max_blocks * MSA_BLOCK;
  const Visible vis{nullptr, window < cap ? window : cap, sinks < cap ? sinks : cap};
  const Shape s = shape_of(p, block_table, num_pool_blocks);
  char* base = static_cast<char*>(ws);
  if (window_on_tc(p, s, pos, vis, c.kv8))
    return cuda_status(launch_window_tc(s, pos, c, vis.window, vis.sinks, q, out,
                                        reinterpret_cast<int*>(base), base + kAlign, st));
  return cuda_status(launch_stream_attn(s, pos, c, vis, q, out, reinterpret_cast<int*>(base),
                                        false, base + kAlign, st));
}

// ---- page operations -------------------------------------------------------
int check_pools(const msa_pool* pools, int npools, PoolSet* ps) {
  if (npools < 0 || npools > MSA_MAX_POOLS || (npools > 0 && !pools)) return MSA_ERR_INVALID_ARG;
  ps->n = npools;
  for (int i = 0; i < npools; ++i) {
    const msa_pool& p = pools[i];
    if (!p.base || p.page_bytes == 0) return MSA_ERR_INVALID_ARG;
    if (p.per_token && p.page_bytes % MSA_BLOCK != 0) return MSA_ERR_INVALID_ARG;
    if (p.page_bytes > ((size_t)1 << 30)) return MSA_ERR_UNSUPPORTED;
    ps->pool[i] = p;
  }
  return MSA_OK;
}

int check_table(int pages, const int32_t* table, int rows, int max_blocks, const int32_t* refs) {
  if (pages < 1 || rows < 1 || max_blocks < 1 || !table || !refs) return MSA_ERR_INVALID_ARG;
  if (((uintptr_t)table & 3u) || ((uintptr_t)refs & 3u)) return MSA_ERR_INVALID_ARG;
  // token counts and page-list words stay in 32 bits
  if ((int64_t)max_blocks * MSA_BLOCK >= ((int64_t)1 << 31) ||
      (int64_t)pages * MSA_BLOCK + MSA_BLOCK >= ((int64_t)1 << 31))
    return MSA_ERR_UNSUPPORTED;
  return MSA_OK;
}

int check_list_len(int n) {
  if (n < 0) return MSA_ERR_INVALID_ARG;
  return n > kMaxBatch ? MSA_ERR_UNSUPPORTED : MSA_OK;
}

// Rows and block ranges of msa_pages_free (rows may repeat) and _alloc.
int check_ranges(const int32_t* row, const int32_t* first, const int32_t* last, int n, int rows,
                 int max_blocks, bool distinct, RowList* rl) {
  const int rc = check_list_len(n);
  if (rc) return rc;
  if (n > 0 && (!row || !first || !last)) return MSA_ERR_INVALID_ARG;
  rl->n = n;
  for (int j = 0; j < n; ++j) {
    if (row[j] < 0 || row[j] >= rows || first[j] < 0 || last[j] < first[j] || last[j] > max_blocks)
      return MSA_ERR_INVALID_ARG;
    for (int k = 0; distinct && k < j; ++k)
      if (row[k] == row[j]) return MSA_ERR_INVALID_ARG;
    rl->a[j] = row[j];
    rl->b[j] = first[j];
    rl->c[j] = last[j];
  }
  return MSA_OK;
}

}  // namespace
}  // namespace msa

using namespace msa;

extern "C" {

int msa_cache_append_q8(const msa_params* p, const int32_t* block_table, int num_pool_blocks,
                        const uint16_t* k_new, const uint16_t* v_new, const uint16_t* k_idx_new,
                        const int32_t* q_start, uint8_t* k_cache, uint8_t* v_cache, int8_t* k_exp,
                        int8_t* v_exp, uint16_t* k_idx_cache, void* ws, size_t ws_bytes,
                        cudaStream_t stream) {
  int rc = validate_params(p);
  if (rc) return rc;
  if (block_table && (rc = validate_pool(block_table, num_pool_blocks))) return rc;
  if (!q_start) return MSA_ERR_INVALID_ARG;
  Positions pos;
  std::memset(&pos, 0, sizeof(pos));
  const int64_t cap = (int64_t)p->max_blocks * MSA_BLOCK;
  for (int b = 0; b < p->B; ++b) {
    if (q_start[b] < 0 || (int64_t)q_start[b] + p->T > cap) return MSA_ERR_INVALID_ARG;
    pos.q_start[b] = q_start[b];
    pos.kv_len[b] = q_start[b] + p->T;
  }
  if (bad(k_new) || bad(v_new) || bad(k_idx_new) || bad(k_cache) || bad(v_cache) || bad(k_exp) ||
      bad(v_exp) || bad(k_idx_cache))
    return MSA_ERR_INVALID_ARG;
  if ((rc = check_ws(ws, ws_bytes, kAlign))) return rc;
  if (p->T == 0) return MSA_OK;
  int* status = static_cast<int*>(ws);
  return cuda_status(launch_cache_append_q8(shape_of(p, block_table, num_pool_blocks), pos, k_new,
                                            v_new, k_idx_new, k_cache, v_cache, k_exp, v_exp,
                                            k_idx_cache, status, stream));
}

size_t msa_q8_workspace_bytes(const msa_params* p) {
  if (validate_params(p) != MSA_OK) return 0;
  return q8_sel_off(p) + align_up((size_t)p->B * p->T * p->G * MSA_TOPK * sizeof(int32_t));
}

int msa_sparse_attn_q8(const msa_params* p, const int32_t* block_table, int num_pool_blocks,
                       const uint16_t* q, const uint8_t* k_cache, const uint8_t* v_cache,
                       const int8_t* k_exp, const int8_t* v_exp, const int32_t* sel,
                       const int32_t* q_start, const int32_t* kv_len, uint16_t* out, void* ws,
                       size_t ws_bytes, cudaStream_t stream) {
  Positions pos;
  int rc = check_call(p, block_table, num_pool_blocks, q_start, kv_len, &pos);
  if (rc) return rc;
  if (bad(q) || bad(k_cache) || bad(v_cache) || bad(k_exp) || bad(v_exp) || bad(sel) || bad(out))
    return MSA_ERR_INVALID_ARG;
  if ((rc = check_ws(ws, ws_bytes, msa_q8_workspace_bytes(p)))) return rc;
  if (p->T == 0) return MSA_OK;
  return run_attn_q8(p, shape_of(p, block_table, num_pool_blocks), pos, q,
                     CacheView{k_cache, v_cache, k_exp, v_exp, true}, sel, out, false, ws, stream);
}

int msa_forward_q8(const msa_params* p, const int32_t* block_table, int num_pool_blocks,
                   const uint16_t* q_idx, const uint16_t* k_idx, const uint16_t* q,
                   const uint8_t* k_cache, const uint8_t* v_cache, const int8_t* k_exp,
                   const int8_t* v_exp, const int32_t* q_start, const int32_t* kv_len,
                   int32_t* sel_out, uint16_t* out, void* ws, size_t ws_bytes,
                   cudaStream_t stream) {
  Positions pos;
  int rc = check_call(p, block_table, num_pool_blocks, q_start, kv_len, &pos);
  if (rc) return rc;
  if (bad(q_idx) || bad(k_idx) || bad(q) || bad(k_cache) || bad(v_cache) || bad(k_exp) ||
      bad(v_exp) || bad(out) || (sel_out && bad(sel_out)))
    return MSA_ERR_INVALID_ARG;
  if ((rc = check_ws(ws, ws_bytes, msa_q8_workspace_bytes(p)))) return rc;
  if (p->T == 0) return MSA_OK;
  const Shape s = shape_of(p, block_table, num_pool_blocks);
  int32_t* sel =
      sel_out ? sel_out : reinterpret_cast<int32_t*>(static_cast<char*>(ws) + q8_sel_off(p));
  if ((rc = run_index_in(p, s, pos, q_idx, k_idx, sel, ws, stream))) return rc;
  return run_attn_q8(p, s, pos, q, CacheView{k_cache, v_cache, k_exp, v_exp, true}, sel, out, true,
                     ws, stream);
}

size_t msa_window_workspace_bytes(const msa_params* p) {
  if (validate_params(p) != MSA_OK) return 0;
  const size_t tc = window_tc_scratch_bytes(shape_of(p)), stream = stream_scratch(p);
  return kAlign + align_up(tc > stream ? tc : stream);
}

int msa_window_attn(const msa_params* p, const int32_t* block_table, int num_pool_blocks,
                    int window, int sinks, const uint16_t* q, const uint16_t* k_cache,
                    const uint16_t* v_cache, const int32_t* q_start, const int32_t* kv_len,
                    uint16_t* out, void* ws, size_t ws_bytes, cudaStream_t stream) {
  return run_window(p, block_table, num_pool_blocks, window, sinks, q,
                    CacheView{k_cache, v_cache, nullptr, nullptr, false}, q_start, kv_len, out, ws,
                    ws_bytes, stream);
}

int msa_window_attn_q8(const msa_params* p, const int32_t* block_table, int num_pool_blocks,
                       int window, int sinks, const uint16_t* q, const uint8_t* k_cache,
                       const uint8_t* v_cache, const int8_t* k_exp, const int8_t* v_exp,
                       const int32_t* q_start, const int32_t* kv_len, uint16_t* out, void* ws,
                       size_t ws_bytes, cudaStream_t stream) {
  return run_window(p, block_table, num_pool_blocks, window, sinks, q,
                    CacheView{k_cache, v_cache, k_exp, v_exp, true}, q_start, kv_len, out, ws,
                    ws_bytes, stream);
}

size_t msa_pages_workspace_bytes(int num_pool_blocks) {
  return num_pool_blocks < 1 ? 0 : pages_workspace_bytes(num_pool_blocks);
}

int msa_pages_copy(const msa_pool* pools, int npools, int num_pool_blocks, const int32_t* src,
                   const int32_t* dst, int n, void* ws, size_t ws_bytes, cudaStream_t stream) {
  PoolSet ps;
  int rc = check_pools(pools, npools, &ps);
  if (rc) return rc;
  if (n < 0 || num_pool_blocks < 1 || (n > 0 && (!src || !dst))) return MSA_ERR_INVALID_ARG;
  if (((uintptr_t)src & 3u) || ((uintptr_t)dst & 3u)) return MSA_ERR_INVALID_ARG;
  if ((rc = check_ws(ws, ws_bytes, msa_pages_workspace_bytes(num_pool_blocks)))) return rc;
  if (n == 0 || npools == 0) return MSA_OK;
  return cuda_status(
      launch_pages_copy(ps, num_pool_blocks, src, dst, n, static_cast<char*>(ws), stream));
}

int msa_pages_fork(const msa_pool* pools, int npools, int num_pool_blocks, int32_t* block_table,
                   int rows, int max_blocks, int32_t* refs, const int32_t* src_rows,
                   const int32_t* dst_rows, const int32_t* len, int n, void* ws, size_t ws_bytes,
                   cudaStream_t stream) {
  PoolSet ps;
  RowList rl;
  int rc = check_pools(pools, npools, &ps);
  if (rc || (rc = check_table(num_pool_blocks, block_table, rows, max_blocks, refs))) return rc;
  if ((rc = check_list_len(n))) return rc;
  if (n > 0 && (!src_rows || !dst_rows || !len)) return MSA_ERR_INVALID_ARG;
  rl.n = n;
  for (int j = 0; j < n; ++j) {
    if (src_rows[j] < 0 || src_rows[j] >= rows || dst_rows[j] < 0 || dst_rows[j] >= rows)
      return MSA_ERR_INVALID_ARG;
    if (len[j] < 0 || len[j] > max_blocks * MSA_BLOCK) return MSA_ERR_INVALID_ARG;
    for (int k = 0; k < n; ++k)
      if (dst_rows[j] == src_rows[k] || (k < j && dst_rows[j] == dst_rows[k]))
        return MSA_ERR_INVALID_ARG;
    rl.a[j] = src_rows[j];
    rl.b[j] = dst_rows[j];
    rl.c[j] = len[j];
  }
  if ((rc = check_ws(ws, ws_bytes, msa_pages_workspace_bytes(num_pool_blocks)))) return rc;
  if (n == 0) return MSA_OK;
  return cuda_status(launch_pages_fork(
      ps, PageTable{block_table, rows, max_blocks, refs, num_pool_blocks}, rl,
      static_cast<char*>(ws), stream));
}

int msa_pages_free(int num_pool_blocks, int32_t* block_table, int rows, int max_blocks,
                   int32_t* refs, const int32_t* row, const int32_t* first, const int32_t* last,
                   int n, void* ws, size_t ws_bytes, cudaStream_t stream) {
  RowList rl;
  int rc = check_table(num_pool_blocks, block_table, rows, max_blocks, refs);
  if (rc || (rc = check_ranges(row, first, last, n, rows, max_blocks, false, &rl))) return rc;
  if ((rc = check_ws(ws, ws_bytes, msa_pages_workspace_bytes(num_pool_blocks)))) return rc;
  if (n == 0) return MSA_OK;
  return cuda_status(
      launch_pages_free(PageTable{block_table, rows, max_blocks, refs, num_pool_blocks}, rl,
                        static_cast<char*>(ws), stream));
}

int msa_pages_alloc(int num_pool_blocks, int32_t* block_table, int rows, int max_blocks,
                    int32_t* refs, const int32_t* row, const int32_t* first, const int32_t* last,
                    int n, void* ws, size_t ws_bytes, cudaStream_t stream) {
  RowList rl;
  int rc = check_table(num_pool_blocks, block_table, rows, max_blocks, refs);
  if (rc || (rc = check_ranges(row, first, last, n, rows, max_blocks, true, &rl))) return rc;
  if ((rc = check_ws(ws, ws_bytes, msa_pages_workspace_bytes(num_pool_blocks)))) return rc;
  if (n == 0) return MSA_OK;
  return cuda_status(
      launch_pages_alloc(PageTable{block_table, rows, max_blocks, refs, num_pool_blocks}, rl,
                         static_cast<char*>(ws), stream));
}

int msa_pages_compact(const msa_pool* pools, int npools, int num_pool_blocks,
                      const int32_t* block_table, int rows, int max_blocks, const int32_t* refs,
                      int32_t* table_out, int32_t* refs_out, int32_t* live, void* ws,
                      size_t ws_bytes, cudaStream_t stream) {
  PoolSet ps;
  int rc = check_pools(pools, npools, &ps);
  if (rc || (rc = check_table(num_pool_blocks, block_table, rows, max_blocks, refs))) return rc;
  if (!table_out || !refs_out || !live || ((uintptr_t)table_out & 3u) ||
      ((uintptr_t)refs_out & 3u) || ((uintptr_t)live & 3u))
    return MSA_ERR_INVALID_ARG;
  if ((rc = check_ws(ws, ws_bytes, msa_pages_workspace_bytes(num_pool_blocks)))) return rc;
  return cuda_status(launch_pages_compact(
      ps,
      PageTable{const_cast<int32_t*>(block_table), rows, max_blocks, const_cast<int32_t*>(refs),
                num_pool_blocks},
      table_out, refs_out, live, static_cast<char*>(ws), stream));
}

}  // extern "C"

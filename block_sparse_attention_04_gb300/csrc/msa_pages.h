// Page operations of paged pools (internal interface).
#pragma once
#include "msa_internal.h"

namespace msa {

constexpr int kMaxPools = MSA_MAX_POOLS;

struct PoolSet {
  msa_pool pool[kMaxPools];
  int n;
};

// A block table [rows][max_blocks] and the reference counts of the pool's
// pages (the number of table entries that map each; 0: free).
struct PageTable {
  int32_t* table;
  int rows, max_blocks;
  int32_t* refs;
  int pages;
};

// Row lists of a call, by value.
struct RowList {
  int n;
  int32_t a[kMaxBatch], b[kMaxBatch], c[kMaxBatch];
};

size_t pages_workspace_bytes(int pages);

cudaError_t launch_pages_copy(const PoolSet& ps, int pages, const int32_t* src, const int32_t* dst,
                              int n, char* ws, cudaStream_t st);
// rows: a = source rows, b = destination rows, c = token counts
cudaError_t launch_pages_fork(const PoolSet& ps, const PageTable& pt, const RowList& rows, char* ws,
                              cudaStream_t st);
// rows: a = rows, [b, c) = block ranges
cudaError_t launch_pages_free(const PageTable& pt, const RowList& rows, char* ws, cudaStream_t st);
cudaError_t launch_pages_alloc(const PageTable& pt, const RowList& rows, char* ws, cudaStream_t st);
cudaError_t launch_pages_compact(const PoolSet& ps, const PageTable& pt, int32_t* table_out,
                                 int32_t* refs_out, int32_t* live, char* ws, cudaStream_t st);

}  // namespace msa

// Launch arguments and launchers of the page tables' bookkeeping and of the copies
// within a paged cache.
#pragma once

#include <cuda_runtime.h>

#include "attn.h"

namespace eba {

struct ReleaseArgs {
  attn_pool_t pool;
  int* table;
  long long table_stride;
  int max_pages, n_seqs;
  const int* first;
  const int* last;
  int* status;
};
cudaError_t launch_release(const ReleaseArgs& a, cudaStream_t stream);

// Fork (n pairs src, dst) or reserve (n sequences).
struct PoolArgs {
  attn_pool_t pool;
  int* table;
  long long table_stride;
  int max_pages, n_seqs, n;
  int* lens;             // reserve: read only
  const int* new_lens;   // reserve
  const int* src;        // fork
  const int* dst;
  int* from;
  int* to;
  int* status;
};
cudaError_t launch_fork(const PoolArgs& a, cudaStream_t stream);
cudaError_t launch_reserve(const PoolArgs& a, cudaStream_t stream);

// Strides in bytes.
struct CopyArgs {
  unsigned char* k;
  unsigned char* v;
  long long k_strides[3], v_strides[3];
  int n_pages, page_size, H_kv;
  int row;  // bytes: 64, 128 or 256
  const int* from;
  const int* to;
  int n;
  int* status;
};
cudaError_t launch_copy(const CopyArgs& a, cudaStream_t stream);

struct GatherArgs {
  unsigned char* k;
  unsigned char* v;
  long long k_strides[3], v_strides[3];
  int n_pages, page_size, H_kv;
  int row;
  const int* table;
  long long table_stride;
  int max_pages, n_seqs;
  const int* places;
  const int* cu;
  int T;
  const int* to_table;
  long long to_stride;
  int to_max_pages;
  const int* to_start;  // null: 0
  bool in_place;        // the tables are the same: a sequence's rows go in order
  int* status;
};
cudaError_t launch_gather(const GatherArgs& a, cudaStream_t stream);

}  // namespace eba

// Launch arguments and launcher of the attention of several drafted tokens per sequence
// over the paged cache.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "attn.h"

namespace eba {

// One CTA on each of 152 SMs; any number of SMs gives the same results.
constexpr int kTreeCtas = 152;
constexpr int kTreeKeys = 128;  // keys of a tile
constexpr int kTreeRows = 128;  // (token, head) rows of an item
// Tiles that an item's end takes as long as, in the split of the list between CTAs. (16 times
// up to 6007 keys, 16 heads of 64: 0 / 1 / 2 / 3 / 5 tiles 90 / 84 / 78 / 76 / 78 us; 32 times up
// to 8191 keys, 8 heads of 128: 136 / 134 / 134 / 132 / 133 us)
constexpr int kTreeEnd = 3;
struct TreeArgs {
  const __nv_bfloat16* q;  // [T, H, d], strides below
  long long q_token, q_head;
  const unsigned char* k;  // the cache's pages
  const unsigned char* v;
  long long k_strides[3], v_strides[3];  // page, slot, head, in bytes
  attn_cache_t cache;
  const int* table;
  long long table_stride;
  const int* lens;
  const int* cu;          // null: one token per sequence
  const long long* mask;  // null: each token sees those before it
  long long mask_stride;
  int words;              // of a token's mask
  unsigned page_mul;      // key / page_size = key * page_mul >> page_shift, for every int >= 0
  int page_shift;
  int box;                // keys of a TMA load: 32 or 16, a divisor of page_size; 0: no TMA
  int max_len;            // keys a table row can hold
  int T, B, H, group;
  int window, sinks;      // window 0: none
  float scale_log2;       // scale * log2(e)
  float o_scale;          // the values' scale
  __nv_bfloat16* o;       // [T, H, d]
  float* lse;             // [T, H]
  // [kTreeCtas]: where the CTA's run begins an item that it does not end: the item's place
  // in the run (0 first, 1 a later one) and its parts; parts 0: no such item
  int2* cut;
  int4* item;             // of the item: sequence, K/V head, query tile
  float* part_o;          // [2 kTreeCtas, 128, d]
  float2* part_ml;        // [2 kTreeCtas, 128]: reference, sum
  int* status;
  unsigned long long limit_ns;
};
// tk, tv: 4-D views (d, H_kv, page_size, n_pages) of the pages, with boxes of a.box rows of 64
// bf16 elements (128-byte swizzle) or of a whole e4m3 row; unused without a.box. ctas: the
// grid. join: items may be cut between CTAs.
cudaError_t launch_tree(const CUtensorMap& tk, const CUtensorMap& tv, const TreeArgs& a, int ctas, bool join, cudaStream_t stream);

}  // namespace eba

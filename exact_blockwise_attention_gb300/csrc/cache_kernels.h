// Launch arguments and launchers of the position rotation, the paged cache's append
// and single-token decode (as kernels.h has those of the attention over tensors).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "attn.h"

namespace eba {

// Rotation of q and k (in[1] with H[1] = 0 heads: q alone). Strides in
// elements: batch, head, token.
struct RopeArgs {
  const void* in[2];
  void* out[2];
  long long si[2][3], so[2][3];
  int H[2];
  const int* pos;  // [axis, batch, token]
  long long pos_axis, pos_batch;
  long long tokens;  // batch * L
  int L;
  int heads_per;  // heads a thread walks (set by the launcher)
  float sign;     // +1 rotates, -1 rotates back (the gradient)
  attn_rope_t rope;
};
cudaError_t launch_rope(RopeArgs& a, int d, cudaStream_t stream);

// New rows into a paged cache. rope.n_pairs = 0: keys go in as they are; pos
// null: a token's position is its place in the cache.
struct AppendArgs {
  const void* k;
  const void* v;
  long long k_token, k_head, v_token, v_head;
  attn_cache_t cache;
  const int* table;
  long long table_stride;
  int max_pages;
  const int* lens;
  const int* cu_new;  // null: one token per sequence
  int n_seqs;
  long long tokens;
  int heads_per;  // set by the launcher
  const int* pos;
  long long pos_axis;
  float k_inv, v_inv;  // 1 / scale of an e4m3 cache
  int* status;
  attn_rope_t rope;
};
cudaError_t launch_append(AppendArgs& a, cudaStream_t stream);

// One new token per sequence over the paged cache. The grid is fixed (two CTAs
// on each of 152 SMs); any number of SMs gives the same results.
constexpr int kDecodeCtas = 304;
// Keys of a tile, 32 KB of keys and values (of each head, a quarter with four).
constexpr int decode_tile_keys(int row_bytes) { return 16384 / row_bytes; }
struct DecodeArgs {
  const __nv_bfloat16* q;  // [B, H, d], strides below
  long long q_seq, q_head;
  const unsigned char* k;  // the cache's pages
  const unsigned char* v;
  long long k_strides[3], v_strides[3];  // page, slot, head, in bytes
  attn_cache_t cache;
  const int* table;
  long long table_stride;
  const int* lens;
  int max_len;  // keys a table row can hold
  int B, H;
  int group;   // query heads per K/V head
  int rows;    // query heads a CTA holds: 8 or 16
  int blocks;  // ceil(group / rows)
  int per_item;  // K/V heads of an item: 1, or 4 neighbouring ones
  int heads;   // H_kv * blocks / per_item: items of a sequence
  int splits;  // > 0: clusters of that many CTAs, one per item; 0: one list of tiles
  float scale_log2;  // scale * log2(e)
  float o_scale;     // the values' scale
  __nv_bfloat16* o;  // [B, H, d]
  float* lse;        // [B, H]
  // Null where no item can be cut between CTAs. Else [kDecodeCtas]: the item that the
  // CTA's run ends in the middle of, and its parts << 16 | runs since its first one << 1
  // | the slot of its first part in that run; parts 0: none that begins in or covers the
  // run.
  int2* cut;
  float* part_o;     // [2 kDecodeCtas, per_item rows, d]
  float2* part_ml;   // [2 kDecodeCtas, per_item rows]: reference, sum
  const int* pos;
  long long pos_axis;
  int* status;
  unsigned long long limit_ns;
  attn_rope_t rope;
};
cudaError_t launch_decode(const DecodeArgs& a, int ctas, bool join, cudaStream_t stream);

}  // namespace eba

// C ABI of the attention library: argument validation, TMA descriptor
// construction, the per-device status word, and kernel launches. Declarations
// and the contract of each entry point are in include/attn.h.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "attn.h"
#include "cache_kernels.h"
#include "kernels.h"

namespace {

constexpr unsigned long long kDefaultWaitNs = 2000000000ull;  // 2 s
constexpr int kMaxDevices = 64;
constexpr float kLog2e = 1.4426950408889634f;

std::atomic<unsigned long long> g_wait_limit_ns{kDefaultWaitNs};
thread_local int t_last_cuda_error = 0;  // cudaError_t of the last failing call

int cuda_fail(cudaError_t e) {
  t_last_cuda_error = static_cast<int>(e);
  return ATTN_ERR_CUDA;
}

// One status word per device, in this module's device globals (no allocation).
__device__ int g_status_word;

template <typename F>
F driver_fn(const char* name) {
  void* p = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPointByVersion(name, &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
      q != cudaDriverEntryPointSuccess)
    return nullptr;
  return reinterpret_cast<F>(p);
}

// Make sure the calling host thread has a CUDA context bound (a fresh thread,
// e.g. an autograd worker, may have none), preferring the device whose context
// is already current. Returns the device, or -1 with the error recorded. When
// ctx_id is given it receives the bound context's process-unique ID (never
// reused, even when a context is destroyed and another is created at the same
// handle), or 0 if the driver cannot tell.
int bind_device(unsigned long long* ctx_id = nullptr) {
  using CtxGetCurrent = CUresult(CUDAAPI*)(CUcontext*);
  using CtxGetDevice = CUresult(CUDAAPI*)(CUdevice*);
  using CtxGetId = CUresult(CUDAAPI*)(CUcontext, unsigned long long*);
  static CtxGetCurrent get_ctx = driver_fn<CtxGetCurrent>("cuCtxGetCurrent");
  static CtxGetDevice get_dev = driver_fn<CtxGetDevice>("cuCtxGetDevice");
  static CtxGetId get_id = driver_fn<CtxGetId>("cuCtxGetId");
  int dev = -1;
  CUcontext ctx = nullptr;
  if (get_ctx && get_dev && get_ctx(&ctx) == CUDA_SUCCESS && ctx) {
    CUdevice d;
    if (get_dev(&d) == CUDA_SUCCESS) dev = static_cast<int>(d);
  }
  cudaError_t e = cudaSuccess;
  if (dev < 0) e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaSetDevice(dev);  // binds the primary context to this thread
  if (e != cudaSuccess) {
    t_last_cuda_error = static_cast<int>(e);
    return -1;
  }
  if (ctx_id) {
    *ctx_id = 0;
    ctx = nullptr;
    unsigned long long id = 0;
    if (get_ctx && get_id && get_ctx(&ctx) == CUDA_SUCCESS && ctx &&
        get_id(ctx, &id) == CUDA_SUCCESS)
      *ctx_id = id;
  }
  return dev;
}

int* status_word_ptr() {
  return static_cast<int*>(eba::symbol_address(&g_status_word, eba::kSymStatusWord));
}

}  // namespace

namespace eba {

void record_cuda_error(int e) { t_last_cuda_error = e; }

// Device addresses of the library's __device__ variables, cached per device
// and symbol together with the ID of the context they were looked up in: a
// different current context (one re-created after a device reset, say) means
// a fresh lookup, so a stale address is never handed to a kernel. Without a
// context ID from the driver every call looks the address up again.
void* symbol_address(const void* symbol, int slot) {
  struct Entry {
    unsigned long long ctx;
    void* addr;
  };
  static std::mutex mu;
  static Entry cache[kMaxDevices][kSymSlots] = {};
  unsigned long long ctx = 0;
  const int dev = bind_device(&ctx);
  if (dev < 0 || dev >= kMaxDevices || slot < 0 || slot >= kSymSlots) return nullptr;
  std::lock_guard<std::mutex> lock(mu);
  Entry& c = cache[dev][slot];
  if (ctx == 0 || c.ctx != ctx || !c.addr) {
    void* p = nullptr;
    cudaError_t e = cudaGetSymbolAddress(&p, symbol);
    if (e != cudaSuccess) {
      t_last_cuda_error = static_cast<int>(e);
      c = Entry{0, nullptr};
      return nullptr;
    }
    c = Entry{ctx, p};
  }
  return c.addr;
}

}  // namespace eba

namespace {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn =
      driver_fn<PFN_cuTensorMapEncodeTiled_v12000>("cuTensorMapEncodeTiled");
  return fn;
}

// 3-D view [B*H, L, d] of a contiguous bf16 [B, H, L, d] tensor; box of
// 64 x 128 x 1 elements (128-byte rows) with the 128-byte swizzle. Rows past L
// read as zero.
bool make_map(CUtensorMap* m, const void* ptr, long long BH, int L, int d) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(L),
                        static_cast<cuuint64_t>(BH)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2,
                           static_cast<cuuint64_t>(L) * static_cast<cuuint64_t>(d) * 2};
  cuuint32_t box[3] = {64, static_cast<cuuint32_t>(eba::kTileRows), 1};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides,
                  box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) t_last_cuda_error = static_cast<int>(r);
  return r == CUDA_SUCCESS;
}

// 3-D view [B*H, L, d] of a contiguous fp32 [B, H, L, d] tensor; box of
// 32 x 128 x 1 elements (128-byte rows, 128-byte swizzle), for TMA reduce-add.
bool make_map_f32(CUtensorMap* m, void* ptr, long long BH, int L, int d) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(L),
                        static_cast<cuuint64_t>(BH)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 4,
                           static_cast<cuuint64_t>(L) * static_cast<cuuint64_t>(d) * 4};
  cuuint32_t box[3] = {32, static_cast<cuuint32_t>(eba::kTileRows), 1};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, ptr, dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) t_last_cuda_error = static_cast<int>(r);
  return r == CUDA_SUCCESS;
}

// 3-D view (d, H, T) of a contiguous token-major [T, H, d] tensor (bf16, or
// fp32 for the dQ accumulator): a box is 128 consecutive tokens of one head,
// 64 bf16 / 32 fp32 columns wide (128-byte rows, 128-byte swizzle), laid out
// in shared memory exactly like a box of the [B*H, L, d] view. Tokens past T
// read as zero.
bool make_map_thd(CUtensorMap* m, const void* ptr, long long T, int H, int d, bool f32) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t esz = f32 ? 4 : 2;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(H),
                        static_cast<cuuint64_t>(T)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * esz,
                           static_cast<cuuint64_t>(H) * static_cast<cuuint64_t>(d) * esz};
  cuuint32_t box[3] = {f32 ? 32u : 64u, 1, static_cast<cuuint32_t>(eba::kTileRows)};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                  const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) t_last_cuda_error = static_cast<int>(r);
  return r == CUDA_SUCCESS;
}

// 3-D view (inner, rows, BH) of a contiguous one-byte (e4m3) tensor
// [BH, rows, inner]; box of 128 x 128 x 1 bytes with the 128-byte swizzle.
// (Q, K: inner = d = 128; V^T: inner = Lk, rows = d.) Elements past the
// extents read as zero.
bool make_map_u8(CUtensorMap* m, const void* ptr, long long BH, int rows, int inner) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(rows),
                        static_cast<cuuint64_t>(BH)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(inner),
                           static_cast<cuuint64_t>(rows) * static_cast<cuuint64_t>(inner)};
  cuuint32_t box[3] = {128, static_cast<cuuint32_t>(eba::kTileRows), 1};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(ptr), dims, strides, box,
                  estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) t_last_cuda_error = static_cast<int>(r);
  return r == CUDA_SUCCESS;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Checks packed-sequence offsets and fills the kernels' table: per sequence,
// forward items are pairs of 128-row query tiles, backward items 128-row key
// tiles. Tq, Tk: the packed totals.
int build_varlen(const int* cu_q, const int* cu_k, int n_seqs, int H, int d, float scale,
                 bool backward, eba::VarlenTable* vt, int* Tq, int* Tk) {
  if (!cu_q || !cu_k || n_seqs < 1 || H < 1) return ATTN_ERR_INVALID_ARG;
  if (n_seqs > ATTN_MAX_SEQS) return ATTN_ERR_UNSUPPORTED;
  if (!std::isfinite(scale) || !(scale > 0.0f)) return ATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  if (cu_q[0] != 0 || cu_k[0] != 0) return ATTN_ERR_INVALID_ARG;
  constexpr int R = eba::kTileRows;
  vt->n_seqs = n_seqs;
  vt->cu_q[0] = vt->cu_k[0] = vt->cu_items[0] = vt->cu_qt[0] = 0;
  long long items = 0, qtiles = 0;
  for (int s = 0; s < n_seqs; ++s) {
    const int lq = cu_q[s + 1] - cu_q[s], lk = cu_k[s + 1] - cu_k[s];
    if (cu_q[s + 1] < cu_q[s] || cu_k[s + 1] < cu_k[s]) return ATTN_ERR_INVALID_ARG;
    const long long nqt = (static_cast<long long>(lq) + R - 1) / R;
    const long long nkt = (static_cast<long long>(lk) + R - 1) / R;
    qtiles += nqt;
    // a backward item is a key tile against the sequence's query tiles: a
    // sequence without queries has none (its dK, dV rows are zeroed apart)
    items += backward ? (lq > 0 ? nkt : 0) : (nqt + 1) / 2;
    if (items * H >= (1ll << 31) || qtiles * R * H >= (1ll << 31)) return ATTN_ERR_INVALID_ARG;
    vt->cu_q[s + 1] = cu_q[s + 1];
    vt->cu_k[s + 1] = cu_k[s + 1];
    vt->cu_items[s + 1] = static_cast<int>(items);
    vt->cu_qt[s + 1] = static_cast<int>(qtiles);
  }
  vt->total = static_cast<int>(items);
  // Work order: sequences by decreasing cost per item (the backward walks a
  // sequence's query tiles per item, the forward its key tiles), ties in
  // sequence order.
  int cost[ATTN_MAX_SEQS];
  for (int s = 0; s < n_seqs; ++s) {
    cost[s] = backward ? vt->cu_qt[s + 1] - vt->cu_qt[s] : (vt->cu_k[s + 1] - vt->cu_k[s] + R - 1) / R;
    vt->order[s] = s;
  }
  std::stable_sort(vt->order, vt->order + n_seqs, [&](int x, int y) { return cost[x] > cost[y]; });
  vt->cu_rank[0] = 0;
  for (int r = 0; r < n_seqs; ++r) {
    const int s = vt->order[r];
    vt->cu_rank[r + 1] = vt->cu_rank[r] + (vt->cu_items[s + 1] - vt->cu_items[s]);
  }
  *Tq = cu_q[n_seqs];
  *Tk = cu_k[n_seqs];
  if (*Tq < 1 || *Tk < 1) return ATTN_ERR_INVALID_ARG;
  return ATTN_OK;
}

int check_sizes(int B, int H, int Lq, int Lk, int d, float scale) {
  if (B < 1 || H < 1 || Lq < 1 || Lk < 1) return ATTN_ERR_INVALID_ARG;
  if (static_cast<long long>(B) * H >= (1ll << 31)) return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !(scale > 0.0f)) return ATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  return ATTN_OK;
}

int check_ptrs(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!p) return ATTN_ERR_INVALID_ARG;
  for (const void* p : ps)
    if (!aligned16(p)) return ATTN_ERR_MISALIGNED;
  return ATTN_OK;
}

// Strides that keep every row 16-byte aligned.
int check_strides(const long long* s, int n, int multiple) {
  for (int i = 0; i < n; ++i) {
    if (s[i] < 0) return ATTN_ERR_INVALID_ARG;
    if (s[i] % multiple != 0) return ATTN_ERR_MISALIGNED;
  }
  return ATTN_OK;
}

int check_rope(const attn_rope_t& r, int d) {
  if (r.n_pairs < 8 || r.n_pairs % 8 != 0 || r.n_pairs > d / 2 || r.n_axes < 1 ||
      r.n_axes > ATTN_MAX_AXES)
    return ATTN_ERR_INVALID_ARG;
  for (int i = 0; i < r.n_pairs; ++i)
    if (r.axis[i] >= r.n_axes) return ATTN_ERR_INVALID_ARG;
  return ATTN_OK;
}

// x mod 1 in units of 2^-64, to nearest.
unsigned long long fraction64(double x) {
  x = std::ldexp(x - std::trunc(x), 32);  // exact, as is each step but the last
  const double whole = std::trunc(x);
  return (static_cast<unsigned long long>(static_cast<long long>(whole)) << 32) +
         static_cast<unsigned long long>(std::llrint(std::ldexp(x - whole, 32)));
}

// Grid limits of the per-row kernels (a thread per 16 elements, heads in y).
bool rows_fit(long long tokens, int d, long long heads) {
  return tokens * (d / 16) < (1ll << 37) && heads <= 65535;
}

int check_cache(const attn_cache_t* c) {
  if (!c) return ATTN_ERR_INVALID_ARG;
  if (c->n_pages < 1 || c->n_pages >= (1ll << 31) || c->page_size < 1 || c->H_kv < 1 ||
      c->H_kv > 65535)
    return ATTN_ERR_INVALID_ARG;
  for (float f : {c->k_scale, c->v_scale})
    if (!std::isfinite(f) || !(f > 0.0f) || !std::isfinite(1.f / f)) return ATTN_ERR_INVALID_ARG;
  if ((c->d != 64 && c->d != 128) || (c->type != ATTN_CACHE_BF16 && c->type != ATTN_CACHE_E4M3))
    return ATTN_ERR_UNSUPPORTED;
  if (c->type == ATTN_CACHE_BF16 && (c->k_scale != 1.f || c->v_scale != 1.f))
    return ATTN_ERR_INVALID_ARG;
  int s = check_ptrs({c->k, c->v});
  const int multiple = c->type == ATTN_CACHE_E4M3 ? 16 : 8;
  if (s == ATTN_OK) s = check_strides(c->k_strides, 3, multiple);
  if (s == ATTN_OK) s = check_strides(c->v_strides, 3, multiple);
  const long long sizes[3] = {c->n_pages, c->page_size, c->H_kv};
  for (int i = 0; i < 3 && s == ATTN_OK; ++i)
    for (long long st : {c->k_strides[i], c->v_strides[i]})
      if (sizes[i] > 1 && st < c->d) s = ATTN_ERR_INVALID_ARG;  // rows apart
  return s;
}

int check_table(const int* table, long long stride, int max_pages, const int* lens, int n_seqs) {
  if (!table || !lens || max_pages < 1 || n_seqs < 1 || stride < 0) return ATTN_ERR_INVALID_ARG;
  return ATTN_OK;
}

// How a decode call is cut up, from what the host knows: the sizes and the keys
// a table can hold. ok: the sizes are within the limits.
struct DecodePlan {
  bool ok;
  int rows, blocks;      // query heads of a CTA (8 or 16), blocks of them in a group
  int per_item;          // K/V heads of an item
  int heads, max_len;    // items of a sequence; keys of a table row
  int splits, ctas;      // see DecodeArgs; the grid
  bool join;             // items may be cut between CTAs
  size_t slots, bytes;   // of the workspace: parts, all
};
DecodePlan decode_plan(int B, int H, int H_kv, int d, long long capacity, int type) {
  DecodePlan p{};
  const int group = H / H_kv;
  // the matrix instruction has 8 columns: groups of up to 8 heads take one set
  // of them, larger ones two at a time
  p.rows = group <= 8 ? 8 : 16;
  p.blocks = (group + p.rows - 1) / p.rows;
  const int row = type == ATTN_CACHE_E4M3 ? d : 2 * d;
  int tile = eba::decode_tile_keys(row);
  p.per_item = 1;
  p.max_len = static_cast<int>(std::min(capacity, (1ll << 31) - 1 - tile));
  p.heads = H_kv * p.blocks;
  long long item_tiles = (p.max_len + tile - 1) / tile;
  long long items = static_cast<long long>(B) * p.heads;
  if (items >= (1ll << 31) || item_tiles * p.heads >= (1ll << 31) ||
      item_tiles * p.heads * B >= (1ll << 31))
    return p;
  p.ok = true;
  // Clusters, where one wave of them leaves each CTA few tiles: one launch instead of
  // two and no workspace, but only as even as the lengths, and with less than a full
  // wave not all SMs. Measured, cluster against list (us; longest sequence, others
  // random down to an eighth): 64 CTAs at 2 tiles each 6.8 / 7.0, at 4 8.2 / 7.9
  // (1 x 8 heads of 128, bf16; the 0.3 us are lost in a replayed graph, but the host
  // needs 18 / 24 for a call), at 8 11.2 / 8.7;
  // 256 CTAs at 8 tiles 12.8 / 14.1 (16 x 8 heads) and
  // 15.9 / 16.4 (e4m3), at 16 20.1 / 20.2 and 23.5 / 20.4. The table decides, not the
  // lengths, which the host does not know: with a table of 131072 keys instead of a tight
  // one (list against cluster) 1 x 333 keys take 7.6 / 6.1, 16 x up to 500 11.3 / 8.7,
  // 4 x up to 2000 of 2 heads 8.3 / 7.9.
  constexpr int wave = eba::kDecodeCtas;
  int splits = 1;
  while (splits < 8 && splits < item_tiles && items * splits * 2 <= wave) splits *= 2;
  const int most = items * splits >= wave * 3 / 4 ? 8 : 4;  // tiles of a CTA
  if (items * splits <= wave && item_tiles <= most * splits) {
    p.splits = splits;
    p.ctas = static_cast<int>(items * splits);
    return p;
  }
  // Rows of at most 128 bytes, and at least 8 of them side by side: four neighbouring
  // heads to an item, so that a CTA reads their rows of a token together; unless that
  // leaves so few items that each is cut into many parts. Measured, fours against
  // single heads (us): 16 sequences x 16 heads of 64, bf16, up to 32000 keys 225 /
  // 255; 32 x 8 heads of 64, e4m3, 16000 keys 57 / 60; 1 x 16 heads of 64 29 / 27;
  // 4 heads of 128, e4m3, 55 / 52.
  if (row <= 128 && H_kv % 4 == 0 && H_kv >= 8 && group <= 8 && items / 4 >= 16) {
    p.per_item = 4;
    p.heads /= 4;
    items /= 4;
    tile /= 4;
    item_tiles = (p.max_len + tile - 1) / tile;
  }
  // no more CTAs than tiles the tables can hold; a single-tile item is never cut
  p.ctas = static_cast<int>(std::min<long long>(wave, items * item_tiles));
  p.join = item_tiles > 1;
  if (!p.join) return p;
  p.slots = 2 * static_cast<size_t>(wave) * p.rows * p.per_item;
  p.bytes = wave * sizeof(int2) + p.slots * (d + 2) * sizeof(float);
  return p;
}

// Short sequences (at most 64 queries and keys) are packed several to a
// 128-row tile; returns the number per tile, or 0 for the per-head tiling.
int packing(int Lq, int Lk) {
  const int L = Lq > Lk ? Lq : Lk;
  return L <= eba::kTileRows / 2 ? eba::kTileRows / L : 0;
}

int fwd_packed(const void* q, const void* k, const void* v, void* o, float* lse, long long BH,
               int Lq, int Lk, int d, int pack, float scale, void* stream) {
  int* status = status_word_ptr();
  if (!status) return ATTN_ERR_CUDA;
  if (BH * Lq >= (1ll << 31) || BH * Lk >= (1ll << 31)) return ATTN_ERR_INVALID_ARG;
  CUtensorMap tq, tk, tv;
  if (!make_map(&tq, q, 1, static_cast<int>(BH * Lq), d) ||
      !make_map(&tk, k, 1, static_cast<int>(BH * Lk), d) ||
      !make_map(&tv, v, 1, static_cast<int>(BH * Lk), d))
    return ATTN_ERR_CUDA;
  eba::FwdArgs a{};
  a.B = 1;
  a.H = 1;
  a.group = 1;
  a.Lq = static_cast<int>(BH * Lq);  // flattened rows: lse / O row = tile row + item offset
  a.Lk = static_cast<int>(BH * Lk);
  a.n_chunks = 1;
  a.bounds[0] = 0;
  a.bounds[1] = a.Lk;
  a.scale_log2 = scale * kLog2e;
  a.o = o;
  a.lse = lse;
  a.status = status;
  a.limit_ns = g_wait_limit_ns.load();
  const eba::PackedTiles pt{pack, static_cast<int>(BH), Lq, Lk};
  cudaError_t e = eba::launch_fwd_packed(tq, tk, tv, a, pt, d, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTN_OK : cuda_fail(e);
}

// Sequences of at most eba::kShortMax queries and keys: the CUDA-core path.
int fwd_short(const void* q, const void* k, const void* v, void* o, float* lse, long long BH,
              int Lq, int Lk, int d, float scale, void* stream) {
  int* status = status_word_ptr();
  if (!status) return ATTN_ERR_CUDA;
  eba::ShortArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.o = o;
  a.lse = lse;
  a.n_seq = BH;
  a.Lq = Lq;
  a.Lk = Lk;
  a.scale_log2 = scale * kLog2e;
  a.status = status;
  a.limit_ns = g_wait_limit_ns.load();
  cudaError_t e = eba::launch_fwd_short(a, d, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTN_OK : cuda_fail(e);
}

// H_kv: K/V heads (H for multi-head attention; a divisor of H for grouped-query).
int fwd_common(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
               int H_kv, int Lq, int Lk, int d, const int* bounds, int n_chunks, float scale,
               bool partial, void* stream) {
  int* status = status_word_ptr();
  if (!status) return ATTN_ERR_CUDA;
  const long long BH = static_cast<long long>(B) * H;
  const long long BHkv = static_cast<long long>(B) * H_kv;
  CUtensorMap tq, tk, tv;
  if (!make_map(&tq, q, BH, Lq, d) || !make_map(&tk, k, BHkv, Lk, d) ||
      !make_map(&tv, v, BHkv, Lk, d))
    return ATTN_ERR_CUDA;
  eba::FwdArgs a{};
  a.B = B;
  a.H = H;
  a.group = H / H_kv;
  a.Lq = Lq;
  a.Lk = Lk;
  a.n_qtiles = (Lq + eba::kTileRows - 1) / eba::kTileRows;
  a.n_pairs = (a.n_qtiles + 1) / 2;
  a.n_chunks = n_chunks;
  a.scale_log2 = scale * kLog2e;
  for (int c = 0; c <= n_chunks; ++c) a.bounds[c] = bounds[c];
  a.o = o;
  a.lse = lse;
  a.o_chunk_stride = BH * Lq * d;
  a.lse_chunk_stride = BH * Lq;
  a.status = status;
  a.limit_ns = g_wait_limit_ns.load();
  if (static_cast<long long>(a.n_pairs) * BH >= (1ll << 31)) return ATTN_ERR_INVALID_ARG;
  cudaError_t e = eba::launch_fwd(tq, tk, tv, a, d, partial, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTN_OK : cuda_fail(e);
}

}  // namespace

extern "C" {

int attn_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
             int Lq, int Lk, int d, float scale, void* stream) {
  int s = check_sizes(B, H, Lq, Lk, d, scale);
  if (s != ATTN_OK) return s;
  if ((s = check_ptrs({q, k, v, o, lse})) != ATTN_OK) return s;
  // Sequences of 5 to 8 tokens: the CUDA-core path (8 x 8 blocks, one warp
  // each). With 4 or fewer on both sides it costs as much per sequence as an
  // 8 x 8 one, and the tensor-core tiles, packing 32 such sequences each, are
  // faster there (measured at B*H = 100352, 4 x 4, d = 64: 74 against 62 us).
  if (std::max(Lq, Lk) <= eba::kShortMax && std::max(Lq, Lk) > eba::kShortMax / 2)
    return fwd_short(q, k, v, o, lse, static_cast<long long>(B) * H, Lq, Lk, d, scale, stream);
  if (const int pack = packing(Lq, Lk))
    return fwd_packed(q, k, v, o, lse, static_cast<long long>(B) * H, Lq, Lk, d, pack, scale,
                      stream);
  const int bounds[2] = {0, Lk};
  return fwd_common(q, k, v, o, lse, B, H, H, Lq, Lk, d, bounds, 1, scale, false, stream);
}

int attn_fwd_fp8(const void* q8, const void* k8, const void* vt8, void* o, float* lse, int B,
                 int H, int Lq, int Lk, int d, float scale, float q_scale, float k_scale,
                 float v_scale, void* stream) {
  int s = check_sizes(B, H, Lq, Lk, d, scale);
  if (s != ATTN_OK) return s;
  for (float f : {q_scale, k_scale, v_scale})
    if (!std::isfinite(f) || !(f > 0.0f)) return ATTN_ERR_INVALID_ARG;
  if (d != 128) return ATTN_ERR_UNSUPPORTED;
  if ((s = check_ptrs({q8, k8, vt8, o, lse})) != ATTN_OK) return s;
  if (Lk % 16 != 0) return ATTN_ERR_MISALIGNED;  // V^T rows must be 16-byte multiples
  int* status = status_word_ptr();
  if (!status) return ATTN_ERR_CUDA;
  const long long BH = static_cast<long long>(B) * H;
  CUtensorMap tq, tk, tvt;
  if (!make_map_u8(&tq, q8, BH, Lq, d) || !make_map_u8(&tk, k8, BH, Lk, d) ||
      !make_map_u8(&tvt, vt8, BH, d, Lk))
    return ATTN_ERR_CUDA;
  eba::FwdArgs a{};
  a.B = B;
  a.H = H;
  a.group = 1;
  a.Lq = Lq;
  a.Lk = Lk;
  a.n_qtiles = (Lq + eba::kTileRows - 1) / eba::kTileRows;
  a.n_pairs = (a.n_qtiles + 1) / 2;
  a.n_chunks = 1;
  a.bounds[0] = 0;
  a.bounds[1] = Lk;
  a.scale_log2 = scale * q_scale * k_scale * kLog2e;
  a.o_scale = v_scale;
  a.o = o;
  a.lse = lse;
  a.status = status;
  a.limit_ns = g_wait_limit_ns.load();
  if (static_cast<long long>(a.n_pairs) * BH >= (1ll << 31)) return ATTN_ERR_INVALID_ARG;
  cudaError_t e = eba::launch_fwd_fp8(tq, tk, tvt, a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTN_OK : cuda_fail(e);
}

int attn_fwd_gqa(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
                 int H_kv, int Lq, int Lk, int d, float scale, void* stream) {
  int s = check_sizes(B, H, Lq, Lk, d, scale);
  if (s != ATTN_OK) return s;
  if (H_kv < 1 || H % H_kv != 0) return ATTN_ERR_INVALID_ARG;
  if ((s = check_ptrs({q, k, v, o, lse})) != ATTN_OK) return s;
  if (H_kv == H) return attn_fwd(q, k, v, o, lse, B, H, Lq, Lk, d, scale, stream);
  const int bounds[2] = {0, Lk};
  return fwd_common(q, k, v, o, lse, B, H, H_kv, Lq, Lk, d, bounds, 1, scale, false, stream);
}

int attn_partial_fwd(const void* q, const void* k, const void* v, float* o_part, float* lse_part,
                     int B, int H, int Lq, int Lk, int d, int k0, int k1, float scale,
                     void* stream) {
  int s = check_sizes(B, H, Lq, Lk, d, scale);
  if (s != ATTN_OK) return s;
  if (k0 < 0 || k1 < k0 || k1 > Lk) return ATTN_ERR_INVALID_ARG;
  if ((s = check_ptrs({q, k, v, o_part, lse_part})) != ATTN_OK) return s;
  const int bounds[2] = {k0, k1};
  return fwd_common(q, k, v, o_part, lse_part, B, H, H, Lq, Lk, d, bounds, 1, scale, true, stream);
}

int attn_split_fwd(const void* q, const void* k, const void* v, float* o_parts, float* lse_parts,
                   int B, int H, int Lq, int Lk, int d, const int* bounds, int n_chunks,
                   float scale, void* stream) {
  int s = check_sizes(B, H, Lq, Lk, d, scale);
  if (s != ATTN_OK) return s;
  if (!bounds) return ATTN_ERR_INVALID_ARG;
  if (n_chunks < 1) return ATTN_ERR_INVALID_ARG;
  if (n_chunks > ATTN_MAX_CHUNKS) return ATTN_ERR_UNSUPPORTED;
  if (bounds[0] != 0 || bounds[n_chunks] != Lk) return ATTN_ERR_INVALID_ARG;
  for (int c = 0; c < n_chunks; ++c)
    if (bounds[c + 1] < bounds[c]) return ATTN_ERR_INVALID_ARG;
  if ((s = check_ptrs({q, k, v, o_parts, lse_parts})) != ATTN_OK) return s;
  return fwd_common(q, k, v, o_parts, lse_parts, B, H, H, Lq, Lk, d, bounds, n_chunks, scale, true,
                    stream);
}

size_t attn_bwd_workspace_size(int B, int H, int Lq, int Lk, int d) {
  if (check_sizes(B, H, Lq, Lk, d, 1.0f) != ATTN_OK) return 0;
  const size_t BH = static_cast<size_t>(B) * H;
  const size_t Lq_pad = (static_cast<size_t>(Lq) + eba::kTileRows - 1) / eba::kTileRows *
                        eba::kTileRows;
  return BH * Lq * d * sizeof(float)      // dQ accumulator
         + 2 * BH * Lq_pad * sizeof(float);  // -lse2 and D
}

int attn_bwd(const void* q, const void* k, const void* v, const void* o, const void* dO,
             const float* lse, void* dq, void* dk, void* dv, int B, int H, int Lq, int Lk, int d,
             float scale, void* workspace, size_t workspace_bytes, void* stream) {
  return attn_bwd_gqa(q, k, v, o, dO, lse, dq, dk, dv, B, H, H, Lq, Lk, d, scale, workspace,
                      workspace_bytes, stream);
}

int attn_bwd_gqa(const void* q, const void* k, const void* v, const void* o, const void* dO,
                 const float* lse, void* dq, void* dk, void* dv, int B, int H, int H_kv, int Lq,
                 int Lk, int d, float scale, void* workspace, size_t workspace_bytes,
                 void* stream) {
  int s = check_sizes(B, H, Lq, Lk, d, scale);
  if (s != ATTN_OK) return s;
  if (H_kv < 1 || H % H_kv != 0) return ATTN_ERR_INVALID_ARG;
  if ((s = check_ptrs({q, k, v, o, dO, lse, dq, dk, dv})) != ATTN_OK) return s;
  if (!workspace || workspace_bytes < attn_bwd_workspace_size(B, H, Lq, Lk, d))
    return ATTN_ERR_WORKSPACE;
  if (!aligned16(workspace)) return ATTN_ERR_MISALIGNED;
  int* status = status_word_ptr();
  if (!status) return ATTN_ERR_CUDA;
  const long long BH = static_cast<long long>(B) * H;
  const long long BHkv = static_cast<long long>(B) * H_kv;
  if (H_kv == H && std::max(Lq, Lk) <= eba::kShortMax && std::max(Lq, Lk) > eba::kShortMax / 2) {
    // Sequences of 5 to 8 tokens: the CUDA-core backward (the workspace is
    // not used; as for the forward, 4 x 4 blocks and below stay on the packed
    // tiles).
    eba::ShortBwdArgs a{};
    a.q = q;
    a.k = k;
    a.v = v;
    a.dO = dO;
    a.lse = lse;
    a.dq = dq;
    a.dk = dk;
    a.dv = dv;
    a.n_seq = BH;
    a.Lq = Lq;
    a.Lk = Lk;
    a.scale = scale;
    a.scale_log2 = scale * kLog2e;
    a.status = status;
    a.limit_ns = g_wait_limit_ns.load();
    cudaError_t e = eba::launch_bwd_short(a, d, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? ATTN_OK : cuda_fail(e);
  }
  CUtensorMap tq, tk, tv, tdo, tdqa;
  float* ws = static_cast<float*>(workspace);
  if (const int pack = H_kv == H ? packing(Lq, Lk) : 0) {
    // Short sequences packed into tiles over the flattened [1, B*H*L, d] views.
    if (BH * Lq >= (1ll << 31) || BH * Lk >= (1ll << 31)) return ATTN_ERR_INVALID_ARG;
    const int rq = static_cast<int>(BH * Lq), rk = static_cast<int>(BH * Lk);
    if (!make_map(&tq, q, 1, rq, d) || !make_map(&tk, k, 1, rk, d) ||
        !make_map(&tv, v, 1, rk, d) || !make_map(&tdo, dO, 1, rq, d) ||
        !make_map_f32(&tdqa, ws, 1, rq, d))
      return ATTN_ERR_CUDA;
    const eba::PackedTiles pt{pack, static_cast<int>(BH), Lq, Lk};
    const int n_tiles = static_cast<int>((BH + pack - 1) / pack);
    eba::BwdArgs a{};
    a.B = 1;
    a.H = 1;
    a.group = 1;
    a.H_kv = 1;
    a.Lq = rq;
    a.Lk = rk;
    a.Lq_pad = n_tiles * eba::kTileRows;  // -lse2 / D: 128 rows per tile
    a.scale = scale;
    a.scale_log2 = scale * kLog2e;
    a.o = o;
    a.dO = dO;
    a.lse = lse;
    a.dq_acc = ws;
    a.nlse2 = ws + static_cast<size_t>(rq) * d;
    a.delta = a.nlse2 + a.Lq_pad;
    a.dq = dq;
    a.dk = dk;
    a.dv = dv;
    a.status = status;
    a.limit_ns = g_wait_limit_ns.load();
    cudaError_t e = eba::launch_bwd_packed(tq, tk, tv, tdo, tdqa, a, pt, d,
                                           static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? ATTN_OK : cuda_fail(e);
  }
  if (!make_map(&tq, q, BH, Lq, d) || !make_map(&tk, k, BHkv, Lk, d) ||
      !make_map(&tv, v, BHkv, Lk, d) || !make_map(&tdo, dO, BH, Lq, d) ||
      !make_map_f32(&tdqa, ws, BH, Lq, d))
    return ATTN_ERR_CUDA;
  eba::BwdArgs a{};
  a.B = B;
  a.H = H;
  a.group = H / H_kv;
  a.H_kv = H_kv;
  a.Lq = Lq;
  a.Lk = Lk;
  a.n_qtiles = (Lq + eba::kTileRows - 1) / eba::kTileRows;
  a.n_ktiles = (Lk + eba::kTileRows - 1) / eba::kTileRows;
  a.Lq_pad = a.n_qtiles * eba::kTileRows;
  a.scale = scale;
  a.scale_log2 = scale * kLog2e;
  a.o = o;
  a.dO = dO;
  a.lse = lse;
  a.dq_acc = ws;
  a.nlse2 = ws + BH * Lq * d;
  a.delta = a.nlse2 + BH * a.Lq_pad;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  a.status = status;
  a.limit_ns = g_wait_limit_ns.load();
  if (static_cast<long long>(a.n_ktiles) * BHkv >= (1ll << 31)) return ATTN_ERR_INVALID_ARG;
  cudaError_t e = eba::launch_bwd(tq, tk, tv, tdo, tdqa, a, d, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTN_OK : cuda_fail(e);
}

int attn_fwd_varlen(const void* q, const void* k, const void* v, void* o, float* lse,
                    const int* cu_seqlens_q, const int* cu_seqlens_k, int n_seqs, int H, int d,
                    float scale, void* stream) {
  return attn_fwd_varlen_gqa(q, k, v, o, lse, cu_seqlens_q, cu_seqlens_k, n_seqs, H, H, d, scale,
                             stream);
}

int attn_fwd_varlen_gqa(const void* q, const void* k, const void* v, void* o, float* lse,
                        const int* cu_seqlens_q, const int* cu_seqlens_k, int n_seqs, int H,
                        int H_kv, int d, float scale, void* stream) {
  eba::VarlenTable vt;
  int Tq = 0, Tk = 0;
  int s = build_varlen(cu_seqlens_q, cu_seqlens_k, n_seqs, H, d, scale, false, &vt, &Tq, &Tk);
  if (s != ATTN_OK) return s;
  if (H_kv < 1 || H % H_kv != 0) return ATTN_ERR_INVALID_ARG;
  if ((s = check_ptrs({q, k, v, o, lse})) != ATTN_OK) return s;
  int* status = status_word_ptr();
  if (!status) return ATTN_ERR_CUDA;
  CUtensorMap tq, tk, tv;
  if (!make_map_thd(&tq, q, Tq, H, d, false) || !make_map_thd(&tk, k, Tk, H_kv, d, false) ||
      !make_map_thd(&tv, v, Tk, H_kv, d, false))
    return ATTN_ERR_CUDA;
  eba::FwdArgs a{};
  a.B = 1;
  a.H = H;
  a.group = H / H_kv;
  a.Lq = Tq;
  a.Lk = Tk;
  a.n_chunks = 1;
  a.scale_log2 = scale * kLog2e;
  a.o = o;
  a.lse = lse;
  a.status = status;
  a.limit_ns = g_wait_limit_ns.load();
  cudaError_t e = eba::launch_fwd_varlen(tq, tk, tv, a, vt, d, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTN_OK : cuda_fail(e);
}

size_t attn_bwd_varlen_workspace_size(int Tq, int H, int d, int n_seqs) {
  if (Tq < 1 || H < 1 || n_seqs < 1 || n_seqs > ATTN_MAX_SEQS || (d != 64 && d != 128)) return 0;
  const size_t rows = static_cast<size_t>(Tq) + static_cast<size_t>(eba::kTileRows) * n_seqs;
  return static_cast<size_t>(Tq) * H * d * sizeof(float)  // dQ accumulator
         + 2 * static_cast<size_t>(H) * rows * sizeof(float);  // -lse2 and D
}

int attn_bwd_varlen(const void* q, const void* k, const void* v, const void* o, const void* dO,
                    const float* lse, void* dq, void* dk, void* dv, const int* cu_seqlens_q,
                    const int* cu_seqlens_k, int n_seqs, int H, int d, float scale,
                    void* workspace, size_t workspace_bytes, void* stream) {
  return attn_bwd_varlen_gqa(q, k, v, o, dO, lse, dq, dk, dv, cu_seqlens_q, cu_seqlens_k, n_seqs,
                             H, H, d, scale, workspace, workspace_bytes, stream);
}

int attn_bwd_varlen_gqa(const void* q, const void* k, const void* v, const void* o,
                        const void* dO, const float* lse, void* dq, void* dk, void* dv,
                        const int* cu_seqlens_q, const int* cu_seqlens_k, int n_seqs, int H,
                        int H_kv, int d, float scale, void* workspace, size_t workspace_bytes,
                        void* stream) {
  eba::VarlenTable vt;
  int Tq = 0, Tk = 0;
  int s = build_varlen(cu_seqlens_q, cu_seqlens_k, n_seqs, H, d, scale, true, &vt, &Tq, &Tk);
  if (s != ATTN_OK) return s;
  if (H_kv < 1 || H % H_kv != 0) return ATTN_ERR_INVALID_ARG;
  if ((s = check_ptrs({q, k, v, o, dO, lse, dq, dk, dv})) != ATTN_OK) return s;
  if (!workspace || workspace_bytes < attn_bwd_varlen_workspace_size(Tq, H, d, n_seqs))
    return ATTN_ERR_WORKSPACE;
  if (!aligned16(workspace)) return ATTN_ERR_MISALIGNED;
  int* status = status_word_ptr();
  if (!status) return ATTN_ERR_CUDA;
  float* ws = static_cast<float*>(workspace);
  CUtensorMap tq, tk, tv, tdo, tdqa;
  if (!make_map_thd(&tq, q, Tq, H, d, false) || !make_map_thd(&tk, k, Tk, H_kv, d, false) ||
      !make_map_thd(&tv, v, Tk, H_kv, d, false) || !make_map_thd(&tdo, dO, Tq, H, d, false) ||
      !make_map_thd(&tdqa, ws, Tq, H, d, true))
    return ATTN_ERR_CUDA;
  eba::BwdArgs a{};
  a.B = 1;
  a.H = H;
  a.group = H / H_kv;
  a.H_kv = H_kv;
  a.Lq = Tq;
  a.Lk = Tk;
  a.Lq_pad = vt.cu_qt[n_seqs] * eba::kTileRows;  // -lse2 / D rows per head
  a.scale = scale;
  a.scale_log2 = scale * kLog2e;
  a.o = o;
  a.dO = dO;
  a.lse = lse;
  a.dq_acc = ws;
  a.nlse2 = ws + static_cast<size_t>(Tq) * H * d;
  a.delta = a.nlse2 + static_cast<size_t>(H) * a.Lq_pad;
  a.dq = dq;
  a.dk = dk;
  a.dv = dv;
  a.status = status;
  a.limit_ns = g_wait_limit_ns.load();
  // Keys of sequences without queries get zero dK, dV (no work item reads
  // them): one fill per run of such sequences, whose rows are contiguous.
  const size_t key_row_bytes = static_cast<size_t>(H_kv) * d * 2;
  for (int s0 = 0; s0 < n_seqs;) {
    if (cu_seqlens_q[s0 + 1] > cu_seqlens_q[s0]) {
      ++s0;
      continue;
    }
    int s1 = s0;
    while (s1 < n_seqs && cu_seqlens_q[s1 + 1] == cu_seqlens_q[s1]) ++s1;
    const size_t off = static_cast<size_t>(cu_seqlens_k[s0]) * key_row_bytes;
    const size_t bytes = static_cast<size_t>(cu_seqlens_k[s1] - cu_seqlens_k[s0]) * key_row_bytes;
    if (bytes > 0) {
      cudaError_t e = cudaMemsetAsync(static_cast<char*>(dk) + off, 0, bytes,
                                      static_cast<cudaStream_t>(stream));
      if (e == cudaSuccess)
        e = cudaMemsetAsync(static_cast<char*>(dv) + off, 0, bytes, static_cast<cudaStream_t>(stream));
      if (e != cudaSuccess) return cuda_fail(e);
    }
    s0 = s1;
  }
  cudaError_t e =
      eba::launch_bwd_varlen(tq, tk, tv, tdo, tdqa, a, vt, d, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTN_OK : cuda_fail(e);
}

int attn_merge(const float* o_parts, const float* lse_parts, int n_chunks, void* o, float* lse,
               int B, int H, int Lq, int d, void* stream) {
  int s = check_sizes(B, H, Lq, 1, d, 1.0f);
  if (s != ATTN_OK) return s;
  if (n_chunks < 1) return ATTN_ERR_INVALID_ARG;
  if ((s = check_ptrs({o_parts, lse_parts, o, lse})) != ATTN_OK) return s;
  if (bind_device() < 0) return ATTN_ERR_CUDA;
  eba::MergeArgs a{};
  a.o_parts = o_parts;
  a.lse_parts = lse_parts;
  a.n_chunks = n_chunks;
  a.rows = static_cast<long long>(B) * H * Lq;
  a.o = o;
  a.lse = lse;
  cudaError_t e = eba::launch_merge(a, d, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTN_OK : cuda_fail(e);
}

int attn_rope_init(attn_rope_t* r, int n_pairs, int n_axes, const int* axis, const double* freq,
                   int interleaved) {
  if (!r || !axis || !freq) return ATTN_ERR_INVALID_ARG;
  if (n_pairs < 8 || n_pairs % 8 != 0 || n_axes < 1) return ATTN_ERR_INVALID_ARG;
  if (n_pairs > ATTN_MAX_PAIRS || n_axes > ATTN_MAX_AXES) return ATTN_ERR_UNSUPPORTED;
  for (int i = 0; i < n_pairs; ++i)
    if (axis[i] < 0 || axis[i] >= n_axes || !std::isfinite(freq[i])) return ATTN_ERR_INVALID_ARG;
  *r = attn_rope_t{};
  r->n_pairs = n_pairs;
  r->n_axes = n_axes;
  r->interleaved = interleaved != 0;
  for (int i = 0; i < n_pairs; ++i) {
    // The product with 1 / (2 pi) in two doubles, off by |freq| 2^-107: in one alone the
    // table would hold 55 bits, which positions near 2^31 bring up to 2^-25 turns.
    constexpr double kHi = 0.15915494309189535, kLo = -9.839338337591243e-18;
    const double x = freq[i] * kHi;
    const double rest = std::fma(freq[i], kHi, -x) + freq[i] * kLo;
    r->axis[i] = static_cast<unsigned char>(axis[i]);
    r->turns[i] = fraction64(x) + fraction64(rest);
  }
  return ATTN_OK;
}

int attn_rope(const attn_rope_t* r, const void* q, const long long* q_strides, void* q_out,
              const long long* q_out_strides, const void* k, const long long* k_strides,
              void* k_out, const long long* k_out_strides, const int* pos,
              const long long* pos_strides, int B, int H_q, int H_k, int L, int d, int inverse,
              void* stream) {
  if (!r || !q_strides || !q_out_strides || !pos || !pos_strides) return ATTN_ERR_INVALID_ARG;
  if (B < 1 || H_q < 1 || H_k < 0 || L < 1) return ATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  int s = check_rope(*r, d);
  if (s != ATTN_OK) return s;
  if ((s = check_ptrs({q, q_out})) != ATTN_OK) return s;
  if ((s = check_strides(q_strides, 3, 8)) != ATTN_OK) return s;
  if ((s = check_strides(q_out_strides, 3, 8)) != ATTN_OK) return s;
  if (H_k > 0) {
    if (!k_strides || !k_out_strides) return ATTN_ERR_INVALID_ARG;
    if ((s = check_ptrs({k, k_out})) != ATTN_OK) return s;
    if ((s = check_strides(k_strides, 3, 8)) != ATTN_OK) return s;
    if ((s = check_strides(k_out_strides, 3, 8)) != ATTN_OK) return s;
  }
  const long long tokens = static_cast<long long>(B) * L;
  if (!rows_fit(tokens, d, static_cast<long long>(H_q) + H_k)) return ATTN_ERR_INVALID_ARG;
  if (bind_device() < 0) return ATTN_ERR_CUDA;
  eba::RopeArgs a{};
  a.in[0] = q;
  a.out[0] = q_out;
  a.in[1] = k;
  a.out[1] = k_out;
  for (int i = 0; i < 3; ++i) {
    a.si[0][i] = q_strides[i];
    a.so[0][i] = q_out_strides[i];
    a.si[1][i] = H_k > 0 ? k_strides[i] : 0;
    a.so[1][i] = H_k > 0 ? k_out_strides[i] : 0;
  }
  a.H[0] = H_q;
  a.H[1] = H_k;
  a.pos = pos;
  a.pos_axis = pos_strides[0];
  a.pos_batch = pos_strides[1];
  a.tokens = tokens;
  a.L = L;
  a.sign = inverse ? -1.f : 1.f;
  a.rope = *r;
  cudaError_t e = eba::launch_rope(a, d, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTN_OK : cuda_fail(e);
}

int attn_cache_append(const attn_cache_t* cache, const void* k, const long long* k_strides,
                      const void* v, const long long* v_strides, const int* page_table,
                      long long table_stride, int max_pages, const int* seq_lens, int n_seqs,
                      const int* cu_new, int T, const attn_rope_t* rope, const int* pos,
                      long long pos_stride, void* stream) {
  int s = check_cache(cache);
  if (s != ATTN_OK) return s;
  if (!k_strides || !v_strides) return ATTN_ERR_INVALID_ARG;
  if ((s = check_table(page_table, table_stride, max_pages, seq_lens, n_seqs)) != ATTN_OK) return s;
  if (T < 1 || (!cu_new && T != n_seqs)) return ATTN_ERR_INVALID_ARG;
  if ((s = check_ptrs({k, v})) != ATTN_OK) return s;
  if ((s = check_strides(k_strides, 2, 8)) != ATTN_OK) return s;
  if ((s = check_strides(v_strides, 2, 8)) != ATTN_OK) return s;
  if (rope) {
    if ((s = check_rope(*rope, cache->d)) != ATTN_OK) return s;
    if (!pos && rope->n_axes != 1) return ATTN_ERR_INVALID_ARG;
  }
  if (!rows_fit(T, cache->d, cache->H_kv)) return ATTN_ERR_INVALID_ARG;
  int* status = status_word_ptr();
  if (!status) return ATTN_ERR_CUDA;
  eba::AppendArgs a{};
  a.k = k;
  a.v = v;
  a.k_token = k_strides[0];
  a.k_head = k_strides[1];
  a.v_token = v_strides[0];
  a.v_head = v_strides[1];
  a.cache = *cache;
  a.table = page_table;
  a.table_stride = table_stride;
  a.max_pages = max_pages;
  a.lens = seq_lens;
  a.cu_new = cu_new;
  a.n_seqs = n_seqs;
  a.tokens = T;
  a.pos = pos;
  a.pos_axis = pos_stride;
  a.k_inv = 1.f / cache->k_scale;
  a.v_inv = 1.f / cache->v_scale;
  a.status = status;
  if (rope) a.rope = *rope;
  cudaError_t e = eba::launch_append(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTN_OK : cuda_fail(e);
}

size_t attn_decode_workspace_size(int B, int H, int H_kv, int d, int type, long long max_keys) {
  if (B < 1 || H < 1 || H_kv < 1 || H % H_kv != 0 || (d != 64 && d != 128) || max_keys < 1 ||
      (type != ATTN_CACHE_BF16 && type != ATTN_CACHE_E4M3))
    return 0;
  const DecodePlan p = decode_plan(B, H, H_kv, d, max_keys, type);
  return p.ok ? p.bytes : 0;
}

int attn_decode(const attn_cache_t* cache, const void* q, const long long* q_strides,
                const int* page_table, long long table_stride, int max_pages, const int* seq_lens,
                int B, int H, float scale, const attn_rope_t* rope, const int* pos,
                long long pos_stride, void* o, float* lse, void* workspace,
                size_t workspace_bytes, void* stream) {
  int s = check_cache(cache);
  if (s != ATTN_OK) return s;
  if (!q_strides) return ATTN_ERR_INVALID_ARG;
  if ((s = check_table(page_table, table_stride, max_pages, seq_lens, B)) != ATTN_OK) return s;
  if (H < 1 || H % cache->H_kv != 0) return ATTN_ERR_INVALID_ARG;
  if (static_cast<long long>(B) * H >= (1ll << 31)) return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(scale * kLog2e) || !(scale > 0.0f)) return ATTN_ERR_INVALID_ARG;
  if ((s = check_ptrs({q, o, lse})) != ATTN_OK) return s;
  if ((s = check_strides(q_strides, 2, 8)) != ATTN_OK) return s;
  if (rope) {
    if ((s = check_rope(*rope, cache->d)) != ATTN_OK) return s;
    if (!pos && rope->n_axes != 1) return ATTN_ERR_INVALID_ARG;
  }
  const DecodePlan p = decode_plan(B, H, cache->H_kv, cache->d,
                                   static_cast<long long>(max_pages) * cache->page_size, cache->type);
  if (!p.ok) return ATTN_ERR_INVALID_ARG;
  if (p.bytes > 0) {
    if (!workspace || workspace_bytes < p.bytes) return ATTN_ERR_WORKSPACE;
    if (!aligned16(workspace)) return ATTN_ERR_MISALIGNED;
  }
  int* status = status_word_ptr();
  if (!status) return ATTN_ERR_CUDA;
  eba::DecodeArgs a{};
  const int esz = cache->type == ATTN_CACHE_E4M3 ? 1 : 2;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.q_seq = q_strides[0];
  a.q_head = q_strides[1];
  a.k = static_cast<const unsigned char*>(cache->k);
  a.v = static_cast<const unsigned char*>(cache->v);
  for (int i = 0; i < 3; ++i) {
    a.k_strides[i] = cache->k_strides[i] * esz;
    a.v_strides[i] = cache->v_strides[i] * esz;
  }
  a.cache = *cache;
  a.table = page_table;
  a.table_stride = table_stride;
  a.lens = seq_lens;
  a.max_len = p.max_len;
  a.B = B;
  a.H = H;
  a.group = H / cache->H_kv;
  a.rows = p.rows;
  a.blocks = p.blocks;
  a.per_item = p.per_item;
  a.heads = p.heads;
  a.splits = p.splits;
  a.scale_log2 = scale * kLog2e;
  a.o_scale = cache->v_scale;
  a.o = static_cast<__nv_bfloat16*>(o);
  a.lse = lse;
  if (p.bytes > 0) {
    a.cut = static_cast<int2*>(workspace);
    a.part_o = reinterpret_cast<float*>(a.cut + eba::kDecodeCtas);
    a.part_ml = reinterpret_cast<float2*>(a.part_o + p.slots * cache->d);
  }
  a.pos = pos;
  a.pos_axis = pos_stride;
  a.status = status;
  if (rope) a.rope = *rope;
  a.limit_ns = g_wait_limit_ns.load();
  cudaError_t e = eba::launch_decode(a, p.ctas, p.join, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? ATTN_OK : cuda_fail(e);
}

const char* attn_status_string(int status) {
  switch (status) {
    case ATTN_OK: return "ok";
    case ATTN_ERR_INVALID_ARG: return "invalid argument";
    case ATTN_ERR_UNSUPPORTED: return "unsupported configuration";
    case ATTN_ERR_MISALIGNED: return "pointer not 16-byte aligned";
    case ATTN_ERR_CUDA: return "CUDA call failed";
    case ATTN_ERR_TIMEOUT: return "an in-kernel wait timed out";
    case ATTN_ERR_WORKSPACE: return "workspace missing or too small";
    case ATTN_ERR_PAGE: return "a cached length or page is out of range";
    default: return "unknown status";
  }
}

int attn_poll_device_status(void* stream) {
  if (bind_device() < 0) return ATTN_ERR_CUDA;
  cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e);
  int value = 0;
  if ((e = cudaMemcpyFromSymbol(&value, g_status_word, sizeof(int))) != cudaSuccess)
    return cuda_fail(e);
  if (value != 0) {
    const int zero = 0;
    if ((e = cudaMemcpyToSymbol(g_status_word, &zero, sizeof(int))) != cudaSuccess)
      return cuda_fail(e);
  }
  if (value == ATTN_OK || value == ATTN_ERR_TIMEOUT || value == ATTN_ERR_PAGE) return value;
  return ATTN_ERR_CUDA;
}

int attn_last_cuda_error(void) { return t_last_cuda_error; }

unsigned long long attn_set_wait_limit_ns(unsigned long long ns) {
  constexpr unsigned long long kMaxWaitNs = 1ull << 62;  // kept positive as a signed 64-bit value
  return g_wait_limit_ns.exchange(ns == 0 ? kDefaultWaitNs : (ns > kMaxWaitNs ? kMaxWaitNs : ns));
}

}  // extern "C"

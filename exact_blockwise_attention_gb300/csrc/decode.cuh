// Attention of one new token per sequence over a paged key-value cache, split
// over the cache's length and joined; or, with a window, over the last keys of the
// cache and its first ones (attn_decode.cu and attn_decode_window.cu build the two).
//
// For each sequence b and query head h (K/V head g = h / G, n = lens[b] keys):
//   s_j = scale q . k_j,  M = max_j s_j,  O = sum_j e^(s_j - M) v_j / L,
//   L = sum_j e^(s_j - M),  lse = M + ln L;
// over parts c of the keys the same sums join exactly:
//   M = max_c M_c,  L = sum_c e^(M_c - M) L_c,  O = sum_c e^(M_c - M) O_c / L.
//
// Every cached element is read once for up to 16 query heads: 2 flops per element
// and head, far below what the card computes per byte, so the kernel is bound
// by HBM reads. (A larger group walks the cache once for each 16 of its heads, in
// part out of L2: 16 x up to 32000 keys, bf16, 16 heads on one K/V head 41 us and
// 188 MB read, 32 heads 56 us and 282 MB, 64 heads 93 us.)
// Measured on GB300, of the rate of a plain copy (6.79 TB/s):
// 64 ragged sequences of up to 8191 keys, 8 heads of 128 for 32, bf16, 1.1 GB
// 176 us, 94 %; 2 x 36864 keys of 32 heads of 128, 1.2 GB 184 us, 95 %; 8 x up
// to 131071 keys, 4 heads of 128 for 64, e4m3, 0.6 GB 105 us, 86 %; 16 x up to
// 12544 keys of 16 heads of 64, bf16, 0.4 GB 71 us, 86 %, the same in e4m3 44 us,
// 69 % (widening: ALU 40 %). What is left is about
// 4 us until the first keys arrive, 3 us of the join, and that the SMs are not
// equally fast: on equal shares the first CTA is done after 137 us, the median
// after 155 and the last after 169. (Handing out the end of each share to who is
// done first cost more in changes of place than it gained.) What it is built
// around:
//  - The work is the list of all 32 KB tiles of all (sequence, K/V head)
//    items, cut into equal runs, one per CTA (two CTAs per SM): long and short
//    sequences balance without the host knowing the lengths, and a call can be
//    captured and replayed with other lengths. An item cut between CTAs leaves
//    fp32 partials, which the join kernel adds up in the order of the keys.
//  - Short caches and few heads, where latency is what counts: one cluster of
//    up to 8 CTAs per item instead, whose parts are joined through the
//    cluster's shared memory: one launch, no workspace and no list of tiles
//    (333 keys of 8 heads of 128 for 32: 6.2 us, and 5 us less on the host).
//  - Two warps of a CTA load and four compute. The loads (cp.async, 16 bytes a
//    lane) fill a ring of three K and three V slots, across item borders; 96 KB
//    of a CTA's 112 are on their way most of the time. Loads by the computing
//    warps themselves left these waiting for addresses (1.1 GB case 181 us,
//    rows of 128 bytes 85 us), TMA tiles of 16 rows arrived later.
//  - A computing warp owns 4 KB of K and of V of each tile, with its own running
//    maximum and sums; the four warps meet only at an item's end.
//  - Four neighbouring K/V heads are one item where rows are short and there are
//    enough of them: their rows of a token are read together (16 heads of 64,
//    e4m3: 57 -> 44 us).
//  - The products use the 16x8x16 warp matrix instruction with the keys as its
//    16 rows and the G query heads as its 8 columns: S^T = K Q^T, then
//    O^T += V^T P^T, with K and V read from shared memory as they lie there
//    (V transposed by ldmatrix) and P^T made from S^T by an 8x8 register
//    transpose. A 128-row tensor-core tile would be almost empty at these
//    heights, and the matrix pipe is 13 % busy (33 % with e4m3 and 16 heads).
//  - bf16 caches: P is split into two bf16 terms (P = hi + lo to 2^-15), so
//    that its rounding stays far below that of the bf16 output; e4m3 caches:
//    K and V widen exactly to fp16, q is scaled per head by a power of two
//    into fp16's range (exact above 2^-28 of the head's largest element) and P
//    is held as fp16, 2^7 to 2^15 at the running maximum (2^-11 relative down to
//    2^-21 of the largest weight, steps of 2^-31 below). (The e4m3 warp
//    instruction takes K as it is, but is slower: 129 instead of 105 us.)
// Scores, maxima, sums and outputs are fp32 throughout.
#pragma once

#include <cuda_fp16.h>

#include <cfloat>

#include "rope.cuh"

namespace eba {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;             // that compute
constexpr int kBlock = kThreads + 64;             // and the two warps that load
constexpr int kAhead = 2;                         // tiles a page number is fetched ahead of its load
constexpr int kSubKeys = 16;                      // keys of a matrix instruction
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kSlack = 8.f;                     // scores may pass the reference by a factor 2^8
constexpr float kF16Shift = 7.f;                  // e4m3 caches: P's largest value is 2^(8 + 7)

// QUAD: an item is four neighbouring K/V heads, one for each computing warp; else it
// is one head, and the warps share its keys.
template <int D, int NB, bool F8, bool QUAD>
struct Layout {
  static constexpr bool kQuad = QUAD;
  static constexpr int kHeads = QUAD ? kWarps : 1;    // K/V heads of an item
  static constexpr int N = 8 * NB;                    // query heads of a K/V head
  static constexpr int kRow = D * (F8 ? 1 : 2);       // bytes of a cached row
  // A warp's step: 4 KB each of K and V, so that what a step costs besides its
  // bytes is paid once for as many bytes (16 keys a step whatever their size:
  // e4m3, 16 heads, 130 instead of 105 us).
  static constexpr int kSub = kRow == 256 ? 1 : 2;
  static constexpr int kRounds = kRow == 64 ? 2 : 1;  // of kSub sets of keys in a step
  static constexpr int kStepKeys = kSubKeys * kSub * kRounds;
  static constexpr int kTileKeys = kWarps / kHeads * kStepKeys;
  static constexpr int kBoxes = kTileKeys / kSubKeys; // sets of 16 keys
  static constexpr int kStep = kStepKeys * kRow;      // bytes of a warp's K (or V) step
  static constexpr int kTile = kWarps * kStep;        // of a tile
  static constexpr int kStages = 96 * 1024 / (2 * kTile);  // K and V slots of the ring
  static constexpr int kQRow = D + 8;                 // 16-bit elements of a staged query row
  static constexpr int kPassCols = QUAD && D == 128 ? 32 : 64;  // of O, written out at a time
  static constexpr int kPassRow = kPassCols + 4;      // floats; +4: conflict-free column writes
  static constexpr int kOffSum = 2 * kStages * kTile;
  static constexpr int kOffQ = kOffSum + kWarps * 8 * kPassRow * 4;
  static constexpr int kOffMl = kOffQ + kHeads * N * kQRow * 2;    // per warp and row: reference, sum
  static constexpr int kOffQs = kOffMl + kWarps * N * 8;  // per row: score factor
  static constexpr int kOffKeys = kOffQs + kHeads * N * 4;  // per stage and 16 keys: those that count
  static constexpr int kOffBar = (kOffKeys + kStages * kBoxes * 2 + 7) / 8 * 8;  // filled K, V, emptied
  static constexpr int kOffScan = kOffBar + kStages * 32;
  static constexpr int kOffFirst = kOffScan + kWarps * 4;
  static constexpr int kOffAbort = kOffFirst + 20;
  static constexpr int kBytes = kOffAbort + 4;
  static_assert(kTileKeys * kHeads == decode_tile_keys(kRow), "");
};

// 16 bytes; the hint keeps L2 from fetching more than a row (64-byte rows of
// several heads lie side by side, and the others are read by other CTAs).
template <int kRow>
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  if constexpr (kRow == 64)
    asm volatile("cp.async.cg.shared.global.L2::64B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(valid ? 16 : 0)
                 : "memory");
  else
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(valid ? 16 : 0)
                 : "memory");
}
// Arrive on `bar` once this lane's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// An 8x8 matrix of 16-bit elements, one 32-bit register a lane, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
template <bool F8>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if constexpr (F8) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  } else {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
}
// Two e4m3 bytes -> two fp16 (exact).
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
  return h;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

// The largest bf16 strictly below p > 0 (0 for 0), as fp32 bits: what is left of
// p is then positive, and both terms of a weight give an infinite value its sign.
__device__ __forceinline__ uint32_t below(float p) {
  return (max(__float_as_uint(p), 1u) - 1u) & 0xFFFF0000u;
}

// A cluster's shared memory: the address of `addr` in CTA `rank`, loads from it,
// and the barrier that orders one CTA's writes before another's reads.
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ float2 ld_cluster2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// Where 16-byte chunk c of row r lies in a tile of kRow-byte rows: permuted so that
// the 8 rows of a matrix load fall into 8 different bank groups.
template <int kRow>
__device__ __forceinline__ uint32_t tile_offset(int r, int c) {
  if constexpr (kRow >= 128) return static_cast<uint32_t>(r * kRow + ((c ^ (r & 7)) << 4));
  return static_cast<uint32_t>(r * kRow + ((c ^ ((r >> 1) & 3)) << 4));
}

// The barrier of the computing warps.
__device__ __forceinline__ void sync_compute() { named_bar_sync(1, kThreads); }

// e4m3: a lane's four consecutive bytes of K serve the two halves of its register
// operand (elements 0, 1 and 8, 9 of the product's order), so the query's elements
// are staged in that order.
__device__ __forceinline__ int q_place(int e) {
  return (e & ~15) + ((e >> 2) & 3) * 2 + (e & 1) + ((e & 2) ? 8 : 0);
}

// A place in the list of tiles: tile t of nt of sequence b (len keys), head hh
// (K/V head and block of query heads).
struct Cursor {
  int b, hh, t, nt, len;
};

__device__ __forceinline__ int clamp_len(const DecodeArgs& a, int b) {
  const int len = a.lens[b];
  return min(max(len, 0), a.max_len);
}
// Windowed: the tiles of a sequence are those of its sinks [0, sunk), then those of
// its window [low, len), which start at the 16 keys that hold low. sunk <= low: a
// sink within the window counts once.
__device__ __forceinline__ int window_low(const DecodeArgs& a, int len) { return max(len - a.window, 0); }
template <int kTileKeys, bool WINDOW>
__device__ __forceinline__ int tiles_of(const DecodeArgs& a, int len) {
  if constexpr (!WINDOW) return (len + kTileKeys - 1) / kTileKeys;
  const int low = window_low(a, len), sunk = min(a.sinks, low);
  return (sunk + kTileKeys - 1) / kTileKeys + (len - (low & -kSubKeys) + kTileKeys - 1) / kTileKeys;
}
// The keys of a tile: 16s of them from `from` on, of which [low, high) count.
struct TileKeys {
  int from, low, high;
};
template <int kTileKeys, bool WINDOW>
__device__ __forceinline__ TileKeys tile_keys(const DecodeArgs& a, int t, int len) {
  if constexpr (!WINDOW) return {t * kTileKeys, 0, len};
  const int low = window_low(a, len), sunk = min(a.sinks, low);
  const int sink_tiles = (sunk + kTileKeys - 1) / kTileKeys;
  if (t < sink_tiles) return {t * kTileKeys, 0, sunk};
  return {(low & -kSubKeys) + (t - sink_tiles) * kTileKeys, low, len};
}

template <int kTileKeys, bool WINDOW>
__device__ __forceinline__ void advance(Cursor& c, const DecodeArgs& a) {
  if (++c.t < c.nt) return;
  c.t = 0;
  if (++c.hh < a.heads) return;
  c.hh = 0;
  c.nt = 0;
  while (c.nt == 0 && ++c.b < a.B) {
    c.len = clamp_len(a, c.b);
    c.nt = tiles_of<kTileKeys, WINDOW>(a, c.len);
  }
}

// The first tile of CTA i: an equal share of all tiles.
__device__ __forceinline__ int first_tile(int i, int tiles, int ctas) {
  return static_cast<int>(static_cast<long long>(i) * tiles / ctas);
}

// A loading warp (one for K, one for V): runs through the CTA's tiles ahead of the
// computing warps and fills the ring's slots as these empty them. Page numbers wait
// in line behind the card's streaming reads, so they are fetched kAhead tiles early.
// The copies are cp.async, 16 bytes a lane: a key that does not count reads nothing
// and leaves zeros, so that its weight 0 gives 0. (Tiled loads of 16 rows by TMA
// took 5 to 15 % longer here: pages of 16 keys make them small, and one thread
// issues each.)
// WHOLE: the page size is a multiple of 16 keys, so that each 16 lie in one page and
// are looked up once; else each key is looked up by itself.
template <typename L, bool WHOLE, bool WINDOW>
__device__ __forceinline__ void load_tiles(const DecodeArgs& a, const unsigned char* from,
                                           const long long (&strides)[3], int half,
                                           unsigned char* smem, Cursor ld, int tiles,
                                           volatile int* s_abort) {
  constexpr int kStages = L::kStages, kTileKeys = L::kTileKeys, kBoxes = L::kBoxes;
  constexpr int kPer = WHOLE ? 1 : kTileKeys / 32;  // look-ups of a lane and tile
  constexpr int kLanes = L::kRow / 16;              // of a row: 16 bytes each
  constexpr int kRows = 32 / (kLanes * L::kHeads);  // keys of an instruction, for each head
  static_assert(kRows >= 1, "");
  const int lane = threadIdx.x & 31;
  const int c = lane % kLanes, r_lane = lane / (kLanes * L::kHeads);
  const int head_lane = lane / kLanes % L::kHeads;
  const uint32_t ring = smem_u32(smem) + half * L::kTile + head_lane * L::kStep;
  const uint32_t bars = smem_u32(smem + L::kOffBar) + half * 8;
  uint16_t* s_keys = reinterpret_cast<uint16_t*>(smem + L::kOffKeys);
  const DeviceStatus st{a.status, a.limit_ns};
  const unsigned char* at = from + c * 16 + head_lane * strides[2] + (WHOLE ? r_lane * strides[1] : 0);
  Cursor look = ld;
  int look_left = tiles;
  int page_of[kAhead][kPer], slot_of[kAhead][kPer];  // slot -1: no such key
  auto look_up = [&]() {
#pragma unroll
    for (int i = 0; i + 1 < kAhead; ++i)
#pragma unroll
      for (int x = 0; x < kPer; ++x)
        page_of[i][x] = page_of[i + 1][x], slot_of[i][x] = slot_of[i + 1][x];
    const TileKeys tk = tile_keys<kTileKeys, WINDOW>(a, look.t, look.len);
#pragma unroll
    for (int x = 0; x < kPer; ++x) {
      const int in = WHOLE ? lane * kSubKeys : lane + 32 * x;
      const int key = tk.from + in;
      page_of[kAhead - 1][x] = 0;
      slot_of[kAhead - 1][x] = -1;
      // (16 keys looked up at once: the window begins within the first of them at most)
      if (look_left > 0 && in < kTileKeys && key < tk.high && (WHOLE || !WINDOW || key >= tk.low)) {
        const int entry = key / a.cache.page_size;
        slot_of[kAhead - 1][x] = key - entry * a.cache.page_size;
        page_of[kAhead - 1][x] = a.table[look.b * a.table_stride + entry];
      }
    }
    if (--look_left > 0) advance<kTileKeys, WINDOW>(look, a);
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) look_up();

  int stage = 0, lap = 0;
#pragma unroll 1
  for (int i = 0; i < tiles; ++i) {
    const long long head = (L::kQuad ? ld.hh * L::kHeads : ld.hh / a.blocks) * strides[2];
    uint32_t keys[kPer];   // that count: WHOLE of this lane's 16, else of 32
    long long off[kPer];   // of the looked-up rows
#pragma unroll
    for (int x = 0; x < kPer; ++x) {
      const int page = page_of[0][x], slot = slot_of[0][x];
      const bool held = slot >= 0;
      const bool ok = held && static_cast<unsigned>(page) < static_cast<unsigned>(a.cache.n_pages);
      if (held && !ok) atomicCAS(a.status, 0, ATTN_ERR_PAGE);
      off[x] = ok ? page * strides[0] + slot * strides[1] + head : 0;
      if constexpr (WHOLE) {
        const TileKeys tk = tile_keys<kTileKeys, WINDOW>(a, ld.t, ld.len);
        const int key = tk.from + lane * kSubKeys;
        keys[x] = ok ? (1u << min(tk.high - key, kSubKeys)) - 1u : 0u;
        if (WINDOW && key < tk.low) keys[x] &= ~0u << (tk.low - key);
      } else {
        keys[x] = __ballot_sync(0xffffffffu, ok);
      }
    }
    look_up();
    const uint32_t full = bars + stage * 16, empty = full + kStages * 16;
    const uint32_t to = ring + stage * 2 * L::kTile;
    if (lap > 0 && !__all_sync(0xffffffffu, mbar_wait(empty, (lap - 1) & 1, s_abort, st))) break;
    if (half == 0) {
      if (WHOLE) {
        if (lane < kBoxes) s_keys[stage * kBoxes + lane] = static_cast<uint16_t>(keys[0]);
      } else if (lane < 2) {
#pragma unroll
        for (int x = 0; x < kPer; ++x)
          s_keys[stage * kBoxes + 2 * x + lane] = static_cast<uint16_t>(keys[x] >> (16 * lane));
      }
      // The copies' arrives below order the copies alone; the masks are ordinary stores
      // and are released by an ordinary arrive.
      __syncwarp();
      if (lane == 0) mbar_arrive(full);
    }
    if constexpr (WHOLE) {
#pragma unroll
      for (int bx = 0; bx < kBoxes; ++bx) {
        const uint32_t mask = __shfl_sync(0xffffffffu, keys[0], bx);
        const unsigned char* p = at + __shfl_sync(0xffffffffu, off[0], bx);
#pragma unroll
        for (int i = 0; i < kSubKeys / kRows; ++i) {
          const int r = i * kRows + r_lane;
          cp_async16<L::kRow>(to + tile_offset<L::kRow>(bx * kSubKeys + r, c), p, (mask >> r) & 1);
          p += kRows * strides[1];
        }
      }
    } else {
#pragma unroll
      for (int x = 0; x < kPer; ++x)
#pragma unroll
        for (int i = 0; i < 32 / kRows; ++i) {
          const int r = i * kRows + r_lane;
          const unsigned char* p = at + __shfl_sync(0xffffffffu, off[x], r);
          cp_async16<L::kRow>(to + tile_offset<L::kRow>(32 * x + r, c), p, (keys[x] >> r) & 1);
        }
    }
    cp_async_arrive(full);
    if (i + 1 < tiles) advance<kTileKeys, WINDOW>(ld, a);
    if (++stage == kStages) stage = 0, ++lap;
  }
  cp_async_wait_all();  // also after a wait that gave up
}

// The run that tile t is in: the last one that does not begin behind it.
__device__ __forceinline__ int run_of(int t, int tiles, int ctas) {
  int i = static_cast<int>(static_cast<long long>(t) * ctas / tiles);
  while (i + 1 < ctas && first_tile(i + 1, tiles, ctas) <= t) ++i;
  return i;
}

template <int D, int NB, bool F8, bool WHOLE, bool QUAD, bool WINDOW>
__global__ void __launch_bounds__(kBlock, 2)
    decode_kernel(const __grid_constant__ DecodeArgs a) {
  using L = Layout<D, NB, F8, QUAD>;
  constexpr int N = L::N;
  constexpr int kStages = L::kStages;
  constexpr int kPassCols = L::kPassCols, kPassRow = L::kPassRow;
  constexpr int kSub = L::kSub, kTileKeys = L::kTileKeys;
  constexpr uint32_t kAllKeys = kSub == 1 ? 0xffffu : 0xffffffffu;
  constexpr int kKSteps = D / 16;  // 16-element steps of a product over d; 16-row tiles of V^T
  extern __shared__ __align__(128) unsigned char smem[];
  int* s_scan = reinterpret_cast<int*>(smem + L::kOffScan);
  Cursor& s_first = *reinterpret_cast<Cursor*>(smem + L::kOffFirst);
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + L::kOffAbort);
  pdl_launch_dependents();
  const uint32_t bars = smem_u32(smem + L::kOffBar);
  // filled: by the copies of 32 lanes, K's also by the masks' arrive; emptied: by 4 warps
  if (threadIdx.x < 4 * kStages)
    mbar_init(bars + threadIdx.x * 8,
              threadIdx.x >= 2 * kStages ? kWarps : threadIdx.x % 2 == 0 ? 33 : 32);
  if (threadIdx.x == 0) *s_abort = 0;
  fence_mbar_init();
  pdl_wait();

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int j4 = lane & 3, u8 = lane >> 2;
  const int cta = blockIdx.x;

  int r0, r1;          // this CTA's tiles
  int G = 1, tiles = 0;  // runs the list of all tiles is cut into, and its length
  if (a.splits) {
    // ---- short caches: one cluster of a.splits CTAs per item ----
    const int it = cta / a.splits, rank = cta - it * a.splits;
    const int b = it / a.heads, raw = a.lens[b];
    const int len = min(max(raw, 0), a.max_len), nt = tiles_of<kTileKeys, WINDOW>(a, len);
    if (tid == 0) {
      if (raw != len) atomicCAS(a.status, 0, ATTN_ERR_PAGE);
      s_first = Cursor{b, it - b * a.heads, first_tile(rank, nt, a.splits), nt, len};
    }
    r0 = first_tile(rank, nt, a.splits);
    r1 = first_tile(rank + 1, nt, a.splits);
  } else {
    // ---- the list of tiles: each thread counts a run of sequences ----
    const int per = (a.B + kThreads - 1) / kThreads;
    const int b0 = min(tid * per, a.B), b1 = tid < kThreads ? min(b0 + per, a.B) : b0;
    int mine = 0;
    for (int b = b0; b < b1; ++b) {
      const int raw = a.lens[b];
      if (cta == 0 && (raw < 0 || raw > a.max_len)) atomicCAS(a.status, 0, ATTN_ERR_PAGE);
      mine += tiles_of<kTileKeys, WINDOW>(a, clamp_len(a, b)) * a.heads;
    }
    int incl = mine;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, incl, m);
      if (lane >= m) incl += o;
    }
    if (lane == 31 && warp < kWarps) s_scan[warp] = incl;
    __syncthreads();
    int before = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      before += w < warp ? s_scan[w] : 0;
      tiles += s_scan[w];
    }
    // no run is empty: with fewer tiles than CTAs the last CTAs have none
    G = max(1, min(static_cast<int>(gridDim.x), tiles));
    r0 = cta < G ? first_tile(cta, tiles, G) : tiles;
    r1 = cta < G ? first_tile(cta + 1, tiles, G) : tiles;
    {
      int at = before + incl - mine;  // first tile of this thread's sequences
      if (r0 < r1 && r0 >= at && r0 < at + mine) {
        for (int b = b0; b < b1; ++b) {
          const int len = clamp_len(a, b), nt = tiles_of<kTileKeys, WINDOW>(a, len);
          if (r0 < at + nt * a.heads) {
            const int in = r0 - at;
            s_first = Cursor{b, in / nt, in % nt, nt, len};
            break;
          }
          at += nt * a.heads;
        }
      }
    }
    // Sequences without keys: O = 0, lse = -inf.
    for (int b = cta; b < a.B; b += gridDim.x) {
      if (clamp_len(a, b) > 0) continue;
      for (int x = tid; x < a.H * D / 8; x += kBlock)
        *reinterpret_cast<uint4*>(a.o + static_cast<long long>(b) * a.H * D + x * 8) =
            make_uint4(0, 0, 0, 0);
      for (int h = tid; h < a.H; h += kBlock) a.lse[static_cast<long long>(b) * a.H + h] = -INFINITY;
    }
  }
  __syncthreads();
  if (!a.splits && r0 >= r1) {
    if (a.cut && tid == 0) a.cut[cta] = make_int2(0, 0);
    return;
  }

  float* s_sum = reinterpret_cast<float*>(smem + L::kOffSum);
  uint16_t* s_q = reinterpret_cast<uint16_t*>(smem + L::kOffQ);
  float2* s_ml = reinterpret_cast<float2*>(smem + L::kOffMl);
  // a split item's part, in the ring once all loads are used: [N][D], [N]
  float* s_part = reinterpret_cast<float*>(smem);
  float2* s_part_ml = reinterpret_cast<float2*>(smem + N * D * 4);
  float* s_qs = reinterpret_cast<float*>(smem + L::kOffQs);

  if (warp >= kWarps) {
    const bool keys = warp == kWarps;
    if (r0 < r1)
      load_tiles<L, WHOLE, WINDOW>(a, keys ? a.k : a.v, keys ? a.k_strides : a.v_strides, keys ? 0 : 1, smem,
                           s_first, r1 - r0, s_abort);
    if (!QUAD && (a.splits > 1 || s_first.nt == 0)) {  // the cluster's barriers below
      cluster_sync();
      cluster_sync();
    }
    return;
  }

  // ---- the query heads of an item: staged for all warps, QUAD: each its own ----
  // Row n: query head g G + blk N + n; rotated where asked, rounded to bf16
  // (the same value the rotation kernel gives); zero behind the group.
  if (QUAD) {
    s_q += warp * N * L::kQRow;
    s_qs += warp * N;
  }
  auto sync_staged = [&]() {
    if (QUAD) __syncwarp(); else sync_compute();
  };
  auto stage_q = [&](const Cursor& c) {
    constexpr int kPer = (QUAD ? 32 : kThreads) / N;  // threads of a row
    constexpr int kPairs = D / 2 / kPer;              // pairs of elements of a thread
    const int n = (QUAD ? lane : tid) / kPer, i = (QUAD ? lane : tid) % kPer;
    const int g = QUAD ? c.hh * L::kHeads + warp : c.hh / a.blocks;
    const int hg = (QUAD ? 0 : c.hh - g * a.blocks) * N + n;
    const __nv_bfloat16* q = a.q + c.b * a.q_seq + (static_cast<long long>(g) * a.group + hg) * a.q_head;
    const int P = a.rope.n_pairs;
    auto places = [&](int pair, int& x, int& y) {
      const bool half = pair < P && !a.rope.interleaved;
      x = half ? pair : 2 * pair;
      y = half ? pair + P : 2 * pair + 1;
    };
    uint32_t both[kPairs];
    float top = 0.f;
#pragma unroll
    for (int p = 0; p < kPairs; ++p) {
      const int pair = i * kPairs + p;
      int ox, oy;
      places(pair, ox, oy);
      float x = hg < a.group ? __bfloat162float(q[ox]) : 0.f;
      float y = hg < a.group ? __bfloat162float(q[oy]) : 0.f;
      if (pair < P) {
        const int pos = a.pos ? a.pos[a.rope.axis[pair] * a.pos_axis + c.b] : c.len - 1;
        float cs, sn;
        rope_cs(pos, a.rope.turns[pair], 1.f, cs, sn);
        rope_turn(x, y, cs, sn);
      }
      both[p] = pack_bf16(x, y);
      x = fabsf(bf16lo_f32(both[p])), y = fabsf(bf16hi_f32(both[p]));
      top = fmaxf(top, fmaxf(x < INFINITY ? x : 0.f, y < INFINITY ? y : 0.f));
    }
    float up = 1.f, down = 1.f;
    if constexpr (F8) {
#pragma unroll
      for (int m = kPer / 2; m > 0; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
      // up = 2^e puts the head's largest element into [2^13, 2^14). e is at least
      // 13 - 127, and at most 126, so that 2^-e is a normal float too: that leaves
      // smaller heads below 2^13, where fp16 still holds all bits that bf16 has there
      // (its smallest number, 2^-133, becomes 2^-7).
      const int floor_log2 = static_cast<int>(__float_as_uint(top) >> 23) - 127;
      const int e = top > 0.f ? min(13 - floor_log2, 126) : 0;
      up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
      down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    }
    // The keys' scale times a power of two is exact. A factor beyond fp32's largest number
    // stays finite, so that scores of 0 are 0.
    if (i == 0) s_qs[n] = fminf(a.scale_log2 * (a.cache.k_scale * down), FLT_MAX);
#pragma unroll
    for (int p = 0; p < kPairs; ++p) {
      int ox, oy;
      places(i * kPairs + p, ox, oy);
      const float x = bf16lo_f32(both[p]) * up, y = bf16hi_f32(both[p]) * up;
      s_q[n * L::kQRow + (F8 ? q_place(ox) : ox)] =
          F8 ? __half_as_ushort(__float2half_rn(x)) : static_cast<uint16_t>(both[p]);
      s_q[n * L::kQRow + (F8 ? q_place(oy) : oy)] =
          F8 ? __half_as_ushort(__float2half_rn(y)) : static_cast<uint16_t>(both[p] >> 16);
    }
  };

  // The query as the product's column operand: registers for one set of columns;
  // two sets would not fit the 168 registers that 12 warps leave each, and are
  // read in every step.
  uint32_t qf[NB == 1 ? kKSteps / 2 : 1][4];
  auto load_q = [&](uint32_t (&f)[4], int nb, int k) {  // of steps k and k + 1
    ldmatrix4(f, smem_u32(s_q + (nb * 8 + (lane & 7)) * L::kQRow + (2 * k + (lane >> 3)) * 8));
  };
  float qs[NB][2];              // score factor of this lane's two columns
  float o[NB][kKSteps][4];
  float top[NB][2], sum[NB][2];
  auto begin_item = [&]() {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int k = 0; k < kKSteps; ++k) {
        if (NB == 1 && k % 2 == 0) load_q(qf[k / 2], 0, k);
#pragma unroll
        for (int x = 0; x < 4; ++x) o[nb][k][x] = 0.f;
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        qs[nb][x] = s_qs[nb * 8 + 2 * j4 + x];
        top[nb][x] = -INFINITY;
        sum[nb][x] = 0.f;
      }
    }
  };

  Cursor cur = s_first;
  int t_begin = cur.t;        // first tile of the item in this run
  bool first_item = true;
  if (r0 < r1) {
    stage_q(cur);
    sync_staged();
    begin_item();
  }

  // A wait that gives up is recorded and ends all waits of the CTA; its warps still
  // meet at every barrier, and what they write is undefined.
  const DeviceStatus st{a.status, a.limit_ns};
  bool live = true;
  auto wait_filled = [&](uint32_t bar, uint32_t parity) {
    if (live) live = __all_sync(0xffffffffu, mbar_wait(bar, parity, s_abort, st));
  };
  int stage = 0;
  uint32_t parity = 0;
#pragma unroll 1
  for (int tile = r0; tile < r1; ++tile) {
    const uint32_t kt = smem_u32(smem) + stage * 2 * L::kTile + warp * L::kStep, vt = kt + L::kTile;
    const uint32_t full = bars + stage * 16, empty = full + kStages * 16;  // K's; V's 8 behind
    wait_filled(full, parity);
#pragma unroll 1
    for (int round = 0; round < L::kRounds; ++round) {
      uint32_t mask;  // the keys that count
      {
        const unsigned char* at =
            smem + L::kOffKeys +
            (stage * L::kBoxes + ((QUAD ? 0 : warp * L::kRounds) + round) * kSub) * 2;
        mask = kSub == 1 ? *reinterpret_cast<const uint16_t*>(at) : *reinterpret_cast<const uint32_t*>(at);
      }
      // S^T = K Q^T: two chains, of the two halves of d or of two sets of keys
      float s[NB][2][4];
      if (mask) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int x = 0; x < 4; ++x) s[nb][0][x] = s[nb][1][x] = 0.f;
#pragma unroll
        for (int k = 0; k < kKSteps; k += 2) {
          uint32_t q[NB][4];
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            if constexpr (NB == 1) {
#pragma unroll
              for (int x = 0; x < 4; ++x) q[nb][x] = qf[k / 2][x];
            } else {
              load_q(q[nb], nb, k);
            }
          }
#pragma unroll
          for (int sub = 0; sub < kSub; ++sub) {
            const int row = (round * kSub + sub) * kSubKeys + (lane & 15);
            if constexpr (F8) {
              uint32_t r[4];
              ldmatrix4(r, kt + tile_offset<L::kRow>(row, k + (lane >> 4)));
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const uint32_t lo = r[2 * x], hi = r[2 * x + 1];
                const uint32_t f[4] = {e4m3x2_f16x2(lo), e4m3x2_f16x2(hi), e4m3x2_f16x2(lo >> 16),
                                       e4m3x2_f16x2(hi >> 16)};
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
                  mma16816<true>(s[nb][kSub == 1 ? x : sub], f, q[nb][2 * x], q[nb][2 * x + 1]);
              }
            } else {
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                uint32_t r[4];
                ldmatrix4(r, kt + tile_offset<L::kRow>(row, 2 * (k + x) + (lane >> 4)));
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
                  mma16816<false>(s[nb][kSub == 1 ? x : sub], r, q[nb][2 * x], q[nb][2 * x + 1]);
              }
            }
          }
        }
      }
      if (round == 0) wait_filled(full + 8, parity);  // V's reads overlap the softmax
      if (round + 1 == L::kRounds) {
        __syncwarp();  // all lanes have read the masks and are done with K
        if (lane == 0) mbar_arrive(empty);
      }
      uint32_t ph[kSub][NB][2], pl[kSub][NB][2];
      if (mask) {
        // online softmax; element x of a lane: key u8 + 8 (x / 2), column 2 j4 + x % 2
        float v[NB][kSub][4];
        bool grew = false;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
          for (int sub = 0; sub < kSub; ++sub) {
#pragma unroll
            for (int x = 0; x < 4; ++x)
              v[nb][sub][x] = (kSub == 1 ? s[nb][0][x] + s[nb][1][x] : s[nb][sub][x]) * qs[nb][x & 1];
            if (mask != kAllKeys) {
#pragma unroll
              for (int x = 0; x < 4; ++x)
                if (!((mask >> (sub * kSubKeys + u8 + 8 * (x >> 1))) & 1)) v[nb][sub][x] = -INFINITY;
            }
#pragma unroll
            for (int x = 0; x < 2; ++x)
              grew |= fmaxf(v[nb][sub][x], v[nb][sub][x + 2]) > top[nb][x] + kSlack;
          }
        }
        // The reference the weights are relative to follows the maximum only when
        // that has grown by more than kSlack: one vote a step instead of a
        // maximum over the lanes and a rescaled output.
        if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              float to = fmaxf(v[nb][0][x], v[nb][0][x + 2]);
              if (kSub == 2) to = fmaxf(to, fmaxf(v[nb][kSub - 1][x], v[nb][kSub - 1][x + 2]));
#pragma unroll
              for (int m = 4; m < 32; m <<= 1) to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, m));
              to = fmaxf(to, top[nb][x]);
              // -inf to -inf (a column whose scores are all -inf) keeps its zeros
              const float f = to == top[nb][x] ? 1.f : ex2_approx(top[nb][x] - to);
              top[nb][x] = to;
              sum[nb][x] *= f;
#pragma unroll
              for (int k = 0; k < kKSteps; ++k) {
                o[nb][k][x] *= f;
                o[nb][k][x + 2] *= f;
              }
            }
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          float ref[2];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            ref[x] = top[nb][x] == -INFINITY ? 0.f : top[nb][x];
            if (F8) ref[x] -= kF16Shift;
          }
#pragma unroll
          for (int sub = 0; sub < kSub; ++sub) {
            float p[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              p[x] = ex2_approx(v[nb][sub][x] - ref[x & 1]);
              sum[nb][x & 1] += p[x];
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              if constexpr (F8) {
                ph[sub][nb][x] = transpose8(pack_f16(p[2 * x], p[2 * x + 1]));
              } else {
                const uint32_t h0 = below(p[2 * x]), h1 = below(p[2 * x + 1]);
                ph[sub][nb][x] = transpose8(__byte_perm(h0, h1, 0x7632));
                pl[sub][nb][x] = transpose8(pack_bf16(p[2 * x] - __uint_as_float(h0),
                                                      p[2 * x + 1] - __uint_as_float(h1)));
              }
            }
          }
        }
        // O^T += V^T P^T
#pragma unroll
        for (int sub = 0; sub < kSub; ++sub) {
          const int set = (round * kSub + sub) * kSubKeys;  // its first row
          if constexpr (F8) {
            // 16-bit units of V hold two columns of one key: after the transposing
            // load a register holds columns 2 u8, 2 u8 + 1 of keys 2 j4, 2 j4 + 1,
            // and rows u8 and u8 + 8 of the product stand for those two columns
#pragma unroll
            for (int k = 0; k < kKSteps; k += 2) {
              uint32_t r[4];
              ldmatrix4_trans(r, vt + tile_offset<L::kRow>(set + (lane & 15), k + (lane >> 4)));
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const uint32_t w0 = __byte_perm(r[2 * x], 0, 0x3120);
                const uint32_t w1 = __byte_perm(r[2 * x + 1], 0, 0x3120);
                const uint32_t f[4] = {e4m3x2_f16x2(w0), e4m3x2_f16x2(w0 >> 16), e4m3x2_f16x2(w1),
                                       e4m3x2_f16x2(w1 >> 16)};
#pragma unroll
                for (int nb = 0; nb < NB; ++nb)
                  mma16816<true>(o[nb][k + x], f, ph[sub][nb][0], ph[sub][nb][1]);
              }
            }
          } else {
            const int vr = set + (lane & 7) + ((lane >> 4) << 3), vc = (lane >> 3) & 1;
#pragma unroll
            for (int k = 0; k < kKSteps; ++k) {
              uint32_t r[4];
              ldmatrix4_trans(r, vt + tile_offset<L::kRow>(vr, 2 * k + vc));
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) {
                mma16816<false>(o[nb][k], r, ph[sub][nb][0], ph[sub][nb][1]);
                mma16816<false>(o[nb][k], r, pl[sub][nb][0], pl[sub][nb][1]);
              }
            }
          }
        }
      }
    }
    __syncwarp();  // all lanes are done with V
    if (lane == 0) mbar_arrive(empty + 8);
    if (++stage == kStages) stage = 0, parity ^= 1;

    const bool item_done = cur.t + 1 == cur.nt;
    if (item_done || tile + 1 == r1) {
      // ---- the item's end, or the run's: join the four warps, or write each's head ----
      const bool whole = t_begin == 0 && item_done;
      const Cursor done = cur;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float l = sum[nb][x];
#pragma unroll
          for (int m = 4; m < 32; m <<= 1) l += __shfl_xor_sync(0xffffffffu, l, m);
          // the reference its weights are relative to; -inf: no weight at all
          float ref = top[nb][x] == -INFINITY ? 0.f : top[nb][x];
          if (F8) ref -= kF16Shift;
          if (top[nb][x] == -INFINITY && l == 0.f) ref = -INFINITY;
          top[nb][x] = ref;
          sum[nb][x] = l;
          if (!QUAD && u8 == 0) s_ml[warp * N + nb * 8 + 2 * j4 + x] = make_float2(ref, l);
        }
      if (!QUAD) sync_compute();
      const bool more = tile + 1 < r1;
      if (more) {
        advance<kTileKeys, WINDOW>(cur, a);
        stage_q(cur);  // every warp holds the old query in registers
      }
      const int part = 2 * cta + (first_item ? 0 : 1);
      // O's columns [c0, c0 + kPassCols) of the warp's rows into its own part of s_sum
      auto put = [&](int nb, int c0, const float (&f)[2]) {
        float* to = s_sum + warp * 8 * kPassRow;
#pragma unroll
        for (int k = 0; k < kPassCols / 16; ++k)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int col = F8 ? k * 16 + 2 * u8 + (x >> 1) : k * 16 + u8 + 8 * (x >> 1);
            to[(2 * j4 + (x & 1)) * kPassRow + col] = o[nb][c0 / 16 + k][x] * f[x & 1];
          }
      };
      if constexpr (QUAD) {
        const int g = done.hh * L::kHeads + warp;
        const long long head0 = static_cast<long long>(done.b) * a.H + g * a.group;
        const long long part0 = (static_cast<long long>(part) * L::kHeads + warp) * N;
        float f[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int row = 2 * j4 + x;
          const float M = top[0][x], l = sum[0][x];
          f[x] = !whole ? 1.f : M == -INFINITY ? 0.f : a.o_scale / l;
          if (u8 == 0 && !whole) a.part_ml[part0 + row] = make_float2(M, l);
          if (u8 == 0 && whole && row < a.group)
            a.lse[head0 + row] = M == -INFINITY ? -INFINITY : (M + lg2_approx(l)) * kLn2;
        }
        constexpr int kCols = kPassCols / 4;  // of a lane
        const int row = lane >> 2, c4 = (lane & 3) * kCols;
#pragma unroll
        for (int c0 = 0; c0 < D; c0 += kPassCols) {
          put(0, c0, f);
          __syncwarp();
          const float* y = s_sum + (warp * 8 + row) * kPassRow + c4;
#pragma unroll
          for (int x = 0; x < kCols; x += 4) {
            const float4 v = *reinterpret_cast<const float4*>(y + x);
            if (!whole)
              *reinterpret_cast<float4*>(a.part_o + (part0 + row) * D + c0 + c4 + x) = v;
            else if (row < a.group)
              *reinterpret_cast<uint2*>(a.o + (head0 + row) * D + c0 + c4 + x) =
                  make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
          }
          __syncwarp();
        }
      } else {
        const int g = done.hh / a.blocks, blk = done.hh - g * a.blocks;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          float f[2];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_ml[w * N + nb * 8 + 2 * j4 + x].x);
            f[x] = top[nb][x] == -INFINITY ? 0.f : ex2_approx(top[nb][x] - M);
          }
          constexpr int kCols = kPassCols / 16;  // of a thread in the sum below
          const int row = tid >> 4, c4 = (tid & 15) * kCols;
          float M = -INFINITY, l = 0.f;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_ml[w * N + nb * 8 + row].x);
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float2 ml = s_ml[w * N + nb * 8 + row];
            l += ml.x == -INFINITY ? 0.f : ml.y * ex2_approx(ml.x - M);
          }
          const int hg = blk * N + nb * 8 + row;
          const long long head = static_cast<long long>(done.b) * a.H + g * a.group + hg;
#pragma unroll
          for (int c0 = 0; c0 < D; c0 += kPassCols) {
            put(nb, c0, f);
            sync_compute();
            float v[kCols] = {};
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
              const float* y = s_sum + (w * 8 + row) * kPassRow + c4;
#pragma unroll
              for (int x = 0; x < kCols; x += 2) {
                const float2 two = *reinterpret_cast<const float2*>(y + x);
                v[x] += two.x, v[x + 1] += two.y;
              }
            }
            if (whole && a.splits <= 1) {
              if (hg < a.group) {
                const float f = M == -INFINITY ? 0.f : a.o_scale / l;
#pragma unroll
                for (int x = 0; x < kCols; x += 2)
                  *reinterpret_cast<uint32_t*>(a.o + head * D + c0 + c4 + x) =
                      pack_bf16(v[x] * f, v[x + 1] * f);
              }
            } else {
              float* to = a.splits > 1 ? s_part + (nb * 8 + row) * D
                                       : a.part_o + (static_cast<long long>(part) * N + nb * 8 + row) * D;
#pragma unroll
              for (int x = 0; x < kCols; x += 2)
                *reinterpret_cast<float2*>(to + c0 + c4 + x) = make_float2(v[x], v[x + 1]);
            }
            sync_compute();
          }
          if ((tid & 15) == 0) {
            if (a.splits > 1)
              s_part_ml[nb * 8 + row] = make_float2(M, l);
            else if (!whole)
              a.part_ml[static_cast<long long>(part) * N + nb * 8 + row] = make_float2(M, l);
            else if (hg < a.group)
              a.lse[head] = M == -INFINITY ? -INFINITY : (M + lg2_approx(l)) * kLn2;
          }
        }
      }
      // What the join kernel needs: the item that this CTA's run ends in the middle of,
      // if the item has its first tile here or covers the whole run.
      if (a.cut && tid == 0 && tile + 1 == r1) {
        int2 cut = make_int2(0, 0);
        if (!item_done && (t_begin == 0 || first_item)) {
          const int t0 = tile - done.t, t1 = t0 + done.nt;  // the item's tiles
          const int c0 = run_of(t0, tiles, G), parts = run_of(t1 - 1, tiles, G) - c0 + 1;
          const int slot = first_tile(c0, tiles, G) == t0 ? 0 : 1;  // of its first part in c0
          cut = make_int2(done.b * a.heads + done.hh, (parts << 16) | ((cta - c0) << 1) | slot);
        }
        a.cut[cta] = cut;
      }
      first_item = false;
      t_begin = 0;
      if (more) {
        if (QUAD) __syncwarp();  // (else the sums' barriers lie between)
        begin_item();
      }
    } else {
      ++cur.t;
    }
  }
  if (!QUAD && (a.splits > 1 || s_first.nt == 0)) {
    // ---- join the cluster's parts, or write an item without keys ----
    const int g = s_first.hh / a.blocks, blk = s_first.hh - g * a.blocks;
    const int rank = cta % a.splits;
    if (r0 >= r1)
      for (int n = tid; n < N; n += kThreads) s_part_ml[n] = make_float2(-INFINITY, 0.f);
    cluster_sync();
    for (int x = rank * kThreads + tid; x < N * D / 4; x += a.splits * kThreads) {
      const int n = x / (D / 4), hg = blk * N + n;
      if (hg >= a.group) continue;
      const uint32_t ml_at = smem_u32(s_part_ml + n), o_at = smem_u32(s_part) + x * 16;
      float M = -INFINITY, l = 0.f;
      for (int w = 0; w < a.splits; ++w) M = fmaxf(M, ld_cluster2(map_rank(ml_at, w)).x);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int w = 0; w < a.splits; ++w) {
        const float2 ml = ld_cluster2(map_rank(ml_at, w));
        if (ml.x == -INFINITY) continue;  // no weight, or no keys and nothing written
        const float f = ex2_approx(ml.x - M);
        const float4 y = ld_cluster4(map_rank(o_at, w));
        l += ml.y * f;
        v.x += y.x * f, v.y += y.y * f, v.z += y.z * f, v.w += y.w * f;
      }
      const long long head = static_cast<long long>(s_first.b) * a.H + g * a.group + hg;
      const float f = M == -INFINITY ? 0.f : a.o_scale / l;
      *reinterpret_cast<uint2*>(a.o + head * D + x % (D / 4) * 4) =
          make_uint2(pack_bf16(v.x * f, v.y * f), pack_bf16(v.z * f, v.w * f));
      if (x % (D / 4) == 0) a.lse[head] = M == -INFINITY ? -INFINITY : (M + lg2_approx(l)) * kLn2;
    }
    cluster_sync();  // the parts stay until all have read them
  }
}

// Items cut between CTAs: their parts are added up in the order of the keys. What
// that costs is the latency of three loads in a row (the cut, the parts, the output)
// and the CTAs that find nothing to do, so there is one CTA for each run (and 8 rows
// of an item): few parts, and the one whose run the item begins in takes a row a
// warp; many, and the first 8 whose runs the item covers take a row each, with all
// their warps. A warp has the loads of 8 parts under way.
constexpr int kJoinWarps = 8, kDeep = 8, kFewParts = 16;
template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps)
    decode_join_kernel(const __grid_constant__ DecodeArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  constexpr int kVec = D / 32;  // columns of a lane
  __shared__ float s_o[kJoinWarps][D];
  __shared__ float2 s_ml[kJoinWarps];
  const int2 cut = a.cut[blockIdx.x];
  const int parts = cut.y >> 16, rank = (cut.y >> 1) & 0x7fff;
  const bool few = parts <= kFewParts;
  if (parts == 0 || rank >= (few ? 1 : kJoinWarps)) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = blockIdx.y * kJoinWarps + (few ? warp : rank);  // row of the item
  const int b = cut.x / a.heads, hh = cut.x - b * a.heads;
  // its query head: of one of the item's K/V heads, or of a block of one head's group
  const int g = a.per_item > 1 ? hh * a.per_item + n / a.rows : hh / a.blocks;
  const int hg = a.per_item > 1 ? n % a.rows : hh % a.blocks * a.rows + n;
  if (hg >= a.group) return;  // (few: a warp of its own; else all warps alike)
  const int c0 = blockIdx.x - rank, N = a.rows * a.per_item;
  float M = -INFINITY, l = 0.f;
  float o[kVec] = {};
  const int step = few ? 1 : kJoinWarps;
  for (int p0 = few ? 0 : warp; p0 < parts; p0 += step * kDeep) {
    float2 ml[kDeep];
    float v[kDeep][kVec];
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      const int p = p0 + u * step;
      if (p >= parts) {
        ml[u] = make_float2(-INFINITY, 0.f);
        continue;
      }
      // part p in the first slot of the p-th CTA after c0, part 0 as recorded
      const long long row = static_cast<long long>(2 * (c0 + p) + (p == 0 ? cut.y & 1 : 0)) * N + n;
      ml[u] = a.part_ml[row];
      const float* from = a.part_o + row * D + lane * kVec;
      if constexpr (kVec == 4) {
        const float4 y = *reinterpret_cast<const float4*>(from);
        v[u][0] = y.x, v[u][1] = y.y, v[u][2] = y.z, v[u][3] = y.w;
      } else {
        const float2 y = *reinterpret_cast<const float2*>(from);
        v[u][0] = y.x, v[u][1] = y.y;
      }
    }
    float to = M;
#pragma unroll
    for (int u = 0; u < kDeep; ++u) to = fmaxf(to, ml[u].x);
    if (to == -INFINITY) continue;  // no weight so far
    const float f = M == -INFINITY ? 0.f : ex2_approx(M - to);
    M = to;
    l *= f;
#pragma unroll
    for (int x = 0; x < kVec; ++x) o[x] *= f;
#pragma unroll
    for (int u = 0; u < kDeep; ++u) {
      if (ml[u].x == -INFINITY) continue;
      const float w = ex2_approx(ml[u].x - to);
      l += ml[u].y * w;
#pragma unroll
      for (int x = 0; x < kVec; ++x) o[x] += v[u][x] * w;
    }
  }
  const long long head = static_cast<long long>(b) * a.H + static_cast<long long>(g) * a.group + hg;
  if (few) {
    const float f = M == -INFINITY ? 0.f : a.o_scale / l;
#pragma unroll
    for (int x = 0; x < kVec; x += 2)
      *reinterpret_cast<uint32_t*>(a.o + head * D + lane * kVec + x) = pack_bf16(o[x] * f, o[x + 1] * f);
    if (lane == 0) a.lse[head] = M == -INFINITY ? -INFINITY : (M + lg2_approx(l)) * kLn2;
    return;
  }
  if (lane == 0) s_ml[warp] = make_float2(M, l);
#pragma unroll
  for (int x = 0; x < kVec; ++x) s_o[warp][lane * kVec + x] = o[x];
  __syncthreads();
  if (threadIdx.x >= D) return;
  M = -INFINITY;
  l = 0.f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) M = fmaxf(M, s_ml[w].x);
  float v = 0.f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) {
    if (s_ml[w].x == -INFINITY) continue;
    const float f = ex2_approx(s_ml[w].x - M);
    l += s_ml[w].y * f;
    v += s_o[w][threadIdx.x] * f;
  }
  const float f = M == -INFINITY ? 0.f : a.o_scale / l;
  a.o[head * D + threadIdx.x] = __float2bfloat16_rn(v * f);
  if (threadIdx.x == 0) a.lse[head] = M == -INFINITY ? -INFINITY : (M + lg2_approx(l)) * kLn2;
}

template <int D, int NB, bool F8, bool QUAD, bool WINDOW>
cudaError_t launch_decode_t(const DecodeArgs& a, int ctas, bool join, cudaStream_t stream) {
  using L = Layout<D, NB, F8, QUAD>;
  static_assert(L::kBytes <= 113 * 1024, "two CTAs share an SM's shared memory");
  auto kern = a.cache.page_size % kSubKeys == 0 ? decode_kernel<D, NB, F8, true, QUAD, WINDOW>
                                                : decode_kernel<D, NB, F8, false, QUAD, WINDOW>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kBlock);
  cfg.dynamicSmemBytes = L::kBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {static_cast<unsigned>(a.splits), 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = a.splits > 1 ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, kern, a);
  if (e != cudaSuccess || !join) return e;
  return launch_pdl(decode_join_kernel<D>, dim3(ctas, a.rows * a.per_item / kJoinWarps),
                    dim3(32 * kJoinWarps), 0, stream, a);
}

template <bool WINDOW>
cudaError_t launch_decode_any(const DecodeArgs& a, int ctas, bool join, cudaStream_t stream) {
  const bool f8 = a.cache.type == ATTN_CACHE_E4M3, two = a.rows == 16, quad = a.per_item > 1;
  if (a.cache.d == 64) {
    if (f8)
      return quad  ? launch_decode_t<64, 1, true, true, WINDOW>(a, ctas, join, stream)
             : two ? launch_decode_t<64, 2, true, false, WINDOW>(a, ctas, join, stream)
                   : launch_decode_t<64, 1, true, false, WINDOW>(a, ctas, join, stream);
    return quad  ? launch_decode_t<64, 1, false, true, WINDOW>(a, ctas, join, stream)
           : two ? launch_decode_t<64, 2, false, false, WINDOW>(a, ctas, join, stream)
                 : launch_decode_t<64, 1, false, false, WINDOW>(a, ctas, join, stream);
  }
  if (f8)
    return quad  ? launch_decode_t<128, 1, true, true, WINDOW>(a, ctas, join, stream)
           : two ? launch_decode_t<128, 2, true, false, WINDOW>(a, ctas, join, stream)
                 : launch_decode_t<128, 1, true, false, WINDOW>(a, ctas, join, stream);
  return two ? launch_decode_t<128, 2, false, false, WINDOW>(a, ctas, join, stream)
             : launch_decode_t<128, 1, false, false, WINDOW>(a, ctas, join, stream);
}

}  // namespace
}  // namespace eba

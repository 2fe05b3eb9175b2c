// Attention of several drafted tokens per sequence over a paged key-value cache.
//
// The rows of a K/V head are the sequence's n tokens times the G query heads that read
// it, n G rows in items of 128. Row r (token i) sees context key j < c within its window
// and those drafted keys c + x whose bit x its mask has:
//   s_j = scale q . k_j,  M = max s_j,  O = sum e^(s_j - M) v_j / L,  L = sum e^(s_j - M),
//   lse = M + ln L,
// and parts of the keys join exactly as in the single-token decode (decode.cuh).
//
// Each cached element is read once for up to 128 rows: up to 256 flops a byte (bf16),
// which the warp matrix instruction of the single-token kernel cannot keep up with and
// tcgen05 can: of a tile of 128 keys of 128 elements, 64 KB and 1.4 us of an SM's share
// of the HBM rate, the products take 0.75 us. So the kernel is built to keep loads on
// their way and every step of a tile short:
//  - The list of all 128-key tiles of all (sequence, K/V head, 128 rows) items is cut
//    into runs of equal cost, one per CTA, as in decode.cuh: lengths need not be known to
//    the host. Items cut between CTAs leave fp32 parts that the join kernel adds up in order.
//  - Pages of a multiple of 16 keys are loaded by TMA, a box of 32 or 16 keys by 64
//    elements to a lane of a warp for the keys and of one for the values, which look
//    their pages up two tiles ahead; boxes that are cut off are loaded row by row, with
//    zeros for the keys that no row of the item sees. Other page sizes: eight warps with
//    cp.async. (Eight warps of cp.async for all: the e4m3 chains below 250 us, by TMA 190.)
//    bf16: three K and three V tiles. e4m3: two of each, and two stages of stored bytes,
//    which the eight warps widen to fp16 (exact).
//  - Both softmax warpgroups share each tile, 64 keys each, a thread a row: one maximum,
//    one accumulator, no joining at an item's end. A row's reference moves when one of
//    its halves passes it by more than 2^8: a vote each tile, an exchange in the few where
//    it does. (The warpgroups in turn, with an accumulator each: the bf16 batch below 141 us,
//    so 131; the rows of 64 elements 112 and 94 us.)
//  - P in columns of its own, bf16 as in the forward pass (fwd.cuh; the row's largest
//    weight's rounding is added to the sum), or with an e4m3 cache fp16 (and q scaled per
//    row by a power of two into fp16's range). O is 2^-8.8 off as a whole, of the single-token
//    decode, whose P is two bf16 terms, 2^-9.2. Two terms here, in one buffer: the bf16 batch
//    below 163 us.
//  - The QK and the PV products are issued by threads of two warps (see fwd.cuh), and
//    loops are rolled: while the roles' code was larger than the instruction cache, its
//    misses took more time than anything else (this, P as one bf16 term instead of two,
//    and eight loading warps instead of four: 293 -> 148 us).
// Measured (one GB300; bytes of the caches at the time of the call): 32 sequences of up to
// 8191 keys, 32 drafts, 8 heads of 128 for 32: 131 us, 5.3 TB/s, 79 % of a copy; 8 of up
// to 131071 e4m3 keys, 12 drafts, 4 heads of 128 for 32: 180 us, 3.4 TB/s; 16 of up to 6007
// keys, 24 drafts, 16 heads of 64: 76 us, 3.7 TB/s. Rows of 256 bytes: HBM, unequal SMs at the
// end, the join. Rows of 128 bytes: a tile takes about 2400 cycles (bf16) and 3000 (e4m3) for
// 1540 of HBM's share. No role's own work is that long (the softmax 2000 of scores, maximum,
// exponentials, vote and waits, however few its rows; a producer 1750; widening 960): the roles
// wait on one another through rings of two and three tiles. Changing one alone gained nothing
// (more slots, two producers for each operand, copies of few rows that share a tile's keys
// among more warps).
// Tensor memory: S_0 [0,128) S_1 [128,256) O [256,256+d) P_0 [384,448) P_1 [448,512).
#include <cuda_fp16.h>

#include <algorithm>
#include <cfloat>

#include "common.cuh"
#include "kernels.h"
#include "tree_kernels.h"

namespace eba {
namespace {

constexpr int kSoftmax = 256;  // threads: two warpgroups
constexpr int kWarpLoad = 8, kWarpIssue = 16;  // first warps of the loaders (of K, of V) and the issuers
constexpr int kWarpTmaK = 18, kWarpTmaV = 19;  // the producers of TMA loads
constexpr int kBlock = 640;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kRegsSoftmax = 136, kRegsLoad = 72, kRegsIssue = 64;
constexpr int kRegsAtLaunch = (256 * kRegsSoftmax + 256 * kRegsLoad + 128 * kRegsIssue) / kBlock;
static_assert(kRegsAtLaunch == 96 && kRegsAtLaunch * kBlock == 256 * kRegsSoftmax + 256 * kRegsLoad + 128 * kRegsIssue,
              "register split must add up to the launch allocation");
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kSlack = 8.f;     // scores may pass the reference by a factor 2^8
constexpr float kF16Shift = 7.f;  // e4m3 caches: P's largest value is 2^(8 + 7)

template <int D, bool F8>
struct Layout {
  static constexpr int kRow = D * (F8 ? 1 : 2);        // bytes of a cached row
  static constexpr int kTile = kTreeKeys * D * 2;      // of 16-bit elements, for the products
  static constexpr int kAtom = kTreeKeys * 128;        // 64 elements wide
  static constexpr int kSlots = F8 ? 2 : 3;            // of K, and of V
  static constexpr int kAhead = 2;                     // tiles on their way
  static constexpr int kRaw = F8 ? kTreeKeys * kRow : 0;  // a stage of stored bytes
  static constexpr int kMasks = 8;                     // tiles whose key masks are kept
  static constexpr int offQ = 0;
  static constexpr int offK = offQ + kTreeRows * D * 2;
  static constexpr int offV = offK + kSlots * kTile;
  static constexpr int offRaw = offV + kSlots * kTile;
  static constexpr int offMl = offRaw + 2 * kAhead * kRaw;  // [2][128]: what the warpgroups exchange
  static constexpr int offQs = offMl + 2 * kTreeRows * 8;  // [128] score factors (e4m3)
  static constexpr int offKeys = offQs + (F8 ? kTreeRows * 4 : 0);  // [kMasks][4]: keys that are there
  static constexpr int kFlags = 16;                    // and their flags (read later)
  static constexpr int offFlag = offKeys + kMasks * 16;  // [kFlags] bytes
  static constexpr int nBar = 4 * kSlots + 2 + 8 + 1 + 2 + (F8 ? 4 * kAhead : 0);
  static constexpr int offBar = offFlag + kFlags;
  static constexpr int offMisc = offBar + nBar * 8;          // tensor memory's address, abort flag
  static constexpr int offScan = offMl;                      // [kBlock / 32], before the items
  static constexpr int offFirst = offMisc + 8;
  static constexpr int kBytes = offFirst + 64;
  // d = 128 fills shared memory to within a few hundred bytes of the limit, leaving no room
  // to realign the base: the kernel checks instead that it lies on a 1024-byte boundary.
  static constexpr bool kAlignSlack = D == 64;
  static constexpr int kAlloc = kBytes + (kAlignSlack ? 1024 : 0);
  static_assert(kAlloc <= 232448, "shared memory over the limit");
  static constexpr uint32_t cS = 0, cO = 256, cP = 384;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(valid ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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
// Instruction descriptor of fp16 operands: idesc_bf16 without the type bits.
__host__ __device__ constexpr uint32_t idesc(int M, int N, bool b_mn, bool f16) {
  return idesc_bf16(M, N, false, b_mn) & ~(f16 ? (1u << 7) | (1u << 10) : 0u);
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// Whether `mine` holds for any thread of a named barrier, at which all of them meet.
__device__ __forceinline__ bool vote_any(int id, int threads, bool mine) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %3, 0;\n\t"
      "bar.red.or.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"(id), "r"(threads), "r"(static_cast<uint32_t>(mine))
      : "memory");
  return any != 0;
}

// ---- the list of tiles -----------------------------------------------------------------

// A sequence: its first row of q, tokens, cached keys (the tokens are the last ones).
// Without its tokens in the cache (an empty slot of a padded batch) it has no items.
struct Seq {
  int c0, n, len, items;
};
__device__ __forceinline__ Seq sequence(const TreeArgs& a, int b) {
  Seq s;
  const int c0 = a.cu ? a.cu[b] : b, c1 = a.cu ? a.cu[b + 1] : b + 1;
  s.c0 = min(max(c0, 0), a.T);
  s.n = min(max(c1, s.c0), a.T) - s.c0;
  s.len = min(max(a.lens[b], 0), a.max_len);
  s.items = s.len >= s.n ? (s.n * a.group + kTreeRows - 1) / kTreeRows : 0;
  return s;
}
// What is wrong with a sequence's numbers.
__device__ __forceinline__ bool faulty(const TreeArgs& a, int b) {
  const int raw = a.lens[b], c0 = a.cu ? a.cu[b] : b, c1 = a.cu ? a.cu[b + 1] : b + 1;
  return raw < 0 || raw > a.max_len || c0 < 0 || c1 < c0 || c1 > a.T || (raw > 0 && raw < c1 - c0);
}

// Keys that any row of an item sees: the sinks [0, sunk), then [low, high), whose tiles
// begin at the 32 keys that hold low.
struct Keys {
  int sunk, low, high;
  __device__ __forceinline__ int sink_tiles() const { return (sunk + kTreeKeys - 1) / kTreeKeys; }
  __device__ __forceinline__ int tiles() const {
    return sink_tiles() + (high - (low & -32) + kTreeKeys - 1) / kTreeKeys;
  }
  // first key of tile t, and the range of those that count
  __device__ __forceinline__ int from(int t) const {
    return t < sink_tiles() ? t * kTreeKeys : (low & -32) + (t - sink_tiles()) * kTreeKeys;
  }
  __device__ __forceinline__ int begin(int t) const { return t < sink_tiles() ? 0 : low; }
  __device__ __forceinline__ int end(int t) const { return t < sink_tiles() ? sunk : high; }
};
__device__ __forceinline__ Keys item_keys(const TreeArgs& a, const Seq& s, int qt) {
  const int ctx = s.len - s.n;
  const int i0 = qt * kTreeRows / a.group, i1 = min((qt * kTreeRows + kTreeRows - 1) / a.group, s.n - 1);
  Keys k;
  // a row's place is ctx + i, or, of a tree, at least ctx
  k.low = a.window == 0 ? 0 : max(0, ctx + (a.mask ? 0 : i0) + 1 - a.window);
  k.high = a.mask ? s.len : ctx + i1 + 1;
  k.sunk = min(a.sinks, k.low);
  return k;
}

// A place in the list: tile t of nt of an item.
struct Cursor {
  int b, hh, qt, t, nt;
  Seq s;
  Keys k;
};
__device__ __forceinline__ void set_item(Cursor& c, const TreeArgs& a) {
  c.k = item_keys(a, c.s, c.qt);
  c.nt = c.k.tiles();
  c.t = 0;
}
__device__ __forceinline__ void next_item(Cursor& c, const TreeArgs& a) {
  if (++c.qt == c.s.items) {
    c.qt = 0;
    if (++c.hh == a.cache.H_kv) {
      c.hh = 0;
      do {
        if (++c.b == a.B) return;  // behind the list: not used
        c.s = sequence(a, c.b);
      } while (c.s.items == 0);
    }
  }
  set_item(c, a);
}
__device__ __forceinline__ void advance(Cursor& c, const TreeArgs& a) {
  if (__builtin_expect(++c.t == c.nt, 0)) next_item(c, a);
}
// Tiles of one of a sequence's heads.
__device__ __forceinline__ int head_tiles(const TreeArgs& a, const Seq& s) {
  int n = 0;
  for (int qt = 0; qt < s.items; ++qt) n += item_keys(a, s, qt).tiles();
  return n;
}

// The list is cut in units: each tile is one, and each item's end kTreeEnd more (0 in short
// runs). A run begins at a unit's tile, or, at the unit of an end, at the next item.
__device__ __forceinline__ int first_unit(int i, int units, int ctas) {
  return static_cast<int>(static_cast<long long>(i) * units / ctas);
}
// The run that unit u is in.
__device__ __forceinline__ int run_of(int u, int units, int ctas) {
  int i = static_cast<int>(static_cast<long long>(u) * ctas / units);
  while (i + 1 < ctas && first_unit(i + 1, units, ctas) <= u) ++i;
  return i;
}

// Whether the list has more units than an int can count; each thread sums up sequences
// [b0, b1). `all` is shared memory. (In line, where it is hardly ever called, its code cost
// the rows of 64 elements below 1 us of 81.)
__device__ __noinline__ bool list_too_long(const TreeArgs& a, unsigned long long* all, int b0, int b1) {
  if (threadIdx.x == 0) *all = 0;
  __syncthreads();
  unsigned long long sum = 0;
  for (int b = b0; b < b1; ++b) {
    const Seq s = sequence(a, b);
    sum += static_cast<unsigned long long>(head_tiles(a, s) + kTreeEnd * s.items) * a.cache.H_kv;
  }
  atomicAdd(all, sum);
  __syncthreads();
  return *all > 0x7fffffffull;
}

// ---- masks -------------------------------------------------------------------------------

// Bits [lo, hi) of a 32-bit word.
__device__ __forceinline__ uint32_t bits(int lo, int hi) {
  lo = min(max(lo, 0), 32);
  hi = min(max(hi, 0), 32);
  const uint32_t below_hi = hi == 32 ? ~0u : (1u << hi) - 1u, below_lo = lo == 32 ? ~0u : (1u << lo) - 1u;
  return below_hi & ~below_lo;
}
// Bits x .. x + 31 of a mask of `words` 64-bit words (0 outside).
__device__ __forceinline__ uint32_t mask_bits(const long long* m, int words, int x) {
  if (x <= -32 || x >= 64 * words) return 0u;
  const uint32_t* w = reinterpret_cast<const uint32_t*>(m);
  const int at = x >> 5, sh = x & 31;  // (x may be negative: at = -1)
  const uint32_t lo = at >= 0 ? w[at] : 0u, hi = at + 1 < 2 * words ? w[at + 1] : 0u;
  return __funnelshift_r(lo, hi, sh);
}

// What the roles need to know of a tile besides its keys.
enum : uint8_t { kFirst = 0x80, kLast = 0x40, kItem = 0x3f };  // of its item in this run; the item's number

// 4-D tiled load: box at coordinates (x, y, z, w) -> shared memory, counted on `bar`. x must
// be a multiple of 16 bytes.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y,
                                            int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}

// TMA: the page size is a multiple of 16 keys (a.box of 16 or 32 of them to a load).
template <int D, bool F8, bool TMA>
__global__ void __launch_bounds__(kBlock, 1)
    tree_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                const __grid_constant__ TreeArgs a) {
  using L = Layout<D, F8>;
  constexpr int kSlots = L::kSlots, kAhead = L::kAhead;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_base = smem_u32(smem_raw);
  if (!L::kAlignSlack && (raw_base & 1023u) != 0) {
    pdl_wait();
    if (threadIdx.x == 0) atomicExch(a.status, DEV_SMEM_ALIGN);
    return;
  }
  const uint32_t sbase = (raw_base + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sbase - raw_base);
  pdl_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  const uint32_t bar0 = sbase + L::offBar;
  auto k_full = [&](int s) { return bar0 + 8u * s; };
  auto k_empty = [&](int s) { return bar0 + 8u * (kSlots + s); };
  auto v_full = [&](int s) { return bar0 + 8u * (2 * kSlots + s); };
  auto v_empty = [&](int s) { return bar0 + 8u * (3 * kSlots + s); };
  const uint32_t b1 = bar0 + 8u * (4 * kSlots);
  const uint32_t q_full = b1, q_empty = b1 + 8;
  // S of a tile is computed; read by the softmax; P is written; O += P V is done
  auto s_full = [&](int i) { return b1 + 16 + 8u * i; };
  auto s_free = [&](int i) { return b1 + 32 + 8u * i; };
  auto p_full = [&](int i) { return b1 + 48 + 8u * i; };
  auto pv_done = [&](int i) { return b1 + 64 + 8u * i; };
  const uint32_t o_free = b1 + 80;  // the item's end has read O
  auto mma_done = [&](int i) { return b1 + 88 + 8u * i; };
  // stages of stored bytes: K's, then V's
  auto raw_full = [&](int s) { return b1 + 104 + 8u * s; };
  auto raw_empty = [&](int s) { return b1 + 104 + 8u * (2 * kAhead + s); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::offMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::offMisc + 4);
  int2* s_scan = reinterpret_cast<int2*>(smem + L::offScan);
  Cursor& s_first = *reinterpret_cast<Cursor*>(smem + L::offFirst);
  int* s_cut = reinterpret_cast<int*>(smem + L::offFirst + sizeof(Cursor));  // tiles before the run, and its end
  static_assert(sizeof(Cursor) + 8 <= 64, "");
  const DeviceStatus st{a.status, a.limit_ns};

  if (tid == 0) {
    for (int s = 0; s < kSlots; ++s) {
      // (TMA: the producer's expectation, and its own copies done)
      mbar_init(k_full(s), TMA && !F8 ? 2 : 128);
      mbar_init(k_empty(s), 1);
      mbar_init(v_full(s), TMA && !F8 ? 2 : 128);
      mbar_init(v_empty(s), 1);
    }
    for (int s = 0; F8 && s < 2 * kAhead; ++s) {
      mbar_init(raw_full(s), 2);
      mbar_init(raw_empty(s), 128);
    }
    mbar_init(q_full, 256);
    mbar_init(q_empty, F8 ? 1 + kSoftmax : 1);  // the item's last product; its factors are read
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full(i), 2);  // the product's commit, and the issuing thread
      mbar_init(s_free(i), kSoftmax);
      mbar_init(p_full(i), kSoftmax);
      mbar_init(pv_done(i), 1);
      mbar_init(mma_done(i), 1);
    }
    mbar_init(o_free, kSoftmax);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kWarpIssue) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  if (TMA && warp == kWarpTmaK && lane == 0) tma_prefetch_desc(&tm_k);
  if (TMA && warp == kWarpTmaV && lane == 0) tma_prefetch_desc(&tm_v);
  pdl_wait();

  // ---- this CTA's run: each thread counts a run of sequences ----
  const int cta = blockIdx.x;
  const int per = (a.B + kBlock - 1) / kBlock;
  const int b0 = min(tid * per, a.B), b_end = min(b0 + per, a.B);
  int2 mine = make_int2(0, 0);  // tiles, items
  bool falls = false;
  for (int b = b0; b < b_end; ++b) {
    if (cta == 0 && faulty(a, b)) atomicCAS(a.status, 0, ATTN_ERR_PAGE);
    falls |= a.cu && a.cu[b + 1] < a.cu[b];
    const Seq s = sequence(a, b);
    mine.x += head_tiles(a, s) * a.cache.H_kv;
    mine.y += s.items * a.cache.H_kv;
  }
  // Where offsets fall, rows may belong to many sequences, and the list need not fit an int, as
  // it does with the host's checks otherwise: a list that does not is not walked.
  // Where offsets fall, rows may belong to many sequences, and the list need not fit an int, as
  // it does with the host's checks otherwise: a list that does not is not walked.
  const bool too_long = __syncthreads_or(falls) &&
                        list_too_long(a, reinterpret_cast<unsigned long long*>(smem + L::offFirst), b0, b_end);
  if (too_long) mine = make_int2(0, 0);
  int2 incl = mine;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl.x, m), y = __shfl_up_sync(0xffffffffu, incl.y, m);
    if (lane >= m) incl.x += x, incl.y += y;
  }
  if (lane == 31) s_scan[warp] = incl;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  int2 before = make_int2(0, 0), all = make_int2(0, 0);
#pragma unroll
  for (int w = 0; w < kBlock / 32; ++w) {
    const int2 x = s_scan[w];
    if (w < warp) before.x += x.x, before.y += x.y;
    all.x += x.x, all.y += x.y;
  }
  const int tiles = all.x;
  const int G = max(1, min(static_cast<int>(gridDim.x), tiles));  // no run is empty
  const int end_units = tiles / G >= 4 * kTreeEnd ? kTreeEnd : 0;
  const int units = tiles + end_units * all.y;
  const int u1 = first_unit(cta + 1, units, G);
  if (cta < G) {
    const int at0 = before.x + incl.x - mine.x, items0 = before.y + incl.y - mine.y;
#pragma unroll 1
    for (int e = 0; e < 2; ++e) {
      const int u = e ? u1 : first_unit(cta, units, G);
      int at = at0, unit = at0 + end_units * items0;
      if (e && cta + 1 == G && tid == 0) s_cut[1] = tiles;
      if (u < unit || u >= unit + mine.x + end_units * mine.y) continue;
      for (int b = b0; b < b_end; ++b) {
        Cursor c;
        c.s = sequence(a, b);
        const int ht = head_tiles(a, c.s), hu = ht + end_units * c.s.items;
        if (u >= unit + hu * a.cache.H_kv) {
          unit += hu * a.cache.H_kv;
          at += ht * a.cache.H_kv;
          continue;
        }
        int in = u - unit;
        c.b = b;
        c.hh = in / hu;
        in -= c.hh * hu;
        at += c.hh * ht;
        for (c.qt = 0;; ++c.qt) {
          set_item(c, a);
          if (in < c.nt + end_units) break;
          in -= c.nt + end_units;
          at += c.nt;
        }
        c.t = min(in, c.nt);
        s_cut[e] = at + c.t;
        if (c.t == c.nt) next_item(c, a);
        if (e == 0) s_first = c;
        break;
      }
    }
  }
  // Sequences without keys, and all rows of a list that is too long: O = 0, lse = -inf.
  auto blank = [&](long long token0, long long tokens, int first, int step) {
    const long long row0 = token0 * a.H, rows = tokens * a.H;
    for (long long x = first; x < rows * (D / 8); x += step)
      *reinterpret_cast<uint4*>(a.o + row0 * D + x * 8) = make_uint4(0, 0, 0, 0);
    for (long long x = first; x < rows; x += step) a.lse[row0 + x] = -INFINITY;
  };
  if (too_long) {
    blank(0, a.T, cta * kBlock + tid, gridDim.x * kBlock);
  } else {
    for (int b = cta; b < a.B; b += gridDim.x) {
      const Seq s = sequence(a, b);
      if (s.items == 0) blank(s.c0, s.n, tid, kBlock);
    }
  }
  __syncthreads();
  const int n_tiles = cta < G && tiles > 0 ? s_cut[1] - s_cut[0] : 0;

  // TMA producer of the keys or the values: lane i has box i / kAtoms of each tile, and half
  // i % kAtoms of its rows.
  auto produce = [&](bool values) {
    constexpr int kAtoms = F8 ? 1 : D / 64;
    constexpr int kLanes = L::kRow / 16, kRows = 32 / kLanes;
    constexpr int kTurns = F8 ? kAhead : kSlots;
    const int box = a.box, bx = lane / kAtoms, atom = lane % kAtoms;
    const bool mine = bx * box < kTreeKeys;
    const uint32_t whole = box == 32 ? ~0u : 0xffffu;
    const uint32_t box_bytes = box * (F8 ? L::kRow : 128);
    const CUtensorMap* map = values ? &tm_v : &tm_k;
    uint32_t* s_keys = reinterpret_cast<uint32_t*>(smem + L::offKeys);
    uint8_t* s_flag = smem + L::offFlag;
    auto full = [&](int i) {
      return F8 ? raw_full((values ? kAhead : 0) + i % kAhead) : values ? v_full(i % kSlots) : k_full(i % kSlots);
    };
    Cursor look = s_first;
    int item = -1, left = n_tiles;
    // looked up two tiles ahead
    int page_of[2] = {}, slot_of[2] = {}, head_of[2] = {}, flag_of[2] = {};
    uint32_t part_of[2] = {};  // the box's keys that count
    int n = -2;
#pragma unroll 1
    for (; n < n_tiles; ++n) {
      if (n >= 0) {
        const int slot = F8 ? (values ? kAhead : 0) + n % kAhead : n % kSlots;
        const uint32_t empty = F8 ? raw_empty(slot) : values ? v_empty(slot) : k_empty(slot);
        if (n >= kTurns && !__all_sync(0xffffffffu, mbar_wait(empty, ((n / kTurns) - 1) & 1, abort_flag, st))) break;
        const bool there = static_cast<unsigned>(page_of[0]) < static_cast<unsigned>(a.cache.n_pages);
        if (part_of[0] && !there) atomicCAS(a.status, 0, ATTN_ERR_PAGE);
        const uint32_t keys = there ? part_of[0] : 0u;
        const bool load = mine && keys == whole;
        const uint32_t loads = __ballot_sync(0xffffffffu, load), boxes = __ballot_sync(0xffffffffu, mine);
        const uint32_t to =
            sbase + (F8 ? L::offRaw + slot * L::kRaw : (values ? L::offV : L::offK) + slot * L::kTile);
        if (lane == 0) mbar_arrive_expect_tx(full(n), __popc(loads) * box_bytes);
        __syncwarp();
        if (load)
          tma_load_4d(to + (F8 ? 0 : atom * L::kAtom) + bx * box_bytes, map, full(n), atom * 64, head_of[0],
                      slot_of[0], page_of[0]);
        if (!values) {
          // the tile's keys that are there, 32 to a word
          uint32_t word = ~0u;
          if (loads != boxes) {
            const uint32_t lo = __shfl_sync(0xffffffffu, keys, (box == 32 ? lane : 2 * lane) * kAtoms & 31);
            const uint32_t up = __shfl_sync(0xffffffffu, keys, (2 * lane + 1) * kAtoms & 31);
            word = box == 32 ? lo : lo | up << 16;
          }
          if (lane < 4) s_keys[(n % L::kMasks) * 4 + lane] = word;
          __syncwarp();
        }
        // (both producers, the same: either may be ahead, and its readers go by it)
        if (lane == 0) s_flag[n % L::kFlags] = static_cast<uint8_t>(flag_of[0]);
        if (__builtin_expect(loads != boxes, 0)) {
          // Boxes that are cut off or not there: row by row, zeros for the keys that do not count.
          uint32_t rest = __ballot_sync(0xffffffffu, mine && atom == 0 && !load);
          const long long st_page = values ? a.v_strides[0] : a.k_strides[0];
          const long long st_slot = values ? a.v_strides[1] : a.k_strides[1];
          const long long st_head = values ? a.v_strides[2] : a.k_strides[2];
          const long long off = keys ? page_of[0] * st_page + slot_of[0] * st_slot + head_of[0] * st_head : 0;
          const int c16 = lane % kLanes, r_lane = lane / kLanes;
#pragma unroll 1
          while (rest) {
            const int from = __ffs(rest) - 1;
            rest &= rest - 1;
            const uint32_t count = __shfl_sync(0xffffffffu, keys, from);
            const unsigned char* p = (values ? a.v : a.k) + __shfl_sync(0xffffffffu, off, from) + c16 * 16;
#pragma unroll 1
            for (int r = r_lane; r < box; r += kRows) {
              const int row = from / kAtoms * box + r;
              const uint32_t at = F8 ? row * L::kRow + c16 * 16 : (c16 >> 3) * L::kAtom + sw128_offset(row, c16 & 7);
              cp_async16(to + at, p + (count >> r & 1 ? r * st_slot : 0), count >> r & 1);
            }
          }
          cp_async_commit();
          cp_async_wait<0>();
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (lane == 0) mbar_arrive(full(n));
      }
      page_of[0] = page_of[1], slot_of[0] = slot_of[1], head_of[0] = head_of[1];
      flag_of[0] = flag_of[1], part_of[0] = part_of[1];
      part_of[1] = 0;
      if (left > 0) {
        const bool first = look.t == 0 || left == n_tiles;
        item += first;
        flag_of[1] = (first ? kFirst : 0) | (look.t + 1 == look.nt ? kLast : 0) | (item & kItem);
        head_of[1] = look.hh;
        const int key = look.k.from(look.t) + bx * box;
        const uint32_t part = mine ? bits(look.k.begin(look.t) - key, look.k.end(look.t) - key) & whole : 0u;
        if (part) {
          const int entry = static_cast<int>(static_cast<uint64_t>(key) * a.page_mul >> a.page_shift);
          slot_of[1] = key - entry * a.cache.page_size;
          page_of[1] = a.table[look.b * a.table_stride + entry];
          part_of[1] = part;
        }
        if (--left > 0) advance(look, a);
      }
    }
    // Every copy started here must land before the CTA may exit. (n: tiles started, also where a
    // wait gave up.)
    for (int i = max(0, n - kTurns); i < n; ++i) mbar_wait_drain(full(i), (i / kTurns) & 1, st);
  };

  if (warp >= kWarpIssue) {
    regs_decrease<kRegsIssue>();
    const int role = warp - kWarpIssue;  // 0: S = Q K^T, 1: O += P V
    if (role < 2 && lane == 0) {
      constexpr uint32_t hi = sdesc_hi(1024);
      constexpr uint32_t id_qk = idesc(kTreeRows, kTreeKeys, false, F8);
      constexpr uint32_t id_pv = idesc(kTreeRows, D, true, F8);
      const uint32_t q_lo = sdesc_lo(sbase + L::offQ, 16), k_lo = sdesc_lo(sbase + L::offK, 16);
      const uint32_t v_lo = sdesc_lo(sbase + L::offV, L::kAtom);
      const volatile uint8_t* s_flag = smem + L::offFlag;
      bool ok = true;
      for (int n = 0; n < n_tiles && ok; ++n) {
        const int slot = n % kSlots, i = n & 1;
        const uint32_t sp = (n / kSlots) & 1, before = ((n >> 1) - 1) & 1;
        if (role == 0) {
          if (!(ok = mbar_wait(k_full(slot), sp, abort_flag, st))) break;
          const int f = s_flag[n % L::kFlags];
          if ((f & kFirst) && !(ok = mbar_wait(q_full, f & 1, abort_flag, st))) break;
          if (n > 1 && !(ok = mbar_wait(s_free(i), before, abort_flag, st))) break;
          tc_fence_after();
#pragma unroll 2
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = ((kk >> 2) * L::kAtom + (kk & 3) * 32) >> 4;
            mma_ss(tmem + L::cS + i * kTreeKeys, sdesc_join(q_lo + off, hi),
                   sdesc_join(k_lo + slot * (L::kTile >> 4) + off, hi), id_qk, kk > 0);
          }
          mma_commit(k_empty(slot));
          if (f & kLast) mma_commit(q_empty);
          mma_commit(s_full(i));
          mbar_arrive(s_full(i));  // what the loaders wrote for the softmax is visible behind this
        } else {
          if (!(ok = mbar_wait(p_full(i), (n >> 1) & 1, abort_flag, st))) break;
          if (!(ok = mbar_wait(v_full(slot), sp, abort_flag, st))) break;
          const int f = s_flag[n % L::kFlags];
          const bool first = f & kFirst;  // overwrites O, once the item before has been read out
          if (first && n > 0 && !(ok = mbar_wait(o_free, ((f & kItem) - 1) & 1, abort_flag, st))) break;
          tc_fence_after();
#pragma unroll 2
          for (int kk = 0; kk < kTreeKeys / 16; ++kk)
            mma_ts(tmem + L::cO, tmem + L::cP + i * (kTreeKeys / 2) + kk * 8,
                   sdesc_join(v_lo + slot * (L::kTile >> 4) + kk * (2048 >> 4), hi), id_pv, !first || kk > 0);
          mma_commit(v_empty(slot));
          mma_commit(pv_done(i));
        }
      }
      // Every MMA this thread issued must be finished before tensor memory is released.
      mma_commit(mma_done(role));
      mbar_wait_drain(mma_done(role), 0, st);
    }
    if constexpr (TMA)
      if (warp >= kWarpTmaK) produce(warp == kWarpTmaV);
  } else if (warp >= kWarpLoad) {
    regs_decrease<kRegsLoad>();
    // An item's query rows, by all of these warps: row x is token x / G, head x % G of the
    // group; zeros behind the last.
    constexpr int kChunks = D / 8;           // 16 bytes of a row each
    constexpr int kStep = 256 / kChunks;     // rows between a thread's
    constexpr int kPer = kTreeRows / kStep;  // of a thread
    const int l = tid - 32 * kWarpLoad, ch = l % kChunks;
    auto fetch_q = [&](const Cursor& c, uint4 (&x)[kPer]) {
      const int rows = min(kTreeRows, c.s.n * a.group - c.qt * kTreeRows);
      const int at = c.qt * kTreeRows + l / kChunks;
      int token = at / a.group, g = at - token * a.group;
      const int step_t = kStep / a.group, step_g = kStep - step_t * a.group;
      const __nv_bfloat16* q = a.q + static_cast<long long>(c.hh) * a.group * a.q_head + ch * 8;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        x[i] = make_uint4(0, 0, 0, 0);
        if (i * kStep + l / kChunks < rows)
          x[i] = *reinterpret_cast<const uint4*>(q + (c.s.c0 + token) * a.q_token + g * a.q_head);
        token += step_t;
        g += step_g;
        if (g >= a.group) g -= a.group, ++token;
      }
    };
    auto store_q = [&](const uint4 (&x)[kPer]) {
      float* s_qs = reinterpret_cast<float*>(smem + L::offQs);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int row = i * kStep + l / kChunks;
        uint32_t y[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        if constexpr (F8) {
          float top = 0.f;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float u = fabsf(bf16lo_f32(y[e])), v = fabsf(bf16hi_f32(y[e]));
            top = fmaxf(top, fmaxf(u < INFINITY ? u : 0.f, v < INFINITY ? v : 0.f));
          }
#pragma unroll
          for (int m = kChunks / 2; m > 0; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
          // 2^e brings the row's largest element into [2^13, 2^14) (see decode.cuh)
          const int floor_log2 = static_cast<int>(__float_as_uint(top) >> 23) - 127;
          const int e2 = top > 0.f ? min(13 - floor_log2, 126) : 0;
          const float up = __uint_as_float(static_cast<uint32_t>(127 + e2) << 23);
          const float down = __uint_as_float(static_cast<uint32_t>(127 - e2) << 23);
          if (ch == 0) s_qs[row] = fminf(a.scale_log2 * (a.cache.k_scale * down), FLT_MAX);
#pragma unroll
          for (int e = 0; e < 4; ++e) y[e] = pack_f16(bf16lo_f32(y[e]) * up, bf16hi_f32(y[e]) * up);
        }
        st_shared_v4(sbase + L::offQ + (ch >> 3) * L::kAtom + sw128_offset(row, ch & 7), y[0], y[1], y[2], y[3]);
      }
      fence_proxy_async_smem();
      mbar_arrive(q_full);
    };
    int item = 0;  // running index in this CTA
    // The query's buffer is free once the previous item's last product has read it.
    auto q_free = [&]() {
      return item == 0 || __all_sync(0xffffffffu, mbar_wait(q_empty, (item - 1) & 1, abort_flag, st));
    };
    Cursor c = s_first;
    if constexpr (TMA && !F8) {
      // ---- the queries alone: the next item's wait in registers ----
      for (int left = n_tiles; left > 0;) {
        uint4 x[kPer];
        fetch_q(c, x);
        if (!q_free()) break;
        store_q(x);
        ++item;
        left -= c.nt - c.t;
        if (left > 0) next_item(c, a);
      }
    } else {
      // ---- warps 0 to 3: keys, 4 to 7: values; rows 32 w .. 32 w + 31 of each tile ----
      const int w = (warp - kWarpLoad) & 3;
      const bool keys = warp < kWarpLoad + 4;
      constexpr int kLanes = L::kRow / 16;  // of a row: 16 bytes each
      constexpr int kRows = 32 / kLanes;    // of an instruction
      constexpr int kLoads = 32 / kRows;    // instructions of 32 rows
      const int c16 = lane % kLanes, r_lane = lane / kLanes;
      const uint32_t tile_base = sbase + (keys ? L::offK : L::offV);
      const uint32_t raw = sbase + L::offRaw + (keys ? 0 : kAhead * L::kRaw) + w * (L::kRaw / 4) + lane * 16;
      uint8_t* s_flag = smem + L::offFlag;
      auto full = [&](int s) { return keys ? k_full(s) : v_full(s); };
      auto empty = [&](int s) { return keys ? k_empty(s) : v_empty(s); };
      // e4m3: where this lane's 16 bytes go, widened (the swizzle repeats after 8 rows)
      constexpr int kWides = F8 ? 8 / kRows : 1;
      uint32_t wide[kWides];
#pragma unroll
      for (int i = 0; i < kWides; ++i)
        wide[i] = (c16 >> 2) * L::kAtom + 32 * w * 128 + sw128_offset(i * kRows + r_lane, (c16 & 3) * 2);
      auto widen = [&](int n) {
        uint4 got[kLoads];
#pragma unroll
        for (int i = 0; i < kLoads; ++i) got[i] = ld_shared_v4(raw + (n % kAhead) * L::kRaw + i * 512);
        const uint32_t to = tile_base + (n % kSlots) * L::kTile;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          const uint4 x = got[i];
          const uint32_t at = to + wide[i % kWides] + i / kWides * 1024;
          st_shared_v4(at, e4m3x2_f16x2(x.x), e4m3x2_f16x2(x.x >> 16), e4m3x2_f16x2(x.y), e4m3x2_f16x2(x.y >> 16));
          // (the row's next chunk: its neighbour)
          st_shared_v4(at ^ 16u, e4m3x2_f16x2(x.z), e4m3x2_f16x2(x.z >> 16), e4m3x2_f16x2(x.w),
                       e4m3x2_f16x2(x.w >> 16));
        }
      };
      auto slot_free = [&](int n) {
        return n < kSlots ||
               __all_sync(0xffffffffu, mbar_wait(empty(n % kSlots), ((n / kSlots) - 1) & 1, abort_flag, st));
      };
      if constexpr (TMA) {
        // e4m3 by TMA: widen only
#pragma unroll 1
        for (int n = 0; n < n_tiles; ++n) {
          const int stage = (keys ? 0 : kAhead) + n % kAhead;
          if (!__all_sync(0xffffffffu, mbar_wait(raw_full(stage), (n / kAhead) & 1, abort_flag, st))) break;
          if (s_flag[n % L::kFlags] & kFirst) {
            if (n > 0) next_item(c, a);
            uint4 x[kPer];
            fetch_q(c, x);
            if (!q_free()) break;
            store_q(x);
            ++item;
          }
          if (!slot_free(n)) break;
          widen(n);
          mbar_arrive(raw_empty(stage));
          fence_proxy_async_smem();
          mbar_arrive(full(n % kSlots));
        }
      } else {
        const unsigned char* base = (keys ? a.k : a.v) + c16 * 16;
        const long long st_page = keys ? a.k_strides[0] : a.v_strides[0];
        const long long st_slot = keys ? a.k_strides[1] : a.v_strides[1];
        const long long st_head = keys ? a.k_strides[2] : a.v_strides[2];
        uint32_t* s_keys = reinterpret_cast<uint32_t*>(smem + L::offKeys);
        // each lane looks its row up, two tiles ahead of the load
        Cursor look = s_first;
        int left = n_tiles, look_item = -1;
        int page_of[2] = {}, slot_of[2] = {-1, -1};  // slot -1: no such key
        int head_of[2] = {}, flag_of[2] = {};
        auto look_up = [&]() {
          page_of[0] = page_of[1], slot_of[0] = slot_of[1], head_of[0] = head_of[1], flag_of[0] = flag_of[1];
          page_of[1] = 0, slot_of[1] = -1;
          if (left <= 0) return;
          const bool first = look.t == 0 || left == n_tiles;
          look_item += first;
          flag_of[1] = (first ? kFirst : 0) | (look.t + 1 == look.nt ? kLast : 0) | (look_item & kItem);
          head_of[1] = look.hh;
          const int key = look.k.from(look.t) + 32 * w + lane;
          if (key >= look.k.begin(look.t) && key < look.k.end(look.t)) {
            const int entry = static_cast<int>(static_cast<uint64_t>(key) * a.page_mul >> a.page_shift);
            slot_of[1] = key - entry * a.cache.page_size;
            page_of[1] = a.table[look.b * a.table_stride + entry];
          }
          if (--left > 0) advance(look, a);
        };
        // bf16: where this lane's 16 bytes go (the swizzle repeats after 8 rows)
        constexpr int kPats = F8 ? 1 : 8 / kRows;
        uint32_t pat[kPats];
#pragma unroll
        for (int i = 0; i < kPats; ++i)
          pat[i] = F8 ? 0u : (c16 >> 3) * L::kAtom + 32 * w * 128 + sw128_offset(i * kRows + r_lane, c16 & 7);
        auto issue = [&](int n) {
          const int page = page_of[0], sl = slot_of[0];
          const bool held = sl >= 0;
          const bool there = held && static_cast<unsigned>(page) < static_cast<unsigned>(a.cache.n_pages);
          if (held && !there) atomicCAS(a.status, 0, ATTN_ERR_PAGE);
          const long long off = there ? page * st_page + sl * st_slot + head_of[0] * st_head : 0;
          const uint32_t rows = __ballot_sync(0xffffffffu, there);
          if (keys && lane == 0) s_keys[(n % L::kMasks) * 4 + w] = rows;
          if (keys && w == 0 && lane == 0) s_flag[n % L::kFlags] = static_cast<uint8_t>(flag_of[0]);
          const uint32_t to = F8 ? raw + (n % kAhead) * L::kRaw : tile_base + (n % kSlots) * L::kTile;
          // (addresses of several rows first: one after the other they wait for each shuffle)
          constexpr int kSet = kLoads < 8 ? kLoads : 8;
#pragma unroll
          for (int i0 = 0; i0 < kLoads; i0 += kSet) {
            const unsigned char* p[kSet];
#pragma unroll
            for (int i = 0; i < kSet; ++i) p[i] = base + __shfl_sync(0xffffffffu, off, (i0 + i) * kRows + r_lane);
#pragma unroll
            for (int i = 0; i < kSet; ++i)
              cp_async16(F8 ? to + (i0 + i) * 512 : to + pat[(i0 + i) % kPats] + (i0 + i) / kPats * 1024, p[i],
                         rows >> ((i0 + i) * kRows + r_lane) & 1);
          }
        };
        // Step n: tile n is handed over, tile n + kAhead fetched, and the one two further looked
        // up. (One loop, also for the first tiles: every copy of this code costs instruction
        // fetches.)
#pragma unroll 1
        for (int n = -kAhead - 2; n < n_tiles; ++n) {
          if (n >= 0) {
            if (c.t == 0 || n == 0) {
              uint4 x[kPer];
              fetch_q(c, x);
              if (!q_free()) break;
              store_q(x);
              ++item;
            }
            if (n + 1 < n_tiles) advance(c, a);
            cp_async_wait<kAhead - 1>();
            if constexpr (F8) {
              if (!slot_free(n)) break;
              widen(n);  // this lane's own bytes
            }
            fence_proxy_async_smem();
            mbar_arrive(full(n % kSlots));
            // bf16: the next tile waits for its slot
            if (!F8 && n + kAhead < n_tiles && !slot_free(n + kAhead)) break;
          }
          if (n + kAhead >= 0 && n + kAhead < n_tiles) issue(n + kAhead);
          cp_async_commit();
          look_up();
        }
        cp_async_wait<0>();
      }
    }
  } else {
    regs_increase<kRegsSoftmax>();
    // ---- softmax: warpgroup g has keys 64 g .. 64 g + 63 of every tile, a thread one row ----
    const int g = warp >> 2, sub = warp & 3;
    const int row = sub * 32 + lane;  // of the item == lane of tensor memory
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(sub * 32) << 16);
    const uint32_t tO = lane_base + L::cO + g * (D / 2);  // the columns that it rescales and writes out
    float* s_max = reinterpret_cast<float*>(smem + L::offMl);   // [warpgroup][row]
    float2* s_sum = reinterpret_cast<float2*>(smem + L::offMl);  // at an item's end
    // A wait that gives up ends all waits; the warps still meet at every barrier, and
    // what they write is undefined.
    bool live = true;
    auto wait = [&](uint32_t bar, uint32_t parity) {
      if (live) live = __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, st));
    };
    Cursor c = s_first;
    int n = 0, item = 0;
    while (n < n_tiles) {
      // ---- an item: its tiles [c.t, c.t + count) are the run's [n, n + count) ----
      const int t_begin = c.t, count = min(c.nt - c.t, n_tiles - n);
      const bool ends = c.t + count == c.nt;
      const int at = c.qt * kTreeRows + row;  // of the sequence's rows
      const bool has = at < c.s.n * a.group;
      const bool some = __any_sync(0xffffffffu, has);
      const int token = has ? at / a.group : 0, ctx = c.s.len - c.s.n;
      const long long* mask = a.mask ? a.mask + (c.s.c0 + token) * a.mask_stride : nullptr;
      int place = ctx + token;
      if (mask) {
        int ones = 0;
        for (int x = 0; x < 2 * a.words; ++x)
          ones += __popc(mask_bits(mask, a.words, 32 * x) & bits(0, c.s.n - 32 * x));
        place = ctx + max(ones, 1) - 1;
      }
      // the context keys that this row sees begin at `near`, and with a chain also the others
      const int near = a.window == 0 ? 0 : place - a.window + 1;
      const int near_most = __reduce_max_sync(0xffffffffu, near);
      float m_used = -INFINITY;
      float l_sum = 0.f, l_fix = 0.f;  // the weights' sum, and what their rounding adds to it
      float qs = a.scale_log2;
#pragma unroll 1
      for (int step = 0; step < count; ++step) {
        const int nn = n + step, i = nn & 1;
        const int k1 = c.k.from(t_begin + step) + 64 * g;
        wait(s_full(i), (nn >> 1) & 1);
        tc_fence_after();
        if (F8 && step == 0) {
          qs = reinterpret_cast<const float*>(smem + L::offQs)[row];
          mbar_arrive(q_empty);
        }
        uint32_t x[64];  // this row's scores
        if (some) {
          tmem_ld32(lane_base + L::cS + i * kTreeKeys + 64 * g, *reinterpret_cast<uint32_t(*)[32]>(x));
          tmem_ld32(lane_base + L::cS + i * kTreeKeys + 64 * g + 32, *reinterpret_cast<uint32_t(*)[32]>(x + 32));
        }
        // the keys that are there; in most tiles all, and all rows see them
        const uint2 there = *reinterpret_cast<const uint2*>(smem + L::offKeys + (nn % L::kMasks) * 16 + 8 * g);
        if (some) {
          tmem_wait_ld();
          reg_pin(*reinterpret_cast<uint32_t(*)[32]>(x));
          reg_pin(*reinterpret_cast<uint32_t(*)[32]>(x + 32));
        }
        tc_fence_before();
        mbar_arrive(s_free(i));  // the tile after the next may be computed
        if (__builtin_expect((there.x & there.y) != ~0u || k1 < near_most || k1 + 64 > ctx, 0)) {
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int k2 = k1 + 32 * y;
            uint32_t u;
            if (mask) {
              u = bits(near - k2, ctx - k2) | bits(0, min(a.sinks, ctx) - k2);
              if (k2 + 32 > ctx) u |= mask_bits(mask, a.words, k2 - ctx) & bits(ctx - k2, c.s.len - k2);
            } else {
              u = bits(near - k2, place + 1 - k2) | bits(0, min(a.sinks, place + 1) - k2);
            }
            u &= y ? there.y : there.x;
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!((u >> e) & 1)) x[32 * y + e] = 0xff800000u;  // -inf
          }
        }
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < 64; e += 8) {
#pragma unroll
          for (int u = 0; u < 4; ++u) m4[u] = fmax3(m4[u], __uint_as_float(x[e + u]), __uint_as_float(x[e + 4 + u]));
        }
        const float mine = some ? fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * qs : -INFINITY;
        // The reference moves when either warpgroup's part of the row passes it by more than
        // kSlack: a vote of both each tile, and an exchange in the few where it does.
        if (__builtin_expect(vote_any(1, kSoftmax, mine > m_used + kSlack), 0)) {
          s_max[g * kTreeRows + row] = mine;
          named_bar_sync(1, kSoftmax);
          const float both = fmaxf(mine, s_max[(1 - g) * kTreeRows + row]);
          const bool bump = both > m_used + kSlack;
          const float alpha = bump ? ex2_approx(m_used - both) : 1.f;
          if (bump) m_used = both;
          l_sum *= alpha;
          l_fix *= alpha;
          if (step > 0) {
            // O holds the products up to the tile before, once that is done
            wait(pv_done(1 - i), ((nn - 1) >> 1) & 1);
            tc_fence_after();
            if (__any_sync(0xffffffffu, bump)) {
#pragma unroll 1
              for (int y = 0; y < D / 64; ++y) {
                uint32_t ov[32];
                tmem_ld32(tO + 32 * y, ov);
                tmem_wait_ld();
                reg_pin(ov);
#pragma unroll
                for (int e = 0; e < 32; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
                tmem_st32(tO + 32 * y, ov);
              }
            }
          }
        }
        // (a row that has seen no key yet has no maximum)
        const float ref = (m_used == -INFINITY ? 0.f : m_used) - (F8 ? kF16Shift : 0.f);
        const float2 qs2 = make_float2(qs, qs), neg = make_float2(-ref, -ref);
        if (nn > 1) {
          wait(pv_done(i), ((nn >> 1) - 1) & 1);  // P of the tile before the last has been used
          tc_fence_after();
        }
        if (some) {
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const uint32_t* y = x + 32 * half + 2 * e;
              const float2 z = fma2(make_float2(__uint_as_float(y[0]), __uint_as_float(y[1])), qs2, neg);
              const float2 p = make_float2(ex2_approx(z.x), ex2_approx(z.y));
              w[e] = F8 ? pack_f16(p.x, p.y) : pack_bf16(p.x, p.y);
              sum[e & 1] = add2(sum[e & 1], p);
            }
            tmem_st16(lane_base + L::cP + i * (kTreeKeys / 2) + 32 * g + 16 * half, w);
          }
          l_sum += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
          // bf16: the rounding of the largest weight (see fwd.cuh: the others' even out)
          const float top = F8 ? 0.f : ex2_approx(mine - ref);
          l_fix += bf16lo_f32(pack_bf16(top, 0.f)) - top;
          tmem_st_wait();
        }
        tc_fence_before();
        mbar_arrive(p_full(i));
      }

      // ---- the item's end, or the run's: the row's sums of both warpgroups, and half of O ----
      {
        const int last = n + count - 1;
        wait(pv_done(last & 1), (last >> 1) & 1);
        tc_fence_after();
        s_sum[g * kTreeRows + row] = make_float2(l_sum, l_fix);
        named_bar_sync(1, kSoftmax);
        const float2 other = s_sum[(1 - g) * kTreeRows + row];
        const float l = l_sum + other.x, rounded = l + (l_fix + other.y);
        // No weight: nothing seen, or only scores of -inf. (A NaN score leaves the maximum as it
        // was, but not the sum: such a row is NaN, its part's reference any finite one.)
        const bool none = m_used == -INFINITY && l == 0.f;
        const float M = none ? -INFINITY : (m_used == -INFINITY ? 0.f : m_used) - (F8 ? kF16Shift : 0.f);
        const bool whole = t_begin == 0 && ends;
        // a part: O as its weights' sum l would have it
        const float mul = none ? 0.f : whole ? a.o_scale / rounded : l / rounded;
        const long long out = (static_cast<long long>(c.s.c0) + token) * a.H + c.hh * a.group + at % a.group;
        const long long slot = 2 * cta + (item == 0 ? 0 : 1);
        if (has && g == 0) {
          if (whole)
            a.lse[out] = none ? -INFINITY : (M + lg2_approx(l)) * kLn2;
          else
            a.part_ml[slot * kTreeRows + row] = make_float2(M, l);
        }
        if (some) {
#pragma unroll 1
          for (int y = 0; y < D / 64; ++y) {
            const int col = g * (D / 2) + 32 * y;
            uint32_t u[32];
            tmem_ld32(tO + 32 * y, u);
            tmem_wait_ld();
            reg_pin(u);
            if (!has) continue;
            float v[32];
            // (a row without a weight: whatever was added)
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = none ? 0.f : __uint_as_float(u[e]) * mul;
            if (whole) {
              uint4* to = reinterpret_cast<uint4*>(a.o + out * D + col);
#pragma unroll
              for (int e = 0; e < 4; ++e)
                to[e] = make_uint4(pack_bf16(v[8 * e], v[8 * e + 1]), pack_bf16(v[8 * e + 2], v[8 * e + 3]),
                                   pack_bf16(v[8 * e + 4], v[8 * e + 5]), pack_bf16(v[8 * e + 6], v[8 * e + 7]));
            } else {
              float4* to = reinterpret_cast<float4*>(a.part_o + (slot * kTreeRows + row) * D + col);
#pragma unroll
              for (int e = 0; e < 8; ++e) to[e] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
            }
          }
        }
        tc_fence_before();
        mbar_arrive(o_free);  // the next item's first product may overwrite O
      }
      n += count;
      if (n == n_tiles && a.cut && tid == 0) {
        // an item that begins in this run and goes on in the next ones
        int parts = 0;
        if (!ends && t_begin == 0) parts = run_of(u1 + c.nt - count - 1, units, G) - cta + 1;
        a.cut[cta] = make_int2(item == 0 ? 0 : 1, parts);
        a.item[cta] = make_int4(c.b, c.hh, c.qt, 0);
      }
      ++item;
      if (n < n_tiles) {
        c.t += count - 1;
        advance(c, a);
      }
    }
    if (n_tiles == 0 && a.cut && tid == 0) a.cut[cta] = make_int2(0, 0);
  }

  // ---- teardown ----
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpIssue) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Items cut between CTAs: their parts, in the order of the keys. blockIdx.x: a run, y: 8 rows.
// Few parts: the blocks of the run that the item begins in, a warp a row. More than 8: those
// of its first 8 runs, a row each, all warps: with the first run's blocks alone, row after
// row, 1501 keys of 8 heads (12 parts each) took 25.0 us in all, so 18.6.
constexpr int kJoinWarps = 8, kDeep = 4, kFewParts = kJoinWarps;
template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps) tree_join_kernel(const __grid_constant__ TreeArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  constexpr int kVec = D / 32;
  __shared__ float s_o[kJoinWarps][D];
  __shared__ float2 s_ml[kJoinWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int run = blockIdx.x;
  int2 cut = lane < kJoinWarps && run >= lane ? a.cut[run - lane] : make_int2(0, 0);
  // (no run is among the first 8 of two such items, or of one and begins another)
  const uint32_t longs = __ballot_sync(0xffffffffu, cut.y > kFewParts);
  const bool few = longs == 0;
  const int behind = few ? 0 : __ffs(longs) - 1, c0 = run - behind;
  cut.x = __shfl_sync(0xffffffffu, cut.x, behind);
  const int parts = __shfl_sync(0xffffffffu, cut.y, behind);
  if (parts == 0) return;
  const int4 it = a.item[c0];
  const Seq s = sequence(a, it.x);
  const int rows = min(kTreeRows, s.n * a.group - it.z * kTreeRows);
  const int row = blockIdx.y * kJoinWarps + (few ? warp : behind);
  if (row >= rows) return;  // (many: all warps alike)
  float M = -INFINITY, l = 0.f, o[kVec] = {};
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
      const long long at = (2 * (c0 + p) + (p == 0 ? cut.x : 0)) * static_cast<long long>(kTreeRows) + row;
      ml[u] = a.part_ml[at];
      const float* from = a.part_o + at * D + lane * kVec;
#pragma unroll
      for (int x = 0; x < kVec; x += 2) {
        const float2 y = *reinterpret_cast<const float2*>(from + x);
        v[u][x] = y.x, v[u][x + 1] = y.y;
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
  const int at = it.z * kTreeRows + row, token = at / a.group;
  const long long out = (static_cast<long long>(s.c0) + token) * a.H + it.y * a.group + at % a.group;
  if (few) {
    const float f = M == -INFINITY ? 0.f : a.o_scale / l;
#pragma unroll
    for (int x = 0; x < kVec; x += 2)
      *reinterpret_cast<uint32_t*>(a.o + out * D + lane * kVec + x) = pack_bf16(o[x] * f, o[x + 1] * f);
    if (lane == 0) a.lse[out] = M == -INFINITY ? -INFINITY : (M + lg2_approx(l)) * kLn2;
    return;
  }
  if (lane == 0) s_ml[warp] = make_float2(M, l);
#pragma unroll
  for (int x = 0; x < kVec; ++x) s_o[warp][lane * kVec + x] = o[x];
  __syncthreads();
  if (threadIdx.x < D) {
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
    a.o[out * D + threadIdx.x] = __float2bfloat16_rn(v * f);
    if (threadIdx.x == 0) a.lse[out] = M == -INFINITY ? -INFINITY : (M + lg2_approx(l)) * kLn2;
  }
}

template <int D, bool F8, bool TMA>
cudaError_t launch_tree_t(const CUtensorMap& tk, const CUtensorMap& tv, const TreeArgs& a, int ctas, bool join,
                          cudaStream_t stream) {
  using L = Layout<D, F8>;
  auto kern = tree_kernel<D, F8, TMA>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kAlloc);
  if (e != cudaSuccess) return e;
  // The warpgroups' register shares must fit the launch allocation, or an increase would
  // wait forever: refuse to launch otherwise.
  cudaFuncAttributes fa;
  e = cudaFuncGetAttributes(&fa, kern);
  if (e != cudaSuccess) return e;
  if (fa.numRegs < kRegsAtLaunch) return cudaErrorInvalidConfiguration;
  e = launch_pdl(kern, dim3(ctas), dim3(kBlock), L::kAlloc, stream, tk, tv, a);
  if (e != cudaSuccess || !join) return e;
  const int rows = std::min(kTreeRows, a.T * a.group);
  return launch_pdl(tree_join_kernel<D>, dim3(ctas, (rows + kJoinWarps - 1) / kJoinWarps),
                    dim3(32 * kJoinWarps), 0, stream, a);
}

template <int D, bool F8>
cudaError_t launch_tree_d(const CUtensorMap& tk, const CUtensorMap& tv, const TreeArgs& a, int ctas, bool join,
                          cudaStream_t stream) {
  return a.box ? launch_tree_t<D, F8, true>(tk, tv, a, ctas, join, stream)
               : launch_tree_t<D, F8, false>(tk, tv, a, ctas, join, stream);
}

}  // namespace

cudaError_t launch_tree(const CUtensorMap& tk, const CUtensorMap& tv, const TreeArgs& a, int ctas, bool join,
                        cudaStream_t stream) {
  const bool f8 = a.cache.type == ATTN_CACHE_E4M3;
  if (a.cache.d == 64)
    return f8 ? launch_tree_d<64, true>(tk, tv, a, ctas, join, stream)
              : launch_tree_d<64, false>(tk, tv, a, ctas, join, stream);
  return f8 ? launch_tree_d<128, true>(tk, tv, a, ctas, join, stream)
            : launch_tree_d<128, false>(tk, tv, a, ctas, join, stream);
}

}  // namespace eba

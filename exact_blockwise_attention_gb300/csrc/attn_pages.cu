// The pages of a paged key-value cache: giving them back, sharing them between forked
// sequences, handing out free ones, and copies within the cache.
//
// A page's state is one number, how many table entries name it; it is free at 0. There
// is no list of free pages to keep in order: a call that needs pages takes the lowest
// free ones, its n-th wanted entry the n-th of them. That needs two prefix sums (of the
// wants in order of the table, of the free pages in order of their numbers) and a pass
// over the counts, and its result depends on the counts alone, not on the order in which
// blocks run or on what was given back when.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "pages_kernels.h"

namespace eba {
namespace {

__device__ __forceinline__ void bad_page(int* status) { atomicCAS(status, 0, ATTN_ERR_PAGE); }

__device__ __forceinline__ int pages_of(int keys, int size) { return keys / size + (keys % size != 0); }

// The sequence that token t belongs to (cu[s] <= t < cu[s + 1]), or -1.
__device__ __forceinline__ int sequence_of(const int* cu, int n, int t) {
  if (t < cu[0] || t >= cu[n]) return -1;
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (cu[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}

// ---- giving pages back ----------------------------------------------------------------

// blockIdx.y: the sequence. Counts are changed by atomic additions of integers: their
// order does not matter.
constexpr int kReleaseThreads = 256;
__global__ void __launch_bounds__(kReleaseThreads)
    release_kernel(const __grid_constant__ ReleaseArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  for (int b = blockIdx.y; b < a.n_seqs; b += gridDim.y) {
    // (both bounds within the table before any entry's index is formed from them)
    const int e0 = min(pages_of(max(a.first[b], 0), a.pool.page_size), a.max_pages);
    const int e1 = min(a.last[b] / a.pool.page_size, a.max_pages);
    int* row = a.table + b * a.table_stride;
    for (long long e = e0 + static_cast<long long>(blockIdx.x) * kReleaseThreads + threadIdx.x; e < e1;
         e += gridDim.x * kReleaseThreads) {
      const int page = row[e];
      if (page < 0) continue;
      row[e] = -1;
      if (page >= a.pool.n_pages) {
        bad_page(a.status);
      } else if (atomicSub(a.pool.refs + page, 1) <= 0) {  // nobody held it
        atomicAdd(a.pool.refs + page, 1);
        bad_page(a.status);
      }
    }
  }
}

// ---- handing out the lowest free pages ---------------------------------------------------

// One cluster. Its warps each take a run of the wanting sequences (or pairs) and a run
// of the pages; two barriers of the cluster separate counting, listing and handing out.
constexpr int kPoolCtas = 8, kPoolWarps = 32;
constexpr int kPoolWorkers = kPoolCtas * kPoolWarps;
constexpr int kPoolDeep = 8;  // loads of a lane under way

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ int ld_remote(const int* p, uint32_t rank) {
  int v;
  uint32_t at;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}
// Orders what the cluster's threads wrote before, in shared and in global memory.
__device__ __forceinline__ void sync_cluster() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

__device__ __forceinline__ int warp_sum(int x) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
  return x;
}

// A sequence's entries [e0, e1), within its row, that may want a page (those that hold
// none do).
__device__ __forceinline__ bool wanted_range(const PoolArgs& a, int b, int& e0, int& e1) {
  const int len = a.lens[b], more = a.new_lens[b];
  if (len < 0 || max(len, more) > static_cast<long long>(a.max_pages) * a.pool.page_size) {
    if ((threadIdx.x & 31) == 0) bad_page(a.status);
    return false;
  }
  e0 = pages_of(len, a.pool.page_size);
  e1 = more > len ? pages_of(more, a.pool.page_size) : e0;
  return true;
}

// Whether a table's entry holds no page.
__device__ __forceinline__ bool wants_page(const PoolArgs& a, int entry) {
  return static_cast<unsigned>(entry) >= static_cast<unsigned>(a.pool.n_pages);
}

// What a fork's pair asks for, kept in a.to between the cluster's barriers.
enum : int { kPairBad = -3, kPairWhole = -2, kPairCopies = -1 };

__device__ __forceinline__ int check_pair(const PoolArgs& a, int i, int lane) {
  const int s = a.src[i], d = a.dst[i];
  bool bad = s < 0 || s >= a.n_seqs || d < 0 || d >= a.n_seqs;
  // a slot that another sequence forks from, or that an earlier pair takes
  bool clash = false;
  for (int j = lane; j < a.n; j += 32) clash |= a.src[j] == d || (j < i && a.dst[j] == d);
  bad |= __any_sync(0xffffffffu, clash);
  int len = 0;
  if (!bad) {
    len = a.lens[s];
    bad = len < 0 || len > static_cast<long long>(a.max_pages) * a.pool.page_size;
  }
  if (bad) {
    if (lane == 0) bad_page(a.status);
    return kPairBad;
  }
  const int whole = len / a.pool.page_size;
  if (len % a.pool.page_size == 0) return kPairWhole;
  const int page = a.table[s * a.table_stride + whole];
  if (page >= a.pool.n_pages && lane == 0) bad_page(a.status);
  return page >= 0 && page < a.pool.n_pages ? kPairCopies : kPairWhole;
}

template <bool FORK>
__global__ void __cluster_dims__(kPoolCtas, 1, 1) __launch_bounds__(32 * kPoolWarps)
    pool_kernel(const __grid_constant__ PoolArgs a) {
  __shared__ int s_want[kPoolWarps], s_free[kPoolWarps], s_total[2];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int worker = rank * kPoolWarps + warp;
  const int size = a.pool.page_size;
  const int u0 = static_cast<int>(static_cast<long long>(worker) * a.n / kPoolWorkers);
  const int u1 = static_cast<int>(static_cast<long long>(worker + 1) * a.n / kPoolWorkers);

  // ---- what is wanted ----
  int want = 0;
  if constexpr (FORK) {
    for (int i = u0; i < u1; ++i) {
      const int kind = check_pair(a, i, lane);
      if (lane == 0) a.to[i] = kind;
      want += kind == kPairCopies;
    }
    sync_cluster();
    // The rows, 256 entries to a warp's step with their loads under way together: whole
    // pages are shared. (One entry after the other: the call took 34 us for 100 rows of 1577, not 26.)
    constexpr int kRun = 32 * kPoolDeep;
    const int parts = (a.max_pages + kRun - 1) / kRun;
    const long long items = static_cast<long long>(a.n) * parts;
    for (long long x = worker; x < items; x += kPoolWorkers) {
      const int i = static_cast<int>(x / parts), part = static_cast<int>(x - static_cast<long long>(i) * parts);
      const int s = a.src[i], d = a.dst[i];
      if (__ldcg(a.to + i) == kPairBad) continue;
      const int* in = a.table + s * a.table_stride;
      int* out = a.table + d * a.table_stride;
      int page[kPoolDeep];
      const int len = a.lens[s];
#pragma unroll
      for (int u = 0; u < kPoolDeep; ++u) {
        const int e = part * kRun + 32 * u + lane;
        page[u] = e < a.max_pages ? in[e] : -1;
      }
      const int whole = len / size;
#pragma unroll
      for (int u = 0; u < kPoolDeep; ++u) {
        const int e = part * kRun + 32 * u + lane;
        if (e >= whole) page[u] = -1;
        if (page[u] >= a.pool.n_pages) {
          bad_page(a.status);
          page[u] = -1;
        }
        if (page[u] >= 0) atomicAdd(a.pool.refs + page[u], 1);
        if (e < a.max_pages) out[e] = max(page[u], -1);
      }
      if (part == 0 && lane == 0) a.lens[d] = len;
    }
    sync_cluster();
  } else {
    for (int b = u0; b < u1; ++b) {
      int e0, e1;
      if (!wanted_range(a, b, e0, e1)) continue;
      const int* row = a.table + b * a.table_stride;
      for (long long e = static_cast<long long>(e0) + lane; e < e1; e += 32) {
        want += wants_page(a, row[e]);
        if (row[e] >= a.pool.n_pages) bad_page(a.status);
      }
    }
    want = warp_sum(want);
  }

  // ---- how many pages of this warp's run are free ----
  const int per = ((a.pool.n_pages - 1) / kPoolWorkers / 32 + 1) * 32;
  const int p0 = static_cast<int>(min(static_cast<long long>(worker) * per, static_cast<long long>(a.pool.n_pages)));
  const int p1 = min(a.pool.n_pages, p0 + min(per, a.pool.n_pages - p0));
  int free = 0;
  for (int p = p0; p < p1; p += 32 * kPoolDeep) {
    int r[kPoolDeep];
#pragma unroll
    for (int i = 0; i < kPoolDeep; ++i) {
      const long long at = static_cast<long long>(p) + 32 * i + lane;
      r[i] = at < p1 ? __ldcg(a.pool.refs + at) : 1;
    }
#pragma unroll
    for (int i = 0; i < kPoolDeep; ++i) free += r[i] == 0;
  }
  free = warp_sum(free);
  if (lane == 0) s_want[warp] = want, s_free[warp] = free;
  __syncthreads();
  // this warp's first want and free page in its CTA's, then the cluster's, order
  int before_want = 0, before_free = 0, all_want = 0, all_free = 0;
  {
    const int w = s_want[lane], f = s_free[lane];
    before_want = warp_sum(lane < warp ? w : 0);
    before_free = warp_sum(lane < warp ? f : 0);
    const int tw = warp_sum(w), tf = warp_sum(f);
    if (threadIdx.x == 0) s_total[0] = tw, s_total[1] = tf;
  }
  sync_cluster();
#pragma unroll
  for (int c = 0; c < kPoolCtas; ++c) {
    const int w = ld_remote(s_total, c), f = ld_remote(s_total + 1, c);
    if (c < static_cast<int>(rank)) before_want += w, before_free += f;
    all_want += w;
    all_free += f;
  }

  // ---- list the pages that are handed out ----
  for (int p = p0; p < p1 && before_free < all_want; p += 32 * kPoolDeep) {
    int r[kPoolDeep];
#pragma unroll
    for (int i = 0; i < kPoolDeep; ++i) {
      const long long at = static_cast<long long>(p) + 32 * i + lane;
      r[i] = at < p1 ? __ldcg(a.pool.refs + at) : 1;
    }
#pragma unroll
    for (int i = 0; i < kPoolDeep; ++i) {
      const uint32_t zeros = __ballot_sync(0xffffffffu, r[i] == 0);
      const int nth = before_free + __popc(zeros & ((1u << lane) - 1u));
      if (r[i] == 0 && nth < all_want) a.pool.scratch[nth] = p + 32 * i + lane;
      before_free += __popc(zeros);
    }
  }
  sync_cluster();

  // ---- hand them out ----
  auto take = [&](int nth) {
    if (nth >= all_free) {
      bad_page(a.status);
      return -1;
    }
    const int page = __ldcg(a.pool.scratch + nth);
    a.pool.refs[page] = 1;
    return page;
  };
  if constexpr (FORK) {
    if (lane == 0)
      for (int i = u0; i < u1; ++i) {
        int from = -1, to = -1;
        if (__ldcg(a.to + i) == kPairCopies) {
          to = take(before_want++);
          const int s = a.src[i], whole = a.lens[s] / size;
          if (to >= 0) {
            from = a.table[s * a.table_stride + whole];
            a.table[a.dst[i] * a.table_stride + whole] = to;
          }
        }
        a.from[i] = from;
        a.to[i] = to;
      }
  } else {
    for (int b = u0; b < u1; ++b) {
      int e0, e1;
      if (!wanted_range(a, b, e0, e1)) continue;
      int* row = a.table + b * a.table_stride;
      for (long long e = e0; e < e1; e += 32) {
        const bool mine = e + lane < e1 && wants_page(a, row[e + lane]);
        const uint32_t wants = __ballot_sync(0xffffffffu, mine);
        if (mine) row[e + lane] = take(before_want + __popc(wants & ((1u << lane) - 1u)));
        before_want += __popc(wants);
      }
    }
  }
}

// ---- copies ------------------------------------------------------------------------------

constexpr int kCopyThreads = 256, kCopyDeep = 4;

// Whole pages. blockIdx.x: the pair, y: a run of its rows' 16-byte units, z: keys, values.
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const __grid_constant__ CopyArgs a) {
  pdl_launch_dependents();
  pdl_wait();
  const int from = a.from[blockIdx.x], to = a.to[blockIdx.x];
  if (from < 0 || to < 0 || from == to) return;
  if (from >= a.n_pages || to >= a.n_pages) {
    if (threadIdx.x == 0) bad_page(a.status);
    return;
  }
  unsigned char* base = blockIdx.z ? a.v : a.k;
  const long long* st = blockIdx.z ? a.v_strides : a.k_strides;
  const int lanes = a.row / 16;  // 4, 8 or 16: units of a row
  const long long units = static_cast<long long>(a.page_size) * a.H_kv * lanes;
  for (long long u0 = (static_cast<long long>(blockIdx.y) * kCopyDeep) * kCopyThreads + threadIdx.x;
       u0 < units; u0 += static_cast<long long>(gridDim.y) * kCopyDeep * kCopyThreads) {
    uint4 x[kCopyDeep];
    long long off[kCopyDeep];
#pragma unroll
    for (int i = 0; i < kCopyDeep; ++i) {
      const long long u = u0 + i * kCopyThreads;
      if (u >= units) continue;
      const long long r = u / lanes;
      const int slot = static_cast<int>(r / a.H_kv), head = static_cast<int>(r - static_cast<long long>(slot) * a.H_kv);
      off[i] = slot * st[1] + head * st[2] + (u - r * lanes) * 16;
      x[i] = *reinterpret_cast<const uint4*>(base + from * st[0] + off[i]);
    }
#pragma unroll
    for (int i = 0; i < kCopyDeep; ++i)
      if (u0 + i * kCopyThreads < units) *reinterpret_cast<uint4*>(base + to * st[0] + off[i]) = x[i];
  }
}

// Chosen tokens, 128 of them at a time: 16 tokens side by side, 16 of a token's 16-byte
// units each (blockIdx.y: which 16 of its keys and values), 8 of such sets under way.
// ORDERED (the rows stay in their sequence's pages): blockIdx.x is the sequence, and its
// tokens go in order, 128 read before any of them is written. A row that does not move
// up is then read before its place is written: the places that a step writes lie before
// those that later steps read.
constexpr int kGatherTokens = 128, kGatherUnits = 16;
template <bool ORDERED>
__global__ void __launch_bounds__(kCopyThreads) gather_kernel(const __grid_constant__ GatherArgs a) {
  __shared__ int s_page[kGatherTokens], s_slot[kGatherTokens];  // page -1: no row to move
  __shared__ int s_to_page[kGatherTokens], s_to_slot[kGatherTokens];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x % kGatherUnits, set = threadIdx.x / kGatherUnits;
  const int per_row = a.row / 16;
  const int unit = blockIdx.y * kGatherUnits + lane;  // of a token's keys, then its values
  const int heads_units = a.H_kv * per_row;
  const bool has = unit < 2 * heads_units, values = unit >= heads_units;
  const int in = unit - (values ? heads_units : 0);
  const long long* st = values ? a.v_strides : a.k_strides;
  unsigned char* base = (values ? a.v : a.k) + in / per_row * st[2] + in % per_row * 16;
  long long t0, t1;
  if (ORDERED) {
    t0 = max(a.cu[blockIdx.x], 0);
    t1 = min(a.cu[blockIdx.x + 1], a.T);
  } else {
    t0 = static_cast<long long>(blockIdx.x) * kGatherTokens;
    t1 = min(t0 + kGatherTokens, static_cast<long long>(a.T));
  }
  for (; t0 < t1; t0 += kGatherTokens) {
    if (threadIdx.x < kGatherTokens) {
      int page = -1, slot = 0, to_page = 0, to_slot = 0;
      const int t = static_cast<int>(t0) + threadIdx.x;
      if (t0 + threadIdx.x < t1) {
        const int b = ORDERED ? static_cast<int>(blockIdx.x) : sequence_of(a.cu, a.n_seqs, t);
        if (b >= 0) {
          const long long place = a.places[t];
          const long long to = (a.to_start ? a.to_start[b] : 0ll) + (t - a.cu[b]);
          const long long room = static_cast<long long>(a.max_pages) * a.page_size;
          const long long to_room = static_cast<long long>(a.to_max_pages) * a.page_size;
          bool ok = place >= 0 && place < room && to >= 0 && to < to_room && !(ORDERED && place < to);
          if (ok) {
            const int e = static_cast<int>(place / a.page_size), z = static_cast<int>(to / a.page_size);
            slot = static_cast<int>(place - static_cast<long long>(e) * a.page_size);
            to_slot = static_cast<int>(to - static_cast<long long>(z) * a.page_size);
            page = a.table[b * a.table_stride + e];
            to_page = a.to_table[b * a.to_stride + z];
            ok = page >= 0 && page < a.n_pages && to_page >= 0 && to_page < a.n_pages;
            if (page == to_page && slot == to_slot) page = -1;  // it is there already
          }
          if (!ok) {
            bad_page(a.status);
            page = -1;
          }
        }
      }
      s_page[threadIdx.x] = page;
      s_slot[threadIdx.x] = slot;
      s_to_page[threadIdx.x] = to_page;
      s_to_slot[threadIdx.x] = to_slot;
    }
    __syncthreads();
    constexpr int kSets = kGatherTokens * kGatherUnits / kCopyThreads;
    uint4 x[kSets];
#pragma unroll
    for (int i = 0; i < kSets; ++i) {
      const int t = i * (kCopyThreads / kGatherUnits) + set;
      if (has && s_page[t] >= 0)
        x[i] = *reinterpret_cast<const uint4*>(base + s_page[t] * st[0] + s_slot[t] * st[1]);
    }
    if (ORDERED) __syncthreads();
#pragma unroll
    for (int i = 0; i < kSets; ++i) {
      const int t = i * (kCopyThreads / kGatherUnits) + set;
      if (has && s_page[t] >= 0)
        *reinterpret_cast<uint4*>(base + s_to_page[t] * st[0] + s_to_slot[t] * st[1]) = x[i];
    }
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_release(const ReleaseArgs& a, cudaStream_t stream) {
  // few blocks a sequence: most calls give back a few pages of each
  const int x = std::min((a.max_pages - 1) / kReleaseThreads + 1, 8);
  return launch_pdl(release_kernel, dim3(x, std::min(a.n_seqs, 65535)), dim3(kReleaseThreads), 0, stream, a);
}

cudaError_t launch_fork(const PoolArgs& a, cudaStream_t stream) {
  return launch_pdl(pool_kernel<true>, dim3(kPoolCtas), dim3(32 * kPoolWarps), 0, stream, a);
}

cudaError_t launch_reserve(const PoolArgs& a, cudaStream_t stream) {
  return launch_pdl(pool_kernel<false>, dim3(kPoolCtas), dim3(32 * kPoolWarps), 0, stream, a);
}

cudaError_t launch_copy(const CopyArgs& a, cudaStream_t stream) {
  const long long units = static_cast<long long>(a.page_size) * a.H_kv * (a.row / 16);
  const long long y = std::min((units + kCopyThreads * kCopyDeep - 1) / (kCopyThreads * kCopyDeep), 1024ll);
  return launch_pdl(copy_kernel, dim3(a.n, static_cast<unsigned>(y), 2), dim3(kCopyThreads), 0, stream, a);
}

cudaError_t launch_gather(const GatherArgs& a, cudaStream_t stream) {
  const int slices = (2 * a.H_kv * (a.row / 16) + kGatherUnits - 1) / kGatherUnits;
  const dim3 block(kCopyThreads);
  if (a.in_place) return launch_pdl(gather_kernel<true>, dim3(a.n_seqs, slices), block, 0, stream, a);
  return launch_pdl(gather_kernel<false>, dim3((a.T + kGatherTokens - 1) / kGatherTokens, slices), block, 0,
                    stream, a);
}

}  // namespace eba

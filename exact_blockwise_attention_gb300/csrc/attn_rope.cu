// Rotary positions over several axes (time, height, width of video tokens),
// and new keys and values written into a paged cache with the keys rotated on
// the way. The rotation and its angles: rope.cuh.
//
// Both kernels are bound by memory: each element is read once and written
// once, with about 3 flops an element. A thread owns 8 pairs of one token (two
// 16-byte vectors) and keeps their 8 cosines and sines in registers while it
// walks several heads, so the trigonometry (about 45 instructions a pair) is
// paid once per group of heads and not per element.
#include "rope.cuh"

namespace eba {
namespace {

constexpr int kRopeThreads = 128;
constexpr int kUnroll = 4;  // heads whose loads are in flight together

// Inputs are read by ordinary loads, not through the read-only path: a kernel that
// begins before the one in front of it is done (pdl_wait) sees them change in its
// lifetime.
struct Vec16 {  // 16 elements of one head: two 16-byte vectors
  uint4 a, b;
};

__device__ __forceinline__ Vec16 load16(const __nv_bfloat16* p, int off_a, int off_b) {
  Vec16 v;
  v.a = *reinterpret_cast<const uint4*>(p + off_a);
  v.b = *reinterpret_cast<const uint4*>(p + off_b);
  return v;
}

__device__ __forceinline__ void widen8(const uint4& v, float (&x)[8]) {
  x[0] = bf16lo_f32(v.x), x[1] = bf16hi_f32(v.x), x[2] = bf16lo_f32(v.y), x[3] = bf16hi_f32(v.y);
  x[4] = bf16lo_f32(v.z), x[5] = bf16hi_f32(v.z), x[6] = bf16lo_f32(v.w), x[7] = bf16hi_f32(v.w);
}

// The cosines and sines of a thread's 8 pairs.
struct Turn8 {
  float c[8], s[8];
};

// 8 pairs: (a[i], b[i]) with halves as pairs, or neighbours (x0 x1) (x2 x3) ...
template <bool INTERLEAVED>
__device__ __forceinline__ void turn16(float (&a)[8], float (&b)[8], const Turn8& t) {
  if constexpr (INTERLEAVED) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      rope_turn(a[2 * i], a[2 * i + 1], t.c[i], t.s[i]);
      rope_turn(b[2 * i], b[2 * i + 1], t.c[i + 4], t.s[i + 4]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) rope_turn(a[i], b[i], t.c[i], t.s[i]);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                    pack_bf16(x[6], x[7]));
}

// Lane i of a token's D / 16: its two vectors' element offsets. Lanes below
// n_pairs / 8 hold rotated pairs; the others elements behind the rotated ones.
template <bool INTERLEAVED>
__device__ __forceinline__ void lane_offsets(int i, int n_pairs, int& off_a, int& off_b) {
  if (INTERLEAVED || 8 * i >= n_pairs) {
    off_a = 16 * i;
    off_b = 16 * i + 8;
  } else {
    off_a = 8 * i;
    off_b = n_pairs + 8 * i;
  }
}

// The rotation's table in shared memory. (As a kernel argument it lies in the
// constant bank, which serves one address at a time: a warp's lanes read 4 or 8
// different pairs, and 16 such reads a thread took longer than the sines and
// cosines.)
struct RopeTable {
  ulonglong2 turns[ATTN_MAX_PAIRS / 2];
  uint2 axis[ATTN_MAX_PAIRS / 8];
};

__device__ __forceinline__ void load_table(RopeTable& t, const attn_rope_t& r) {
  const int i = threadIdx.x;
  if (i < ATTN_MAX_PAIRS) {
    reinterpret_cast<unsigned long long*>(t.turns)[i] = r.turns[i];
    reinterpret_cast<unsigned char*>(t.axis)[i] = r.axis[i];
  }
  __syncthreads();
}

// cos, sin of pairs 8 i .. 8 i + 7 at the positions p of the axes.
__device__ __forceinline__ void lane_turn(const RopeTable& r, int i, const int (&p)[ATTN_MAX_AXES],
                                          float sign, Turn8& t) {
  const uint2 ax = r.axis[i];
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    const ulonglong2 turns = r.turns[4 * i + j / 2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int axis = ((j < 4 ? ax.x : ax.y) >> (8 * ((j + u) % 4))) & 0xff;
      int pj = p[0];
#pragma unroll
      for (int a = 1; a < ATTN_MAX_AXES; ++a) pj = axis == a ? p[a] : pj;
      rope_cs(pj, u ? turns.y : turns.x, sign, t.c[j + u], t.s[j + u]);
    }
  }
}

__device__ __forceinline__ void load_positions(int (&p)[ATTN_MAX_AXES], int n_axes, const int* pos,
                                               long long stride) {
#pragma unroll
  for (int a = 0; a < ATTN_MAX_AXES; ++a) p[a] = a < n_axes ? pos[a * stride] : 0;
}

template <int D, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
  pdl_launch_dependents();
  __shared__ RopeTable s_table;
  load_table(s_table, a.rope);  // kernel arguments alone: before the previous kernel is done
  pdl_wait();
  constexpr int kLanes = D / 16;
  const long long id = static_cast<long long>(blockIdx.x) * kRopeThreads + threadIdx.x;
  const int i = static_cast<int>(id % kLanes);
  const long long token = id / kLanes;
  if (token >= a.tokens) return;
  const long long b = token / a.L;
  const long long l = token - b * a.L;
  const int h0 = blockIdx.y * a.heads_per;
  const int h1 = min(h0 + a.heads_per, a.H[0] + a.H[1]);
  int off_a, off_b;
  lane_offsets<INTERLEAVED>(i, a.rope.n_pairs, off_a, off_b);
  const bool turns = 8 * i < a.rope.n_pairs;
  const __nv_bfloat16* src[2];
  __nv_bfloat16* dst[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    src[x] = static_cast<const __nv_bfloat16*>(a.in[x]) + b * a.si[x][0] + l * a.si[x][2];
    dst[x] = static_cast<__nv_bfloat16*>(a.out[x]) + b * a.so[x][0] + l * a.so[x][2];
  }
  auto from = [&](int h) {
    return h < a.H[0] ? src[0] + h * a.si[0][1] : src[1] + (h - a.H[0]) * a.si[1][1];
  };
  auto to = [&](int h) {
    return h < a.H[0] ? dst[0] + h * a.so[0][1] : dst[1] + (h - a.H[0]) * a.so[1][1];
  };
  // the first heads' loads go out before the trigonometry
  Vec16 v[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u)
    if (h0 + u < h1) v[u] = load16(from(h0 + u), off_a, off_b);
  Turn8 t;
  if (turns) {
    int p[ATTN_MAX_AXES];
    load_positions(p, a.rope.n_axes, a.pos + b * a.pos_batch + l, a.pos_axis);
    lane_turn(s_table, i, p, a.sign, t);
  }
  for (int h = h0; h < h1; h += kUnroll) {
    if (h > h0) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
        if (h + u < h1) v[u] = load16(from(h + u), off_a, off_b);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (h + u >= h1) break;
      __nv_bfloat16* o = to(h + u);
      if (turns) {
        float x[8], y[8];
        widen8(v[u].a, x);
        widen8(v[u].b, y);
        turn16<INTERLEAVED>(x, y, t);
        v[u].a = pack8(x);  // the one rounding, to the output's type
        v[u].b = pack8(y);
      }
      *reinterpret_cast<uint4*>(o + off_a) = v[u].a;
      *reinterpret_cast<uint4*>(o + off_b) = v[u].b;
    }
  }
}

// ---------------------------------------------------------------------------
// New rows into the pages
// ---------------------------------------------------------------------------

// The sequence of token t: the s with cu[s] <= t < cu[s + 1], or -1 for a
// token outside [cu[0], cu[n]).
__device__ __forceinline__ int find_sequence(const int* cu, int n, long long t) {
  if (t < cu[0] || t >= cu[n]) return -1;
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}

// Where token t goes: its place in its sequence, the table entry of its page
// (null: it is not written) and its slot. A place out of range is recorded in
// the status word; the entry's page is checked when it is used, so that its load
// overlaps the trigonometry.
struct Place {
  const int* entry;
  int at, slot;
};
__device__ __forceinline__ Place find_place(const AppendArgs& a, long long t) {
  Place p{nullptr, 0, 0};
  int s;
  long long back;  // new tokens of the sequence from this one on
  if (a.cu_new) {
    s = find_sequence(a.cu_new, a.n_seqs, t);
    if (s < 0) return p;  // behind the last sequence: padding
    back = a.cu_new[s + 1] - t;
  } else {
    s = static_cast<int>(t);
    back = 1;
  }
  const int len = a.lens[s];
  if (len == 0) return p;  // an empty slot of the batch
  const long long at = len - back;
  // (at >= len: offsets that decrease)
  if (at < 0 || at >= len || at >= static_cast<long long>(a.max_pages) * a.cache.page_size) {
    atomicCAS(a.status, 0, ATTN_ERR_PAGE);
    return p;
  }
  p.at = static_cast<int>(at);
  const int entry = p.at / a.cache.page_size;
  p.slot = p.at - entry * a.cache.page_size;
  p.entry = a.table + s * a.table_stride + entry;
  return p;
}

// x times the rounded reciprocal of the scale, and e4m3 to nearest: the product is within
// 2^-23 of the quotient, so next to a tie of two e4m3 numbers it may take the other one
// (of the 65280 finite bf16 numbers, 30 at scale 0.03, none at 0.0125). The quotient costs
// more than that is worth: 5 x 4999 tokens of 8 heads of 128 take 43 us by division, 33
// by the product corrected with its remainder and 30 with the reciprocal as two floats,
// instead of 27.6.
__device__ __forceinline__ uint2 pack8_e4m3(const float (&x)[8], float inv) {
  return make_uint2(pack_e4m3x4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv),
                    pack_e4m3x4(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv));
}

// blockIdx.z: the keys' or the values' half of the work (a thread that did both
// would hold twice the registers, and its values would wait for its keys' angles).
// Six CTAs an SM leave 80 registers: enough for bf16, while e4m3 spills 8 or 9 of them
// (four CTAs, without spills: the same 27.6 us; five 28.3).
template <int D, bool INTERLEAVED, bool F8>
__global__ void __launch_bounds__(kRopeThreads, 6)
    append_kernel(const __grid_constant__ AppendArgs a) {
  pdl_launch_dependents();
  __shared__ RopeTable s_table;
  load_table(s_table, a.rope);  // kernel arguments alone: before the previous kernel is done
  pdl_wait();
  constexpr int kLanes = D / 16;
  const long long id = static_cast<long long>(blockIdx.x) * kRopeThreads + threadIdx.x;
  const int i = static_cast<int>(id % kLanes);
  const long long token = id / kLanes;
  if (token >= a.tokens) return;
  const bool keys = blockIdx.z == 0;
  const int h0 = blockIdx.y * a.heads_per;
  const int h1 = min(h0 + a.heads_per, a.cache.H_kv);
  const bool turns = keys && 8 * i < a.rope.n_pairs;
  int off_a, off_b;
  lane_offsets<INTERLEAVED>(i, keys ? a.rope.n_pairs : 0, off_a, off_b);
  const attn_cache_t& c = a.cache;
  const long long in_head = keys ? a.k_head : a.v_head;
  const __nv_bfloat16* in = keys ? static_cast<const __nv_bfloat16*>(a.k) + token * a.k_token
                                 : static_cast<const __nv_bfloat16*>(a.v) + token * a.v_token;
  Vec16 v[kUnroll];
  auto fetch = [&](int h) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (h + u < h1) v[u] = load16(in + (h + u) * in_head, off_a, off_b);
  };
  fetch(h0);
  int pos[ATTN_MAX_AXES] = {};
  if (turns && a.pos) load_positions(pos, a.rope.n_axes, a.pos + token, a.pos_axis);
  const Place place = find_place(a, token);
  if (!place.entry) return;
  const int page = *place.entry;
  Turn8 t;
  if (turns) {
    if (!a.pos) pos[0] = place.at;  // one axis: the place in the sequence
    lane_turn(s_table, i, pos, 1.f, t);
  }
  if (page < 0 || page >= c.n_pages) {
    atomicCAS(a.status, 0, ATTN_ERR_PAGE);
    return;
  }
  const long long* st = keys ? c.k_strides : c.v_strides;
  const long long out_head = st[2];
  const long long row = page * st[0] + place.slot * st[1];
  for (int h = h0; h < h1; h += kUnroll) {
    if (h > h0) fetch(h);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (h + u >= h1) break;
      const long long to = row + (h + u) * out_head;
      float x[8], y[8];
      if (F8 || turns) {
        widen8(v[u].a, x);
        widen8(v[u].b, y);
        if (turns) turn16<INTERLEAVED>(x, y, t);
      }
      if constexpr (F8) {
        // no bf16 in between: fp32 straight to e4m3 (to nearest, saturating)
        unsigned char* p = static_cast<unsigned char*>(keys ? c.k : c.v) + to;
        const float inv = keys ? a.k_inv : a.v_inv;
        *reinterpret_cast<uint2*>(p + off_a) = pack8_e4m3(x, inv);
        *reinterpret_cast<uint2*>(p + off_b) = pack8_e4m3(y, inv);
      } else {
        if (turns) {
          v[u].a = pack8(x);
          v[u].b = pack8(y);
        }
        __nv_bfloat16* p = static_cast<__nv_bfloat16*>(keys ? c.k : c.v) + to;
        *reinterpret_cast<uint4*>(p + off_a) = v[u].a;
        *reinterpret_cast<uint4*>(p + off_b) = v[u].b;
      }
    }
  }
}

// Heads a thread walks: 8 where that leaves 512 threads for each SM, fewer for
// few tokens, where spreading the heads over more threads is what shortens the
// call.
int heads_per_thread(long long lanes, int heads) {  // lanes: threads for each head
  int per = 8;
  while (per > 1 && lanes * ((heads + per - 1) / per) < 152ll * 512) per /= 2;
  return per;
}

template <typename Args, typename F>
cudaError_t launch_rows(Args& a, int lanes, int heads, int parts, F kern, cudaStream_t stream) {
  const long long threads = a.tokens * lanes;
  a.heads_per = heads_per_thread(threads * parts, heads);
  const dim3 grid(static_cast<unsigned>((threads + kRopeThreads - 1) / kRopeThreads),
                  static_cast<unsigned>((heads + a.heads_per - 1) / a.heads_per),
                  static_cast<unsigned>(parts));
  return launch_pdl(kern, grid, dim3(kRopeThreads), 0, stream, a);
}

template <int D>
cudaError_t launch_rope_d(RopeArgs& a, cudaStream_t stream) {
  const int heads = a.H[0] + a.H[1];
  return a.rope.interleaved ? launch_rows(a, D / 16, heads, 1, rope_kernel<D, true>, stream)
                            : launch_rows(a, D / 16, heads, 1, rope_kernel<D, false>, stream);
}

template <int D, bool F8>
cudaError_t launch_append_d(AppendArgs& a, cudaStream_t stream) {
  const int heads = a.cache.H_kv;
  return a.rope.interleaved ? launch_rows(a, D / 16, heads, 2, append_kernel<D, true, F8>, stream)
                            : launch_rows(a, D / 16, heads, 2, append_kernel<D, false, F8>, stream);
}

}  // namespace

cudaError_t launch_rope(RopeArgs& a, int d, cudaStream_t stream) {
  return d == 64 ? launch_rope_d<64>(a, stream) : launch_rope_d<128>(a, stream);
}

cudaError_t launch_append(AppendArgs& a, cudaStream_t stream) {
  const bool f8 = a.cache.type == ATTN_CACHE_E4M3;
  if (a.cache.d == 64)
    return f8 ? launch_append_d<64, true>(a, stream) : launch_append_d<64, false>(a, stream);
  return f8 ? launch_append_d<128, true>(a, stream) : launch_append_d<128, false>(a, stream);
}

}  // namespace eba

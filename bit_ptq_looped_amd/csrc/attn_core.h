// Shared by the decode and prefill kernels of the attention over the paged
// key-value cache: visibility, operands, the layout of tiles in LDS, joining of
// partial results.  attention.hip describes the method.
#pragma once

#include "kv_internal.h"
#include "quant_core.h"

namespace loopq {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4* lds_s16x4;

constexpr int kDecodeGroups = 512;   // work-groups of the decode launch, four pieces each
constexpr int kDecodePieces = kDecodeGroups * 4;
constexpr int kDecodeRows = 16;      // query heads of an item
constexpr int kDecodeKeys = 32;      // keys of a tile
constexpr int kPrefillGroups = 256;  // work-groups of the prefill launch
constexpr int kPrefillSlots = 2 * kPrefillGroups;
constexpr int kPrefillRows = 256;    // (query, head) rows of an item, at most
constexpr int kPrefillKeys = 64;

// A split item: how many parts it has and which.  One record per decode piece
// (of the item whose first part is the piece's last) or per prefill slot (of
// the item whose first part took it); parts is 0 where there is none.
struct __attribute__((aligned(16))) JoinRecord {
  int32_t parts, row, item, tile;
};

// A prefill task: key tiles k0 .. k1 - 1 of a query tile, for one key head.
struct PrefillTask {
  int32_t row, first, n, len;   // the row, its first query, its queries, its tokens
  int32_t tile, lo, hi;         // the query tile, positions of its first and last query
  int32_t head, from;           // its key tiles: `head` from 0, then from `from` on
  int32_t k0, k1;
  int32_t part, parts, slot;    // of the item: this part, all, the first one's slot if there are several
  int32_t pad[2];
};

// what a launch needs beside the caller's arguments
struct AttnPlan {
  float* part;            // partial results: [slot][rows][head_dim], then
  float* ml;              // their m and l: [slot][2][rows]
  JoinRecord* records;
  int32_t* row_tiles;     // prefill: query tiles before each row, [rows + 1]
  PrefillTask* tasks;     // prefill: the tasks of one key head
  int32_t* head;          // prefill: {tasks of a key head, slots of a key head, key heads of a block}
  int32_t* next;          // tasks handed out, of each eighth of the tasks
  int32_t most_tiles;     // prefill: query tiles, at most
  const uint16_t* zeros;  // 256 zero bytes, cleared by the plan launch
  float c;                // |scale| log2(e), or 1 for a scale of 0
  float qmul;             // sign of the scale: queries are taken times this
};

hipError_t launch_attn_decode(const AttnArgs& a, const AttnPlan& pl, hipStream_t s);
hipError_t launch_attn_prefill(const AttnArgs& a, const AttnPlan& pl, hipStream_t s);

__device__ __forceinline__ int row_len(const AttnArgs& a, int row) {
  const int64_t cap = (int64_t)a.width << a.page_shift;
  const int64_t n = a.lens[row];
  return (int)(n < 0 ? 0 : n > cap ? cap : n);
}

// the row's queries: the first and their number, inside [0, queries)
__device__ __forceinline__ int row_queries(const AttnArgs& a, int row, int* first) {
  const int s = min(max(a.cu[row], 0), a.queries);
  const int e = min(max(a.cu[row + 1], s), a.queries);
  *first = s;
  return e - s;
}

// Tiles of 2^shift keys that queries at positions lo .. hi can see: `head`
// tiles from key 0 (sinks), then those from tile `from` on; their number.
struct Tiles {
  int head, from, n;
  __device__ __forceinline__ int at(int i) const { return i < head ? i : from + i - head; }
};
__device__ __forceinline__ Tiles visible_tiles(const AttnArgs& a, int lo, int hi, int shift) {
  Tiles t{0, 0, 0};
  if (hi < 0) return t;
  const int64_t low = a.window > 0 ? max((int64_t)lo - a.window + 1, (int64_t)0) : 0;  // first key in the window
  t.from = (int)(low >> shift);
  t.head = (int)min((int64_t)t.from, ((int64_t)a.sinks + (1 << shift) - 1) >> shift);
  t.n = t.head + (hi >> shift) - t.from + 1;
  return t;
}

// bits 0 .. n - 1
__device__ __forceinline__ uint64_t below(int64_t n) { return n <= 0 ? 0 : n >= 64 ? ~0ull : (1ull << n) - 1; }

// every fourth bit of x, 16 of them
__device__ __forceinline__ uint16_t every_fourth(uint64_t x) {
  x &= 0x1111111111111111ull;
  x = (x | (x >> 3)) & 0x0303030303030303ull;
  x = (x | (x >> 6)) & 0x000f000f000f000full;
  x = (x | (x >> 12)) & 0x000000ff000000ffull;
  return (uint16_t)(x | (x >> 24));
}

__device__ __forceinline__ bool sees(const AttnArgs& a, int p, int j) {
  return j <= p && (a.window == 0 || p - j < a.window || j < a.sinks);
}

// the last i in [0, n) with p[i] <= u
template <class T>
__device__ __forceinline__ int find(const T* p, int n, T u) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p[mid] <= u) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Eight query elements as N bf16 planes of an MFMA operand.  fp32 has three: the
// leading bits cut off twice, and the rest, which 8 bits hold.  No plane has
// another sign than the element, and none is 0 unless the element is (2^-126
// where nothing is left): all planes times an infinite key are that infinity.
template <int N>
__device__ __forceinline__ void query_planes(const u32x4 (&raw)[N == 1 ? 1 : 2], float mul, bf16x8 (&q)[N]) {
  if (N == 1 && mul == 1.0f) {
    q[0] = __builtin_bit_cast(bf16x8, raw[0]);
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float x = mul * (N == 1 ? bf16_bits_to_float(e & 1 ? raw[0][e >> 1] >> 16 : raw[0][e >> 1] & 0xffffu) : __uint_as_float(raw[N > 1 ? e >> 2 : 0][e & 3]));
    const float least = fminf(fabsf(x), 0x1p-126f);
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const float t = n + 1 < N && x == x ? __uint_as_float(__float_as_uint(x) & 0xffff0000u) : x;
      q[n][e] = (__bf16)t;
      x = copysignf(fabsf(t) == INFINITY ? least : fmaxf(fabsf(x - t), least), t);
    }
  }
}
template <int N>
__device__ __forceinline__ void load_query(const AttnArgs& a, float mul, int64_t at, bool in, bf16x8 (&q)[N]) {
  u32x4 raw[N == 1 ? 1 : 2];
#pragma unroll
  for (int x = 0; x < (N == 1 ? 1 : 2); ++x) {
    raw[x] = u32x4{0, 0, 0, 0};
    if (in) raw[x] = *reinterpret_cast<const u32x4*>(reinterpret_cast<const char*>(a.q) + at * (N == 1 ? 2 : 4) + 16 * x);
  }
  query_planes(raw, mul, q);
}

// Eight weights as N bf16 planes: one, rounded to nearest; or the leading bits
// cut off for all but the last, so that no plane is negative, and none 0 unless
// the weight is (2^-126 where nothing is left): every plane times an infinite
// value then is that infinity.
template <int N>
__device__ __forceinline__ void split_weights(const float (&p)[8], bf16x8 (&w)[N]) {
  float x[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = p[e];
#pragma unroll
  for (int n = 0; n < N; ++n) {
    u32x4 b;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      b[e] = n + 1 < N ? __builtin_amdgcn_perm(__float_as_uint(x[2 * e + 1]), __float_as_uint(x[2 * e]), 0x07060302u)
                       : bf16x2_rne(x[2 * e], x[2 * e + 1]);
    w[n] = __builtin_bit_cast(bf16x8, b);
    if (n + 1 < N)
#pragma unroll
      for (int e = 0; e < 8; ++e)
        x[e] = fmaxf(x[e] - __uint_as_float(__float_as_uint(x[e]) & 0xffff0000u), fminf(p[e], 0x1p-126f));
  }
}

template <int N>
struct Planes {
  static constexpr int n = N;
};

// Place of 16-byte chunk ch of a key's row in a tile of 2^LOG keys in LDS:
// blocks of four chunks (32 columns), the key's 64 bytes of each block in one
// run, chunks permuted by the key: reads of one chunk of 16 keys and transposing
// reads of four keys each spread over all banks.  ROWS also permutes the keys by
// the block, which does the same for writes of whole rows.
template <int LOG, bool ROWS>
__device__ __forceinline__ int chunk_at(int key, int ch) {
  return ((ch >> 2) << (LOG + 2)) + ((ROWS ? key ^ ((ch >> 2) & 3) : key) << 2) + ((ch & 3) ^ ((key >> 2) & 3));
}

__device__ __forceinline__ u32x2 read_tr(const u32x4* tile, int chunk, int half) {
  const char* p = reinterpret_cast<const char*>(tile) + chunk * 16 + half * 8;
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(p)));
}

__device__ __forceinline__ bf16x8 join_halves(u32x2 x, u32x2 y) {
  return __builtin_bit_cast(bf16x8, u32x4{x[0], x[1], y[0], y[1]});
}

template <int D>
__device__ __forceinline__ void store_row(const AttnArgs& a, int64_t at, const float (&o)[2], float l) {
  const int lane = threadIdx.x & 63;
  const float f = l > 0.0f || l != l ? 1.0f / l : 0.0f;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int d = lane + 64 * h;
    if (d >= D) break;
    if (a.bf16) reinterpret_cast<uint16_t*>(a.out)[at + d] = (uint16_t)bf16x2_rne(o[h] * f, 0.0f);
    else reinterpret_cast<float*>(a.out)[at + d] = o[h] * f;
  }
}

// Parts first, first + step, ... of n of one row, one wave: columns lane and
// lane + 64 of the sum at the reference m of all n parts, and l.  Bound by trips
// to memory (the parts come from other XCDs), so that the first eight parts are on
// their way before m is known.
template <int D, int ROWS, class F>
__device__ __forceinline__ float join_parts(const AttnPlan& pl, int n, int first, int step, int r, F slot_of, float (&o)[2]) {
  const int lane = threadIdx.x & 63;
  float p[8][2], pm[8], psum[8];
  const auto load = [&](int i0) {  // no branches, so that all are one trip
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const int64_t slot = slot_of(min(i0 + x * step, n - 1));
      const float* at = pl.part + (slot * ROWS + r) * D;
      pm[x] = pl.ml[slot * 2 * ROWS + r];
      psum[x] = pl.ml[(slot * 2 + 1) * ROWS + r];
      p[x][0] = at[lane];
      if (D > 64) p[x][1] = at[min(lane + 64, D - 1)];
    }
  };
  load(first);
  float m = -INFINITY;
  for (int i = lane; i < n; i += 64) m = fmaxf(m, pl.ml[slot_of(i) * 2 * ROWS + r]);
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
  const float ref = m == -INFINITY ? 0.0f : m;
  float l = 0.0f;
  o[0] = o[1] = 0.0f;
  for (int i0 = first; i0 < n; i0 += 8 * step) {
    if (i0 != first) load(i0);
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const bool in = i0 + x * step < n;  // the last part stands in for those past it
      const float f = __builtin_amdgcn_exp2f(pm[x] - ref);
      l = in ? fmaf(f, psum[x], l) : l;
      o[0] = in ? fmaf(f, p[x][0], o[0]) : o[0];
      if (D > 64) o[1] = in ? fmaf(f, p[x][1], o[1]) : o[1];
    }
  }
  return l;
}

// The records among n that stand for an item, into `list` in their order (the
// same in every work-group), with their place; their number.  256 threads, 2048
// records at a time so that they are one trip to memory; ends with a barrier.
struct SplitItem {
  int32_t parts, row, item, tile, at;
};
__device__ __forceinline__ int split_items(const JoinRecord* records, int n, SplitItem* list) {
  __shared__ int count[32];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int base = 0;
  for (int i0 = 0; i0 < n; i0 += 2048) {
    JoinRecord rec[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const int i = i0 + 256 * c + tid;
      rec[c] = i < n ? records[i] : JoinRecord{0, 0, 0, 0};
    }
    uint64_t is[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      is[c] = __ballot(rec[c].parts > 0);
      if (lane == 0) count[4 * c + wave] = __popcll(is[c]);
    }
    __syncthreads();
    const int mine = lane < 32 ? count[lane] : 0;
    int upto = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up(upto, off, 64);
      if (lane >= off) upto += y;
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const int at = base + __shfl(upto - mine, 4 * c + wave, 64) + __popcll(is[c] & ((1ull << lane) - 1));
      if ((is[c] >> lane) & 1) list[at] = SplitItem{rec[c].parts, rec[c].row, rec[c].item, rec[c].tile, i0 + 256 * c + tid};
    }
    base += __shfl(upto, 31, 64);
    __syncthreads();
  }
  return base;
}

}  // namespace loopq

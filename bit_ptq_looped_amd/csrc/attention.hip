// Attention over the paged key-value cache (include/loopq_kv.h): one new token
// a row (decode), or several (prefill), with a sliding window and sinks.
//
// For a query q with the visible keys J:  s_j = scale q . k_j,
// out = sum_J 2^(t_j - m) v_j / sum_J 2^(t_j - m),  t_j = s_j log2(e), m a running
// reference at or near the maximum, all sums in fp32 (one pass over the keys;
// m, l and the sums are rescaled when the reference grows).
//
// Both products run on the bf16 MFMA, transposed: S^T = K Q^T puts a query in a
// column, so its keys lie in the registers of two (four) lanes and the softmax
// needs one (two) lane exchanges; P^T then is the second product's B operand as
// it stands, O^T = V^T P^T, since the order of the summed keys is free as long
// as both operands keep the same: slot e of lane group h holds key
// 4h + e % 4 + 8 (e / 4) of its 16 (prefill), or 4h + e % 4 + 16 (e / 4) of its
// 32 (decode).  V^T comes from the row-major tile in LDS by transposing reads.
// fp32 queries and weights are split into three bf16 planes (24 bits), whose
// products with the bf16 keys and values are exact; bf16 queries are exact
// alone.
//
// Work is cut by length, not by row: the visible key tiles of all (row, key
// head, query tile) items form one line, cut into equal pieces, one per wave
// (decode) or work-group (prefill).  Lengths are read on the device, so ragged
// rows balance and the launch shape never depends on them.  An item that lies
// in one piece is finished there; the others leave (m, l, O) per piece, at most
// two a piece, and a second launch joins them in the order of the keys: the
// result depends on the inputs alone.
#include "kv_internal.h"
#include "quant_core.h"

namespace loopq {
namespace {

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
constexpr int kPrefillGroups = 512;  // work-groups of the prefill launch
constexpr int kPrefillSlots = 2 * kPrefillGroups;
constexpr int kPrefillRows = 128;    // (query, head) rows of an item
constexpr int kPrefillKeys = 64;

// what a launch needs beside the caller's arguments
struct AttnPlan {
  float* part;            // partial results: [slot][rows][head_dim], then
  float* ml;              // their m and l: [slot][2][rows]
  int64_t* row_task;      // prefill: tasks before each row, [rows + 1]
  int64_t* row_slot;      // prefill: slots before each row, [rows + 1]
  int64_t* row_tiles;     // prefill: query tiles before each row, [rows + 1]
  int32_t* tile_task;     // prefill: tasks before each query tile, within its row and key head
  int32_t* tile_slot;     // the same for slots
  int64_t* head;          // prefill: {most key tiles of a task}, then
  int32_t* next;          // tasks handed out, of each eighth of the tasks
  const uint16_t* zeros;  // 256 zero bytes, cleared by the plan launch
  float c;                // |scale| log2(e), or 1 for a scale of 0
  float qmul;             // sign of the scale: queries are taken times this
};

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

// exclusive prefix of n values f(i) into LDS, out[n] their sum (the work-group's
// 256 threads; ends with a barrier)
template <class F>
__device__ __forceinline__ void block_prefix(int n, int64_t* out, F f) {
  __shared__ int64_t part[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int64_t base = 0;
  for (int i0 = 0; i0 < n; i0 += 256) {
    const int i = i0 + tid;
    const int64_t v = i < n ? f(i) : 0;
    int64_t x = v;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int64_t y = __shfl_up(x, off, 64);
      if (lane >= off) x += y;
    }
    if (lane == 63) part[wave] = x;
    __syncthreads();
    int64_t before = base, all = base;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      before += w < wave ? part[w] : 0;
      all += part[w];
    }
    if (i < n) out[i] = before + x - v;
    base = all;
    __syncthreads();
  }
  if (tid == 0) out[n] = base;
  __syncthreads();
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

__device__ __forceinline__ float bf16_of(const void* p, int64_t i, int bf16) {
  return bf16 ? bf16_bits_to_float(reinterpret_cast<const uint16_t*>(p)[i]) : reinterpret_cast<const float*>(p)[i];
}

// eight query elements as N bf16 planes of an MFMA operand
template <int N>
__device__ __forceinline__ void load_query(const AttnArgs& a, float mul, int64_t at, bool in, bf16x8 (&q)[N]) {
  float x[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = 0.0f;
  if (in) {
    if (N == 1) {
      const u32x4 u = *reinterpret_cast<const u32x4*>(reinterpret_cast<const uint16_t*>(a.q) + at);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = mul * bf16_bits_to_float(e & 1 ? u[e >> 1] >> 16 : u[e >> 1] & 0xffffu);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = mul * reinterpret_cast<const float*>(a.q)[at + e];
    }
  }
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      q[n][e] = (__bf16)x[e];
      x[e] -= (float)q[n][e];
    }
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

// ------------------------------------------------------------------- decode

__device__ __forceinline__ void decode_prefix(const AttnArgs& a, int items, int64_t* prefix) {
  block_prefix(a.rows, prefix, [&](int r) {
    const int p = row_len(a, r) - 1;
    return (int64_t)visible_tiles(a, p, p, 5).n * items;
  });
}

__device__ __forceinline__ int64_t decode_piece(int64_t total) {
  const int64_t n = (total + kDecodePieces - 1) / kDecodePieces;
  return n < 2 ? 2 : n;
}

template <int D, bool F32>
__global__ __launch_bounds__(256, 2) void decode_attn_kernel(AttnArgs a, AttnPlan pl) {
  constexpr int NQ = F32 ? 3 : 1, NP = F32 ? 3 : 2;
  constexpr int C = D / 8;               // chunks of a row
  constexpr int NV = kDecodeKeys * C / 64;  // chunks of a tile per lane
  __shared__ u32x4 s_v[4][kDecodeKeys * C];
  extern __shared__ int64_t s_prefix[];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n16 = lane & 15, g = lane >> 4;
  const int gts = (a.group + kDecodeRows - 1) / kDecodeRows, items = a.heads * gts;
  decode_prefix(a, items, s_prefix);
  const int64_t total = s_prefix[a.rows], piece = decode_piece(total);
  const int idx = (int)blockIdx.x * 4 + wave;
  int64_t u = idx * piece;
  const int64_t u_end = min(u + piece, total);
  u32x4* tile = s_v[wave];

  while (u < u_end) {
    const int row = find(s_prefix, a.rows, u);
    const int len = row_len(a, row), pos = len - 1;
    const Tiles tl = visible_tiles(a, pos, pos, 5);
    const int item = (int)((u - s_prefix[row]) / tl.n);
    const int64_t i0 = s_prefix[row] + (int64_t)item * tl.n;
    const int first = (int)(u - i0), last = (int)(min(u_end - i0, (int64_t)tl.n));  // tiles of this piece
    const int kvh = item / gts, gt = item - kvh * gts;
    const int head = gt * kDecodeRows + n16;  // in the group
    const bool has = head < a.group;
    const int hq = kvh * a.group + head;
    const int32_t* table = a.table + (int64_t)row * a.width;

    bf16x8 q[D / 32][NQ];
#pragma unroll
    for (int c = 0; c < D / 32; ++c)
      load_query<NQ>(a, pl.qmul, row * a.ldq + (int64_t)hq * D + 32 * c + 8 * g, has, q[c]);

    f32x4 o[D / 16];
#pragma unroll
    for (int d = 0; d < D / 16; ++d) o[d] = f32x4{0, 0, 0, 0};
    float m = -INFINITY, l = 0.0f;

    // lane x (mod 32) looks after key x of a tile: its page, or -1 if it is hidden
    const auto page_of = [&](int i) {
      const int j = (tl.at(i) << 5) + (lane & 31);
      int page = -1;
      if (sees(a, pos, j)) {
        page = table[j >> a.page_shift];
      }
      return page;  // as it stands in the table: the load is not waited for here
    };
    const auto real = [&](int page) { return (uint32_t)page < (uint32_t)a.num_pages ? page : -1; };
    u32x4 kr[2][D / 32], vr[NV];
    const auto load_tile = [&](int i, int page) {
      const int j0 = tl.at(i) << 5;
      const int in_page = (1 << a.page_shift) - 1;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int key = 16 * t + n16, pg = __shfl(page, key, 64);
        const uint16_t* p = a.pool + pg * a.page_stride + (((int64_t)kvh << a.page_shift) + ((j0 + key) & in_page)) * D + 8 * g;
        if (pg >= 0)
#pragma unroll
          for (int c = 0; c < D / 32; ++c) kr[t][c] = *reinterpret_cast<const u32x4*>(p + 32 * c);
      }
#pragma unroll
      for (int x = 0; x < NV; ++x) {
        const int at = lane + 64 * x, key = at / C, ch = at - key * C, pg = __shfl(page, key, 64);
        const uint16_t* p = a.pool + a.plane + pg * a.page_stride +
                            (((int64_t)kvh << a.page_shift) + ((j0 + key) & in_page)) * D + 8 * ch;
        vr[x] = u32x4{0, 0, 0, 0};  // a hidden key's values count for nothing, whatever they hold
        if (pg >= 0) vr[x] = *reinterpret_cast<const u32x4*>(p);
      }
    };

    int page = real(page_of(first));
    uint32_t seen = (uint32_t)__ballot(page >= 0);
    load_tile(first, page);
    page = first + 1 < last ? page_of(first + 1) : -1;
    for (int i = first; i < last; ++i) {
      // S^T: rows 4 g + r of key tile t, column n16
      f32x4 s[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        s[t] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int c = 0; c < D / 32; ++c)
#pragma unroll
          for (int n = NQ - 1; n >= 0; --n)
            s[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, kr[t][c]), q[c][n], s[t], 0, 0, 0);
      }
      // V to LDS, then the next tile's loads
#pragma unroll
      for (int x = 0; x < NV; ++x) {
        const int at = lane + 64 * x, key = at / C, ch = at - key * C;
        tile[chunk_at<5, true>(key, ch)] = vr[x];
      }
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      const uint32_t now = seen;
      if (i + 1 < last) {
        page = real(page);
        seen = (uint32_t)__ballot(page >= 0);
        load_tile(i + 1, page);
        page = i + 2 < last ? page_of(i + 2) : -1;
      }
      if (now != 0xffffffffu) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (!((now >> (16 * t + 4 * g + r)) & 1)) s[t][r] = -INFINITY;
      }
      float top = fmaxf(fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[0][2], s[0][3])),
                        fmaxf(fmaxf(s[1][0], s[1][1]), fmaxf(s[1][2], s[1][3])));
      top = fmaxf(top, __shfl_xor(top, 16, 64));
      top = fmaxf(top, __shfl_xor(top, 32, 64));
      top *= pl.c;
      if (__any(top > m)) {
        const float mn = fmaxf(m, top);
        const float f = __builtin_amdgcn_exp2f(m - (mn == -INFINITY ? 0.0f : mn));
        m = mn;
        l *= f;
#pragma unroll
        for (int d = 0; d < D / 16; ++d) o[d] *= f;
      }
      const float ref = m == -INFINITY ? 0.0f : m;
      float p[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        p[e] = __builtin_amdgcn_exp2f(fmaf(s[e >> 2][e & 3], pl.c, -ref));
        l += p[e];
      }
      bf16x8 w[NP];
      split_weights<NP>(p, w);
#pragma unroll
      for (int d = 0; d < D / 16; ++d) {
        const int x = lane & 15, key = 4 * g + (x >> 2), ch = 2 * d + ((x & 3) >> 1);
        const bf16x8 vt = join_halves(read_tr(tile, chunk_at<5, true>(key, ch), x & 1), read_tr(tile, chunk_at<5, true>(key + 16, ch), x & 1));
#pragma unroll
        for (int n = NP - 1; n >= 0; --n) o[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vt, w[n], o[d], 0, 0, 0);
      }
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
    l += __shfl_xor(l, 16, 64);
    l += __shfl_xor(l, 32, 64);
    if (first == 0 && last == tl.n) {
      const float f = l > 0.0f || l != l ? 1.0f / l : 0.0f;
      if (has) {
        const int64_t at = row * a.ldo + (int64_t)hq * D + 4 * g;
#pragma unroll
        for (int d = 0; d < D / 16; ++d) {
          const f32x4 r = o[d] * f;
          if (a.bf16)
            *reinterpret_cast<u32x2*>(reinterpret_cast<uint16_t*>(a.out) + at + 16 * d) = u32x2{bf16x2_rne(r[0], r[1]), bf16x2_rne(r[2], r[3])};
          else
            *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(a.out) + at + 16 * d) = r;
        }
      }
    } else if (has) {
      const int64_t slot = (int64_t)idx * 2 + (first == 0 && u != idx * piece ? 1 : 0);
      float* dst = pl.part + (slot * kDecodeRows + n16) * D + 4 * g;
#pragma unroll
      for (int d = 0; d < D / 16; ++d) *reinterpret_cast<f32x4*>(dst + 16 * d) = o[d];
      if (g == 0) {
        pl.ml[slot * 2 * kDecodeRows + n16] = m;
        pl.ml[(slot * 2 + 1) * kDecodeRows + n16] = l;
      }
    }
    u = i0 + last;
  }
  // rows without a visible key belong to no piece
  if (blockIdx.x == 0)
    for (int r = 0; r < a.rows; ++r)
      if (s_prefix[r + 1] == s_prefix[r])
        for (int d = tid; d < a.heads * a.group * D; d += 256) {
          if (a.bf16) reinterpret_cast<uint16_t*>(a.out)[r * a.ldo + d] = 0;
          else reinterpret_cast<float*>(a.out)[r * a.ldo + d] = 0.0f;
        }
}

// Joins the n parts of one item for one of its rows, one wave: columns lane and
// lane + 64 of the result (unscaled by 1 / l) and l.
template <int D, int ROWS, class F>
__device__ __forceinline__ float join_row(const AttnPlan& pl, int n, int r, F slot_of, float (&o)[2]) {
  const int lane = threadIdx.x & 63;
  float m = -INFINITY;
  for (int i = lane; i < n; i += 64) m = fmaxf(m, pl.ml[slot_of(i) * 2 * ROWS + r]);
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
  const float ref = m == -INFINITY ? 0.0f : m;
  float l = 0.0f;
  o[0] = o[1] = 0.0f;
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const int64_t slot = slot_of(i);
    const float f = __builtin_amdgcn_exp2f(pl.ml[slot * 2 * ROWS + r] - ref);
    const float* p = pl.part + (slot * ROWS + r) * D;
    l = fmaf(f, pl.ml[(slot * 2 + 1) * ROWS + r], l);
    o[0] = fmaf(f, p[lane], o[0]);
    if (D > 64) o[1] = fmaf(f, lane + 64 < D ? p[lane + 64] : 0.0f, o[1]);
  }
  return l;
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

// One work-group per cut between two pieces; the first cut inside an item joins it.
template <int D>
__global__ __launch_bounds__(256) void decode_join_kernel(AttnArgs a, AttnPlan pl) {
  extern __shared__ int64_t s_prefix[];
  const int gts = (a.group + kDecodeRows - 1) / kDecodeRows, items = a.heads * gts;
  decode_prefix(a, items, s_prefix);
  const int64_t total = s_prefix[a.rows], piece = decode_piece(total);
  const int64_t cut = ((int64_t)blockIdx.x + 1) * piece;
  if (cut >= total) return;
  const int row = find(s_prefix, a.rows, cut);
  const int64_t n = (s_prefix[row + 1] - s_prefix[row]) / items;
  const int item = (int)((cut - s_prefix[row]) / n);
  const int64_t i0 = s_prefix[row] + item * n, w0 = i0 / piece;
  if (i0 == cut || w0 != blockIdx.x) return;
  const int64_t w1 = (i0 + n - 1) / piece;
  const int kvh = item / gts, gt = item - kvh * gts;
  for (int r = threadIdx.x >> 6; r < min(kDecodeRows, a.group - gt * kDecodeRows); r += 4) {
    float o[2];
    const int64_t slot0 = w0 * 2 + (i0 != w0 * piece);
    const float l = join_row<D, kDecodeRows>(pl, (int)(w1 - w0) + 1, r, [&](int i) { return i ? (w0 + i) * 2 : slot0; }, o);
    store_row<D>(a, row * a.ldo + (int64_t)(kvh * a.group + gt * kDecodeRows + r) * D, o, l);
  }
}

// ------------------------------------------------------------------ prefill

// Rows of a query tile are (query, head of the group) pairs, heads fastest.
__device__ __forceinline__ int query_tiles(const AttnArgs& a, int n) {
  return (int)(((int64_t)n * a.group + kPrefillRows - 1) / kPrefillRows);
}
__device__ __forceinline__ Tiles tile_keys(const AttnArgs& a, int t, int n, int len, int* lo, int* hi) {
  const int64_t r0 = (int64_t)t * kPrefillRows, r1 = min(r0 + kPrefillRows, (int64_t)n * a.group) - 1;
  *lo = len - n + (int)(r0 / a.group);
  *hi = len - n + (int)(r1 / a.group);
  return visible_tiles(a, *lo, *hi, 6);
}

// the larger of lanes x and x + 32, in both
__device__ __forceinline__ float max_halves(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// x of the wave's first lane, as a scalar
__device__ __forceinline__ int64_t uniform(int64_t x) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)x), hi = __builtin_amdgcn_readfirstlane((uint32_t)(x >> 32));
  return (int64_t)(((uint64_t)hi << 32) | lo);
}

// inclusive sum over the wave
__device__ __forceinline__ int64_t wave_sum(int64_t x) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int64_t y = __shfl_up(x, off, 64);
    if (lane >= off) x += y;
  }
  return x;
}

// p[0 .. n) to its exclusive prefix, p[n] the sum, by 1024 threads; barriers on both sides
__device__ __forceinline__ int64_t prefix_in_place(int64_t* p, int n) {
  __shared__ int64_t part[16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int64_t base = 0;
  __syncthreads();
  for (int i0 = 0; i0 < n; i0 += 1024) {
    const int i = i0 + tid;
    const int64_t v = i < n ? p[i] : 0, x = wave_sum(v);
    if (lane == 63) part[wave] = x;
    __syncthreads();
    int64_t before = base;
    for (int w = 0; w < 16; ++w) {
      before += w < wave ? part[w] : 0;
      base += part[w];
    }
    if (i < n) p[i] = before + x - v;
    __syncthreads();
  }
  if (tid == 0) p[n] = base;
  __syncthreads();
  return base;
}

// One work-group.  A task is an item or, where an item has more than L key
// tiles, a part of it of at most L; L is a work-group's even share of all key
// tiles, so that few long items are split over the whole chip and many stay
// whole.  Slots take the results of split items' tasks: at most 2 tiles / L.
__global__ __launch_bounds__(1024) void prefill_plan_kernel(AttnArgs a, AttnPlan pl) {
  __shared__ unsigned long long s_sum;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (tid < 64) reinterpret_cast<uint32_t*>(const_cast<uint16_t*>(pl.zeros))[tid] = 0;
  if (tid < 8) pl.next[tid] = 0;
  if (tid == 0) s_sum = 0;
  for (int r = tid; r < a.rows; r += 1024) {
    int first;
    pl.row_tiles[r] = query_tiles(a, row_queries(a, r, &first));
  }
  prefix_in_place(pl.row_tiles, a.rows);
  for (int pass = 0; pass < 2; ++pass) {
    const int64_t L = pass ? pl.head[0] : 0;
    for (int r = wave; r < a.rows; r += 16) {  // a wave per row
      int first;
      const int n = row_queries(a, r, &first), len = row_len(a, r), qt = query_tiles(a, n);
      int64_t tasks = 0, slots = 0;
      for (int t0 = 0; t0 < qt; t0 += 64) {
        const int t = t0 + lane;
        int lo, hi;
        const int64_t keys = t < qt ? tile_keys(a, t, n, len, &lo, &hi).n : 0;
        if (pass == 0) {
          tasks += keys;
        } else {
          const int64_t parts = (keys + L - 1) / L, x = wave_sum(parts), y = wave_sum(parts > 1 ? parts : 0);
          if (t < qt) {
            pl.tile_task[pl.row_tiles[r] + t] = (int32_t)(tasks + x - parts);
            pl.tile_slot[pl.row_tiles[r] + t] = (int32_t)(slots + y - (parts > 1 ? parts : 0));
          }
          tasks += __shfl(x, 63, 64);
          slots += __shfl(y, 63, 64);
        }
      }
      if (pass == 0) {
        const int64_t x = wave_sum(tasks);
        if (lane == 63) atomicAdd(&s_sum, (unsigned long long)(x * a.heads));
      } else if (lane == 0) {
        pl.row_task[r] = tasks * a.heads;
        pl.row_slot[r] = slots * a.heads;
      }
    }
    __syncthreads();
    if (pass == 0 && tid == 0) pl.head[0] = max((int64_t)4, ((int64_t)s_sum + kPrefillGroups - 1) / kPrefillGroups);
    __syncthreads();
  }
  prefix_in_place(pl.row_task, a.rows);
  prefix_in_place(pl.row_slot, a.rows);
}

struct PrefillItem {
  int row, kvh, tile, part, n, len, first;  // first: the row's first query
  int lo, hi;                               // positions of the tile's queries
  Tiles tl;
  int from, to;                             // key tiles of the task
  int64_t slot;                             // of the item's first task, if there are several
};
// Task x by the prefixes of tasks, or of slots.  Within a key head the query
// tiles go from the last to the first, which has the fewest keys.
__device__ __forceinline__ PrefillItem prefill_item(const AttnArgs& a, const AttnPlan& pl, int64_t x, bool by_slot) {
  PrefillItem it;
  const int64_t* rows = by_slot ? pl.row_slot : pl.row_task;
  it.row = find(rows, a.rows, x);
  it.n = row_queries(a, it.row, &it.first);
  it.len = row_len(a, it.row);
  const int64_t per = (rows[it.row + 1] - rows[it.row]) / a.heads;
  x -= rows[it.row];
  it.kvh = (int)(x / per);
  x -= it.kvh * per;
  if (!by_slot) x = per - 1 - x;
  const int64_t t0 = pl.row_tiles[it.row];
  const int32_t* before = (by_slot ? pl.tile_slot : pl.tile_task) + t0;
  it.tile = find(before, (int)(pl.row_tiles[it.row + 1] - t0), (int32_t)x);
  it.part = (int)x - before[it.tile];
  it.tl = tile_keys(a, it.tile, it.n, it.len, &it.lo, &it.hi);
  const int64_t L = pl.head[0];
  it.from = (int)(it.part * L);
  it.to = (int)min((it.part + 1) * L, (int64_t)it.tl.n);
  it.slot = pl.row_slot[it.row] + it.kvh * ((pl.row_slot[it.row + 1] - pl.row_slot[it.row]) / a.heads) + pl.tile_slot[t0 + it.tile];
  return it;
}

// The next task for a work-group of eighth e, or -1: each XCD has an eighth of
// the tasks (neighbours share keys, and with them an L2), then helps out in the
// others.  Which work-group takes a task does not change its result.
__device__ __forceinline__ int64_t next_task(const AttnPlan& pl, int64_t tasks, int* e, int* tries) {
  for (; *tries < 8; ++*tries, *e = (*e + 1) & 7) {
    const int64_t lo = tasks * *e / 8, hi = tasks * (*e + 1) / 8;
    const int64_t x = lo + atomicAdd(pl.next + *e, 1);
    if (x < hi) return x;
  }
  return -1;
}

// 16 bytes per lane from src + OFF (bytes, per lane) to LDS at byte dst + 16
// lane (dst a scalar), without passing the registers.  The compiler does not see the write: a
// reader waits for loads_done() and the barrier after it.  The offset counts for
// the target, too; one wait state lies between the write of m0 and its use.
template <int OFF>
__device__ __forceinline__ void load_lds16(const void* src, uint32_t dst) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off offset:%2" ::"s"(dst - OFF), "v"(src), "n"(OFF)
               : "memory", "m0");
}
__device__ __forceinline__ uint32_t lds_offset(const void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
}
__device__ __forceinline__ void loads_done() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

__device__ __forceinline__ bool finite_bf16x2(uint32_t w) {
  return (w & 0x7f80u) != 0x7f80u && (w & 0x7f800000u) != 0x7f800000u;
}

// whether every key of a tile of 64 has a page
__device__ __forceinline__ bool tile_has_pages(const AttnArgs& a, const int32_t* table, int tile) {
  bool ok = true;
  for (int j = tile << 6; j < (tile + 1) << 6; j += min(64, 1 << a.page_shift))
    ok &= (uint32_t)table[j >> a.page_shift] < (uint32_t)a.num_pages;
  return ok;
}

// A work-group takes 128 rows, 32 a wave, over tiles of 64 keys; K and V of the
// next tile are on their way to LDS while this one is multiplied.  Keys that no
// query of the item sees are read from a line of zeros.
template <int D, bool F32>
__global__ __launch_bounds__(256, F32 ? 1 : 2) void prefill_attn_kernel(AttnArgs a, AttnPlan pl) {
  constexpr int NQ = F32 ? 3 : 1;
  constexpr int C = D / 8, S = D / 32;  // chunks and blocks of a row
  constexpr int kTile = kPrefillKeys * C;
  __shared__ u32x4 s_k[2 * kTile], s_v[2 * kTile];
  __shared__ __attribute__((aligned(8))) uint16_t s_valid[2][4];  // keys of a tile that some query sees, 16 a wave
  __shared__ int64_t s_task;
  __shared__ int s_bad;  // a tile that some query sees in part had a value that is not finite
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n32 = lane & 31, h = lane >> 5;
  const int64_t tasks = pl.row_task[a.rows];
  const int in_page = (1 << a.page_shift) - 1;
  int eighth = blockIdx.x & 7, tries = 0;  // work-groups go round the eight XCDs

  // this lane's share of a tile's copy: its key, and a chunk of each block
  const int wave0 = __builtin_amdgcn_readfirstlane(wave);
  const uint32_t to_k = lds_offset(s_k) + wave0 * 1024, to_v = lds_offset(s_v) + wave0 * 1024;
  const int my_key = wave * 16 + (lane >> 2), my_off = 8 * ((lane & 3) ^ (lane >> 4));
  // chunks this lane multiplies
  int k_at[D / 16], v_at[S][2];
#pragma unroll
  for (int c = 0; c < D / 16; ++c) k_at[c] = chunk_at<6, false>(n32, 2 * c + h);
  {
    const int x = lane & 15, g = lane >> 4;
#pragma unroll
    for (int d = 0; d < S; ++d)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        v_at[d][e] = chunk_at<6, false>(4 * h + 8 * e + (x >> 2), 4 * d + 2 * (g & 1) + ((x & 3) >> 1)) * 2 + (x & 1);
  }

  for (;;) {
    if (tid == 0) {
      s_task = next_task(pl, tasks, &eighth, &tries);
      s_bad = 0;
    }
    __syncthreads();
    const int64_t task = uniform(s_task);
    if (task < 0) return;
    const PrefillItem it = prefill_item(a, pl, task, false);
    const int first = it.from, last = it.to;
    const int32_t* table = a.table + (int64_t)it.row * a.width;
    const int64_t rows = (int64_t)it.n * a.group;
    const int64_t rr = (int64_t)it.tile * kPrefillRows + wave * 32 + n32;
    const bool has = rr < rows;
    const int64_t rq = has ? rr : rows - 1;
    const int qi = (int)(rq / a.group), hq = it.kvh * a.group + (int)(rq - (int64_t)qi * a.group);
    const int pos = it.len - it.n + qi;  // position of this lane's query
    // bf16 weights are rounded by up to 2^-8 of themselves; over many keys that
    // averages out, with few the weights take a second plane
    const bool few = !F32 && (it.lo < 255 || (a.window > 0 && a.window < 256));

    bf16x8 q[D / 16][NQ];
#pragma unroll
    for (int c = 0; c < D / 16; ++c)
      load_query<NQ>(a, pl.qmul, (int64_t)(it.first + qi) * a.ldq + (int64_t)hq * D + 16 * c + 8 * h, true, q[c]);

    f32x16 o[S];
#pragma unroll
    for (int d = 0; d < S; ++d)
#pragma unroll
      for (int r = 0; r < 16; ++r) o[d][r] = 0.0f;
    float m = -INFINITY, l = 0.0f;

    // page of this lane's key of tile i, -1 if no query of the item sees the key
    const auto page_of = [&](int i) {
      const int j = (it.tl.at(i) << 6) + my_key;
      int page = -1;
      if (j <= it.hi && (a.window == 0 || it.lo - j < a.window || j < a.sinks)) page = table[j >> a.page_shift];
      return page;  // as it stands in the table: the load is not waited for here
    };
    const auto copy_tile = [&](int i, int page, int buf) {
      const bool in = (uint32_t)page < (uint32_t)a.num_pages;
      const unsigned long long there = __ballot(in);
      if (lane == 0) s_valid[buf][wave] = every_fourth(there);
      const int j = (it.tl.at(i) << 6) + my_key;
      const uint16_t* k = a.pool + (uint32_t)page * a.page_stride + (((int64_t)it.kvh << a.page_shift) + (j & in_page)) * D + my_off;
      const uint16_t* v = k + a.plane;
      if (!in) k = v = pl.zeros;
      const uint32_t dk = to_k + buf * (kTile * 16), dv = to_v + buf * (kTile * 16);
      load_lds16<0>(k, dk);
      load_lds16<64>(k, dk + 4096);
      if (S > 2) load_lds16<128>(k, dk + 8192);
      if (S > 3) load_lds16<192>(k, dk + 12288);
      load_lds16<0>(v, dv);
      load_lds16<64>(v, dv + 4096);
      if (S > 2) load_lds16<128>(v, dv + 8192);
      if (S > 3) load_lds16<192>(v, dv + 12288);
    };
    const auto all_see = [&](int j0) {
      return j0 + 63 <= it.lo && (a.window == 0 || it.hi - j0 < a.window || j0 + 63 < a.sinks);
    };
    const auto run_tiles = [&](auto planes) {
    constexpr int NP = decltype(planes)::n;
    int page = page_of(first);
    copy_tile(first, page, 0);
    page = first + 1 < last ? page_of(first + 1) : -1;
    int buf = 0;
    for (int i = first; i < last; ++i, buf ^= 1) {
      const int j0 = it.tl.at(i) << 6;
      loads_done();
      __syncthreads();
      const uint64_t valid = (uint64_t)uniform(*reinterpret_cast<const int64_t*>(s_valid[buf]));
      // every query of the item sees every key of the tile
      const bool whole = valid == ~0ull && all_see(j0);
      if (!whole) {
        // A weight of 0 does not keep out a value that is infinite or NaN:
        // such values leave the tile here, and reach the queries that see them
        // at the item's end.
#pragma unroll
        for (int x = 0; x < kTile / 256; ++x) {
          const int at = tid + 256 * x;
          u32x4 v = s_v[buf * kTile + at];
          bool fix = false;
#pragma unroll
          for (int e = 0; e < 4; ++e) fix |= !finite_bf16x2(v[e]);
          if (fix) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if ((v[e] & 0x7f80u) == 0x7f80u) v[e] &= 0xffff0000u;
              if ((v[e] & 0x7f800000u) == 0x7f800000u) v[e] &= 0xffffu;
            }
            s_v[buf * kTile + at] = v;
            s_bad = 1;
          }
        }
        __syncthreads();
      }
      if (i + 1 < last) {
        const int next = page;
        page = i + 2 < last ? page_of(i + 2) : -1;
        copy_tile(i + 1, next, buf ^ 1);
      }
      __builtin_amdgcn_sched_barrier(0);
      const u32x4 *kt = s_k + buf * kTile, *vt = s_v + buf * kTile;
      // all reads of K ahead of its products
      u32x4 kf[D / 16][2];
#pragma unroll
      for (int c = 0; c < D / 16; ++c)
#pragma unroll
        for (int t = 0; t < 2; ++t) kf[c][t] = kt[k_at[c] + t * 128];
      __builtin_amdgcn_sched_barrier(0);
      f32x16 s[2];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) s[t][r] = 0.0f;
#pragma unroll
      for (int c = 0; c < D / 16; ++c)
#pragma unroll
        for (int n = NQ - 1; n >= 0; --n)
#pragma unroll
          for (int t = 0; t < 2; ++t)
            s[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, kf[c][t]), q[c][n], s[t], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
      // V of the first two key quarters while the products finish
      bf16x8 vf[2][S];
      const auto read_v = [&](int kc) {
#pragma unroll
        for (int d = 0; d < S; ++d)
          vf[kc & 1][d] = join_halves(read_tr(vt, (v_at[d][0] >> 1) + kc * 64, v_at[d][0] & 1),
                                      read_tr(vt, (v_at[d][1] >> 1) + kc * 64, v_at[d][1] & 1));
      };
      read_v(0);
      read_v(1);
      __builtin_amdgcn_sched_barrier(0);
      if (!whole) {
        uint64_t seen = below(pos - j0 + 1) & valid;
        if (a.window > 0) seen &= ~below((int64_t)pos - a.window + 1 - j0) | below((int64_t)a.sinks - j0);
        seen >>= 4 * h;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const uint32_t w = (uint32_t)(seen >> (32 * t));
#pragma unroll
          for (int r = 0; r < 16; ++r)
            if (!(w & (1u << (8 * (r >> 2) + (r & 3))))) s[t][r] = -INFINITY;
        }
      }
      float top = s[0][0];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int r = 0; r < 16; ++r) top = fmaxf(top, s[t][r]);
      top = max_halves(top) * pl.c;
      // the reference follows only when it is left far behind: weights up to 2^8
      // are as exact, and rescaling costs a pass over o
      if (__any(top > m + 8.0f)) {
        const float mn = fmaxf(m, top);
        const float f = __builtin_amdgcn_exp2f(m - (mn == -INFINITY ? 0.0f : mn));
        m = mn;
        l *= f;
#pragma unroll
        for (int d = 0; d < S; ++d) o[d] *= f;
      }
      const float ref = m == -INFINITY ? 0.0f : m;
      bf16x8 w[2][NP];
      const auto weights = [&](int kc) {
        float p[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          p[e] = __builtin_amdgcn_exp2f(fmaf(s[kc >> 1][8 * (kc & 1) + e], pl.c, -ref));
          if (NP > 1) l += p[e];
        }
        split_weights<NP>(p, w[kc & 1]);
        if (NP == 1) {  // the sum of the rounded weights: what rounding does to all of them alike cancels
          typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
          const bf16x2 one = {(__bf16)1.0f, (__bf16)1.0f};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            l = __builtin_amdgcn_fdot2_f32_bf16(bf16x2{w[kc & 1][0][2 * e], w[kc & 1][0][2 * e + 1]}, one, l, false);
        }
      };
      weights(0);
      __builtin_amdgcn_sched_barrier(0);
      // the next quarter's weights are formed beside this one's products
#pragma unroll
      for (int kc = 0; kc < 4; ++kc) {
        if (kc < 3) weights(kc + 1);
#pragma unroll
        for (int d = 0; d < S; ++d)
#pragma unroll
          for (int n = NP - 1; n >= 0; --n) o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf[kc & 1][d], w[kc & 1][n], o[d], 0, 0, 0);
        if (kc < 2) read_v(kc + 2);
        if (NP == 1 && kc < 3) {
#pragma unroll
          for (int d = 0; d < S; ++d) {
            __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);    // a product,
            __builtin_amdgcn_sched_group_barrier(0x402, 7, 0);  // its share of the vector work
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    };
    if constexpr (F32) run_tiles(Planes<3>());
    else if (few) run_tiles(Planes<2>());
    else run_tiles(Planes<1>());
    __syncthreads();  // the next item's first tile goes over a buffer that may still be read
    if (s_bad) {
      for (int j = it.tl.at(first) << 6; j <= it.hi; ++j) {
        const int tile = j >> 6, i = tile < it.tl.head ? tile : tile - it.tl.from + it.tl.head;
        if ((tile >= it.tl.head && tile < it.tl.from) || i < first || i >= last) continue;
        const int page = table[j >> a.page_shift];
        // a tile that every query saw whole kept its values
        if ((uint32_t)page >= (uint32_t)a.num_pages || !sees(a, pos, j)) continue;
        if (all_see(tile << 6) && tile_has_pages(a, table, tile)) continue;
        const uint16_t* v = a.pool + a.plane + page * a.page_stride + (((int64_t)it.kvh << a.page_shift) + (j & in_page)) * D + 4 * h;
#pragma unroll
        for (int d = 0; d < S; ++d)
#pragma unroll
          for (int r = 0; r < 16; r += 4) {
            const u32x2 y = *reinterpret_cast<const u32x2*>(v + 32 * d + 2 * r);
            if (finite_bf16x2(y[0]) && finite_bf16x2(y[1])) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float z = bf16_bits_to_float(e & 1 ? y[e >> 1] >> 16 : y[e >> 1] & 0xffffu);
              if (!(fabsf(z) < INFINITY)) o[d][r + e] += z;
            }
          }
      }
    }
    __syncthreads();
    l += __shfl_xor(l, 32, 64);
    if (first == 0 && last == it.tl.n) {
      const float f = l > 0.0f || l != l ? 1.0f / l : 0.0f;
      if (has) {
        const int64_t at = (int64_t)(it.first + qi) * a.ldo + (int64_t)hq * D + 4 * h;
#pragma unroll
        for (int d = 0; d < S; ++d)
#pragma unroll
          for (int r = 0; r < 16; r += 4) {
            const f32x4 v = f32x4{o[d][r], o[d][r + 1], o[d][r + 2], o[d][r + 3]} * f;
            if (a.bf16)
              *reinterpret_cast<u32x2*>(reinterpret_cast<uint16_t*>(a.out) + at + 32 * d + 2 * r) = u32x2{bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3])};
            else
              *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(a.out) + at + 32 * d + 2 * r) = v;
          }
      }
    } else {
      const int64_t slot = it.slot + it.part;
      const int r0 = wave * 32 + n32;
      float* dst = pl.part + (slot * kPrefillRows + r0) * D + 4 * h;
#pragma unroll
      for (int d = 0; d < S; ++d)
#pragma unroll
        for (int r = 0; r < 16; r += 4)
          *reinterpret_cast<f32x4*>(dst + 32 * d + 2 * r) = f32x4{o[d][r], o[d][r + 1], o[d][r + 2], o[d][r + 3]};
      if (h == 0) {
        pl.ml[slot * 2 * kPrefillRows + r0] = m;
        pl.ml[(slot * 2 + 1) * kPrefillRows + r0] = l;
      }
    }
  }
}

// Joins split items (grid.x: slots, an item's first one joins it; grid.y: quarters of the rows),
// and clears rows whose query tile no key tile belongs to.
template <int D>
__global__ __launch_bounds__(256) void prefill_join_kernel(AttnArgs a, AttnPlan pl) {
  const int wave = threadIdx.x >> 6;
  if (blockIdx.x < pl.row_slot[a.rows]) {
    const PrefillItem it = prefill_item(a, pl, blockIdx.x, true);
    if (it.part == 0) {
      const int64_t slot = it.slot, L = pl.head[0];
      const int parts = (int)((it.tl.n + L - 1) / L);
      for (int r = blockIdx.y * 32 + wave; r < (int)blockIdx.y * 32 + 32; r += 4) {
        const int64_t rr = (int64_t)it.tile * kPrefillRows + r;
        if (rr >= (int64_t)it.n * a.group) break;
        float o[2];
        const float l = join_row<D, kPrefillRows>(pl, parts, r, [&](int i) { return slot + i; }, o);
        const int qi = (int)(rr / a.group), hq = it.kvh * a.group + (int)(rr - (int64_t)qi * a.group);
        store_row<D>(a, (int64_t)(it.first + qi) * a.ldo + (int64_t)hq * D, o, l);
      }
    }
  }
  // queries at negative positions whose whole tile sees nothing
  for (int row = blockIdx.x * 4 + blockIdx.y; row < a.rows; row += gridDim.x * 4) {
    int first;
    const int n = row_queries(a, row, &first), len = row_len(a, row);
    if (n <= len) continue;
    for (int t = 0; t < query_tiles(a, n); ++t) {
      int lo, hi;
      if (tile_keys(a, t, n, len, &lo, &hi).n > 0) break;
      const int q0 = (int)((int64_t)t * kPrefillRows / a.group);
      const int64_t r1 = min(((int64_t)t + 1) * kPrefillRows, (int64_t)n * a.group);
      (void)q0;
      for (int64_t r = (int64_t)t * kPrefillRows + wave; r < r1; r += 4) {
        const int qi = (int)(r / a.group), g = (int)(r - (int64_t)qi * a.group);
        const float z[2] = {0.0f, 0.0f};
        for (int kvh = 0; kvh < a.heads; ++kvh)
          store_row<D>(a, (int64_t)(first + qi) * a.ldo + (int64_t)(kvh * a.group + g) * D, z, 0.0f);
      }
    }
  }
}

struct AttnSizes {
  size_t part, ml, row, tile;
  size_t all() const { return part + ml + 3 * row + 2 * tile + 512; }
};
size_t up256(int64_t b) { return (size_t)((b + 255) / 256 * 256); }
AttnSizes attn_sizes(int64_t queries, int heads_q, int64_t rows, int D) {
  const int64_t n = max((int64_t)kDecodePieces * 2 * kDecodeRows, (int64_t)kPrefillSlots * kPrefillRows);
  AttnSizes s;
  s.part = up256(n * D * 4);
  s.ml = up256(n * 2 * 4);
  s.row = up256((rows + 1) * 8);
  s.tile = up256((queries * heads_q / kPrefillRows + rows + 1) * 4);
  return s;
}

template <int D, bool F32>
hipError_t launch(const AttnArgs& a, const AttnPlan& pl, hipStream_t s) {
  if (!a.cu) {
    const int lds = (a.rows + 1) * 8;
    const void* f = reinterpret_cast<const void*>(decode_attn_kernel<D, F32>);
    hipError_t e = prepare_launch(f, lds, 256);
    if (e == hipSuccess) e = prepare_launch(reinterpret_cast<const void*>(decode_join_kernel<D>), lds, 256);
    if (e != hipSuccess) return e;
    decode_attn_kernel<D, F32><<<kDecodeGroups, 256, lds, s>>>(a, pl);
    decode_join_kernel<D><<<kDecodePieces - 1, 256, lds, s>>>(a, pl);
    return hipGetLastError();
  }
  prefill_plan_kernel<<<1, 1024, 0, s>>>(a, pl);
  prefill_attn_kernel<D, F32><<<kPrefillGroups, 256, 0, s>>>(a, pl);
  prefill_join_kernel<D><<<dim3(kPrefillSlots, 4), 256, 0, s>>>(a, pl);
  return hipGetLastError();
}

}  // namespace

size_t attn_workspace_bytes(int64_t queries, int heads_q, int64_t rows, int head_dim) {
  return attn_sizes(queries, heads_q, rows, head_dim).all();
}

hipError_t launch_attn(const AttnArgs& a, hipStream_t s) {
  const AttnSizes z = attn_sizes(a.queries, a.heads * a.group, a.rows, a.head_dim);
  char* p = reinterpret_cast<char*>(a.ws);
  AttnPlan pl;
  pl.part = reinterpret_cast<float*>(p);
  pl.ml = reinterpret_cast<float*>(p += z.part);
  pl.row_task = reinterpret_cast<int64_t*>(p += z.ml);
  pl.row_slot = reinterpret_cast<int64_t*>(p += z.row);
  pl.row_tiles = reinterpret_cast<int64_t*>(p += z.row);
  pl.tile_task = reinterpret_cast<int32_t*>(p += z.row);
  pl.tile_slot = reinterpret_cast<int32_t*>(p += z.tile);
  pl.zeros = reinterpret_cast<uint16_t*>(p += z.tile);
  pl.head = reinterpret_cast<int64_t*>(p += 256);
  pl.next = reinterpret_cast<int32_t*>(p + 64);
  // t = s c with c > 0, so that the largest score has the largest t
  const float log2e = 1.4426950408889634f;
  pl.qmul = a.scale > 0.0f ? 1.0f : a.scale < 0.0f ? -1.0f : 0.0f;
  pl.c = a.scale != 0.0f ? fabsf(a.scale) * log2e : 1.0f;
  switch (a.head_dim) {
    case 64: return a.bf16 ? launch<64, false>(a, pl, s) : launch<64, true>(a, pl, s);
    case 96: return a.bf16 ? launch<96, false>(a, pl, s) : launch<96, true>(a, pl, s);
    default: return a.bf16 ? launch<128, false>(a, pl, s) : launch<128, true>(a, pl, s);
  }
}

}  // namespace loopq

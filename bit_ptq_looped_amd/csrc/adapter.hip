// Low-rank adapters of many requests beside a shared projection
// (include/loopq_block.h has the definitions):
//   z_m = scale_a A_a x_m,  y_m += B_a z_m,  a = ids[m].
//
// Two launches: the first forms z (fp32, in the workspace), the second adds its
// product to y.  Rows without an adapter cost their id's read.
#include "block_internal.h"
#include "quant_core.h"

namespace loopq {
namespace {

// the row's adapter, or -1
__device__ __forceinline__ int adapter_of(const AdapterArgs& a, int64_t m) {
  const int id = a.ids[m];
  return id >= 0 && id < a.adapters ? id : -1;
}
__device__ __forceinline__ int rank_of(const AdapterArgs& a, int id) {
  if (a.ranks == nullptr) return a.R;
  const int r = a.ranks[id];
  return r < 0 ? 0 : r > a.R ? a.R : r;
}

// the same for an adapter of the whole wave: a scalar load, which the vector loads under way need not wait for
__device__ __forceinline__ int wave_rank_of(const AdapterArgs& a, int id) {
  if (a.ranks == nullptr) return a.R;
  typedef const int32_t __attribute__((address_space(4))) * constant_ints;
  const int r = ((constant_ints)(uintptr_t)a.ranks)[id];
  return r < 0 ? 0 : r > a.R ? a.R : r;
}

__device__ __forceinline__ void eight_bf16(const uint4& u, float (&v)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// ---------------------------------------------------------------- few rows

constexpr int kRanks = 2;  // ranks a wave takes

// A wave forms kRanks of a row's z: products of 8 elements a lane and step, the
// lanes added up by a butterfly.
template <int BF>
__global__ __launch_bounds__(256) void shrink_rows_kernel(AdapterArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t m = blockIdx.x;
  const int j0 = (blockIdx.y * 4 + (threadIdx.x >> 6)) * kRanks;
  const int id = adapter_of(a, m);
  if (id < 0) return;
  const int rank = rank_of(a, id);
  if (j0 >= rank) return;
  const uint16_t* A = a.A + ((int64_t)id * a.R + j0) * a.K;
  float acc[kRanks] = {};
#pragma unroll 4
  for (int k = 8 * lane; k < a.K; k += 512) {
    float x[8];
    if constexpr (BF) {
      eight_bf16(*reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.x) + m * a.ldx + k), x);
    } else {
      const float4* p = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(a.x) + m * a.ldx + k);
      const float4 u = p[0], v = p[1];
      x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w, x[4] = v.x, x[5] = v.y, x[6] = v.z, x[7] = v.w;
    }
#pragma unroll
    for (int j = 0; j < kRanks; ++j) {
      if (j0 + j >= rank) break;
      float w[8];
      eight_bf16(*reinterpret_cast<const uint4*>(A + (int64_t)j * a.K + k), w);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[j] = __builtin_fmaf(x[i], w[i], acc[j]);
    }
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1)
#pragma unroll
    for (int j = 0; j < kRanks; ++j) acc[j] += __shfl_xor(acc[j], o);
  if (lane == 0) {
    const float s = a.scales[id];
#pragma unroll
    for (int j = 0; j < kRanks; ++j)
      if (j0 + j < rank) a.z[m * a.R + j0 + j] = s * acc[j];
  }
}

// A wave adds to 64 elements of a row of y.  C = 2^k >= R / 8 lanes share an
// element, eight ranks each (one 16-byte read of B), in C passes over the 64;
// lane l keeps the element of pass l % C.
template <int C>
__global__ __launch_bounds__(256) void expand_rows_kernel(AdapterArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t m = blockIdx.x;
  const int n0 = (blockIdx.y * 4 + (threadIdx.x >> 6)) * 64;
  if (n0 >= a.N) return;
  const int id = adapter_of(a, m);
  if (id < 0) return;
  const int rank = rank_of(a, id);
  const int c = lane % C, per = 64 / C;
  const int n_mine = n0 + c * per + lane / C;
  float* y = a.y + m * a.ldy;
  float old = 0.0f;
  if (n_mine < a.N) old = y[n_mine];
  const int have = max(0, min(8, rank - 8 * c));  // ranks of this lane
  float z[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] = i < have ? a.z[m * a.R + 8 * c + i] : 0.0f;
  const uint16_t* B = a.B + ((int64_t)id * a.N) * a.R + 8 * c;
  uint4 b[C];
#pragma unroll
  for (int p = 0; p < C; ++p) {
    const int n = n0 + p * per + lane / C;
    b[p] = n < a.N && have > 0 ? *reinterpret_cast<const uint4*>(B + (int64_t)n * a.R) : uint4{0u, 0u, 0u, 0u};
  }
  float mine = 0.0f;
#pragma unroll
  for (int p = 0; p < C; ++p) {
    float w[8];
    eight_bf16(b[p], w);
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v = __builtin_fmaf(z[i], i < have ? w[i] : 0.0f, v);
#pragma unroll
    for (int o = 1; o < C; o <<= 1) v += __shfl_xor(v, o);
    if (c == p) mine = v;
  }
  if (n_mine < a.N) y[n_mine] = old + mine;
}

hipError_t launch_rows(const AdapterArgs& a, hipStream_t s) {
  const dim3 shrink(a.rows, (a.R + 4 * kRanks - 1) / (4 * kRanks));
  if (a.x_bf16) shrink_rows_kernel<1><<<shrink, 256, 0, s>>>(a);
  else shrink_rows_kernel<0><<<shrink, 256, 0, s>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const dim3 expand(a.rows, (a.N + 255) / 256);
  const int c = a.R / 8;
  void (*fn)(AdapterArgs) = c <= 1   ? expand_rows_kernel<1>
                            : c <= 2 ? expand_rows_kernel<2>
                            : c <= 4 ? expand_rows_kernel<4>
                            : c <= 8 ? expand_rows_kernel<8>
                                     : expand_rows_kernel<16>;
  fn<<<expand, 256, 0, s>>>(a);
  return hipGetLastError();
}

// --------------------------------------------------------------- many rows
//
// Both products on the bf16 MFMA (16x16x32): the adapter's rows are the first
// operand, the tokens the second, so that a lane holds four consecutive ranks
// (outputs) of one token, 16 bytes of z (y).  fp32 values enter as three exact
// bf16 planes, smallest first, so products are exact and sums fp32.  A tile of
// tokens goes through each adapter that occurs in it, whole, and every token
// keeps the result of its own: no sorting, no zeros multiplied into other rows
// (an infinity in one adapter stays with its tokens), and the cost of a mixed
// tile is its number of adapters, which for prompts is one or two.

constexpr int kTile = 32;  // tokens of a shrink work-group
constexpr int kMaxSplits = 8;

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Adapters of a wave's tokens, one after the other: lane l (of `lanes`) holds the
// id of token l; next() takes the first one left.
struct Adapters {
  uint64_t left;
  int id;
  __device__ __forceinline__ Adapters(int id_, uint64_t lanes) : left(__ballot(id_ >= 0) & lanes), id(id_) {}
  __device__ __forceinline__ int next() {
    const int a = __builtin_amdgcn_readlane(id, __ffsll((unsigned long long)left) - 1);
    left &= ~__ballot(id == a);
    return a;
  }
};

// How many adapters occur.
__device__ __forceinline__ int count_of(Adapters all) {
  int n = 0;
  for (; all.left; ++n) all.next();
  return n;
}

// Loads and stores go through buffer resources of less than 2^31 bytes, so that a
// lane without a part in one names the place kNone, past the end: the load gives 0
// and the store is dropped, without a branch around each.
constexpr uint32_t kNone = 0x80000000u;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t resource(const void* p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, 0x00020000);
}
__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t r, uint32_t at) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0));
}

// z partial sums: work-group (tile, split) of 4 waves.  K is cut into steps of KS
// MFMA (32 KS elements), the split's steps into four runs, whose sums are added in
// their order through LDS: a wave takes one run of every adapter or, in a tile of
// more than kFew adapters, the four runs of every fourth adapter (the sums are the
// same).  Two sets of registers: the next step is loaded while one is multiplied.
// RT: rank tiles of 16 (R <= 16 RT).
constexpr int kFew = 4;

template <int BF, int RT, int KS>
__global__ __launch_bounds__(256) void shrink_tile_kernel(AdapterArgs a) {
  constexpr int LD = 16 * RT + 4;
  __shared__ float sum[4][kTile][LD];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int li = lane & 15, lq = lane >> 4;
  const int64_t m0 = (int64_t)blockIdx.x * kTile;
  const int64_t mine = m0 + (lane & 31);
  const int id = mine < a.rows ? adapter_of(a, mine) : -1;
  Adapters todo(id, 0xFFFFFFFFull);
  if (todo.left == 0) return;
  const bool mixed = count_of(todo) > kFew;
  const int steps = (a.K + 32 * KS - 1) / (32 * KS);
  int first[5];  // of each run, and the end (K <= 65536 and splits <= 8: 32 bits do)
#pragma unroll
  for (int r = 0; r < 5; ++r) first[r] = (uint32_t)steps * (blockIdx.y * 4 + r) / (gridDim.y * 4);
  const int c0 = mixed ? first[0] : wave == 0 ? first[0] : wave == 1 ? first[1] : wave == 2 ? first[2] : first[3];
  const int c1 = mixed ? first[4] : wave == 0 ? first[1] : wave == 1 ? first[2] : wave == 2 ? first[3] : first[4];
  constexpr int item = BF ? 2 : 4;
  const auto xr = resource(reinterpret_cast<const char*>(a.x) + m0 * a.ldx * item, (kTile - 1) * a.ldx * item + a.K * item);
  int ids[2];
  uint32_t xat[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    ids[h] = __shfl(id, 16 * h + li);
    xat[h] = (uint32_t)((16 * h + li) * a.ldx * item);
  }
  // this wave's adapters: all, or every fourth
  int skip = mixed ? wave : 0;
  auto next_adapter = [&]() {
    for (; todo.left && skip > 0; --skip) todo.next();
    if (mixed) skip = 3;
    return todo.left ? todo.next() : -1;
  };
  struct Step {
    u32x4 x[KS][2][BF ? 1 : 2];
    u32x4 w[KS][RT];
  };
  // always the same number of loads, so that the wait for one step leaves the next one's under way
  auto load = [&](Step& s, int ad, int rank, int c) {
    const auto wr = resource(a.A + (int64_t)max(ad, 0) * a.R * a.K, ad < 0 ? 0 : (int64_t)rank * a.K * 2);  // rows from the rank on lie outside
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      const int k = (c * KS + i) * 32 + 8 * lq;
      const bool in = k < a.K;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t at = in && ad >= 0 && ids[h] == ad ? xat[h] + (uint32_t)(k * item) : kNone;
#pragma unroll
        for (int p = 0; p < (BF ? 1 : 2); ++p) s.x[i][h][p] = load16(xr, at + 16 * p);
      }
#pragma unroll
      for (int t = 0; t < RT; ++t) s.w[i][t] = load16(wr, in ? (uint32_t)(((16 * t + li) * a.K + k) * 2) : kNone);
    }
  };
  v4f acc[2][RT];
  auto multiply = [&](const Step& s, int ad, int c) {
    int run = wave, begin = c0, end = c1;
    if (mixed) {
      run = c < first[1] ? 0 : c < first[2] ? 1 : c < first[3] ? 2 : 3;
      begin = c < first[1] ? first[0] : c < first[2] ? first[1] : c < first[3] ? first[2] : first[3];
      end = c < first[1] ? first[1] : c < first[2] ? first[2] : c < first[3] ? first[3] : first[4];
    }
    if (c == begin) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int t = 0; t < RT; ++t) acc[h][t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    }
#pragma unroll
    for (int i = 0; i < KS; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if constexpr (BF) {
#pragma unroll
          for (int t = 0; t < RT; ++t) acc[h][t] = s2_mm(s.w[i][t], s.x[i][h][0], acc[h][t]);
        } else {
          float v[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[e] = __uint_as_float(s.x[i][h][0][e]);
            v[4 + e] = __uint_as_float(s.x[i][h][1][e]);
          }
          v4u planes[3];
          planes8(v, planes);
#pragma unroll
          for (int p = 2; p >= 0; --p)
#pragma unroll
            for (int t = 0; t < RT; ++t) acc[h][t] = s2_mm(s.w[i][t], planes[p], acc[h][t]);
        }
      }
    if (c + 1 < end) return;
    mfma_settle_before_join();
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (ids[h] == ad) {
#pragma unroll
        for (int t = 0; t < RT; ++t) *reinterpret_cast<v4f*>(&sum[run][16 * h + li][16 * t + 4 * lq]) = acc[h][t];
      }
  };
  int ad = c0 < c1 ? next_adapter() : -1;
  if (ad >= 0) {
    int rank = wave_rank_of(a, ad), c = c0;
    auto advance = [&]() {
      if (++c < c1) return;
      ad = next_adapter();
      if (ad >= 0) rank = wave_rank_of(a, ad);
      c = c0;
    };
    Step s0, s1;
    load(s0, ad, rank, c);
    for (;;) {
      int at = c, of = ad;
      advance();
      load(s1, ad, rank, c);
      multiply(s0, of, at);
      if (ad < 0) break;
      at = c, of = ad;
      advance();
      load(s0, ad, rank, c);
      multiply(s1, of, at);
      if (ad < 0) break;
    }
  }
  __syncthreads();
  float* z = a.z + ((int64_t)blockIdx.y * a.rows + m0) * a.R;
  for (int i = threadIdx.x; i < kTile * a.R; i += 256) {
    const int m = i / a.R, j = i - m * a.R;
    if (m0 + m >= a.rows) continue;
    const int own = adapter_of(a, m0 + m);
    if (own < 0 || j >= rank_of(a, own)) continue;
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < 4; ++w)
      if (first[w] < first[w + 1]) v += sum[w][m][j];
    z[i] = a.scales[own] * v;
  }
}

// y += B z: a wave takes 16 tokens and a stripe of N, 64 outputs a step; the four
// waves of a work-group lie side by side in N.  Two sets of registers: the next
// (adapter, step) is loaded while one is multiplied.  RS: steps of 32 ranks
// (R <= 32 RS).  VEC: y in 16-byte accesses (aligned rows, N % 4 == 0).
template <int RS, bool VEC>
__global__ __launch_bounds__(256) void expand_tile_kernel(AdapterArgs a, int splits, int stripe, int stripes) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int li = lane & 15, lq = lane >> 4;
  const int group = blockIdx.x / stripes;
  const int64_t m = (int64_t)group * 16 + li;
  const int id = m < a.rows ? adapter_of(a, m) : -1;
  Adapters todo(id, 0xFFFFull);
  if (todo.left == 0) return;
  const int n_begin = (blockIdx.x - group * stripes) * stripe + 64 * wave;
  const int n_end = min(a.N, (blockIdx.x - group * stripes) * stripe + stripe);
  if (n_begin >= n_end) return;
  const auto yr = resource(a.y + (int64_t)group * 16 * a.ldy, 15 * a.ldy * 4 + (int64_t)a.N * 4);
  const uint32_t yat = (uint32_t)(li * a.ldy * 4);
  struct Step {
    v4f old[4];
    u32x4 b[RS][4];
  };
  // always the same number of loads, so that the wait for one step leaves the next one's under way
  auto load = [&](Step& s, int ad, int rank, int n0) {
    const auto br = resource(a.B + (int64_t)max(ad, 0) * a.N * a.R, ad < 0 ? 0 : (int64_t)a.N * a.R * 2);  // outputs from N on lie outside
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = n0 + 16 * i + li;
#pragma unroll
      for (int t = 0; t < RS; ++t) {
        const int j = 32 * t + 8 * lq;
        s.b[t][i] = load16(br, j < rank ? (uint32_t)((n * a.R + j) * 2) : kNone);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = n0 + 16 * i + 4 * lq;
      if constexpr (VEC) {
        s.old[i] = __builtin_bit_cast(v4f, load16(yr, id == ad && ad >= 0 && n < a.N ? yat + 4u * n : kNone));
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          s.old[i][e] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(yr, id == ad && ad >= 0 && n + e < a.N ? yat + 4u * (n + e) : kNone, 0, 0));
      }
    }
  };
  int ad = todo.next(), rank = wave_rank_of(a, ad), n0 = n_begin;
  Step s0, s1;
  load(s0, ad, rank, n0);
  v4u z[RS][3];
  const int mine = id >= 0 ? rank_of(a, id) : 0;
#pragma unroll
  for (int t = 0; t < RS; ++t) {
    const int j = 32 * t + 8 * lq;
    float v[8] = {};
    if (j < mine) {
      for (int sp = 0; sp < splits; ++sp) {
        const v4f* p = reinterpret_cast<const v4f*>(a.z + ((int64_t)sp * a.rows + m) * a.R + j);
        const v4f u0 = p[0], u1 = p[1];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[e] += u0[e];
          v[4 + e] += u1[e];
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = j + e < mine ? v[e] : 0.0f;
    planes8(v, z[t]);
  }
  auto multiply = [&](Step& s, int of, int of_rank, int at) {
    if (of_rank & 7) {  // a lane may have read ranks that the adapter does not have
#pragma unroll
      for (int t = 0; t < RS; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int have = of_rank - (32 * t + 8 * lq + 2 * e);
          const uint32_t keep = have >= 2 ? 0xFFFFFFFFu : have == 1 ? 0x0000FFFFu : 0u;
#pragma unroll
          for (int i = 0; i < 4; ++i) s.b[t][i][e] &= keep;
        }
    }
    v4f acc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int p = 2; p >= 0; --p)
#pragma unroll
      for (int t = 0; t < RS; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] = s2_mm(s.b[t][i], z[t][p], acc[i]);
    mfma_settle_before_join();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = at + 16 * i + 4 * lq;
      const v4f v = s.old[i] + acc[i];
      if constexpr (VEC) {
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), yr, id == of && n < a.N ? yat + 4u * n : kNone, 0, 0);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[e]), yr, id == of && n + e < a.N ? yat + 4u * (n + e) : kNone, 0, 0);
      }
    }
  };
  auto advance = [&]() {
    if ((n0 += 256) < n_end) return;
    ad = todo.left ? todo.next() : -1;
    if (ad >= 0) rank = wave_rank_of(a, ad);
    n0 = n_begin;
  };
  for (;;) {
    int at = n0, of = ad, of_rank = rank;
    advance();
    load(s1, ad, rank, n0);
    multiply(s0, of, of_rank, at);
    if (ad < 0) break;
    at = n0, of = ad, of_rank = rank;
    advance();
    load(s0, ad, rank, n0);
    multiply(s1, of, of_rank, at);
    if (ad < 0) break;
  }
}

int splits_for(int64_t rows, int K) {
  const int64_t tiles = (rows + kTile - 1) / kTile;
  const int64_t want = 768 / tiles, most = (K + 511) / 512;
  const int64_t n = want < most ? want : most;
  return (int)(n < 1 ? 1 : n > kMaxSplits ? kMaxSplits : n);
}

// KS: what two steps' registers leave room for two or three waves a SIMD
template <int RT, int KS_BF, int KS_F32>
void shrink_tiles(const AdapterArgs& a, dim3 grid, hipStream_t s) {
  if (a.x_bf16) shrink_tile_kernel<1, RT, KS_BF><<<grid, 256, 0, s>>>(a);
  else shrink_tile_kernel<0, RT, KS_F32><<<grid, 256, 0, s>>>(a);
}
template <int RS>
void expand_tiles(const AdapterArgs& a, int grid, int splits, int stripe, int stripes, hipStream_t s) {
  if (a.ldy % 4 == 0 && a.N % 4 == 0 && reinterpret_cast<uintptr_t>(a.y) % 16 == 0)
    expand_tile_kernel<RS, true><<<grid, 256, 0, s>>>(a, splits, stripe, stripes);
  else
    expand_tile_kernel<RS, false><<<grid, 256, 0, s>>>(a, splits, stripe, stripes);
}

hipError_t launch_tiles(const AdapterArgs& a, hipStream_t s) {
  const int splits = splits_for(a.rows, a.K);
  const dim3 shrink((a.rows + kTile - 1) / kTile, splits);
  if (a.R <= 16) shrink_tiles<1, 4, 2>(a, shrink, s);
  else if (a.R <= 32) shrink_tiles<2, 4, 2>(a, shrink, s);
  else if (a.R <= 64) shrink_tiles<4, 2, 2>(a, shrink, s);
  else shrink_tiles<8, 1, 1>(a, shrink, s);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int groups = (a.rows + 15) / 16, steps = (a.N + 255) / 256;
  int stripes = (2048 + groups - 1) / groups;
  if (stripes > steps) stripes = steps;
  const int stripe = (steps + stripes - 1) / stripes * 256;
  stripes = (a.N + stripe - 1) / stripe;
  if (a.R <= 32) expand_tiles<1>(a, groups * stripes, splits, stripe, stripes, s);
  else if (a.R <= 64) expand_tiles<2>(a, groups * stripes, splits, stripe, stripes, s);
  else expand_tiles<4>(a, groups * stripes, splits, stripe, stripes, s);
  return hipGetLastError();
}

}  // namespace

// z of each split of K (at most what splits_for gives for any K)
size_t adapter_workspace_bytes(int64_t rows, int max_rank) {
  return (size_t)(splits_for(rows > 0 ? rows : 1, 1 << 30) * rows * max_rank * 4 + 255) / 256 * 256;
}

hipError_t launch_adapter(const AdapterArgs& a, hipStream_t s) {
  return a.rows <= 64 ? launch_rows(a, s) : launch_tiles(a, s);
}

}  // namespace loopq

// Low-rank adapters of many requests beside a shared projection
// (include/loopq_block.h has the definitions):
//   z_m = scale_a A_a x_m,  y_m += B_a z_m,  a = ids[m].
//
// z goes through the workspace (fp32) from the launches that form it to the one that
// adds its product to y, or stays in one launch (few rows).  Rows without an adapter
// cost their id's read.  What bounds it: for prompts the bytes of x and twice those of
// y, which are far more than the adapters' and whose products take the matrix units a
// tenth of that time; for few rows the launch and its trips to memory.
// 8192 bf16 rows of nine requests, one without an adapter, K 2560, N 6912, rank 64: 120 us
// (24 + 6 + 90; 458 MB at the 4.8 TB/s of a large copy are 95); 1500 of K 6912, N 2560, rank
// 32, from the last-level cache: 28 (13 + 4 + 11); 48 rows of 32 adapters, K 2560, N 7680,
// rank 16: 7.7; one such row 5.2.
#include <algorithm>
#include <type_traits>

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
//
// fp32 FMA of the vector units; A and B are read with 16 bytes a lane, eight
// neighbours of K (ranks) each: a row reads its adapter from an L2 or the last-level
// cache whatever its neighbours do.

// Sums of V[0 .. n - 1] over the wave's lanes.  Two values change halves with one
// swap of 32 lanes, then of 16: a lane goes on with a quarter of them; four
// steps within 16 lanes finish.  sums() leaves value i of the V in the lanes
// 16 q .. 16 q + 15 of v[i / 4], q = i % 4.
template <int S>
__device__ __forceinline__ float swap_add(float x, float y) {
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  u32x2 r;
  if constexpr (S == 32) r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(y), false, false);
  else r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(y), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
template <int CTRL>
__device__ __forceinline__ float dpp_add(float x) {
  return x + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xF, 0xF, false));
}
template <int N>
__device__ __forceinline__ void sums(float (&v)[N]) {
  static_assert(N % 4 == 0, "four values share a lane's 16");
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    // lanes 0-15: value 4 i, 16-31: 4 i + 1, 32-47: 4 i + 2, 48-63: 4 i + 3
    const float a = swap_add<32>(v[4 * i], v[4 * i + 2]), b = swap_add<32>(v[4 * i + 1], v[4 * i + 3]);
    float x = swap_add<16>(a, b);
    x = dpp_add<0xB1>(x);
    x = dpp_add<0x4E>(x);
    x = dpp_add<0x141>(x);
    v[i] = dpp_add<0x140>(x);
  }
}

// A wave forms J ranks of a token's z, 512 elements of K a step: every `step`-th of them
// from k0 on.  The sum of rank i of the J is in the lanes 16 i .. 16 i + 15.
constexpr int J = 4;
template <int BF>
__device__ __forceinline__ float four_ranks(const AdapterArgs& a, int64_t m, int id, int rank, int j0, int k0, int step) {
  const int lane = threadIdx.x & 63;
  const uint16_t* A = a.A + ((int64_t)id * a.R + j0) * a.K;
  float acc[J] = {};
#pragma unroll 2
  for (int k = k0 + 8 * lane; k < a.K; k += step) {
    uint4 w[J];
#pragma unroll
    for (int j = 0; j < J; ++j) w[j] = *reinterpret_cast<const uint4*>(A + (int64_t)(j0 + j < rank ? j : 0) * a.K + k);
    float x[8];
    if constexpr (BF) {
      eight_bf16(*reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.x) + m * a.ldx + k), x);
    } else {
      const float4* p = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(a.x) + m * a.ldx + k);
      const float4 u = p[0], v = p[1];
      x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w, x[4] = v.x, x[5] = v.y, x[6] = v.z, x[7] = v.w;
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {
      float u[8];
      eight_bf16(w[j], u);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[j] = __builtin_fmaf(x[i], u[i], acc[j]);
    }
  }
  sums(acc);
  return acc[0];
}

// A wave adds to 64 outputs of a token of y.  C = 2^k >= R / 8 lanes share an output,
// eight ranks each (one 16-byte read of B), in C passes over the 64; lane l keeps the
// output of pass l % C.
template <int C>
struct Outputs {
  static constexpr int per = 64 / C;
  uint4 b[C];
  float* y;
  float old;
  int c, have;
  bool in;
  __device__ __forceinline__ void load(const AdapterArgs& a, int64_t m, int id, int rank, int n0) {
    const int lane = threadIdx.x & 63;
    c = lane % C;
    const int n_mine = n0 + c * per + lane / C;
    in = n_mine < a.N;
    y = a.y + m * a.ldy + n_mine;
    old = in ? *y : 0.0f;
    have = max(0, min(8, rank - 8 * c));  // ranks of this lane
    const uint16_t* B = a.B + ((int64_t)id * a.N) * a.R + 8 * c;
#pragma unroll
    for (int p = 0; p < C; ++p) {
      const int n = n0 + p * per + lane / C;
      b[p] = n < a.N && have > 0 ? *reinterpret_cast<const uint4*>(B + (int64_t)n * a.R) : uint4{0u, 0u, 0u, 0u};
    }
  }
  __device__ __forceinline__ void add(const float (&z)[8]) {  // 0 past the lane's ranks
    float mine = 0.0f;
#pragma unroll
    for (int p = 0; p < C; ++p) {
      float w[8];
      eight_bf16(b[p], w);
      float v = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) v = __builtin_fmaf(z[i], i < have ? w[i] : 0.0f, v);
      if constexpr (C > 1) v = dpp_add<0xB1>(v);
      if constexpr (C > 2) v = dpp_add<0x4E>(v);
      if constexpr (C > 4) v = dpp_add<0x141>(v);
      if constexpr (C > 8) v = dpp_add<0x140>(v);
      if (c == p) mine = v;
    }
    if (in) *y = old + mine;
  }
};

template <int BF>
__global__ __launch_bounds__(256) void shrink_rows_kernel(AdapterArgs a) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t m = blockIdx.x;
  const int j0 = (blockIdx.y * 4 + wave) * J;
  const int id = __builtin_amdgcn_readfirstlane(adapter_of(a, m));
  if (id < 0) return;
  const int rank = wave_rank_of(a, id);
  if (j0 >= rank) return;
  const float z = four_ranks<BF>(a, m, id, rank, j0, 0, 512);
  const int j = j0 + (lane >> 4);
  if ((lane & 15) == 0 && j < rank) a.z[m * a.R + j] = a.scales[id] * z;
}

template <int C>
__global__ __launch_bounds__(256) void expand_rows_kernel(AdapterArgs a) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t m = blockIdx.x;
  const int n0 = (blockIdx.y * 4 + wave) * 64;
  if (n0 >= a.N) return;
  const int id = __builtin_amdgcn_readfirstlane(adapter_of(a, m));
  if (id < 0) return;
  Outputs<C> out;
  out.load(a, m, id, wave_rank_of(a, id), n0);
  float z[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] = i < out.have ? a.z[m * a.R + 8 * out.c + i] : 0.0f;
  out.add(z);
}

// Both in one launch: 16 waves form the token's z for themselves, in fours of ranks and
// parts of K, and add to 1024 outputs, whose y and B are on their way meanwhile.
constexpr int kWide = 1024;
constexpr int kTokenMaxRank = 32;
template <int BF, int C>
__global__ __launch_bounds__(1024) void token_kernel(AdapterArgs a) {
  __shared__ float sz[16 * J];  // [part][rank]
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t m = blockIdx.x;
  const int id = __builtin_amdgcn_readfirstlane(adapter_of(a, m));
  if (id < 0) return;
  const int rank = wave_rank_of(a, id);
  const int n0 = blockIdx.y * kWide + 64 * wave;
  Outputs<C> out;
  out.load(a, m, id, rank, n0);
  const int fours = a.R / J, parts = 16 / fours, part = wave / fours, j0 = (wave - part * fours) * J;
  if (part < parts && j0 < rank) {
    const float z = four_ranks<BF>(a, m, id, rank, j0, 512 * part, 512 * parts);
    if ((lane & 15) == 0) sz[part * a.R + j0 + (lane >> 4)] = z;
  }
  __syncthreads();
  const float s = a.scales[id];
  float z[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float v = 0.0f;
    if (i < out.have) {
      for (int part = 0; part < parts; ++part) v += sz[part * a.R + 8 * out.c + i];
    }
    z[i] = s * v;
  }
  if (n0 < a.N) out.add(z);
}

template <int C>
hipError_t launch_rows_of(const AdapterArgs& a, hipStream_t s) {
  // One launch while A is read again for few stripes: alone on the card it takes what two take
  // (rank 16, K 2560, N 7680: a row 5.2 us and 5.5, 48 rows 7.7 and 7.8, 160 17 and 14), and
  // the call costs 2.5 us less of the host.  From rank 64 on a work-group has too much of A to
  // itself (a row 8.3 us and 6.4).
  if constexpr (8 * C <= kTokenMaxRank) {
    const int stripes = (a.N + kWide - 1) / kWide;
    if ((int64_t)a.rows * stripes * a.R * a.K <= 1 << 24) {
      const dim3 grid(a.rows, stripes);
      if (a.x_bf16) token_kernel<1, C><<<grid, 1024, 0, s>>>(a);
      else token_kernel<0, C><<<grid, 1024, 0, s>>>(a);
      return hipGetLastError();
    }
  }
  const dim3 shrink(a.rows, (a.R + 4 * J - 1) / (4 * J));
  if (a.x_bf16) shrink_rows_kernel<1><<<shrink, 256, 0, s>>>(a);
  else shrink_rows_kernel<0><<<shrink, 256, 0, s>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  expand_rows_kernel<C><<<dim3(a.rows, (a.N + 255) / 256), 256, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_rows(const AdapterArgs& a, hipStream_t s) {
  const int c = a.R / 8;
  return c <= 1   ? launch_rows_of<1>(a, s)
         : c <= 2 ? launch_rows_of<2>(a, s)
         : c <= 4 ? launch_rows_of<4>(a, s)
         : c <= 8 ? launch_rows_of<8>(a, s)
                  : launch_rows_of<16>(a, s);
}

// --------------------------------------------------------------- many rows
//
// Both products on the bf16 MFMA.  fp32 values enter as three exact bf16 planes,
// smallest first, so products are exact and sums fp32.  A tile of tokens goes
// through each adapter that occurs in it, whole, and every token keeps the result
// of its own: no zeros multiplied into other rows (an infinity in one adapter stays
// with its tokens), and a tile costs its number of adapters.  For prompts that is one
// or two; tokens in any order are first put in the order of their adapters.
//
// An MFMA operand wants neighbouring lanes in different rows, memory wants them side
// by side: four lanes in four rows take four times the address cycles.  So what a
// work-group shares goes through LDS, and y is read and written an element a lane,
// 32 side by side.  A tile of more than kFew adapters goes without LDS: its waves
// take the adapters of their own tokens one by one, operands straight from memory (2048
// rows of 48 adapters, rank 16: 35 us with kFew 3, 46 with 6, 49 with 12).  The
// products and sums of a token are the same, in the same order, either way.

constexpr int kTile = 64;    // tokens of a shrink work-group, 16 a wave
constexpr int kTokens = 128; // tokens of an expand work-group, 32 a wave
constexpr int kFew = 3;
constexpr int kMaxSplits = 16;  // what they add to z's bytes would show

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));

__device__ __forceinline__ v16f mm32(const u32x4& a, const u32x4& b, v16f c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

// Adapters of up to 64 tokens, one after the other: lane l holds the id of token l;
// next() takes the first one left.
struct Adapters {
  uint64_t left;
  int id;
  __device__ __forceinline__ Adapters(int id_, uint64_t lanes) : left(__ballot(id_ >= 0) & lanes), id(id_) {}
  __device__ __forceinline__ int next() {
    const int a = __builtin_amdgcn_readlane(id, __ffsll((unsigned long long)left) - 1);
    left &= ~__ballot(id == a);
    return a;
  }
  __device__ __forceinline__ int next_or_none() { return left ? next() : -1; }
};

// Loads and stores go through buffer resources of less than 2^31 bytes, so that a
// lane without a part in one names the place kNone, past the end: the load gives 0
// and the store is dropped, without a branch around each.
constexpr uint32_t kNone = 0x80000000u;

// Tokens in any order are put in the order of their adapters, segment by segment, so
// that a wave meets few of them.  Every shrink work-group of a segment does this for
// itself, 3 us, less than a launch.  1024 fp32 rows of 48 adapters in any order, rank 64,
// K and N 2560: 41 us, as they come 156; 4096 of 32, rank 32, K and N 2048: 37 and 114.
constexpr int kSegment = 1024;
constexpr int kRuns = 32;  // two more adapters a tile, on average
// key: the place in the segment, and above its ten bits the adapter (a.adapters: none, or
// past the last row).  False, and nothing written, where ids change at most kRuns times from
// row to row.  Sorted by one bit of the adapter after the other, stably, four places a thread.
// share: 20 ints.
__device__ __forceinline__ bool order_segment(const AdapterArgs& a, int64_t base, uint32_t* key, int* share) {
  constexpr int E = kSegment / 256;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int count = (int)min((int64_t)kSegment, a.rows - base);
  int id[E], before[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int i = 256 * e + tid;
    id[e] = adapter_of(a, base + min(i, count - 1));
    before[e] = adapter_of(a, base + min(max(i - 1, 0), count - 1));
  }
  int runs = 0;
#pragma unroll
  for (int e = 0; e < E; ++e) runs += __popcll(__ballot(id[e] != before[e]));
  if (lane == 0) share[16 + wave] = runs;
  __syncthreads();
  if (share[16] + share[17] + share[18] + share[19] <= kRuns) return false;
  uint32_t v[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int i = 256 * e + tid;
    v[e] = (uint32_t)(i < count && id[e] >= 0 ? id[e] : a.adapters) * kSegment + i;
  }
  for (uint32_t bit = kSegment; bit <= (uint32_t)a.adapters * kSegment; bit *= 2) {
    uint64_t zeros[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      zeros[e] = __ballot(!(v[e] & bit));
      if (lane == 0) share[4 * e + wave] = __popcll(zeros[e]);
    }
    __syncthreads();
    int all = 0, at[E];
#pragma unroll
    for (int q = 0; q < 4 * E; ++q) {
      if (q % 4 == 0) at[q / 4] = all;
      const int n = share[q];
      if (q % 4 < wave) at[q / 4] += n;
      all += n;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int z = at[e] + __popcll(zeros[e] & ((1ull << lane) - 1));
      key[v[e] & bit ? all + 256 * e + tid - z : z] = v[e];
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = key[256 * e + tid];
  }
  return true;
}
__device__ __forceinline__ __amdgpu_buffer_rsrc_t resource(const void* p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, 0x00020000);
}
__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t r, uint32_t at) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0));
}

// acc[t] += A x of 32 elements of K: RT rank tiles of 16, 16 tokens
template <int BF, int RT>
__device__ __forceinline__ void shrink_mm(const u32x4 (&w)[RT], const u32x4 (&x)[BF ? 1 : 2], v4f (&acc)[RT]) {
  if constexpr (BF) {
#pragma unroll
    for (int t = 0; t < RT; ++t) acc[t] = s2_mm(w[t], x[0], acc[t]);
  } else {
    float v[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = __uint_as_float(x[0][e]);
      v[4 + e] = __uint_as_float(x[1][e]);
    }
    v4u planes[3];
    planes8(v, planes);
#pragma unroll
    for (int p = 2; p >= 0; --p)
#pragma unroll
      for (int t = 0; t < RT; ++t) acc[t] = s2_mm(w[t], planes[p], acc[t]);
  }
}

// z partial sums (16x16x32 MFMA, ranks the first operand, tokens the second: a lane
// ends with four ranks of a token): work-group (tile of 64 tokens, split of K), 16
// tokens a wave.  K goes in chunks of 256 bytes a row of x, two of them on their way
// while one is multiplied.
// RT: rank tiles of 16 (R <= 16 RT).
template <int BF, int RT>
__global__ __launch_bounds__(256) void shrink_tile_kernel(AdapterArgs a) {
  constexpr int item = BF ? 2 : 4;
  constexpr int KC = 256 / item;         // elements of a chunk
  constexpr int XS = 256 + 16;           // bytes of a row in LDS: 16 spread the rows over the banks
  constexpr int WS = KC * 2 + 16;
  constexpr int WL = KC / 8;             // lanes of a row of A
  constexpr int WN = (16 * RT * WL + 255) / 256;
  __shared__ __attribute__((aligned(16))) char sx[kTile * XS];
  __shared__ __attribute__((aligned(16))) char sw[16 * RT * WS];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int li = lane & 15, lq = lane >> 4;
  const int64_t m0 = (int64_t)blockIdx.x * kTile;
  // the token of this lane's place
  int64_t base = m0, row = m0 + lane;
  int id = row < a.rows ? adapter_of(a, row) : -1;
  if (a.sort) {
    uint32_t* key = reinterpret_cast<uint32_t*>(sx);
    static_assert(sizeof(sx) >= kSegment * 4 && sizeof(sw) >= 80, "the keys of a segment fit");
    base = m0 / kSegment * kSegment;
    if (order_segment(a, base, key, reinterpret_cast<int*>(sw))) {
      const uint32_t k = key[(int)(m0 - base) + lane];
      row = base + k % kSegment;
      id = (int)(k / kSegment) < a.adapters ? (int)(k / kSegment) : -1;
    }
  }
  if (blockIdx.y == 0 && wave == 0 && m0 + lane < a.rows) a.order[m0 + lane] = int2{(int)row, id};
  Adapters todo(id, ~0ull);
  if (todo.left == 0) return;
  int few = 0;
  for (Adapters all = todo; all.left && few <= kFew; ++few) all.next();
  const int chunks = (a.K + KC - 1) / KC;
  const int c0 = (uint32_t)chunks * blockIdx.y / gridDim.y, c1 = (uint32_t)chunks * (blockIdx.y + 1) / gridDim.y;
  const auto xr = resource(reinterpret_cast<const char*>(a.x) + base * a.ldx * item, ((a.sort ? kSegment : kTile) - 1) * a.ldx * item + a.K * item);
  const uint32_t row_at = (uint32_t)((row - base) * a.ldx * item);
  const int my_id = __shfl(id, 16 * wave + li);  // the token of this lane's results
  float* z = a.z + ((int64_t)blockIdx.y * a.rows + m0 + 16 * wave + li) * a.R;
  v4f acc[RT];
  auto finish = [&](int ad, int rank) {
    mfma_settle_before_join();
    if (my_id != ad) return;
    const float s = a.scales[ad];
#pragma unroll
    for (int t = 0; t < RT; ++t)  // rows of z are whole multiples of eight: what lies past the rank is never read
      if (16 * t + 4 * lq < rank) *reinterpret_cast<v4f*>(z + 16 * t + 4 * lq) = v4f{s * acc[t][0], s * acc[t][1], s * acc[t][2], s * acc[t][3]};
  };
  auto clear = [&]() {
#pragma unroll
    for (int t = 0; t < RT; ++t) acc[t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  };

  if (few <= kFew) {
    int xid[4];
    uint32_t xat[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      xid[i] = __shfl(id, (int)(threadIdx.x >> 4) + 16 * i);
      xat[i] = __shfl(row_at, (int)(threadIdx.x >> 4) + 16 * i);
    }
    while (todo.left) {
      const int ad = todo.next(), rank = wave_rank_of(a, ad);
      const auto wr = resource(a.A + (int64_t)ad * a.R * a.K, (int64_t)rank * a.K * 2);  // rows from the rank on lie outside
      struct Chunk {
        u32x4 x[4], w[WN];
      };
      // always the same number of loads, so that the wait for one chunk leaves the next ones under way
      auto load = [&](Chunk& s, int c) {
        const int kx = c * KC + (int)(threadIdx.x & 15) * (16 / item);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          s.x[i] = load16(xr, xid[i] == ad && kx < a.K && c < c1 ? xat[i] + (uint32_t)(kx * item) : kNone);
        const int kw = c * KC + (int)(threadIdx.x % WL) * 8;
#pragma unroll
        for (int i = 0; i < WN; ++i) {
          const int j = (int)threadIdx.x / WL + i * (256 / WL);
          s.w[i] = load16(wr, kw < a.K && c < c1 ? (uint32_t)((j * a.K + kw) * 2) : kNone);
        }
      };
      auto multiply = [&](Chunk& s, int next) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 4; ++i) *reinterpret_cast<u32x4*>(sx + ((int)(threadIdx.x >> 4) + 16 * i) * XS + (threadIdx.x & 15) * 16) = s.x[i];
#pragma unroll
        for (int i = 0; i < WN; ++i) {
          const int j = (int)threadIdx.x / WL + i * (256 / WL);
          if (16 * RT * WL >= 256 || j < 16 * RT) *reinterpret_cast<u32x4*>(sw + j * WS + (threadIdx.x % WL) * 16) = s.w[i];
        }
        __syncthreads();
        load(s, next);
#pragma unroll
        for (int k = 0; k < KC / 32; ++k) {
          u32x4 xo[BF ? 1 : 2], wo[RT];
#pragma unroll
          for (int p = 0; p < (BF ? 1 : 2); ++p)
            xo[p] = *reinterpret_cast<const u32x4*>(sx + (16 * wave + li) * XS + (32 * k + 8 * lq) * item + 16 * p);
#pragma unroll
          for (int t = 0; t < RT; ++t) wo[t] = *reinterpret_cast<const u32x4*>(sw + (16 * t + li) * WS + (32 * k + 8 * lq) * 2);
          shrink_mm<BF, RT>(wo, xo, acc);
        }
      };
      clear();
      Chunk s0, s1;
      load(s0, c0);
      load(s1, c0 + 1);
      for (int c = c0;;) {
        multiply(s0, c + 2);
        if (++c >= c1) break;
        multiply(s1, c + 2);
        if (++c >= c1) break;
      }
      finish(ad, rank);
    }
    return;
  }

  // many adapters: a wave for itself, two register sets of KS MFMA steps each
  constexpr int KS = RT == 1 ? 4 : RT <= 4 ? 2 : 1;
  struct Step {
    u32x4 x[KS][BF ? 1 : 2];
    u32x4 w[KS][RT];
    int ad, rank, k0;
  };
  Adapters own(my_id, 0xFFFFull);
  const uint32_t xat = __shfl(row_at, 16 * wave + li);
  const int k_begin = c0 * KC, k_end = min(a.K, c1 * KC);
  if (own.left == 0 || k_begin >= k_end) return;
  int ad = own.next(), rank = wave_rank_of(a, ad), k0 = k_begin;
  // the step at hand, and on to the next; always the same number of loads, so that the
  // wait for one step leaves the next one's under way
  auto load = [&](Step& s) {
    s.ad = ad, s.rank = rank, s.k0 = k0;
    const auto wr = resource(a.A + (int64_t)max(ad, 0) * a.R * a.K, ad < 0 ? 0 : (int64_t)rank * a.K * 2);
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      const int k = k0 + 32 * i + 8 * lq;
      const bool in = k < k_end;
#pragma unroll
      for (int p = 0; p < (BF ? 1 : 2); ++p)
        s.x[i][p] = load16(xr, in && ad >= 0 && my_id == ad ? xat + (uint32_t)(k * item + 16 * p) : kNone);
#pragma unroll
      for (int t = 0; t < RT; ++t) s.w[i][t] = load16(wr, in ? (uint32_t)(((16 * t + li) * a.K + k) * 2) : kNone);
    }
    if ((k0 += 32 * KS) < k_end) return;
    k0 = k_begin;
    ad = ad < 0 ? -1 : own.next_or_none();
    if (ad >= 0) rank = wave_rank_of(a, ad);
  };
  auto multiply = [&](const Step& s) {
    if (s.k0 == k_begin) clear();
#pragma unroll
    for (int i = 0; i < KS; ++i) shrink_mm<BF, RT>(s.w[i], s.x[i], acc);
    if (s.k0 + 32 * KS >= k_end) finish(s.ad, s.rank);
  };
  Step s0, s1;
  load(s0);
  for (;;) {
    load(s1);
    multiply(s0);
    if (s1.ad < 0) return;
    load(s0);
    multiply(s1);
    if (s0.ad < 0) return;
  }
}

// The splits' sums of z, added in their order, as three bf16 planes: [row][R / 8][3][8].
// A thread takes eight ranks of a place's token; ranks that its adapter does not have are 0.
// (Read by the next kernel itself, 16 splits of 1500 tokens cost it 9 us in each of 40
// stripes of N, this launch 3.)
__global__ __launch_bounds__(256) void join_kernel(AdapterArgs a, int splits) {
  const int per = a.R / 8;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t m = i / per;
  if (m >= a.rows) return;
  const int id = a.order[m].y;
  if (id < 0) return;
  const int j = (int)(i - m * per) * 8, rank = rank_of(a, id);
  float v[8] = {};
  if (j < rank) {
    const float* at = a.z + m * a.R + j;
#pragma unroll 4
    for (int sp = 0; sp < splits; ++sp) {
      const v4f* p = reinterpret_cast<const v4f*>(at + (int64_t)sp * a.rows * a.R);
      const v4f u0 = p[0], u1 = p[1];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] += u0[e];
        v[4 + e] += u1[e];
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = j + e < rank ? v[e] : 0.0f;
  v4u planes[3];
  planes8(v, planes);
  v4u* to = reinterpret_cast<v4u*>(a.planes) + i * 3;
#pragma unroll
  for (int p = 0; p < 3; ++p) to[p] = planes[p];
}

// y += B z (32x32x16 MFMA, tokens the first operand, outputs the second: a lane ends
// with 16 tokens of one output): work-group (128 tokens, stripe of N), 32 tokens a
// wave.  NB outputs of B go through LDS at a time; the next ones, and their y, are
// loaded while some are multiplied.  RS: steps of 16 ranks (R <= 16 RS).
template <int RS>
__global__ __launch_bounds__(256, RS <= 4 ? 2 : 1) void expand_tile_kernel(AdapterArgs a, int stripe, int stripes) {
  constexpr int NB = 64;                 // outputs of a block
  constexpr int BS = 32 * RS + 16;       // bytes of a row of B in LDS
  constexpr int BL = 2 * RS;             // lanes of a row
  constexpr int BN = NB * BL / 256;      // loads of a thread
  static_assert(NB * BL % 256 == 0 || NB * BL == 128, "a block is whole loads of the work-group");
  __shared__ __attribute__((aligned(16))) char sb[NB * BS];
  __shared__ __attribute__((aligned(16))) uint32_t sy[kTokens];  // where the tokens' rows of y begin
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int li = lane & 31, lh = lane >> 5;
  const int group = blockIdx.x / stripes;
  const int64_t t0 = (int64_t)group * kTokens;
  // ids of all the tokens (two a lane) decide the form, those of this wave's 32 the work
  const int2 first = t0 + lane < a.rows ? a.order[t0 + lane] : int2{0, -1};
  const int2 second = t0 + 64 + lane < a.rows ? a.order[t0 + 64 + lane] : int2{0, -1};
  const int id_a = first.y, id_b = second.y;
  const int64_t m0 = t0 + 32 * wave;
  const int64_t base = a.sort ? t0 / kSegment * kSegment : m0;
  const int row = __shfl(wave < 2 ? first.x : second.x, 32 * (wave & 1) + li);
  if (lane < 32) sy[32 * wave + li] = (uint32_t)((row - base) * a.ldy * 4);
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // read by this wave only
  const int id = __shfl(wave < 2 ? id_a : id_b, 32 * (wave & 1) + li);
  const bool straight = __ballot((id_a >= 0 && first.x != t0 + lane) || (id_b >= 0 && second.x != t0 + 64 + lane)) == 0;
  Adapters lower(id_a, ~0ull), upper(id_b, ~0ull);
  if (lower.left == 0 && upper.left == 0) return;
  int few = 0;
  {
    Adapters l = lower, u = upper;
    for (; l.left && few <= kFew; ++few) {
      const int ad = l.next();
      u.left &= ~__ballot(u.id == ad);
    }
    for (; u.left && few <= kFew; ++few) u.next();
  }
  const int n_begin = (blockIdx.x - group * stripes) * stripe, n_end = min(a.N, n_begin + stripe);
  const auto yr = resource(a.y + base * a.ldy, ((a.sort ? kSegment : 32) - 1) * a.ldy * 4 + (int64_t)a.N * 4);
  // z of the wave's tokens
  u32x4 z[RS][3];
  auto load_z = [&]() {
    const auto zr = resource(a.planes + m0 * a.R * 3, (int64_t)32 * a.R * 6);
#pragma unroll
    for (int t = 0; t < RS; ++t) {
      const int j = 16 * t + 8 * lh;
      const uint32_t at = id >= 0 && j < a.R ? (uint32_t)((li * a.R + j) * 6) : kNone;
#pragma unroll
      for (int p = 0; p < 3; ++p) z[t][p] = load16(zr, at + 16 * p);
    }
  };
  // Element e of a result is token 8 (e / 4) + 4 lh + e % 4, output li.  Tokens of other
  // adapters are masked.
  // (lane_tokens: bit 8 (e / 4) + e % 4 is the lane's token e)
  auto lane_tokens = [&](uint64_t is) { return lh ? (uint32_t)(is >> 4) : (uint32_t)is; };
  uint32_t mine_of = 0;
  bool whole = false;
  auto set_tokens = [&](uint64_t is) {
    mine_of = lane_tokens(is);
    whole = is == ~0ull;
    return is != 0;
  };
  // f(e, place of element e in y, the part of it that is the wave's).  Tokens of a tile that
  // is straight lie a row apart, those of another where sy says.
  const uint32_t lane_at = (uint32_t)((m0 - base + 4 * lh) * a.ldy * 4);
  auto each_y = [&](auto straight, int n, auto f) {
    const uint32_t at = 4u * (n + li), mine = n + li < n_end ? mine_of : 0u;
    if constexpr (straight) {
      const uint32_t to = n + li < n_end ? lane_at + at : kNone;
#pragma unroll
      for (int e = 0; e < 16; ++e)
        f(e, whole || (mine_of & (1u << (8 * (e / 4) + e % 4))) ? to : kNone, (int)((8 * (e / 4) + e % 4) * a.ldy * 4));
      return;
    }
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const u32x4 r = *reinterpret_cast<const u32x4*>(sy + 32 * wave + 8 * g + 4 * lh);
#pragma unroll
      for (int i = 0; i < 4; ++i) f(4 * g + i, mine & (1u << (8 * g + i)) ? r[i] + at : kNone, 0);
    }
  };
  auto load_y = [&](auto straight, v16f& old, int n) {
    each_y(straight, n, [&](int e, uint32_t at, int wave_at) { old[e] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(yr, at, wave_at, 0)); });
  };
  auto store_y = [&](auto straight, const v16f& old, const v16f& v, int n) {
    each_y(straight, n, [&](int e, uint32_t at, int wave_at) { __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(old[e] + v[e]), yr, at, wave_at, 0); });
  };
  // ranks that an adapter does not have among a lane's eight of step t
  auto cut = [&](u32x4 v, int t, int rank) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int have = rank - (16 * t + 8 * lh + 2 * e);
      v[e] &= have >= 2 ? 0xFFFFFFFFu : have == 1 ? 0x0000FFFFu : 0u;
    }
    return v;
  };
  auto multiply = [&](const u32x4 (&b)[RS], const v16f& old, int n) {
    v16f acc = {};
#pragma unroll
    for (int p = 2; p >= 0; --p)
#pragma unroll
      for (int t = 0; t < RS; ++t) acc = mm32(z[t][p], b[t], acc);
    mfma_settle_before_join();
    store_y(std::true_type{}, old, acc, n);
  };

  if (few <= kFew && straight) {
    bool have_z = false;
    while (lower.left || upper.left) {
      int ad;
      if (lower.left) {
        ad = lower.next();
        upper.left &= ~__ballot(upper.id == ad);
      } else {
        ad = upper.next();
      }
      const int rank = wave_rank_of(a, ad);
      const bool any = set_tokens(__ballot(id == ad));
      const auto br = resource(a.B + (int64_t)ad * a.N * a.R, (int64_t)a.N * a.R * 2);  // outputs from N on lie outside
      u32x4 b[BN > 0 ? BN : 1];
      auto load_b = [&](int n0) {
#pragma unroll
        for (int i = 0; i < (BN > 0 ? BN : 1); ++i) {
          const int n = (int)threadIdx.x / BL + i * (256 / BL), j = (int)(threadIdx.x % BL) * 8;
          b[i] = load16(br, j < rank && n0 < n_end ? (uint32_t)(((n0 + n) * a.R + j) * 2) : kNone);
        }
      };
      auto stage_b = [&]() {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < (BN > 0 ? BN : 1); ++i) {
          const int n = (int)threadIdx.x / BL + i * (256 / BL);
          if (BN > 0 || n < NB) *reinterpret_cast<u32x4*>(sb + n * BS + (threadIdx.x % BL) * 16) = b[i];
        }
        __syncthreads();
      };
      load_b(n_begin);
      if (!any) {  // another wave's adapter: help with B
        for (int n0 = n_begin; n0 < n_end; n0 += NB) {
          stage_b();
          load_b(n0 + NB);
        }
        continue;
      }
      v16f old[2];
      load_y(std::true_type{}, old[0], n_begin);
      load_y(std::true_type{}, old[1], n_begin + 32);
      if (!have_z) load_z();
      have_z = true;
      for (int n0 = n_begin; n0 < n_end; n0 += NB) {
        stage_b();
        load_b(n0 + NB);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          u32x4 bo[RS];
#pragma unroll
          for (int t = 0; t < RS; ++t) bo[t] = *reinterpret_cast<const u32x4*>(sb + (32 * h + li) * BS + (16 * t + 8 * lh) * 2);
          if (rank & 7) {
#pragma unroll
            for (int t = 0; t < RS; ++t) bo[t] = cut(bo[t], t, rank);
          }
          multiply(bo, old[h], n0 + 32 * h);
          load_y(std::true_type{}, old[h], n0 + NB + 32 * h);
        }
      }
    }
    return;
  }

  // many adapters: a wave for itself, 64 outputs at a time through its adapters; the
  // result of each token is picked from its own's, y is read and written once
  Adapters own(id, 0xFFFFFFFFull);
  if (own.left == 0) return;
  load_z();
  set_tokens(__ballot(id >= 0));
  struct Part {
    u32x4 b[2][RS];
    int ad, rank;
  };
  for (int n = n_begin; n < n_end; n += NB) {
    v16f old[2], got[2] = {};
    load_y(std::false_type{}, old[0], n);
    load_y(std::false_type{}, old[1], n + 32);
    Adapters left = own;
    // the next adapter's part of B; always the same number of loads, so that the wait for
    // one part leaves the next one's under way
    auto load_part = [&](Part& s) {
      s.ad = left.next_or_none();
      s.rank = s.ad >= 0 ? wave_rank_of(a, s.ad) : 0;
      const auto br = resource(a.B + (int64_t)max(s.ad, 0) * a.N * a.R, (int64_t)a.N * a.R * 2);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int t = 0; t < RS; ++t) {
          const int j = 16 * t + 8 * lh;
          s.b[h][t] = load16(br, j < s.rank ? (uint32_t)(((n + 32 * h + li) * a.R + j) * 2) : kNone);
        }
    };
    auto pick = [&](Part& s) {
      const uint32_t is = lane_tokens(__ballot(id == s.ad));
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (s.rank & 7) {
#pragma unroll
          for (int t = 0; t < RS; ++t) s.b[h][t] = cut(s.b[h][t], t, s.rank);
        }
        v16f acc = {};
#pragma unroll
        for (int p = 2; p >= 0; --p)
#pragma unroll
          for (int t = 0; t < RS; ++t) acc = mm32(z[t][p], s.b[h][t], acc);
        mfma_settle_before_join();
#pragma unroll
        for (int e = 0; e < 16; ++e) got[h][e] = is & (1u << (8 * (e / 4) + e % 4)) ? acc[e] : got[h][e];
      }
    };
    Part p0, p1;
    load_part(p0);
    for (;;) {
      load_part(p1);
      pick(p0);
      if (p1.ad < 0) break;
      load_part(p0);
      pick(p1);
      if (p0.ad < 0) break;
    }
    store_y(std::false_type{}, old[0], got[0], n);
    store_y(std::false_type{}, old[1], got[1], n + 32);
  }
}

// Two work-groups a CU, each with 128 elements of K at least.  The prompts of the head
// of this file: 2 splits 23.4 us, 4 (this rule) 23.0, 8 26.7, 16 30.8; fp32 x: 42, 39, 39, 43.
constexpr int kShrinkGroups = 512;
int splits_for(int64_t rows, int K) {
  const int64_t tiles = (rows + kTile - 1) / kTile;
  const int64_t want = kShrinkGroups / tiles, most = (K + 127) / 128;
  const int64_t n = want < most ? want : most;
  return (int)(n < 1 ? 1 : n > kMaxSplits ? kMaxSplits : n);
}

template <int RT>
void shrink_tiles(const AdapterArgs& a, dim3 grid, hipStream_t s) {
  if (a.x_bf16) shrink_tile_kernel<1, RT><<<grid, 256, 0, s>>>(a);
  else shrink_tile_kernel<0, RT><<<grid, 256, 0, s>>>(a);
}

hipError_t launch_tiles(const AdapterArgs& a, hipStream_t s) {
  const int splits = splits_for(a.rows, a.K);
  const dim3 shrink((a.rows + kTile - 1) / kTile, splits);
  if (a.R <= 16) shrink_tiles<1>(a, shrink, s);
  else if (a.R <= 32) shrink_tiles<2>(a, shrink, s);
  else if (a.R <= 64) shrink_tiles<4>(a, shrink, s);
  else shrink_tiles<8>(a, shrink, s);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  join_kernel<<<(unsigned)(((int64_t)a.rows * (a.R / 8) + 255) / 256), 256, 0, s>>>(a, splits);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int groups = (a.rows + kTokens - 1) / kTokens, blocks = (a.N + 63) / 64;
  // six and four work-groups a CU, of which two and one fit at once
  int stripes = ((a.R <= 64 ? 1536 : 1024) + groups - 1) / groups;
  if (stripes > blocks) stripes = blocks;
  const int stripe = (blocks + stripes - 1) / stripes * 64;
  stripes = (a.N + stripe - 1) / stripe;
  void (*fn)(AdapterArgs, int, int) = a.R <= 16   ? expand_tile_kernel<1>
                                           : a.R <= 32 ? expand_tile_kernel<2>
                                           : a.R <= 64 ? expand_tile_kernel<4>
                                                       : expand_tile_kernel<8>;
  fn<<<groups * stripes, 256, 0, s>>>(a, stripe, stripes);
  return hipGetLastError();
}

}  // namespace

// z of each split of K, its planes, the order.  splits_for falls in steps as rows grow, so
// splits times rows goes up and down: room is taken for the most that it reaches for any
// number of rows up to this one and any K, and what serves a batch serves every smaller one.
static size_t sums_bytes(int64_t rows, int max_rank) {
  const int64_t split = std::min<int64_t>(kMaxSplits * rows, kShrinkGroups * kTile);
  return (size_t)(std::max(rows, split) * max_rank * 4 + 255) / 256 * 256;
}
static size_t planes_bytes(int64_t rows, int max_rank) { return (size_t)(rows * max_rank * 6 + 255) / 256 * 256; }
size_t adapter_workspace_bytes(int64_t rows, int max_rank) {
  return sums_bytes(rows, max_rank) + planes_bytes(rows, max_rank) + (size_t)(rows * 8 + 255) / 256 * 256;
}

hipError_t launch_adapter(AdapterArgs a, hipStream_t s) {
  char* at = reinterpret_cast<char*>(a.z) + sums_bytes(a.rows, a.R);
  a.planes = reinterpret_cast<uint16_t*>(at);
  a.order = reinterpret_cast<int2*>(at + planes_bytes(a.rows, a.R));
  // a segment's rows of x and of y lie within 2^31 bytes, but for matrices of far wider rows
  const int64_t most = (int64_t)1 << 31, item = a.x_bf16 ? 2 : 4;
  a.sort = (kSegment - 1) * a.ldx * item + a.K * item < most && (kSegment - 1) * a.ldy * 4 + (int64_t)a.N * 4 < most;
  // Few rows go one by one: tiles cost 14 us (in any order 20 and more) before they do
  // anything, rows what they read.  The rule leaves out the rank and the order of the ids, so
  // near the border it takes the slower form in places.  One by one and in tiles, of 4 adapters
  // (the rule's choice starred), K of 2560: rank 16, N of 2560: 256 rows *9 and 14 us, 400 *12
  // and 16, 600 16 and *17, those in any order 16 and *25; N of 6912: 256 rows *16 and 15;
  // rank 64, N of 2560: 400 rows *22 and 21, 600 in any order 30 and *35; N of 6912: 256 rows
  // *29 and 18.  Over 60 sizes around the border (96 to 600 rows, ranks 16 and 64) it takes 5%
  // more time than the better form on average, 65% at worst.
  return (int64_t)a.rows * (a.K + a.N) <= 5 << 19 ? launch_rows(a, s) : launch_tiles(a, s);
}

}  // namespace loopq

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

}  // namespace

size_t adapter_workspace_bytes(int64_t rows, int max_rank) { return (size_t)(rows * max_rank * 4 + 255) / 256 * 256; }

hipError_t launch_adapter(const AdapterArgs& a, hipStream_t s) { return launch_rows(a, s); }

}  // namespace loopq

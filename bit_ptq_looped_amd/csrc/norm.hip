// The residual's addition, the root-mean-square norm and the next linear's
// input, in one pass (include/loopq_block.h has the definitions).
//
// h = x + residual; r = fl32(1 / sqrt(mean h^2 + eps)); z = (h r) w; out: h, z,
// or the Eq.(4) codes and steps of z.  A row's elements stay in registers from
// the load to the last store, so each input is read once and each output
// written once: the kernel is bound by those bytes.
//
// The mean is taken in 64 bits: a square of an fp32 number is exact there (48
// bits) and the sum of 2^15 of them carries an error below 2^-37 of an fp32
// ulp's half, so r is one fp32 number whatever the order of summation, and with
// it the codes, which are compared bit for bit like every code of this library.
// It costs one conversion and one fp64 FMA an element, about a sixth of the
// vector issue of a kernel that waits for memory.
#include "block_internal.h"
#include "quant_core.h"

namespace loopq {
namespace {

__device__ __forceinline__ float4 load4(const void* p, int64_t at, bool bf16) {
  if (bf16) {
    const uint2 u = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(p) + at);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xFFFF0000u));
  }
  return *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(p) + at);
}

__device__ __forceinline__ uint2 round4(const float4& v) {
  return uint2{bf16x2_rne(v.x, v.y), bf16x2_rne(v.z, v.w)};
}

__device__ __forceinline__ void store4(void* p, int64_t at, const float4& v, bool bf16) {
  if (bf16) *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p) + at) = round4(v);
  else *reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + at) = v;
}

// Sum and maximum over the T threads of a row: T <= 64 lanes of one wave, or
// the whole work-group of T threads (part: one value a wave).  Every thread gets
// the same bits, the order is fixed.
template <int T>
__device__ __forceinline__ double row_sum(double v, double* part) {
#pragma unroll
  for (int o = (T < 64 ? T : 64) / 2; o > 0; o >>= 1) v += __shfl_xor(v, o);
  if constexpr (T > 64) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = part[0];
#pragma unroll
    for (int w = 1; w < T / 64; ++w) v += part[w];
  }
  return v;
}
template <int T>
__device__ __forceinline__ float row_max(float v, float* part) {
#pragma unroll
  for (int o = (T < 64 ? T : 64) / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
  if constexpr (T > 64) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = part[0];
#pragma unroll
    for (int w = 1; w < T / 64; ++w) v = fmaxf(v, part[w]);
  }
  return v;
}

__device__ __forceinline__ float amax4(const float4& v) {
  return fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
}

// T threads a row, NC runs of four elements a thread (K <= 4 T NC): run c of
// thread l starts at 4 (l + T c), so a load instruction of a wave covers 64
// consecutive runs, and a group of 32 elements lies in eight consecutive lanes.
// X: x is bf16.  R: residual none (0), fp32 (1), bf16 (2).
template <int T, int NC, int X, int R>
__global__ __launch_bounds__(T < 256 ? 256 : T) void norm_kernel(NormArgs a) {
  __shared__ double part_sum[T > 64 ? T / 64 : 1];
  __shared__ float part_max[T > 64 ? T / 64 : 1];
  const int64_t row = a.row0 + (T < 256 ? (int64_t)blockIdx.x * (256 / T) + threadIdx.x / T : (int64_t)blockIdx.x);
  if (row >= a.rows) return;  // all T threads of a row together
  const int l = T < 256 ? threadIdx.x % T : threadIdx.x;
  float4 h[NC], w[NC];
  auto k_of = [&](int c) { return 4 * (l + T * c); };
  {
    float4 q[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int k = k_of(c);
      h[c] = k < a.K ? load4(a.x, row * a.ldx + k, X) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if constexpr (R != 0) q[c] = k < a.K ? load4(a.res, row * a.ldr + k, R == 2) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    if constexpr (R != 0) {
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        h[c] = make_float4(h[c].x + q[c].x, h[c].y + q[c].y, h[c].z + q[c].z, h[c].w + q[c].w);
        if constexpr (R == 2) {
          const uint2 u = round4(h[c]);
          h[c] = make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                             __uint_as_float(u.y & 0xFFFF0000u));
        }
      }
    }
  }
  if (a.w != nullptr) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
      if (k_of(c) < a.K) w[c] = *reinterpret_cast<const float4*>(a.w + k_of(c));
  }
  double ss = 0.0;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const double e0 = h[c].x, e1 = h[c].y, e2 = h[c].z, e3 = h[c].w;
    ss = __builtin_fma(e0, e0, ss);
    ss = __builtin_fma(e1, e1, ss);
    ss = __builtin_fma(e2, e2, ss);
    ss = __builtin_fma(e3, e3, ss);
  }
  const double mean = row_sum<T>(ss, part_sum) / (double)a.K;
  const bool finite = mean < __builtin_huge_val();  // false for NaN: fp32 squares do not overflow 64 bits
  const float r = (float)(1.0 / __builtin_sqrt(mean + (double)a.eps));

  if (R != 0 && a.sum != nullptr) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
      if (k_of(c) < a.K) store4(a.sum, row * a.lds + k_of(c), h[c], R == 2);
  }
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    h[c] = make_float4(h[c].x * r, h[c].y * r, h[c].z * r, h[c].w * r);
    if (a.w != nullptr) h[c] = make_float4(h[c].x * w[c].x, h[c].y * w[c].y, h[c].z * w[c].z, h[c].w * w[c].w);
  }
  if (a.y != nullptr) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
      if (k_of(c) < a.K) store4(a.y, row * a.ldy + k_of(c), h[c], a.y_bf16);
  }
  if (a.codes == nullptr) return;
  const float rq = 1.0f / a.qmax;
  float row_step = 0.0f;
  if (a.per_token) {
    float m = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c)
      if (k_of(c) < a.K) m = fmaxf(m, amax4(h[c]));
    row_step = step_of(row_max<T>(m, part_max), a.clip, a.qmax, rq);
  }
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int k = k_of(c);
    float s = row_step;
    if (!a.per_token) s = step_of(group8_max(amax4(h[c])), a.clip, a.qmax, rq);
    uint32_t packed = codes4(h[c], s, a.qmax);
    if (!finite) {
      packed = 0u;
      s = __builtin_nanf("");
    }
    if (k < a.K) {
      *reinterpret_cast<uint32_t*>(a.codes + row * a.K + k) = packed;
      if ((l & 7) == 0) a.steps[row * (a.K / 32) + k / 32] = s;
    }
  }
}

template <int T, int NC>
hipError_t launch_form(NormArgs a, hipStream_t s) {
  const int r = a.res == nullptr ? 0 : a.res_bf16 ? 2 : 1;
  void (*fn)(NormArgs) = a.x_bf16 ? (r == 0 ? norm_kernel<T, NC, 1, 0> : r == 1 ? norm_kernel<T, NC, 1, 1> : norm_kernel<T, NC, 1, 2>)
                                  : (r == 0 ? norm_kernel<T, NC, 0, 0> : r == 1 ? norm_kernel<T, NC, 0, 1> : norm_kernel<T, NC, 0, 2>);
  constexpr int block = T < 256 ? 256 : T, per = block / T;
  // a launch has fewer than 2^32 work-items
  constexpr int64_t most = ((((int64_t)1 << 32) - block) / block) * per;
  for (int64_t at = 0; at < a.rows; at += most) {
    NormArgs b = a;
    b.row0 = at;
    const int64_t n = a.rows - at < most ? a.rows - at : most;
    fn<<<(unsigned)((n + per - 1) / per), block, 0, s>>>(b);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_rms_norm(NormArgs a, hipStream_t s) {
  const int K = a.K;
  if (a.rows < 1024 && K > 512) {  // few rows: a work-group each
    if (K <= 1024) return launch_form<256, 1>(a, s);
    if (K <= 2048) return launch_form<256, 2>(a, s);
    if (K <= 4096) return launch_form<256, 4>(a, s);
  }
  if (K <= 32) return launch_form<8, 1>(a, s);
  if (K <= 64) return launch_form<16, 1>(a, s);
  if (K <= 128) return launch_form<32, 1>(a, s);
  if (K <= 256) return launch_form<64, 1>(a, s);
  if (K <= 512) return launch_form<64, 2>(a, s);
  if (K <= 1024) return launch_form<64, 4>(a, s);
  if (K <= 2048) return launch_form<64, 8>(a, s);
  if (K <= 2560) return launch_form<64, 10>(a, s);
  if (K <= 4096) return launch_form<64, 16>(a, s);
  if (K <= 8192) return launch_form<256, 8>(a, s);
  if (K <= 16384) return launch_form<1024, 4>(a, s);
  return launch_form<1024, 8>(a, s);
}

}  // namespace loopq

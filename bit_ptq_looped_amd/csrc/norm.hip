// The residual's addition, the root-mean-square norm and the next linear's
// input, in one pass (include/loopq_block.h has the definitions).
//
// h = x + residual; r = fl32(1 / sqrt(mean h^2 + eps)); z = (h r) w; out: h, z,
// or the Eq.(4) codes and steps of z.  A row's elements stay in registers from
// the load to the last store, so each input is read once and each output
// written once: the kernel is bound by those bytes, but where bf16 rows without a
// residual become codes.  There some 26 vector instructions an element (the squares in 64
// bits, the quotients and their check, packing) take 87% of the launch's cycles.
//
// The mean is taken in 64 bits: a square of an fp32 number is exact there (48 bits), the
// sum of a row's squares is rounded at most 52 times on the way of any of them (4 NC - 1 in
// a thread, 6 between lanes, 15 between waves, in the longest form), and 1 / K, the
// product with it and eps take a rounding each: 55 2^-53, of which the root takes half.
// With the root's own 2^-52 the value that becomes r is within 2^-48 of itself.  So r is one
// fp32 number whatever the order of summation, but for a row whose exact value lies that
// close to the border between two of them (less than one in 2^23), and with it the codes,
// which are compared bit for bit like every code of this library.
// It costs one conversion and one fp64 FMA an element, in a kernel that waits for
// memory: 8192 rows of 2560, fp32 with an fp32 residual into sums and 8-bit codes, take
// 50 us (275 MB, 5.5 TB/s; a large copy reaches 4.8), bf16 to bf16 19, 4096 of 6912 bf16
// with one step a token 26; one row of 2048 2.5, of which most is the launch.
#include "block_internal.h"
#include "quant_core.h"

namespace loopq {
namespace {

// Threads a CU is given, at most: a CU holds 512 to 2048 by the form's registers (1280 as
// <256, 3>, 1024 as <256, 7> of bf16), so four to sixteen times that, and a work-group takes
// a few rows where there are very many while the last ones end together.  8192 rows
// of 2560, fp32 with an fp32 residual: 2048 threads 54 us, 8192 50; bf16 18.2 and 18.5.
constexpr int kNormThreads = 8192;

// four consecutive elements as they lie
template <int BF>
struct Run {
  uint32_t u[BF ? 2 : 4];
  __device__ __forceinline__ void load(const void* p, int64_t at) {
    if constexpr (BF) {
      const uint2 v = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(p) + at);
      u[0] = v.x, u[1] = v.y;
    } else {
      const uint4 v = *reinterpret_cast<const uint4*>(reinterpret_cast<const float*>(p) + at);
      u[0] = v.x, u[1] = v.y, u[2] = v.z, u[3] = v.w;
    }
  }
  __device__ __forceinline__ float4 floats() const {
    if constexpr (BF)
      return make_float4(__uint_as_float(u[0] << 16), __uint_as_float(u[0] & 0xFFFF0000u), __uint_as_float(u[1] << 16),
                         __uint_as_float(u[1] & 0xFFFF0000u));
    else
      return make_float4(__uint_as_float(u[0]), __uint_as_float(u[1]), __uint_as_float(u[2]), __uint_as_float(u[3]));
  }
};

__device__ __forceinline__ uint2 round4(const float4& v) {
  return uint2{bf16x2_rne(v.x, v.y), bf16x2_rne(v.z, v.w)};
}

__device__ __forceinline__ void store4(void* p, int64_t at, const float4& v, bool bf16) {
  if (bf16) *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(p) + at) = round4(v);
  else *reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + at) = v;
}

// Sum and maximum over the T threads of a row: T <= 64 lanes of one wave, or
// the whole work-group of T threads (part: one value a wave).  Every thread gets
// the same bits, the order is fixed.  Lanes exchange by DPP within 16 and by the
// swaps of 16 and 32 lanes: no trip through LDS.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}
// v of the lane 2^S away, in the sense of a butterfly over aligned runs of 2^(S+1) lanes:
// the other of the pair, the quad's other half, the mirrored half row, the mirrored row
template <int S>
__device__ __forceinline__ uint32_t across(uint32_t v) {
  if constexpr (S == 0) return dpp<0xB1>(v);
  else if constexpr (S == 1) return dpp<0x4E>(v);
  else if constexpr (S == 2) return dpp<0x141>(v);
  else return dpp<0x140>(v);
}
// both halves of 2 x 16 or 2 x 32 lanes, in every lane: {lower, upper}
template <int S>
__device__ __forceinline__ void halves(uint32_t v, uint32_t* lower, uint32_t* upper) {
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  u32x2 r;
  if constexpr (S == 4) r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  else r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  *lower = r[0];
  *upper = r[1];
}
template <int S>
__device__ __forceinline__ double sum_step(double v) {
  const uint64_t u = __double_as_longlong(v);
  if constexpr (S < 4) {
    const uint64_t w = (uint64_t)across<S>((uint32_t)(u >> 32)) << 32 | across<S>((uint32_t)u);
    return v + __longlong_as_double((long long)w);
  } else {
    uint32_t l0, l1, h0, h1;
    halves<S>((uint32_t)u, &l0, &l1);
    halves<S>((uint32_t)(u >> 32), &h0, &h1);
    return __longlong_as_double((long long)((uint64_t)h0 << 32 | l0)) + __longlong_as_double((long long)((uint64_t)h1 << 32 | l1));
  }
}
template <int S>
__device__ __forceinline__ float max_step(float v) {
  if constexpr (S < 4) {
    return fmaxf(v, __uint_as_float(across<S>(__float_as_uint(v))));
  } else {
    uint32_t a, b;
    halves<S>(__float_as_uint(v), &a, &b);
    return fmaxf(__uint_as_float(a), __uint_as_float(b));
  }
}
template <int T>
__device__ __forceinline__ double row_sum(double v, double* part) {
  v = sum_step<0>(v);
  v = sum_step<1>(v);
  v = sum_step<2>(v);
  if constexpr (T >= 16) v = sum_step<3>(v);
  if constexpr (T >= 32) v = sum_step<4>(v);
  if constexpr (T >= 64) v = sum_step<5>(v);
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
  v = max_step<0>(v);
  v = max_step<1>(v);
  v = max_step<2>(v);
  if constexpr (T >= 16) v = max_step<3>(v);
  if constexpr (T >= 32) v = max_step<4>(v);
  if constexpr (T >= 64) v = max_step<5>(v);
  if constexpr (T > 64) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = part[0];
#pragma unroll
    for (int w = 1; w < T / 64; ++w) v = fmaxf(v, part[w]);
  }
  return v;
}

// fl32(1 / sqrt(mean + eps)).  The hardware's reciprocal root y carries some 24 bits; with
// e = 1 - v y^2 the root is y (1 - e)^(-1/2) = y (1 + e / 2 + 3 e^2 / 8 + ..), and what is left
// out, 5 e^3 / 16, lies below 2^-65: e is off by the rounding of v y, at most 2^-53, which
// halves, and the last FMA rounds once more.  Below 2^-52 together.
__device__ __forceinline__ float reciprocal_root(double mean, double eps) {
  const double v = mean + eps;
  const double y = __builtin_amdgcn_rsq(v);
  const double e = __builtin_fma(-v * y, y, 1.0);
  const float r = (float)__builtin_fma(y * e, __builtin_fma(0.375, e, 0.5), y);
  return v < __builtin_huge_val() ? r : (float)y;  // infinite: 0, NaN: NaN
}

__device__ __forceinline__ float amax4(const float4& v) {
  return fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
}

// T threads a row, NC runs of four elements a thread (K <= 4 T NC): run c of
// thread l starts at 4 (l + T c), so a load instruction of a wave covers 64
// consecutive runs, and a group of 32 elements lies in eight consecutive lanes.
// A work-group (or its 256 / T parts) goes on from row to row: the next row is
// loaded while one is worked on, and the weights are read once.  T = 1024 takes one
// row only: its 16 waves have 128 registers each, and the next row would spill.
// X: x is bf16.  R: residual none (0), fp32 (1), bf16 (2).
template <int T, int NC, int X, int R>
__global__ __launch_bounds__(T < 128 ? 256 : T) void norm_kernel(NormArgs a) {
  constexpr int W = T > 64 ? T / 64 : 1;
  __shared__ double part_sum[2][W];  // in turns: a wave may be a row ahead of another
  __shared__ float part_max[2][W];
  const int64_t step = (int64_t)gridDim.x * (T < 128 ? 256 / T : 1);
  constexpr bool ahead = T < 1024;
  int64_t row = a.row0 + (T < 128 ? (int64_t)blockIdx.x * (256 / T) + threadIdx.x / T : (int64_t)blockIdx.x);
  if (row >= a.rows) return;  // all T threads of a row together
  const int l = T < 128 ? threadIdx.x % T : threadIdx.x;
  auto k_of = [&](int c) { return 4 * (l + T * c); };
  Run<X> x[NC];
  Run<R == 2> q[R != 0 ? NC : 1];
  auto load = [&](int64_t m) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
      if (k_of(c) < a.K) x[c].load(a.x, m * a.ldx + k_of(c));
    if constexpr (R != 0) {
#pragma unroll
      for (int c = 0; c < NC; ++c)
        if (k_of(c) < a.K) q[c].load(a.res, m * a.ldr + k_of(c));
    }
  };
  load(row);
  float4 w[NC];
  if (a.w != nullptr) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
      if (k_of(c) < a.K) w[c] = *reinterpret_cast<const float4*>(a.w + k_of(c));
  }
  const float rq = 1.0f / a.qmax;
  for (int turn = 0; row < a.rows; row = ahead ? row + step : a.rows, turn ^= 1) {
    float4 h[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      h[c] = x[c].floats();
      if constexpr (R != 0) {
        const float4 v = q[c].floats();
        h[c] = make_float4(h[c].x + v.x, h[c].y + v.y, h[c].z + v.z, h[c].w + v.w);
        if constexpr (R == 2) {
          const uint2 u = round4(h[c]);
          h[c] = make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                             __uint_as_float(u.y & 0xFFFF0000u));
        }
      }
      if (k_of(c) >= a.K) h[c] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    if (ahead && row + step < a.rows) load(row + step);
    double ss = 0.0;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const double e0 = h[c].x, e1 = h[c].y, e2 = h[c].z, e3 = h[c].w;
      ss = __builtin_fma(e0, e0, ss);
      ss = __builtin_fma(e1, e1, ss);
      ss = __builtin_fma(e2, e2, ss);
      ss = __builtin_fma(e3, e3, ss);
    }
    const double mean = row_sum<T>(ss, part_sum[turn]) * a.inv_k;
    const bool finite = mean < __builtin_huge_val();  // false for NaN: fp32 squares do not overflow 64 bits
    const float r = reciprocal_root(mean, (double)a.eps);

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
    if (a.codes == nullptr) continue;
    float row_step = 0.0f;
    if (a.per_token) {
      float m = 0.0f;
#pragma unroll
      for (int c = 0; c < NC; ++c)
        if (k_of(c) < a.K) m = fmaxf(m, amax4(h[c]));
      row_step = step_of(row_max<T>(m, part_max[turn]), a.clip, a.qmax, rq);
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
}

template <int T, int NC>
hipError_t launch_form(const NormArgs& a, hipStream_t s) {
  const int r = a.res == nullptr ? 0 : a.res_bf16 ? 2 : 1;
  void (*fn)(NormArgs) = a.x_bf16 ? (r == 0 ? norm_kernel<T, NC, 1, 0> : r == 1 ? norm_kernel<T, NC, 1, 1> : norm_kernel<T, NC, 1, 2>)
                                  : (r == 0 ? norm_kernel<T, NC, 0, 0> : r == 1 ? norm_kernel<T, NC, 0, 1> : norm_kernel<T, NC, 0, 2>);
  constexpr int block = T < 128 ? 256 : T, per = block / T;
  // a launch has fewer than 2^32 work-items
  constexpr int64_t most = T < 1024 ? (int64_t)1 << 31 : ((int64_t)1 << 22) - 1;
  NormArgs b = a;
  for (b.row0 = 0; b.row0 < a.rows; b.row0 += most) {
    const int64_t left = a.rows - b.row0, groups = ((left < most ? left : most) + per - 1) / per;
    const int64_t held = (int64_t)device_cu_count() * kNormThreads / block;
    fn<<<(unsigned)(T < 1024 && held < groups ? held : groups), block, 0, s>>>(b);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_rms_norm(const NormArgs& a, hipStream_t s) {
  // Two to seven runs a thread, but one for the shortest rows and for few rows, and eight
  // for the longest.  With fewer, a wave's own work (the root, the exchange
  // between lanes, its start) shows: 8192 bf16 rows of 2560 take 18.2 us as <256, 3> and
  // 20.4 as <512, 2>, 4096 of 6912 with one step a token 27 as <256, 7>, 31 as <512, 4>.
  // With more, too few waves fit a CU: the 8192 rows take 20.8 us as <64, 10>.
  auto fits = [&](int t, int nc) { return a.K <= 4 * t * nc; };
  if (fits(8, 1)) return launch_form<8, 1>(a, s);
  if (fits(8, 2)) return launch_form<8, 2>(a, s);
  if (fits(16, 2)) return launch_form<16, 2>(a, s);
  if (fits(32, 2)) return launch_form<32, 2>(a, s);
  if (fits(64, 2)) return launch_form<64, 2>(a, s);
  if (a.rows < 512) {  // few rows: the time of one counts (48 rows of 2560: <256, 3> 3.6 us, <512, 2> 3.4)
    if (fits(256, 1)) return launch_form<256, 1>(a, s);
    if (fits(512, 1)) return launch_form<512, 1>(a, s);
    if (fits(512, 2)) return launch_form<512, 2>(a, s);
    if (fits(1024, 2)) return launch_form<1024, 2>(a, s);
  }
  if (fits(128, 2)) return launch_form<128, 2>(a, s);
  if (fits(256, 2)) return launch_form<256, 2>(a, s);
  if (fits(256, 3)) return launch_form<256, 3>(a, s);
  if (fits(256, 5)) return launch_form<256, 5>(a, s);
  if (fits(256, 7)) return launch_form<256, 7>(a, s);
  if (fits(512, 4)) return launch_form<512, 4>(a, s);
  if (fits(1024, 3)) return launch_form<1024, 3>(a, s);
  if (fits(1024, 5)) return launch_form<1024, 5>(a, s);
  return launch_form<1024, 8>(a, s);
}

}  // namespace loopq

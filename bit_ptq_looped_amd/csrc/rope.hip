// Rotary positions, alone and with the cache write (include/loopq_block.h has
// the definitions).
//
// A wave takes one token and a range of its heads: lane i < rot_dim / 2 forms
// the sine and cosine of frequency i once, for all of these heads.  The angle is
// taken in turns, p inv_freq / 2 pi, in 64 bits, where the fraction of a turn is
// what is left after the nearest whole number is taken off exactly; so far
// positions cost no precision, and sine and cosine of half turns (sincospif)
// need no reduction of their own.  The work is bound by the bytes of the
// tensors: the first heads' loads are issued before the position is looked up.
//
// The row of a token is found by a search of the wave, 64 probes of cu at once:
// one trip to memory for up to 64 rows, two up to 4096.
#include "block_internal.h"
#include "quant_core.h"

namespace loopq {
namespace {

struct Place {
  double pos;
  bool skip;   // behind the last row: nothing is written
  bool paged;  // the position has a page
  uint16_t* dst;  // head 0's keys of the token in the slab
};

__device__ __forceinline__ Place find_place(const RopeArgs& a, int64_t t, int lane) {
  Place p{0.0, false, false, nullptr};
  if (a.positions != nullptr) {
    p.pos = (double)a.positions[t];
    return p;
  }
  int lo = 0, hi = a.t.rows;
  const int32_t first = a.cu[0], last = a.cu[hi];
  while (hi - lo > 1) {  // cu[lo] <= t < cu[hi]
    const int step = (hi - lo + 63) >> 6;
    const int64_t at = (int64_t)lo + (int64_t)(lane + 1) * step;
    const bool below = at < hi && a.cu[at < hi ? at : lo] <= t;
    const int n = __popcll(__ballot(below));
    lo += n * step;
    hi = min(hi, lo + step);
  }
  lo = __builtin_amdgcn_readfirstlane(lo);
  p.skip = t < first || t >= last;
  if (p.skip) return p;
  const int64_t cap = (int64_t)a.t.width << a.page_shift;
  int64_t n = a.t.lens[lo];
  n = n < 0 ? 0 : n > cap ? cap : n;
  const int64_t pos = n - a.cu[lo + 1] + t;
  p.pos = (double)pos;
  if (pos < 0 || pos >= cap) return p;
  const int page = a.t.table[(int64_t)lo * a.t.width + (pos >> a.page_shift)];
  p.paged = page >= 0 && page < a.t.pages;
  if (p.paged) p.dst = a.pool + (int64_t)page * a.page_stride + (pos & ((1 << a.page_shift) - 1)) * a.head_dim;
  return p;
}

// magnitude times sine and cosine of lane i's frequency
__device__ __forceinline__ void turn_of(const RopeArgs& a, double pos, int i, float* c, float* s) {
  const double turns = pos * (a.inv_freq[i] * 0.15915494309189533577);  // 1 / 2 pi
  const float half_turns = 2.0f * (float)(turns - __builtin_rint(turns));
  float cs, sn;
  sincospif(half_turns, &sn, &cs);
  *c = a.magnitude * cs;
  *s = a.magnitude * sn;
}

// The head of a token: which tensor it is in, and its index there.
__device__ __forceinline__ int part_of(const RopeArgs& a, int head, int* at) {
  int p = 0;
  if (head >= a.part[0].heads) {
    head -= a.part[0].heads;
    p = 1;
    if (head >= a.part[1].heads) {
      head -= a.part[1].heads;
      p = 2;
    }
  }
  *at = head;
  return p;
}

template <int BF>
struct Eight {
  uint4 raw[BF ? 1 : 2];
  __device__ __forceinline__ void load(const void* p, int64_t at) {
    const uint4* s = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(p) + at * (BF ? 2 : 4));
    raw[0] = s[0];
    if constexpr (!BF) raw[1] = s[1];
  }
  __device__ __forceinline__ void floats(float (&v)[8]) const {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(raw);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (BF) v[i] = __uint_as_float((i & 1) ? u[i / 2] & 0xFFFF0000u : u[i / 2] << 16);
      else v[i] = __uint_as_float(u[i]);
    }
  }
};

__device__ __forceinline__ void store8(void* p, int64_t at, const float (&v)[8], bool bf16) {
  if (bf16) {
    *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(p) + at) =
        uint4{bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]), bf16x2_rne(v[4], v[5]), bf16x2_rne(v[6], v[7])};
  } else {
    float4* d = reinterpret_cast<float4*>(reinterpret_cast<float*>(p) + at);
    d[0] = make_float4(v[0], v[1], v[2], v[3]);
    d[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

// rot_dim a multiple of 16: a lane takes sixteen elements of a head, the two
// halves of eight pairs (HALF) or eight pairs side by side, in 16-byte accesses.
// 64 / (D / 16) heads a pass; the next pass is loaded while one is turned.
template <int D, int BF>
__global__ __launch_bounds__(256) void rope_vec_kernel(RopeArgs a) {
  constexpr int S = D / 16, HP = 64 / S;
  const int lane = threadIdx.x & 63;
  const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t t = w / a.split;
  if (t >= a.tokens) return;
  const int slot = lane % S, hl = lane / S;
  const int h0 = (int)(w - t * a.split) * a.per;
  const int h1 = min(h0 + a.per, a.heads);
  const bool turned = slot < a.rot / 16;
  const int e0 = !a.pairs && turned ? 8 * slot : 16 * slot;
  const int e1 = !a.pairs && turned ? a.rot / 2 + 8 * slot : 16 * slot + 8;
  Eight<BF> x0, x1;
  auto load = [&](int head) {
    if (hl < HP && head < h1) {
      int at;
      const RopePart& p = a.part[part_of(a, head, &at)];
      const int64_t base = t * p.ld_in + (int64_t)at * D;
      x0.load(p.in, base + e0);
      x1.load(p.in, base + e1);
    }
  };
  load(h0 + hl);
  const Place pl = find_place(a, t, lane);
  if (pl.skip) return;
  float cl = 0.0f, sl = 0.0f;
  if (lane < a.rot / 2) turn_of(a, pl.pos, lane, &cl, &sl);
  float c[8], s[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    c[j] = __shfl(cl, (8 * slot + j) & 63);
    s[j] = __shfl(sl, (8 * slot + j) & 63);
  }
  for (int head = h0 + hl; head - hl < h1; head += HP) {
    float u[8], v[8];
    x0.floats(u);
    x1.floats(v);
    load(head + HP);
    if (hl >= HP || head >= h1) continue;
    int at;
    const int which = part_of(a, head, &at);
    if (which != 2 && turned) {
      if (a.pairs) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float p = u[2 * j], q = u[2 * j + 1], y = v[2 * j], z = v[2 * j + 1];
          u[2 * j] = p * c[j] - q * s[j];
          u[2 * j + 1] = q * c[j] + p * s[j];
          v[2 * j] = y * c[4 + j] - z * s[4 + j];
          v[2 * j + 1] = z * c[4 + j] + y * s[4 + j];
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float p = u[j], q = v[j];
          u[j] = p * c[j] - q * s[j];
          v[j] = q * c[j] + p * s[j];
        }
      }
    }
    // the values of a head lie as its keys and values do: whole elements of the turned part,
    // so a value's sixteen elements are the lane's whatever they are
    if (which == 0) {
      const RopePart& p = a.part[0];
      const int64_t base = t * p.ld_out + (int64_t)at * D;
      store8(p.out, base + e0, u, p.out_bf16);
      store8(p.out, base + e1, v, p.out_bf16);
    } else if (pl.paged) {
      uint16_t* d = pl.dst + ((int64_t)at << a.page_shift) * D + (which == 2 ? a.plane : 0);
      store8(d, e0, u, true);
      store8(d, e1, v, true);
    }
  }
}

__device__ __forceinline__ float load1(const void* p, int64_t at, bool bf16) {
  return bf16 ? bf16_bits_to_float(reinterpret_cast<const uint16_t*>(p)[at]) : reinterpret_cast<const float*>(p)[at];
}
__device__ __forceinline__ void store1(void* p, int64_t at, float v, bool bf16) {
  if (bf16) reinterpret_cast<uint16_t*>(p)[at] = (uint16_t)bf16x2_rne(v, v);
  else reinterpret_cast<float*>(p)[at] = v;
}

// Any even rot_dim: lane i takes pair i of a head and elements rot_dim + i and
// rot_dim + i + 64 of its rest, single elements side by side, U heads at a time.
__global__ __launch_bounds__(256) void rope_any_kernel(RopeArgs a) {
  constexpr int U = 4;
  const int lane = threadIdx.x & 63;
  const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t t = w / a.split;
  if (t >= a.tokens) return;
  const int D = a.head_dim;
  const int h0 = (int)(w - t * a.split) * a.per;
  const int h1 = min(h0 + a.per, a.heads);
  const Place pl = find_place(a, t, lane);
  if (pl.skip) return;
  const bool pair = lane < a.rot / 2;
  const int ea = a.pairs ? 2 * lane : lane, eb = a.pairs ? 2 * lane + 1 : lane + a.rot / 2;
  float c = 0.0f, s = 0.0f;
  if (pair) turn_of(a, pl.pos, lane, &c, &s);
  for (int g = h0; g < h1; g += U) {
    float x[U][4];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (g + j >= h1) break;
      int at;
      const int which = part_of(a, g + j, &at);
      const RopePart& p = a.part[which];
      const int64_t base = t * p.ld_in + (int64_t)at * D;
      const int from = which == 2 ? 0 : a.rot;
      if (which != 2 && pair) {
        x[j][0] = load1(p.in, base + ea, a.in_bf16);
        x[j][1] = load1(p.in, base + eb, a.in_bf16);
      }
      if (from + lane < D) x[j][2] = load1(p.in, base + from + lane, a.in_bf16);
      if (from + lane + 64 < D) x[j][3] = load1(p.in, base + from + lane + 64, a.in_bf16);
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (g + j >= h1) break;
      int at;
      const int which = part_of(a, g + j, &at);
      void* d;
      int64_t base = 0;
      bool bf16 = true;
      if (which == 0) {
        d = a.part[0].out;
        base = t * a.part[0].ld_out + (int64_t)at * D;
        bf16 = a.part[0].out_bf16;
      } else {
        if (!pl.paged) continue;
        d = pl.dst + ((int64_t)at << a.page_shift) * D + (which == 2 ? a.plane : 0);
      }
      const int from = which == 2 ? 0 : a.rot;
      if (which != 2 && pair) {
        store1(d, base + ea, x[j][0] * c - x[j][1] * s, bf16);
        store1(d, base + eb, x[j][1] * c + x[j][0] * s, bf16);
      }
      if (from + lane < D) store1(d, base + from + lane, x[j][2], bf16);
      if (from + lane + 64 < D) store1(d, base + from + lane + 64, x[j][3], bf16);
    }
  }
}

}  // namespace

hipError_t launch_rope(RopeArgs a, hipStream_t s) {
  const bool vec = a.rot % 16 == 0;
  const int step = vec ? 64 / (a.head_dim / 16) : 4;  // heads of a pass
  const int passes = (a.heads + step - 1) / step;
  // a token's heads are shared out among waves while there are few tokens
  const int want = (int)((4096 + (int64_t)a.tokens - 1) / a.tokens);
  int split = want < passes ? want : passes;
  a.per = (passes + split - 1) / split * step;
  a.split = (a.heads + a.per - 1) / a.per;
  const unsigned grid = (unsigned)(((int64_t)a.tokens * a.split + 3) / 4);
  void (*fn)(RopeArgs) = rope_any_kernel;
  if (vec) {
    if (a.head_dim == 64) fn = a.in_bf16 ? rope_vec_kernel<64, 1> : rope_vec_kernel<64, 0>;
    else if (a.head_dim == 96) fn = a.in_bf16 ? rope_vec_kernel<96, 1> : rope_vec_kernel<96, 0>;
    else fn = a.in_bf16 ? rope_vec_kernel<128, 1> : rope_vec_kernel<128, 0>;
  }
  fn<<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace loopq

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
// 8192 tokens of 32 heads of 128: bf16 28 us, fp32 53 (4.8 and 5.0 TB/s, a large
// copy reaches 4.8); 16384 tokens of 16 heads each of fp32 queries, keys and values,
// keys and values into the cache, queries out in bf16: 117 (5.2 TB/s); a single token
// 3.0, of which all but a fraction is the launch.
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

// Any even rot_dim: a lane takes eight elements of a head.  Pairs side by side lie
// within them; halves rot_dim / 2 apart lie where no 16-byte access starts, so a
// wave's heads pass through its part of LDS (nine places for eight elements, so that
// 64 lanes a run apart hit 64 banks).  8192 tokens of 32 heads, bf16, 100 of 128
// elements turned: 30 us (single elements a lane, in 2-byte accesses: 108).
template <int D, int BF>
__global__ __launch_bounds__(256) void rope_any_kernel(RopeArgs a) {
  constexpr int S = D / 8, HP = 64 / S;
  __shared__ float row[4][64 * 9];
  const int lane = threadIdx.x & 63;
  const int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t t = w / a.split;
  if (t >= a.tokens) return;
  const int slot = lane % S, hl = lane / S, e0 = 8 * slot;
  const int h0 = (int)(w - t * a.split) * a.per;
  const int h1 = min(h0 + a.per, a.heads);
  Eight<BF> x;
  auto load = [&](int head) {
    if (hl < HP && head < h1) {
      int at;
      const RopePart& p = a.part[part_of(a, head, &at)];
      x.load(p.in, t * p.ld_in + (int64_t)at * D + e0);
    }
  };
  load(h0 + hl);
  const Place pl = find_place(a, t, lane);
  if (pl.skip) return;
  float cl = 0.0f, sl = 0.0f;
  if (lane < a.rot / 2) turn_of(a, pl.pos, lane, &cl, &sl);
  // element j becomes c x + s (the other of its pair), s with its sign
  float c[8], s[8];
  int other[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int e = e0 + j, half = a.rot / 2;
    const bool second = a.pairs ? j & 1 : e >= half;
    const int i = a.pairs ? e >> 1 : second ? e - half : e;
    const float sj = __shfl(sl, i & 63);
    c[j] = __shfl(cl, i & 63);
    s[j] = second ? sj : -sj;
    const int o = e >= a.rot ? e : second ? e - half : e + half;
    other[j] = hl * S * 9 + o + (o >> 3);
  }
  float* mine = row[threadIdx.x >> 6];
  for (int head = h0 + hl; head - hl < h1; head += HP) {
    float u[8], v[8];
    x.floats(u);
    load(head + HP);
    if (a.pairs) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = u[j ^ 1];
    } else {  // the other lanes' elements: LDS operations of a wave complete in order
      if (hl < HP) {
#pragma unroll
        for (int j = 0; j < 8; ++j) mine[9 * lane + j] = u[j];
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      if (hl < HP) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = mine[other[j]];
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    if (hl >= HP || head >= h1) continue;
    int at;
    const int which = part_of(a, head, &at);
    if (which != 2) {
#pragma unroll
      for (int j = 0; j < 8; ++j) u[j] = e0 + j < a.rot ? u[j] * c[j] + v[j] * s[j] : u[j];
    }
    if (which == 0) store8(a.part[0].out, t * a.part[0].ld_out + (int64_t)at * D + e0, u, a.part[0].out_bf16);
    else if (pl.paged) store8(pl.dst + ((int64_t)at << a.page_shift) * D + (which == 2 ? a.plane : 0), e0, u, true);
  }
}

}  // namespace

hipError_t launch_rope(RopeArgs a, hipStream_t s) {
  // where the halves of pairs start at 16 bytes too, LDS is not needed: 8192 tokens of 27
  // heads of 96 in bf16 take 16.4 us (through LDS 20.3), of 32 of 128 in fp32 53 (60)
  const bool vec = a.rot % 16 == 0;
  const int step = 64 / (a.head_dim / (vec ? 16 : 8));  // heads of a pass
  const int passes = (a.heads + step - 1) / step;
  // a token's heads are shared out among waves while there are few tokens: 4096 waves are
  // four a SIMD, which is what finds room (five in bf16) by rope_vec_kernel's registers
  const int want = (int)((4096 + (int64_t)a.tokens - 1) / a.tokens);
  int split = want < passes ? want : passes;
  a.per = (passes + split - 1) / split * step;
  a.split = (a.heads + a.per - 1) / a.per;
  const unsigned grid = (unsigned)(((int64_t)a.tokens * a.split + 3) / 4);
  void (*fn)(RopeArgs);
  if (vec) {
    if (a.head_dim == 64) fn = a.in_bf16 ? rope_vec_kernel<64, 1> : rope_vec_kernel<64, 0>;
    else if (a.head_dim == 96) fn = a.in_bf16 ? rope_vec_kernel<96, 1> : rope_vec_kernel<96, 0>;
    else fn = a.in_bf16 ? rope_vec_kernel<128, 1> : rope_vec_kernel<128, 0>;
  } else {
    if (a.head_dim == 64) fn = a.in_bf16 ? rope_any_kernel<64, 1> : rope_any_kernel<64, 0>;
    else if (a.head_dim == 96) fn = a.in_bf16 ? rope_any_kernel<96, 1> : rope_any_kernel<96, 0>;
    else fn = a.in_bf16 ? rope_any_kernel<128, 1> : rope_any_kernel<128, 0>;
  }
  fn<<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace loopq

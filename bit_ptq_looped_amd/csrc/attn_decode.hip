// Attention of one new token per row over the paged cache (attention.hip has
// the method).
//
// Bound by the bytes of K and V, each read once: a tile of 32 keys is 16 KB at
// D = 128, and a wave keeps the next one in flight in registers while it works on
// one, 2048 waves of them (32 MB) over the chip.  48 rows of up to 8192 tokens, 20
// heads of 128, bf16: 2.08 GB in 367 us, 5.7 TB/s; 3 rows of 131071 tokens, 4 key
// heads for 32 query heads, fp32 queries: 0.81 GB in 165 us, 4.9 TB/s (212 us while the
// three planes of the queries spilled registers in the loop: a reload waits for the
// loads before it).  A kernel that only reads reaches 6.5 TB/s.  Short rows are bound by
// trips: a wave asks for its second tile when the first has come.
#include "attn_core.h"

namespace loopq {
namespace {

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

// Tiles first .. last - 1 (at least one) of a query tile's keys, by one wave: O^T
// in registers (lane: head lane % 16, columns 16 d + 4 (lane / 16) + r), the
// reference m and l = the sum of the weights.  `tile` and `rows` are the wave's own
// LDS.  K goes from memory to the product's operand, V through LDS to be
// transposed; the next tile's loads are issued before this one's weights are
// formed.
template <int D, bool F32>
__device__ __forceinline__ void decode_tiles(const AttnArgs& a, const AttnPlan& pl, int row, int kvh, int hq, bool has, int pos,
                                             const Tiles& tl, int first, int last, u32x4* tile, const char** rows, f32x4 (&o)[D / 16],
                                             float& m, float& l) {
  constexpr int NQ = F32 ? 3 : 1, NP = F32 ? 3 : 2;
  constexpr int C = D / 8;                  // chunks of a row
  constexpr int NV = kDecodeKeys * C / 64;  // chunks of a tile per lane
  const int lane = threadIdx.x & 63, n16 = lane & 15, g = lane >> 4;
  const int32_t* table = a.table + (int64_t)row * a.width;
  m = -INFINITY;
  l = 0.0f;
  bf16x8 q[D / 32][NQ];
#pragma unroll
  for (int c = 0; c < D / 32; ++c)
    load_query<NQ>(a, pl.qmul, row * a.ldq + (int64_t)hq * D + 32 * c + 8 * g, has, q[c]);

#pragma unroll
  for (int d = 0; d < D / 16; ++d) o[d] = f32x4{0, 0, 0, 0};

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
  // Where the keys' rows start goes through LDS: a load needs one address from
  // there and an offset.  A hidden key reads the pool's first row instead.
  const char* const pool = reinterpret_cast<const char*>(a.pool);
  u32x4 kr[2][D / 32], vr[NV];
  const auto load_tile = [&](int i, int page) {
    const int in_page = ((tl.at(i) << 5) + lane) & ((1 << a.page_shift) - 1);
    if (lane < kDecodeKeys)
      rows[lane] = page < 0 ? pool : pool + 2 * (page * a.page_stride + (((int64_t)kvh << a.page_shift) + in_page) * D);
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const char* p = rows[16 * t + n16] + 16 * g;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) kr[t][c] = *reinterpret_cast<const u32x4*>(p + 64 * c);
    }
#pragma unroll
    for (int x = 0; x < NV; ++x) {
      const int at = lane + 64 * x, key = at / C, ch = at - key * C;
      vr[x] = *reinterpret_cast<const u32x4*>(rows[key] + 2 * a.plane + 16 * ch);
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
    const uint32_t now = seen;
    if (now != 0xffffffffu) {  // a hidden key's values count for nothing, whatever was read
#pragma unroll
      for (int x = 0; x < NV; ++x)
        if (!((now >> ((lane + 64 * x) / C)) & 1)) vr[x] = u32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int x = 0; x < NV; ++x) {
      const int at = lane + 64 * x, key = at / C, ch = at - key * C;
      tile[chunk_at<5, true>(key, ch)] = vr[x];
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    mfma_settle_before_join();
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
  mfma_settle_before_join();
  l += __shfl_xor(l, 16, 64);
  l += __shfl_xor(l, 32, 64);
}

// one head's result from a lane's columns
template <int D>
__device__ __forceinline__ void store_columns(const AttnArgs& a, int64_t at, const f32x4 (&o)[D / 16], float l) {
  const float f = l > 0.0f || l != l ? 1.0f / l : 0.0f;
#pragma unroll
  for (int d = 0; d < D / 16; ++d) {
    const f32x4 r = o[d] * f;
    if (a.bf16)
      *reinterpret_cast<u32x2*>(reinterpret_cast<uint16_t*>(a.out) + at + 16 * d) = u32x2{bf16x2_rne(r[0], r[1]), bf16x2_rne(r[2], r[3])};
    else
      *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(a.out) + at + 16 * d) = r;
  }
}

// A piece of the line of tiles per wave: 2048 pieces are two work-groups for each
// CU, as many as the registers hold.
template <int D, bool F32>
__global__ __launch_bounds__(256, 2) void decode_attn_kernel(AttnArgs a, AttnPlan pl) {
  __shared__ u32x4 s_v[4][kDecodeKeys * D / 8];
  __shared__ const char* s_rows[4][kDecodeKeys];
  extern __shared__ int64_t s_prefix[];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n16 = lane & 15, g = lane >> 4;
  const int gts = (a.group + kDecodeRows - 1) / kDecodeRows, items = a.heads * gts;
  decode_prefix(a, items, s_prefix);
  const int64_t total = s_prefix[a.rows], piece = decode_piece(total);
  const int idx = (int)blockIdx.x * 4 + wave;
  int64_t u = idx * piece;
  const int64_t u_end = min(u + piece, total);
  u32x4* tile = s_v[wave];
  if (lane == 0) pl.records[idx].parts = 0;

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
    f32x4 o[D / 16];
    float m, l;
    decode_tiles<D, F32>(a, pl, row, kvh, hq, has, pos, tl, first, last, tile, s_rows[wave], o, m, l);
    if (first == 0 && last == tl.n) {
      if (has) store_columns<D>(a, row * a.ldo + (int64_t)hq * D + 4 * g, o, l);
    } else if (has) {
      const int second = first == 0 && u != idx * piece;
      const int64_t slot = (int64_t)idx * 2 + second;
      float* dst = pl.part + (slot * kDecodeRows + n16) * D + 4 * g;
#pragma unroll
      for (int d = 0; d < D / 16; ++d) *reinterpret_cast<f32x4*>(dst + 16 * d) = o[d];
      if (g == 0) {
        pl.ml[slot * 2 * kDecodeRows + n16] = m;
        pl.ml[(slot * 2 + 1) * kDecodeRows + n16] = l;
      }
      if (lane == 0 && first == 0)  // the item goes on in the pieces after this one
        pl.records[idx] = JoinRecord{(int)((i0 + tl.n - 1) / piece) - idx + 1, row, item, second};
    }
    u = i0 + last;
  }
  // rows without a visible key belong to no piece
  for (int r = blockIdx.x; r < a.rows; r += gridDim.x)
    if (s_prefix[r + 1] == s_prefix[r])
      for (int d = tid; d < a.heads * a.group * D; d += 256) {
        if (a.bf16) reinterpret_cast<uint16_t*>(a.out)[r * a.ldo + d] = 0;
        else reinterpret_cast<float*>(a.out)[r * a.ldo + d] = 0.0f;
      }
}

// Short rows: a work-group per item, an eighth of its tiles a wave, joined in
// LDS, so that there is no second launch and no trip through memory.
constexpr int kShortWaves = 8;
template <int D, bool F32>
__global__ __launch_bounds__(64 * kShortWaves, 2) void decode_short_kernel(AttnArgs a, AttnPlan pl) {
  __shared__ u32x4 s_v[kShortWaves][kDecodeKeys * D / 8];  // a wave's V tile, then its O: [16][D] floats, as many bytes
  __shared__ const char* s_rows[kShortWaves][kDecodeKeys];
  __shared__ float s_m[kShortWaves][kDecodeRows], s_l[kShortWaves][kDecodeRows];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), n16 = lane & 15, g = lane >> 4;
  const int gts = (a.group + kDecodeRows - 1) / kDecodeRows, items = a.heads * gts;
  const int row = blockIdx.x / items, item = blockIdx.x - row * items;
  const int kvh = item / gts, gt = item - kvh * gts, head = gt * kDecodeRows + n16, hq = kvh * a.group + head;
  const bool has = head < a.group;
  const int pos = row_len(a, row) - 1;
  const Tiles tl = visible_tiles(a, pos, pos, 5);
  const int per = (tl.n + kShortWaves - 1) / kShortWaves, first = wave * per, last = min(first + per, tl.n);
  float m = -INFINITY, l = 0.0f;
  if (first < last) {
    f32x4 o[D / 16];
    decode_tiles<D, F32>(a, pl, row, kvh, hq, has, pos, tl, first, last, s_v[wave], s_rows[wave], o, m, l);
    float* so = reinterpret_cast<float*>(s_v[wave]) + n16 * D + 4 * g;
#pragma unroll
    for (int d = 0; d < D / 16; ++d) *reinterpret_cast<f32x4*>(so + 16 * d) = o[d];
  }
  if (g == 0) {
    s_m[wave][n16] = m;
    s_l[wave][n16] = l;
  }
  __syncthreads();
  const int heads = min(kDecodeRows, a.group - gt * kDecodeRows);
  for (int e = tid; e < heads * D; e += 64 * kShortWaves) {
    const int r = e / D;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kShortWaves; ++w) top = fmaxf(top, s_m[w][r]);
    const float ref = top == -INFINITY ? 0.0f : top;
    float sum = 0.0f, x = 0.0f;
#pragma unroll
    for (int w = 0; w < kShortWaves; ++w) {
      if (w * per >= tl.n) break;  // the wave had no tile
      const float f = __builtin_amdgcn_exp2f(s_m[w][r] - ref);
      sum = fmaf(f, s_l[w][r], sum);
      x = fmaf(f, reinterpret_cast<const float*>(s_v[w])[e], x);
    }
    x *= sum > 0.0f || sum != sum ? 1.0f / sum : 0.0f;
    const int64_t at = row * a.ldo + (int64_t)(kvh * a.group + gt * kDecodeRows) * D + e;
    if (a.bf16) reinterpret_cast<uint16_t*>(a.out)[at] = (uint16_t)bf16x2_rne(x, 0.0f);
    else reinterpret_cast<float*>(a.out)[at] = x;
  }
}

// Joins split items: one work-group per (item, head), its four waves a quarter
// of the parts each, added in the order of the waves.  Trips to memory: the
// records, then m and the first parts, then eight parts a wave at a time; 9 us for
// 960 items of two or three parts, 11 us for 12 items of 170 (4 us with nothing to do).
template <int D>
__global__ __launch_bounds__(256) void decode_join_kernel(AttnArgs a, AttnPlan pl) {
  __shared__ SplitItem s_list[kDecodePieces];
  __shared__ float s_o[4][2][64], s_l[4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int gts = (a.group + kDecodeRows - 1) / kDecodeRows, heads = min(kDecodeRows, a.group);
  const int n = split_items(pl.records, kDecodePieces, s_list);
  for (int x = blockIdx.x; x < n * heads; x += gridDim.x) {
    const SplitItem rec = s_list[x / heads];
    const int w0 = rec.at, r = x % heads;
    const int kvh = rec.item / gts, gt = rec.item - kvh * gts;
    if (r >= a.group - gt * kDecodeRows) continue;
    float o[2];
    const float l = join_parts<D, kDecodeRows>(pl, rec.parts, wave, 4, r,
                                               [&](int i) { return (int64_t)(w0 + i) * 2 + (i ? 0 : rec.tile); }, o);
    s_o[wave][0][lane] = o[0];
    s_o[wave][1][lane] = o[1];
    if (lane == 0) s_l[wave] = l;
    __syncthreads();
    if (wave == 0) {
#pragma unroll
      for (int h = 0; h < 2; ++h) o[h] = s_o[0][h][lane] + s_o[1][h][lane] + s_o[2][h][lane] + s_o[3][h][lane];
      store_row<D>(a, rec.row * a.ldo + (int64_t)(kvh * a.group + gt * kDecodeRows + r) * D, o, s_l[0] + s_l[1] + s_l[2] + s_l[3]);
    }
    __syncthreads();
  }
}

template <int D, bool F32>
hipError_t launch(const AttnArgs& a, const AttnPlan& pl, hipStream_t s) {
  // By what the table has room for, since lengths are not known here, and the
  // number of items: with one item a work-group, more than 640 queue up, and the
  // cut line's second launch is the smaller cost.  D = 128, bf16, every row
  // full, us (short, cut): 16 items: 128 keys 6.0, 12.6; 512 keys 10.3, 12.7; 1024
  // keys 15.2, 12.7; 4096 keys 43, 15.  128 items: 512 keys 11.4, 14.8; 2048 keys 27,
  // 32; 4096 keys 54, 52.  640 items: 128 keys 19.1, 21.1; 512 keys 37.4, 37.7.  1280
  // items: 128 keys 31, 28; 512 keys 69, 66; 2048 keys 237, 249.
  const int items = a.heads * ((a.group + kDecodeRows - 1) / kDecodeRows);
  const int64_t room = (int64_t)a.width << a.page_shift, n = (int64_t)a.rows * items;
  const bool launchable = n * (64 * kShortWaves) < ((int64_t)1 << 32);  // work-items of one launch
  if (launchable && (room <= 512 ? n <= 640 : room <= 2048 && n >= 128)) {
    decode_short_kernel<D, F32><<<(unsigned)n, 64 * kShortWaves, 0, s>>>(a, pl);
    return hipGetLastError();
  }
  const int lds = (a.rows + 1) * 8;
  const hipError_t e = prepare_launch(reinterpret_cast<const void*>(decode_attn_kernel<D, F32>), lds, 256);
  if (e != hipSuccess) return e;
  decode_attn_kernel<D, F32><<<kDecodeGroups, 256, lds, s>>>(a, pl);
  decode_join_kernel<D><<<kDecodeGroups, 256, 0, s>>>(a, pl);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_decode(const AttnArgs& a, const AttnPlan& pl, hipStream_t s) {
  switch (a.head_dim) {
    case 64: return a.bf16 ? launch<64, false>(a, pl, s) : launch<64, true>(a, pl, s);
    case 96: return a.bf16 ? launch<96, false>(a, pl, s) : launch<96, true>(a, pl, s);
    default: return a.bf16 ? launch<128, false>(a, pl, s) : launch<128, true>(a, pl, s);
  }
}

}  // namespace loopq

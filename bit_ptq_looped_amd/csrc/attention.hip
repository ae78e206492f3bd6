// Attention over the paged key-value cache (include/loopq_kv.h).
//
// One wave per query and head, one pass over the keys it can see, 64 at a time:
// lane j forms s_j = scale q . k_j, the wave keeps the running maximum m, the
// sum l of exp(s_j - m) and the sums of exp(s_j - m) v_j (two columns of v a
// lane), rescaled by exp(m_old - m_new) when m grows.  All in fp32.
#include "kv_internal.h"
#include "quant_core.h"

namespace loopq {
namespace {

template <int D>
__global__ __launch_bounds__(64) void attn_simple_kernel(AttnArgs a) {
  __shared__ float sq[D];
  const int lane = threadIdx.x;
  const int head = blockIdx.x % (a.heads * a.group), t = blockIdx.x / (a.heads * a.group);
  int row = t, pos = 0;
  const int64_t cap = (int64_t)a.width << a.page_shift;
  if (a.cu) {
    if (a.cu[a.rows] <= t || a.cu[0] > t) return;
    int lo = 0, hi = a.rows;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.cu[mid] <= t) lo = mid;
      else hi = mid;
    }
    row = lo;
    pos = (int)min((int64_t)max(a.lens[row], 0), cap) - a.cu[row + 1] + t;
  } else {
    pos = (int)min((int64_t)max(a.lens[row], 0), cap) - 1;
  }
  for (int d = lane; d < D; d += 64) {
    const int64_t i = t * a.ldq + (int64_t)head * D + d;
    sq[d] = a.bf16 ? bf16_bits_to_float(reinterpret_cast<const uint16_t*>(a.q)[i]) : reinterpret_cast<const float*>(a.q)[i];
  }
  __syncthreads();
  const int kvh = head / a.group;
  float m = -INFINITY, l = 0.0f, o[2] = {0.0f, 0.0f};
  const int64_t low = a.window > 0 ? (int64_t)pos - a.window + 1 : 0;
  for (int64_t j0 = 0; j0 <= pos; j0 += 64) {
    if (j0 + 63 < low && j0 >= a.sinks) continue;
    const int64_t j = j0 + lane;
    bool seen = j <= pos && (j >= low || j < a.sinks);
    int64_t at = 0;
    if (seen) {
      const int page = a.table[(int64_t)row * a.width + (j >> a.page_shift)];
      seen = page >= 0 && page < a.num_pages;
      at = page * a.page_stride + (((int64_t)kvh << a.page_shift) + (j & ((1 << a.page_shift) - 1))) * D;
    }
    float s = -INFINITY;
    if (seen) {
      float acc = 0.0f;
      for (int d = 0; d < D; d += 8) {
        const uint4 u = *reinterpret_cast<const uint4*>(a.pool + at + d);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc = fmaf(bf16_bits_to_float(w[i] & 0xffffu), sq[d + 2 * i], acc);
          acc = fmaf(bf16_bits_to_float(w[i] >> 16), sq[d + 2 * i + 1], acc);
        }
      }
      s = acc * a.scale;
    }
    float top = s;
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, 64));
    const float mn = fmaxf(m, top);
    if (!__any(seen)) continue;
    const float p = seen ? expf(s - mn) : 0.0f;
    const float c = m == -INFINITY ? 0.0f : expf(m - mn);
    float sum = p;
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) sum += __shfl_xor(sum, off, 64);
    l = l * c + sum;
    m = mn;
    o[0] *= c;
    o[1] *= c;
    for (int i = 0; i < 64; ++i) {
      if (!__shfl((int)seen, i, 64)) continue;
      const float pi = __shfl(p, i, 64);
      const int64_t ai = __shfl(at, i, 64) + a.plane;
      o[0] = fmaf(pi, bf16_bits_to_float(a.pool[ai + lane]), o[0]);
      if (D > 64 && lane + 64 < D) o[1] = fmaf(pi, bf16_bits_to_float(a.pool[ai + 64 + lane]), o[1]);
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int d = lane + 64 * h;
    if (d >= D) break;
    const float r = l > 0.0f ? o[h] / l : 0.0f;
    const int64_t i = t * a.ldo + (int64_t)head * D + d;
    if (a.bf16) reinterpret_cast<uint16_t*>(a.out)[i] = (uint16_t)bf16x2_rne(r, r);
    else reinterpret_cast<float*>(a.out)[i] = r;
  }
}

}  // namespace

size_t attn_workspace_bytes(int64_t, int, int64_t, int) { return 256; }

hipError_t launch_attn(const AttnArgs& a, hipStream_t s) {
  const int grid = a.queries * a.heads * a.group;
  if (a.head_dim == 64) attn_simple_kernel<64><<<grid, 64, 0, s>>>(a);
  else if (a.head_dim == 96) attn_simple_kernel<96><<<grid, 64, 0, s>>>(a);
  else attn_simple_kernel<128><<<grid, 64, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace loopq

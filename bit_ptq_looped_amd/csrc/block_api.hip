// C ABI of the block's parts between its linears and the attention (declared in
// include/loopq_block.h): host-side checks and dispatch on the caller's stream.
#include <math.h>

#include "arg_checks.h"
#include "block_internal.h"

using namespace loopq;

namespace {

bool is_dtype(int d) { return d == LOOPQ_F32 || d == LOOPQ_BF16; }

// A matrix of a call: rows of `bytes` bytes, `ld` bytes apart.
struct Rows {
  const void* p;
  int64_t ld, bytes;
};

bool share(const Rows& a, const Rows& b, int64_t rows) {
  return a.p && b.p && rows_overlap(a.p, a.ld, a.bytes, b.p, b.ld, b.bytes, rows);
}
bool same(const Rows& a, const Rows& b) { return a.p == b.p && a.ld == b.ld && a.bytes == b.bytes; }

int32_t check_dims(int heads, int head_dim) {
  if (heads <= 0 || head_dim <= 0) return LOOPQ_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 96 && head_dim != 128) return LOOPQ_ERR_UNSUPPORTED;
  return (int64_t)heads * head_dim > (1 << 20) ? LOOPQ_ERR_UNSUPPORTED : LOOPQ_OK;
}

int32_t check_rope(const loopq_rope_spec* r, int head_dim) {
  if (!r || !r->inv_freq || !isfinite(r->magnitude)) return LOOPQ_ERR_INVALID_ARG;
  if (r->layout != LOOPQ_ROPE_HALF && r->layout != LOOPQ_ROPE_PAIRS) return LOOPQ_ERR_INVALID_ARG;
  if (r->rot_dim < 2 || r->rot_dim % 2 || r->rot_dim > head_dim) return LOOPQ_ERR_UNSUPPORTED;
  return aligned(r->inv_freq, 8) ? LOOPQ_OK : LOOPQ_ERR_ALIGNMENT;
}

// tokens of a rotary call: a launch has fewer than 2^32 work-items, 64 a token (and a
// token is shared by several waves only where there are fewer than 4096)
constexpr int32_t kRopeMaxTokens = (1 << 26) - 4;

RopeArgs rope_args(const loopq_rope_spec* r, int32_t dtype, int32_t tokens, int32_t head_dim) {
  RopeArgs a = {};
  a.in_bf16 = dtype == LOOPQ_BF16;
  a.tokens = tokens;
  a.head_dim = head_dim;
  a.rot = r->rot_dim;
  a.pairs = r->layout == LOOPQ_ROPE_PAIRS;
  a.inv_freq = r->inv_freq;
  a.magnitude = r->magnitude;
  return a;
}

RopePart part(const void* in, int64_t ld_in, void* out, int64_t ld_out, int heads, int head_dim, int out_bf16, int tokens) {
  const int64_t width = (int64_t)heads * head_dim;
  return RopePart{in, out, tokens > 1 ? ld_in : width, tokens > 1 ? ld_out : width, heads, out_bf16};
}

}  // namespace

extern "C" {

int32_t loopq_rms_norm(const void* x, int64_t ldx, int32_t x_dtype, const void* residual, int64_t ldr, int32_t res_dtype,
                       int32_t rows, int32_t K, const float* weight, float eps, void* sum_out, int64_t lds, void* y,
                       int64_t ldy, int32_t y_dtype, int8_t* codes, float* steps, float clip, int32_t bits_a,
                       int32_t per_token, void* stream) {
  if (rows < 0 || K <= 0) return LOOPQ_ERR_INVALID_ARG;
  if (!(eps > 0.0f) || !isfinite(eps)) return LOOPQ_ERR_INVALID_ARG;
  if (K % 8 || K > kNormMaxK || (codes && K % 32)) return LOOPQ_ERR_UNSUPPORTED;
  if (!is_dtype(x_dtype) || (residual && !is_dtype(res_dtype)) || (y && !is_dtype(y_dtype))) return LOOPQ_ERR_UNSUPPORTED;
  if (codes && bits_a != 4 && bits_a != 8) return LOOPQ_ERR_UNSUPPORTED;
  if (codes && (!(clip > 0.0f) || !isfinite(clip))) return LOOPQ_ERR_INVALID_ARG;
  if (rows == 0) return LOOPQ_OK;
  if ((!y && !codes) || (sum_out && !residual) || (codes && !steps)) return LOOPQ_ERR_INVALID_ARG;
  int32_t st = check_rows(x, ldx, K, rows, x_dtype);
  if (st == LOOPQ_OK && residual) st = check_rows(residual, ldr, K, rows, res_dtype);
  if (st == LOOPQ_OK && sum_out) st = check_rows(sum_out, lds, K, rows, res_dtype);
  if (st == LOOPQ_OK && y) st = check_rows(y, ldy, K, rows, y_dtype);
  if (st != LOOPQ_OK) return st;
  if (!aligned(weight, 16) || (codes && (!aligned(codes, 16) || !aligned(steps, 4)))) return LOOPQ_ERR_ALIGNMENT;
  // a single row's distance is nobody's
  if (rows == 1) ldx = ldr = lds = ldy = K;
  const int xb = item_bytes(x_dtype), rb = item_bytes(res_dtype), yb = item_bytes(y_dtype);
  const Rows in[2] = {{x, ldx * xb, (int64_t)K * xb}, {residual, ldr * rb, (int64_t)K * rb}};
  const Rows sum = {sum_out, lds * rb, (int64_t)K * rb}, out = {y, ldy * yb, (int64_t)K * yb};
  const size_t n = (size_t)rows * K;
  for (const Rows* o : {&sum, &out}) {
    for (int i = 0; i < 2; ++i)
      if (share(in[i], *o, rows) && !same(in[i], *o)) return LOOPQ_ERR_INVALID_ARG;
    if (o->p && weight && overlap(weight, (size_t)K * 4, o->p, (rows - 1) * o->ld + o->bytes)) return LOOPQ_ERR_INVALID_ARG;
  }
  if (share(sum, out, rows)) return LOOPQ_ERR_INVALID_ARG;
  if (codes) {
    const Rows all[4] = {in[0], in[1], sum, out};
    for (const Rows& m : all)
      if (m.p && (overlap(m.p, (rows - 1) * m.ld + m.bytes, codes, n) || overlap(m.p, (rows - 1) * m.ld + m.bytes, steps, n / 8)))
        return LOOPQ_ERR_INVALID_ARG;
    if (overlap(codes, n, steps, n / 8)) return LOOPQ_ERR_INVALID_ARG;
    if (weight && (overlap(weight, (size_t)K * 4, codes, n) || overlap(weight, (size_t)K * 4, steps, n / 8)))
      return LOOPQ_ERR_INVALID_ARG;
  }
  NormArgs a;
  a.x = x;
  a.res = residual;
  a.w = weight;
  a.sum = sum_out;
  a.y = y;
  a.codes = codes;
  a.steps = steps;
  a.ldx = ldx;
  a.ldr = ldr;
  a.lds = lds;
  a.ldy = ldy;
  a.rows = rows;
  a.K = K;
  a.x_bf16 = x_dtype == LOOPQ_BF16;
  a.res_bf16 = residual && res_dtype == LOOPQ_BF16;
  a.y_bf16 = y && y_dtype == LOOPQ_BF16;
  a.per_token = per_token != 0;
  a.eps = eps;
  a.inv_k = 1.0 / K;
  a.clip = codes ? clip : 1.0f;
  a.qmax = codes && bits_a == 4 ? 7.0f : 127.0f;
  hipStream_t s = as_stream(stream);
  TimingScope ts(LOOPQ_KERNEL_NORM, s);
  return hip_status(launch_rms_norm(a, s));
}

int32_t loopq_rope_frequencies(int32_t scaling, int32_t rot_dim, double base, double factor, double length, double low,
                               double high, double* inv_freq) {
  if (!inv_freq || !(base > 1.0)) return LOOPQ_ERR_INVALID_ARG;
  if (scaling < LOOPQ_ROPE_PLAIN || scaling > LOOPQ_ROPE_PARTS) return LOOPQ_ERR_INVALID_ARG;
  if (rot_dim < 2 || rot_dim > 128 || rot_dim % 2 || (scaling == LOOPQ_ROPE_BASE && rot_dim < 4)) return LOOPQ_ERR_UNSUPPORTED;
  if (scaling != LOOPQ_ROPE_PLAIN && (!(factor >= 1.0) || !isfinite(factor))) return LOOPQ_ERR_INVALID_ARG;
  if (scaling == LOOPQ_ROPE_PARTS &&
      (!(length > 0.0) || !isfinite(length) || !(low >= 0.0) || !(high > low) || !isfinite(high)))
    return LOOPQ_ERR_INVALID_ARG;
  if (scaling == LOOPQ_ROPE_BASE) base *= pow(factor, (double)rot_dim / (rot_dim - 2));
  if (!isfinite(base)) return LOOPQ_ERR_INVALID_ARG;
  for (int i = 0; i < rot_dim / 2; ++i) {
    double f = pow(base, -2.0 * i / rot_dim);
    if (scaling == LOOPQ_ROPE_LINEAR) f /= factor;
    if (scaling == LOOPQ_ROPE_PARTS) {
      double g = (length * f / 6.283185307179586477 - low) / (high - low);
      g = g < 0.0 ? 0.0 : g > 1.0 ? 1.0 : g;
      f = g * f + (1.0 - g) * f / factor;
    }
    inv_freq[i] = f;
  }
  return LOOPQ_OK;
}

int32_t loopq_rope(const void* x, int64_t ldx, int32_t dtype, int32_t tokens, int32_t heads, int32_t head_dim,
                   const int32_t* positions, const loopq_rope_spec* rope, void* out, int64_t ldo, void* stream) {
  int32_t st = check_dims(heads, head_dim);
  if (st == LOOPQ_OK) st = check_rope(rope, head_dim);
  if (st != LOOPQ_OK) return st;
  if (!is_dtype(dtype)) return LOOPQ_ERR_UNSUPPORTED;
  if (tokens < 0) return LOOPQ_ERR_INVALID_ARG;
  if (tokens > kRopeMaxTokens) return LOOPQ_ERR_UNSUPPORTED;
  if (tokens == 0) return LOOPQ_OK;
  if (!positions) return LOOPQ_ERR_INVALID_ARG;
  const int64_t width = (int64_t)heads * head_dim;
  st = check_rows(x, ldx, width, tokens, dtype);
  if (st == LOOPQ_OK) st = check_rows(out, ldo, width, tokens, dtype);
  if (st != LOOPQ_OK) return st;
  if (!aligned(positions, 4)) return LOOPQ_ERR_ALIGNMENT;
  RopeArgs a = rope_args(rope, dtype, tokens, head_dim);
  a.part[0] = part(x, ldx, out, ldo, heads, head_dim, a.in_bf16, tokens);
  const int item = item_bytes(dtype);
  const Rows in = {x, a.part[0].ld_in * item, width * item}, to = {out, a.part[0].ld_out * item, width * item};
  if (share(in, to, tokens) && !same(in, to)) return LOOPQ_ERR_INVALID_ARG;
  a.positions = positions;
  a.heads = heads;
  hipStream_t s = as_stream(stream);
  TimingScope ts(LOOPQ_KERNEL_ROPE, s);
  return hip_status(launch_rope(a, s));
}

int32_t loopq_kv_write_rope(const loopq_kv_pool* pool, int32_t slab, const loopq_kv_table* table, const int32_t* cu,
                            const loopq_rope_spec* rope, const void* k, int64_t ldk, const void* v, int64_t ldv,
                            int32_t dtype, int32_t tokens, const void* q, int64_t ldq, int32_t heads_q, void* q_out,
                            int64_t ldqo, int32_t q_dtype, void* stream) {
  int32_t st = check_pool(pool);
  if (st == LOOPQ_OK) st = check_table(table);
  if (st == LOOPQ_OK) st = check_rope(rope, pool->head_dim);
  if (st != LOOPQ_OK) return st;
  if (!q != !q_out) return LOOPQ_ERR_INVALID_ARG;
  if (!is_dtype(dtype) || (q && !is_dtype(q_dtype))) return LOOPQ_ERR_UNSUPPORTED;
  if (q && (st = check_dims(heads_q, pool->head_dim)) != LOOPQ_OK) return st;
  if (slab < 0 || slab >= pool->slabs || tokens < 0 || table->num_pages != pool->num_pages) return LOOPQ_ERR_INVALID_ARG;
  if (tokens > kRopeMaxTokens) return LOOPQ_ERR_UNSUPPORTED;
  if (tokens == 0 || table->rows == 0) return LOOPQ_OK;
  if (!cu) return LOOPQ_ERR_INVALID_ARG;
  if (!aligned(cu, 4)) return LOOPQ_ERR_ALIGNMENT;
  const int d = pool->head_dim;
  const int64_t width = (int64_t)pool->heads * d;
  st = check_rows(k, ldk, width, tokens, dtype);
  if (st == LOOPQ_OK) st = check_rows(v, ldv, width, tokens, dtype);
  if (st == LOOPQ_OK && q) st = check_rows(q, ldq, (int64_t)heads_q * d, tokens, dtype);
  if (st == LOOPQ_OK && q) st = check_rows(q_out, ldqo, (int64_t)heads_q * d, tokens, q_dtype);
  if (st != LOOPQ_OK) return st;
  RopeArgs a = rope_args(rope, dtype, tokens, d);
  a.part[0] = part(q, ldq, q_out, ldqo, q ? heads_q : 0, d, q && q_dtype == LOOPQ_BF16, tokens);
  a.part[1] = part(k, ldk, nullptr, 0, pool->heads, d, 1, tokens);
  a.part[2] = part(v, ldv, nullptr, 0, pool->heads, d, 1, tokens);
  if (q) {
    const int item = item_bytes(dtype), qi = item_bytes(q_dtype);
    const Rows to = {q_out, a.part[0].ld_out * qi, (int64_t)heads_q * d * qi};
    for (int i = 0; i < 3; ++i) {
      const Rows in = {a.part[i].in, a.part[i].ld_in * item, (int64_t)a.part[i].heads * d * item};
      if (share(in, to, tokens) && !(i == 0 && same(in, to))) return LOOPQ_ERR_INVALID_ARG;
    }
  }
  a.cu = cu;
  a.t = table_of(table);
  a.plane = (int64_t)pool->heads * pool->page_size * d;
  a.page_stride = pool->slabs * 2 * a.plane;
  a.pool = reinterpret_cast<uint16_t*>(pool->data) + slab * 2 * a.plane;
  a.page_shift = 31 - __builtin_clz((unsigned)pool->page_size);
  a.heads = a.part[0].heads + 2 * pool->heads;
  hipStream_t s = as_stream(stream);
  TimingScope ts(LOOPQ_KERNEL_ROPE, s);
  return hip_status(launch_rope(a, s));
}

int32_t loopq_adapter_workspace_bytes(int32_t rows, int32_t max_rank, size_t* bytes) {
  if (!bytes || rows < 0 || max_rank <= 0) return LOOPQ_ERR_INVALID_ARG;
  if (max_rank % 8 || max_rank > kAdapterMaxRank) return LOOPQ_ERR_UNSUPPORTED;
  *bytes = adapter_workspace_bytes(rows, max_rank);
  return LOOPQ_OK;
}

int32_t loopq_adapter_apply(const void* x, int64_t ldx, int32_t dtype, int32_t rows, int32_t K, int32_t N,
                            const int32_t* ids, const void* A, const void* B, const float* scales, const int32_t* ranks,
                            int32_t adapters, int32_t max_rank, float* y, int64_t ldy, void* workspace,
                            size_t workspace_bytes, void* stream) {
  if (rows < 0 || K <= 0 || N <= 0 || adapters <= 0 || max_rank <= 0) return LOOPQ_ERR_INVALID_ARG;
  if (!is_dtype(dtype)) return LOOPQ_ERR_UNSUPPORTED;
  if (K % 8 || K > 65536 || N > (1 << 20) || adapters > (1 << 16)) return LOOPQ_ERR_UNSUPPORTED;
  if (max_rank % 8 || max_rank > kAdapterMaxRank || rows > kAdapterMaxRows) return LOOPQ_ERR_UNSUPPORTED;
  if (rows == 0) return LOOPQ_OK;
  if (!ids || !A || !B || !scales || !y) return LOOPQ_ERR_INVALID_ARG;
  int32_t st = check_rows(x, ldx, K, rows, dtype);
  if (st != LOOPQ_OK) return st;
  if (rows > 1 && ldy < N) return LOOPQ_ERR_INVALID_ARG;
  if (rows > 1 && (ldx >= kAdapterMaxLdx / item_bytes(dtype) || ldy >= kAdapterMaxLdy / 4)) return LOOPQ_ERR_UNSUPPORTED;
  if (!aligned(ids, 4) || !aligned(A, 16) || !aligned(B, 16) || !aligned(scales, 4) || !aligned(ranks, 4) || !aligned(y, 4))
    return LOOPQ_ERR_ALIGNMENT;
  AdapterArgs a;
  a.x = x;
  a.ldx = rows > 1 ? ldx : K;
  a.x_bf16 = dtype == LOOPQ_BF16;
  a.rows = rows;
  a.K = K;
  a.N = N;
  a.ids = ids;
  a.A = reinterpret_cast<const uint16_t*>(A);
  a.B = reinterpret_cast<const uint16_t*>(B);
  a.scales = scales;
  a.ranks = ranks;
  a.adapters = adapters;
  a.R = max_rank;
  a.y = y;
  a.ldy = rows > 1 ? ldy : N;
  const int item = item_bytes(dtype);
  if (share({x, a.ldx * item, (int64_t)K * item}, {y, a.ldy * 4, (int64_t)N * 4}, rows)) return LOOPQ_ERR_INVALID_ARG;
  st = check_workspace(workspace, workspace_bytes, adapter_workspace_bytes(rows, max_rank));
  if (st != LOOPQ_OK) return st;
  a.z = reinterpret_cast<float*>(workspace);
  hipStream_t s = as_stream(stream);
  TimingScope ts(LOOPQ_KERNEL_ADAPTER, s);
  return hip_status(launch_adapter(a, s));
}

}  // extern "C"

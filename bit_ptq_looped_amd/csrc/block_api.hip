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
  a.row0 = 0;
  a.rows = rows;
  a.K = K;
  a.x_bf16 = x_dtype == LOOPQ_BF16;
  a.res_bf16 = residual && res_dtype == LOOPQ_BF16;
  a.y_bf16 = y && y_dtype == LOOPQ_BF16;
  a.per_token = per_token != 0;
  a.eps = eps;
  a.clip = codes ? clip : 1.0f;
  a.qmax = codes && bits_a == 4 ? 7.0f : 127.0f;
  hipStream_t s = as_stream(stream);
  TimingScope ts(LOOPQ_KERNEL_NORM, s);
  return hip_status(launch_rms_norm(a, s));
}

}  // extern "C"

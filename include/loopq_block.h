/*
 * loopq_block.h -- what a block of a looped transformer needs between its
 * quantized linears (include/loopq.h) and the attention (include/loopq_kv.h),
 * for AMD Instinct MI355X (gfx950): the residual's addition with the
 * root-mean-square norm.
 *
 * The conventions of loopq.h hold: device pointers unless the name ends in
 * _host, work is enqueued on `stream` and the call returns, the caller owns
 * every buffer, arguments are checked on the host before any HIP call.  A call
 * of no rows is a no-op.  Buffers must not overlap unless a call says so.
 * "16-byte aligned rows" means the pointer and, where there is more than one
 * row, the distance from a row to the next; columns of the same wider rows
 * qualify.
 */
#ifndef LOOPQ_BLOCK_H
#define LOOPQ_BLOCK_H

#include "loopq_kv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Residual, RMS norm and what the next linear takes, in one pass over the rows.
 *
 *   h = x + residual, rounded to the residual's type (h = x without a residual)
 *   r = fl32(1 / sqrt(mean_k h_k^2 + eps)), the mean, root and quotient in fp64
 *   z_k = fl32(fl32(h_k r) w_k)        (fl32(h_k r) without a weight)
 *
 * x [rows][K] in x_dtype; residual, sum_out [rows][K] in res_dtype; weight fp32
 * [K]; y [rows][K] in y_dtype.  residual, weight, sum_out, y and codes may each
 * be NULL, sum_out only with a residual; y or codes is given.  sum_out receives h
 * (the norm is of h as it is kept there, given or not), y receives z, rounded
 * to y_dtype.
 * codes int8 [rows][K] and steps fp32 [rows][K/32], both contiguous, receive
 * Eq.(4) of z as loopq_quant_act (per_token 0) or loopq_quant_act_per_token
 * (per_token 1) without a transform forms them from z: bitwise the same, ready
 * for loopq_gemm_codes.  clip > 0 and finite, bits_a 4 or 8 (both ignored without
 * codes).
 * In 64 bits the order of the sum does not show in r (but where the exact value
 * lies within some 2^-50 of a border between two fp32 numbers), so y, codes and
 * steps are functions of the inputs, not of the launch.
 * A row that holds an infinity or NaN (after the rounding of h) has steps of NaN
 * and codes of 0; its y is what the formulas give.
 *
 * sum_out may be the residual or x itself, and y may be x or the residual itself
 * (the same address, type and row distance).
 * x, residual, sum_out, y: 16-byte aligned rows, at least K elements apart;
 * weight, codes: 16-byte aligned; steps: 4-byte.
 * K % 8 == 0 (K % 32 == 0 with codes), K <= 32768, eps > 0 and finite. */
int32_t loopq_rms_norm(const void* x, int64_t ldx, int32_t x_dtype, const void* residual, int64_t ldr,
                       int32_t res_dtype, int32_t rows, int32_t K, const float* weight, float eps,
                       void* sum_out, int64_t lds, void* y, int64_t ldy, int32_t y_dtype,
                       int8_t* codes, float* steps, float clip, int32_t bits_a, int32_t per_token,
                       void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LOOPQ_BLOCK_H */

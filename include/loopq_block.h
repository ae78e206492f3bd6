/*
 * loopq_block.h -- what a block of a looped transformer needs between its
 * quantized linears (include/loopq.h) and the attention (include/loopq_kv.h),
 * for AMD Instinct MI355X (gfx950): the residual's addition with the
 * root-mean-square norm, rotary positions, and low-rank adapters of many
 * requests beside a shared projection.
 *
 * The conventions of loopq.h hold: device pointers unless the name ends in
 * _host, work is enqueued on `stream` and the call returns, the caller owns
 * every buffer, arguments are checked on the host before any HIP call.  A call
 * of no rows is a no-op.  Buffers must not overlap unless a call says so.
 * "16-byte aligned rows" means the pointer and, where there is more than one
 * row, the distance from a row to the next; columns of the same wider rows
 * qualify.  Values read from device memory (ids, ranks, positions, lengths,
 * page tables) are never trusted with an address.
 */
#ifndef LOOPQ_BLOCK_H
#define LOOPQ_BLOCK_H

#include "loopq_kv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Residual, RMS norm and what the next linear takes, in one pass over the rows.
 *
 *   h = fl32(x + residual), rounded to the residual's type (h = x without a residual)
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
 * What 64 bits round stays below 2^-48 of r before it is rounded to fp32.  So the
 * order of the sum does not show in r, and y, codes and steps are functions of the
 * inputs, not of the launch, but for a row whose exact 1 / sqrt lies within 2^-48 of
 * itself of the border between two fp32 numbers (less than one row in 2^23).
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

/* Which elements of a head form the pair that frequency i turns. */
typedef enum {
  LOOPQ_ROPE_HALF = 0,  /* x[i] and x[i + rot_dim / 2] */
  LOOPQ_ROPE_PAIRS = 1  /* x[2 i] and x[2 i + 1] */
} loopq_rope_layout;

/* Rotary positions: the pair (a, b) of frequency i at position p becomes
 *   m (a cos t - b sin t), m (b cos t + a sin t),  t = p inv_freq[i],
 * for i < rot_dim / 2; elements from rot_dim on stay as they are.  inv_freq fp64
 * [rot_dim / 2] (device, 8-byte aligned; radians a position), magnitude m
 * finite, rot_dim even, 2 .. head_dim.  t is reduced in fp64; sine, cosine and
 * the turn are fp32 (sines and cosines within 3e-7 up to positions of 2^24),
 * results are rounded once.  The turn by -p undoes the turn by p (and, times m,
 * takes gradients back through it). */
typedef struct {
  const double* inv_freq;
  int32_t rot_dim, layout;
  float magnitude;
} loopq_rope_spec;

/* How loopq_rope_frequencies treats contexts `factor` times as long. */
typedef enum {
  LOOPQ_ROPE_PLAIN = 0,  /* f_i = base^(-2 i / rot_dim) */
  LOOPQ_ROPE_LINEAR = 1, /* f_i / factor */
  LOOPQ_ROPE_BASE = 2,   /* base times factor^(rot_dim / (rot_dim - 2)): the slowest turns by f / factor, the fastest as before */
  LOOPQ_ROPE_PARTS = 3   /* g f_i + (1 - g) f_i / factor, g = (length f_i / 2 pi - low) / (high - low) within [0, 1]:
                            what turns over `high` times within the original length stays, what turns less than
                            `low` times is stretched */
} loopq_rope_scaling;

/* The frequencies of a scaling as fp64 [rot_dim / 2] in host memory (host only).
 * base > 1; factor >= 1 (ignored by PLAIN); length > 0 and 0 <= low < high
 * (PARTS only); all finite, the longer base of BASE too.  rot_dim even, 2 .. 128 (from 4 on for BASE). */
int32_t loopq_rope_frequencies(int32_t scaling, int32_t rot_dim, double base, double factor, double length,
                               double low, double high, double* inv_freq_host);

/* x, out [tokens][heads][head_dim] in `dtype`, tokens ldx and ldo elements apart,
 * 16-byte aligned rows; positions int32 [tokens] (any sign).  out may be x itself
 * (the same address and distance) or, with ldx = ldo, other columns of the same
 * wider rows.  head_dim 64, 96 or 128; heads * head_dim <= 2^20. */
int32_t loopq_rope(const void* x, int64_t ldx, int32_t dtype, int32_t tokens, int32_t heads, int32_t head_dim,
                   const int32_t* positions, const loopq_rope_spec* rope_host, void* out, int64_t ldo, void* stream);

/* loopq_kv_write with rotary positions, and the new tokens' queries: k is turned
 * and then, with v as it is, rounded to bf16 and written to the slab; q is turned
 * into q_out.  Token i of the n that cu gives row b (the last of its lens[b]
 * tokens, see loopq_kv_write) is at position lens[b] - n + i.  cu, k, v, dtype,
 * tokens as for loopq_kv_write (but rows of q, k and v from cu[rows] up to tokens
 * may be read, without effect): a token whose position has no page is dropped (its
 * q is turned all the same).  q [tokens][heads_q][head_dim] in `dtype`, q_out the
 * same shape in q_dtype (bf16 queries suit loopq_attn_prefill), 16-byte aligned
 * rows ldq and ldqo elements apart; q_out may be q itself (the same address,
 * type and distance) or other columns of the same wider rows.  q and q_out may
 * both be NULL (heads_q is ignored then).  Rows of q_out from cu[rows] on are not
 * written.  heads_q * head_dim <= 2^20. */
int32_t loopq_kv_write_rope(const loopq_kv_pool* pool_host, int32_t slab, const loopq_kv_table* table_host,
                            const int32_t* cu, const loopq_rope_spec* rope_host, const void* k, int64_t ldk,
                            const void* v, int64_t ldv, int32_t dtype, int32_t tokens, const void* q, int64_t ldq,
                            int32_t heads_q, void* q_out, int64_t ldqo, int32_t q_dtype, void* stream);

/* Low-rank adapters of many requests, added to a shared projection's result:
 *   y_m += scales[a] B_a (A_a x_m),  a = ids[m],
 * for every row m whose id is an adapter's (0 <= ids[m] < adapters); other rows
 * of y are neither read nor written.  x [rows][K] in `dtype` (the input of the
 * linear that wrote y), 16-byte aligned rows ldx elements apart; y fp32
 * [rows][N], rows ldy elements apart, 4-byte aligned.  A bf16
 * [adapters][max_rank][K] and B bf16 [adapters][N][max_rank], contiguous, 16-byte
 * aligned.  ids int32 [rows] in any order (rows of one request side by side cost
 * least); scales fp32 [adapters]; ranks int32 [adapters] or NULL: adapter a uses
 * the first ranks[a] (within 0 .. max_rank) rows of A_a and columns of B_a, the rest
 * is not used, whatever it holds.  ids, scales, ranks: device, 4-byte aligned.
 * Products of x and A and of A x and B are formed from all bits of their factors
 * (of 2^-100 and more in magnitude), sums are fp32 in an order that depends on
 * the sizes only: a row's result does not depend on other rows' ids.  An infinity
 * or NaN in a row or an adapter reaches no row but its own (there an infinity may
 * end as NaN).
 * max_rank a multiple of 8 up to 128; K % 8 == 0, K <= 65536; N <= 2^20;
 * adapters <= 2^16; rows <= 2^20; ldx < 2^24 (fp32: 2^23),
 * ldy < 2^24.  Workspace: loopq_adapter_workspace_bytes(rows, max_rank), which
 * never falls as either grows: one of a program's largest batch and rank serves all
 * of its calls.  Two calls that share one must not overlap. */
int32_t loopq_adapter_workspace_bytes(int32_t rows, int32_t max_rank, size_t* bytes_host);
int32_t loopq_adapter_apply(const void* x, int64_t ldx, int32_t dtype, int32_t rows, int32_t K, int32_t N,
                            const int32_t* ids, const void* A, const void* B, const float* scales,
                            const int32_t* ranks, int32_t adapters, int32_t max_rank, float* y, int64_t ldy,
                            void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* LOOPQ_BLOCK_H */

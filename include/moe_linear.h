/*
 * moe_linear.h - dense products with int4 affine group-quantised weights
 * (the projections around the experts: mixer inputs and outputs, head gates,
 * the vocabulary).  For x of T tokens:
 *
 *   y[t][n] = sum_k x[t][k] * W[n][k],   W[n][k] = s[n, k/G] * q[n,k] + b[n, k/G]
 *
 * with q in 0..15 and fp16 s, b in groups of G inputs, as for the experts
 * (moe.h).  Products of x and q are exact and sums are fp32 in a fixed order
 * (bitwise repeatable) that depends on n_tokens: a token's results may differ in
 * their last bits between batches.  Each output is rounded once to out_dtype.
 *
 * Weights are laid out once on the device by moe_linear_pack.  A value
 * outside a type's range overflows to infinity as a conversion does.  Sums are
 * formed as 16 s (sum (1 + q/16) x) + (b - 16 s) (sum x) over up to 256 columns,
 * two parts that nearly cancel: they need 512 max|x[t]| (1 + 16 max|s| + max|b|)
 * within fp32's range (3.4e38), which every fp16 x and a bf16 x of up to 10^34
 * with |s|, |b| of up to 3 have; beyond, y[t] may be infinite or NaN where the
 * sum itself is not.  A non-finite x[t] reaches y[t] only.  The conventions of moe.h hold
 * (caller-owned device buffers, work on the given stream only, negative
 * status and moe_last_error on refusal, n_tokens == 0 a no-op).
 */
#ifndef MOE_AMD_MOE_LINEAR_H
#define MOE_AMD_MOE_LINEAR_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { MOE_F32 = 3 };

/* in_dim K:     a multiple of 64, 64..65536
 * out_dim N:    1..2^20, any
 * group_size G: 32, 64 or 128, dividing K
 * act_dtype:    MOE_F16 or MOE_BF16 (x)
 * out_dtype:    MOE_F16, MOE_BF16 or MOE_F32 (y) */
typedef struct {
  int32_t in_dim, out_dim, group_size, act_dtype, out_dtype;
} moe_linear_desc;

/* Bytes of the packed weights (0 for unsupported sizes).  N is padded to
 * N' = the next multiple of 32; two sections follow each other:
 *   values  N' * K / 2 bytes: the 32-row pair-tiles of the expert blob's down
 *           section (moe.h: block p * K/64 + c holds rows 32p..32p+31,
 *           columns 64c..64c+63);
 *   scales  4 * N' * K / G bytes: [s_A, b_A, s_B, b_B] fp16 of (pair-tile p,
 *           group g, row n of tile A / B) at ((p * K/G + g) * 16 + n) * 8.
 * Padding rows are zero. */
uint64_t moe_linear_bytes(int32_t in_dim, int32_t out_dim, int32_t group_size);

/* Device-side packer.  q: [N][K/8] 32-bit words, value 8i + j of a row in
 * bits 4j..4j+3 of its word i; scale, bias: [N][K/G] fp16 bits; packed:
 * moe_linear_bytes() bytes, 256-byte aligned.  All device buffers. */
moe_status moe_linear_pack(int32_t in_dim, int32_t out_dim, int32_t group_size, const uint32_t* q,
                           const uint16_t* scale, const uint16_t* bias, uint8_t* packed, moe_stream stream);

/* y [T][N] (out_dtype, rows back to back) of x [T][K] (16-byte aligned) and
 * the packed weights.  n_tokens up to 2^20, and ceil(n_tokens / 128) *
 * ceil(N / 128) up to 2^23 - 8. */
moe_status moe_linear_forward(const moe_linear_desc* desc, const uint8_t* packed, const void* x, int32_t n_tokens,
                              void* y, moe_stream stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_AMD_MOE_LINEAR_H */

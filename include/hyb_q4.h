/*
 * hyb_q4.h -- C ABI of libhyb's 4-bit weights with group scales and their
 * product.
 *
 * A weight (n x k, out x in) is held as e2m1 codes (1 sign, 2 exponent, 1
 * mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives) with one
 * power-of-two scale per group of 32 columns of a row: 4.25 bits a weight.
 * Groups start at column 0; a row's last may be shorter.
 *
 * Scale of a group: 2^e with the smallest integer e, -125 <= e <= 125, that
 * brings the group's largest magnitude to 7 * 2^e or less (7 rounds to 6: no
 * element is off by more than half the spacing of the codes' top binade); 1 for
 * a group of zeros.  Code of an element a: a / 2^e (exact) rounded once, to
 * nearest, halves to the even code, at most 6; the sign is kept.  A group that
 * holds a NaN or an infinity stands for NaN throughout.  A value read back,
 * code * 2^e, is exact in fp32 and bf16 (2 significant bits, no smaller than
 * 2^-126), and in fp16 within that type's range.
 *
 * Product: Y[i, j] = sum_c X[i, c] W[j, c] over the values that the codes stand
 * for, X in 16 bits as it is.  The products are exact and are summed in fp32.
 * For fp16 activations the values of a row are carried relative to the row's
 * largest scale: exact for scales down to 2^-36 of it, values of smaller ones
 * may count as zero.  For bf16 ones, values and products below 2^-126 may.
 *
 * Storage "HYB4": rows are rounded up to 16 (a panel), columns to 128 (a
 * step); what is behind the matrix's edge holds code 0.
 *   codes   element (r, c) in byte
 *           ((r/16) * steps + c/128) * 1024 + ((c%32)/8) * 256 + (r%16) * 16
 *           + ((c%128)/32) * 4 + (c%8)/2,   steps = ceil(k/128),
 *           low half for even c, high half for odd c
 *   scales  e + 127 (255: a NaN group) of row r and group g = c/32 in byte
 *           ((g/16) * rows16 + r) * 16 + g%16, g up to 16 ceil(steps/4);
 *           rows16 = rows rounded up to 16; unused bytes 127.  Behind them, one
 *           byte per row: the largest byte of its groups that are neither all
 *           zeros nor NaN (127 if there is none).
 *
 * Conventions as in hyb.h and hyb_f8.h: device pointers are plain addresses,
 * calls check their arguments on the host, enqueue on `stream` and return;
 * nothing is allocated; outputs must not overlap inputs; hyb_last_error has the
 * detail of a failed call.  Calls may be captured into a graph.
 */
#ifndef HYB_Q4_H_
#define HYB_Q4_H_

#include "hyb.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Device addresses of one 4-bit weight (owned by the caller), both 16-byte
 * aligned; may be NULL where hyb_q4_size gives 0 bytes. */
typedef struct {
  void* codes;
  void* scales;
} hyb_q4;

/* Bytes of the two buffers of an n x k weight (0 when n or k is 0).  Host
 * only.  0 <= n <= 2^27 - 16, 0 <= k <= 2^22, else HYB_ERR_SHAPE. */
hyb_status hyb_q4_size(int64_t n, int64_t k, size_t* code_bytes, size_t* scale_bytes);

/* Quantise A (n x k of `dtype`, HYB_F16, HYB_BF16 or HYB_F32, row stride
 * lda >= k elements, element-aligned; 16-byte aligned rows are read fastest)
 * into dst. */
hyb_status hyb_q4_quantize(const void* a, int32_t dtype, int64_t n, int64_t k, int64_t lda, const hyb_q4* dst,
                           void* stream);

/* The values that the codes stand for, n x k of `dtype` (any of the three;
 * rounded to nearest, halves to even, where fp16 does not hold one), row stride
 * lda >= k. */
hyb_status hyb_q4_dequantize(const hyb_q4* src, int64_t n, int64_t k, void* a, int32_t dtype, int64_t lda,
                             void* stream);

/* Y = X W^T for any number 0 <= m <= 2^22 of tokens, one included.  (A launch bounds n
 * m: ceil(n/128) ceil(m/16) below 2^23 is always taken, what is beyond may be
 * HYB_ERR_UNSUPPORTED.)  Row strides, here and above, are at most 2^31.
 *   x   device m x k of x_dtype (HYB_BF16 or HYB_F16), row stride ldx >= k,
 *       element-aligned (16-byte aligned rows are read fastest)
 *   y   device m x n of y_dtype (HYB_F32, HYB_BF16 or HYB_F16; 16-bit outputs
 *       are rounded to nearest even from the fp32 sum), row stride ldy >= n,
 *       element-aligned.  k = 0 gives zeros.
 * The workspace (device, 16-byte aligned, no initial contents, the bytes of
 * hyb_q4_gemm_workspace_size for the current device; may be 0) holds
 * activations laid out for the matrix units and the fp32 sums of products whose
 * k is cut into parts, which are added in a fixed order; calls that overlap on
 * one buffer race. */
hyb_status hyb_q4_gemm_workspace_size(int64_t n, int64_t k, int32_t m, size_t* bytes);
hyb_status hyb_q4_gemm(const hyb_q4* w, int64_t n, int64_t k, const void* x, int32_t x_dtype, int32_t m, int64_t ldx,
                       void* y, int32_t y_dtype, int64_t ldy, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* HYB_Q4_H_ */

/*
 * hyb_f8.h -- C ABI of libhyb's 8-bit block-scaled matrices and their product.
 *
 * A matrix (rows x k) is held as e4m3 codes (1 sign, 4 exponent, 3 mantissa
 * bits, largest finite value 448) with one power-of-two scale per block:
 *   HYB_F8_WEIGHT  blocks of 128 rows x 128 columns (a weight, out x in)
 *   HYB_F8_ROWS    blocks of 1 row x 128 columns (activations)
 * Blocks start at row 0 and column 0; the last ones may be shorter.
 *
 * Scale of a block: 2^e with the smallest integer e, -127 <= e, that brings
 * the block's largest finite magnitude to 448 * 2^e or less; 1 for a block
 * without a finite non-zero element.  Code of an element a: a / 2^e (exact)
 * rounded once to e4m3, to nearest, halves to even.  NaN and infinities
 * become the NaN code 0xFF (they do not enter the scale), so an output they
 * reach is NaN.  A value read back, code * 2^e, is exact in the type that was
 * quantised, unless the code rounded up past that type's largest number.
 *
 * Product: Y[i, j] = sum_c X[i, c] W[j, c] over the values that the codes
 * stand for.  The products are exact and are summed in fp32, for an fp32
 * output without further loss.  For a 16-bit output the sums of 128 columns
 * may come from the 8-bit matrix instruction, which drops bits of a product
 * that lie far below the largest of the 128: an error of at most 2^-11 of that
 * largest product, ahead of the output's own rounding.  Values, products and
 * sums below 2^-126, the smallest normal number of fp32 and bf16, may count as
 * zero: a weight of 1e-38 may add nothing, however large its activation.
 *
 * Storage "HYB8", both kinds: rows are rounded up to 16 (a panel), columns to
 * 128 (a step); what is behind the matrix's edge holds code 0.
 *   codes   element (r, c) at byte
 *           ((r/16) * steps + c/128) * 2048 + ((c%128)/64) * 1024
 *           + ((c%64)/16) * 256 + (r%16) * 16 + c%16,   steps = ceil(k/128)
 *   scales  byte e + 127 of row r and step s in the 32-bit little-endian word
 *           (s/4) * rows16 + r, bits 8 (s%4) .. 8 (s%4) + 7; rows16 = rows
 *           rounded up to 16; unused bytes 127.  (A weight's block scale is
 *           written for each of its rows.)
 *
 * Conventions as in hyb.h: device pointers are plain addresses, calls check
 * their arguments on the host, enqueue on `stream` and return; nothing is
 * allocated; outputs must not overlap inputs; hyb_last_error has the detail
 * of a failed call.  Calls may be captured into a graph.
 */
#ifndef HYB_F8_H_
#define HYB_F8_H_

#include "hyb.h"

#ifdef __cplusplus
extern "C" {
#endif

enum { HYB_F8_WEIGHT = 1, HYB_F8_ROWS = 2 };

/* Device addresses of one quantised matrix (owned by the caller), both
 * 16-byte aligned; may be NULL where hyb_f8_size gives 0 bytes. */
typedef struct {
  void* codes;
  void* scales;
} hyb_f8;

/* Bytes of the two buffers of a rows x k matrix (the same for both kinds;
 * 0 when rows or k is 0).  Host only.  0 <= rows <= 2^27 - 16, 0 <= k <= 2^22,
 * else HYB_ERR_SHAPE. */
hyb_status hyb_f8_size(int64_t rows, int64_t k, size_t* code_bytes, size_t* scale_bytes);

/* Quantise A (rows x k of `dtype`, HYB_F16, HYB_BF16 or HYB_F32, row stride
 * lda >= k elements, element-aligned; 16-byte aligned rows are read fastest)
 * into dst. */
hyb_status hyb_f8_quantize(const void* a, int32_t dtype, int64_t rows, int64_t k, int64_t lda, int32_t kind,
                           const hyb_f8* dst, void* stream);

/* The values that the codes stand for, rows x k of `dtype` (any of the three;
 * exact for the type that was quantised, for HYB_F32 and, from 2^-130 on, for
 * HYB_BF16, rounded to nearest, halves to even, otherwise), row stride
 * lda >= k. */
hyb_status hyb_f8_dequantize(const hyb_f8* src, int64_t rows, int64_t k, void* a, int32_t dtype, int64_t lda,
                             void* stream);

/* Y = X W^T for any number m >= 0 of tokens, one included: w is n x k
 * (HYB_F8_WEIGHT), x is m x k (HYB_F8_ROWS), y device m x n of y_dtype
 * (HYB_F32, HYB_BF16 or HYB_F16; 16-bit outputs are rounded to nearest even
 * from the fp32 sum), row stride ldy >= n, element-aligned (4 elements wide
 * stores where the rows are aligned for them).  k = 0 gives zeros.
 * Products whose tiles would leave compute units idle cut k into parts and
 * add the parts' fp32 sums in a fixed order: they keep the sums in
 * `workspace` (device, 16-byte aligned, no initial contents needed, the
 * bytes of hyb_f8_gemm_workspace_size for the current device; calls that
 * overlap on one buffer race).  workspace_bytes = 0 runs unsplit; a positive
 * size below the need is HYB_ERR_INVALID_ARG. */
hyb_status hyb_f8_gemm_workspace_size(int64_t n, int64_t k, int32_t m, size_t* bytes);
hyb_status hyb_f8_gemm(const hyb_f8* w, int64_t n, int64_t k, const hyb_f8* x, int32_t m, void* y, int32_t y_dtype,
                       int64_t ldy, void* workspace, size_t workspace_bytes, void* stream);

/* hyb_f8_quantize of x (m x k of x_dtype, row stride ldx) and hyb_f8_gemm in
 * one call, for activations that one product reads.  The workspace (bytes of
 * hyb_f8_linear_workspace_size, 16-byte aligned, as above) is needed: it holds
 * the codes as well.  The result is bitwise that of the two calls. */
hyb_status hyb_f8_linear_workspace_size(int64_t n, int64_t k, int32_t m, size_t* bytes);
hyb_status hyb_f8_linear(const hyb_f8* w, int64_t n, int64_t k, const void* x, int32_t x_dtype, int32_t m, int64_t ldx,
                         void* y, int32_t y_dtype, int64_t ldy, void* workspace, size_t workspace_bytes,
                         void* stream);

#ifdef __cplusplus
}
#endif
#endif /* HYB_F8_H_ */

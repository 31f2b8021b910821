/*
 * lnq_fp4.h -- C ABI of the library's microscaled 4-bit floating-point operators (sm_100a).
 *
 * The uniform 4-bit counterpart of lnq_pack_codes and lnq_lut_gemv (lnq.h): where LNQ gives each
 * output row a codebook of its own, these formats store a matrix as 4-bit floating-point codes
 * with one 8-bit scale per block of consecutive elements of a row, which the tensor cores
 * multiply as they are.
 *
 * A code is an E2M1 number: bit 3 the sign, bits 2-0 the magnitude out of
 * {0, 0.5, 1, 1.5, 2, 3, 4, 6}. Two formats:
 *   LNQ_FP4_MX  blocks of B = 32; the scale byte b is a power of two (E8M0), s = 2^(b - 127),
 *               255 = NaN. There is no matrix scale (t = 1): pass NULL.
 *   LNQ_FP4_NV  blocks of B = 16; the scale byte is an E4M3 number without sign (bit 7 is zero),
 *               127 = NaN; t is a positive 32-bit scale for the whole matrix, in device memory
 *               (NULL: t = 1).
 * The element stands for  code * s * t.
 *
 * Layout of a matrix of `rows` rows and d columns, all in device memory:
 *   codes   [rows][lnq_fp4_code_bytes(d)]          element i in byte i / 2, even i in the low half
 *   scales  [rows][lnq_fp4_scale_bytes(d, fmt)]    block k in byte k
 *   Both row pitches are those of d rounded up to a multiple of 128 (64 bytes of codes, 4 (MX) or
 *   8 (NV) bytes of scales per 128 elements). Bytes that lie wholly behind the row's last element
 *   or block may hold anything; where d is odd, the upper half of the last byte is zero.
 *   lnq_fp4_quantize writes zeros behind the row.
 *   Alignment: codes 16 bytes; scales 4 (MX) or 8 (NV) bytes; t 4 bytes; x and y their element.
 *
 * The conventions on streams, ownership and errors are those of lnq.h. No operator here takes a
 * workspace or allocates device memory, and inputs and outputs must not overlap. A size of zero
 * rows is a valid call that does nothing (its pointers may be NULL). Results do not depend on
 * timing: no floating-point atomics, every sum in an order fixed by the sizes and the device.
 *
 * Grouped operators: `offsets` is a device array of experts + 1 int32 row numbers; the rows
 * offsets[e] .. offsets[e+1] - 1 of the activations use matrix e. Rows before offsets[0] or from
 * offsets[experts] on are neither read nor written. The values are read on the device, where each
 * is limited to 0 .. n and to no less than the largest before it, so that no array of offsets
 * leads outside the arrays.
 */
#ifndef LNQ_FP4_H
#define LNQ_FP4_H

#include "lnq.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { LNQ_FP4_MX = 0, LNQ_FP4_NV = 1 } lnq_fp4_format;

/* Types of unquantised matrices. */
typedef enum { LNQ_F32 = 0, LNQ_BF16 = 1, LNQ_F16 = 2 } lnq_dtype;

/* Largest sizes the operators take: elements of a row, rows of a matrix (of all experts' matrices
 * together), experts. */
#define LNQ_FP4_MAX_D (1ll << 24)
#define LNQ_FP4_MAX_ROWS (1ll << 30)
#define LNQ_FP4_MAX_EXPERTS 1024

/* Bytes per row of codes and of scales (0 if d or fmt is invalid). */
LNQ_API int64_t lnq_fp4_code_bytes(int64_t d);
LNQ_API int64_t lnq_fp4_scale_bytes(int64_t d, lnq_fp4_format fmt);

/* t[0] = (largest finite |x|) / 2688, rounded to 32 bits: the matrix scale with which the largest
 * element gets the largest code (6) and block scale (448). 1 where that quotient rounds to zero.
 *   x [rows][ldx] of type xt, columns 0 .. d-1 read; t one float, out.
 * Requirements: rows >= 0 (0 gives t = 1; x may be NULL), 1 <= d <= ldx. */
LNQ_API lnq_status lnq_fp4_tensor_scale(const void *x, lnq_dtype xt, int64_t rows, int64_t d,
                                        int64_t ldx, float *t, lnq_stream_t stream);

/* Quantises x [rows][ldx] (type xt, columns 0 .. d-1) to codes and scales.
 *   MX: s = 2^e, e = floor(log2(amax)) - 2 limited to -127 .. 125, amax = max |x| of the block.
 *   NV: s = amax / (6 t), rounded to the nearest E4M3 number (ties to even), at most 448.
 *   code = x / (s t), rounded to the nearest E2M1 number (ties to the even code), at most 6 in
 *   magnitude; 0 where s = 0.
 * Both roundings are those of the exact quotients. A block that holds a NaN or an infinity, and
 * every block where t is not a positive finite number, gets the NaN scale and zero codes.
 * Requirements: rows >= 0, 1 <= d <= ldx, d <= LNQ_FP4_MAX_D; t NULL for MX. */
LNQ_API lnq_status lnq_fp4_quantize(const void *x, lnq_dtype xt, int64_t rows, int64_t d,
                                    int64_t ldx, lnq_fp4_format fmt, const float *t,
                                    uint8_t *codes, uint8_t *scales, lnq_stream_t stream);

/* y [rows][ldy] (type yt, columns 0 .. d-1 written) = code * s * t. code * s is exact; the product
 * with t is rounded to 32 bits and then, for the 16-bit types, to the type (infinite where it
 * does not fit). */
LNQ_API lnq_status lnq_fp4_dequantize(const uint8_t *codes, const uint8_t *scales, int64_t rows,
                                      int64_t d, lnq_fp4_format fmt, const float *t, void *y,
                                      lnq_dtype yt, int64_t ldy, lnq_stream_t stream);

/* y[b][j] = sum_i x[b][i] w[j][i] for b < nb: unquantised activations times a quantised matrix,
 * for the few rows of a decoding step (any nb >= 0 is taken; the weights are read once for every
 * 32 rows of bf16, 16 of f16 or 10 of f32 x, and lnq_fp4_gemm is the operator for prompts).
 *   x [nb][ldx] of type xt; codes, scales [d_out] rows of d_in; y [nb][ldy] of type yt, out.
 * Arithmetic: every product is exact, the sums are 32-bit, the product of t with the finished sum is
 * rounded to 32 bits and then to y's type. (Bits of a 32-bit x below 2^-133, and of a product before t
 * below 2^-142, may be dropped.) */
LNQ_API lnq_status lnq_fp4_gemv(const void *x, lnq_dtype xt, int64_t nb, int64_t ldx,
                                const uint8_t *codes, const uint8_t *scales, const float *t,
                                int64_t d_out, int64_t d_in, lnq_fp4_format fmt, void *y,
                                lnq_dtype yt, int64_t ldy, lnq_stream_t stream);

/* lnq_fp4_gemv with the rows of x grouped by expert: codes and scales hold `experts` matrices of
 * d_out rows one after another, t is [experts] (or NULL). A pass over a matrix takes the rows of an
 * average group (n / experts, rounded up to 8, 16, 24 or 32 rows of bf16, half of that of f16, 2, 5, 8
 * or 10 of f32); a larger group reads its matrix once for each such number of rows. */
LNQ_API lnq_status lnq_fp4_grouped_gemv(const void *x, lnq_dtype xt, int64_t n, int64_t ldx,
                                        const int32_t *offsets, int64_t experts,
                                        const uint8_t *codes, const uint8_t *scales,
                                        const float *t, int64_t d_out, int64_t d_in,
                                        lnq_fp4_format fmt, void *y, lnq_dtype yt, int64_t ldy,
                                        lnq_stream_t stream);

/* y[b][j] = sum_i a[b][i] w[j][i]: the product of two quantised matrices of one format, on the
 * block-scaled tensor cores.
 *   a: codes and scales of [n] rows of d_in, matrix scale ta; w: of [d_out] rows, matrix scale
 *   tw; y [n][ldy] of type yt, out.
 * Arithmetic: products of codes and block scales are exact, the sums 32-bit (24 bits, cut off); ta
 * and tw multiply the finished sum, each product rounded to 32 bits and the last one to yt. Where
 * the sum times one of them would leave the 32-bit range and the result does not, nothing is lost. */
LNQ_API lnq_status lnq_fp4_gemm(const uint8_t *a_codes, const uint8_t *a_scales, const float *ta,
                                int64_t n, const uint8_t *w_codes, const uint8_t *w_scales,
                                const float *tw, int64_t d_out, int64_t d_in,
                                lnq_fp4_format fmt, void *y, lnq_dtype yt, int64_t ldy,
                                lnq_stream_t stream);

/* lnq_fp4_gemm with the rows of a grouped by expert: w_codes and w_scales hold `experts` matrices
 * of d_out rows one after another, tw is [experts] (or NULL). */
LNQ_API lnq_status lnq_fp4_grouped_gemm(const uint8_t *a_codes, const uint8_t *a_scales,
                                        const float *ta, int64_t n, const int32_t *offsets,
                                        int64_t experts, const uint8_t *w_codes,
                                        const uint8_t *w_scales, const float *tw, int64_t d_out,
                                        int64_t d_in, lnq_fp4_format fmt, void *y, lnq_dtype yt,
                                        int64_t ldy, lnq_stream_t stream);

/* Synchronises `stream` and reports whether a bounded wait inside an lnq_fp4_* product has given up
 * (LNQ_ERR_TIMEOUT: the results of the calls concerned are incomplete), on the current device:
 *   a stream: in a product called on it, or in one captured into a graph, wherever the graph ran;
 *   the default stream (NULL): in any product of the device;
 * each since the stream's last report, or since the library was loaded. Every stream has reports of
 * its own, and one stream's takes nothing from another's; callers that share a stream share them.
 * Streams beyond the first thousand may share a count, and then both report; a stream that got the
 * handle of a destroyed one also got its reports. */
LNQ_API lnq_status lnq_fp4_check(lnq_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LNQ_FP4_H */

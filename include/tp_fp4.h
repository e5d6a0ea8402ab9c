/*
 * tp_fp4.h - C ABI of libtpmlp's four-bit operators on one GB300 (sm_103a):
 * microscaled quantisation, the product of two quantised matrices, and the MLP
 * block's forward on four-bit weights.  Status codes, tp_mlp_status_string() and
 * tp_mlp_last_detail() are shared with tp_mlp.h.
 *
 * A matrix [rows, cols] is quantised along its rows in blocks of consecutive
 * elements (the last block of a row may be short).  An element is an E2M1 code
 * (0 .5 1 1.5 2 3 4 6 with a sign); a block has one scale:
 *
 *   TPFP4_NV   blocks of 16, scale s in E4M3, one power of two g for the matrix:
 *              s    = e4m3(amax / (6 g))      nearest even, at most 448
 *              code = e2m1(x / (s g))         nearest even, at most 6
 *              value = code s g.  g is given, or the smallest power of two
 *              with max |x| <= 2688 g (1 for a matrix of zeros; infinities and
 *              NaNs are not counted).  A block whose s is 0 has codes of 0.
 *   TPFP4_MX   blocks of 32, scale s = 2^e in E8M0 (Open Compute Project,
 *              "Microscaling Formats (MX)", v1.0): e = floor(log2 amax) - 2, at
 *              least -127 (s = 1 for a block of zeros), code = e2m1(x / s),
 *              value = code s; g = 1.
 *
 * With a g far above what a matrix needs small blocks are lost: one whose largest |x|
 * is at most 6 g 2^-10 (0.0059 for g = 1) has s = 0 and values of 0, and below 6 g 2^-6
 * (0.094) s is one of E4M3's few subnormal numbers.
 *
 * Quotients are not rounded before the code is chosen: every code is the one
 * the definition gives (a code of zero may have either sign).  A block that holds
 * an infinity or a NaN has the scale's NaN, and its values are NaN.
 *
 * The product of A [T, K] and B [N, K], both quantised along K in the same
 * format, is C[t, n] = g_A g_B sum_k A[t, k] B[n, k] (+ bias[n]): the tensor
 * cores multiply the codes and the blocks' scales exactly and add in fp32; one
 * rounding to C's type.  Repeated calls are bit-identical.
 *
 * Conventions
 * -----------
 * - Plain matrices are bf16 (TPMLP_BF16) or fp32 (TPMLP_FP32), row-major with
 *   any row stride >= the number of columns, aligned to their element; 32-byte
 *   aligned rows are read fastest.  What lies between rows may be read, and is
 *   never written.  A packed matrix is one buffer of
 *   tp_fp4_bytes bytes, 256-byte aligned, whose first 4096 bytes hold the status
 *   word of the products that read it as A (16 bytes), g (fp32) and scratch.
 * - rows and cols are 1 .. 2^28 (rows of a plain matrix: 0 .. 2^28).
 * - Pointers are DEVICE pointers the caller owns; the library never allocates
 *   device memory.  Calls only enqueue work on `stream`.  No output shares
 *   memory with an input (TPMLP_ERR_ARG).  Every function returns a status
 *   code and touches no output when argument validation fails.
 */
#ifndef TP_FP4_H_
#define TP_FP4_H_

#include <stddef.h>

#include "tp_mlp.h"

#ifdef __cplusplus
extern "C" {
#endif

#define TPFP4_NV 0
#define TPFP4_MX 1

/* Bytes of a packed [rows, cols] matrix (0 for a bad format or size), and the
 * offsets of its parts (-1 likewise):
 *   TPFP4_CODES   two codes a byte, in tiles of 128 rows x 256 columns (16 KB),
 *                 tile (r / 128, c / 256) being number n = (r / 128)
 *                 ceil(cols / 256) + c / 256: columns 32 u .. 32 u + 31 of row r
 *                 (u of the tile) are the 16 bytes at 16384 n + (r mod 128) 128 +
 *                 (u xor (r mod 8)) 16 (shared memory's 128-byte swizzle), two
 *                 columns a byte, the even one in the low nibble; zeros past cols
 *   TPFP4_SCALES  one byte a block, in tiles of the same rows and columns (2048
 *                 bytes NV, 1024 MX): the scale of block b = (c mod 256) / 16
 *                 (NV) or / 32 (MX) of row r at n times that + (b / 4) 512 +
 *                 (r mod 32) 16 + ((r mod 128) / 32) 4 + b mod 4; 0 (NV) or 127
 *                 (MX) past cols
 * What lies in rows past the matrix is not defined. */
size_t tp_fp4_bytes(long long rows, long long cols, int format);
long long tp_fp4_offset(long long rows, long long cols, int format, int which);
#define TPFP4_CODES  0
#define TPFP4_SCALES 1

/* Quantise x [rows, cols] along its rows into a packed [rows, cols], or
 * (transpose = 1) along its columns into a packed [cols, rows], the transposed
 * matrix.
 *   scale    NV: g, a power of two from 2^-126 to 2^127, or 0 to take it from
 *            the matrix (x is read twice); MX: 0 or 1
 *   like     NV with scale = 0: a packed matrix whose g is taken instead, or NULL
 *   colsum   [cols] fp32, the sums of x's columns (a bias gradient, in a fixed
 *            order; transpose = 1 only), or NULL
 *   workspace  tp_fp4_colsum_workspace_bytes(rows, cols) bytes, 16-byte
 *            aligned, used only with colsum
 * rows = 0 (transpose = 0) enqueues nothing, and leaves the header as it is. */
int tp_fp4_quantize(long long rows, long long cols, int dtype, const void* x,
                    long long row_stride, int transpose, int format,
                    double scale, const void* like, void* packed,
                    size_t packed_bytes, float* colsum, void* workspace,
                    size_t workspace_bytes, void* stream);
size_t tp_fp4_colsum_workspace_bytes(long long rows, long long cols);

/* x [rows >= 1, cols] both ways in one pass: along its rows into `packed`
 * [rows, cols], along its columns into packed_t [cols, rows]; the rest as above.
 * The same results as the two calls one by one. */
int tp_fp4_quantize_both(long long rows, long long cols, int dtype, const void* x,
                         long long row_stride, int format, double scale,
                         void* packed, size_t packed_bytes, void* packed_t,
                         size_t packed_t_bytes, float* colsum, void* workspace,
                         size_t workspace_bytes, void* stream);

/* The values of a packed [rows, cols] matrix, written as `dtype` (exact in bf16
 * too, but for values out of its range). */
int tp_fp4_dequantize(long long rows, long long cols, int format,
                      const void* packed, size_t packed_bytes, int dtype,
                      void* out, long long row_stride, void* stream);

/* C [T, N] (`dtype`, row stride ldc) from packed A [T, K] and B [N, K].  bias
 * [N] fp32 or NULL.  status: 16 bytes that the caller zeroed, where the first error
 * of all calls that are given them stays until tp_fp4_check, or NULL for A's status
 * word.  T = 0 enqueues nothing. */
int tp_fp4_matmul(long long T, long long N, long long K, int format,
                  const void* A, size_t a_bytes, const void* B, size_t b_bytes,
                  const float* bias, int dtype, void* C, long long ldc,
                  void* status, void* stream);

/* Both in one call, for a layer y = x W: x [T, K] (x_dtype, x_stride) quantised
 * (x_scale as tp_fp4_quantize's scale) times the packed W [N, K].  xq is scratch of
 * tp_fp4_bytes(T, K, format) bytes; status as above (NULL: xq's).  The product
 * starts to load W while x is quantised, and up to 8 rows of bf16 (4 of
 * fp32) with a given x_scale are quantised by the product itself.  xq and C share no memory with the rest. */
int tp_fp4_linear(long long T, long long N, long long K, int x_dtype,
                  const void* x, long long x_stride, int format, double x_scale,
                  void* xq, size_t xq_bytes, const void* W, size_t w_bytes,
                  const float* bias, int dtype, void* C, long long ldc,
                  void* status, void* stream);

/* Waits for `stream`, then reads and clears a status word: that of a packed matrix
 * that products read as A, or one given to the calls: TPMLP_OK, TPMLP_ERR_TIMEOUT (a bounded device wait
 * gave up; that product's C is undefined) or TPMLP_ERR_CUDA. */
int tp_fp4_check(void* status, void* stream);

/* ---- the MLP block's forward on four-bit weights ------------------------
 *   Xq = quantised Xn (= LayerNorm(X) rounded to bf16, or X), H = Xq Aq + b1,
 *   Y = GeLU(H) (fp32, within 2.2e-7 in all and 4e-3 of itself down to H = -6),
 *   Yq = quantised Y, Z = Yq Bq + b2 [+ X], one rounding to
 * bf16.  A and B are quantised along the products' inner dimension (NV: g from
 * each); x_scale and y_scale are NV's g of Xn and Y (MX: 0 or 1): powers of two that
 * the caller knows, not taken from Xn and Y; blocks far below 448 g are held coarsely
 * or not at all (see TPFP4_NV).  The t shards
 * are consecutive ranges of the second product's one sum, so Z does not depend
 * on t.  The handle must be TPMLP_BF16 without dropout (TPMLP_ERR_ARG). */
size_t tp_fp4_mlp_weights_bytes(const tp_mlp_handle* handle, int format);
int tp_fp4_mlp_pack_weights(tp_mlp_handle* handle, int format, const void* A,
                            const void* B, void* packed, size_t packed_bytes,
                            void* stream);
size_t tp_fp4_mlp_workspace_bytes(const tp_mlp_handle* handle, int tokens,
                                  int format);
/* status: 16 bytes of device memory, 16-byte aligned, that the caller zeroed, where
 * the first error of all the handle's tp_fp4_mlp_forward calls from here on stays
 * until tp_fp4_check reads it; or NULL, as a new handle has it: a call's error is left
 * in its own workspace, where the next call on that workspace clears it. */
int tp_fp4_mlp_set_status(tp_mlp_handle* handle, void* status);
/* Arguments as tp_mlp_forward_fp8; packed and workspace 256-byte aligned;
 * tp_mlp_check reads the workspace's status, where tp_fp4_mlp_set_status has not
 * given another place. */
int tp_fp4_mlp_forward(tp_mlp_handle* handle, int tokens, int format,
                       const void* X, const void* packed, const float* bias1,
                       const float* bias2, const float* ln_gamma,
                       const float* ln_beta, double x_scale, double y_scale,
                       void* Z, void* workspace, size_t workspace_bytes,
                       void* stream);

#ifdef __cplusplus
}
#endif
#endif /* TP_FP4_H_ */

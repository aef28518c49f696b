/*
 * muon_linear.h - C ABI of the 8-bit operators of linear layers on one gfx950 GPU (same
 * library, same conventions and status codes as muon.h): the product in 8-bit integers with a
 * scale for each token and channel, activation checkpoints in 8 bits, and the weight gradient
 * that is formed from one.
 *
 * Why they are here: the gradients that the optimizer step reads come from the products of the
 * linear layers whose matrices it owns, y = x W^T with x tokens x inputs and W outputs x
 * inputs.  A layer runs
 *   forward    xq = codes of x's rows;  y = xq . wq^T             muon_int8_linear
 *              kept = codes of x's blocks, instead of x           muon_quantize
 *   backward   wt = codes of W's columns; gq = codes of dy's rows;
 *              dx = gq . wt^T                                     muon_int8_linear
 *              dw = [dw +] dy^T kept                              muon_weight_grad
 * and dw is the `grad` of a muon_matrix, or of a muon_grad list.
 *
 * Codes: 8-bit integers q in [-127, 127] with scales s, each standing for q s.
 *   by row    one scale for each row r: s = max |x_rc| / 127 (fp32), and q_rc is the integer
 *             nearest to 127 x_rc / max |x_r|, a value in the middle between two going to the
 *             even one: exactly, whatever x's type.  A row of zeros has scale 0.
 *   by block  one scale for each 128 columns of a row (the last block may be shorter): the
 *             smallest power of two s = 2^e, -126 <= e <= 121, with max |x| <= 127 s where
 *             there is one, and q = x / s rounded to the nearest integer (ties to even), no
 *             further from 0 than 127.  The value q s is a bf16 number, so nothing is rounded
 *             a second time when a checkpoint is read.
 *   A row (a block) that holds a NaN or an infinity has a NaN scale and codes 0: everything
 *   formed from it is NaN, as everything formed from x would be NaN or infinite.
 *
 * Products: muon_int8_matmul and muon_int8_linear sum in 32-bit integers, exactly (at most
 * 131071 columns), and round that sum to fp32, its two products with the scales, and the
 * result's type.  Where a sum times its first scale leaves the fp32 range the result is
 * infinite.  muon_weight_grad's products of bf16 dy with the decoded
 * checkpoint are exact and summed in fp32; for an fp32 dy the products run in fp32.
 * Accumulation adds to the old gradient in fp32; a bf16 result is rounded to nearest even once.
 * Sums are taken in an order that depends on sizes only: results are bitwise reproducible.
 */
#ifndef MUON_LINEAR_H
#define MUON_LINEAR_H

#include "muon.h"

#ifdef __cplusplus
extern "C" {
#endif

/* rows x cols elements of `dtype` (muon_dtype) in device memory, aligned to their size; row r
 * begins ld elements after row r - 1 (ld >= cols where there are two rows).  No element (rows
 * or cols 0): data may be NULL. */
typedef struct muon_view {
  void* data;
  int64_t rows;
  int64_t cols;
  int64_t ld;
  int32_t dtype;
  int32_t reserved; /* must be 0 */
} muon_view;

/* Bytes from one row of codes to the next. */
#define MUON_CODES_PITCH(cols) (((int64_t)(cols) + 127) / 128 * 128)

/* Codes of a rows x cols matrix.  q: rows * MUON_CODES_PITCH(cols) bytes, 16-byte aligned, a
 * row's bytes behind its cols codes being 0 (muon_quantize writes them so).  scale: fp32,
 * 4-byte aligned, rows values (block 0) or rows * ceil(cols / 128), row by row (block 128). */
typedef struct muon_codes {
  void* q;
  float* scale;
  int64_t rows;
  int64_t cols;
  int32_t block;    /* 0: one scale a row, 128: one for each 128 columns of a row */
  int32_t reserved; /* must be 0 */
} muon_codes;

/* Sizes: rows and cols from 0 to 2^30; muon_int8_matmul and muon_int8_linear sum over at most 131071
 * columns; muon_weight_grad of a bf16 dy takes at most 2^24 - 8 columns of dy and of x; and results
 * of more than 2^23 tiles of 128 x 128 (2^26 columns for up to 64 rows) are refused.  `workspace` is device memory of at least the size that
 * the call's _size function gives for the same arguments (0: NULL will do), 256-byte aligned, owned by the caller and
 * written by nothing else until the stream has passed the call; its contents do not matter, and
 * calls in flight at once need one each.  An output may overlap no input, no other output and
 * not the workspace (MUON_EALIAS); interleaved rows of one wider buffer do not overlap. */

/* codes <- the codes of x: of its rows, or with transpose != 0 of its columns (codes->rows =
 * x->cols, codes->cols = x->rows; block 0 only). */
int muon_quantize_size(const muon_view* x, int32_t transpose, size_t* bytes);
int muon_quantize(const muon_view* x, int32_t transpose, const muon_codes* codes, void* workspace,
                  size_t workspace_bytes, void* hip_stream);

/* out <- the values that the codes stand for, the fp32 product q s rounded to out's type. */
int muon_dequantize(const muon_codes* codes, const muon_view* out, void* hip_stream);

/* out (a->rows x b->rows) <- a b^T, from codes by row. */
int muon_int8_matmul_size(const muon_codes* a, const muon_codes* b, size_t* bytes);
int muon_int8_matmul(const muon_codes* a, const muon_codes* b, const muon_view* out, void* workspace,
                     size_t workspace_bytes, void* hip_stream);

/* out (x->rows x w->rows) <- (codes of x's rows) w^T: muon_quantize and muon_int8_matmul, bit for
 * bit, in one launch for a few rows. */
int muon_int8_linear_size(const muon_view* x, const muon_codes* w, size_t* bytes);
int muon_int8_linear(const muon_view* x, const muon_codes* w, const muon_view* out, void* workspace,
                     size_t workspace_bytes, void* hip_stream);

/* out (dy->cols x x->cols) <- dy^T x, or out + dy^T x with accumulate != 0, from x's codes by
 * block; dy->rows = x->rows. */
int muon_weight_grad_size(const muon_view* dy, const muon_codes* x, size_t* bytes);
int muon_weight_grad(const muon_view* dy, const muon_codes* x, const muon_view* out, int32_t accumulate,
                     void* workspace, size_t workspace_bytes, void* hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* MUON_LINEAR_H */

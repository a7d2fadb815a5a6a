/*
 * f8_gemm.h -- matrix products on 8-bit floating-point operands with one FP32 scale for each
 * block of 128 along the contraction, and the quantiser that makes such operands, for one
 * NVIDIA GB300 (sm_103a), C ABI. Part of the same library as sgemm_f32.h, whose conventions on
 * memory, streams and asynchrony hold here too.
 *
 * Formats: F8_E4M3 (largest number 448, no infinity) and F8_E5M2 (largest finite 57344).
 *
 * A quantised matrix is a row-major byte matrix q (leading dimension ldq) and FP32 scales s. The
 * value of element (i, j) is q(i, j) * s of its block. Blocks are 1 x 128, 128 x 1 or 128 x 128
 * elements, counted from element (0, 0); the last blocks of a row or column may be shorter.
 */
#ifndef F8_GEMM_H_
#define F8_GEMM_H_

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st *cudaStream_t;

enum { F8_E4M3 = 0, F8_E5M2 = 1 };               /* formats of quantised operands */
enum { F8_D_F32 = 0, F8_D_BF16 = 1, F8_D_F16 = 2 }; /* types of x and of D */

/* Quantise x (rows x cols, row-major, leading dimension ldx, type x_type): for each block b
 *   s_b = max(max_{b} |x| / F, 2^-126), F the format's largest number; with pow2 != 0 the least
 *         power of two that is not smaller (then x / s_b is exact, and so are later products
 *         with s_b)
 *   q   = x / s_b, rounded once to the format (nearest, ties to even; FP32 division)
 * A block with a NaN gets a NaN scale, one with an infinity an infinite scale, so that neither
 * is lost in a product.
 *
 * One or two results from one read of x (the second is left out with qc = NULL).
 *   q,  s  blocks of block_rows x block_cols, one of 1 x 128, 128 x 1, 128 x 128
 *   qc, sc blocks of 128 x 1; only together with 1 x 128 blocks in q
 * Scale of block (bi, bj) at s[bi * s_row + bj * s_col], sc[bi * sc_row + bj * sc_col].
 * Bytes of q between cols and ldq are not written.
 *
 * Returns 0, -i for the first illegal argument (rows = 1, cols = 2, x = 3, x_type = 4, ldx = 5,
 * block_rows = 6, block_cols = 7, format = 8, q = 10, ldq = 11, s = 12, s_row = 13, s_col = 14,
 * qc = 15, ldqc = 16, sc = 17, sc_row = 18, sc_col = 19), or a cudaError_t. */
int f8_quantize(int rows, int cols, const void *x, int x_type, int ldx, int block_rows,
                int block_cols, int format, int pow2, void *q, int ldq, float *s,
                long long s_row, long long s_col, void *qc, int ldqc, float *sc,
                long long sc_row, long long sc_col, cudaStream_t stream);

/* D = alpha * op(A) * op(B) + beta * D with
 *   op(A)(i, k) = qA(i, k) * sA(i / a_rows, k / 128)
 *   op(B)(k, j) = qB(k, j) * sB(k / 128, j / b_cols)
 * and the storage of sgemm_f32_ex: transa = 0: A stored M x K, 1: K x M; transb = 0: B stored
 * K x N, 1: N x K; D is M x N, row-major, of type d_type.
 *   a_rows, b_cols   1 or 128: rows of op(A), columns of op(B) that share a scale
 *   a_scale_mn, a_scale_k   strides of a_scale from one (group of) row(s) of op(A) to the next
 *                    and from one block of k to the next; b_scale_mn, b_scale_k alike for the
 *                    columns of op(B)
 * A and B are 16-byte aligned with leading dimensions that are multiples of 16 (TMA reads them;
 * the padding is not read). Scales may be any numbers up to 2^88 whose products sA * sB are from 2^-126
 * to 2^88, blocks of zeros with any finite scale: beyond that, scaled sums leave the range of FP32 or
 * lose bits although D may hold them.
 *
 * Products of a block are summed by the tensor core in FP32, the blocks in FP32 registers, in an
 * order fixed by the shape: the same call gives the same bits. beta == 0 does not read D;
 * alpha == 0 or K == 0 does not read A, B or their scales. D must not overlap A or B.
 *
 * Returns 0, -i for the first illegal argument in this signature's order (transa = 1, ...,
 * ldd = 24), or a cudaError_t. */
int f8_gemm(int transa, int transb, int M, int N, int K, float alpha, const void *A,
            int a_format, int lda, const float *a_scale, int a_rows, long long a_scale_mn,
            long long a_scale_k, const void *B, int b_format, int ldb, const float *b_scale,
            int b_cols, long long b_scale_mn, long long b_scale_k, float beta, void *D,
            int d_type, int ldd, cudaStream_t stream);

/* The arguments of f8_quantize and of f8_gemm, in their order, as structures: one pointer crosses a
 * language binding faster than 20 to 26 values. */
typedef struct {
  int rows, cols;
  const void *x;
  int x_type, ldx, block_rows, block_cols, format, pow2;
  void *q;
  int ldq;
  float *s;
  long long s_row, s_col;
  void *qc;
  int ldqc;
  float *sc;
  long long sc_row, sc_col;
  cudaStream_t stream;
} f8_quantize_args;

typedef struct {
  int transa, transb, M, N, K;
  float alpha;
  const void *A;
  int a_format, lda;
  const float *a_scale;
  int a_rows;
  long long a_scale_mn, a_scale_k;
  const void *B;
  int b_format, ldb;
  const float *b_scale;
  int b_cols;
  long long b_scale_mn, b_scale_k;
  float beta;
  void *D;
  int d_type, ldd;
  cudaStream_t stream;
} f8_gemm_args;

/* The calls themselves, with the same return codes. `args` is read during the call only. */
int f8_quantize_with(const f8_quantize_args *args);
int f8_gemm_with(const f8_gemm_args *args);

/* How f8_gemm runs a product on a GPU with num_sms SMs (0: the current device; without one a whole
 * GB300). Any pointer may be NULL.
 *   exchanged   1 if the columns of D run along the instruction's 128 rows (few rows in D)
 *   tile_cols   16, 32, 64, 128, or 256 for tiles of 256 x 256 by pairs of blocks
 *   split       blocks that share a tile's sum, each with its part of k
 * Returns 0 or -i for the first illegal argument (M, N and K of 1 or more). */
int f8_gemm_plan(int transa, int transb, int M, int N, int K, int a_rows, int b_cols, int num_sms,
                 int *exchanged, int *tile_cols, int *split);

/* Reads and clears the device status word of f8_gemm (synchronising copy on the legacy stream: wait
 * first for calls on streams that do not wait for it): 0 = fine, 1 - 4 = a wait gave up after about a
 * second and the call's result is not to be used. Returns 0 or a cudaError_t. */
int f8_gemm_status(int *status);

#ifdef __cplusplus
}
#endif
#endif

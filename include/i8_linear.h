/*
 * i8_linear.h -- a linear layer on 8-bit integers with one FP32 scale for each token and each output
 * channel, and the quantiser that makes such operands, for one NVIDIA GB300 (sm_103a), C ABI. Part of
 * the same library as sgemm_f32.h, whose conventions on memory, streams, asynchrony and workspaces
 * hold here too.
 *
 * A quantised matrix is a row-major matrix q of signed bytes (leading dimension ldq) and one FP32
 * scale for each row: element (i, j) stands for q(i, j) * scale(i).
 */
#ifndef I8_LINEAR_H_
#define I8_LINEAR_H_

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st *cudaStream_t;

enum { I8_F32 = 0, I8_BF16 = 1, I8_F16 = 2 }; /* types of x and of D */

/* Quantise each row of x (rows x cols, row-major, leading dimension ldx, type x_type):
 *     a     = max(max |x| along the row, 2^-119)
 *     scale = a / 127                                     (FP32 division)
 *     q     = x * (127 / a) rounded to a whole number     (FP32 division, exact product; nearest,
 *                                                          ties to even): from -127 to 127
 * A row with a NaN or an infinity gets a NaN scale and zeros, so that its products are NaN. Bytes of q
 * between cols and ldq are not written. cols == 0 writes the scales of rows of zeros.
 *
 * Returns 0, -i for the first illegal argument in this signature's order (rows = 1, cols = 2, x = 3,
 * x_type = 4, ldx = 5, q = 6, ldq = 7, scale = 8), or a cudaError_t. x and scale are aligned to their
 * elements. */
int i8_quantize(int rows, int cols, const void *x, int x_type, int ldx, void *q, int ldq, float *scale,
                cudaStream_t stream);

/* D = x w^T with scales, bias and what was there:
 *     D(i, j) = x_scale(i) w_scale(j) sum_k qx(i, k) qw(j, k) + bias(j) + beta D(i, j)
 * x is M x K and w is N x K, both with k contiguous, 16-byte aligned and with leading dimensions that
 * are multiples of 16; the padding is not read. All 256 values of a byte are allowed. bias (N FP32
 * numbers) may be NULL. D is M x N, row-major, of type d_type.
 *
 * The sum over k is the exact whole number (K is at most 131071, so that 32 bits hold it), whatever
 * way the product runs; scales, bias and beta are applied in FP32, with one rounding to d_type. The
 * product of the two scales is formed first: where it leaves FP32's range, so does the result.
 * beta == 0 does not read D; K == 0 does not read x, w or their scales. D must not overlap x or w. D, bias
 * and the scales are aligned to their elements.
 *
 * Returns 0, -i for the first illegal argument in this signature's order (M = 1, N = 2, K = 3, x = 4,
 * ldx = 5, x_scale = 6, w = 7, ldw = 8, w_scale = 9, bias = 10, D = 12, d_type = 13, ldd = 14), or a
 * cudaError_t. */
int i8_linear(int M, int N, int K, const void *x, int ldx, const float *x_scale, const void *w, int ldw,
              const float *w_scale, const float *bias, float beta, void *D, int d_type, int ldd,
              cudaStream_t stream);

/* The arguments of both in their order, as structures: one pointer crosses a language binding faster
 * than 9 to 15 values. */
typedef struct {
  int rows, cols;
  const void *x;
  int x_type, ldx;
  void *q;
  int ldq;
  float *scale;
  cudaStream_t stream;
} i8_quantize_args;

typedef struct {
  int M, N, K;
  const void *x;
  int ldx;
  const float *x_scale;
  const void *w;
  int ldw;
  const float *w_scale, *bias;
  float beta;
  void *D;
  int d_type, ldd;
  cudaStream_t stream;
} i8_linear_args;

/* The calls themselves, with the same return codes (-1 without arguments). `args` is read during the
 * call only. */
int i8_quantize_with(const i8_quantize_args *args);
int i8_linear_with(const i8_linear_args *args);

/* How i8_linear runs a product on a GPU with num_sms SMs (0: the current device; without one a whole
 * GB300). Any pointer may be NULL.
 *   tile_tokens    rows of x per tile: 16, 32, 64 or 128; 0 for the kernel of one or two rows, which has none
 *   tile_channels  rows of w per tile: 128, or 256 where two blocks share a tile (0 as above)
 *   split          blocks that share a tile's sum, each with its part of k
 * Returns 0 or -i for the first illegal argument (M, N and K of 1 or more). */
int i8_linear_plan(int M, int N, int K, int num_sms, int *tile_tokens, int *tile_channels, int *split);

/* Reads and clears the device status word of i8_linear (synchronising copy on the legacy stream: wait
 * first for calls on streams that do not wait for it): 0 = fine, 1 - 4 = a wait gave up after about a
 * second and the call's result is not to be used. Returns 0 or a cudaError_t. */
int i8_linear_status(int *status);

#ifdef __cplusplus
}
#endif
#endif

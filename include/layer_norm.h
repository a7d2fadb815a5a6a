/*
 * layer_norm.h -- layer norm over the rows of a matrix and its gradients for one NVIDIA GB300
 * (sm_103a), C ABI. Part of the same library as sgemm_f32.h, whose conventions on memory, streams,
 * asynchrony and workspaces hold here too.
 */
#ifndef LAYER_NORM_H_
#define LAYER_NORM_H_

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st *cudaStream_t;

enum { LN_F32 = 0, LN_BF16 = 1, LN_F16 = 2 }; /* types of x, y, dy, dx, weight and bias */

/* For each row of x (rows x cols, row-major, leading dimension ldx, type x_type):
 *     mean = sum x / cols,  var = sum (x - mean)^2 / cols,  rstd = 1 / sqrt(var + eps)
 *     y    = (x - mean) rstd weight + bias                    (rounded once, to x_type)
 * weight and bias (cols elements of type w_type each) may be NULL: 1 and 0. mean and rstd (rows FP32
 * numbers each), which layer_norm_backward takes, may be NULL.
 *
 * Sums are FP32 (in rows of more than 16384 elements with 48 bits), in an order fixed by the shape, the type
 * and whether rows are 16-byte aligned: the same call gives the same bits. Where the mean is more than 4 times the
 * spread it is corrected by the mean of the distances from it, so that a spread of a few last places counts and a
 * constant row has its number as the mean and no variance. y takes the mean before its rounding to FP32.
 *
 * Magnitudes up to 2^62 / sqrt(cols) are held (2^50 in rows of up to 2^24 elements): their squares' sum stays in FP32.
 * Where the variance does not, rstd is 0 and y the bias. Downwards the variance and eps together have to be 2^-120 or
 * more, below which squares lose bits: a matter of eps == 0 alone. A NaN or an infinity makes its own row NaN, and so
 * does eps == 0 a constant row, whose rstd is infinite. y may be x itself with ldy = ldx, and must not overlap it
 * otherwise.
 *
 * Returns 0, -i for the first illegal argument in this signature's order (rows = 1 (>= 0), cols = 2
 * (>= 1), x = 3, x_type = 4, ldx = 5, weight = 6, bias = 7, w_type = 8, eps = 9 (>= 0, finite),
 * y = 10, ldy = 11, mean = 12, rstd = 13), or a cudaError_t. Arrays are aligned to their elements. */
int layer_norm(int rows, int cols, const void *x, int x_type, int ldx, const void *weight,
               const void *bias, int w_type, float eps, void *y, int ldy, float *mean, float *rstd,
               cudaStream_t stream);

/* Gradients of layer_norm from that of y (dy; dy and dx have x's type), with h = (x - mean) rstd and
 * g = dy weight:
 *     dx      = rstd (g - sum g / cols - h sum (g h) / cols)     along each row
 *     dweight = sum over the rows of dy h + beta dweight         (cols FP32 numbers)
 *     dbias   = sum over the rows of dy   + beta dbias           (cols FP32 numbers)
 * weight may be NULL (1), and so may dx, dweight and dbias, each of which is then left out. beta == 0
 * does not read dweight and dbias; with rows == 0 they become beta times themselves. dx may be dy or
 * x itself with the same leading dimension, and must not overlap them otherwise.
 *
 * Sums along rows are FP32 (with 48 bits in rows of more than 12288 elements, or of more than 16384 where they
 * are of 16 bits and 16-byte aligned), those over the rows FP32 within a block (at most 500 rows one after the
 * other) and 64-bit beyond, in an order fixed by the shape, the type, that alignment and the device: the same call
 * gives the same bits. The mean is the FP32 number that is given: where a spread is few of its last places, h carries
 * its rounding. The workspace (layer_norm_backward_workspace_size bytes at most) is a stream-ordered allocation from
 * the library's pool.
 *
 * Returns 0, -i for the first illegal argument in this signature's order (rows = 1 (>= 0), cols = 2
 * (>= 1), dy = 3, lddy = 4, x = 5, x_type = 6, ldx = 7, mean = 8, rstd = 9, weight = 10, w_type = 11,
 * dx = 12, lddx = 13, dweight = 14, dbias = 15), or a cudaError_t. Arrays are aligned to their elements. */
int layer_norm_backward(int rows, int cols, const void *dy, int lddy, const void *x, int x_type,
                        int ldx, const float *mean, const float *rstd, const void *weight,
                        int w_type, void *dx, int lddx, float *dweight, float *dbias, float beta,
                        cudaStream_t stream);

/* Bytes of workspace that layer_norm_backward takes at most from the library's pool on the current device
 * (without one: on a whole GB300); FP32 rows that are not 16-byte aligned take the most. Returns 0 or -1, -2 for an
 * illegal rows, cols. */
int layer_norm_backward_workspace_size(int rows, int cols, size_t *bytes);

/* The arguments of both in their order, as structures: one pointer crosses a language binding faster
 * than 14 to 17 values. */
typedef struct {
  int rows, cols;
  const void *x;
  int x_type, ldx;
  const void *weight, *bias;
  int w_type;
  float eps;
  void *y;
  int ldy;
  float *mean, *rstd;
  cudaStream_t stream;
} layer_norm_args;

typedef struct {
  int rows, cols;
  const void *dy;
  int lddy;
  const void *x;
  int x_type, ldx;
  const float *mean, *rstd;
  const void *weight;
  int w_type;
  void *dx;
  int lddx;
  float *dweight, *dbias;
  float beta;
  cudaStream_t stream;
} layer_norm_backward_args;

/* The calls themselves, with the same return codes (-1 without arguments). `args` is read during the
 * call only. */
int layer_norm_with(const layer_norm_args *args);
int layer_norm_backward_with(const layer_norm_backward_args *args);

#ifdef __cplusplus
}
#endif
#endif

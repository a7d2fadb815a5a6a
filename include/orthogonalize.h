/*
 * orthogonalize.h -- orthogonalising a matrix by Newton-Schulz products for one NVIDIA GB300
 * (sm_103a), C ABI. Part of the same library as sgemm_f32.h, whose conventions on memory,
 * streams, asynchrony and workspaces hold here too.
 */
#ifndef ORTHOGONALIZE_H_
#define ORTHOGONALIZE_H_

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st *cudaStream_t;

enum { NS_F32 = 0, NS_BF16 = 1, NS_F16 = 2 }; /* types of G and of out */

/* For each of `batch` matrices G (rows x cols, row-major, leading dimension ldg, the next one
 * g_stride elements further):
 *     X_0 = G / (|G|_F + eps)
 *     X_{t+1} = a X_t + (b S + c S^2) X_t,  S = X_t X_t^T   (rows <= cols; else the same on the
 *                                                            transposed matrix)
 *     out = alpha X_steps + beta out
 * coefficients = {a, b, c}, the same in every step, read by the host during the call. With those
 * of a Newton-Schulz iteration X tends to the orthogonal factor U V^T of G = U s V^T.
 *
 * All products run on the tensor cores in FP32 fidelity: every factor is the sum of two FP16
 * numbers (22 bits) under a power-of-two scale that the host derives from the coefficients, and
 * sums are FP32. There is one rounding to out's type, at the end. The order of every sum is
 * fixed by the shape: the same call gives the same bits.
 *
 * G is not changed (out may be G itself when type and strides are the same). beta == 0 does not
 * read out. A zero matrix gives zeros. A NaN or an infinity in a matrix makes its result NaN and
 * leaves the other matrices of the batch alone.
 *
 * The workspace (ns_orthogonalize_workspace_size bytes) is a stream-ordered allocation from the
 * library's pool.
 *
 * Returns 0, -i for the first illegal argument (batch = 1, rows = 2, cols = 3, G = 4, g_type = 5,
 * ldg = 6, g_stride = 7, steps = 8 (0 .. 64), coefficients = 9 (not NULL, finite, and such that
 * |X| stays below 2^60), eps = 10 (>= 0), out = 13, out_type = 14, ldo = 15, o_stride = 16), or a
 * cudaError_t. */
int ns_orthogonalize(int batch, int rows, int cols, const void *G, int g_type, int ldg,
                     long long g_stride, int steps, const float *coefficients, float eps,
                     float alpha, float beta, void *out, int out_type, int ldo,
                     long long o_stride, cudaStream_t stream);

/* Bytes of workspace that the call takes from the library's pool on the current device (without
 * one: on a whole GB300). Returns 0 or -1, -2, -3 for a negative batch, rows or cols. */
int ns_orthogonalize_workspace_size(int batch, int rows, int cols, size_t *bytes);

/* How ns_orthogonalize runs a problem on a GPU with num_sms SMs (0: the current device; without one a
 * whole GB300). Any pointer may be NULL.
 *   tile_cols   64 or 128 (tiles of 128 rows), or 256 for tiles of 256 x 256 by pairs of blocks
 *   tiles, whole, split   for each of the three products of a step (X X^T, S S, R X): its tiles in the
 *               whole batch, how many of them are computed in one piece, and in how many parts along k
 *               the others are (1 if there are none)
 * Returns 0, -i for the first illegal argument (sizes of 1 or more), or a cudaError_t. */
int ns_orthogonalize_plan(int batch, int rows, int cols, int num_sms, int *tile_cols, int tiles[3],
                          int whole[3], int split[3]);

/* Reads and clears the device status word of ns_orthogonalize (synchronising copy on the legacy
 * stream: wait first for calls on streams that do not wait for it): 0 = fine, 1 - 4 = a wait gave up
 * and the call's result is not to be used. A wait gives up after about a second where
 * it is for a block's own copies and instructions, and after eight to ten where it depends on the
 * other blocks. Returns 0 or a cudaError_t. */
int ns_orthogonalize_status(int *status);

#ifdef __cplusplus
}
#endif
#endif

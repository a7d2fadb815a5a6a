/*
 * grad_clip.h -- the norm of all gradients together, and clipping them by it, for one NVIDIA GB300
 * (sm_103a), C ABI. Part of the same library as sgemm_f32.h, whose conventions on memory, streams,
 * asynchrony and workspaces hold here too.
 */
#ifndef GRAD_CLIP_H_
#define GRAD_CLIP_H_

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st *cudaStream_t;

enum { GC_F32 = 0, GC_BF16 = 1, GC_F16 = 2 }; /* types of gradients and results */

/* Of `count` arrays, the i-th of sizes[i] elements of type types[i] at grads[i]:
 *     norm   = sqrt(sum of squares of all elements)
 *     factor = min(1, max_norm / (norm + eps))               (64 bits, rounded once to FP32)
 *     out[i] = grads[i] * factor                              (FP32, rounded once to out_types[i])
 * The lists are read by the host during the call; the arrays are device memory, aligned to their
 * elements. norm (one FP32 number in device memory) may be NULL. out == NULL leaves the second part
 * out. out[i] may be grads[i] itself with the same type (in place; a factor of 1 then writes
 * nothing); apart from that no result may overlap a gradient or another result.
 *
 * Squares are summed in FP32, 64 of them at a time, and those sums in 64 bits; arrays whose squares
 * leave FP32's range are scaled. So all finite gradients are handled, and a norm beyond FP32 is
 * written as infinity while its factor is still right. The order is fixed by the sizes and the device: the
 * same call gives the same bits. An infinity among the gradients makes the norm infinite and the
 * factor 0 (the infinite elements become NaN), a NaN makes both NaN. max_norm may be infinite (only
 * the norm is of interest, or elements are converted; an infinite norm then gives NaN).
 *
 * The workspace is a stream-ordered allocation from the library's pool.
 *
 * Returns 0, -i for the first illegal argument (count = 1, grads = 2, types = 3, sizes = 4, max_norm =
 * 5 (>= 0), eps = 6 (>= 0, finite), out = 7 (entries, their alignment and overlaps), out_types = 8,
 * norm = 9 (aligned)), or a cudaError_t. */
int clip_grad_norm(int count, const void *const *grads, const int *types, const long long *sizes,
                   double max_norm, double eps, void *const *out, const int *out_types, float *norm,
                   cudaStream_t stream);

#ifdef __cplusplus
}
#endif
#endif

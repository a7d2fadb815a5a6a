// What the operators on whole rows share (layer norm, its gradients, the quantiser to 8-bit
// integers): a row of up to 16384 elements lies in the registers of 8 to 1024 neighbouring threads,
// packed as it was loaded, in chunks of 8 elements per thread.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "sgemm_ffma.cuh"
#include "sgemm_internal.h"
#include "sgemm_plan.h"
#include "tc_common.cuh"

namespace sgemm {
namespace rows {

// Types of elements: W words hold 8 of them; value(): number n of a word as FP32; pack(): numbers
// rounded once, to nearest even.
struct F32 {
  static constexpr int W = 8, SIZE = 4, TYPE = tcx::OUT_F32;
  static __device__ __forceinline__ float value(uint32_t w, int) { return __uint_as_float(w); }
};
struct BF16 {
  static constexpr int W = 4, SIZE = 2, TYPE = tcx::OUT_BF16;
  static __device__ __forceinline__ float value(uint32_t w, int n) {
    return __uint_as_float(n ? w & 0xffff0000u : w << 16);
  }
};
struct F16 {
  static constexpr int W = 4, SIZE = 2, TYPE = tcx::OUT_F16;
  static __device__ __forceinline__ float value(uint32_t w, int n) {
    return __half2float(__ushort_as_half((unsigned short)(n ? w >> 16 : w & 0xffffu)));
  }
};

template <class T>
struct Chunk {
  uint32_t w[T::W];
  __device__ __forceinline__ float operator[](int j) const {
    return T::W == 8 ? T::value(w[j % T::W], 0) : T::value(w[j / 2], j & 1);
  }
};

template <class T>
__device__ __forceinline__ void pack(const float (&v)[8], Chunk<T> &c) {
  if constexpr (T::W == 8) {
#pragma unroll
    for (int j = 0; j < 8; ++j) c.w[j] = __float_as_uint(v[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) c.w[j] = tcx::pack_out(T::TYPE, v[2 * j], v[2 * j + 1]);
  }
}

// How TPR threads share a row: chunk c of thread t holds, with VEC (rows are 16-byte aligned), 8
// neighbouring elements, else elements that are TPR apart, so that a warp reads neighbours either
// way. Of a chunk's elements the first count() exist.
template <int TPR, bool VEC>
struct Share {
  int cols, t;
  __device__ __forceinline__ int col(int c, int j) const {
    return VEC ? (c * TPR + t) * 8 + j : (c * 8 + j) * TPR + t;
  }
  __device__ __forceinline__ int count(int c) const {
    const int n = VEC ? cols - col(c, 0) : (cols - col(c, 0) + TPR - 1) / TPR;
    return n < 0 ? 0 : n > 8 ? 8 : n;
  }
  // Elements that do not exist are zero.
  template <class T>
  __device__ __forceinline__ void load(const void *row, int c, int n, Chunk<T> &v) const {
    const char *src = reinterpret_cast<const char *>(row);
    if (VEC && n == 8) {
      const uint4 *s = reinterpret_cast<const uint4 *>(src + (long long)col(c, 0) * T::SIZE);
#pragma unroll
      for (int i = 0; i < T::W; i += 4) {
        const uint4 u = __ldcs(s + i / 4);
        v.w[i] = u.x, v.w[i + 1] = u.y, v.w[i + 2] = u.z, v.w[i + 3] = u.w;
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < T::W; ++i) v.w[i] = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) {
        const int at = col(c, j);
        if (T::W == 8)
          v.w[j % T::W] = __ldcs(reinterpret_cast<const uint32_t *>(src) + at);
        else
          v.w[j / 2] |= (uint32_t)__ldcs(reinterpret_cast<const uint16_t *>(src) + at) << (16 * (j & 1));
      }
  }
  template <class T>
  __device__ __forceinline__ void store(void *row, int c, int n, const Chunk<T> &v) const {
    char *dst = reinterpret_cast<char *>(row);
    if (VEC && n == 8) {
      uint4 *d = reinterpret_cast<uint4 *>(dst + (long long)col(c, 0) * T::SIZE);
#pragma unroll
      for (int i = 0; i < T::W; i += 4) d[i / 4] = make_uint4(v.w[i], v.w[i + 1], v.w[i + 2], v.w[i + 3]);
      return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) {
        const int at = col(c, j);
        if (T::W == 8)
          reinterpret_cast<uint32_t *>(dst)[at] = v.w[j % T::W];
        else
          reinterpret_cast<uint16_t *>(dst)[at] = (uint16_t)(v.w[j / 2] >> (16 * (j & 1)));
      }
  }
};

// A vector of parameters (a weight, a bias) in any of the types; 1 or 0 where there is none.
struct Vector {
  const void *ptr;
  int type;
  __device__ __forceinline__ float at(int i, float otherwise) const {
    return ptr ? tcx::load_out(ptr, type, i) : otherwise;
  }
};

// Sums over the TPR threads of a row, the same bits in each of them. `turn` alternates between calls
// of a kernel, so that one barrier is enough: whoever writes a buffer again has passed the barrier
// of the call in between, before which everybody had read it.
template <int TPR>
__device__ __forceinline__ float2 row_sum(float2 v, float2 (*part)[32], int turn) {
#pragma unroll
  for (int d = 1; d < (TPR < 32 ? TPR : 32); d *= 2) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, d);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, d);
  }
  if constexpr (TPR > 32) {
    if ((threadIdx.x & 31) == 0) part[turn][threadIdx.x >> 5] = v;
    __syncthreads();
    v = part[turn][0];
#pragma unroll
    for (int w = 1; w < TPR / 32; ++w) {
      const float2 u = part[turn][w];
      v.x += u.x;
      v.y += u.y;
    }
  }
  return v;
}

// Threads per row and chunks per thread for rows of `cols` elements; 8 chunks' worth more would spill.
struct Layout {
  int tpr, chunks;
};
constexpr int kLongest = 16384;  // elements of a row that stays in registers

constexpr bool aligned(uintptr_t ptr, long long ld_bytes) { return ptr % 16 == 0 && ld_bytes % 16 == 0; }

}  // namespace rows
}  // namespace sgemm

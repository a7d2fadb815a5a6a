// Quantiser of the 8-bit block-scaled product: for each block b of x
//   s_b = max(max |x| / F, 2^-126), q = round(x / s_b)
// with blocks of 1 x 128, 128 x 1, 128 x 128, or the first two at once from one read.
//
// Bound by HBM: sizeof(x) bytes in and one byte (two for the pair) out for each element.
//  * rows_kernel (1 x 128): 16 lanes hold one block, 8 neighbouring elements each, so a block's
//    maximum is four shuffles; a warp holds U blocks per half, all reads issued first.
//  * tile_kernel (the other layouts): a CTA of 256 threads holds a 128 x 128 tile in registers,
//    64 elements per thread (8 rows of 8 neighbouring columns); row maxima are shuffles, column
//    maxima and the tile's maximum meet in shared memory.
// Maxima are taken on the bits of |x| as integers, whose order is that of the numbers with
// infinity and then NaN on top, so that neither is lost.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/f8_gemm.h"
#include "sgemm_ffma.cuh"
#include "sgemm_internal.h"
#include "sgemm_plan.h"

namespace sgemm {
namespace f8 {

struct Result {
  uint8_t *q;
  long long ldq;
  float *s;
  long long s_row, s_col;
  int vec;             // 8-byte stores to q are aligned
};

struct QuantParams {
  int rows, cols;
  const void *x;
  long long ldx;
  int vec;             // 16-byte loads of x are aligned
  int format, pow2;
  Result a, c;         // a: rows or the only result; c: columns
};

// Eight neighbouring elements of row r from column c, as FP32 (0 out of range).
template <class T>
__device__ __forceinline__ void load8(const QuantParams &p, int r, int c, float (&v)[8]) {
  const T *src = reinterpret_cast<const T *>(p.x) + r * p.ldx + c;
  if (r < p.rows && p.vec && c + 8 <= p.cols) {
    if constexpr (sizeof(T) == 4) {
      const float4 a = __ldcs(reinterpret_cast<const float4 *>(src));
      const float4 b = __ldcs(reinterpret_cast<const float4 *>(src) + 1);
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
      v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
      const uint4 u = __ldcs(reinterpret_cast<const uint4 *>(src));
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float2 f;
        if constexpr (sizeof(T) == 2 && T::is_bf16)
          f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w[j]));
        else
          f = __half22float2(*reinterpret_cast<const __half2 *>(&w[j]));
        v[2 * j] = f.x;
        v[2 * j + 1] = f.y;
      }
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    v[j] = 0.0f;
    if (r < p.rows && c + j < p.cols) v[j] = src[j].value();
  }
}

struct F32 {
  float f;
  static constexpr bool is_bf16 = false;
  __device__ float value() const { return f; }
};
struct BF16 {
  __nv_bfloat16 f;
  static constexpr bool is_bf16 = true;
  __device__ float value() const { return __bfloat162float(f); }
};
struct F16 {
  __half f;
  static constexpr bool is_bf16 = false;
  __device__ float value() const { return __half2float(f); }
};

__device__ __forceinline__ uint32_t bits_abs(float x) { return __float_as_uint(x) & 0x7fffffffu; }

__device__ __forceinline__ uint32_t max8(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = max(m, bits_abs(v[j]));
  return m;
}

__device__ __forceinline__ float scale_of(uint32_t amax, int format, int pow2) {
  const uint32_t least = 0x00800000u;  // 2^-126
  uint32_t s = __float_as_uint(__fdiv_rn(__uint_as_float(amax), format ? 57344.0f : 448.0f));
  s = max(s, least);                   // (positive, infinite or NaN: ordered as integers)
  if (pow2 && s < 0x7f800000u) s = (s + 0x007fffffu) & 0xff800000u;
  return __uint_as_float(s);
}

// Two numbers to two bytes, nearest with ties to even, limited to the largest finite number;
// NaN stays NaN. The first number goes to the low byte.
__device__ __forceinline__ uint32_t round2(float lo, float hi, int format) {
  uint16_t r;
  if (format)
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;\n" : "=h"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ void store8(const Result &o, const QuantParams &p, int r, int c,
                                       const float (&y)[8]) {
  if (r >= p.rows || c >= p.cols) return;
  uint2 w;
  w.x = round2(y[0], y[1], p.format) | round2(y[2], y[3], p.format) << 16;
  w.y = round2(y[4], y[5], p.format) | round2(y[6], y[7], p.format) << 16;
  uint8_t *dst = o.q + r * o.ldq + c;
  if (o.vec && c + 8 <= p.cols) {
    *reinterpret_cast<uint2 *>(dst) = w;
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (c + j < p.cols) dst[j] = (uint8_t)((j < 4 ? w.x >> (8 * j) : w.y >> (8 * j - 32)) & 0xff);
}

// Maximum over the 16 lanes of a half-warp.
__device__ __forceinline__ uint32_t half_max(uint32_t m) {
#pragma unroll
  for (int d = 1; d < 16; d *= 2) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
  return m;
}

// 1 x 128 blocks: unit u = row * blocks + block, 2 U units per warp.
template <class T, int U>
__global__ void __launch_bounds__(256) rows_kernel(const QuantParams p) {
  griddep_wait();  // (launched with programmatic dependent launch: see launch_1d)
  const int lane = threadIdx.x & 31, sub = lane & 15, half = lane >> 4;
  const int blocks = (p.cols + 127) / 128;
  const long long units = (long long)p.rows * blocks;
  const long long warps = (long long)gridDim.x * 8;
  const long long w0 = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  for (long long u0 = w0 * 2 * U; u0 < units; u0 += warps * 2 * U) {
    float v[U][8];
    int r[U], c[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const long long u = u0 + 2 * i + half;
      r[i] = u < units ? (int)(u / blocks) : p.rows;
      c[i] = (int)(u % blocks) * 128 + sub * 8;
      load8<T>(p, r[i], c[i], v[i]);
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const float s = scale_of(half_max(max8(v[i])), p.format, p.pow2);
      if (sub == 0 && r[i] < p.rows) p.a.s[r[i] * p.a.s_row + (c[i] >> 7) * p.a.s_col] = s;
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = __fdiv_rn(v[i][j], s);
      store8(p.a, p, r[i], c[i], v[i]);
    }
  }
  griddep_launch_dependents();
}

enum { COLS = 0, SQUARE = 1, PAIR = 2 };

// One 128 x 128 tile per CTA: thread (g = tid / 16, sub = tid % 16) holds columns 8 sub .. + 7 of
// rows g, g + 16, ..., g + 112.
template <class T, int WHICH>
__global__ void __launch_bounds__(256) tile_kernel(const QuantParams p, int tiles_c) {
  griddep_wait();
  __shared__ uint32_t top[8][128];
  __shared__ float scale[128];
  const int tid = threadIdx.x, sub = tid & 15, g = tid >> 4, warp = tid >> 5;
  const int br = blockIdx.x / tiles_c, bc = blockIdx.x % tiles_c;
  const int r0 = br * 128 + g, c0 = bc * 128 + sub * 8;
  float v[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) load8<T>(p, r0 + 16 * i, c0, v[i]);

  if constexpr (WHICH == SQUARE) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, max8(v[i]));
    m = __reduce_max_sync(0xffffffffu, m);
    if ((tid & 31) == 0) top[0][warp] = m;
    __syncthreads();
    m = top[0][0];
#pragma unroll
    for (int w = 1; w < 8; ++w) m = max(m, top[0][w]);
    const float s = scale_of(m, p.format, p.pow2);
    if (tid == 0) p.a.s[br * p.a.s_row + bc * p.a.s_col] = s;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = __fdiv_rn(v[i][j], s);
      store8(p.a, p, r0 + 16 * i, c0, v[i]);
    }
  } else {
    const Result &o = WHICH == PAIR ? p.c : p.a;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, bits_abs(v[i][j]));
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 16));
      if ((tid & 16) == 0) top[warp][sub * 8 + j] = m;
    }
    __syncthreads();
    if (tid < 128) {
      uint32_t m = top[0][tid];
#pragma unroll
      for (int w = 1; w < 8; ++w) m = max(m, top[w][tid]);
      const float s = scale_of(m, p.format, p.pow2);
      scale[tid] = s;
      const int c = bc * 128 + tid;
      if (c < p.cols) o.s[br * o.s_row + c * o.s_col] = s;
    }
    __syncthreads();
    float sc[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) sc[j] = scale[sub * 8 + j];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = __fdiv_rn(v[i][j], sc[j]);
      store8(o, p, r0 + 16 * i, c0, y);
    }
    if constexpr (WHICH == PAIR) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = r0 + 16 * i;
        const float s = scale_of(half_max(max8(v[i])), p.format, p.pow2);
        if (sub == 0 && r < p.rows) p.a.s[r * p.a.s_row + bc * p.a.s_col] = s;
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = __fdiv_rn(v[i][j], s);
        store8(p.a, p, r, c0, v[i]);
      }
    }
  }
  griddep_launch_dependents();
}

template <class T>
static cudaError_t launch_quantize(const QuantParams &p, int which, int sms, cudaStream_t stream) {
  if (which < 0) {
    const long long units = (long long)p.rows * ceil_div(p.cols, 128);
    // two blocks in flight per half-warp once every SM has several warps of work
    if (units >= 4LL * 8 * 8 * sms) {
      const long long grid = std::min<long long>(ceil_div(units, 8 * 4), 8LL * sms);
      return launch_1d(rows_kernel<T, 2>, (int)grid, 256, 0, 1, stream, p);
    }
    return launch_1d(rows_kernel<T, 1>, (int)ceil_div(units, 8 * 2), 256, 0, 1, stream, p);
  }
  const int tiles_c = (int)ceil_div(p.cols, 128);
  const long long tiles = (long long)tiles_c * ceil_div(p.rows, 128);
  if (tiles > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  if (which == SQUARE)
    return launch_1d(tile_kernel<T, SQUARE>, (int)tiles, 256, 0, 1, stream, p, tiles_c);
  if (which == COLS)
    return launch_1d(tile_kernel<T, COLS>, (int)tiles, 256, 0, 1, stream, p, tiles_c);
  return launch_1d(tile_kernel<T, PAIR>, (int)tiles, 256, 0, 1, stream, p, tiles_c);
}

}  // namespace f8
}  // namespace sgemm

using namespace sgemm;

extern "C" int f8_quantize(int rows, int cols, const void *x, int x_type, int ldx, int block_rows,
                           int block_cols, int format, int pow2, void *q, int ldq, float *s,
                           long long s_row, long long s_col, void *qc, int ldqc, float *sc,
                           long long sc_row, long long sc_col, cudaStream_t stream) {
  const bool any = rows > 0 && cols > 0;
  if (rows < 0) return -1;
  if (cols < 0) return -2;
  if (any && x == nullptr) return -3;
  if (x_type != F8_D_F32 && x_type != F8_D_BF16 && x_type != F8_D_F16) return -4;
  const int size = x_type == F8_D_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(x) % size != 0) return -3;
  if (ldx < std::max(1, cols)) return -5;
  if (block_rows != 1 && block_rows != 128) return -6;
  if ((block_cols != 1 && block_cols != 128) || (block_rows == 1 && block_cols == 1)) return -7;
  if (format != F8_E4M3 && format != F8_E5M2) return -8;
  if (any && q == nullptr) return -10;
  if (ldq < std::max(1, cols)) return -11;
  if (any && s == nullptr) return -12;
  if (s_row < 0) return -13;
  if (s_col < 0) return -14;
  if (qc != nullptr) {
    if (block_rows != 1) return -15;
    if (ldqc < std::max(1, cols)) return -16;
    if (any && sc == nullptr) return -17;
    if (sc_row < 0) return -18;
    if (sc_col < 0) return -19;
  }
  if (!any) return 0;
  int sms = 0;
  cudaError_t e = device_setup(&sms);
  if (e != cudaSuccess) return (int)e;
  const auto aligned = [](const void *ptr, long long ld_bytes, unsigned to) {
    return reinterpret_cast<uintptr_t>(ptr) % to == 0 && ld_bytes % to == 0;
  };
  f8::QuantParams p{};
  p.rows = rows;
  p.cols = cols;
  p.x = x;
  p.ldx = ldx;
  p.vec = aligned(x, (long long)ldx * size, 16);
  p.format = format;
  p.pow2 = pow2 != 0;
  p.a = f8::Result{static_cast<uint8_t *>(q), ldq, s, s_row, s_col, aligned(q, ldq, 8)};
  p.c = f8::Result{static_cast<uint8_t *>(qc), ldqc, sc, sc_row, sc_col, aligned(qc, ldqc, 8)};
  const int which = qc != nullptr ? f8::PAIR
                    : block_rows == 1 ? -1
                    : block_cols == 1 ? f8::COLS
                                      : f8::SQUARE;
  if (x_type == F8_D_F32) return (int)f8::launch_quantize<f8::F32>(p, which, sms, stream);
  if (x_type == F8_D_BF16) return (int)f8::launch_quantize<f8::BF16>(p, which, sms, stream);
  return (int)f8::launch_quantize<f8::F16>(p, which, sms, stream);
}

// Quantiser of the 8-bit block-scaled product: for each block b of x
//   s_b = max(max |x| / F, 2^-126), q = round(x / s_b)
// with blocks of 1 x 128, 128 x 1, 128 x 128, or the first two at once from one read.
//
// Bound by HBM: sizeof(x) bytes in and one byte (two for the pair) out for each element. What
// stands in the way is arithmetic, so there is little of it per element:
//  * x stays packed in registers as it was loaded, 16 neighbouring elements per thread, which
//    spreads the work on a scale over many of them. Maxima of magnitudes are one instruction for
//    two 16-bit numbers; NaN wins over everything, so that it is not lost.
//  * No division per element. With r = 1 / s to 2^-23 the product y = x r is within 2^-22 of
//    x / s. Let m be y rounded to 5 significant bits: every tie of the 8-bit formats is such a
//    number. The remainder x - m s is exact in one FMA, and m + (x - m s) r is x / s corrected by
//    one step of Markstein's remainder iteration: exact next to a tie, where m is the tie and the
//    remainder tiny, and within an FP32 rounding elsewhere, where nothing depends on it. So q is
//    what the correctly rounded FP32 quotient gives, for three packed FP32 instructions per two
//    elements. m s has bits down to 2^-33 s (e4m3; 2^-40 s for e5m2), which FP32 no longer holds for
//    s under 2^-116 (2^-109): blocks with s under 2^-100 are computed from 2^64 x and 2^64 s.
//  * rows_kernel (1 x 128): 8 lanes hold one block, so a block's maximum is three shuffles.
//  * tile_kernel (the other layouts): a CTA holds a 128 x 128 tile in registers, 32 of them per
//    thread; row maxima are shuffles, column maxima and the tile's maximum meet in shared memory.
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
  int vec;             // 16-byte stores to q are aligned
};

struct QuantParams {
  int rows, cols;
  const void *x;
  long long ldx;
  int vec;             // 16-byte loads of x are aligned
  int format, pow2;
  Result a, c;         // a: rows or the only result; c: columns
};

// Types of x: 16 neighbouring elements are W words. larger(): the larger magnitudes of two words
// (with either sign; NaN over all); top(): the largest magnitude in a word, and value(): number n
// of a word, as FP32; scaled(): a word's numbers times powers of two whose results the type holds.
// SMALL: scales under kSmallScale occur. CTAS: of rows_kernel per SM, for the registers, where the
// compiler alone takes too many (BF16 with 37 for 31: 18.0 us, not 17.0, for 8192 x 4096); 0: it does not.
struct F32 {
  static constexpr int W = 16, CTAS = 0;
  static constexpr bool SMALL = true;
  static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
    uint32_t m;
    asm("max.NaN.xorsign.abs.f32 %0, %1, %2;\n" : "=r"(m) : "r"(a), "r"(b));
    return m;
  }
  static __device__ __forceinline__ float top(uint32_t w) { return fabsf(__uint_as_float(w)); }
  static __device__ __forceinline__ float value(uint32_t w, int) { return __uint_as_float(w); }
  static __device__ __forceinline__ uint32_t scaled(uint32_t w, float f, float) {
    return __float_as_uint(__uint_as_float(w) * f);
  }
};
struct BF16 {
  static constexpr int W = 8, CTAS = 8;
  static constexpr bool SMALL = true;
  static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
    uint32_t m;
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;\n" : "=r"(m) : "r"(a), "r"(b));
    return m;
  }
  static __device__ __forceinline__ float top(uint32_t w) {
    w &= 0x7fff7fffu;
    return __uint_as_float(max(w & 0xffff0000u, w << 16));
  }
  static __device__ __forceinline__ float value(uint32_t w, int n) {
    return __uint_as_float(n ? w & 0xffff0000u : w << 16);
  }
  static __device__ __forceinline__ uint32_t scaled(uint32_t w, float lo, float hi) {
    return __float_as_uint(value(w, 0) * lo) >> 16 |
           (__float_as_uint(value(w, 1) * hi) & 0xffff0000u);  // (a NaN has bits below, too)
  }
};
struct F16 {
  static constexpr int W = 8, CTAS = 0;
  static constexpr bool SMALL = false;  // (its smallest number is 2^-24)
  static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
    uint32_t m;
    asm("max.NaN.xorsign.abs.f16x2 %0, %1, %2;\n" : "=r"(m) : "r"(a), "r"(b));
    return m;
  }
  static __device__ __forceinline__ float top(uint32_t w) {
    w &= 0x7fff7fffu;
    return __half2float(__ushort_as_half((unsigned short)max(w >> 16, w & 0xffffu)));
  }
  static __device__ __forceinline__ float value(uint32_t w, int n) {
    return __half2float(__ushort_as_half((unsigned short)(n ? w >> 16 : w & 0xffffu)));
  }
};

template <class T>
struct Sixteen {
  uint32_t w[T::W];
};

// Element j (0 .. 15).
template <class T>
__device__ __forceinline__ float at(const Sixteen<T> &v, int j) {
  return T::W == 16 ? T::value(v.w[j], 0) : T::value(v.w[j / 2], j & 1);
}

// n of 16 neighbouring elements from src (0 for the others).
template <class T>
__device__ __forceinline__ void load16(const char *src, bool vec, int n, Sixteen<T> &v) {
  if (vec && n >= 16) {
#pragma unroll
    for (int i = 0; i < T::W; i += 4) {
      const uint4 u = __ldcs(reinterpret_cast<const uint4 *>(src) + i / 4);
      v.w[i] = u.x, v.w[i + 1] = u.y, v.w[i + 2] = u.z, v.w[i + 3] = u.w;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < T::W; ++i) v.w[i] = 0;
#pragma unroll
  for (int j = 0; j < 16; ++j)
    if (j < n) {
      if (T::W == 16)
        v.w[j % T::W] = reinterpret_cast<const uint32_t *>(src)[j];
      else
        v.w[j / 2] |= (uint32_t)reinterpret_cast<const uint16_t *>(src)[j] << (16 * (j & 1));
    }
}

template <class T>
__device__ __forceinline__ uint32_t max16(const Sixteen<T> &v) {
  uint32_t m = v.w[0];
#pragma unroll
  for (int i = 1; i < T::W; ++i) m = T::larger(m, v.w[i]);
  return m;
}

// A block's scale, and what its elements are multiplied with: r = 1 / s and -s.
struct Scale {
  float s, r, minus;
};
constexpr float kSmallScale = 0x1p-100f, kUp = 0x1p64f, kDown = 0x1p-64f;

__device__ __forceinline__ Scale scale_of(float amax, int format, int pow2) {
  const uint32_t least = 0x00800000u, inf = 0x7f800000u;  // 2^-126
  uint32_t b = __float_as_uint(__fdiv_rn(amax, format ? 57344.0f : 448.0f));
  b = max(b, least);                   // (positive, infinite or NaN: ordered as integers)
  if (pow2 && b < inf) b = (b + 0x007fffffu) & 0xff800000u;
  Scale o;
  o.s = __uint_as_float(b);
  if (pow2 && b < inf)
    o.r = __uint_as_float(0x7f000000u - b);  // (an amax is under 2^128: b < 2^120)
  else
    asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(o.r) : "f"(o.s));
  // an infinite or NaN scale takes no part in the remainder: r = 0 or NaN decides alone
  o.minus = b < inf ? -o.s : 0.0f;
  return o;
}

// Two numbers to two bytes, nearest with ties to even, limited to the largest finite number;
// NaN stays NaN. The first number goes to the low byte.
template <int FORMAT>
__device__ __forceinline__ uint32_t round2(float lo, float hi) {
  uint16_t r;
  if (FORMAT)
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;\n" : "=h"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// q of two elements; r, minus: both elements' factors.
template <int FORMAT>
__device__ __forceinline__ uint32_t quantize2(float x0, float x1, unsigned long long r,
                                              unsigned long long minus) {
  const unsigned long long x = pack2(x0, x1);
  unsigned long long y, rest;
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(y) : "l"(x), "l"(r));
  const float2 v = unpack2(y);
  const unsigned long long m =
      pack2(__uint_as_float((__float_as_uint(v.x) + 0x40000u) & 0xfff80000u),
            __uint_as_float((__float_as_uint(v.y) + 0x40000u) & 0xfff80000u));
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(rest) : "l"(m), "l"(minus), "l"(x));
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(y) : "l"(rest), "l"(r), "l"(m));
  const float2 t = unpack2(y);
  return round2<FORMAT>(t.x, t.y);
}

template <class T, int FORMAT>
__device__ __forceinline__ uint4 quantize16(const Sixteen<T> &v, const Scale &s) {
  uint32_t w[4];
  const unsigned long long r = pack2(s.r, s.r), minus = pack2(s.minus, s.minus);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = quantize2<FORMAT>(at<T>(v, 4 * i), at<T>(v, 4 * i + 1), r, minus) |
           quantize2<FORMAT>(at<T>(v, 4 * i + 2), at<T>(v, 4 * i + 3), r, minus) << 16;
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// A small scale's factors for 2^64 x.
__device__ __forceinline__ void raise(Scale &s) {
  s.r *= kDown;
  s.minus *= kUp;
}

// v times f, a power of two (exact).
template <class T>
__device__ __forceinline__ void scale16(Sixteen<T> &v, float f) {
#pragma unroll
  for (int i = 0; i < T::W; ++i) v.w[i] = T::scaled(v.w[i], f, f);
}

// The first n of 16 bytes.
__device__ __forceinline__ void store16(uint8_t *dst, bool vec, int n, const uint4 &w) {
  if (vec && n >= 16) {
    *reinterpret_cast<uint4 *>(dst) = w;
    return;
  }
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int j = 0; j < 16; ++j)
    if (j < n) dst[j] = (uint8_t)(u[j / 4] >> (8 * (j & 3)));
}

// Scale of the block that 8 neighbouring lanes hold, from each lane's magnitudes.
template <class T>
__device__ __forceinline__ Scale lanes_scale(uint32_t m, int format, int pow2) {
#pragma unroll
  for (int d = 1; d < 8; d *= 2) m = T::larger(m, __shfl_xor_sync(0xffffffffu, m, d));
  return scale_of(T::top(m), format, pow2);
}

// 1 x 128 blocks: unit u = row * blocks + block; a warp takes 4 neighbouring units at a time, so that
// it reads 1 KB (of 16 bits) at once and a block's maximum stays within 8 lanes. No shared memory, 31
// registers: 72% of the warps resident. 8192 x 4096 BF16: 16.8 us, 6.1 TB/s
// (90% of a copy's rate). 1 x 4096: 1.3 us.
template <class T, int FORMAT>
__global__ void __launch_bounds__(256, T::CTAS) rows_kernel(const QuantParams p) {
  griddep_wait();  // (launched with programmatic dependent launch: see launch_1d)
  constexpr int size = T::W == 16 ? 4 : 2;
  const int lane = threadIdx.x & 31, sub = lane & 7;
  const int blocks = (int)(((unsigned)p.cols + 127) / 128);
  const long long units = (long long)p.rows * blocks;
  const long long step = (long long)gridDim.x * 8 * 4;
  const int step_r = (int)(step / blocks), step_b = (int)(step % blocks);
  long long u = ((long long)blockIdx.x * 8 + (threadIdx.x >> 5)) * 4;
  const long long mine = u + (lane >> 3);
  unsigned r = (unsigned)(mine / blocks);  // (up to rows + 2: past 31 bits where rows are most)
  int b = (int)(mine % blocks);
  for (; u < units; u += step) {
    const int c = b * 128 + sub * 16;
    const int n = r < (unsigned)p.rows ? p.cols - c : 0;
    Sixteen<T> v;
    load16<T>(reinterpret_cast<const char *>(p.x) + (r * p.ldx + c) * size, p.vec, n, v);
    Scale s = lanes_scale<T>(max16<T>(v), FORMAT, p.pow2);
    if (sub == 0 && r < (unsigned)p.rows) p.a.s[r * p.a.s_row + b * p.a.s_col] = s.s;
    if constexpr (T::SMALL) {
      if (s.s < kSmallScale) {
        raise(s);
        scale16<T>(v, kUp);
      }
    }
    store16(p.a.q + r * p.a.ldq + c, p.a.vec, n, quantize16<T, FORMAT>(v, s));
    r += step_r;
    b += step_b;
    if (b >= blocks) {
      b -= blocks;
      ++r;
    }
  }
  griddep_launch_dependents();
}

enum { COLS = 0, SQUARE = 1, PAIR = 2 };

// One 128 x 128 tile per CTA of 8 G threads: thread (g = tid / 8, sub = tid % 8) holds columns
// 16 sub .. + 15 of rows g, g + G, ...: 32 registers of x. The tile stays in registers from its one
// read to its last use, so a CTA has no loads under way while it computes and stores: several CTAs
// per SM overlap instead, as many as the registers allow (34 to 47% of the warps). 14336 x 4096
// FP32 in squares: 49 us, 6.0 TB/s, 89% of a copy's rate. 8192 x 4096 BF16 by rows and by columns at
// once: 34 us, 4.0 TB/s, with twice the arithmetic per byte read; two calls, by rows and by columns,
// take 16.8 + 25.8 us. (CTAs of 512 threads with half as many elements each: 44 us for 35, 23 for 16 in
// squares; a column's maximum then takes as many shuffles for half as many rows.)
template <class T>
constexpr int kRowGroups = T::W == 16 ? 64 : 32;

template <class T, int FORMAT, int WHICH>
__global__ void __launch_bounds__(8 * kRowGroups<T>, T::W == 16 ? 2 : WHICH == PAIR ? 3 : 4)
    tile_kernel(const QuantParams p, int tiles_c) {
  griddep_wait();
  constexpr int size = T::W == 16 ? 4 : 2;
  constexpr int G = kRowGroups<T>, WARPS = G / 4, ROWS = 128 / G;
  __shared__ uint32_t top[WARPS][8 * T::W];
  __shared__ __align__(16) float col_r[128], col_minus[128], col_up[128];
  const int tid = threadIdx.x, sub = tid & 7, g = tid >> 3, warp = tid >> 5;
  const int br = blockIdx.x / tiles_c, bc = blockIdx.x % tiles_c;
  const int r0 = br * 128 + g, c0 = bc * 128 + sub * 16;
  const int n = p.cols - c0;
  Sixteen<T> v[ROWS];
  const char *src = reinterpret_cast<const char *>(p.x) + (r0 * p.ldx + c0) * size;
#pragma unroll
  for (int i = 0; i < ROWS; ++i)
    load16<T>(src + i * (G * p.ldx * size), p.vec, r0 + G * i < p.rows ? n : 0, v[i]);

  if constexpr (WHICH == SQUARE) {
    uint32_t m = max16<T>(v[0]);
#pragma unroll
    for (int i = 1; i < ROWS; ++i) m = T::larger(m, max16<T>(v[i]));
#pragma unroll
    for (int d = 1; d < 32; d *= 2) m = T::larger(m, __shfl_xor_sync(0xffffffffu, m, d));
    if ((tid & 31) == 0) top[warp][0] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WARPS; ++w) m = T::larger(m, top[w][0]);
    Scale s = scale_of(T::top(m), FORMAT, p.pow2);
    if (tid == 0) p.a.s[br * p.a.s_row + bc * p.a.s_col] = s.s;
    if constexpr (T::SMALL) {
      if (s.s < kSmallScale) {
        raise(s);
#pragma unroll
        for (int i = 0; i < ROWS; ++i) scale16<T>(v[i], kUp);
      }
    }
    uint8_t *dst = p.a.q + r0 * p.a.ldq + c0;
#pragma unroll
    for (int i = 0; i < ROWS; ++i)
      store16(dst + i * (G * p.a.ldq), p.a.vec, r0 + G * i < p.rows ? n : 0,
              quantize16<T, FORMAT>(v[i], s));
  } else {
    const Result &o = WHICH == PAIR ? p.c : p.a;
#pragma unroll
    for (int k = 0; k < T::W; ++k) {
      uint32_t m = v[0].w[k];
#pragma unroll
      for (int i = 1; i < ROWS; ++i) m = T::larger(m, v[i].w[k]);
      m = T::larger(m, __shfl_xor_sync(0xffffffffu, m, 8));
      m = T::larger(m, __shfl_xor_sync(0xffffffffu, m, 16));
      if ((tid & 31) < 8) top[warp][sub * T::W + k] = m;
    }
    __syncthreads();
    bool small = false;
    if (tid < 128) {  // column tid of the tile
      const int word = T::W == 16 ? tid : tid / 2;
      uint32_t m = top[0][word];
#pragma unroll
      for (int w = 1; w < WARPS; ++w) m = T::larger(m, top[w][word]);
      const float amax = fabsf(T::value(m, tid & 1));
      Scale s = scale_of(amax, FORMAT, p.pow2);
      if constexpr (T::SMALL) {
        small = s.s < kSmallScale && amax > 0.0f;  // (a column of zeros needs no correction)
        col_up[tid] = small ? kUp : 1.0f;
        if (small) raise(s);
      }
      col_r[tid] = s.r;
      col_minus[tid] = s.minus;
      if (bc * 128 + tid < p.cols) o.s[br * o.s_row + (bc * 128 + tid) * o.s_col] = s.s;
    }
    if constexpr (WHICH == PAIR) {
      uint8_t *dst = p.a.q + r0 * p.a.ldq + c0;
#pragma unroll
      for (int i = 0; i < ROWS; ++i) {
        const int r = r0 + G * i;
        Scale s = lanes_scale<T>(max16<T>(v[i]), FORMAT, p.pow2);
        if (sub == 0 && r < p.rows) p.a.s[r * p.a.s_row + bc * p.a.s_col] = s.s;
        if constexpr (T::SMALL) {
          if (s.s < kSmallScale) {
            raise(s);
            scale16<T>(v[i], kUp);
          }
        }
        store16(dst + i * (G * p.a.ldq), p.a.vec, r < p.rows ? n : 0,
                quantize16<T, FORMAT>(v[i], s));
        if constexpr (T::SMALL) {
          if (s.s < kSmallScale) scale16<T>(v[i], kDown);  // (the columns have their own scales)
        }
      }
    }
    if constexpr (!T::SMALL) {
      __syncthreads();
    } else {
      if (__syncthreads_or(small)) {
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
#pragma unroll
          for (int k = 0; k < T::W; ++k) {
            const int c = sub * 16 + k * (16 / T::W);
            v[i].w[k] = T::scaled(v[i].w[k], col_up[c], col_up[c + (T::W == 8)]);
          }
      }
    }
    uint8_t *dst = o.q + r0 * o.ldq + c0;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      uint32_t w[4];
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const int c = sub * 16 + 4 * h;
        const float4 f = *reinterpret_cast<const float4 *>(col_r + c);
        const float4 d = *reinterpret_cast<const float4 *>(col_minus + c);
        w[h] = quantize2<FORMAT>(at<T>(v[i], 4 * h), at<T>(v[i], 4 * h + 1), pack2(f.x, f.y),
                                 pack2(d.x, d.y)) |
               quantize2<FORMAT>(at<T>(v[i], 4 * h + 2), at<T>(v[i], 4 * h + 3), pack2(f.z, f.w),
                                 pack2(d.z, d.w))
                   << 16;
      }
      store16(dst + i * (G * o.ldq), o.vec, r0 + G * i < p.rows ? n : 0,
              make_uint4(w[0], w[1], w[2], w[3]));
    }
  }
  griddep_launch_dependents();
}

template <class T, int FORMAT>
static cudaError_t launch_quantize(const QuantParams &p, int which, int sms, cudaStream_t stream) {
  if (which < 0) {
    const long long units = (long long)p.rows * ceil_div(p.cols, 128);
    const long long grid = std::min<long long>(ceil_div(units, 8 * 4), 8LL * sms);
    return launch_1d(rows_kernel<T, FORMAT>, (int)grid, 256, 0, 1, stream, p);
  }
  const int tiles_c = (int)ceil_div(p.cols, 128);
  const long long tiles = (long long)tiles_c * ceil_div(p.rows, 128);
  if (tiles > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  constexpr int threads = 8 * kRowGroups<T>;
  if (which == SQUARE)
    return launch_1d(tile_kernel<T, FORMAT, SQUARE>, (int)tiles, threads, 0, 1, stream, p, tiles_c);
  if (which == COLS)
    return launch_1d(tile_kernel<T, FORMAT, COLS>, (int)tiles, threads, 0, 1, stream, p, tiles_c);
  return launch_1d(tile_kernel<T, FORMAT, PAIR>, (int)tiles, threads, 0, 1, stream, p, tiles_c);
}

template <class T>
static cudaError_t launch_quantize(const QuantParams &p, int which, int sms, cudaStream_t stream) {
  return p.format ? launch_quantize<T, F8_E5M2>(p, which, sms, stream)
                  : launch_quantize<T, F8_E4M3>(p, which, sms, stream);
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
  const auto misplaced = [](const float *at) { return reinterpret_cast<uintptr_t>(at) % 4 != 0; };
  if (any && (s == nullptr || misplaced(s))) return -12;
  if (s_row < 0) return -13;
  if (s_col < 0) return -14;
  if (qc != nullptr) {
    if (block_rows != 1) return -15;
    if (ldqc < std::max(1, cols)) return -16;
    if (any && (sc == nullptr || misplaced(sc))) return -17;
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
  p.a = f8::Result{static_cast<uint8_t *>(q), ldq, s, s_row, s_col, aligned(q, ldq, 16)};
  p.c = f8::Result{static_cast<uint8_t *>(qc), ldqc, sc, sc_row, sc_col, aligned(qc, ldqc, 16)};
  const int which = qc != nullptr ? f8::PAIR
                    : block_rows == 1 ? -1
                    : block_cols == 1 ? f8::COLS
                                      : f8::SQUARE;
  if (x_type == F8_D_F32) return (int)f8::launch_quantize<f8::F32>(p, which, sms, stream);
  if (x_type == F8_D_BF16) return (int)f8::launch_quantize<f8::BF16>(p, which, sms, stream);
  return (int)f8::launch_quantize<f8::F16>(p, which, sms, stream);
}

extern "C" int f8_quantize_with(const f8_quantize_args *a) {
  if (a == nullptr) return -1;
  return f8_quantize(a->rows, a->cols, a->x, a->x_type, a->ldx, a->block_rows, a->block_cols,
                     a->format, a->pow2, a->q, a->ldq, a->s, a->s_row, a->s_col, a->qc, a->ldqc,
                     a->sc, a->sc_row, a->sc_col, a->stream);
}

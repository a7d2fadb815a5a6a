// What the operators on whole rows share (layer norm, its gradients, the quantiser to 8-bit
// integers): a row of up to 16384 elements lies in the registers of 8 to 1024 neighbouring threads,
// packed as it was loaded, in chunks of 8 elements per thread.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

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

// Two FP32 numbers in one instruction.
using Two = unsigned long long;
__device__ __forceinline__ Two both(float v) { return pack2(v, v); }
__device__ __forceinline__ Two add2(Two a, Two b) {
  Two d;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ Two mul2(Two a, Two b) {
  Two d;
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
  Two d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ float sum2(Two v) {
  const float2 f = unpack2(v);
  return f.x + f.y;
}

// Elements 2 i and 2 i + 1 of a chunk, to FP32 and back.
template <class T>
__device__ __forceinline__ Two pair(const Chunk<T> &c, int i) {
  return pack2(c[2 * i], c[2 * i + 1]);
}
template <class T>
__device__ __forceinline__ void set_pair(Chunk<T> &c, int i, Two v) {
  const float2 f = unpack2(v);
  if constexpr (T::W == 8) {
    c.w[2 * i % T::W] = __float_as_uint(f.x);
    c.w[(2 * i + 1) % T::W] = __float_as_uint(f.y);
  } else {
    c.w[i] = tcx::pack_out(T::TYPE, f.x, f.y);
  }
}
// Zero instead of the elements from number n on.
__device__ __forceinline__ Two first(Two v, int i, int n) {
  const float2 f = unpack2(v);
  return pack2(2 * i < n ? f.x : 0.0f, 2 * i + 1 < n ? f.y : 0.0f);
}

// How TPR threads share a row: chunk c of thread t holds, with VEC (rows are 16-byte aligned), pieces of
// E neighbouring elements (16 bytes) that are TPR pieces apart, else elements that are TPR apart, so
// that a warp reads neighbours either way. Of a chunk's elements the first count() exist.
template <class T, int TPR, bool VEC>
struct Share {
  static constexpr int E = VEC ? 16 / T::SIZE : 1, PIECES = 8 / E;
  int cols, t;
  __device__ __forceinline__ int col(int c, int j) const { return ((c * PIECES + j / E) * TPR + t) * E + j % E; }
  __device__ __forceinline__ int count(int c) const {
    int n = 0;
#pragma unroll
    for (int i = 0; i < PIECES; ++i) n += min(E, max(0, cols - col(c, i * E)));
    return n;
  }
  // Elements that do not exist are zero.
  __device__ __forceinline__ void load(const void *row, int c, int n, Chunk<T> &v) const {
    const char *src = reinterpret_cast<const char *>(row);
    if (VEC && n == 8) {
#pragma unroll
      for (int i = 0; i < PIECES; ++i) {
        const uint4 u = *reinterpret_cast<const uint4 *>(src + (long long)col(c, i * E) * T::SIZE);
        v.w[4 * i] = u.x, v.w[4 * i + 1] = u.y, v.w[4 * i + 2] = u.z, v.w[4 * i + 3] = u.w;
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
  __device__ __forceinline__ void store(void *row, int c, int n, const Chunk<T> &v) const {
    char *dst = reinterpret_cast<char *>(row);
    if (VEC && n == 8) {
#pragma unroll
      for (int i = 0; i < PIECES; ++i)
        *reinterpret_cast<uint4 *>(dst + (long long)col(c, i * E) * T::SIZE) =
            make_uint4(v.w[4 * i], v.w[4 * i + 1], v.w[4 * i + 2], v.w[4 * i + 3]);
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

// A thread's chunks of the rows to come, of INPUTS matrices: with VEC as asynchronous copies into its own
// places of a ring in shared memory, DEPTH rows ahead (what one row's registers hold under way does not
// fill HBM's latency: layer norm of 8192 x 4096 BF16 took 37 us so and 32 with the ring, when
// numbers were still taken one by one: 22 now), else one row ahead in registers.
// Nobody else reads them, so there is nothing to wait for but the thread's own copies.
template <class T, int TPR, int CH, bool VEC, int INPUTS, int DEPTH, int THREADS>
struct Ahead {
  using S = Share<T, TPR, VEC>;
  static constexpr int ROW = THREADS * CH * 8 * T::SIZE;  // bytes of the CTA's rows of one input
  static constexpr int BYTES = VEC ? DEPTH * INPUTS * ROW : 0;
  S sh;
  int n[CH];
  bool whole;                     // every chunk has its 8 elements
  long long rows, row, step;      // row: the next one to fetch
  const char *from[INPUTS];       // that row of each input
  long long ld[INPUTS];           // bytes from there to the one after it
  uint32_t at;                    // this thread's place in the ring
  int slot;
  Chunk<T> next[VEC ? 1 : INPUTS][VEC ? 1 : CH];

  // Rows `row`, `row` + step, ... of inputs that begin at `input`, with leading dimensions in bytes.
  __device__ __forceinline__ Ahead(int cols, void *ring, const char *const (&input)[INPUTS],
                                   const long long (&pitch)[INPUTS], int rows_, long long row_, long long step_)
      : sh{cols, (int)(threadIdx.x % TPR)}, rows(rows_), row(row_), step(step_), slot(0) {
    at = VEC ? saddr(ring) + threadIdx.x * 16 : 0;
    whole = true;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      n[c] = sh.count(c);
      whole &= n[c] == 8;
    }
#pragma unroll
    for (int i = 0; i < INPUTS; ++i) {
      from[i] = input[i] + row * pitch[i];
      ld[i] = step * pitch[i];
    }
  }
  __device__ __forceinline__ void begin() {
    if constexpr (VEC) {
#pragma unroll
      for (int d = 0; d < DEPTH - 1; ++d) copy(d);
    } else {
      fetch();
    }
  }
  // The chunks of the oldest row under way (of one past the last: anything).
  __device__ __forceinline__ void take(Chunk<T> (&v)[INPUTS][CH]) {
    if constexpr (VEC) {
      cp_async_wait<DEPTH - 2>();
#pragma unroll
      for (int i = 0; i < INPUTS; ++i)
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int q = 0; q < S::PIECES; ++q) {
            uint32_t(&w)[T::W] = v[i][c].w;
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];\n"
                         : "=r"(w[4 * q]), "=r"(w[4 * q + 1]), "=r"(w[4 * q + 2]), "=r"(w[4 * q + 3])
                         : "r"(place(slot, i, c, q))
                         : "memory");
          }
      copy(slot == 0 ? DEPTH - 1 : slot - 1);
      slot = slot == DEPTH - 1 ? 0 : slot + 1;
    } else {
#pragma unroll
      for (int i = 0; i < INPUTS; ++i)
#pragma unroll
        for (int c = 0; c < CH; ++c) v[i][c] = next[i][c];
      fetch();
    }
  }

 private:
  __device__ __forceinline__ uint32_t place(int slot_, int i, int c, int q) const {
    return at + slot_ * (INPUTS * ROW) + ((i * CH + c) * S::PIECES + q) * (THREADS * 16);
  }
  __device__ __forceinline__ void advance() {
    row += step;
#pragma unroll
    for (int i = 0; i < INPUTS; ++i) from[i] += ld[i];
  }
  __device__ __forceinline__ void copy(int slot_) {
    if (row < rows) {
#pragma unroll
      for (int i = 0; i < INPUTS; ++i)
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int q = 0; q < S::PIECES; ++q) {
            const int col = sh.col(c, q * S::E);
            if (whole) {
              cp_async_16(place(slot_, i, c, q), from[i] + col * T::SIZE, 16);
            } else {
              const int have = min(S::E, sh.cols - col) * T::SIZE;
              cp_async_16(place(slot_, i, c, q), from[i] + (have > 0 ? col * T::SIZE : 0), max(0, have));
            }
          }
    }
    cp_async_commit();
    advance();
  }
  __device__ __forceinline__ void fetch() {
#pragma unroll
    for (int i = 0; i < INPUTS; ++i)
#pragma unroll
      for (int c = 0; c < CH; ++c) sh.load(from[i], c, row < rows ? n[c] : 0, next[i][c]);
    advance();
  }
};

// A vector of parameters (a weight, a bias) in any of the types; `otherwise` where there is none.
struct Vector {
  const void *ptr;
  int type;
  int vec;             // 16-byte aligned
  __device__ __forceinline__ float at(int i, float otherwise) const {
    return ptr ? tcx::load_out(ptr, type, i) : otherwise;
  }
};

// The same from element `at` on.
__device__ __forceinline__ Vector from(const Vector &p, long long at) {
  const int size = p.type == tcx::OUT_F32 ? 4 : 2;
  return {p.ptr ? static_cast<const char *>(p.ptr) + at * size : nullptr, p.type, p.vec};
}

// Rows that do not stay in registers are taken in blocks of 8 elements per thread of a CTA: what `each` does
// with block after block, given the columns from its first one on and that one's number.
template <class T, int TPR, bool VEC, class Each>
__device__ __forceinline__ void blocks(int cols, Each &&each) {
  for (long long at = 0; at < cols; at += 8 * TPR)
    each(Share<T, TPR, VEC>{(int)(cols - at), (int)threadIdx.x}, at);
}

// The parameters of chunk c's columns (0 past the last one).
template <class S>
__device__ __forceinline__ void parameters(const Vector &p, const S &sh, int c, int n, float otherwise, Two (&to)[4]) {
  float v[8];
  if (S::E > 1 && p.ptr && p.vec && n == 8) {
    constexpr int E = S::E;
#pragma unroll
    for (int q = 0; q < S::PIECES; ++q) {
      const long long at = sh.col(c, q * E);
      if (p.type == tcx::OUT_F32) {
#pragma unroll
        for (int j = 0; j < E; j += 4) {
          const float4 f = *reinterpret_cast<const float4 *>(static_cast<const float *>(p.ptr) + at + j);
          v[q * E + j] = f.x, v[q * E + j + 1] = f.y, v[q * E + j + 2] = f.z, v[q * E + j + 3] = f.w;
        }
      } else {
#pragma unroll
        for (int j = 0; j < E; j += 4) {
          const uint2 u = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(p.ptr) + at + j);
          const uint32_t w[2] = {u.x, u.y};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            v[q * E + j + i] = p.type == tcx::OUT_BF16 ? BF16::value(w[i / 2], i & 1) : F16::value(w[i / 2], i & 1);
        }
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < n ? p.at(sh.col(c, j), otherwise) : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) to[i] = pack2(v[2 * i], v[2 * i + 1]);
}

// Sums of N numbers over the TPR threads of a row (one of ROWS rows of a CTA), the same bits in each of
// them. `turn` alternates between calls of a kernel, so that one barrier is enough: whoever writes a
// buffer again has passed the barrier of the call in between, before which everybody had read it.
// (TPR: up to 32, 64, or a multiple of 128.)
template <int TPR, int N, int ROWS = 1>
struct RowSums {
  float part[TPR > 32 ? ROWS : 1][2][N][TPR < 128 ? 4 : TPR / 32];
};
template <int TPR, int N, int ROWS>
__device__ __forceinline__ void row_sum(float (&v)[N], RowSums<TPR, N, ROWS> &sums, int turn) {
#pragma unroll
  for (int d = 1; d < (TPR < 32 ? TPR : 32); d *= 2)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], d);
  if constexpr (TPR > 32) {
    const int row = ROWS == 1 ? 0 : threadIdx.x / TPR;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) sums.part[row][turn][i][threadIdx.x % TPR >> 5] = v[i];
    if (ROWS == 1)
      __syncthreads();
    else
      tcx::named_barrier(1 + row, TPR);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float4 *from = reinterpret_cast<const float4 *>(sums.part[row][turn][i]);
      float4 s = from[0];
#pragma unroll
      for (int w = 1; w < TPR / 128; ++w) {
        const float4 u = from[w];
        s.x += u.x, s.y += u.y, s.z += u.z, s.w += u.w;
      }
      v[i] = TPR < 128 ? s.x + s.y : (s.x + s.y) + (s.z + s.w);
    }
  }
}

// A sum of two FP32 numbers, hi + lo, as exact as 48 bits: for long sums, where 64-bit additions would be
// what takes the time (two per cycle and SM). add(): the sum of hi and v without a rounding (Knuth's
// two-sum), the rest into lo.
struct Long {
  float hi = 0.0f, lo = 0.0f;
  __device__ __forceinline__ void add(float v) {
    const float s = hi + v, b = s - hi;
    lo += (hi - (s - b)) + (v - b);
    hi = s;
  }
  __device__ __forceinline__ void add(const Long &v) {
    add(v.hi);
    lo += v.lo;
  }
  // (where hi is infinite or NaN lo may be NaN: hi says it)
  __device__ __forceinline__ float over(long long n) const {
    return isfinite(hi) ? (float)(((double)hi + (double)lo) / (double)n) : hi;
  }
};

// Over the 1024 threads of a CTA; the sum in the first one. Not twice without a barrier in between.
__device__ __forceinline__ Long cta_sum(Long v, Long *part) {
#pragma unroll
  for (int d = 16; d > 0; d /= 2) {
    Long u;
    u.hi = __shfl_down_sync(0xffffffffu, v.hi, d);
    u.lo = __shfl_down_sync(0xffffffffu, v.lo, d);
    v.add(u);
  }
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x < 32) {
    v = part[threadIdx.x];
#pragma unroll
    for (int d = 16; d > 0; d /= 2) {
      Long u;
      u.hi = __shfl_down_sync(0xffffffffu, v.hi, d);
      u.lo = __shfl_down_sync(0xffffffffu, v.lo, d);
      v.add(u);
    }
  }
  return v;
}

// s / n for the FP32 number n of elements, with r = 1 / n: the quotient corrected by its remainder.
__device__ __forceinline__ float over(float s, float n, float r) {
  const float q = s * r;
  return isfinite(q) ? fmaf(fmaf(-q, n, s), r, q) : q;
}

// Once per kernel and device: leave to use `bytes` of dynamic shared memory.
constexpr int kDevices = 64;
template <class F>
static cudaError_t allow_bytes(F kernel, int bytes, std::once_flag (&once)[kDevices], cudaError_t (&set)[kDevices]) {
  if (bytes <= 16 * 1024) return cudaSuccess;  // (48 KB with what is static go without)
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kDevices) return cudaErrorInvalidDevice;
  std::call_once(once[dev], [&] {
    set[dev] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  });
  return set[dev];
}

constexpr int kLongest = 16384;  // elements of a row that stays in registers

constexpr bool aligned(uintptr_t ptr, long long ld_bytes) { return ptr % 16 == 0 && ld_bytes % 16 == 0; }

}  // namespace rows
}  // namespace sgemm

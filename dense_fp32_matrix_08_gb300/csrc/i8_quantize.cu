// Quantiser to 8-bit integers with a scale for each row:
//   a = max(max |x|, 2^-119), scale = a / 127, q = x (127 / a) rounded to a whole number
//
// Bound by HBM: x is read once and a byte written for each element. A row stays packed in registers
// between its maximum and its result. The product with 127 / a is rounded once, to a whole number, by
// the addition of 1.5 * 2^23 in the same FMA, which leaves q in the low byte: |q| is at most 127, since
// a (127 / a) (1 + 2^-24) is nearer to 127 than to 128. 8192 x 4096 BF16: 16.1 us, 6.2 TB/s, 92% of a copy's
// rate; 1 x 4096: 1.2 us.
#include <algorithm>

#include "../../include/i8_linear.h"
#include "row_common.cuh"

namespace sgemm {
namespace i8q {

using namespace rows;

struct Params {
  int rows, cols;
  const char *x;
  long long ldx;       // bytes
  uint8_t *q;
  long long ldq;
  float *scale;
  int vec_q;           // 8-byte stores to q are aligned
};

// The larger magnitudes of two words (with either sign; NaN over all), and the largest one in a word.
template <class T>
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) {
  uint32_t m;
  if constexpr (T::TYPE == tcx::OUT_F32)
    asm("max.NaN.xorsign.abs.f32 %0, %1, %2;\n" : "=r"(m) : "r"(a), "r"(b));
  else if constexpr (T::TYPE == tcx::OUT_BF16)
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;\n" : "=r"(m) : "r"(a), "r"(b));
  else
    asm("max.NaN.xorsign.abs.f16x2 %0, %1, %2;\n" : "=r"(m) : "r"(a), "r"(b));
  return m;
}
template <class T>
__device__ __forceinline__ uint32_t top(uint32_t w) {  // FP32 bits of a magnitude
  if constexpr (T::TYPE == tcx::OUT_F32) return w & 0x7fffffffu;
  w &= 0x7fff7fffu;
  if constexpr (T::TYPE == tcx::OUT_BF16) return max(w & 0xffff0000u, w << 16);
  return __float_as_uint(__half2float(__ushort_as_half((unsigned short)max(w >> 16, w & 0xffffu))));
}

// Largest magnitude over a row's threads: FP32 bits, ordered as integers (a NaN is the largest).
template <int TPR>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t (*part)[32], int turn) {
#pragma unroll
  for (int d = 1; d < (TPR < 32 ? TPR : 32); d *= 2) v = max(v, __shfl_xor_sync(0xffffffffu, v, d));
  if constexpr (TPR > 32) {
    if ((threadIdx.x & 31) == 0) part[turn][threadIdx.x >> 5] = v;
    __syncthreads();
    v = part[turn][0];
#pragma unroll
    for (int w = 1; w < TPR / 32; ++w) v = max(v, part[turn][w]);
  }
  return v;
}

struct Scale {
  float s, r;  // scale, and what x is multiplied with
  bool finite;
};
__device__ __forceinline__ Scale scale_of(uint32_t bits) {
  Scale o;
  const float a = fmaxf(__uint_as_float(bits), 0x1p-119f);
  o.finite = bits < 0x7f800000u;
  o.s = o.finite ? __fdiv_rn(a, 127.0f) : __uint_as_float(0x7fc00000u);
  o.r = __fdiv_rn(127.0f, a);
  return o;
}
// q in the low byte.
__device__ __forceinline__ uint32_t rounded(float x, const Scale &s) {
  return __float_as_uint(fmaf(x, s.r, 12582912.0f));
}
__device__ __forceinline__ uint32_t four(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// q of chunk c, of which n elements exist.
template <bool VEC, class T, class S>
__device__ __forceinline__ void put(const Params &p, const Scale &s, const S &sh, uint8_t *to, int c, int n,
                                    const Chunk<T> &v) {
  uint32_t q[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) q[j] = s.finite ? rounded(v[j], s) : 0;
  if (VEC && p.vec_q && n == 8) {
    const uint32_t lo = four(q[0], q[1], q[2], q[3]), hi = four(q[4], q[5], q[6], q[7]);
    if constexpr (S::E == 8) {
      *reinterpret_cast<uint2 *>(to + sh.col(c, 0)) = make_uint2(lo, hi);
    } else {
      *reinterpret_cast<uint32_t *>(to + sh.col(c, 0)) = lo;
      *reinterpret_cast<uint32_t *>(to + sh.col(c, 4)) = hi;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) to[sh.col(c, j)] = (uint8_t)q[j];
  }
}

// Rows under way. More than it takes costs time: 8192 x 4096 BF16 16.1 us with three, 18.3 with two; FP32 25.6 with
// two, 26.5 with three, but 16384 x 1024 FP32 13.7 with three, 15.7 with two.
template <class T, int TPR, int CH>
constexpr int kDepth = T::SIZE == 4 && TPR * CH >= 256 ? 2 : 3;

template <class T, int TPR, int CH, bool VEC>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR, TPR < 128 ? 8 : 1024 / TPR) quantize_kernel(const Params p) {
  constexpr int THREADS = TPR < 128 ? 128 : TPR, RPB = THREADS / TPR;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ uint32_t part[2][32];
  const long long step = (long long)gridDim.x * RPB;
  long long base = (long long)blockIdx.x * RPB;  // (the same for a whole CTA)
  long long row = base + threadIdx.x / TPR;
  Ahead<T, TPR, CH, VEC, 1, kDepth<T, TPR, CH>, THREADS> ahead(p.cols, ring, {p.x}, {p.ldx}, p.rows, row, step);
  const auto &sh = ahead.sh;
  const auto &n = ahead.n;
  const bool once = step >= p.rows;  // (a launch that takes a while lets the next one begin at its end)
  if (once) griddep_launch_dependents();
  griddep_wait();  // (launched with programmatic dependent launch: see launch_1d)
  ahead.begin();
  for (int turn = 0; base < p.rows; base += step, row += step, turn ^= 1) {
    Chunk<T> in[1][CH];
    ahead.take(in);
    const Chunk<T>(&v)[CH] = in[0];
    uint32_t m = v[0].w[0];
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int i = 0; i < T::W; ++i) m = larger<T>(m, v[c].w[i]);
    const Scale s = scale_of(row_max<TPR>(top<T>(m), part, turn));
    if (row < p.rows) {
      if (sh.t == 0) p.scale[row] = s.s;
      uint8_t *to = p.q + row * p.ldq;
#pragma unroll
      for (int c = 0; c < CH; ++c) put<VEC>(p, s, sh, to, c, n[c], v[c]);
    }
  }
  if (!once) griddep_launch_dependents();
}

// Rows of any length: a CTA reads its row twice.
template <class T, bool VEC>
__global__ void __launch_bounds__(1024) quantize_long_kernel(const Params p) {
  __shared__ uint32_t part[2][32];
  griddep_launch_dependents();
  griddep_wait();
  int turn = 0;
  for (long long row = blockIdx.x; row < p.rows; row += gridDim.x, turn ^= 1) {
    const char *x = p.x + row * p.ldx;
    uint32_t m = 0;
    blocks<T, 1024, VEC>(p.cols, [&](const auto &sh, long long at) {
      Chunk<T> v;
      sh.load(x + at * T::SIZE, 0, sh.count(0), v);
#pragma unroll
      for (int i = 0; i < T::W; ++i) m = larger<T>(m, v.w[i]);
    });
    const Scale s = scale_of(row_max<1024>(top<T>(m), part, turn));
    if (threadIdx.x == 0) p.scale[row] = s.s;
    blocks<T, 1024, VEC>(p.cols, [&](const auto &sh, long long at) {
      const int n = sh.count(0);
      Chunk<T> v;
      sh.load(x + at * T::SIZE, 0, n, v);
      put<VEC>(p, s, sh, p.q + row * p.ldq + at, 0, n, v);
    });
  }
}

template <class T, int TPR, int CH, bool VEC>
static cudaError_t launch(const Params &p, int sms, cudaStream_t stream) {
  constexpr int threads = TPR < 128 ? 128 : TPR, rpb = threads / TPR;
  constexpr int bytes = Ahead<T, TPR, CH, VEC, 1, kDepth<T, TPR, CH>, threads>::BYTES;
  static cudaError_t set[kDevices];
  static std::once_flag once[kDevices];
  const cudaError_t e = allow_bytes(quantize_kernel<T, TPR, CH, VEC>, bytes, once, set);
  if (e != cudaSuccess) return e;
  const long long grid = std::min<long long>(ceil_div(p.rows, rpb), (long long)sms * (1024 / threads));
  return launch_1d(quantize_kernel<T, TPR, CH, VEC>, (int)grid, threads, bytes, 1, stream, p);
}
template <class T, int TPR, int CH>
static cudaError_t launch(const Params &p, bool vec, int sms, cudaStream_t stream) {
  return vec ? launch<T, TPR, CH, true>(p, sms, stream) : launch<T, TPR, CH, false>(p, sms, stream);
}

template <class T>
static cudaError_t run(const Params &p, bool vec, int sms, cudaStream_t stream) {
  if (p.cols <= 64) return launch<T, 8, 1>(p, vec, sms, stream);
  if (p.cols <= 256) return launch<T, 32, 1>(p, vec, sms, stream);
  if (p.cols <= 512) return launch<T, 32, 2>(p, vec, sms, stream);
  // (a warp per row needs no barrier, where its registers hold it: 16384 x 1024 BF16 11.2 us with 128 threads on
  // a row, 9.9 so; FP32 13.8 and 15.9)
  if (p.cols <= 1024) {
    if constexpr (T::SIZE == 4) return launch<T, 128, 1>(p, vec, sms, stream);
    else return vec ? launch<T, 32, 4, true>(p, sms, stream) : launch<T, 128, 1, false>(p, sms, stream);
  }
  if (p.cols <= 2048) return launch<T, 128, 2>(p, vec, sms, stream);
  if (p.cols <= 4096) return launch<T, 256, 2>(p, vec, sms, stream);
  if (p.cols <= 6144) return launch<T, 384, 2>(p, vec, sms, stream);
  if (p.cols <= 8192) return launch<T, 512, 2>(p, vec, sms, stream);
  if (p.cols <= 12288) return launch<T, 768, 2>(p, vec, sms, stream);
  if (p.cols <= kLongest) return launch<T, 1024, 2>(p, vec, sms, stream);
  return launch_1d(vec ? quantize_long_kernel<T, true> : quantize_long_kernel<T, false>, std::min(p.rows, 2 * sms),
                   1024, 0, 1, stream, p);
}

}  // namespace i8q
}  // namespace sgemm

using namespace sgemm;

extern "C" int i8_quantize(int rows, int cols, const void *x, int x_type, int ldx, void *q, int ldq,
                           float *scale, cudaStream_t stream) {
  const bool any = rows > 0 && cols > 0;
  if (rows < 0) return -1;
  if (cols < 0) return -2;
  if (any && x == nullptr) return -3;
  if (x_type != I8_F32 && x_type != I8_BF16 && x_type != I8_F16) return -4;
  const int size = x_type == I8_F32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(x) % size != 0) return -3;
  if (ldx < std::max(1, cols)) return -5;
  if (any && q == nullptr) return -6;
  if (ldq < std::max(1, cols)) return -7;
  if ((rows > 0 && scale == nullptr) || reinterpret_cast<uintptr_t>(scale) % 4 != 0) return -8;
  if (rows == 0) return 0;
  int sms = 0;
  const cudaError_t e = device_setup(&sms);
  if (e != cudaSuccess) return (int)e;
  const auto at = [](const void *ptr) { return reinterpret_cast<uintptr_t>(ptr); };
  i8q::Params p{};
  p.rows = rows;
  p.cols = cols;
  p.x = static_cast<const char *>(x);
  p.ldx = (long long)ldx * size;
  p.q = static_cast<uint8_t *>(q);
  p.ldq = ldq;
  p.scale = scale;
  p.vec_q = at(q) % 8 == 0 && (rows == 1 || ldq % 8 == 0);
  const bool vec = rows::aligned(at(x), rows > 1 ? p.ldx : 0);
  if (x_type == I8_F32) return (int)i8q::run<rows::F32>(p, vec, sms, stream);
  if (x_type == I8_BF16) return (int)i8q::run<rows::BF16>(p, vec, sms, stream);
  return (int)i8q::run<rows::F16>(p, vec, sms, stream);
}

extern "C" int i8_quantize_with(const i8_quantize_args *a) {
  if (a == nullptr) return -1;
  return i8_quantize(a->rows, a->cols, a->x, a->x_type, a->ldx, a->q, a->ldq, a->scale, a->stream);
}

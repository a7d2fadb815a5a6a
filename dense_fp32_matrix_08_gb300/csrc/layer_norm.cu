// Layer norm over the rows of x:
//   mean = sum x / n, var = sum (x - mean)^2 / n, rstd = 1 / sqrt(var + eps), y = (x - mean) rstd w + b
//
// Bound by HBM: each element is read and written once. A row stays in registers from its one read to
// its last use, so that the variance is the mean of the squared distances themselves: no difference
// of large sums. The FP32 sum of a row gives its mean m to at most 53 u mean|x| (u = 2^-24). Where that is not far
// below the spread (far_off), the distances from m, exact there, are added up for what m lacks, e = sum (x - m) / n,
// and the variance is taken again, from (x - m) - e: a constant row has var 0 and y = b.
//
// 8192 x 4096 BF16: 22.0 us, 6.1 TB/s, 90% of a copy's rate, issue slots 59% busy (pairs of FP32 numbers per
// instruction: one by one they were 71% busy and it took 32 us); FP32 41 us, 96%. With means of 10 times the spread
// 32 and 41 us (corrected for every row, of whatever mean, 25.5 and 41). 1 x 4096: 1.7 us. 16384 x 1024 BF16 11.7 us,
// 84%; 16384 x 512 7.1, 70%: the sums' exchanges weigh more there. 2048 x 16384 BF16 35.5 us, 56%: one row at a time
// per SM. Rows at any alignment come element by element: 8192 x 4095 BF16 40 us, 4096 x 12287 83 (72 without the
// correction's registers).
#include <algorithm>
#include <cmath>

#include "../../include/layer_norm.h"
#include "row_common.cuh"

namespace sgemm {
namespace ln {

using namespace rows;

struct Params {
  int rows, cols;
  const char *x;
  long long ldx;       // bytes
  Vector weight, bias;
  float eps, n, r;     // n = cols, r = 1 / n
  char *y;
  long long ldy;       // bytes
  float *mean, *rstd;
};

// CTAs of norm_kernel per SM: 768 threads with 80 registers each (one CTA for rows of 8193 to 12288 elements); 512 with
// 128 where a thread of a warp has 32 elements, 384 with 160 where these are FP32 (16384 x 1024 21.3 us, 23.1 with 512,
// whose registers spill); 1024 with 64 where it has 8, or aligned 16-bit rows have 6145 to 8192 elements, or rows more
// than 12288. FP32 rows of 6145 to 8192 elements and rows that are not aligned: one CTA of 512 (4096 x 8192 FP32 42 us,
// with two of them 46 to 55; BF16 24.8, with one 27.8).
template <class T, int TPR, int CH, bool VEC>
constexpr int kPerSm = TPR < 128    ? (CH > 2 ? (T::SIZE == 4 ? 3 : 4) : 6)
                       : CH == 1    ? 1024 / TPR
                       : TPR <= 384 ? 768 / TPR
                                    : (TPR == 512 && VEC && T::SIZE == 2 ? 2 : 1);
// Rows under way. More than it takes costs time: 8192 x 4096 FP32 takes 41.0 us with two, 46.7 with three, BF16
// 22.6 with three, 22.9 with four and 24.8 with two; where a row's bytes are few, or a CTA is alone on its SM, FP32
// rows need three as well (16384 x 1024: 21.5 us, 24.1 with two; 4096 x 8192: 42 and 45).
template <class T, int TPR, int CH>
constexpr int kDepth = T::SIZE == 4 && TPR * CH >= 256 && TPR != 512 ? 2 : 3;

// Whether the mean `near` may be off by what counts: where it is above 4 times the root of q, the mean square of the
// distances from it. (Below, it is off by at most 53 u (4 + 1) of the spread. Both may be 0: the squares of the
// smallest numbers are.)
__device__ __forceinline__ bool far_off(float near, float q) { return near * near >= 16.0f * q && q < INFINITY; }

// TPR threads on a row, CTAs of TPR (at least 128) threads that take rows in turn. The parameters of a
// thread's columns stay in its registers. 1024 threads have none for that: those of 16-bit rows lie in shared memory
// behind the ring, each thread's in places of its own (2048 x 16384 BF16 35.5 us, 45 where they are read from L2
// for each row); FP32 rows need the room for the ring.
template <class T, int TPR, bool VEC>
constexpr bool kShared = TPR == 1024 && VEC && T::SIZE == 2;
template <class T, int TPR, int CH, bool VEC>
constexpr int kRing = Ahead<T, TPR, CH, VEC, 1, kDepth<T, TPR, CH>, TPR < 128 ? 128 : TPR>::BYTES;
template <class T, int TPR, int CH, bool VEC>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR, kPerSm<T, TPR, CH, VEC>) norm_kernel(const Params p) {
  constexpr int THREADS = TPR < 128 ? 128 : TPR, RPB = THREADS / TPR;
  constexpr bool HOLD = TPR < 1024, SHARED = kShared<T, TPR, VEC>;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ __align__(16) RowSums<TPR, 1> sums, again;
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
  Two w[HOLD ? CH : 1][4], b[HOLD ? CH : 1][4];
  if constexpr (HOLD) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      parameters(p.weight, sh, c, n[c], 1.0f, w[c]);
      parameters(p.bias, sh, c, n[c], 0.0f, b[c]);
    }
  }
  ulonglong2 *mine = reinterpret_cast<ulonglong2 *>(ring + kRing<T, TPR, CH, VEC>) + threadIdx.x;
  if constexpr (SHARED) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      parameters(p.weight, sh, c, n[c], 1.0f, w[0]);
      parameters(p.bias, sh, c, n[c], 0.0f, b[0]);
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        mine[(c * 4 + i) * THREADS] = make_ulonglong2(w[0][i], w[0][i + 1]);
        mine[(c * 4 + i + 1) * THREADS] = make_ulonglong2(b[0][i], b[0][i + 1]);
      }
    }
  }
  char *to = p.y + row * p.ldy;
  for (; base < p.rows; base += step, row += step, to += step * p.ldy) {
    Chunk<T> in[1][CH];
    ahead.take(in);
    Two d[CH][4], total = 0;
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        d[c][i] = pair(in[0][c], i);
        total = add2(total, d[c][i]);
      }
    float s[1] = {sum2(total)};
    row_sum(s, sums, 0);
    float mean = over(s[0], p.n, p.r);
    const Two minus = both(-mean);
    total = 0;
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        d[c][i] = add2(d[c][i], minus);
        if (!ahead.whole) d[c][i] = first(d[c][i], i, n[c]);
        total = fma2(d[c][i], d[c][i], total);
      }
    s[0] = sum2(total);
    row_sum(s, sums, 1);
    float var = over(s[0], p.n, p.r);
    const bool off = far_off(mean, var);
    if (TPR < 32 ? __any_sync(0xffffffffu, off) : off) {  // (the same for a row's threads)
      total = 0;
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) total = add2(total, d[c][i]);
      s[0] = sum2(total);
      row_sum(s, again, 0);
      const float e = TPR >= 32 || off ? over(s[0], p.n, p.r) : 0.0f;  // (a warp's other rows keep what they have)
      mean += e;
      const Two rest = both(-e);
      total = 0;
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          d[c][i] = add2(d[c][i], rest);
          if (!ahead.whole) d[c][i] = first(d[c][i], i, n[c]);
          total = fma2(d[c][i], d[c][i], total);
        }
      s[0] = sum2(total);
      row_sum(s, again, 1);
      var = over(s[0], p.n, p.r);
    }
    // 1 / sqrt, with one step of Newton's iteration where it is neither 0 nor infinite
    const float v = var + p.eps;
    float rstd = rsqrtf(v);
    if (v > 0.0f && v < INFINITY) rstd = fmaf(0.5f * rstd, fmaf(-v * rstd, rstd, 1.0f), rstd);
    if (row < p.rows) {
      if (sh.t == 0) {
        if (p.mean) p.mean[row] = mean;
        if (p.rstd) p.rstd[row] = rstd;
      }
      const Two r2 = both(rstd);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        if constexpr (SHARED) {
#pragma unroll
          for (int i = 0; i < 4; i += 2) {
            const ulonglong2 wi = mine[(c * 4 + i) * THREADS], bi = mine[(c * 4 + i + 1) * THREADS];
            w[0][i] = wi.x, w[0][i + 1] = wi.y, b[0][i] = bi.x, b[0][i + 1] = bi.y;
          }
        } else if constexpr (!HOLD) {
          parameters(p.weight, sh, c, n[c], 1.0f, w[0]);
          parameters(p.bias, sh, c, n[c], 0.0f, b[0]);
        }
        Chunk<T> out;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          set_pair(out, i, fma2(mul2(d[c][i], r2), w[HOLD ? c : 0][i], b[HOLD ? c : 0][i]));
        sh.store(to, c, n[c], out);
      }
    }
  }
  if (!once) griddep_launch_dependents();
}

// Rows of any length: a CTA reads its row three times (for the mean, the variance and the result; from
// caches after the first). 8 elements at a time are added up in FP32, the rest as Long. With 64-bit sums
// 2048 x 16392 BF16 took 450 us, most of it in the CTA-wide ones.
template <class T, bool VEC>
__global__ void __launch_bounds__(1024) norm_long_kernel(const Params p) {
  __shared__ Long part[2][32];
  __shared__ float told[4];
  griddep_launch_dependents();
  griddep_wait();
  for (long long row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const char *x = p.x + row * p.ldx;
    Long total;
    blocks<T, 1024, VEC>(p.cols, [&](const auto &sh, long long at) {
      Chunk<T> v;
      sh.load(x + at * T::SIZE, 0, sh.count(0), v);
      Two s = pair(v, 0);
#pragma unroll
      for (int i = 1; i < 4; ++i) s = add2(s, pair(v, i));
      total.add(sum2(s));
    });
    total = cta_sum(total, part[0]);
    if (threadIdx.x == 0) told[0] = total.over(p.cols);
    __syncthreads();
    const float near = told[0];
    const Two minus = both(-near);
    float e = 0.0f;
    // (x - near) - e, or its square, of 8 elements at a time
    const auto distances = [&](bool squares) {
      Long sum;
      const Two rest = both(-e);
      blocks<T, 1024, VEC>(p.cols, [&](const auto &sh, long long at) {
        const int n = sh.count(0);
        Chunk<T> v;
        sh.load(x + at * T::SIZE, 0, n, v);
        Two s = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const Two d = first(add2(add2(pair(v, i), minus), rest), i, n);
          s = squares ? fma2(d, d, s) : add2(d, s);
        }
        sum.add(sum2(s));
      });
      return sum;
    };
    total = cta_sum(distances(true), part[1]);
    if (threadIdx.x == 0) told[1] = total.over(p.cols);
    __syncthreads();
    float var = told[1];
    if (far_off(near, var)) {
      total = cta_sum(distances(false), part[0]);
      if (threadIdx.x == 0) told[2] = total.over(p.cols);
      __syncthreads();
      e = told[2];
      total = cta_sum(distances(true), part[1]);
      if (threadIdx.x == 0) told[3] = total.over(p.cols);
      __syncthreads();
      var = told[3];
    }
    const float rstd = __frsqrt_rn(var + p.eps);
    if (threadIdx.x == 0) {
      if (p.mean) p.mean[row] = near + e;
      if (p.rstd) p.rstd[row] = rstd;
    }
    char *y = p.y + row * p.ldy;
    const Two rest = both(-e), r2 = both(rstd);
    blocks<T, 1024, VEC>(p.cols, [&](const auto &sh, long long at) {
      const int n = sh.count(0);
      Chunk<T> v, out;
      sh.load(x + at * T::SIZE, 0, n, v);
      Two w[4], b[4];
      parameters(from(p.weight, at), sh, 0, n, 1.0f, w);
      parameters(from(p.bias, at), sh, 0, n, 0.0f, b);
#pragma unroll
      for (int i = 0; i < 4; ++i) set_pair(out, i, fma2(mul2(add2(add2(pair(v, i), minus), rest), r2), w[i], b[i]));
      sh.store(y + at * T::SIZE, 0, n, out);
    });
  }
}

template <class T, int TPR, int CH, bool VEC>
static cudaError_t launch(const Params &p, int sms, cudaStream_t stream) {
  constexpr int threads = TPR < 128 ? 128 : TPR, rpb = threads / TPR;
  constexpr int bytes = kRing<T, TPR, CH, VEC> + (kShared<T, TPR, VEC> ? 2 * CH * 8 * 4 * threads : 0);
  static cudaError_t set[kDevices];
  static std::once_flag once[kDevices];
  const cudaError_t e = allow_bytes(norm_kernel<T, TPR, CH, VEC>, bytes, once, set);
  if (e != cudaSuccess) return e;
  const long long grid = std::min<long long>(ceil_div(p.rows, rpb), (long long)sms * kPerSm<T, TPR, CH, VEC>);
  return launch_1d(norm_kernel<T, TPR, CH, VEC>, (int)grid, threads, bytes, 1, stream, p);
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
  // (a warp per row needs no barrier, but aligned rows for its registers: 16384 x 1024 BF16 15.1 us with 128
  // threads on a row, 11.7 so. Rows that come element by element have 8 of them per thread where that is faster: 16384
  // x 1023 BF16 18.2 us, with 768 threads per SM 22.8; 8192 x 4095 BF16 40.2, with 16 per thread 43.2, but FP32 48.6
  // and 47.7.)
  if (p.cols <= 1024) return vec ? launch<T, 32, 4, true>(p, sms, stream) : launch<T, 128, 1, false>(p, sms, stream);
  if constexpr (T::SIZE == 2) {
    if (!vec && p.cols <= 2048) return launch<T, 256, 1, false>(p, sms, stream);
    if (!vec && p.cols <= 4096) return launch<T, 512, 1, false>(p, sms, stream);
    if (p.cols <= 2048) return launch<T, 128, 2, true>(p, sms, stream);
    if (p.cols <= 4096) return launch<T, 256, 2, true>(p, sms, stream);
  } else {
    if (p.cols <= 2048) return launch<T, 128, 2>(p, vec, sms, stream);
    if (p.cols <= 4096) return launch<T, 256, 2>(p, vec, sms, stream);
  }
  if (p.cols <= 6144) return launch<T, 384, 2>(p, vec, sms, stream);
  if (p.cols <= 8192) return launch<T, 512, 2>(p, vec, sms, stream);
  if (p.cols <= 12288) return launch<T, 768, 2>(p, vec, sms, stream);
  if (p.cols <= kLongest) return launch<T, 1024, 2>(p, vec, sms, stream);
  return launch_1d(vec ? norm_long_kernel<T, true> : norm_long_kernel<T, false>, std::min(p.rows, 2 * sms), 1024, 0,
                   1, stream, p);
}

}  // namespace ln
}  // namespace sgemm

using namespace sgemm;

extern "C" int layer_norm(int rows, int cols, const void *x, int x_type, int ldx, const void *weight,
                          const void *bias, int w_type, float eps, void *y, int ldy, float *mean,
                          float *rstd, cudaStream_t stream) {
  const auto known = [](int t) { return t == LN_F32 || t == LN_BF16 || t == LN_F16; };
  const auto misplaced = [](const void *q, int t) {
    return reinterpret_cast<uintptr_t>(q) % (t == LN_F32 ? 4 : 2) != 0;
  };
  if (rows < 0) return -1;
  if (cols < 1) return -2;
  if (rows > 0 && x == nullptr) return -3;
  if (!known(x_type)) return -4;
  if (misplaced(x, x_type)) return -3;
  if (ldx < cols) return -5;
  if (!known(w_type)) return -8;
  if (misplaced(weight, w_type)) return -6;
  if (misplaced(bias, w_type)) return -7;
  if (!(eps >= 0.0f) || std::isinf(eps)) return -9;
  if (rows > 0 && y == nullptr) return -10;
  if (misplaced(y, x_type)) return -10;
  if (ldy < cols) return -11;
  if (misplaced(mean, LN_F32)) return -12;
  if (misplaced(rstd, LN_F32)) return -13;
  if (rows == 0) return 0;
  int sms = 0;
  const cudaError_t e = device_setup(&sms);
  if (e != cudaSuccess) return (int)e;
  const long long size = x_type == LN_F32 ? 4 : 2;
  ln::Params p{};
  p.rows = rows;
  p.cols = cols;
  p.x = static_cast<const char *>(x);
  p.ldx = ldx * size;
  p.weight = {weight, w_type, reinterpret_cast<uintptr_t>(weight) % 16 == 0};
  p.bias = {bias, w_type, reinterpret_cast<uintptr_t>(bias) % 16 == 0};
  p.eps = eps;
  p.n = (float)cols;
  p.r = 1.0f / p.n;
  p.y = static_cast<char *>(y);
  p.ldy = ldy * size;
  p.mean = mean;
  p.rstd = rstd;
  const bool vec = rows::aligned(reinterpret_cast<uintptr_t>(x), rows > 1 ? p.ldx : 0) &&
                   rows::aligned(reinterpret_cast<uintptr_t>(y), rows > 1 ? p.ldy : 0);
  if (x_type == LN_F32) return (int)ln::run<rows::F32>(p, vec, sms, stream);
  if (x_type == LN_BF16) return (int)ln::run<rows::BF16>(p, vec, sms, stream);
  return (int)ln::run<rows::F16>(p, vec, sms, stream);
}

extern "C" int layer_norm_with(const layer_norm_args *a) {
  if (a == nullptr) return -1;
  return layer_norm(a->rows, a->cols, a->x, a->x_type, a->ldx, a->weight, a->bias, a->w_type, a->eps,
                    a->y, a->ldy, a->mean, a->rstd, a->stream);
}

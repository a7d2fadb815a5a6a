// Gradients of layer norm. With h = (x - mean) rstd and g = dy w, along each row of n elements
//   dx = rstd (g - sum g / n - h sum (g h) / n)
// and over the rows dw = sum dy h, db = sum dy.
//
// Bound by HBM: dy and x are read and dx is written once. A row stays in registers between its two
// sums and its result. dw and db are added up in the registers of the thread that holds the column,
// over all rows that it gets (500 at most, so that FP32 holds such a sum); those of a CTA meet in shared
// memory, the CTAs' sums in the workspace, where reduce_kernel adds them in a fixed order.
// 8192 x 4096 BF16: 39.7 us, 5.1 TB/s. Without dw and db 34.2 (87% of a copy's rate): the sums' registers
// leave 16 warps per SM, issue slots 50% busy; the rest is the sums' way. FP32: 63 us, 6.4 TB/s (94%).
// 4099 x 777 FP32: 12.5, of which 3.5 are for the sums; its rows are not aligned, so that they come element by
// element. Longer rows than registers hold are read twice: 2048 x 16384 FP32 128 us (BF16, in registers, 72).
#include <algorithm>
#include <cmath>

#include "../../include/layer_norm.h"
#include "row_common.cuh"

namespace sgemm {
namespace lnb {

using namespace rows;

constexpr int kMostRows = 500;  // rows that a thread adds up in FP32
// Elements of a row that stays in registers beside the sums: any, and 16-bit ones that are aligned.
constexpr int kLongestHere = 12288, kLongestPacked = kLongest;

struct Params {
  int rows, cols;
  const char *dy, *x;
  long long lddy, ldx;      // bytes
  const float *mean, *rstd;
  Vector weight;
  float n, r;               // cols, 1 / cols
  char *dx;
  long long lddx;           // bytes
  float *part;              // sums of dw, then of db: [2][parts][pitch]; NULL: neither is wanted
  int parts;
  long long pitch;          // cols rounded up to a multiple of 4
  float2 *along;            // rows that do not stay in registers: sum g / n, sum (g h) / n
};

// One CTA of 512 threads per SM, with up to 128 registers each (768 with 80, 1024 with 64 for the longest rows): as
// many rows at a time as that makes, and one sum of each column per SM.
template <int TPR>
constexpr int kThreads = TPR > 512 ? TPR : 512;
// Rows under way. More than it takes costs time: 8192 x 4096 FP32 63 us with two, 66 with three; FP32 rows of 1024
// and less are short enough for three (16384 x 1024 36.5 us, 38.3 with two); BF16 40.0 with three, 41.0 with two.
// (Three of 16384 16-bit elements have no room.)
template <class T, int TPR, int CH>
constexpr int kDepth = (T::SIZE == 4 && TPR * CH >= 256) || TPR == 1024 ? 2 : 3;

// Whether the weight of a thread's columns lies in shared memory, in places of the thread's own, instead of registers:
// for rows of 8193 elements and more, where it fits. (4096 x 12288 BF16 77 us, 93 with it in registers that spill, 149
// with the rows read twice. FP32 142, with registers that spill: read again from L2 for each row 152, rows read
// twice 208.)
template <class T, int TPR, bool VEC>
constexpr bool kShared = TPR > 512 && VEC && T::SIZE == 2;

// Dynamic shared memory: the ring of rows to come and behind it such a weight; at the end the sums of the CTA's rows.
template <class T, int TPR, int CH, bool VEC>
constexpr int kRing = Ahead<T, TPR, CH, VEC, 2, kDepth<T, TPR, CH>, kThreads<TPR>>::BYTES;
template <class T, int TPR, int CH, bool VEC>
constexpr int kBytes = std::max(kRing<T, TPR, CH, VEC> + (kShared<T, TPR, VEC> ? TPR * CH * 8 * 4 : 0),
                                TPR < kThreads<TPR> ? kThreads<TPR> * 2 * CH * 8 * 4 : 0);

template <class T, int TPR, int CH, bool VEC>
__global__ void __launch_bounds__(kThreads<TPR>, 1) backward_kernel(const Params p) {
  constexpr int RPB = kThreads<TPR> / TPR;
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ __align__(16) RowSums<TPR, 2, RPB> sums;
  const long long step = (long long)gridDim.x * RPB;
  long long base = (long long)blockIdx.x * RPB;  // (the same for a whole CTA)
  long long row = base + threadIdx.x / TPR;
  Ahead<T, TPR, CH, VEC, 2, kDepth<T, TPR, CH>, kThreads<TPR>> ahead(p.cols, ring, {p.x, p.dy}, {p.ldx, p.lddy},
                                                                      p.rows, row, step);
  const auto &sh = ahead.sh;
  const auto &n = ahead.n;
  griddep_wait();  // (launched with programmatic dependent launch: see launch_1d)
  ahead.begin();
  float next_mean = row < p.rows ? p.mean[row] : 0.0f, next_rstd = row < p.rows ? p.rstd[row] : 0.0f;
  constexpr bool SHARED = kShared<T, TPR, VEC>;
  Two held[SHARED ? 1 : CH][4], dw[CH][4], db[CH][4];
  ulonglong2 *mine = reinterpret_cast<ulonglong2 *>(ring + kRing<T, TPR, CH, VEC>) + threadIdx.x;
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    Two(&w)[4] = held[SHARED ? 0 : c];
    parameters(p.weight, sh, c, n[c], 1.0f, w);
    if constexpr (SHARED) {
      mine[2 * c * TPR] = make_ulonglong2(w[0], w[1]);
      mine[(2 * c + 1) * TPR] = make_ulonglong2(w[2], w[3]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) dw[c][i] = db[c][i] = 0;
  }
  // The weight of chunk c: w[i] of its elements 2 i and 2 i + 1.
  const auto weight = [&](int c, Two (&w)[4]) {
    if constexpr (SHARED) {
      const ulonglong2 a = mine[2 * c * TPR], b = mine[(2 * c + 1) * TPR];
      w[0] = a.x, w[1] = a.y, w[2] = b.x, w[3] = b.y;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = held[c][i];
    }
  };
  char *to = p.dx + row * p.lddx;
  int turn = 0;
  for (; base < p.rows; base += step, row += step, to += step * p.lddx, turn ^= 1) {
    Chunk<T> v[2][CH];
    ahead.take(v);
    const float mean = next_mean, rstd = next_rstd;
    next_mean = row + step < p.rows ? p.mean[row + step] : 0.0f;
    next_rstd = row + step < p.rows ? p.rstd[row + step] : 0.0f;
    const bool in = row < p.rows;
    const Two minus = both(-mean), r2 = both(rstd);
    float s[2] = {0.0f, 0.0f};
    // h and g stay in registers between the two passes where there is room for them
    constexpr bool KEEP = VEC && T::SIZE == 2 && TPR <= 512;
    Two kept[KEEP ? CH : 1][4][2];
    if (in) {
      Two sg = 0, sgh = 0;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        Two w[4];
        weight(c, w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // (elements that do not exist have dy = 0, so they add nothing where rstd and mean are finite,
          // and where those are not the row is NaN anyway)
          const Two d = pair(v[1][c], i), h = mul2(add2(pair(v[0][c], i), minus), r2), g = mul2(d, w[i]);
          dw[c][i] = fma2(d, h, dw[c][i]);
          db[c][i] = add2(db[c][i], d);
          sg = add2(sg, g);
          sgh = fma2(g, h, sgh);
          if constexpr (KEEP) kept[c][i][0] = h, kept[c][i][1] = g;
        }
      }
      s[0] = sum2(sg);
      s[1] = sum2(sgh);
    }
    if (p.dx == nullptr) continue;
    row_sum(s, sums, turn);
    if (in) {
      const Two s1 = both(-over(s[0], p.n, p.r)), s2 = both(-over(s[1], p.n, p.r));
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        Chunk<T> out;
        Two w[4];
        if constexpr (!KEEP) weight(c, w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          Two h, g;
          if constexpr (KEEP) {
            h = kept[c][i][0];
            g = add2(kept[c][i][1], s1);
          } else {
            h = mul2(add2(pair(v[0][c], i), minus), r2);
            g = fma2(pair(v[1][c], i), w[i], s1);
          }
          set_pair(out, i, mul2(fma2(h, s2, g), r2));
        }
        sh.store(to, c, n[c], out);
      }
    }
  }
  if (p.part) {
    float f[2][CH][8];
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 a = unpack2(dw[c][i]), e = unpack2(db[c][i]);
        f[0][c][2 * i] = a.x, f[0][c][2 * i + 1] = a.y, f[1][c][2 * i] = e.x, f[1][c][2 * i + 1] = e.y;
      }
    // four sums of chunk c from j on, to the workspace (element by element 8192 x 4096 BF16 took 7 us more)
    const auto leave = [&](int which, int c, int j, int have, const Share<T, TPR, VEC> &at, const float4 &v) {
      float *out = p.part + ((long long)which * p.parts + blockIdx.x) * p.pitch;
      const float u[4] = {v.x, v.y, v.z, v.w};
      if (VEC && j + 4 <= have) {
        *reinterpret_cast<float4 *>(out + at.col(c, j)) = v;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (j + i < have) out[at.col(c, j + i)] = u[i];
      }
    };
    if constexpr (TPR == kThreads<TPR>) {
#pragma unroll
      for (int which = 0; which < 2; ++which)
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
          for (int j = 0; j < 8; j += 4)
            leave(which, c, j, n[c], sh, make_float4(f[which][c][j], f[which][c][j + 1], f[which][c][j + 2],
                                                     f[which][c][j + 3]));
    } else {
      // those of the rows that the CTA had at a time: within warps, then from all of them
      constexpr int U = TPR < 32 ? 32 : TPR, UNITS = kThreads<TPR> / U;
      cp_async_wait<0>();
      __syncthreads();  // (the ring is done with)
      float4 *meet = reinterpret_cast<float4 *>(ring);  // [which][c][j / 4][unit][thread]
      const int unit = threadIdx.x / U, t = threadIdx.x % U;
#pragma unroll
      for (int which = 0; which < 2; ++which)
#pragma unroll
        for (int c = 0; c < CH; ++c) {
#pragma unroll
          for (int d = TPR; d < 32; d *= 2)
#pragma unroll
            for (int j = 0; j < 8; ++j) f[which][c][j] += __shfl_xor_sync(0xffffffffu, f[which][c][j], d);
#pragma unroll
          for (int j = 0; j < 8; j += 4)
            meet[(((which * CH + c) * 2 + j / 4) * UNITS + unit) * U + t] =
                make_float4(f[which][c][j], f[which][c][j + 1], f[which][c][j + 2], f[which][c][j + 3]);
        }
      __syncthreads();
      for (int i = threadIdx.x; i < 2 * CH * 2 * U; i += kThreads<TPR>) {
        const int t2 = i % U, k = i / U, which = k / (2 * CH), c = k / 2 % CH, j = k % 2 * 4;
        if (t2 >= TPR) continue;  // (a narrow row's other copies)
        float4 v = meet[k * UNITS * U + t2];
#pragma unroll
        for (int q = 1; q < UNITS; ++q) {
          const float4 u = meet[(k * UNITS + q) * U + t2];
          v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
        }
        const Share<T, TPR, VEC> at{p.cols, t2};
        leave(which, c, j, at.count(c), at, v);
      }
    }
  }
  griddep_launch_dependents();
}

// Rows of any length, first half: the two sums along each row, 8 elements at a time in FP32, the rest as
// Long.
template <class T, bool VEC>
__global__ void __launch_bounds__(1024) along_kernel(const Params p) {
  __shared__ Long part[2][2][32];
  griddep_wait();
  int turn = 0;
  for (long long row = blockIdx.x; row < p.rows; row += gridDim.x, turn ^= 1) {
    const char *x = p.x + row * p.ldx, *dy = p.dy + row * p.lddy;
    const Two minus = both(-p.mean[row]), r2 = both(p.rstd[row]);
    Long a, b;
    blocks<T, 1024, VEC>(p.cols, [&](const auto &sh, long long at) {
      const int n = sh.count(0);
      Chunk<T> vx, vd;
      sh.load(x + at * T::SIZE, 0, n, vx);
      sh.load(dy + at * T::SIZE, 0, n, vd);
      Two w[4], sa = 0, sb = 0;
      parameters(rows::from(p.weight, at), sh, 0, n, 1.0f, w);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const Two g = mul2(pair(vd, i), w[i]);
        sa = add2(sa, g);
        sb = fma2(g, mul2(add2(pair(vx, i), minus), r2), sb);
      }
      a.add(sum2(sa));
      b.add(sum2(sb));
    });
    a = cta_sum(a, part[turn][0]);
    b = cta_sum(b, part[turn][1]);
    if (threadIdx.x == 0) p.along[row] = make_float2(a.over(p.cols), b.over(p.cols));
  }
  griddep_launch_dependents();
}

// Second half: CTA (i, j) takes 2048 columns of the j-th part of the rows.
constexpr int kLongCols = 2048;
template <class T, bool VEC>
__global__ void __launch_bounds__(256) across_kernel(const Params p, int col_blocks, int rows_each) {
  griddep_wait();
  const int block = blockIdx.x % col_blocks, chunk = blockIdx.x / col_blocks;
  const long long c0 = (long long)block * kLongCols;
  const Share<T, 256, VEC> sh{(int)min(p.cols - c0, (long long)kLongCols), (int)threadIdx.x};
  const int n = sh.count(0);
  const long long r0 = (long long)chunk * rows_each;
  const long long r1 = r0 + rows_each < p.rows ? r0 + rows_each : p.rows;
  Two w[4], dw[4] = {}, db[4] = {};
  parameters(rows::from(p.weight, c0), sh, 0, n, 1.0f, w);
#pragma unroll 2
  for (long long row = r0; row < r1; ++row) {
    Chunk<T> vx, vd, out;
    sh.load(p.x + row * p.ldx + c0 * T::SIZE, 0, n, vx);
    sh.load(p.dy + row * p.lddy + c0 * T::SIZE, 0, n, vd);
    const float2 s = p.dx ? p.along[row] : make_float2(0.0f, 0.0f);
    const Two minus = both(-p.mean[row]), r2 = both(p.rstd[row]), s1 = both(-s.x), s2 = both(-s.y);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const Two d = pair(vd, i), h = mul2(add2(pair(vx, i), minus), r2);
      dw[i] = fma2(d, h, dw[i]);
      db[i] = add2(db[i], d);
      set_pair(out, i, mul2(fma2(h, s2, fma2(d, w[i], s1)), r2));
    }
    if (p.dx) sh.store(p.dx + row * p.lddx + c0 * T::SIZE, 0, n, out);
  }
  if (p.part) {
    float *to = p.part + chunk * p.pitch + c0, *tb = to + p.parts * p.pitch;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = unpack2(dw[i]), e = unpack2(db[i]);
      if (2 * i < n) to[sh.col(0, 2 * i)] = a.x, tb[sh.col(0, 2 * i)] = e.x;
      if (2 * i + 1 < n) to[sh.col(0, 2 * i + 1)] = a.y, tb[sh.col(0, 2 * i + 1)] = e.y;
    }
  }
  griddep_launch_dependents();
}

// dweight (block < blocks) or dbias: 32 columns per CTA, its 8 warps take the parts in turn, 16 of them at
// a time in FP32 and the rest in 64 bits. With the parts' way to L2 5 us of the 41 of 8192 x 4096 BF16.
// (CTAs of 32 warps took 7 us longer.)
constexpr int kReduceWarps = 8;
__global__ void __launch_bounds__(32 * kReduceWarps)
    reduce_kernel(const float *part, int parts, int cols, long long pitch, int blocks, float *dweight,
                  float *dbias, float beta) {
  __shared__ double sums[kReduceWarps][32];
  griddep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool second = (int)blockIdx.x >= blocks;
  const long long col = (long long)(blockIdx.x - (second ? blocks : 0)) * 32 + lane;
  float *out = second ? dbias : dweight;
  if (out == nullptr) return;
  double total = 0.0;
  if (col < cols) {
    const float *from = part + (second ? parts * pitch : 0) + col;
    for (int r0 = warp; r0 < parts; r0 += 16 * kReduceWarps) {
      float v[16], s = 0.0f;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int r = r0 + kReduceWarps * j;
        v[j] = r < parts ? from[r * pitch] : 0.0f;
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) s += v[j];
      total += s;
    }
  }
  sums[warp][lane] = total;
  __syncthreads();
  if (warp == 0 && col < cols) {
#pragma unroll
    for (int w = 1; w < kReduceWarps; ++w) total += sums[w][lane];
    out[col] = beta != 0.0f ? (float)((double)beta * out[col] + total) : (float)total;
  }
  griddep_launch_dependents();
}

// ------------------------------------------------------------------------------------
// Host side

struct Plan {
  int tpr;          // threads on a row; 0: rows do not stay in registers
  int grid, parts;  // CTAs and sums of dw that they leave
  int rows_each;    // (tpr == 0) rows of a sum
};

// Threads on a row; 0: rows do not stay in registers. A thread with 16 elements waits as long for its row's sums as
// one with 8: 16384 x 1024 BF16 26.9 us with 128 threads on a row, 22.5 with 64; 4099 x 777 BF16, element by element,
// 17.0 and 13.8. `one_by_one`: FP32 rows that are not aligned, which come element by element and with 16 of them take
// more registers than there are: 4099 x 777 12.6 us with 128 threads, 17.8 with 64; 8192 x 4095 80 with 512, 135 with
// 256. `packed`: 16-bit rows that are aligned, of which 1024 threads hold the longest ones, with registers that
// spill: 2048 x 16384 72 us, read twice 96.
static int threads_on(int cols, bool one_by_one, bool packed) {
  const int more = one_by_one ? 2 : 1;
  return cols <= 64     ? 8
         : cols <= 256  ? 32
         : cols <= 512  ? 32 * more
         : cols <= 1024 ? 64 * more
         : cols <= 2048 ? 128 * more
         : cols <= 4096 ? 256 * more
         : cols <= 8192 ? 512
         : cols <= kLongestHere ? 768
         : cols <= kLongestPacked && packed ? 1024 : 0;
}

static Plan make_plan(int rows, int cols, int tpr, int sms) {
  Plan pl{tpr};
  if (tpr) {
    const long long most = ceil_div(rows, tpr > 512 ? 1 : 512 / tpr);
    pl.grid = (int)std::min<long long>(most, std::max<long long>(sms, ceil_div(most, kMostRows)));
    pl.parts = pl.grid;
  } else {
    const long long blocks = ceil_div(cols, kLongCols);
    pl.rows_each = (int)std::max<long long>(1, std::min<long long>(kMostRows, rows * blocks / (8LL * sms)));
    pl.parts = (int)ceil_div(rows, pl.rows_each);
  }
  return pl;
}

static size_t along_bytes(const Plan &pl, int rows) {
  return pl.tpr ? 0 : ((size_t)rows * sizeof(float2) + 255) / 256 * 256;
}
static long long pitch_of(int cols) { return ceil_div(cols, 4) * 4; }
static size_t part_bytes(const Plan &pl, int cols) { return (size_t)2 * pl.parts * pitch_of(cols) * sizeof(float); }

template <class T, int TPR, int CH, bool VEC>
static cudaError_t launch(const Params &p, int grid, cudaStream_t stream) {
  constexpr int bytes = kBytes<T, TPR, CH, VEC>;
  static cudaError_t set[kDevices];
  static std::once_flag once[kDevices];
  const cudaError_t e = allow_bytes(backward_kernel<T, TPR, CH, VEC>, bytes, once, set);
  return e != cudaSuccess ? e : launch_1d(backward_kernel<T, TPR, CH, VEC>, grid, kThreads<TPR>, bytes, 1, stream, p);
}
template <class T, int TPR, int CH>
static cudaError_t launch(const Params &p, bool vec, int grid, cudaStream_t stream) {
  return vec ? launch<T, TPR, CH, true>(p, grid, stream) : launch<T, TPR, CH, false>(p, grid, stream);
}

template <class T>
static cudaError_t run(const Params &p, const Plan &pl, bool vec, int sms, cudaStream_t stream) {
  if (p.cols <= 64) return launch<T, 8, 1>(p, vec, pl.grid, stream);
  if (p.cols <= 256) return launch<T, 32, 1>(p, vec, pl.grid, stream);
  if (p.cols <= 4096) {
    if constexpr (T::SIZE == 4) {
      switch (vec ? 0 : pl.tpr) {
        case 64: return launch<T, 64, 1, false>(p, pl.grid, stream);
        case 128: return launch<T, 128, 1, false>(p, pl.grid, stream);
        case 256: return launch<T, 256, 1, false>(p, pl.grid, stream);
        case 512: return launch<T, 512, 1, false>(p, pl.grid, stream);
      }
      switch (pl.tpr) {
        case 32: return launch<T, 32, 2, true>(p, pl.grid, stream);
        case 64: return launch<T, 64, 2, true>(p, pl.grid, stream);
        case 128: return launch<T, 128, 2, true>(p, pl.grid, stream);
        default: return launch<T, 256, 2, true>(p, pl.grid, stream);
      }
    } else {
      switch (pl.tpr) {
        case 32: return launch<T, 32, 2>(p, vec, pl.grid, stream);
        case 64: return launch<T, 64, 2>(p, vec, pl.grid, stream);
        case 128: return launch<T, 128, 2>(p, vec, pl.grid, stream);
        default: return launch<T, 256, 2>(p, vec, pl.grid, stream);
      }
    }
  }
  if (p.cols <= 8192) return launch<T, 512, 2>(p, vec, pl.grid, stream);
  if (p.cols <= kLongestHere) return launch<T, 768, 2>(p, vec, pl.grid, stream);
  if constexpr (T::SIZE == 2) {
    if (pl.tpr == 1024) return launch<T, 1024, 2, true>(p, pl.grid, stream);
  }
  if (p.dx) {
    const cudaError_t e = launch_1d(vec ? along_kernel<T, true> : along_kernel<T, false>, std::min(p.rows, 2 * sms),
                                    1024, 0, 1, stream, p);
    if (e != cudaSuccess) return e;
  }
  const long long blocks = ceil_div(p.cols, kLongCols), grid = blocks * pl.parts;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  return launch_1d(vec ? across_kernel<T, true> : across_kernel<T, false>, (int)grid, 256, 0, 1, stream, p, (int)blocks,
                   pl.rows_each);
}

}  // namespace lnb
}  // namespace sgemm

using namespace sgemm;

extern "C" int layer_norm_backward_workspace_size(int rows, int cols, size_t *bytes) {
  if (rows < 0) return -1;
  if (cols < 1) return -2;
  if (bytes == nullptr) return 0;
  *bytes = 0;
  if (rows == 0) return 0;
  int sms = 0;
  if (device_setup(&sms) != cudaSuccess) {
    (void)cudaGetLastError();
    sms = 152;  // no device here: the answer for a whole GB300
  }
  // (the more threads on a row, the more sums; rows that are read twice leave as many as any)
  const lnb::Plan pl = lnb::make_plan(rows, cols, lnb::threads_on(cols, true, false), sms);
  *bytes = lnb::along_bytes(pl, rows) + lnb::part_bytes(pl, cols);
  return 0;
}

extern "C" int layer_norm_backward(int rows, int cols, const void *dy, int lddy, const void *x,
                                   int x_type, int ldx, const float *mean, const float *rstd,
                                   const void *weight, int w_type, void *dx, int lddx, float *dweight,
                                   float *dbias, float beta, cudaStream_t stream) {
  const auto known = [](int t) { return t == LN_F32 || t == LN_BF16 || t == LN_F16; };
  const auto misplaced = [](const void *q, int t) {
    return reinterpret_cast<uintptr_t>(q) % (t == LN_F32 ? 4 : 2) != 0;
  };
  if (rows < 0) return -1;
  if (cols < 1) return -2;
  if (rows > 0 && dy == nullptr) return -3;
  if (lddy < cols) return -4;
  if (rows > 0 && x == nullptr) return -5;
  if (!known(x_type)) return -6;
  if (misplaced(dy, x_type)) return -3;
  if (misplaced(x, x_type)) return -5;
  if (ldx < cols) return -7;
  if ((rows > 0 && mean == nullptr) || misplaced(mean, LN_F32)) return -8;
  if ((rows > 0 && rstd == nullptr) || misplaced(rstd, LN_F32)) return -9;
  if (!known(w_type)) return -11;
  if (misplaced(weight, w_type)) return -10;
  if (misplaced(dx, x_type)) return -12;
  if (dx != nullptr && lddx < cols) return -13;
  if (misplaced(dweight, LN_F32)) return -14;
  if (misplaced(dbias, LN_F32)) return -15;
  if (dx == nullptr && dweight == nullptr && dbias == nullptr) return 0;
  const bool sums = dweight != nullptr || dbias != nullptr;
  if (rows == 0 && (!sums || beta == 1.0f)) return 0;
  int sms = 0;
  cudaError_t e = device_setup(&sms);
  if (e != cudaSuccess) return (int)e;
  const int blocks = (int)ceil_div(cols, 32);
  if (rows == 0)
    return (int)launch_1d(lnb::reduce_kernel, 2 * blocks, 32 * lnb::kReduceWarps, 0, 1, stream,
                          static_cast<const float *>(nullptr), 0, cols, 0LL, blocks, dweight, dbias, beta);
  const long long size = x_type == LN_F32 ? 4 : 2;
  lnb::Params p{};
  p.rows = rows;
  p.cols = cols;
  p.dy = static_cast<const char *>(dy);
  p.lddy = lddy * size;
  p.x = static_cast<const char *>(x);
  p.ldx = ldx * size;
  p.mean = mean;
  p.rstd = rstd;
  p.weight = {weight, w_type, reinterpret_cast<uintptr_t>(weight) % 16 == 0};
  p.n = (float)cols;
  p.r = 1.0f / p.n;
  p.dx = static_cast<char *>(dx);
  p.lddx = lddx * size;
  const auto at = [](const void *q) { return reinterpret_cast<uintptr_t>(q); };
  const bool vec = rows::aligned(at(dy), rows > 1 ? p.lddy : 0) &&
                   rows::aligned(at(x), rows > 1 ? p.ldx : 0) &&
                   (dx == nullptr || rows::aligned(at(dx), rows > 1 ? p.lddx : 0));
  const int tpr = lnb::threads_on(cols, size == 4 && !vec, size == 2 && vec);
  const lnb::Plan pl = lnb::make_plan(rows, cols, tpr, sms);
  p.parts = pl.parts;
  p.pitch = lnb::pitch_of(cols);
  const size_t along = dx ? lnb::along_bytes(pl, rows) : 0;
  const size_t bytes = along + (sums ? lnb::part_bytes(pl, cols) : 0);
  char *ws = nullptr;
  if (bytes > 0) {
    e = cudaMallocFromPoolAsync(reinterpret_cast<void **>(&ws), bytes, workspace_pool(), stream);
    if (e != cudaSuccess) return (int)e;
    p.along = reinterpret_cast<float2 *>(ws);
    if (sums) p.part = reinterpret_cast<float *>(ws + along);
  }
  e = x_type == LN_F32    ? lnb::run<rows::F32>(p, pl, vec, sms, stream)
      : x_type == LN_BF16 ? lnb::run<rows::BF16>(p, pl, vec, sms, stream)
                          : lnb::run<rows::F16>(p, pl, vec, sms, stream);
  if (e == cudaSuccess && sums)
    e = launch_1d(lnb::reduce_kernel, 2 * blocks, 32 * lnb::kReduceWarps, 0, 1, stream,
                  static_cast<const float *>(p.part), pl.parts, cols, p.pitch, blocks, dweight, dbias, beta);
  if (ws != nullptr) {
    const cudaError_t ef = cudaFreeAsync(ws, stream);
    if (e == cudaSuccess) e = ef;
  }
  return (int)e;
}

extern "C" int layer_norm_backward_with(const layer_norm_backward_args *a) {
  if (a == nullptr) return -1;
  return layer_norm_backward(a->rows, a->cols, a->dy, a->lddy, a->x, a->x_type, a->ldx, a->mean, a->rstd,
                             a->weight, a->w_type, a->dx, a->lddx, a->dweight, a->dbias, a->beta,
                             a->stream);
}

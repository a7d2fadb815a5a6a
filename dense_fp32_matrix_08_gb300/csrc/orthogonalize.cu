// Orthogonalising a matrix by Newton-Schulz products on the 5th-generation tensor cores:
//   X_0 = G / (|G|_F + eps);  X <- a X + (b S + c S^2) X, S = X X^T, `steps` times
// on the orientation with fewer rows (m x n, m <= n).
//
// FP32 fidelity on FP16 tensor cores. Every matrix is kept as hi + lo, two FP16 numbers: hi = the
// value rounded to 11 bits, lo = the remainder, so hi + lo carries 22 bits, and a product is
// hi hi' + hi lo' + lo hi' (lo lo' is 2^-22 of it). One FP16 product alone loses what matters
// here: rounding noise of the strong directions of X lands on the weak ones, and those are what
// the iteration amplifies (a random matrix of rank 16 plus 5% noise comes out 2% wrong with one
// FP16 product, 17% with BF16). FP16 has few exponents, so each matrix carries a power-of-two
// scale. The host derives it from the coefficients: |X_0| <= 1 in the spectral norm, the
// polynomial bounds every later norm, and no element exceeds the norm.
//
// Three products per step:
//   GRAM   S = X X^T              both operands K-major
//   POLY   R = b S + c S^2
//   APPLY  X' = R X + a X         X read MN-major: no transposed copy of it is ever made
// S and R are symmetric: only the tiles on or below the diagonal are computed and stored. A k step
// to the right of the diagonal block reads the transposed tile below it, as an MN-major operand.
// (Storing both halves made the stores of a tile 10000 of 24000 cycles longer.)
//
// The tensor core's own additions cut what lies below the sum that they meet. So its accumulators,
// up to four, are read out after each step of 64 k and added up in FP32 registers, and a X is added in
// the epilogue: the largest term passes no tensor core. Results of every type are made so and rounded
// once. Off the exact result, five steps, plain 32-bit products in brackets: 4096 x 4096
// 5.6e-7 (3.2e-6), 256 x 256 6.8e-7 (1.7e-6), 128 x 1000 7.4e-7 (1.4e-6), 32 x 16 7.7e-7 (8.4e-7),
// 20 x 3000 1.1e-6 (1.1e-6), the last three with what Cfg::FINE adds. With a I in R and one accumulator
// per step 4096 x 4096 and 256 x 256 had 1.1 and 1.4e-6, with chunks of 512 k ten times that.
//
// A call is two launches: norm_kernel (sums of squares) and ns_kernel, which stays resident and
// runs all products with a grid-wide barrier between them. With a launch for each product the
// chain of 15 small products of a 256 x 256 matrix took 175 us, most of it launches.
//
// Tiles of ns_kernel, chosen by choose(): 256 x 256 by a CTA pair, 128 x 128 or 128 x 64 by one
// CTA. Tiles that do not fill the SMs once more are split along k: the parts of their sums go to the
// workspace in FP32 and are added in order after another barrier.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "../../include/orthogonalize.h"
#include "sgemm_internal.h"
#include "sgemm_plan.h"
#include "tc_common.cuh"

namespace sgemm {
namespace ns {

using namespace tcx;

constexpr int BK = 64;                    // k per stage: 128 bytes of FP16
constexpr int BOX = 64;                   // rows of a small TMA box
constexpr int BOX_BYTES = BOX * 128;
constexpr int MAX_STEPS = 64;

// FINE, for short sides of one tile: lo lo' is added, a step's accumulators are added up before they meet
// the longer sum, and where the registers hold it that sum runs over 8 steps first (EIGHTS). What
// 22-bit factors and a long FP32 sum lose is then no more than plain 32-bit products lose; without it 20 x
// 3000 was off by 1.2 times as much on average, by 2.1 times at most. It costs 1% there, 4% in large
// batches, and would cost 7% at 512 x 512, where the error is below half of plain products' without it.
template <int TN_, bool PAIR_, bool FINE_>
struct Cfg {
  static constexpr int TN = TN_;                        // tile columns
  static constexpr bool PAIR = PAIR_, FINE = FINE_, EIGHTS = FINE && TN == 64;
  static constexpr int BS = PAIR ? 256 : 128;           // tile rows; sizes are padded to it
  static constexpr int QN = PAIR ? TN / 2 : TN;         // columns of Q that a CTA holds
  static constexpr int P_TILE = 128 * 128, Q_TILE = QN * 128;  // bytes of hi or lo
  static constexpr int STAGE_BYTES = 2 * (P_TILE + Q_TILE);
  static constexpr int STAGES = TN == 64 ? 4 : 3;
  static constexpr int GROUPS = 2;                      // epilogue groups of four warps
  static constexpr int COLS = TN / GROUPS;
  static constexpr int EPI_WARPS = 4 * GROUPS, THREADS = 32 * (4 + EPI_WARPS);
  // accumulators of a k step (see the MMA issuer): as many as TMEM holds twice, four at most
  static constexpr int ACCS = TN == 64 ? 4 : TN == 128 ? 2 : 1;
  static constexpr int TMEM_COLS = 2 * ACCS * TN;
  static constexpr int SLOTS = BS / 32 * (TN / 32);     // 32 x 32 blocks of a tile
  static constexpr int BAR_BYTES = 8 * (2 * STAGES + 4) + 16;
  static constexpr int SMEM_BYTES =
      1024 + STAGES * STAGE_BYTES + EPI_WARPS * TURN_BYTES + BAR_BYTES;
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory per CTA");
  static_assert(COLS % 32 == 0 && 128 * 129 * 4 <= STAGES * STAGE_BYTES, "epilogue blocks");
  // kind::f16: D in FP32 (bits 4-5 = 1), FP16 operands (bits 7-9, 10-12 = 0), MN-major Q (bit 16)
  // where asked, N / 8 (bits 17-22), M / 16 (bits 24-28).
  static constexpr uint32_t IDESC =
      (1u << 4) | ((uint32_t)(TN >> 3) << 17) | ((uint32_t)(BS >> 4) << 24);
};

enum { GRAM = 0, POLY = 1, APPLY = 2 };

struct Input {
  const void *g;
  int type, rows, cols;
  long long ld, stride;
  int vec;                 // matrices without gaps, 16-byte aligned
  int rows_vec;            // 16-byte loads of rows are aligned
};

struct Params {
  int batch, steps;
  int mp, np;              // padded sizes of the short and the long side
  // per product: tiles of a matrix, tiles of the batch computed whole, parts of the others' sums
  int tiles[3], whole[3], split[3];
  long long half;          // rows between the hi and the lo part of a matrix: batch * mp
  __half *x[2], *s, *r;
  float *partial;
  unsigned *counter;       // arrivals at the grid-wide barrier
  Input in;
  const double *part;      // pieces of the sums of squares
  int parts;
  double eps;
  float x_scale;
  // per step: factors of the sums of the three products, of S in R, and of X in the next X
  float f[MAX_STEPS][3], fs[MAX_STEPS], fx[MAX_STEPS];
  // the result
  void *user;
  int user_type, tall, m, n, vec;
  long long ldu, user_stride;
  float alpha, beta;
};

// Tensor maps of both X buffers, S and R, in boxes of 128 rows (K-major tiles of 128 rows) and of 64
// (K-major tiles of 64 rows; MN-major tiles, whose box rows are the k of a step).
struct Maps {
  CUtensorMap large[4], small[4];
};

// Device status word: 0 = fine; 1, 2, 3 = a wait of the producer, the MMA issuer or the epilogue
// gave up, 4 = a wait at the grid-wide barrier did.
__device__ int g_ns_status;

__device__ __forceinline__ uint32_t pack_half(__half a, __half b) {
  const __half2 h = __halves2half2(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// ---- Grid-wide barrier: every CTA arrives once per use, and not before the use before is complete;
// the count only grows. Work that a CTA
// does before its arrival is visible to whoever has seen the count, TMA copies included.
__device__ __forceinline__ void proxy_fence() { asm volatile("fence.proxy.async;\n" ::: "memory"); }

__device__ __forceinline__ void grid_arrive(unsigned *counter) {  // one thread, after a CTA barrier
  asm volatile("red.release.gpu.global.add.u32 [%0], 1;\n" ::"l"(counter) : "memory");
}

// Limit of a wait at the barrier, whose end other CTAs' work decides. A product's first operands, and
// its first sums, come after the barrier and one and two waits of this CTA's own: those are waited for
// that much longer. Every other wait is for the CTA's own (or its partner's) copies and instructions.
constexpr unsigned long long kGridLimitNs = 8 * kWaitLimitNs;
constexpr unsigned long long kFirstLimitNs = kGridLimitNs + kWaitLimitNs;

// One warp; false if the count has not been reached after kGridLimitNs. copies: TMA copies follow.
__device__ __forceinline__ bool grid_wait(const unsigned *counter, unsigned target, bool copies) {
  bool ok = true;
  if ((threadIdx.x & 31) == 0) {
    unsigned v;
    unsigned long long t0 = 0;
    for (uint32_t i = 0;; ++i) {
      asm volatile("ld.acquire.gpu.global.u32 %0, [%1];\n" : "=r"(v) : "l"(counter) : "memory");
      if (v >= target) break;
      if ((i & 255u) == 255u) {
        const unsigned long long t = global_ns();
        if (t0 == 0) t0 = t;
        if (t - t0 > kGridLimitNs || i >= (1u << 31)) {
          ok = false;
          break;
        }
      }
    }
    if (copies) proxy_fence();  // (they read what other CTAs' plain stores wrote)
    if (!ok) atomicCAS(&g_ns_status, 0, 4);
  }
  ok = __all_sync(0xffffffffu, ok);
  __syncwarp();  // (a vote orders no memory: what lane 0 has acquired is now visible to all)
  return ok;
}

// Units of a product: the tiles computed whole, then the parts of the others.
__device__ __forceinline__ int units_of(const Params &p, int mode) {
  return p.whole[mode] + (p.batch * p.tiles[mode] - p.whole[mode]) * p.split[mode];
}

struct Unit {
  int mat, tp, tq;  // matrix, tile row and column
  int part;         // index of the part among all parts, -1 for a whole tile
  int k0, k1;       // steps of k
};

// Tile t of the batch. Tiles of the symmetric products are those on or below the diagonal, row by
// row (BS / TN of them in a diagonal block).
template <class C>
__device__ __forceinline__ void tile_at(const Params &p, int mode, int t, Unit &u) {
  u.mat = t / p.tiles[mode];
  t %= p.tiles[mode];
  if (mode == APPLY) {
    tile_coords(t, p.mp / C::BS, p.np / C::TN, 4, u.tp, u.tq);
    return;
  }
  constexpr int Q = C::BS / C::TN;
  int i = (int)((sqrtf(8.0f * (t / Q) + 1.0f) - 1.0f) * 0.5f);
  while (Q * (i + 1) * (i + 2) / 2 <= t) ++i;
  while (Q * i * (i + 1) / 2 > t) --i;
  u.tp = i;
  u.tq = t - Q * i * (i + 1) / 2;
}

template <class C>
__device__ __forceinline__ Unit unit_at(const Params &p, int mode, int i) {
  Unit u;
  const int KT = (mode == GRAM ? p.np : p.mp) / BK, S = p.split[mode];
  u.part = i - p.whole[mode];
  u.k0 = 0;
  u.k1 = KT;
  int t = i;
  if (u.part >= 0) {
    const int sp = u.part % S;
    t = p.whole[mode] + u.part / S;
    u.k0 = (int)((long long)KT * sp / S);
    u.k1 = (int)((long long)KT * (sp + 1) / S);
  } else {
    u.part = -1;
  }
  tile_at<C>(p, mode, t, u);
  return u;
}

// Whether step k (elements) of a symmetric operand's rows from `row` lies to the right of their
// diagonal block, where only the transposed tile is stored.
template <class C>
__device__ __forceinline__ bool beyond(int row, int k) {
  return k >= (row / C::BS + 1) * C::BS;
}

// What becomes of 32 x 32 sums of a product at (row0, col0) of matrix `mat`: v holds 32 columns of
// one row per lane. One copy of this code serves all products (ns_kernel): each CTA runs it once or
// twice between two barriers, and what it costs then is mostly the fetching of its instructions.
__device__ __forceinline__ void finish(const Params &p, int mode, int step, int mat, int row0,
                                       int col0, uint8_t *buf, int lane,
                                       float (&v)[32]) {
  const bool result = mode == APPLY && step == p.steps - 1;
  if (result && (row0 >= p.m || col0 >= p.n)) return;
  const float f = p.f[step][mode];
#pragma unroll
  for (int j = 0; j < 32; ++j) v[j] *= f;
  const int part = lane & 3, sub = lane >> 2;  // 16-byte piece and row of 8 of coalesced accesses
  const long long ld = mode == APPLY ? p.np : p.mp, lo = p.half * ld;
  const long long row = (long long)mat * p.mp + row0;  // in the buffer
  if (mode != GRAM) {
    const float fs = mode == POLY ? p.fs[step] : p.fx[step];
    const __half *s = (mode == POLY ? p.s : p.x[step & 1]) + (row + sub) * ld + col0 + 8 * part;
    uint4 in[2][4];  // both halves are on their way before the first is used
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        in[h][i] = __ldcg(reinterpret_cast<const uint4 *>(s + h * lo + 8 * i * ld));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < 4; ++i) *turn_at(buf, 8 * i + sub, part) = in[h][i];
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint4 u = *turn_at(buf, lane, j);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&w[e]));
          v[8 * j + 2 * e] = fmaf(fs, a.x, v[8 * j + 2 * e]);
          v[8 * j + 2 * e + 1] = fmaf(fs, a.y, v[8 * j + 2 * e + 1]);
        }
      }
      __syncwarp();
    }
  }
  if (result) {
    const int size = p.user_type == NS_F32 ? 4 : 2;
    void *out = reinterpret_cast<char *>(p.user) + mat * p.user_stride * size;
    if (!p.tall) {
      store_rows<32>(Out{out, p.user_type, p.ldu, p.m, p.n, p.alpha, p.beta, p.vec}, buf, lane, row0,
                     col0, v);
    } else if (row0 + lane < p.m) {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (col0 + j < p.n)
          finish_out(out, p.user_type, (col0 + j) * p.ldu + row0 + lane, p.alpha * v[j], p.beta);
    }
    return;
  }
  // hi, then lo = what hi leaves
  __half *base = mode == GRAM ? p.s : mode == POLY ? p.r : p.x[(step + 1) & 1];
  __half *o = base + (row + sub) * ld + col0 + 8 * part;
#pragma unroll 1
  for (int h = 0; h < 2; ++h, o += lo) {
    uint32_t w[16];
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      const __half2 a = __floats2half2_rn(v[j], v[j + 1]);
      w[j / 2] = *reinterpret_cast<const uint32_t *>(&a);
      const float2 b = __half22float2(a);
      v[j] -= b.x;
      v[j + 1] -= b.y;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *turn_at(buf, lane, j) = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<uint4 *>(o + 8 * i * ld) = *turn_at(buf, 8 * i + sub, part);
    __syncwarp();
  }
}

// ------------------------------------------------------------------------------------
// Norm and start values.

__device__ __forceinline__ float load(const void *x, int type, long long i) {
  return load_out(x, type, i);
}

// Squares of numbers over 2^64 overflow FP32 and those under 2^-64 vanish, so each thread sums
// the squares of x, of x 2^-70 and of x 2^70; the last step takes the sum that did neither.
constexpr float kDown = 0x1p-70f, kUp = 0x1p70f;

__device__ __forceinline__ void add_square(float (&s)[3], float x) {
  s[0] = fmaf(x, x, s[0]);
  s[1] = fmaf(x * kDown, x * kDown, s[1]);
  s[2] = fmaf(x * kUp, x * kUp, s[2]);
}

// Block b of matrix b / parts: its share of the matrix, in an order fixed by the shape. Block 0 also
// resets the counter of the grid-wide barrier.
__global__ void __launch_bounds__(256)
    norm_kernel(const Input in, double *part, int parts, unsigned *counter) {
  griddep_wait();
  __shared__ double red[3][8];
  if (blockIdx.x == 0 && threadIdx.x == 0) *counter = 0;
  const int mat = blockIdx.x / parts, piece = blockIdx.x % parts;
  const long long total = (long long)in.rows * in.cols, eights = (total + 7) / 8;
  const long long first = eights * piece / parts * 8;
  const long long last = min(total, eights * (piece + 1) / parts * 8);
  float s[3] = {0.0f, 0.0f, 0.0f};
  if (in.vec) {
    const int size = in.type == NS_F32 ? 4 : 2, per = 16 / size;  // (last - first) % 8 == 0 but at the end
    const char *g = reinterpret_cast<const char *>(in.g) + mat * in.stride * size;
#pragma unroll 4
    for (long long i = first + threadIdx.x * per; i + per <= last; i += 256 * per) {
      const uint4 u = *reinterpret_cast<const uint4 *>(g + i * size);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (in.type == NS_F32) {
          add_square(s, __uint_as_float(w[e]));
        } else if (in.type == NS_BF16) {
          add_square(s, __uint_as_float(w[e] << 16));
          add_square(s, __uint_as_float(w[e] & 0xffff0000u));
        } else {
          const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&w[e]));
          add_square(s, a.x);
          add_square(s, a.y);
        }
      }
    }
    const long long tail = last - (last - first) % per + threadIdx.x;
    if (tail < last) add_square(s, load(g, in.type, tail));
  } else {
    long long i = first + threadIdx.x;
    int r = (int)(i / in.cols), c = (int)(i % in.cols);
    const int step_r = 256 / in.cols, step_c = 256 % in.cols;
#pragma unroll 4
    for (; i < last; i += 256) {
      add_square(s, load(in.g, in.type, mat * in.stride + r * in.ld + c));
      r += step_r;
      c += step_c;
      if (c >= in.cols) {
        c -= in.cols;
        ++r;
      }
    }
  }
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    double d = s[q];
#pragma unroll
    for (int o = 16; o > 0; o /= 2) d += __shfl_xor_sync(0xffffffffu, d, o);
    if ((threadIdx.x & 31) == 0) red[q][threadIdx.x >> 5] = d;
  }
  __syncthreads();
  if (threadIdx.x < 3) {
    double d = 0.0;
    for (int w = 0; w < 8; ++w) d += red[threadIdx.x][w];
    part[(long long)blockIdx.x * 3 + threadIdx.x] = d;
  }
}

// What X_0 of matrix `mat` is multiplied with, in two factors, by one warp.
__device__ __forceinline__ void start_factors(const Params &p, int mat, float *mul) {
  const int lane = threadIdx.x & 31;
  double s[3] = {0.0, 0.0, 0.0};
  for (int i = lane; i < p.parts; i += 32)
    for (int q = 0; q < 3; ++q) s[q] += p.part[((long long)mat * p.parts + i) * 3 + q];
#pragma unroll
  for (int q = 0; q < 3; ++q)
#pragma unroll
    for (int o = 16; o > 0; o /= 2) s[q] += __shfl_xor_sync(0xffffffffu, s[q], o);
  if (lane == 0) {
    // a sum of NaN fails every comparison and stays NaN
    double pre = 1.0, sum = s[0];
    if (s[0] > 1e35) {
      pre = kDown;
      sum = s[1];
    } else if (s[0] < 1e-25) {
      pre = kUp;
      sum = s[2];
    }
    const double norm = sqrt(sum) / pre;
    mul[0] = (float)pre;
    mul[1] = norm + p.eps > 0.0 ? (float)(p.x_scale / (norm + p.eps) / pre) : (float)(norm * 0.0);
  }
}

// Eight neighbouring elements of row r from column c (0 out of range).
__device__ __forceinline__ void load8(const Input &in, const char *g, int r, int c, float (&v)[8]) {
  const int size = in.type == NS_F32 ? 4 : 2;
  if (in.rows_vec && r < in.rows && c + 8 <= in.cols) {
    const uint4 *q = reinterpret_cast<const uint4 *>(g + (r * in.ld + c) * size);
    const uint4 u = __ldg(q);
    if (in.type == NS_F32) {
      const uint4 u2 = __ldg(q + 1);
      const uint32_t w[8] = {u.x, u.y, u.z, u.w, u2.x, u2.y, u2.z, u2.w};
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(w[e]);
    } else {
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (in.type == NS_BF16) {
          v[2 * e] = __uint_as_float(w[e] << 16);
          v[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
        } else {
          const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&w[e]));
          v[2 * e] = a.x;
          v[2 * e + 1] = a.y;
        }
      }
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    v[e] = r < in.rows && c + e < in.cols ? load(g, in.type, r * in.ld + c + e) : 0.0f;
}

// X_0 times its scale as hi and lo, in the short orientation, with zero padding. 128 x 128 tiles by
// whole CTAs; a tall G is turned in t (128 x 129).
__device__ __forceinline__ void start(const Params &p, float *t, float *mul) {
  const int tiles_n = p.np / 128, per = tiles_n * (p.mp / 128), nt = blockDim.x;
  const long long lo = p.half * p.np;
  const Input &in = p.in;
  const int size = in.type == NS_F32 ? 4 : 2;
  int known = -1;
  for (int u = blockIdx.x; u < per * p.batch; u += gridDim.x) {
    const int mat = u / per, tile = u % per;
    const int r0 = tile / tiles_n * 128, c0 = tile % tiles_n * 128;
    const char *g = reinterpret_cast<const char *>(in.g) + mat * in.stride * size;
    if (mat != known) {
      __syncthreads();
      if (threadIdx.x < 32) start_factors(p, mat, mul);
      __syncthreads();
      known = mat;
    }
    const float pre = mul[0], f = mul[1];
    if (p.tall) {
      __syncthreads();  // the last tile has been read
#pragma unroll 2
      for (int e = threadIdx.x; e < 2048; e += nt) {
        const int m = 8 * (e & 15), n = e >> 4;  // G is n x m
        float v[8];
        load8(in, g, c0 + n, r0 + m, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) t[(m + j) * 129 + n] = v[j];
      }
      __syncthreads();
    }
#pragma unroll 2
    for (int e = threadIdx.x; e < 2048; e += nt) {
      const int n = 8 * (e & 15), m = e >> 4;
      float v[8];
      if (p.tall) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = t[m * 129 + n + j];
      } else {
        load8(in, g, r0 + m, c0 + n, v);
      }
      uint32_t hi[4], lw[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float a = v[2 * j] * pre * f, b = v[2 * j + 1] * pre * f;
        const __half ha = __float2half_rn(a), hb = __float2half_rn(b);
        hi[j] = pack_half(ha, hb);
        lw[j] = pack_half(__float2half_rn(a - __half2float(ha)), __float2half_rn(b - __half2float(hb)));
      }
      __half *o = p.x[0] + ((long long)mat * p.mp + r0 + m) * p.np + c0 + n;
      *reinterpret_cast<uint4 *>(o) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      *reinterpret_cast<uint4 *>(o + lo) = make_uint4(lw[0], lw[1], lw[2], lw[3]);
    }
  }
}

// steps == 0: out = alpha X_0 + beta out.
__global__ void __launch_bounds__(256) copy_kernel(const Params p) {
  __shared__ float mul[2];
  const long long total = (long long)p.in.rows * p.in.cols;
  const int size = p.user_type == NS_F32 ? 4 : 2;
  for (int mat = blockIdx.y; mat < p.batch; mat += gridDim.y) {
    __syncthreads();  // (mul has been read)
    if (threadIdx.x < 32) start_factors(p, mat, mul);
    __syncthreads();
    void *out = reinterpret_cast<char *>(p.user) + mat * p.user_stride * size;
    for (long long i = blockIdx.x * 256LL + threadIdx.x; i < total; i += gridDim.x * 256LL) {
      const long long r = i / p.in.cols, c = i % p.in.cols;
      const float x = load(p.in.g, p.in.type, mat * p.in.stride + r * p.in.ld + c) * mul[0] * mul[1];
      finish_out(out, p.user_type, r * p.ldu + c, p.alpha * x, p.beta);
    }
  }
}

// ------------------------------------------------------------------------------------
// All products. Warp 0: TMA producer, warp 1: MMA issuer (one elected lane of each); warps 4 ..:
// epilogue, a group of four warps owns COLS columns of the tile, warp w of it TMEM lanes (rows)
// 32 (w % 4) .. + 31. All warps together make the start values.
//
// What bounds it, five steps each. 4096 x 4096 FP32, pairs: 2900 us; three FP16 MMAs per product, the
// instructions alone 2160 (1.9 PFLOP/s), the rest the last, partial round of tiles and their stores.
// 8 x 1024 x 1024 BF16, 128 x 128 tiles: 673 us, 270 of them MMAs; a product is 2 to 4 rounds of
// tiles, and the barrier, the first loads and the last stores of a product overlap nothing.
// 4097 x 777 BF16: 364 us, the same with products of one round. (16-bit results summed 256 k in one
// accumulator, with a I in R, took 545 and 318 us, for several times the error before the rounding.)
// 256 x 256 FP32: 119 us, 7 to 8 us for each of 15 dependent products: barrier 2, first loads 1.5, k steps
// 1.5, stores 1 to 2.

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1)
    ns_kernel(const __grid_constant__ Maps maps, const __grid_constant__ Params p) {
  constexpr bool PAIR = C::PAIR;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = saddr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t *sbase = smem_raw + (base - raw);
  const uint32_t bars = base + C::STAGES * C::STAGE_BYTES + C::EPI_WARPS * TURN_BYTES;
  const uint32_t acc_full = bars + 8 * (2 * C::STAGES), acc_empty = acc_full + 16;
  const uint32_t tmem_slot = acc_empty + 16;
  volatile uint32_t *tmem_slot_ptr =
      reinterpret_cast<volatile uint32_t *>(smem_raw + (tmem_slot - raw));
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int cta = PAIR ? (int)(blockIdx.x & 1u) : 0;
  const int first = (int)(PAIR ? blockIdx.x >> 1 : blockIdx.x);
  const int stride = (int)(PAIR ? gridDim.x >> 1 : gridDim.x);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(bars + 8 * s, 1);
      mbar_init(bars + 8 * (C::STAGES + s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_full + 8 * b, 1);
      mbar_init(acc_empty + 8 * b, PAIR ? 2 * C::EPI_WARPS : C::EPI_WARPS);
    }
    mbar_init_fence();
    for (int i = 0; i < 4; ++i) {
      tma_prefetch_map(&maps.large[i]);
      tma_prefetch_map(&maps.small[i]);
    }
  }
  __syncwarp();
  if (warp == 0) {
    if constexpr (PAIR) {
      tmem_alloc_pair(tmem_slot, C::TMEM_COLS);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_slot, C::TMEM_COLS);
      tmem_relinquish();
    }
  }
  {
    __shared__ float mul[2];
    start(p, reinterpret_cast<float *>(sbase), mul);
  }
  proxy_fence();
  fence_before();
  __syncthreads();
  if (threadIdx.x == 0) grid_arrive(p.counter);  // (orders this CTA's use of shared memory too)
  if constexpr (PAIR) cluster_sync_all();        // the other CTA's barriers are initialised
  fence_after();
  const uint32_t tmem = *tmem_slot_ptr;
  unsigned passed = gridDim.x;                   // count of the barrier uses so far

  if (warp < 4) {
    if constexpr (PAIR) reg_dealloc<56>();       // 384 x 168 = 128 x 56 + 256 x 224
    if (warp == 0) {
      // ---- TMA producer: P hi, P lo, Q hi, Q lo of each k step
      Ring<C::STAGES> st;
      int issued = 0;  // (up to STAGES)
      bool ok = true;
      for (int ph = 0; ph < 3 * p.steps && ok; ++ph) {
        const int mode = ph % 3, step = ph / 3;
        ok = grid_wait(p.counter, passed, true);
        if (!ok) break;
        const int x = step & 1;
        const int ip = mode == GRAM ? x : mode + 1, iq = mode == POLY ? 2 : x;  // maps of P and Q
        const int total = units_of(p, mode);
        for (int i = first; i < total && ok; i += stride) {
          const Unit u = unit_at<C>(p, mode, i);
          const int y0 = u.mat * p.mp, p0 = u.tp * C::BS + cta * 128;
          const int q0 = u.tq * C::TN + cta * (PAIR ? C::QN : 0);
          for (int kt = u.k0; kt < u.k1; ++kt) {
            ok = __all_sync(0xffffffffu,
                            wait_short(bars + 8 * (C::STAGES + st.slot), st.parity ^ 1u));
            if (!ok) {
              if (lane == 0) atomicCAS(&g_ns_status, 0, 1);
              break;
            }
            if (elect_one()) {
              const uint32_t dst = base + st.slot * C::STAGE_BYTES;
              const uint32_t full = PAIR ? in_cta(bars + 8 * st.slot, 0) : bars + 8 * st.slot;
              const int k = kt * BK;
              if (!PAIR || cta == 0)
                mbar_expect_tx(bars + 8 * st.slot, (PAIR ? 2 : 1) * C::STAGE_BYTES);
              const auto get = [&](uint32_t to, const CUtensorMap *m, int x, int y) {
                if constexpr (PAIR)
                  tma_load_2d_pair(to, m, x, y, full);
                else
                  tma_load_2d(to, m, x, y, full);
              };
              // rows [r0, + ROWS) of an operand at this step of k: K-major, or MN-major from rows
              // [k, + 64) of the matrix
              const bool pt = mode != GRAM && beyond<C>(p0, k);
              const bool qt = mode == APPLY || (mode == POLY && beyond<C>(q0, k));
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int y = y0 + (h ? (int)p.half : 0);
                const uint32_t dp = dst + h * C::P_TILE, dq = dst + 2 * C::P_TILE + h * C::Q_TILE;
                if (pt) {
                  get(dp, &maps.small[ip], p0, y + k);
                  get(dp + BOX_BYTES, &maps.small[ip], p0 + BOX, y + k);
                } else {
                  get(dp, &maps.large[ip], k, y + p0);
                }
                if (qt) {
#pragma unroll
                  for (int c = 0; c < C::QN / BOX; ++c)
                    get(dq + c * BOX_BYTES, &maps.small[iq], q0 + BOX * c, y + k);
                } else {
                  get(dq, C::QN == 128 ? &maps.large[iq] : &maps.small[iq], k, y + q0);
                }
              }
            }
            __syncwarp();
            issued = min(issued + 1, C::STAGES);
            st.next();
          }
        }
        passed += gridDim.x * (p.split[mode] > 1 ? 2u : 1u);
      }
      // the last loads issued must have landed before this warp leaves (a pair's: the leader waits
      // for both, and the CTAs leave together)
      for (; issued > 0 && (!PAIR || cta == 0); --issued) {
        st.parity ^= st.slot == 0 ? 1u : 0u;
        st.slot = st.slot == 0 ? C::STAGES - 1 : st.slot - 1;
        wait_short(bars + 8 * st.slot, st.parity);
      }
    } else if (warp == 1 && (!PAIR || cta == 0)) {
      // ---- MMA issuer: one k step per set of TMEM accumulators, the corrections first, so that only
      // hi hi' meets a sum of full size. An instruction aligns its 16 products with the accumulator
      // and cuts what lies below: the larger the sum it meets, the more. So hi hi' of a step's four
      // instructions go to ACCS accumulators in turn.
      const uint64_t ph0 = sw128_desc(base, BOX_BYTES), pl0 = ph0 + (C::P_TILE >> 4);
      const uint64_t qh0 = ph0 + (2 * C::P_TILE >> 4), ql0 = qh0 + (C::Q_TILE >> 4);
      Ring<C::STAGES> st;
      Ring<2> buf;
      bool ok = true;
      for (int ph = 0; ph < 3 * p.steps && ok; ++ph) {
        const int mode = ph % 3;
        const int total = units_of(p, mode);
        unsigned long long limit = kFirstLimitNs;
        for (int i = first; i < total && ok; i += stride) {
          const Unit u = unit_at<C>(p, mode, i);
          for (int kt = u.k0; kt < u.k1; ++kt) {
            ok = __all_sync(0xffffffffu, wait_short(acc_empty + 8 * buf.slot, buf.parity ^ 1u) &&
                                             wait_short(bars + 8 * st.slot, st.parity, limit));
            limit = kWaitLimitNs;
            if (!ok) {
              if (lane == 0) atomicCAS(&g_ns_status, 0, 2);
              break;
            }
            fence_after();
            if (elect_one()) {
              const uint32_t at = st.slot * (uint32_t)(C::STAGE_BYTES >> 4);
              const uint32_t acc = tmem + buf.slot * (C::ACCS * C::TN);
              // (both CTAs of a pair have the same k beyond their diagonal block: blocks of 256)
              const bool pt = mode != GRAM && beyond<C>(u.tp * C::BS, kt * BK);
              const bool qt = mode == APPLY || (mode == POLY && beyond<C>(u.tq * C::TN, kt * BK));
              const uint32_t idesc = C::IDESC | (pt ? 1u << 15 : 0u) | (qt ? 1u << 16 : 0u);
              const uint32_t adv_p = (pt ? 16 * 128 : 32) >> 4, adv_q = (qt ? 16 * 128 : 32) >> 4;
              const auto mma = [&](uint32_t d, uint64_t a, uint64_t b, uint32_t more) {
                if constexpr (PAIR)
                  mma_f16_pair(d, a, b, idesc, more);
                else
                  mma_f16(d, a, b, idesc, more);
              };
#pragma unroll
              for (uint32_t kk = 0; kk < BK / 16; ++kk) {
                if (C::FINE) mma(acc, pl0 + at + kk * adv_p, ql0 + at + kk * adv_q, kk != 0);
                mma(acc, pl0 + at + kk * adv_p, qh0 + at + kk * adv_q, C::FINE || kk != 0);
                mma(acc, ph0 + at + kk * adv_p, ql0 + at + kk * adv_q, 1u);
              }
#pragma unroll
              for (uint32_t kk = 0; kk < BK / 16; ++kk) {
                const uint32_t n = kk % C::ACCS;
                mma(acc + n * C::TN, ph0 + at + kk * adv_p, qh0 + at + kk * adv_q,
                    n == 0 || kk >= C::ACCS);
              }
              if constexpr (PAIR) {
                mma_commit_pair(bars + 8 * (C::STAGES + st.slot));
                mma_commit_pair(acc_full + 8 * buf.slot);
              } else {
                mma_commit(bars + 8 * (C::STAGES + st.slot));
                mma_commit(acc_full + 8 * buf.slot);
              }
            }
            __syncwarp();
            st.next();
            buf.next();
          }
        }
      }
    }
  } else {
    // ---- epilogue. After a wait that gave up a warp goes on without its sums, so that it still
    // arrives at the barriers of its CTA.
    if constexpr (PAIR) reg_alloc<224>();
    const int grp = (warp - 4) >> 2, quad = warp & 3;
    const uint32_t src0 = tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)(grp * C::COLS);
    uint8_t *turn = sbase + C::STAGES * C::STAGE_BYTES + (warp - 4) * TURN_BYTES;
    Ring<2> buf;
    bool ok = true;
    for (int ph = 0; ph < 3 * p.steps; ++ph) {
      const int mode = ph % 3, step = ph / 3;
      const int S = p.split[mode], whole = p.whole[mode], total = units_of(p, mode);
      // pass 0: this CTA's units; pass 1, where sums are split: their parts added in order, one
      // 32 x 32 block per warp at a time
#pragma unroll 1
      for (int pass = 0; pass < (S > 1 ? 2 : 1); ++pass) {
        const int end = pass ? (p.batch * p.tiles[mode] - whole) * C::SLOTS : total;
        const int by = pass ? (int)gridDim.x * C::EPI_WARPS : stride;
#pragma unroll 1
        for (int i = pass ? (int)blockIdx.x * C::EPI_WARPS + warp - 4 : first; i < end; i += by) {
          float acc[C::COLS], eights[C::EIGHTS ? C::COLS : 1];
#pragma unroll
          for (int j = 0; j < C::COLS; ++j) acc[j] = 0.0f;
          if constexpr (C::EIGHTS) {
#pragma unroll
            for (int j = 0; j < C::COLS; ++j) eights[j] = 0.0f;
          }
          Unit u;
          int row0, col0;
          if (pass == 0) {
            unsigned long long limit = kWaitLimitNs + (i == first ? kFirstLimitNs : 0);
            u = unit_at<C>(p, mode, i);
            row0 = u.tp * C::BS + cta * 128 + quad * 32;
            col0 = u.tq * C::TN + grp * C::COLS;
            for (int kt = u.k0; kt < u.k1 && ok; ++kt) {
              ok = __all_sync(0xffffffffu, wait_short(acc_full + 8 * buf.slot, buf.parity, limit));
              limit = kWaitLimitNs;
              if (!ok) {
                if (lane == 0) atomicCAS(&g_ns_status, 0, 3);
                break;
              }
              // (S will be read for R, or X for the next X: this CTA's producer has seen them written
              // before its first copy, and this makes them visible to this warp)
              if (mode != GRAM && kt == u.k0)
                ok = grid_wait(p.counter, passed, false);
              fence_after();
              if constexpr (C::FINE) {
                const uint32_t src = src0 + buf.slot * (C::ACCS * C::TN);
#pragma unroll
                for (int j0 = 0; j0 < C::COLS; j0 += 16) {
                  uint32_t v[C::ACCS][16];
#pragma unroll
                  for (int n = 0; n < C::ACCS; ++n) tmem_ld(src + (uint32_t)(n * C::TN + j0), v[n]);
#pragma unroll
                  for (int n = 0; n < C::ACCS; ++n) tmem_wait_ld(v[n]);
#pragma unroll
                  for (int j = 0; j < 16; ++j) {
                    float s = __uint_as_float(v[0][j]);
#pragma unroll
                    for (int n = 1; n < C::ACCS; ++n) s += __uint_as_float(v[n][j]);
                    if constexpr (C::EIGHTS)
                      eights[j0 + j] += s;
                    else
                      acc[j0 + j] += s;
                  }
                }
                if constexpr (C::EIGHTS) {
                  if (((kt - u.k0) & 7) == 7 || kt == u.k1 - 1) {
#pragma unroll
                    for (int j = 0; j < C::COLS; ++j) {
                      acc[j] += eights[j];
                      eights[j] = 0.0f;
                    }
                  }
                }
              } else {
#pragma unroll 1
                for (int n = 0; n < C::ACCS; ++n) {
                  const uint32_t src = src0 + (buf.slot * C::ACCS + n) * C::TN;
#pragma unroll
                  for (int j0 = 0; j0 < C::COLS; j0 += 16) {
                    uint32_t v[16];
                    tmem_ld(src + (uint32_t)j0, v);
                    tmem_wait_ld(v);
#pragma unroll
                    for (int j = 0; j < 16; ++j) acc[j0 + j] += __uint_as_float(v[j]);
                  }
                }
              }
              fence_before();
              __syncwarp();
              if (lane == 0) {
                if constexpr (PAIR)
                  arrive_in(in_cta(acc_empty + 8 * buf.slot, 0));
                else
                  mbar_arrive(acc_empty + 8 * buf.slot);
              }
              buf.next();
            }
          } else {
            const int t = i / C::SLOTS, slot = i % C::SLOTS;
            tile_at<C>(p, mode, whole + t, u);
            u.part = -1;
            row0 = u.tp * C::BS + slot / (C::TN / 32) * 32;
            col0 = u.tq * C::TN + slot % (C::TN / 32) * 32;
            const float4 *from = reinterpret_cast<const float4 *>(
                p.partial + ((long long)t * S * C::SLOTS + slot) * 1024) + lane;
#pragma unroll 4
            for (int q = 0; q < S; ++q) {
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const float4 v = __ldcg(from + q * (C::SLOTS * 256) + 32 * j);
                acc[4 * j] += v.x;
                acc[4 * j + 1] += v.y;
                acc[4 * j + 2] += v.z;
                acc[4 * j + 3] += v.w;
              }
            }
          }
#pragma unroll 1
          for (int j0 = 0; j0 < (pass ? 32 : C::COLS); j0 += 32) {
            float v[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) {  // (acc stays in registers: no index that varies)
              v[j] = acc[j];
#pragma unroll
              for (int c = 32; c < C::COLS; c += 32)
                if (j0 == c) v[j] = acc[c + j];
            }
            if (u.part < 0) {
              finish(p, mode, step, u.mat, row0, col0 + j0, turn, lane, v);
            } else {
              const int slot = (cta * 4 + quad) * (C::TN / 32) + (grp * C::COLS + j0) / 32;
              float4 *o = reinterpret_cast<float4 *>(
                  p.partial + ((long long)u.part * C::SLOTS + slot) * 1024) + lane;
#pragma unroll
              for (int j = 0; j < 8; ++j)
                o[32 * j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
            }
          }
        }
        named_barrier(1, 32 * C::EPI_WARPS);
        if (warp == 4) {
          // (a CTA without work in this product must not arrive while others are still to arrive
          // for the one before)
          if (pass == 0 && first >= total) ok = grid_wait(p.counter, passed, false) && ok;
          if (lane == 0) grid_arrive(p.counter);
          __syncwarp();
        }
        if (S > 1 && pass == 0) ok = grid_wait(p.counter, passed + gridDim.x, false) && ok;
      }
      passed += gridDim.x * (S > 1 ? 2u : 1u);
    }
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  if constexpr (PAIR) {
    cluster_sync_all();  // no instruction, copy or arrival of the other CTA is under way
    if (warp == 0) tmem_dealloc_pair(tmem, C::TMEM_COLS);
  } else {
    if (warp == 0) tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// ------------------------------------------------------------------------------------
// Host side

using Pair = Cfg<256, true, false>;
using Wide = Cfg<128, false, false>;
using Narrow = Cfg<64, false, false>;
using FineWide = Cfg<128, false, true>;
using FineNarrow = Cfg<64, false, true>;

// How a problem runs: tile shape and parts of the sums, with the sizes that follow.
struct Plan {
  int shape;                    // 0 Pair, 1 Wide, 2 Narrow
  long long mp, np;             // short and long side, padded
  long long tiles[3], whole[3];
  int split[3];
  int parts;                    // pieces of a matrix in the norm
  long long ctas;
  size_t x, s, partial, bytes;  // elements of one X and one S (FP16) and of the partials (FP32)
};

// Estimated time of a plan in cycles. A k step of 64 costs its MMAs (12 instructions of TN / 2
// cycles) or the copy of its operands, whichever is longer (measured: about 50 bytes per cycle and
// SM with every SM loading, 64 with few); a product also costs its barrier and the stores of a
// CTA's tiles, and a split sum another barrier and pass.
static double cost(const Plan &q, int shape, int batch, long long mp, long long np, long long slots,
                   Plan *out) {
  static const int rows[3] = {Pair::BS, Wide::BS, Narrow::BS}, tn[3] = {256, 128, 64};
  static const double mma[3] = {1536, 768, 384};
  static const double bytes[3] = {Pair::STAGE_BYTES, Wide::STAGE_BYTES, Narrow::STAGE_BYTES};
  static const double tile[3] = {14000, 5000, 3000};
  *out = q;
  const long long tm = mp / rows[shape], per = rows[shape] / tn[shape];
  out->tiles[GRAM] = out->tiles[POLY] = per * tm * (tm + 1) / 2;
  out->tiles[APPLY] = tm * (np / tn[shape]);
  double total = 0.0;
  for (int mode = 0; mode < 3; ++mode) {
    const long long t = out->tiles[mode] * batch, KT = (mode == GRAM ? np : mp) / BK;
    double best = 1e300;
    for (int all = 0; all < 2; ++all) {  // the last, partial round of tiles split, or all of them
      const long long full = all ? 0 : t / slots * slots, rest = t - full;
      for (int S = 1; S <= 16 && S <= KT; ++S) {
        if (S > 1 && (rest == 0 || rest * S > slots)) break;
        const long long units = full + rest * S;
        const double step =
            std::max(mma[shape], bytes[shape] / (64.0 - 14.0 * std::min(1.0, (double)units / slots)));
        const double c = (S > 1 ? full / slots : (t + slots - 1) / slots) * (step * KT + tile[shape]) +
                         2500.0 + (S > 1 ? step * ((KT + S - 1) / S) + tile[shape] + 8000.0 + 500.0 * S : 0.0);
        if (c < best) {
          best = c;
          out->split[mode] = S;
          out->whole[mode] = S > 1 ? full : t;
        }
      }
    }
    total += best;
  }
  return total;
}

static Plan choose(int batch, int rows, int cols, int sms, const int *pairs) {
  Plan best{};
  const long long m = std::min(rows, cols), n = std::max(rows, cols);
  double least = 1e300;
  for (int shape = 0; shape < 3; ++shape) {
    const int unit = shape == 0 ? Pair::BS : 128;
    const long long mp = ceil_div(m, unit) * unit, np = ceil_div(n, unit) * unit;
    Plan q{};
    q.shape = shape;
    q.mp = mp;
    q.np = np;
    const long long slots = shape == 0 ? *pairs : sms;
    if (slots < 1) continue;
    Plan w;
    const double c = cost(q, shape, batch, mp, np, slots, &w);
    if (c < least) {
      least = c;
      best = w;
    }
  }
  const long long slots = best.shape == 0 ? *pairs : sms;
  long long units = 1;
  size_t most = 0;
  const int area = best.shape == 0 ? 256 * 256 : best.shape == 1 ? 128 * 128 : 128 * 64;
  for (int mode = 0; mode < 3; ++mode) {
    const long long parts = (best.tiles[mode] * batch - best.whole[mode]) * best.split[mode];
    units = std::max(units, best.whole[mode] + parts);
    most = std::max(most, (size_t)parts * area);
  }
  best.ctas = std::min(units, slots) * (best.shape == 0 ? 2 : 1);
  best.parts = (int)std::min<long long>(592, ceil_div(m * n, 8192));
  best.x = (size_t)2 * batch * best.mp * best.np;
  best.s = (size_t)2 * batch * best.mp * best.mp;
  best.partial = most;
  best.bytes = 2 * (2 * best.x + 2 * best.s) + 4 * best.partial +
               (size_t)3 * batch * best.parts * sizeof(double) + 256;
  return best;
}

// Bounds of the spectral norms: of X_t in bx[0 .. steps], of R in br[t], each with a margin of 2% for
// the roundings. With y = x^2 the polynomials are r(y) = b y + c y^2 and x (a + r(x^2)); on [0, bx[t]]
// their extremes lie at the ends or where the derivative vanishes. False where a bound leaves the range
// of FP32 scales.
static bool bounds(const float *co, int steps, double *bx, double *br) {
  const double a = co[0], b = co[1], c = co[2];
  const double disc = 9.0 * b * b - 20.0 * a * c, w = std::sqrt(std::max(disc, 0.0));
  // zeros of r'(y) = b + 2 c y and of (x r(x^2))' = a + 3 b y + 5 c y^2 (NaN or infinite where
  // there is none: no comparison takes those)
  const double zeros[4] = {-b / (2.0 * c), (-3.0 * b + w) / (10.0 * c), (-3.0 * b - w) / (10.0 * c),
                           -a / (3.0 * b)};
  bx[0] = 1.02;
  for (int t = 0; t < steps; ++t) {
    const double top = bx[t] * bx[t];
    double mx = 0.0, mr = 0.0;
    const auto at = [&](double y) {
      const double r = y * (b + y * c);
      mr = std::max(mr, std::fabs(r));
      mx = std::max(mx, std::fabs(a + r) * std::sqrt(y));
    };
    at(0.0);
    at(top);
    for (double y : zeros)
      if (y > 0.0 && y < top) at(y);
    bx[t + 1] = std::max(1.02 * mx, 1e-12);
    br[t] = std::max(1.02 * mr, 1e-12);
    if (!(bx[t + 1] < 0x1p60) || !(br[t] < 0x1p60)) return false;
  }
  return true;
}

// Power of two that takes numbers up to `bound` below 2^14 (FP16 ends at 65504).
static float scale_for(double bound) { return (float)std::exp2(14.0 - std::ceil(std::log2(bound))); }

struct Device {
  std::once_flag once;
  cudaError_t err = cudaSuccess;
  int pairs = 0;  // CTA pairs resident at once
};
static Device g_dev[64];

static cudaError_t kernel_setup(const int **pairs) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  Device &d = g_dev[dev];
  std::call_once(d.once, [&d]() {
    const auto set = [](auto k, int bytes) {
      return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    };
    d.err = set(ns_kernel<Pair>, Pair::SMEM_BYTES);
    if (d.err == cudaSuccess) d.err = set(ns_kernel<Wide>, Wide::SMEM_BYTES);
    if (d.err == cudaSuccess) d.err = set(ns_kernel<Narrow>, Narrow::SMEM_BYTES);
    if (d.err == cudaSuccess) d.err = set(ns_kernel<FineWide>, FineWide::SMEM_BYTES);
    if (d.err == cudaSuccess) d.err = set(ns_kernel<FineNarrow>, FineNarrow::SMEM_BYTES);
    if (d.err == cudaSuccess)
      d.pairs = cluster_ctas_of(ns_kernel<Pair>, Pair::THREADS, Pair::SMEM_BYTES, 2) / 2;
  });
  *pairs = &d.pairs;
  return d.err;
}

// All CTAs wait for one another, so the launch is cooperative: it starts when all fit.
template <class C>
static cudaError_t launch(const Maps &m, const Params &p, int ctas, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas, 1, 1);
  cfg.blockDim = dim3(C::THREADS, 1, 1);
  cfg.dynamicSmemBytes = C::SMEM_BYTES;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = C::PAIR ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, ns_kernel<C>, m, p);
}

static cudaError_t run(const Plan &l, const float *co, const double *bx, const double *br,
                       Params &p, char *ws, cudaStream_t stream) {
  p.mp = (int)l.mp;
  p.np = (int)l.np;
  p.half = p.batch * l.mp;
  p.x[0] = reinterpret_cast<__half *>(ws);
  p.x[1] = p.x[0] + l.x;
  p.s = p.x[1] + l.x;
  p.r = p.s + l.s;
  p.partial = reinterpret_cast<float *>(p.r + l.s);
  double *part = reinterpret_cast<double *>(p.partial + l.partial);
  p.part = part;
  p.parts = l.parts;
  p.counter = reinterpret_cast<unsigned *>(part + (size_t)3 * p.batch * l.parts);
  p.x_scale = p.steps > 0 ? scale_for(bx[0]) : 1.0f;
  const long long rows = 2 * p.half;  // hi, then lo
  long long units = (long long)p.batch * l.parts;
  for (int mode = 0; mode < 3; ++mode) {
    p.tiles[mode] = (int)l.tiles[mode];
    p.whole[mode] = (int)l.whole[mode];
    p.split[mode] = l.split[mode];
    units = std::max(units, p.batch * l.tiles[mode] * l.split[mode] * 64);
  }
  units = std::max(units, l.mp / 128 * (l.np / 128) * p.batch);
  if (rows > 0x7fffffffLL || l.np > 0x7fffffffLL || units > 0x7fffffffLL)
    return cudaErrorInvalidConfiguration;
  cudaError_t e = launch_1d(norm_kernel, p.batch * l.parts, 256, 0, 1, stream, p.in, part, l.parts,
                            p.counter);
  if (e != cudaSuccess) return e;
  if (p.steps == 0) {
    const long long blocks = std::min<long long>(1024, ceil_div((long long)p.m * p.n, 1024));
    const unsigned mats = (unsigned)std::min(p.batch, 65535);  // (the most of a grid's y)
    copy_kernel<<<dim3((unsigned)blocks, mats), 256, 0, stream>>>(p);
    return cudaGetLastError();
  }
  float sx = p.x_scale;
  for (int t = 0; t < p.steps; ++t) {
    const float ss = scale_for(bx[t] * bx[t]), sr = scale_for(br[t]), sn = scale_for(bx[t + 1]);
    p.f[t][GRAM] = ss / (sx * sx);
    p.f[t][POLY] = (float)((double)co[2] * sr / ((double)ss * ss));
    p.fs[t] = (float)((double)co[1] * sr / ss);
    const float out = t + 1 < p.steps ? sn : 1.0f;  // scale of what the step leaves
    p.f[t][APPLY] = out / (sr * sx);
    p.fx[t] = (float)((double)co[0] * out / sx);
    sx = sn;
  }
  Maps m;
  const __half *const at[4] = {p.x[0], p.x[1], p.s, p.r};
  for (int i = 0; i < 4; ++i) {
    const long long ld = i < 2 ? l.np : l.mp;
    if (!encode_map_2d_narrow(&m.large[i], at[i], 2, rows, ld, ld, 128) ||
        !encode_map_2d_narrow(&m.small[i], at[i], 2, rows, ld, ld, BOX))
      return cudaErrorInvalidValue;
  }
  const bool fine = l.mp == 128;
  if (l.shape == 0) return launch<Pair>(m, p, (int)l.ctas, stream);
  if (l.shape == 1)
    return fine ? launch<FineWide>(m, p, (int)l.ctas, stream) : launch<Wide>(m, p, (int)l.ctas, stream);
  return fine ? launch<FineNarrow>(m, p, (int)l.ctas, stream)
              : launch<Narrow>(m, p, (int)l.ctas, stream);
}

}  // namespace ns
}  // namespace sgemm

using namespace sgemm;

extern "C" int ns_orthogonalize_workspace_size(int batch, int rows, int cols, size_t *bytes) {
  if (batch < 0) return -1;
  if (rows < 0) return -2;
  if (cols < 0) return -3;
  if (bytes == nullptr) return 0;
  *bytes = 0;
  if (batch == 0 || rows == 0 || cols == 0) return 0;
  int sms = 0;
  const int whole = 76, *pairs = nullptr;
  if (device_setup(&sms) != cudaSuccess || ns::kernel_setup(&pairs) != cudaSuccess) {
    (void)cudaGetLastError();
    sms = 152;  // no device here: the answer for a whole GB300
    pairs = &whole;
  }
  *bytes = ns::choose(batch, rows, cols, sms, pairs).bytes;
  return 0;
}

extern "C" int ns_orthogonalize_plan(int batch, int rows, int cols, int num_sms, int *tile_cols,
                                     int tiles[3], int whole[3], int split[3]) {
  if (batch < 1) return -1;
  if (rows < 1) return -2;
  if (cols < 1) return -3;
  if (num_sms < 0) return -4;
  int sms = num_sms, pairs = num_sms / 2;
  const int *at_once = nullptr;
  if (num_sms == 0) {
    if (device_setup(&sms) == cudaSuccess && ns::kernel_setup(&at_once) == cudaSuccess) {
      pairs = *at_once;
    } else {
      (void)cudaGetLastError();
      sms = 152;  // no device here: the answer for a whole GB300
      pairs = 76;
    }
  }
  const ns::Plan l = ns::choose(batch, rows, cols, sms, &pairs);
  if (tile_cols) *tile_cols = 256 >> l.shape;
  for (int mode = 0; mode < 3; ++mode) {
    if (l.tiles[mode] * batch > 0x7fffffffLL) return (int)cudaErrorInvalidConfiguration;
    if (tiles) tiles[mode] = (int)(l.tiles[mode] * batch);
    if (whole) whole[mode] = (int)l.whole[mode];
    if (split) split[mode] = l.split[mode];
  }
  return 0;
}

extern "C" int ns_orthogonalize(int batch, int rows, int cols, const void *G, int g_type, int ldg,
                                long long g_stride, int steps, const float *coefficients,
                                float eps, float alpha, float beta, void *out, int out_type,
                                int ldo, long long o_stride, cudaStream_t stream) {
  const bool any = batch > 0 && rows > 0 && cols > 0;
  const auto known = [](int t) { return t == NS_F32 || t == NS_BF16 || t == NS_F16; };
  const auto misplaced = [](const void *q, int t) {
    return reinterpret_cast<uintptr_t>(q) % (t == NS_F32 ? 4 : 2) != 0;
  };
  if (batch < 0) return -1;
  if (rows < 0) return -2;
  if (cols < 0) return -3;
  if (any && G == nullptr) return -4;
  if (!known(g_type)) return -5;
  if (misplaced(G, g_type)) return -4;
  if (ldg < std::max(1, cols)) return -6;
  if (g_stride < 0) return -7;
  if (steps < 0 || steps > 64) return -8;
  double bx[65], br[64];
  if (coefficients == nullptr || !std::isfinite(coefficients[0]) ||
      !std::isfinite(coefficients[1]) || !std::isfinite(coefficients[2]) ||
      !ns::bounds(coefficients, steps, bx, br)) return -9;
  if (!(eps >= 0.0f)) return -10;
  if (any && out == nullptr) return -13;
  if (!known(out_type)) return -14;
  if (misplaced(out, out_type)) return -13;
  if (ldo < std::max(1, cols)) return -15;
  if (o_stride < 0 || (batch > 1 && o_stride < (long long)(rows - 1) * ldo + cols)) return -16;
  if (!any) return 0;

  int sms = 0;
  const int *pairs = nullptr;
  cudaError_t e = device_setup(&sms);
  if (e == cudaSuccess) e = ns::kernel_setup(&pairs);
  if (e != cudaSuccess) return (int)e;
  const ns::Plan l = ns::choose(batch, rows, cols, sms, pairs);
  const auto aligned = [](const void *q, long long a, long long b, int t) {
    const int size = t == NS_F32 ? 4 : 2;
    return reinterpret_cast<uintptr_t>(q) % 16 == 0 && a * size % 16 == 0 && b * size % 16 == 0;
  };
  ns::Params p{};
  p.batch = batch;
  p.steps = steps;
  p.in = ns::Input{G, g_type, rows, cols, ldg, g_stride,
                   (ldg == cols || rows == 1) && aligned(G, 0, batch > 1 ? g_stride : 0, g_type),
                   aligned(G, ldg, batch > 1 ? g_stride : 0, g_type)};
  p.eps = eps;
  p.user = out;
  p.user_type = out_type;
  p.tall = rows > cols;
  p.m = std::min(rows, cols);
  p.n = std::max(rows, cols);
  p.vec = aligned(out, ldo, batch > 1 ? o_stride : 0, out_type);
  p.ldu = ldo;
  p.user_stride = o_stride;
  p.alpha = alpha;
  p.beta = beta;
  char *ws = nullptr;
  e = cudaMallocFromPoolAsync(reinterpret_cast<void **>(&ws), l.bytes, workspace_pool(), stream);
  if (e != cudaSuccess) return (int)e;
  e = ns::run(l, coefficients, bx, br, p, ws, stream);
  const cudaError_t ef = cudaFreeAsync(ws, stream);
  return (int)(e == cudaSuccess ? ef : e);
}

extern "C" int ns_orthogonalize_status(int *status) {
  int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, ns::g_ns_status, sizeof(int));
  if (e != cudaSuccess) return (int)e;
  const int zero = 0;
  e = cudaMemcpyToSymbol(ns::g_ns_status, &zero, sizeof(int));
  if (status) *status = v;
  return (int)e;
}

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
// Three products per step, each one launch of ns_kernel over 128 x 128 tiles:
//   GRAM   S = X X^T              both operands K-major; S is symmetric: tiles on or below the
//                                 diagonal, each written twice
//   POLY   R = a I + b S + c S^2  S symmetric, so K-major twice; R symmetric too
//   APPLY  X' = R X               X read MN-major: no transposed copy of it is ever made
// The identity in R makes X' one product with no addend. The tensor core's
// accumulator is read out after every 64 k and added up in FP32 registers: its own additions
// truncate (with 512 k per accumulator the result at 8 x 1024 x 1024 is 1.5e-5 off, with 64 1.4e-6,
// and 32-bit products give 2.7e-6).
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

constexpr int BT = 128;                   // tile rows and columns
constexpr int BK = 64;                    // k per stage: 128 bytes of FP16
constexpr int TILE_BYTES = BT * BK * 2;   // one operand tile, hi or lo
constexpr int STAGE_BYTES = 4 * TILE_BYTES;
constexpr int STAGES = 3;
constexpr int GROUPS = 2, COLS = BT / GROUPS;
constexpr int EPI_WARPS = 4 * GROUPS, THREADS = 32 * (4 + EPI_WARPS);
constexpr int TMEM_COLS = 2 * BT;
constexpr int BAR_BYTES = 8 * (2 * STAGES + 4) + 16;
constexpr int SMEM_BYTES = 1024 + STAGES * STAGE_BYTES + BAR_BYTES;
static_assert(SMEM_BYTES <= 227 * 1024, "shared memory per CTA");

// kind::f16: D in FP32 (bits 4-5 = 1), FP16 operands (bits 7-9, 10-12 = 0), MN-major Q (bit 16)
// where asked, N / 8 (bits 17-22), M / 16 (bits 24-28).
constexpr uint32_t IDESC = (1u << 4) | ((uint32_t)(BT >> 3) << 17) | ((uint32_t)(BT >> 4) << 24);

enum { GRAM = 0, POLY = 1, APPLY = 2 };

struct Params {
  int batch, mp, np;       // padded sizes of the short and the long side
  int K;                   // contraction: np for GRAM, mp else
  int tiles;               // per matrix
  int tiles_q;             // APPLY: tiles along n
  long long lo_p, lo_q;    // rows between the hi and the lo part of an operand
  float f;                 // factor of the sum
  __half *out;             // hi; lo is lo_out elements further
  long long lo_out;
  const __half *s;         // POLY: S (hi), lo is lo_s elements further
  long long lo_s;
  float fs, diag;          // POLY: factor of S, value added on the diagonal
  // last APPLY: the result in the caller's orientation and type
  void *user;
  int user_type, tall, m, n;
  long long ldu, user_stride;
  float alpha, beta;
};

// Device status word: 0 = fine; 1, 2, 3 = a wait of the producer, the MMA issuer or the
// epilogue gave up.
__device__ int g_ns_status;

__device__ __forceinline__ uint32_t pack_half(__half a, __half b) {
  const __half2 h = __halves2half2(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ void split(float v, __half &hi, __half &lo) {
  hi = __float2half_rn(v);
  lo = __float2half_rn(v - __half2float(hi));
}

// Tile `t` of a matrix: on and below the diagonal for the symmetric results, else all.
template <int MODE>
__device__ __forceinline__ void tile_of(const Params &p, int t, int &tp, int &tq) {
  if constexpr (MODE == APPLY) {
    tile_coords(t, p.mp / BT, p.tiles_q, 8, tp, tq);
  } else {
    int i = (int)((sqrtf(8.0f * t + 1.0f) - 1.0f) * 0.5f);
    while ((i + 1) * (i + 2) / 2 <= t) ++i;
    while (i * (i + 1) / 2 > t) --i;
    tp = i;
    tq = t - i * (i + 1) / 2;
  }
}

template <int MODE, bool LAST>
__global__ void __launch_bounds__(THREADS, 1)
    ns_kernel(const __grid_constant__ CUtensorMap map_p, const __grid_constant__ CUtensorMap map_q,
              const Params p) {
  using namespace tcx;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = saddr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  const uint32_t bars = base + STAGES * STAGE_BYTES;
  const uint32_t acc_full = bars + 8 * (2 * STAGES), acc_empty = acc_full + 16;
  const uint32_t tmem_slot = acc_empty + 16;
  volatile uint32_t *tmem_slot_ptr =
      reinterpret_cast<volatile uint32_t *>(smem_raw + (tmem_slot - raw));
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int total = p.tiles * p.batch;
  const int KT = p.K / BK;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(bars + 8 * s, 1);
      mbar_init(bars + 8 * (STAGES + s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_full + 8 * b, 1);
      mbar_init(acc_empty + 8 * b, EPI_WARPS);
    }
    mbar_init_fence();
    tma_prefetch_map(&map_p);
    tma_prefetch_map(&map_q);
  }
  if (warp == 0) {
    tmem_alloc(tmem_slot, TMEM_COLS);
    tmem_relinquish();
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = *tmem_slot_ptr;
  griddep_wait();  // (launched with programmatic dependent launch: see launch_1d)

  if (warp == 0) {
    // ---- TMA producer: P hi, P lo, Q hi, Q lo of each k step, 64-row boxes of 8 KB
    Ring<STAGES> st;
    int issued = 0;  // (up to STAGES)
    bool ok = true;
    for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
      int tp, tq;
      tile_of<MODE>(p, t % p.tiles, tp, tq);
      const int y0 = t / p.tiles * p.mp;  // first row of the matrix in its buffer
      for (int kt = 0; kt < KT; ++kt) {
        if (!wait_short(bars + 8 * (STAGES + st.slot), st.parity ^ 1u)) {
          if (lane == 0) atomicCAS(&g_ns_status, 0, 1);
          ok = false;
          break;
        }
        if (elect_one()) {
          const uint32_t dst = base + st.slot * STAGE_BYTES, full = bars + 8 * st.slot;
          const int k = kt * BK;
          mbar_expect_tx(full, STAGE_BYTES);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int yp = y0 + (h ? (int)p.lo_p : 0), yq = y0 + (h ? (int)p.lo_q : 0);
            const uint32_t dp = dst + h * TILE_BYTES, dq = dp + 2 * TILE_BYTES;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              tma_load_2d(dp + c * 8192, &map_p, k, yp + tp * BT + 64 * c, full);
              if (MODE == APPLY)
                tma_load_2d(dq + c * 8192, &map_q, tq * BT + 64 * c, yq + k, full);
              else
                tma_load_2d(dq + c * 8192, &map_q, k, yq + tq * BT + 64 * c, full);
            }
          }
        }
        __syncwarp();
        issued = min(issued + 1, STAGES);
        st.next();
      }
    }
    // the last loads issued must have landed before this warp leaves
    for (; issued > 0; --issued) {
      st.parity ^= st.slot == 0 ? 1u : 0u;
      st.slot = st.slot == 0 ? STAGES - 1 : st.slot - 1;
      wait_short(bars + 8 * st.slot, st.parity);
    }
  } else if (warp == 1) {
    // ---- MMA issuer: one k step per TMEM accumulator, the corrections first, so that only four
    // additions meet a sum of full size
    constexpr uint32_t idesc = IDESC | (MODE == APPLY ? 1u << 16 : 0u);
    constexpr uint32_t adv_q = MODE == APPLY ? 16 * 128 : 32;
    Ring<STAGES> st;
    Ring<2> buf;
    bool ok = true;
    for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
      for (int kt = 0; kt < KT; ++kt) {
        if (!wait_short(acc_empty + 8 * buf.slot, buf.parity ^ 1u) ||
            !wait_short(bars + 8 * st.slot, st.parity)) {
          if (lane == 0) atomicCAS(&g_ns_status, 0, 2);
          ok = false;
          break;
        }
        fence_after();
        if (elect_one()) {
          const uint32_t src = base + st.slot * STAGE_BYTES, acc = tmem + buf.slot * BT;
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk) {
            const uint64_t ph = sw128_desc(src + kk * 32, 16);
            const uint64_t pl = sw128_desc(src + TILE_BYTES + kk * 32, 16);
            const uint64_t qh = sw128_desc(src + 2 * TILE_BYTES + kk * adv_q, 8192);
            const uint64_t ql = sw128_desc(src + 3 * TILE_BYTES + kk * adv_q, 8192);
            mma_f16(acc, pl, qh, idesc, kk != 0 ? 1u : 0u);
            mma_f16(acc, ph, ql, idesc, 1u);
          }
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk)
            mma_f16(acc, sw128_desc(src + kk * 32, 16),
                    sw128_desc(src + 2 * TILE_BYTES + kk * adv_q, 8192), idesc, 1u);
          mma_commit(bars + 8 * (STAGES + st.slot));
          mma_commit(acc_full + 8 * buf.slot);
        }
        __syncwarp();
        st.next();
        buf.next();
      }
    }
  } else if (warp >= 4) {
    // ---- epilogue: group grp of four warps owns 64 columns, one row per thread
    const int grp = (warp - 4) >> 2, quad = warp & 3;
    const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)(grp * COLS);
    Ring<2> buf;
    bool ok = true;
    for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
      int tp, tq;
      tile_of<MODE>(p, t % p.tiles, tp, tq);
      const int mat = t / p.tiles;
      const int row = tp * BT + quad * 32 + lane, col0 = tq * BT + grp * COLS;
      float acc[COLS];
#pragma unroll
      for (int j = 0; j < COLS; ++j) acc[j] = 0.0f;
      for (int kt = 0; kt < KT; ++kt) {
        ok = __all_sync(0xffffffffu, wait_short(acc_full + 8 * buf.slot, buf.parity));
        if (!ok) {
          if (lane == 0) atomicCAS(&g_ns_status, 0, 3);
          break;
        }
        fence_after();
#pragma unroll
        for (int j0 = 0; j0 < COLS; j0 += 32) {
          uint32_t v[32];
          tmem_ld(lane_base + buf.slot * BT + (uint32_t)j0, v);
          tmem_wait_ld(v);
#pragma unroll
          for (int j = 0; j < 32; ++j) acc[j0 + j] += __uint_as_float(v[j]);
        }
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acc_empty + 8 * buf.slot);
        buf.next();
      }
      if (!ok) break;

      if constexpr (LAST) {
        if (row < p.m) {
#pragma unroll
          for (int j = 0; j < COLS; ++j) {
            const int col = col0 + j;
            if (col < p.n) {
              const long long at = mat * p.user_stride +
                                   (p.tall ? col * p.ldu + row : row * p.ldu + col);
              float v = p.alpha * (acc[j] * p.f);
              if (p.user_type == NS_F32) {
                float *d = reinterpret_cast<float *>(p.user) + at;
                *d = p.beta != 0.0f ? fmaf(p.beta, *d, v) : v;
              } else if (p.user_type == NS_BF16) {
                __nv_bfloat16 *d = reinterpret_cast<__nv_bfloat16 *>(p.user) + at;
                if (p.beta != 0.0f) v = fmaf(p.beta, __bfloat162float(*d), v);
                *d = __float2bfloat16_rn(v);
              } else {
                __half *d = reinterpret_cast<__half *>(p.user) + at;
                if (p.beta != 0.0f) v = fmaf(p.beta, __half2float(*d), v);
                *d = __float2half_rn(v);
              }
            }
          }
        }
      } else {
        const long long ld = MODE == APPLY ? p.np : p.mp;
        __half *o = p.out + ((long long)mat * p.mp + row) * ld + col0;
        const __half *sh = MODE == POLY ? p.s + ((long long)mat * p.mp + row) * ld + col0 : nullptr;
#pragma unroll
        for (int j0 = 0; j0 < COLS; j0 += 8) {
          float v[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = acc[j0 + j] * p.f;
          if constexpr (MODE == POLY) {
            const uint4 uh = *reinterpret_cast<const uint4 *>(sh + j0);
            const uint4 ul = *reinterpret_cast<const uint4 *>(sh + p.lo_s + j0);
            const uint32_t wh[4] = {uh.x, uh.y, uh.z, uh.w}, wl[4] = {ul.x, ul.y, ul.z, ul.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&wh[j]));
              const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&wl[j]));
              v[2 * j] = fmaf(p.fs, a.x + b.x, v[2 * j]);
              v[2 * j + 1] = fmaf(p.fs, a.y + b.y, v[2 * j + 1]);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (row == col0 + j0 + j) v[j] += p.diag;
          }
          __half hi[8], lo[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) split(v[j], hi[j], lo[j]);
          *reinterpret_cast<uint4 *>(o + j0) =
              make_uint4(pack_half(hi[0], hi[1]), pack_half(hi[2], hi[3]),
                         pack_half(hi[4], hi[5]), pack_half(hi[6], hi[7]));
          *reinterpret_cast<uint4 *>(o + p.lo_out + j0) =
              make_uint4(pack_half(lo[0], lo[1]), pack_half(lo[2], lo[3]),
                         pack_half(lo[4], lo[5]), pack_half(lo[6], lo[7]));
          if (MODE != APPLY && tp != tq) {
            __half *mir = p.out + ((long long)mat * p.mp + col0 + j0) * ld + row;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              mir[j * ld] = hi[j];
              mir[j * ld + p.lo_out] = lo[j];
            }
          }
        }
      }
    }
  }
  __syncwarp();
  griddep_launch_dependents();
  fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, TMEM_COLS);
}

// ------------------------------------------------------------------------------------
// Norm and start values.

template <class T>
__device__ __forceinline__ float load(const void *x, long long i) {
  return (float)reinterpret_cast<const T *>(x)[i];
}
__device__ __forceinline__ float load(const void *x, int type, long long i) {
  if (type == NS_F32) return load<float>(x, i);
  if (type == NS_BF16) return load<__nv_bfloat16>(x, i);
  return load<__half>(x, i);
}

// Squares of numbers over 2^64 overflow FP32 and those under 2^-64 vanish, so each thread sums
// the squares of x, of x 2^-70 and of x 2^70; the last step takes the sum that did neither.
constexpr float kDown = 0x1p-70f, kUp = 0x1p70f;

struct Input {
  const void *g;
  int type, rows, cols;
  long long ld, stride;
};

__global__ void __launch_bounds__(256) norm_kernel(const Input in, double *part, int parts) {
  griddep_wait();
  __shared__ double red[3][8];
  const int mat = blockIdx.x / parts, piece = blockIdx.x % parts;
  const long long total = (long long)in.rows * in.cols;
  const long long first = total * piece / parts, last = total * (piece + 1) / parts;
  float s[3] = {0.0f, 0.0f, 0.0f};
  long long i = first + threadIdx.x;
  int r = (int)(i / in.cols), c = (int)(i % in.cols);
  for (; i < last; i += 256) {
    const float x = load(in.g, in.type, mat * in.stride + r * in.ld + c);
    s[0] = fmaf(x, x, s[0]);
    s[1] = fmaf(x * kDown, x * kDown, s[1]);
    s[2] = fmaf(x * kUp, x * kUp, s[2]);
    for (c += 256; c >= in.cols; c -= in.cols) ++r;
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
  griddep_launch_dependents();
}

// X_0 times its scale, split, in the short orientation, with zero padding. 64 x 64 tiles; a tall
// G is turned in shared memory.
__global__ void __launch_bounds__(256)
    start_kernel(const Input in, const double *part, int parts, double eps, float scale, int tall,
                 int mp, int np, __half *x, long long lo) {
  griddep_wait();
  __shared__ float t[64][65];
  __shared__ float mul[2];
  const int tiles_n = np / 64, per = tiles_n * (mp / 64);
  const int mat = blockIdx.x / per, tile = blockIdx.x % per;
  const int r0 = tile / tiles_n * 64, c0 = tile % tiles_n * 64;
  if (threadIdx.x < 32) {
    double s[3] = {0.0, 0.0, 0.0};
    for (int i = threadIdx.x; i < parts; i += 32)
      for (int q = 0; q < 3; ++q) s[q] += part[((long long)mat * parts + i) * 3 + q];
#pragma unroll
    for (int q = 0; q < 3; ++q)
#pragma unroll
      for (int o = 16; o > 0; o /= 2) s[q] += __shfl_xor_sync(0xffffffffu, s[q], o);
    if (threadIdx.x == 0) {
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
      mul[1] = norm + eps > 0.0 ? (float)(scale / (norm + eps) / pre) : (float)(norm * 0.0);
    }
  }
  __syncthreads();
  const float pre = mul[0], f = mul[1];
  const int a = threadIdx.x & 63, b = threadIdx.x >> 6;
  if (tall) {
#pragma unroll 4
    for (int i = 0; i < 16; ++i) {
      const int n = c0 + b + 4 * i, m = r0 + a;  // G is n x m
      t[a][b + 4 * i] = n < in.rows && m < in.cols
                            ? load(in.g, in.type, mat * in.stride + n * in.ld + m)
                            : 0.0f;
    }
    __syncthreads();
  }
#pragma unroll 4
  for (int i = 0; i < 16; ++i) {
    const int m = r0 + b + 4 * i, n = c0 + a;
    float v;
    if (tall)
      v = t[b + 4 * i][a];
    else
      v = m < in.rows && n < in.cols ? load(in.g, in.type, mat * in.stride + m * in.ld + n) : 0.0f;
    __half hi, lw;
    split(v * pre * f, hi, lw);
    __half *o = x + ((long long)mat * mp + m) * np + n;
    o[0] = hi;
    o[lo] = lw;
  }
  griddep_launch_dependents();
}

// steps == 0: out = alpha X_0 + beta out.
__global__ void __launch_bounds__(256)
    copy_kernel(const __half *x, long long lo, float f, Params p) {
  griddep_wait();
  const long long total = (long long)p.batch * p.m * p.n;
  for (long long i = blockIdx.x * 256LL + threadIdx.x; i < total; i += gridDim.x * 256LL) {
    const int mat = (int)(i / ((long long)p.m * p.n));
    const long long e = i % ((long long)p.m * p.n);
    const int row = (int)(e / p.n), col = (int)(e % p.n);
    const __half *s = x + ((long long)mat * p.mp + row) * p.np + col;
    const long long at =
        mat * p.user_stride + (p.tall ? col * p.ldu + row : row * p.ldu + col);
    float v = p.alpha * (f * (__half2float(s[0]) + __half2float(s[lo])));
    if (p.beta != 0.0f) v = fmaf(p.beta, load(p.user, p.user_type, at), v);
    if (p.user_type == NS_F32)
      reinterpret_cast<float *>(p.user)[at] = v;
    else if (p.user_type == NS_BF16)
      reinterpret_cast<__nv_bfloat16 *>(p.user)[at] = __float2bfloat16_rn(v);
    else
      reinterpret_cast<__half *>(p.user)[at] = __float2half_rn(v);
  }
}

// ------------------------------------------------------------------------------------
// Host side

struct Layout {
  long long m, n, mp, np;       // short and long side, padded to whole tiles
  int parts;                    // pieces of a matrix in the norm
  size_t x, s, part, bytes;     // element counts (FP16) of one X, of one S; bytes of all
};

static Layout layout(int batch, int rows, int cols) {
  Layout l;
  l.m = std::min(rows, cols);
  l.n = std::max(rows, cols);
  l.mp = ceil_div(l.m, BT) * BT;
  l.np = ceil_div(l.n, BT) * BT;
  l.parts = (int)std::min<long long>(128, ceil_div(l.m * l.n, 4096));
  l.x = (size_t)2 * batch * l.mp * l.np;
  l.s = (size_t)2 * batch * l.mp * l.mp;
  l.part = (size_t)3 * batch * l.parts * sizeof(double);
  l.bytes = 2 * (2 * l.x + 2 * l.s) + l.part;
  return l;
}

// Bounds of the spectral norms: of X_t in bx[0 .. steps], of a I + b S + c S^2 in br[t], each with
// a margin of 2% for the roundings. With y = x^2 the polynomials are r(y) = a + b y + c y^2 and
// x r(x^2); on [0, bx[t]] their extremes lie at the ends or where the derivative vanishes. False
// where a bound leaves the range of FP32 scales.
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
      const double r = std::fabs(a + y * (b + y * c));
      mr = std::max(mr, r);
      mx = std::max(mx, r * std::sqrt(y));
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

static std::once_flag g_once[64];
static cudaError_t g_err[64];

static cudaError_t kernel_setup() {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::call_once(g_once[dev], [dev]() {
    const auto set = [](auto k) {
      return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
    };
    cudaError_t err = set(ns_kernel<GRAM, false>);
    if (err == cudaSuccess) err = set(ns_kernel<POLY, false>);
    if (err == cudaSuccess) err = set(ns_kernel<APPLY, false>);
    if (err == cudaSuccess) err = set(ns_kernel<APPLY, true>);
    g_err[dev] = err;
  });
  return g_err[dev];
}

static cudaError_t run(const Layout &l, const Input &in, int batch, int steps, const float *co,
                       const double *bx, const double *br, float eps, Params p, __half *ws,
                       int sms, cudaStream_t stream) {
  __half *x[2] = {ws, ws + l.x};
  __half *s = x[1] + l.x, *r = s + l.s;
  double *part = reinterpret_cast<double *>(r + l.s);
  const long long rows = 2LL * batch * l.mp;   // hi, then lo
  if (rows > 0x7fffffffLL || l.np > 0x7fffffffLL) return cudaErrorInvalidValue;
  CUtensorMap mx[2], ms, mr;
  if (!encode_map_2d_narrow(&mx[0], x[0], 2, rows, l.np, l.np, 64) ||
      !encode_map_2d_narrow(&mx[1], x[1], 2, rows, l.np, l.np, 64) ||
      !encode_map_2d_narrow(&ms, s, 2, rows, l.mp, l.mp, 64) ||
      !encode_map_2d_narrow(&mr, r, 2, rows, l.mp, l.mp, 64))
    return cudaErrorInvalidValue;
  const long long starts = (l.mp / 64) * (l.np / 64) * batch;
  const long long tm = l.mp / BT, tn = l.np / BT;
  if (starts > 0x7fffffffLL || (long long)batch * l.parts > 0x7fffffffLL)
    return cudaErrorInvalidConfiguration;
  float sx = scale_for(bx[0]);
  cudaError_t e = launch_1d(norm_kernel, batch * l.parts, 256, 0, 1, stream, in, part, l.parts);
  if (e == cudaSuccess)
    e = launch_1d(start_kernel, (int)starts, 256, 0, 1, stream, in, part, l.parts, (double)eps, sx,
                  p.tall, (int)l.mp, (int)l.np, x[0], (long long)(l.x / 2));
  if (e != cudaSuccess) return e;
  p.mp = (int)l.mp;
  p.np = (int)l.np;
  if (steps == 0) {
    const long long blocks = std::min<long long>(8LL * sms, ceil_div(batch * l.m * l.n, 256));
    return launch_1d(copy_kernel, (int)blocks, 256, 0, 1, stream, x[0], (long long)(l.x / 2),
                     1.0f / sx, p);
  }
  const long long half_rows = (long long)batch * l.mp;
  p.lo_p = p.lo_q = half_rows;
  const auto grid = [&](long long tiles) { return (int)std::min<long long>(tiles * batch, sms); };
  for (int t = 0; t < steps; ++t) {
    const float ss = scale_for(bx[t] * bx[t]), sr = scale_for(br[t]), sn = scale_for(bx[t + 1]);
    Params q = p;
    q.K = (int)l.np;
    q.tiles = (int)(tm * (tm + 1) / 2);
    q.f = ss / (sx * sx);
    q.out = s;
    q.lo_out = (long long)(l.s / 2);
    e = launch_1d(ns_kernel<GRAM, false>, grid(q.tiles), THREADS, SMEM_BYTES, 1, stream, mx[t & 1],
                  mx[t & 1], q);
    if (e != cudaSuccess) return e;
    q.K = (int)l.mp;
    q.f = (float)((double)co[2] * sr / ((double)ss * ss));
    q.fs = (float)((double)co[1] * sr / ss);
    q.diag = co[0] * sr;
    q.s = s;
    q.lo_s = (long long)(l.s / 2);
    q.out = r;
    e = launch_1d(ns_kernel<POLY, false>, grid(q.tiles), THREADS, SMEM_BYTES, 1, stream, ms, ms, q);
    if (e != cudaSuccess) return e;
    q.tiles = (int)(tm * tn);
    q.tiles_q = (int)tn;
    q.lo_out = (long long)(l.x / 2);
    q.out = x[(t + 1) & 1];
    if (t + 1 < steps) {
      q.f = sn / (sr * sx);
      e = launch_1d(ns_kernel<APPLY, false>, grid(q.tiles), THREADS, SMEM_BYTES, 1, stream, mr,
                    mx[t & 1], q);
    } else {
      q.f = 1.0f / (sr * sx);
      e = launch_1d(ns_kernel<APPLY, true>, grid(q.tiles), THREADS, SMEM_BYTES, 1, stream, mr,
                    mx[t & 1], q);
    }
    if (e != cudaSuccess) return e;
    sx = sn;
  }
  return cudaSuccess;
}

}  // namespace ns
}  // namespace sgemm

using namespace sgemm;

extern "C" int ns_orthogonalize_workspace_size(int batch, int rows, int cols, size_t *bytes) {
  if (batch < 0) return -1;
  if (rows < 0) return -2;
  if (cols < 0) return -3;
  if (bytes) *bytes = batch == 0 || rows == 0 || cols == 0 ? 0 : ns::layout(batch, rows, cols).bytes;
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
  cudaError_t e = device_setup(&sms);
  if (e == cudaSuccess) e = ns::kernel_setup();
  if (e != cudaSuccess) return (int)e;
  const ns::Layout l = ns::layout(batch, rows, cols);
  ns::Params p{};
  p.batch = batch;
  p.user = out;
  p.user_type = out_type;
  p.tall = rows > cols;
  p.m = (int)l.m;
  p.n = (int)l.n;
  p.ldu = ldo;
  p.user_stride = o_stride;
  p.alpha = alpha;
  p.beta = beta;
  __half *ws = nullptr;
  e = cudaMallocFromPoolAsync(reinterpret_cast<void **>(&ws), l.bytes, workspace_pool(), stream);
  if (e != cudaSuccess) return (int)e;
  const ns::Input in{G, g_type, rows, cols, ldg, g_stride};
  e = ns::run(l, in, batch, steps, coefficients, bx, br, eps, p, ws, sms, stream);
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

// The linear layer on 8-bit integers for few rows of x (a few tokens in serving), and the conversion of
// int8 to FP16 in front of large products.
//
// Few rows: bound by HBM, the weight is read once. A warp takes four channels (rows of w) and a part
// of k; each lane multiplies 16 bytes of each of them with the same 16 bytes of each row of x, four
// products per instruction (dp4a), and adds them up in 32-bit integers. x stays in L1. The sums are
// whole numbers, so that any order of adding them gives the same bits.
#include <algorithm>

#include "i8_internal.h"
#include "sgemm_ffma.cuh"
#include "sgemm_internal.h"
#include "sgemm_plan.h"
#include "tc_common.cuh"

namespace sgemm {
namespace i8 {

constexpr int kDotRows = 2;    // rows of x for which dp4a is as fast as the weight arrives
constexpr int kWarps = 8;      // per CTA
constexpr int kChannels = 4;   // per warp

struct FewParams {
  int M, N, K;
  Operand x, w;
  Result d;
  int parts;           // warps of a CTA that share the channels, each with its part of k
};

// 16 bytes from k on; those past K are zero and not read. (x has been written by the kernel before this
// one, which may still run when a CTA of this one begins: no load by the non-coherent path.)
__device__ __forceinline__ uint4 load16(const int8_t *row, int k, int K, bool stream) {
  if (k + 16 <= K) {
    const uint4 *s = reinterpret_cast<const uint4 *>(row + k);
    return stream ? __ldcs(s) : *s;
  }
  uint32_t u[4] = {};
#pragma unroll
  for (int j = 0; j < 16; ++j)
    if (k + j < K) u[j / 4] |= (uint32_t)(uint8_t)row[k + j] << (8 * (j & 3));
  return make_uint4(u[0], u[1], u[2], u[3]);
}

__device__ __forceinline__ int dot16(const uint4 &a, const uint4 &b, int c) {
  c = __dp4a((int)a.x, (int)b.x, c);
  c = __dp4a((int)a.y, (int)b.y, c);
  c = __dp4a((int)a.z, (int)b.z, c);
  return __dp4a((int)a.w, (int)b.w, c);
}

template <int MT>
__global__ void __launch_bounds__(32 * kWarps) few_kernel(const FewParams p) {
  __shared__ int sums[kWarps][kChannels][MT];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int groups = kWarps / p.parts;  // of channels per CTA
  const int part = warp % p.parts;
  const long long n0 = ((long long)blockIdx.x * groups + warp / p.parts) * kChannels;
  // the part's k, in steps of 512
  const int steps = (p.K + 511) / 512;
  const int k0 = (int)((long long)steps * part / p.parts) * 512;
  const int k1 = min(p.K, (int)((long long)steps * (part + 1) / p.parts) * 512);
  const int8_t *w[kChannels];
#pragma unroll
  for (int c = 0; c < kChannels; ++c) w[c] = p.w.q + min(n0 + c, (long long)p.N - 1) * p.w.ld;
  int acc[kChannels][MT] = {};
  griddep_wait();  // (launched with programmatic dependent launch: see launch_1d)
#pragma unroll 2
  for (int k = k0 + 16 * lane; k < k1; k += 512) {
    uint4 wv[kChannels];
#pragma unroll
    for (int c = 0; c < kChannels; ++c) wv[c] = load16(w[c], k, p.K, true);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const uint4 xv = load16(p.x.q + (MT == 1 ? 0 : min(m, p.M - 1) * p.x.ld), k, p.K, false);
#pragma unroll
      for (int c = 0; c < kChannels; ++c) acc[c][m] = dot16(wv[c], xv, acc[c][m]);
    }
  }
#pragma unroll
  for (int c = 0; c < kChannels; ++c)
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int s = __reduce_add_sync(0xffffffffu, acc[c][m]);
      if (lane == 0) sums[warp][c][m] = s;
    }
  __syncthreads();
  for (int i = threadIdx.x; i < groups * kChannels * MT; i += 32 * kWarps) {
    const int c = i % (groups * kChannels), m = i / (groups * kChannels);
    const long long n = (long long)blockIdx.x * groups * kChannels + c;
    if (n < p.N && m < p.M) {
      int s = 0;
      for (int q = 0; q < p.parts; ++q) s += sums[c / kChannels * p.parts + q][c % kChannels][m];
      const float y = fmaf((float)s, p.w.scale[n] * p.x.scale[m], p.d.bias ? p.d.bias[n] : 0.0f);
      tcx::finish_out(p.d.ptr, p.d.type, m * p.d.ld + n, y, p.d.beta);
    }
  }
  griddep_launch_dependents();
}

// More rows than that (up to 32): the same on warp-wide matrix instructions (mma.sync, FP16 operands, FP32
// sums). tcgen05 would need tiles of 128 channels per CTA, its accumulators' set-up and their way back for
// a handful of tokens; here the weight goes from memory to registers, is converted there and used. A
// warp multiplies 16 channels with 8 NT rows of x; which k a lane's operands stand for is the same for
// both operands, and that is all the sum needs, so each lane converts 16 neighbouring bytes of two
// channels at a time. x is converted once per CTA, 1024 of k at a time, into shared memory, in the order
// in which the lanes take it. FP32 holds the sums of 1024 k exactly. The CTAs of a cluster take a part
// of k each and add their sums up through distributed shared memory.
constexpr int kStep = 128;     // k of a warp at a time: twice 16 for each of 4 lanes
constexpr int kRound = 8;      // steps for which x is in shared memory
constexpr int kSomeWarps = 4;  // per CTA
constexpr int kSomeChannels = 16 * kSomeWarps;
constexpr int kPitch = kSomeChannels + 4;  // of the sums

template <int NT>
struct Some {
  static constexpr int TOK = 8 * NT;
  static constexpr int RAW = TOK * kStep * kRound;  // bytes of x as it comes
  static constexpr int BYTES = 3 * RAW;             // and in FP16
  static_assert(TOK * kPitch * 4 <= 2 * RAW, "the sums take the place of x");
};

__device__ __forceinline__ void mma_16x8x16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t word(const uint4 &v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// p.parts: CTAs of a cluster.
template <int NT>
__global__ void __launch_bounds__(32 * kSomeWarps, NT == 4 ? 3 : 4) some_kernel(const FewParams p) {
  using S = Some<NT>;
  extern __shared__ __align__(16) uint8_t smem[];
  uint8_t *raw = smem + 2 * S::RAW;  // [step][n][half][lane] 16 bytes; before it FP16: [step][n][quarter][lane]
  const uint32_t raw_at = saddr(raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int rank = (int)(blockIdx.x % (unsigned)p.parts);
  const long long n0 = (long long)(blockIdx.x / (unsigned)p.parts) * kSomeChannels;
  const int steps = (p.K + kStep - 1) / kStep;
  const int s0 = (int)((long long)steps * rank / p.parts), s1 = (int)((long long)steps * (rank + 1) / p.parts);
  const int8_t *w[2];
#pragma unroll
  for (int c = 0; c < 2; ++c) w[c] = p.w.q + min(n0 + 16 * warp + 8 * c + g, (long long)p.N - 1) * p.w.ld;
  uint4 ahead[2][2][2];  // two steps' bytes of two channels
  const auto load = [&](uint4 (&v)[2][2], int s) {
    if (s < s1) {
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h) v[c][h] = load16(w[c], s * kStep + 64 * h + 16 * t, p.K, true);
      __syncwarp();  // (lanes at the end of a row took longer)
    }
  };
  // x of the steps from `s` on: thread (g, t) of a warp copies what lane (g, t) will use
  const auto copy = [&](int s) {
    const int pieces = min(kRound, s1 - s) * NT * 2;
    for (int i = warp; i < pieces; i += kSomeWarps) {
      const int h = i & 1, n = i / 2 % NT, at = i / (2 * NT);
      const int token = 8 * n + g, k = (s + at) * kStep + 64 * h + 16 * t;
      const int bytes = token < p.M ? max(0, min(16, p.K - k)) : 0;
      cp_async_16(raw_at + i * 512 + lane * 16, p.x.q + (bytes ? token * p.x.ld + k : 0), bytes);
    }
    cp_async_commit();
  };
  float acc[NT][4];
  int total[NT][4] = {};
  griddep_wait();
  copy(s0);
  load(ahead[0], s0);
  load(ahead[1], s0 + 1);
  const auto multiply = [&](const uint4 (&v)[2][2], int at) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint4 b[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n)
          b[n] = *reinterpret_cast<const uint4 *>(smem + ((at * NT + n) * 4 + 2 * h + q) * 512 + lane * 16);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t a[4];
          tcx::halves(word(v[0][h], 2 * q + j), a[0], a[2]);
          tcx::halves(word(v[1][h], 2 * q + j), a[1], a[3]);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma_16x8x16(acc[n], a, word(b[n], 2 * j), word(b[n], 2 * j + 1));
        }
      }
  };
  for (int r = s0; r < s1; r += kRound) {
    const int count = min(kRound, s1 - r);
    cp_async_wait<0>();
    __syncthreads();  // (x has come, and everybody is done with the last round's)
    for (int i = warp; i < count * NT * 2; i += kSomeWarps) {
      const uint4 u = *reinterpret_cast<const uint4 *>(raw + i * 512 + lane * 16);
      uint4 lo, hi;
      tcx::halves(u.x, lo.x, lo.y);
      tcx::halves(u.y, lo.z, lo.w);
      tcx::halves(u.z, hi.x, hi.y);
      tcx::halves(u.w, hi.z, hi.w);
      *reinterpret_cast<uint4 *>(smem + 2 * i * 512 + lane * 16) = lo;
      *reinterpret_cast<uint4 *>(smem + (2 * i + 1) * 512 + lane * 16) = hi;
    }
    __syncthreads();
    if (r + kRound < s1) copy(r + kRound);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][i] = 0.0f;
    for (int at = 0; at < count; at += 2) {
      uint4 v[2][2][2];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i / 4][i / 2 % 2][i % 2] = ahead[i / 4][i / 2 % 2][i % 2];
      load(ahead[0], r + at + 2);
      load(ahead[1], r + at + 3);
      multiply(v[0], at);
      if (at + 1 < count) multiply(v[1], at + 1);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) total[n][i] += __float2int_rn(acc[n][i]);
  }
  __syncthreads();
  int *sums = reinterpret_cast<int *>(smem);  // [token][channel]
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      sums[(8 * n + 2 * t + (i & 1)) * kPitch + 16 * warp + 8 * (i >> 1) + g] = total[n][i];
  if (p.parts > 1)
    cluster_sync_all();
  else
    __syncthreads();
  for (int i = rank * 32 * kSomeWarps + tid; i < kSomeChannels * S::TOK; i += p.parts * 32 * kSomeWarps) {
    const int c = i % kSomeChannels, m = i / kSomeChannels;
    const long long n = n0 + c;
    if (n < p.N && m < p.M) {
      int s = 0;
      if (p.parts > 1) {
        for (int q = 0; q < p.parts; ++q)
          s += __float_as_int(tcx::ld_cluster1(saddr(sums + m * kPitch + c), (uint32_t)q));
      } else {
        s = sums[m * kPitch + c];
      }
      const float y = fmaf((float)s, p.w.scale[n] * p.x.scale[m], p.d.bias ? p.d.bias[n] : 0.0f);
      tcx::finish_out(p.d.ptr, p.d.type, m * p.d.ld + n, y, p.d.beta);
    }
  }
  __syncwarp();
  if (p.parts > 1) cluster_sync_all();  // no CTA leaves while another may still read its sums
  griddep_launch_dependents();
}

template <int NT>
static cudaError_t launch_some(FewParams p, int sms, cudaStream_t stream) {
  // as many CTAs as are resident at once, and at least two rounds of x for each
  const long long columns = ceil_div(p.N, kSomeChannels);
  const int at_once = (NT == 4 ? 2 : 4) * sms, steps = (int)ceil_div(p.K, kStep);
  while (p.parts < 8 && 2 * columns * p.parts <= at_once && 2 * p.parts <= steps) p.parts *= 2;
  return launch_1d(some_kernel<NT>, (int)(columns * p.parts), 32 * kSomeWarps, Some<NT>::BYTES, p.parts, stream, p);
}

cudaError_t launch_few(int M, int N, int K, const Operand &x, const Operand &w, const Result &d, int sms,
                       cudaStream_t stream) {
  FewParams p{M, N, K, x, w, d, 1};
  if (M > kDotRows)
    return M <= 8    ? launch_some<1>(p, sms, stream)
           : M <= 16 ? launch_some<2>(p, sms, stream)
                     : launch_some<4>(p, sms, stream);
  // more warps on the same channels where there are too few of them to fill the GPU
  const long long groups = ceil_div(N, kChannels);
  while (p.parts < kWarps && groups * p.parts < 16LL * sms && 512 * p.parts < K) p.parts *= 2;
  const int grid = (int)ceil_div(groups * p.parts, kWarps);
  if (M == 1) return launch_1d(few_kernel<1>, grid, 32 * kWarps, 0, 1, stream, p);
  return launch_1d(few_kernel<2>, grid, 32 * kWarps, 0, 1, stream, p);
}

cudaError_t few_setup() {
  const auto set = [](void (*kernel)(FewParams), int bytes) {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  };
  cudaError_t e = set(some_kernel<1>, Some<1>::BYTES);
  if (e == cudaSuccess) e = set(some_kernel<2>, Some<2>::BYTES);
  if (e == cudaSuccess) e = set(some_kernel<4>, Some<4>::BYTES);
  return e;
}

// ------------------------------------------------------------------------------------

__global__ void __launch_bounds__(256) unpack_kernel(const int8_t *q, long long ldq, int rows, int K,
                                                     __half *out, long long ldo) {
  griddep_wait();
  const int chunks = (K + 15) / 16;
  const long long total = (long long)rows * chunks;
  for (long long i = blockIdx.x * 256LL + threadIdx.x; i < total; i += 256LL * gridDim.x) {
    const long long r = i / chunks;
    const int k = (int)(i % chunks) * 16;
    const uint4 v = load16(q + r * ldq, k, K, false);
    uint4 lo, hi;
    tcx::halves(v.x, lo.x, lo.y);
    tcx::halves(v.y, lo.z, lo.w);
    tcx::halves(v.z, hi.x, hi.y);
    tcx::halves(v.w, hi.z, hi.w);
    uint4 *d = reinterpret_cast<uint4 *>(out + r * ldo + k);  // (the workspace's rows have room)
    d[0] = lo;
    d[1] = hi;
  }
  griddep_launch_dependents();
}

cudaError_t launch_unpack(int rows, int K, const Operand &q, void *out, long long ldo, int sms,
                          cudaStream_t stream) {
  const long long total = (long long)rows * ceil_div(K, 16);
  const long long grid = std::min<long long>(ceil_div(total, 256), 8LL * sms);
  return launch_1d(unpack_kernel, (int)grid, 256, 0, 1, stream, q.q, q.ld, rows, K,
                   static_cast<__half *>(out), ldo);
}

}  // namespace i8
}  // namespace sgemm

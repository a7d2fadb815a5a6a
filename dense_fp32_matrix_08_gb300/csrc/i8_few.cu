// The linear layer on 8-bit integers for few rows of x (a few tokens in serving), and the conversion of
// int8 to FP16 in front of large products.
//
// Few rows: bound by HBM, the weight is read once. A warp takes four channels (rows of w) and a part
// of k; each lane multiplies 16 bytes of each of them with the same 16 bytes of each row of x, four
// products per instruction (dp4a), and adds them up in 32-bit integers. x stays in L1. The sums are
// whole numbers, so that any order of adding them gives the same bits. 1 x 14336 x 4096: 10.0 us, 5.9 TB/s
// (87% of a copy's rate); 1 x 4096 x 14336: 9.1 us; 1 x 4096 x 4096: 3.1 us, in a stream of calls. Four CTAs
// per SM, 64 registers (of which two rows spill 24 bytes, one none): with five more spills (1 x 4096 x 14336: 14.3
// us), with three there is too little under way (13.9).
#include <algorithm>

#include "i8_internal.h"
#include "sgemm_ffma.cuh"
#include "sgemm_internal.h"
#include "sgemm_plan.h"
#include "tc_common.cuh"

namespace sgemm {
namespace i8 {

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
__global__ void __launch_bounds__(32 * kWarps, 4) few_kernel(const FewParams p) {
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
  // The weight's first part begins its way to L2 while the kernel before this one still runs. (To L2 only,
  // where what that kernel may yet write to it is seen.) The next launch may take what room there is.
  // 1 x 4096 x 4096, one call after the other: 4.3 us without, 3.1 so; 1 x 14336 x 4096: 11.0 and 10.0, 10.9
  // with twice as much.
#pragma unroll
  for (int c = 0; c < kChannels; ++c)
    for (int k = k0 + 128 * lane; k < min(k1, k0 + 1024); k += 128 * 32)
      asm volatile("prefetch.global.L2 [%0];\n" ::"l"(w[c] + k));
  griddep_launch_dependents();
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
}

cudaError_t launch_few(int M, int N, int K, const Operand &x, const Operand &w, const Result &d, int sms,
                       cudaStream_t stream) {
  FewParams p{M, N, K, x, w, d, 1};
  // more warps on the same channels where there are too few of them to fill the GPU
  const long long groups = ceil_div(N, kChannels);
  while (p.parts < kWarps && groups * p.parts < 16LL * sms && 512 * p.parts < K) p.parts *= 2;
  const int grid = (int)ceil_div(groups * p.parts, kWarps);
  if (M == 1) return launch_1d(few_kernel<1>, grid, 32 * kWarps, 0, 1, stream, p);
  return launch_1d(few_kernel<2>, grid, 32 * kWarps, 0, 1, stream, p);
}

// ------------------------------------------------------------------------------------

__global__ void __launch_bounds__(256) unpack_kernel(const int8_t *q, long long ldq, int rows, int K,
                                                     __half *out, long long ldo) {
  griddep_launch_dependents();
  griddep_wait();
  const int chunks = (K + 15) / 16;
  const long long start = blockIdx.x * 256LL + threadIdx.x, step = 256LL * gridDim.x;
  const int step_r = (int)(step / chunks), step_c = (int)(step % chunks);
  long long r = start / chunks;
  int c = (int)(start % chunks);
  for (; r < rows; r += step_r, c += step_c) {
    if (c >= chunks) {
      c -= chunks;
      if (++r >= rows) break;
    }
    const int k = c * 16;
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

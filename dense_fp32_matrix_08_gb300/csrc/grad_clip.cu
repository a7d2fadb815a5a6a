// The norm of many arrays together, and the arrays times min(1, max_norm / (norm + eps)).
//
// Bound by HBM: every element is read for the norm, and read again and written for the result. Two
// launches however many arrays there are (for each 960 of them): square_kernel leaves one sum of
// squares per CTA; every CTA of scale_kernel adds all of them up, in the same order, and scales its
// part. The arrays are cut into pieces of kPiece elements that the CTAs take in turn. scale_kernel
// takes them backwards, so that the last ones read for the norm come from L2. 235 M FP32 gradients: 149 us
// for the norm (6.3 TB/s, 93% of a copy's rate), 441 to 445 with the result in other arrays, 415 being the
// time of the bytes at a copy's rate. 200 small arrays of two types: 19 us, two launches and little else.
#include <algorithm>
#include <cmath>
#include <vector>

#include "../../include/grad_clip.h"
#include "sgemm_ffma.cuh"
#include "sgemm_internal.h"
#include "sgemm_plan.h"
#include "tc_common.cuh"

namespace sgemm {
namespace gc {

constexpr int kThreads = 512, kPerSm = 4;  // CTAs per SM
constexpr int kPiece = 64 * kThreads;       // elements

struct Array {
  const void *in;
  void *out;
  long long n;
  int first;                 // its first piece in this launch
  uint8_t type, out_type;
};

template <int MOST>
struct Params {
  Array a[MOST];
  int count, pieces;         // arrays and pieces of this launch
  double *sums;              // of each CTA of all launches of square_kernel
  int slot, slots;           // this launch's first one; all of them
  double max_norm, eps;
  float *norm;
};

// The array that piece `at` belongs to.
template <int MOST>
__device__ __forceinline__ const Array &array_of(const Params<MOST> &p, int at) {
  int lo = 0, hi = p.count;  // a[lo].first <= at < a[hi].first
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (p.a[mid].first <= at) lo = mid; else hi = mid;
  }
  return p.a[lo];
}

// What a thread takes at a time: 8 elements of 8 kThreads, as 16-byte accesses side by side: 8 neighbours, or
// (FP32) 4 and the 4 that are 4 kThreads further.
__device__ __forceinline__ int place(int type, int j) {
  return type == GC_F32 ? threadIdx.x * 4 + (j >= 4 ? kThreads * 4 - 4 : 0) + j : threadIdx.x * 8 + j;
}

// Elements place(0 .. 7) from i on; those that do not exist are zero.
__device__ __forceinline__ void load8(const Array &a, long long i, bool vec, float (&v)[8]) {
  if (vec && i + kThreads * 8 <= a.n) {
    if (a.type == GC_F32) {
      const float4 *s = reinterpret_cast<const float4 *>(static_cast<const float *>(a.in) + i) + threadIdx.x;
      const float4 x = s[0], y = s[kThreads];
      v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w, v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
    } else {
      const uint4 u = *(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.in) + i) + threadIdx.x);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (a.type == GC_BF16) {
          v[2 * j] = __uint_as_float(w[j] << 16);
          v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        } else {
          const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[j]));
          v[2 * j] = f.x;
          v[2 * j + 1] = f.y;
        }
      }
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const long long at = i + place(a.type, j);
    v[j] = at < a.n ? tcx::load_out(a.in, a.type, at) : 0.0f;
  }
}

__device__ __forceinline__ void store8(const Array &a, long long i, bool vec, const float (&v)[8]) {
  if (vec && i + kThreads * 8 <= a.n) {
#pragma unroll
    for (int j = 0; j < 8; j += 4) {
      const long long at = i + place(a.type, j);
      if (a.out_type == GC_F32)
        __stcs(reinterpret_cast<float4 *>(static_cast<float *>(a.out) + at), make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]));
      else if (a.type == GC_F32 || j == 0) {
        const uint32_t lo = tcx::pack_out(a.out_type, v[j], v[j + 1]), hi = tcx::pack_out(a.out_type, v[j + 2], v[j + 3]);
        uint16_t *to = static_cast<uint16_t *>(a.out) + at;
        if (a.type == GC_F32)
          __stcs(reinterpret_cast<uint2 *>(to), make_uint2(lo, hi));
        else
          __stcs(reinterpret_cast<uint4 *>(to), make_uint4(lo, hi, tcx::pack_out(a.out_type, v[4], v[5]),
                                                           tcx::pack_out(a.out_type, v[6], v[7])));
      }
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const long long at = i + place(a.type, j);
    if (at < a.n) tcx::store_out(a.out, a.out_type, at, v[j]);
  }
}

__device__ __forceinline__ bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Sum of squares of a thread's elements of a piece, in a scale in which FP32 holds it.
__device__ __forceinline__ double thread_squares(const Array &a, long long at, bool vec) {
  float s = 0.0f;
  uint32_t any = 0;
  const int count = (int)min((long long)kPiece, a.n - at);
#pragma unroll 4
  for (int k = 0; k < count; k += kThreads * 8) {
    float v[8];
    load8(a, at + k, vec, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      s = fmaf(v[j], v[j], s);
      any |= __float_as_uint(v[j]);
    }
  }
  any &= 0x7fffffffu;
  // 64 squares: a sum above 2^-90 has lost nothing that counts to numbers under 2^-126, and one under
  // 2^120 is exact enough as it is. Else the elements once more, times 2^100 or 2^-70.
  if (any == 0 || (s > 0x1p-90f && s < 0x1p120f)) return s;
  const float up = s < 1.0f ? 0x1p100f : 0x1p-70f;
  s = 0.0f;
  for (int k = 0; k < count; k += kThreads * 8) {
    float v[8];
    load8(a, at + k, vec, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) s = fmaf(v[j] * up, v[j] * up, s);
  }
  return (double)s * (up > 1.0f ? 0x1p-200 : 0x1p140);
}

// Sum of `count` numbers by a warp, in each of its lanes. (64-bit additions run at two per cycle and SM: one
// warp of a CTA makes them.)
__device__ __forceinline__ double warp_sum(const double *v, int count) {
  double s = 0.0;
  for (int i = threadIdx.x & 31; i < count; i += 32) s += v[i];
#pragma unroll
  for (int d = 1; d < 32; d *= 2) s += __shfl_xor_sync(0xffffffffu, s, d);
  return s;
}

template <int MOST>
__global__ void __launch_bounds__(kThreads, kPerSm) square_kernel(const __grid_constant__ Params<MOST> p) {
  griddep_wait();  // (launched with programmatic dependent launch: see launch_1d)
  double sum = 0.0;
  for (int at = blockIdx.x; at < p.pieces; at += gridDim.x) {
    const Array &a = array_of(p, at);
    sum += thread_squares(a, (long long)(at - a.first) * kPiece, aligned16(a.in));
  }
  __shared__ double part[kThreads];
  part[threadIdx.x] = sum;
  __syncthreads();
  if (threadIdx.x < 32) {
    sum = warp_sum(part, kThreads);
    if (threadIdx.x == 0) p.sums[p.slot + blockIdx.x] = sum;
  }
  griddep_launch_dependents();
}

// WRITE: also the scaled arrays; else the norm only (one CTA).
template <int MOST, bool WRITE>
__global__ void __launch_bounds__(kThreads, kPerSm) scale_kernel(const __grid_constant__ Params<MOST> p) {
  griddep_wait();
  __shared__ double total;
  if (threadIdx.x < 32) {
    const double sum = warp_sum(p.sums, p.slots);
    if (threadIdx.x == 0) total = sqrt(sum);
  }
  __syncthreads();
  const double norm = total;
  if (blockIdx.x == 0 && threadIdx.x == 0 && p.norm) *p.norm = (float)norm;
  if constexpr (WRITE) {
    const double ratio = p.max_norm / (norm + p.eps);
    // (NaN stays; 0 / 0 is no reason for one)
    const bool whole = ratio >= 1.0 || norm == 0.0;
    // a factor near the end of FP32's range or below it in two parts, of which neither loses bits: x less is exact
    // wherever x ratio is not below FP32's smallest number
    const bool low = ratio < 0x1p-100, lowest = ratio < 0x1p-190;
    const float factor = whole ? 1.0f : (float)(ratio * (lowest ? 0x1p149 : low ? 0x1p64 : 1.0));
    const float less = whole || !low ? 1.0f : lowest ? 0x1p-149f : 0x1p-64f;
    for (int at = p.pieces - 1 - blockIdx.x; at >= 0; at -= gridDim.x) {
      const Array &a = array_of(p, at);
      if (whole && a.in == a.out) continue;
      const bool vec = aligned16(a.in), vec_out = aligned16(a.out);
      const long long from = (long long)(at - a.first) * kPiece;
      const int count = (int)min((long long)kPiece, a.n - from);
#pragma unroll 4
      for (int k = 0; k < count; k += kThreads * 8) {
        float v[8];
        load8(a, from + k, vec, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = v[j] * less * factor;
        store8(a, from + k, vec_out, v);
      }
    }
  }
  griddep_launch_dependents();
}

static int size_of(int type) { return type == GC_F32 ? 4 : 2; }

// Whether a result overlaps a gradient that is not the same array, or another result.
static bool overlapping(int count, const void *const *grads, const int *types, const long long *sizes,
                        void *const *out, const int *out_types) {
  struct Span {
    uintptr_t from, to;
    bool written;
    int of;
  };
  std::vector<Span> spans;
  spans.reserve(2 * (size_t)count);
  for (int i = 0; i < count; ++i) {
    if (sizes[i] == 0) continue;
    const uintptr_t g = reinterpret_cast<uintptr_t>(grads[i]), o = reinterpret_cast<uintptr_t>(out[i]);
    spans.push_back({o, o + (uintptr_t)sizes[i] * size_of(out_types[i]), true, i});
    if (g != o || types[i] != out_types[i])
      spans.push_back({g, g + (uintptr_t)sizes[i] * size_of(types[i]), false, i});
  }
  std::sort(spans.begin(), spans.end(), [](const Span &a, const Span &b) { return a.from < b.from; });
  uintptr_t read_to = 0, written_to = 0;  // ends of what began so far
  for (const Span &s : spans) {
    if (s.from < written_to || (s.written && s.from < read_to)) return true;
    uintptr_t &end = s.written ? written_to : read_to;
    end = std::max(end, s.to);
  }
  return false;
}

struct Call {
  int count;
  const void *const *grads;
  const int *types;
  const long long *sizes;
  double max_norm, eps;
  void *const *out;
  const int *out_types;
  float *norm;
  cudaStream_t stream;
};

// Fills `p` with arrays from `i` on that are not empty; returns the next one.
template <int MOST>
static int fill(Params<MOST> &p, const Call &c, int i) {
  p.count = p.pieces = 0;
  for (; i < c.count && p.count < MOST; ++i) {
    if (c.sizes[i] == 0) continue;
    const long long pieces = ceil_div(c.sizes[i], kPiece);
    if (p.pieces + pieces > 0x3fffffff) break;
    p.a[p.count++] = {c.grads[i], c.out ? c.out[i] : nullptr, c.sizes[i], p.pieces, (uint8_t)c.types[i],
                      (uint8_t)(c.out ? c.out_types[i] : 0)};
    p.pieces += (int)pieces;
  }
  return i;
}

template <int MOST>
static cudaError_t run(const Call &c, int launches, int sms) {
  const int most = kPerSm * sms;  // CTAs of a launch
  double *ws = nullptr;
  cudaError_t e = cudaMallocFromPoolAsync(reinterpret_cast<void **>(&ws),
                                          sizeof(double) * (size_t)most * launches, workspace_pool(), c.stream);
  if (e != cudaSuccess) return e;
  static thread_local Params<MOST> p;
  p.sums = ws;
  p.max_norm = c.max_norm;
  p.eps = c.eps;
  p.norm = c.norm;
  p.slots = 0;
  int i = 0;
  do {
    i = fill(p, c, i);
    const int grid = std::min(p.pieces, most);
    p.slot = p.slots;
    p.slots += grid;
    if (grid > 0) e = launch_1d(square_kernel<MOST>, grid, kThreads, 0, 1, c.stream, p);
  } while (e == cudaSuccess && i < c.count);
  if (c.out == nullptr) {
    if (e == cudaSuccess) e = launch_1d(scale_kernel<MOST, false>, 1, kThreads, 0, 1, c.stream, p);
  } else {
    i = 0;
    do {
      i = fill(p, c, i);
      if (e == cudaSuccess)
        e = launch_1d(scale_kernel<MOST, true>, std::max(1, std::min(p.pieces, most)), kThreads, 0, 1,
                      c.stream, p);
    } while (e == cudaSuccess && i < c.count);
  }
  const cudaError_t ef = cudaFreeAsync(ws, c.stream);
  return e == cudaSuccess ? ef : e;
}

}  // namespace gc
}  // namespace sgemm

using namespace sgemm;

extern "C" int clip_grad_norm(int count, const void *const *grads, const int *types,
                              const long long *sizes, double max_norm, double eps, void *const *out,
                              const int *out_types, float *norm, cudaStream_t stream) {
  const auto known = [](int t) { return t == GC_F32 || t == GC_BF16 || t == GC_F16; };
  const auto misplaced = [](const void *q, int t) {
    return reinterpret_cast<uintptr_t>(q) % gc::size_of(t) != 0;
  };
  if (count < 0) return -1;
  if (count > 0 && grads == nullptr) return -2;
  if (count > 0 && types == nullptr) return -3;
  if (count > 0 && sizes == nullptr) return -4;
  long long arrays = 0, pieces = 0;
  for (int i = 0; i < count; ++i) {
    if (!known(types[i])) return -3;
    if (sizes[i] < 0 || sizes[i] > (1LL << 42)) return -4;
    if (sizes[i] > 0 && (grads[i] == nullptr || misplaced(grads[i], types[i]))) return -2;
    arrays += sizes[i] > 0;
    pieces += ceil_div(sizes[i], gc::kPiece);
  }
  if (!(max_norm >= 0.0)) return -5;
  if (!(eps >= 0.0) || std::isinf(eps)) return -6;
  if (out != nullptr && count > 0) {
    if (out_types == nullptr) return -8;
    for (int i = 0; i < count; ++i) {
      if (!known(out_types[i])) return -8;
      if (sizes[i] > 0 && (out[i] == nullptr || misplaced(out[i], out_types[i]))) return -7;
    }
    if (gc::overlapping(count, grads, types, sizes, out, out_types)) return -7;
  }
  if (misplaced(norm, GC_F32)) return -9;
  if (arrays == 0 && norm == nullptr) return 0;
  int sms = 0;
  const cudaError_t e = device_setup(&sms);
  if (e != cudaSuccess) return (int)e;
  const gc::Call c{count, grads, types, sizes, max_norm, eps, out, out_types, norm, stream};
  // launches: full tables, and each time that the pieces of one would be too many
  const auto launches = [&](int most) { return (int)(ceil_div(arrays, most) + pieces / 0x3fffffff * 2 + 1); };
  // (the table is copied for each launch: 6.5 us for a call of 20 arrays, 11 of 200, 30 of 900)
  return arrays <= 32    ? (int)gc::run<32>(c, launches(32), sms)
         : arrays <= 240 ? (int)gc::run<240>(c, launches(240), sms)
                         : (int)gc::run<960>(c, launches(960), sms);
}

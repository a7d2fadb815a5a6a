// What the tensor-core operators (8-bit product, orthogonalisation) share: PTX wrappers of
// the 5th-generation tensor cores (tcgen05, TMEM) and of thread-block clusters, and shared
// memory descriptors of the operand layouts that TMA writes.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "sgemm_ffma.cuh"
#include "sgemm_ptx.cuh"

namespace sgemm {
namespace tcx {

// Wait for the phase of parity `parity`, by default with the limit of mbar_wait (sgemm_ptx.cuh). A try suspends
// the thread for as long as the hardware chooses, so that waiting warps leave the issue slots and the
// shared memory port to the others (a limit of one's own costs the 8-bit product's epilogue seven
// instructions of 150 per block and 2% of its time); the global timer is read between tries only.
// Lanes may answer differently when the limit runs out while the phase completes, so a warp that goes
// on to something that needs all of its lanes (elect.sync, tcgen05.ld) takes a vote on the answer: some
// lanes that left the loop alone would keep the others waiting for ever.
__device__ __forceinline__ bool try_wait_suspended(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n"
      ".reg .pred p;\n"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      "selp.u32 %0, 1, 0, p;\n"
      "}\n"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}

__device__ __forceinline__ bool wait_short(uint32_t bar, uint32_t parity,
                                           unsigned long long limit = kWaitLimitNs) {
  if (try_wait_suspended(bar, parity)) return true;
  const unsigned long long t0 = global_ns();
  for (uint32_t i = 0; i < (1u << 30); ++i) {  // (should the timer not advance)
    if (try_wait_suspended(bar, parity)) return true;
    if (global_ns() - t0 > limit) return false;
  }
  return false;
}

// Position in a ring of N slots: the slot and the parity of its use (0 for the first, 1 for the
// second, ...). A consumer waits for the slot's "full" phase of this parity, a producer for the
// "empty" phase of the opposite one (which a fresh mbarrier counts as complete).
template <uint32_t N>
struct Ring {
  uint32_t slot = 0, parity = 0;
  __device__ __forceinline__ void next() {
    if constexpr ((N & (N - 1)) == 0) {
      parity ^= (slot + 1) / N;
      slot = (slot + 1) % N;
    } else if (++slot == N) {
      slot = 0;
      parity ^= 1u;
    }
  }
};

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile(
      "{\n"
      ".reg .pred p;\n"
      "elect.sync _|p, 0xffffffff;\n"
      "selp.u32 %0, 1, 0, p;\n"
      "}\n"
      : "=r"(e));
  return e != 0;
}

__device__ __forceinline__ void fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory");
}

__device__ __forceinline__ void tmem_alloc(uint32_t slot, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(slot),
               "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void tmem_relinquish() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(taddr), "r"(ncols)
               : "memory");
}

// Arrive on `bar` once every tcgen05.mma this thread issued so far has completed.
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(bar)
      : "memory");
}

// D[tmem] (+)= P[smem] * Q[smem]^T on 8-bit floating-point operands, K = 32.
__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t pdesc, uint64_t qdesc,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n"
      ".reg .pred p;\n"
      "setp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n"
      "}\n" ::"r"(d_tmem),
      "l"(pdesc), "l"(qdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// D[tmem] (+)= P[smem] * Q[smem]^T on fp16 operands, K = 16.
__device__ __forceinline__ void mma_f16(uint32_t d_tmem, uint64_t pdesc, uint64_t qdesc,
                                        uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n"
      ".reg .pred p;\n"
      "setp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n"
      "}\n" ::"r"(d_tmem),
      "l"(pdesc), "l"(qdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// ---- CTA pairs (cta_group::2): the two CTAs of a cluster work on one accumulator tile of 256
// rows. Each holds its 128 rows of P and half of Q in its own shared memory (at the same offsets)
// and its 128 rows of the accumulator in its own TMEM; CTA 0, the leader, issues the instructions
// for both. Allocation is made by one warp of each CTA.
__device__ __forceinline__ void tmem_alloc_pair(uint32_t slot, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(slot),
               "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void tmem_relinquish_pair() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;\n" ::"r"(taddr), "r"(ncols)
               : "memory");
}

// Arrive on `bar` of both CTAs once every pair instruction this thread issued so far has completed.
__device__ __forceinline__ void mma_commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;\n" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}

__device__ __forceinline__ void mma_f8_pair(uint32_t d_tmem, uint64_t pdesc, uint64_t qdesc,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n"
      ".reg .pred p;\n"
      "setp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n"
      "}\n" ::"r"(d_tmem),
      "l"(pdesc), "l"(qdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void mma_f16_pair(uint32_t d_tmem, uint64_t pdesc, uint64_t qdesc,
                                             uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n"
      ".reg .pred p;\n"
      "setp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n"
      "}\n" ::"r"(d_tmem),
      "l"(pdesc), "l"(qdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// The same with P in TMEM: lane i of its columns holds row i, two fp16 numbers of k per column.
__device__ __forceinline__ void mma_f16_tmem(uint32_t d_tmem, uint32_t p_tmem, uint64_t qdesc,
                                             uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n"
      ".reg .pred p;\n"
      "setp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n"
      "}\n" ::"r"(d_tmem),
      "r"(p_tmem), "l"(qdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_f16_tmem_pair(uint32_t d_tmem, uint32_t p_tmem, uint64_t qdesc,
                                                  uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n"
      ".reg .pred p;\n"
      "setp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n"
      "}\n" ::"r"(d_tmem),
      "r"(p_tmem), "l"(qdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 32 columns of this thread's TMEM lane; complete after tmem_wait_st().
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};\n" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]),
      "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]),
      "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]),
      "r"(v[29]), "r"(v[30]), "r"(v[31])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
}

// Address of the same shared memory location in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t in_cta(uint32_t local, uint32_t rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(a) : "r"(local), "r"(rank));
  return a;
}

// Arrive on another CTA's barrier. (No release at cluster scope, which costs about 2000 cycles: what
// it reports, reads of TMEM, is ordered by the tcgen05 fences.)
__device__ __forceinline__ void arrive_in(uint32_t cluster_bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];\n" ::"r"(cluster_bar)
               : "memory");
}

// 2-D tile copy into this CTA's shared memory, completing `cluster_bar` of either CTA of the pair.
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst, const CUtensorMap *map, int x, int y,
                                                 uint32_t cluster_bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile"
      ".mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(cluster_bar)
      : "memory");
}

// A tile of a copy to come, to L2.
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap *map, int x, int y) {
  asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];\n" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(x), "r"(y)
               : "memory");
}

// 32 (16) consecutive FP32 accumulator columns of this thread's TMEM lane, readable after
// tmem_wait_ld().
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, "
      "[%32];\n"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]),
        "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]),
        "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
        "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]),
        "=r"(v[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]),
        "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(taddr)
      : "memory");
}
// Wait for this thread's loads from TMEM; no use of v moves before it.
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]),
                 "+r"(v[6]), "+r"(v[7]), "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]),
                 "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]), "+r"(v[16]), "+r"(v[17]),
                 "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]),
                 "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]),
                 "+r"(v[30]), "+r"(v[31])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]),
                 "+r"(v[6]), "+r"(v[7]), "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]),
                 "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15])
               :
               : "memory");
}

// Shared-memory matrix descriptor of an operand that TMA wrote with the 128-byte swizzle
// from 128-byte-wide boxes (descriptor version 1 in bits 46-47, swizzle mode 2 in 61-63).
//  * K-major (a row of the box is 128 bytes of k for one row of the operand): 8-row groups
//    are 1024 bytes apart (stride offset); the leading offset is not used. The next K step
//    of 32 bytes adds 32 to the start address.
//  * MN-major (a row of the box is 128 bytes along the operand's rows, for one k): 8-k groups
//    are 1024 bytes apart (stride offset), and the next 128 bytes of rows are `lead` bytes
//    further (leading offset). The next K step of n adds 128 n bytes to the start address.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t smem_addr, uint32_t lead) {
  uint64_t d = (uint64_t)((smem_addr & 0x3FFFFu) >> 4);
  d |= (uint64_t)((lead >> 4) & 0x3FFFu) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

// Four signed bytes as FP16 numbers, exactly: with the sign bits flipped a byte b is 1024 + 128 + b as
// the low bits of 0x6400.
__device__ __forceinline__ void halves(uint32_t w, uint32_t &lo, uint32_t &hi) {
  const uint32_t u = w ^ 0x80808080u;
  const __half2 bias = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
  const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
  const __half2 x = __hsub2(*reinterpret_cast<const __half2 *>(&a), bias);
  const __half2 y = __hsub2(*reinterpret_cast<const __half2 *>(&b), bias);
  lo = *reinterpret_cast<const uint32_t *>(&x);
  hi = *reinterpret_cast<const uint32_t *>(&y);
}

// Registers per thread of a warpgroup, down or up (its four warps all execute it).
template <int N>
__device__ __forceinline__ void reg_dealloc() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_alloc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N));
}

// Barrier among `threads` threads of the CTA (id 1 .. 15; 0 is __syncthreads), whole warps: a warp
// of which some lanes are still elsewhere would be counted twice.
__device__ __forceinline__ void named_barrier(int id, int threads) {
  __syncwarp();
  asm volatile("bar.sync %0, %1;\n" ::"r"(id), "r"(threads) : "memory");
}

// This thread's arrival at `bar` once its cp.async copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];\n" ::"r"(bar) : "memory");
}

// MN-major operand in boxes of `row` bytes along its rows (128, 64 or 32, which is also the span of
// the swizzle TMA wrote it with; modes 2, 4, 6): 8-k groups are 8 rows apart.
__device__ __forceinline__ uint64_t mn_desc(uint32_t smem_addr, uint32_t row, uint32_t lead) {
  uint64_t d = (uint64_t)((smem_addr & 0x3FFFFu) >> 4);
  d |= (uint64_t)((lead >> 4) & 0x3FFFu) << 16;
  d |= (uint64_t)(8 * row >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)(row == 128 ? 2 : row == 64 ? 4 : 6) << 61;
  return d;
}

// One FP32 number of CTA `rank`'s shared memory at the offset of the local address `local`.
__device__ __forceinline__ float ld_cluster1(uint32_t local, uint32_t rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];\n" : "=f"(v) : "r"(in_cta(local, rank)) : "memory");
  return v;
}

// ---- Results on their way out. A warp's buffer of 2 KB holds 64 bytes of each of 32 rows as four
// 16-byte pieces; piece j of row r lies at j ^ (r / 2 % 4), so that 8 neighbouring rows' pieces,
// and the four pieces of 2 neighbouring rows, lie in different banks. Lanes put the rows that they
// hold and take what neighbouring lanes then store side by side (or the other way round).
constexpr int TURN_BYTES = 32 * 64;

__device__ __forceinline__ uint4 *turn_at(uint8_t *buf, int row, int piece) {
  return reinterpret_cast<uint4 *>(buf + row * 64 + ((piece ^ (row >> 1 & 3)) << 4));
}

enum { OUT_F32 = 0, OUT_BF16 = 1, OUT_F16 = 2 };

// A row-major result out = alpha * v + beta * out; rows and cols: what exists of it.
struct Out {
  void *ptr;
  int type;
  long long ld;
  int rows, cols;
  float alpha, beta;
  int vec;  // 16-byte accesses to rows are aligned
};

__device__ __forceinline__ float load_out(const void *ptr, int type, long long at) {
  if (type == OUT_F32) return reinterpret_cast<const float *>(ptr)[at];
  if (type == OUT_BF16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(ptr)[at]);
  return __half2float(reinterpret_cast<const __half *>(ptr)[at]);
}

__device__ __forceinline__ void store_out(void *ptr, int type, long long at, float v) {
  if (type == OUT_F32)
    reinterpret_cast<float *>(ptr)[at] = v;
  else if (type == OUT_BF16)
    reinterpret_cast<__nv_bfloat16 *>(ptr)[at] = __float2bfloat16_rn(v);
  else
    reinterpret_cast<__half *>(ptr)[at] = __float2half_rn(v);
}

// out[at] = y + beta * out[at]
__device__ __forceinline__ void finish_out(void *ptr, int type, long long at, float y, float beta) {
  store_out(ptr, type, at, beta != 0.0f ? fmaf(beta, load_out(ptr, type, at), y) : y);
}

__device__ __forceinline__ uint32_t pack_out(int type, float a, float b) {
  if (type == OUT_BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
  }
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// CN (16 or 32) neighbouring columns from `col` of 32 rows, one per lane, the first is row0.
template <int CN>
__device__ __forceinline__ void store_rows(const Out &o, uint8_t *buf, int lane, int row0, int col,
                                           const float (&v)[CN]) {
  const int rows = min(32, o.rows - row0), cols = min(CN, o.cols - col);
  if (o.vec && o.beta == 0.0f && o.type != OUT_F32) {
    // packed: 2 CN bytes of a row
#pragma unroll
    for (int j = 0; j < CN; j += 8)
      *turn_at(buf, lane, j / 8) =
          make_uint4(pack_out(o.type, o.alpha * v[j], o.alpha * v[j + 1]),
                     pack_out(o.type, o.alpha * v[j + 2], o.alpha * v[j + 3]),
                     pack_out(o.type, o.alpha * v[j + 4], o.alpha * v[j + 5]),
                     pack_out(o.type, o.alpha * v[j + 6], o.alpha * v[j + 7]));
    __syncwarp();
    constexpr int LANES = CN / 8;  // per row
    const int c = 8 * (lane % LANES);
#pragma unroll
    for (int r = lane / LANES; r < 32; r += 32 / LANES) {
      const uint4 w = *turn_at(buf, r, lane % LANES);
      if (r >= rows) continue;
      uint16_t *d = reinterpret_cast<uint16_t *>(o.ptr) + (row0 + r) * o.ld + col + c;
      if (c + 8 <= cols) {
        *reinterpret_cast<uint4 *>(d) = w;
      } else {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (c + j < cols) d[j] = (uint16_t)(u[j / 2] >> (16 * (j & 1)));
      }
    }
    __syncwarp();
    return;
  }
#pragma unroll
  for (int h = 0; h < CN; h += 16) {  // 16 columns at a time in FP32
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *reinterpret_cast<float4 *>(turn_at(buf, lane, j)) =
          make_float4(o.alpha * v[h + 4 * j], o.alpha * v[h + 4 * j + 1],
                      o.alpha * v[h + 4 * j + 2], o.alpha * v[h + 4 * j + 3]);
    __syncwarp();
    if (o.vec && o.type == OUT_F32) {
      const int c = 4 * (lane & 3);
#pragma unroll
      for (int r = lane >> 2; r < 32; r += 8) {
        float4 w = *reinterpret_cast<const float4 *>(turn_at(buf, r, lane & 3));
        if (r >= rows || h + c >= cols) continue;
        float *d = reinterpret_cast<float *>(o.ptr) + (row0 + r) * o.ld + col + h + c;
        if (h + c + 4 <= cols) {
          if (o.beta != 0.0f) {
            const float4 q = *reinterpret_cast<const float4 *>(d);
            w = make_float4(fmaf(o.beta, q.x, w.x), fmaf(o.beta, q.y, w.y), fmaf(o.beta, q.z, w.z),
                            fmaf(o.beta, q.w, w.w));
          }
          *reinterpret_cast<float4 *>(d) = w;
        } else {
          const float y[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (h + c + j < cols) d[j] = o.beta != 0.0f ? fmaf(o.beta, d[j], y[j]) : y[j];
        }
      }
    } else {
      const int c = lane & 15;
#pragma unroll 4
      for (int r = lane >> 4; r < 32; r += 2) {
        const float y = reinterpret_cast<const float *>(turn_at(buf, r, c >> 2))[c & 3];
        if (r < rows && h + c < cols)
          finish_out(o.ptr, o.type, (row0 + r) * o.ld + col + h + c, y, o.beta);
      }
    }
    __syncwarp();
  }
}

}  // namespace tcx

// Tensor map of a rows x cols row-major matrix of 1- or 2-byte elements (row stride ld
// elements, a multiple of 16 bytes; ptr 16-byte aligned) in boxes of span bytes x box_rows, swizzled
// over that span (128, 64 or 32); elements out of range read as zero. False if the driver rejects it.
bool encode_map_2d_narrow(CUtensorMap *map, const void *ptr, int elem_bytes, long long rows,
                          long long cols, long long ld, int box_rows, int span = 128);

}  // namespace sgemm

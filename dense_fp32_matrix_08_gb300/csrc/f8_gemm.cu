// D = alpha * op(A) * op(B) + beta * D on 8-bit floating-point operands with one FP32 scale
// for each block of 128 along k, on the 5th-generation tensor cores of sm_103a:
//
//   D[i][j] = alpha * sum_kb sA[i][kb] * sB[kb][j] * (sum_{k in block kb} qA[i][k] * qB[k][j])
//             + beta * D[i][j]
//
// The inner sums (128 products of two 8-bit numbers) run in the tensor core with FP32
// accumulation; the outer sum over the blocks runs in FP32 registers, because its terms carry
// different scales. One accumulator tile in TMEM therefore holds one block of k only: while
// the tensor core fills one TMEM buffer, the epilogue warps read the previous one, scale it
// and add it to their registers.
//
// The kernel sees the product as P (128 rows per tile) times Q (TN columns per tile). P = op(A)
// and Q = op(B) for products with many rows. With few rows (serving: a few tokens) the roles are
// exchanged, P = op(B)^T and Q = op(A)^T, so that the 128-row side of the instruction holds rows
// of the weight and none of it is wasted on absent tokens.
//
// Both operands may be stored with k contiguous or with the other index contiguous: TMA writes
// either into the 128-byte-swizzled layout that the instruction's descriptors read (K-major or
// MN-major), so no transposed copy is ever made.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <mutex>

#include "../../include/f8_gemm.h"
#include "sgemm_internal.h"
#include "sgemm_plan.h"
#include "tc_common.cuh"

namespace sgemm {
namespace f8 {

constexpr int BP = 128;                  // rows of P per tile
constexpr int BK = 128;                  // k per block = per pipeline stage
constexpr int P_BYTES = BP * BK;
constexpr int MAX_CLUSTER = 8;
constexpr int PART_PITCH = BP;           // column pitch of a cluster's partial tiles (floats)

// PAIR: two CTAs share a tile of 256 rows and TN columns (tcgen05 cta_group::2), each with its 128
// rows of P and half of Q.
template <int TN_, bool PAIR_ = false>
struct Cfg {
  static constexpr int TN = TN_;
  static constexpr bool PAIR = PAIR_;
  static constexpr int QN = PAIR ? TN / 2 : TN;     // columns of Q that this CTA holds
  static constexpr int GROUPS = PAIR ? 4 : TN >= 128 ? 2 : 1;  // epilogue groups of four warps
  static constexpr int COLS = TN / GROUPS;          // accumulator columns of a group
  static constexpr int EPI_WARPS = 4 * GROUPS;
  static constexpr int THREADS = 32 * (4 + EPI_WARPS);
  static constexpr int Q_BYTES = QN * BK;
  static constexpr int STAGE_BYTES = P_BYTES + Q_BYTES;
  // (Half as many stages for the narrow tiles, so that the next call's CTA fits beside this one's,
  // measured 12 to 15% slower at 1x14336x4096 and 256x4096x4096 and gained nothing on short sums.)
  static constexpr int STAGES = PAIR ? 5 : TN >= 64 ? 6 : TN == 32 ? 8 : 10;
  // A pair's tile is computed in two parts of 128 columns with accumulators of their own, each read
  // by two of the epilogue groups: the tensor core fills one while the other is read and handed
  // back. (One group of four warps per part, 128 sums per thread, was 13% slower at
  // 8192x14336x4096: 485 against 429 us.)
  static constexpr int PARTS = PAIR ? 2 : 1;
  static constexpr int PART = TN / PARTS;           // columns of one accumulator
  static constexpr int NBUF = PAIR ? 2 : 4;         // accumulators per part
  static constexpr int ACC_COLS = PART < 32 ? 32 : PART;
  static constexpr int TMEM_COLS = PARTS * NBUF * ACC_COLS;
  static constexpr int ACC_WARPS = EPI_WARPS / PARTS * (PAIR ? 2 : 1);  // readers of one
  // scales of a k block: 128 of P (one if its rows share it), then TN of Q (one for each 128)
  static constexpr int SC_DEPTH = TN == 16 ? 6 : 4;
  static constexpr int SC_BYTES = SC_DEPTH * (BP + TN) * 4;
  static constexpr int TURN_BYTES = EPI_WARPS * tcx::TURN_BYTES;
  static constexpr int BAR_BYTES = 8 * (2 * STAGES + 2 * PARTS * NBUF + 2 * SC_DEPTH) + 16;
  static constexpr int SMEM_BYTES =
      1024 + STAGES * STAGE_BYTES + SC_BYTES + TURN_BYTES + BAR_BYTES;
  static_assert((int)F8_D_F32 == tcx::OUT_F32 && (int)F8_D_BF16 == tcx::OUT_BF16 &&
                (int)F8_D_F16 == tcx::OUT_F16, "types of D");
  // Two warps take turns with the k blocks of a single CTA. Each must see every use of a slot it
  // waits on (a barrier tells only odd uses from even ones), so slots alternate as the blocks do.
  static_assert(PAIR || (STAGES % 2 == 0 && NBUF % 2 == 0), "each slot belongs to one issuer");
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory per CTA");
  static_assert(TMEM_COLS <= 512, "TMEM columns");
  static_assert(PAIR || TN <= 128, "an MN-major Q is one box");
  static_assert(PART_PITCH * TN * 4 <= STAGES * STAGE_BYTES, "a partial tile fits in the ring");
};

struct Side {          // one operand as the kernel sees it
  int extent;          // rows of P, columns of Q
  int mn_major;        // stored with this extent contiguous
  const float *scale;
  int shift;           // 7: one scale for 128 of the extent, 0: one for each
  long long s_mn, s_k; // scale strides along the extent and along the k blocks
};

struct Params {
  Side p, q;
  int KB;              // k blocks
  int tiles_p, tiles_q, group_p;
  int split;           // CTAs of a cluster, each with its range of k blocks
  uint32_t idesc;
  float alpha, beta;
  void *D;
  int d_type;
  long long d_p, d_q;  // strides of D along P and Q; one of them is 1
  int vec;             // 16-byte stores along the contiguous index are aligned
};

// Device status word: 0 = fine; 1, 2, 3, 4 = a wait of the producer, the MMA issuer, the epilogue
// or the scale loader gave up.
__device__ int g_f8_status;

__device__ __forceinline__ unsigned long long mul2(unsigned long long a, unsigned long long b) {
  unsigned long long d;
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

__device__ __forceinline__ void store1(const Params &p, int row, int col, float v) {
  if (row < p.p.extent && col < p.q.extent)
    tcx::finish_out(p.D, p.d_type, row * p.d_p + col * p.d_q, p.alpha * v, p.beta);
}

// Warp 0: TMA producer, warps 1 and 3: MMA issuers (one elected lane of each), warp 2: scale loader.
// Warps 4 ..: epilogue; a group of four warps owns COLS columns of the tile, warp w of it TMEM lanes
// (tile rows) 32 (w % 4) .. + 31, one row per thread.
// QVEC: Q has a scale for each column (else one for each 128, the same for a whole group).
//
// What bounds it. 8192 x 14336 x 4096, BF16 result: 400 us, 2.4 PFLOP/s, the tensor core 60% busy. For
// each block of k an epilogue warp executes about 145 instructions on its 64 accumulators per lane
// (32 of them the packed multiply-adds), which fills 65% of the issue slots; the rest is the time an
// accumulator takes from the tensor core to the epilogue and back, and TMEM holds only two per part.
// 4096 x 4096 x 8192 with a scale for each column of Q: 203 us, 1.4 PFLOP/s, the tensor core 33% and the
// issue slots 44% busy: 3.4 rounds of tiles take the time of four, and in them twice the multiplies and
// the reads of the scales make that way longer. (The accumulators as 16 x 256-bit fragments, which need a
// quarter of the scales per lane, took 218 us for 210 then.) 4099 x 3001 x 777: 27 us, 19 with rows of 3008:
// unaligned 16-bit rows are stored element by element. (As 4-byte pairs: 33.5 us for 28.6 then, more
// partial sectors per instruction.) 1 x 4096 x 4096 with the weight in memory: 7.0 us, 2.4 TB/s (5.5
// from L2), most of it the start of the CTAs, the first bytes' way and the clusters' exchange.
template <int TN, bool QVEC, bool PAIR>
__global__ void __launch_bounds__(Cfg<TN, PAIR>::THREADS, 1)
    f8_kernel(const __grid_constant__ CUtensorMap map_p, const __grid_constant__ CUtensorMap map_q,
              const Params p) {
  using C = Cfg<TN, PAIR>;
  using namespace tcx;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = saddr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t *sbase = smem_raw + (base - raw);
  float *scales = reinterpret_cast<float *>(sbase + C::STAGES * C::STAGE_BYTES);
  const uint32_t bars = base + C::STAGES * C::STAGE_BYTES + C::SC_BYTES + C::TURN_BYTES;
  const uint32_t acc_full = bars + 8 * (2 * C::STAGES);
  const uint32_t acc_empty = acc_full + 8 * C::PARTS * C::NBUF;
  const uint32_t sc_full = acc_empty + 8 * C::PARTS * C::NBUF, sc_empty = sc_full + 8 * C::SC_DEPTH;
  const uint32_t tmem_slot = sc_empty + 8 * C::SC_DEPTH;
  volatile uint32_t *tmem_slot_ptr =
      reinterpret_cast<volatile uint32_t *>(smem_raw + (tmem_slot - raw));

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  // a cluster is S CTAs with a range of k blocks each, or a pair on one tile of 256 rows
  const int S = PAIR ? 1 : p.split, CS = PAIR ? 2 : S;
  const int cta = CS > 1 ? (int)(blockIdx.x % (unsigned)CS) : 0;  // rank in the cluster
  const int rank = PAIR ? 0 : cta;
  const int first = (int)(blockIdx.x / (unsigned)CS), step = (int)(gridDim.x / (unsigned)CS);
  const int units = PAIR ? (p.tiles_p + 1) / 2 : p.tiles_p;       // rows of tiles
  const int tiles = units * p.tiles_q;
  const int kb0 = (int)((long long)p.KB * rank / S);
  const int kb1 = (int)((long long)p.KB * (rank + 1) / S);

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(bars + 8 * s, 1);
      mbar_init(bars + 8 * (C::STAGES + s), C::PARTS);
    }
    for (int b = 0; b < C::PARTS * C::NBUF; ++b) {
      mbar_init(acc_full + 8 * b, 1);
      mbar_init(acc_empty + 8 * b, C::ACC_WARPS);
    }
    for (int d = 0; d < C::SC_DEPTH; ++d) {
      mbar_init(sc_full + 8 * d, 32);
      mbar_init(sc_empty + 8 * d, C::EPI_WARPS);
    }
    mbar_init_fence();
    tma_prefetch_map(&map_p);
    tma_prefetch_map(&map_q);
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
  fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync_all();  // the other CTA's barriers are initialised
  fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot_ptr, 0);  // (uniform)
  griddep_wait();  // (launched with programmatic dependent launch: see launch_1d)
  // (every CTA of the grid is resident, so the next launch may take what room is left)
  griddep_launch_dependents();

  const auto tile_at = [&](int t, int &tp, int &tq) {
    tile_coords(t, units, p.tiles_q, p.group_p, tp, tq);
    if (PAIR) tp = 2 * tp + cta;
  };

  if (warp < 4) {
  // a pair's 640 threads x 96 registers at launch = 128 x 64 + 512 x 104
  if constexpr (PAIR) reg_dealloc<64>();
  if (warp == 0) {
    // ---- TMA producer: the k blocks of this CTA's tiles, in order, through the ring of stages
    Ring<C::STAGES> st;
    int issued = 0;  // (up to STAGES)
    bool ok = true;
    for (int t = first; t < tiles && ok; t += step) {
      int tp, tq;
      tile_at(t, tp, tq);
      for (int kb = kb0; kb < kb1; ++kb) {
        ok = __all_sync(0xffffffffu, wait_short(bars + 8 * (C::STAGES + st.slot), st.parity ^ 1u));
        if (!ok) {
          if (lane == 0) atomicCAS(&g_f8_status, 0, 1);
          break;
        }
        if (elect_one()) {
          const uint32_t dst = base + st.slot * C::STAGE_BYTES, full = bars + 8 * st.slot;
          const int k = kb * BK, p0 = tp * BP, q0 = tq * TN + cta * (PAIR ? C::QN : 0);
          if constexpr (PAIR) {  // both CTAs' copies complete the leader's barrier
            const uint32_t lead = in_cta(full, 0);
            if (cta == 0) mbar_expect_tx(full, 2 * C::STAGE_BYTES);
            tma_load_2d_pair(dst, &map_p, p.p.mn_major ? p0 : k, p.p.mn_major ? k : p0, lead);
            tma_load_2d_pair(dst + P_BYTES, &map_q, p.q.mn_major ? q0 : k, p.q.mn_major ? k : q0,
                             lead);
          } else {
            mbar_expect_tx(full, C::STAGE_BYTES);
            tma_load_2d(dst, &map_p, p.p.mn_major ? p0 : k, p.p.mn_major ? k : p0, full);
            tma_load_2d(dst + P_BYTES, &map_q, p.q.mn_major ? q0 : k, p.q.mn_major ? k : q0, full);
          }
        }
        __syncwarp();
        issued = min(issued + 1, C::STAGES);
        st.next();
      }
    }
    // the last loads issued must have landed before this warp leaves (a pair's: the leader waits for
    // both, and the CTAs leave together)
    for (; issued > 0 && (!PAIR || cta == 0); --issued) {
      st.parity ^= st.slot == 0 ? 1u : 0u;
      st.slot = st.slot == 0 ? C::STAGES - 1 : st.slot - 1;
      wait_short(bars + 8 * st.slot, st.parity);
    }
  } else if (warp == 1 || warp == 3) {
    // ---- MMA issuers. What a warp does for one accumulator (two waits, four instructions, the
    // commits) takes longer than the tensor core takes for 128 columns, so two warps share it:
    // each issues one part of every k block of a pair, else every other k block.
    const int me = warp >> 1;
    const uint32_t lead_q = 128 * BK;
    const uint32_t adv_p = (p.p.mn_major ? 32 * 128 : 32) >> 4;
    constexpr uint32_t row_q = TN < 128 ? TN : 128;  // bytes of a k of an MN-major Q
    const uint32_t adv_q = (p.q.mn_major ? 32 * row_q : 32) >> 4;
    const uint64_t pd0 = sw128_desc(base, 16);
    // a part's 64 rows of this CTA's Q: 8 KB further, or 64 bytes into the rows of k
    const uint32_t q_at = base + P_BYTES + (PAIR ? me * (p.q.mn_major ? 64 : 64 * 128) : 0);
    const uint64_t qd0 = p.q.mn_major ? mn_desc(q_at, row_q, lead_q) : sw128_desc(q_at, 16);
    const uint32_t acc0 = PAIR ? me * C::NBUF : 0;
    Ring<C::STAGES> st;
    Ring<C::NBUF> buf;
    bool ok = true;
    int mine = me;  // (not a pair) k blocks until the next one of this warp
    for (int t = first; t < tiles && ok && (!PAIR || cta == 0); t += step) {
      for (int kb = kb0; kb < kb1; ++kb) {
        if (PAIR || mine == 0) {
          const uint32_t a = acc0 + buf.slot;
          ok = __all_sync(0xffffffffu, wait_short(bars + 8 * st.slot, st.parity) &&
                                           wait_short(acc_empty + 8 * a, buf.parity ^ 1u));
          if (!ok) {
            if (lane == 0) atomicCAS(&g_f8_status, 0, 2);
            break;
          }
          fence_after();
          if (elect_one()) {
            const uint32_t at = st.slot * (uint32_t)(C::STAGE_BYTES >> 4);
            const uint32_t d = tmem + a * C::ACC_COLS;
#pragma unroll
            for (uint32_t kk = 0; kk < BK / 32; ++kk) {
              if constexpr (PAIR)
                mma_f8_pair(d, pd0 + at + kk * adv_p, qd0 + at + kk * adv_q, p.idesc, kk != 0);
              else
                mma_f8(d, pd0 + at + kk * adv_p, qd0 + at + kk * adv_q, p.idesc, kk != 0);
            }
            // once these have completed the stage is free of this warp, and the accumulator complete
            // (in this order: who has seen the last accumulator knows that no arrival is to come)
            if constexpr (PAIR) {
              mma_commit_pair(bars + 8 * (C::STAGES + st.slot));
              mma_commit_pair(acc_full + 8 * a);
            } else {
              mma_commit(bars + 8 * (C::STAGES + st.slot));
              mma_commit(acc_full + 8 * a);
            }
          }
          __syncwarp();
        }
        mine ^= 1;
        st.next();
        buf.next();
      }
    }
  } else if (warp == 2) {
    // ---- scale loader: the scales of each k block, several blocks ahead of the epilogue, which
    // would otherwise wait for memory once per block; 0 out of range
    Ring<C::SC_DEPTH> sl;
    bool ok = true;
    for (int t = first; t < tiles && ok; t += step) {
      int tp, tq;
      tile_at(t, tp, tq);
      for (int kb = kb0; kb < kb1; ++kb) {
        ok = __all_sync(0xffffffffu, wait_short(sc_empty + 8 * sl.slot, sl.parity ^ 1u));
        if (!ok) {
          if (lane == 0) atomicCAS(&g_f8_status, 0, 4);
          break;
        }
        const uint32_t dst = saddr(scales + sl.slot * (BP + TN));
        const float *ps = p.p.scale + kb * p.p.s_k, *qs = p.q.scale + kb * p.q.s_k;
        if (p.p.shift) {
          const bool in = tp * BP < p.p.extent;  // (a pair's second CTA may have no rows)
          if (lane == 0) cp_async_4(dst, in ? ps + tp * p.p.s_mn : ps, in ? 4 : 0);
        } else {
#pragma unroll
          for (int i = lane; i < BP; i += 32) {
            const int row = tp * BP + i;
            const bool in = row < p.p.extent;
            cp_async_4(dst + 4 * i, in ? ps + row * p.p.s_mn : ps, in ? 4 : 0);
          }
        }
#pragma unroll
        for (int i = lane; i < (QVEC ? TN : (TN + 127) / 128); i += 32) {
          const int col = tq * TN + (QVEC ? i : 128 * i);
          const bool in = col < p.q.extent;
          cp_async_4(dst + 4 * (BP + i), in ? qs + (QVEC ? col : col >> 7) * p.q.s_mn : qs,
                     in ? 4 : 0);
        }
        cp_async_arrive(sc_full + 8 * sl.slot);
        sl.next();
      }
    }
    cp_async_commit();
    cp_async_wait<0>();
  }
  } else {
    // ---- epilogue
    if constexpr (PAIR) reg_alloc<104>();
    const int grp = (warp - 4) >> 2, quad = warp & 3;
    // accumulators and columns of this group: a quarter of a pair's tile is 64 columns of the half
    // of Q that CTA grp % 2 holds, in the accumulators of part grp / 2
    const uint32_t acc0 = PAIR ? (grp >> 1) * C::NBUF : 0;
    const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16) + acc0 * C::ACC_COLS +
                               (uint32_t)((PAIR ? grp & 1 : grp) * C::COLS);
    const int tile_col = PAIR ? 128 * (grp & 1) + 64 * (grp >> 1) : grp * C::COLS;
    const int p_at = p.p.shift ? 0 : quad * 32 + lane;
    const uint32_t full0 = acc_full + 8 * acc0;
    const uint32_t empty0 = PAIR ? in_cta(acc_empty + 8 * acc0, 0) : acc_empty;  // (the leader's)
    Ring<C::NBUF> buf;
    Ring<C::SC_DEPTH> sl;
    bool ok = true;
    for (int t = first; t < tiles && ok; t += step) {
      int tp, tq;
      tile_at(t, tp, tq);
      const int row0 = tp * BP + quad * 32, col0 = tq * TN + tile_col;
      unsigned long long acc[C::COLS / 2];
#pragma unroll
      for (int j = 0; j < C::COLS / 2; ++j) acc[j] = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        ok = __all_sync(0xffffffffu, wait_short(sc_full + 8 * sl.slot, sl.parity) &&
                                         wait_short(full0 + 8 * buf.slot, buf.parity));
        if (!ok) {
          if (lane == 0) atomicCAS(&g_f8_status, 0, 3);
          break;
        }
        fence_after();
        const float *sc = scales + sl.slot * (BP + TN);
        const float *sqb = sc + BP + (QVEC ? tile_col : tile_col / 128);
        const float s = QVEC ? sc[p_at] : sc[p_at] * sqb[0];
        const unsigned long long s2 = pack2(s, s);
        // TMEM is read 32 columns at a time, the next while these are scaled and added. A pair's
        // 96 registers hold one lot only (16 and 16: 431 us, not 402, at 8192x14336x4096), or
        // two of 16 beside the scales of the columns (32 spills: 235 us, not 205, at
        // 4096x4096x8192).
        constexpr bool AHEAD = !PAIR || QVEC;
        constexpr int CH = (PAIR && QVEC) || C::COLS < 32 ? 16 : 32;
        uint32_t v[AHEAD ? 2 : 1][CH];
        const uint32_t src = lane_base + buf.slot * C::ACC_COLS;
        tmem_ld(src, v[0]);
#pragma unroll
        for (int c = 0; c < C::COLS; c += CH) {
          uint32_t(&w)[CH] = v[AHEAD ? c / CH % 2 : 0];
          if (!AHEAD && c > 0) tmem_ld(src + (uint32_t)c, w);
          tmem_wait_ld(w);
          if (AHEAD && c + CH < C::COLS)
            tmem_ld(src + (uint32_t)(c + CH), v[(c / CH + 1) % 2]);
#pragma unroll
          for (int j = 0; j < CH; j += 4) {
            unsigned long long lo = pack2(__uint_as_float(w[j]), __uint_as_float(w[j + 1]));
            unsigned long long hi = pack2(__uint_as_float(w[j + 2]), __uint_as_float(w[j + 3]));
            if constexpr (QVEC) {
              const float4 f = *reinterpret_cast<const float4 *>(sqb + c + j);
              lo = mul2(lo, pack2(f.x, f.y));
              hi = mul2(hi, pack2(f.z, f.w));
            }
            ffma2(acc[(c + j) / 2], lo, s2);
            ffma2(acc[(c + j) / 2 + 1], hi, s2);
          }
        }
        fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (PAIR)
            arrive_in(empty0 + 8 * buf.slot);
          else
            mbar_arrive(empty0 + 8 * buf.slot);
          mbar_arrive(sc_empty + 8 * sl.slot);
        }
        buf.next();
        sl.next();
      }
      if (!ok) break;
      if (S == 1 && p.d_q == 1) {
        uint8_t *turn = reinterpret_cast<uint8_t *>(scales + C::SC_DEPTH * (BP + TN)) +
                        (warp - 4) * TURN_BYTES;
        const Out out{p.D, p.d_type, p.d_p, p.p.extent, p.q.extent, p.alpha, p.beta, p.vec};
        constexpr int CN = C::COLS < 32 ? 16 : 32;
#pragma unroll
        for (int c = 0; c < C::COLS; c += CN) {
          float v[CN];
#pragma unroll
          for (int j = 0; j < CN; j += 2) {
            const float2 f = unpack2(acc[(c + j) / 2]);
            v[j] = f.x;
            v[j + 1] = f.y;
          }
          if (row0 < p.p.extent && col0 + c < p.q.extent)
            store_rows<CN>(out, turn, lane, row0, col0 + c, v);
        }
      } else if (S == 1) {  // P of D's columns: the lanes hold neighbouring elements
#pragma unroll
        for (int c = 0; c < C::COLS; c += 2) {
          const float2 f = unpack2(acc[c / 2]);
          store1(p, row0 + lane, col0 + c, f.x);
          store1(p, row0 + lane, col0 + c + 1, f.y);
        }
      } else {
        // partial tile -> the ring, which every MMA of this CTA has finished reading (the
        // last accumulator is complete): [column][row]
        float *part = reinterpret_cast<float *>(sbase);
#pragma unroll
        for (int j = 0; j < C::COLS; j += 2) {
          const float2 f = unpack2(acc[j / 2]);
          part[(tile_col + j) * PART_PITCH + quad * 32 + lane] = f.x;
          part[(tile_col + j + 1) * PART_PITCH + quad * 32 + lane] = f.y;
        }
      }
    }
  }
  __syncwarp();
  if (S > 1) {
    // CTA `rank` finishes columns [rank * TN / S, (rank + 1) * TN / S): partials in rank order, a
    // warp 32 rows (one per lane) by 8 columns at a time
    cluster_sync_all();
    if (warp >= 4) {
      int tp, tq;
      tile_at(first, tp, tq);
      const int c0 = TN * rank / S, c1 = min(TN * (rank + 1) / S, p.q.extent - tq * TN);
      const int quads = min(4, (p.p.extent - tp * BP + 31) / 32);
      uint8_t *turn = reinterpret_cast<uint8_t *>(scales + C::SC_DEPTH * (BP + TN)) +
                      (warp - 4) * TURN_BYTES;
      const Out out{p.D, p.d_type, p.d_p, p.p.extent, p.q.extent, p.alpha, p.beta, p.vec};
      const int wide = TN / S >= 16 && p.d_q == 1 ? 16 : 8;  // columns of a block
      const int blocks = c1 > c0 ? (c1 - c0 + wide - 1) / wide * quads : 0;
      for (int b = warp - 4; b < blocks; b += C::EPI_WARPS) {
        const int r = b % quads * 32, c = c0 + b / quads * wide;
        float v[16];
#pragma unroll
        for (int h = 0; h < 16; h += 8) {
          if (h >= wide) break;
          float w[MAX_CLUSTER][8];
#pragma unroll
          for (int q = 0; q < MAX_CLUSTER; ++q)  // all loads in flight before the adds
            if (q < S) {
              // Only what is used below: a load that nothing waits for could still be under way
              // when the other CTA leaves.
#pragma unroll
              for (int j = 0; j < 8; ++j)
                if (c + h + j < c1)
                  w[q][j] = ld_cluster1(
                      base + (uint32_t)((c + h + j) * PART_PITCH + r + lane) * 4, (uint32_t)q);
            }
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            v[h + j] = 0.0f;
            if (c + h + j < c1) {
              v[h + j] = w[0][j];
#pragma unroll
              for (int q = 1; q < MAX_CLUSTER; ++q)
                if (q < S) v[h + j] += w[q][j];
            }
          }
        }
        if (wide == 16) {
          store_rows<16>(out, turn, lane, tp * BP + r, tq * TN + c, v);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (c + j < c1) store1(p, tp * BP + r + lane, tq * TN + c + j, v[j]);
        }
      }
    }
    __syncwarp();
    cluster_sync_all();  // no CTA leaves while another may still read its partial
  }
  fence_before();
  __syncthreads();
  if constexpr (PAIR) {
    cluster_sync_all();  // no instruction, copy or arrival of the other CTA is under way
    if (warp == 0) tmem_dealloc_pair(tmem, C::TMEM_COLS);
  } else {
    if (warp == 0) tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// D = beta * D (k == 0 or alpha == 0; 0 when beta == 0, without reading D).
__global__ void f8_scale_kernel(Params p, int M, int N, long long ldd) {
  griddep_wait();
  const long long total = (long long)M * N;
  for (long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x; i < total;
       i += (long long)gridDim.x * blockDim.x) {
    const long long at = i / N * ldd + i % N;
    tcx::finish_out(p.D, p.d_type, at, 0.0f, p.beta);
  }
}

// ------------------------------------------------------------------------------------
// Host side

struct Plan {
  bool swap;   // P = op(B)^T
  bool pair;   // two CTAs per tile of 256 rows
  int tn, split;
};

// Estimated time of a plan in units of 64 cycles, from times measured on GB300 with every plan
// forced on 24 shapes: what a block of k costs a CTA (more where Q has a scale for each column), the
// stores of a tile (three times that where the lanes hold D's rows), and a cluster's exchange (twice
// where they do: 64 x 4096 x 4096 took 9.7 us so, against 7.6 in one piece). The estimate's choice is
// within 5% of the best plan, or within 1 us where a call takes less than 6.
static Plan make_plan(int M, int N, int KB, bool a_mn, bool b_mn, bool a_vec, bool b_vec, int sms) {
  Plan best{false, false, 128, 1};
  double best_cost = 1e300;
  static const int tns[5] = {256, 128, 64, 32, 16};
  static const double block[5] = {16, 9.5, 7, 6, 6}, block_vec[5] = {24, 14, 9, 7, 6};
  static const double store[5] = {70, 25, 15, 10, 8};
  for (int swap = 0; swap < 2; ++swap)
    for (int i = 0; i < 5; ++i) {
      const int tn = tns[i], P = swap ? N : M, Q = swap ? M : N;
      const bool pair = tn == 256, vec = swap ? a_vec : b_vec;
      if ((swap ? a_mn : b_mn) && tn < 32) continue;  // (the narrowest swizzle spans 32 bytes)
      const long long tiles = (long long)ceil_div(P, pair ? 2 * BP : BP) * ceil_div(Q, tn);
      for (int S = 1; S <= MAX_CLUSTER; S *= 2) {
        // (clusters of 8 sit in one GPC each: more than about 12 of them do not run at once)
        if (S > 1 && (pair || S > KB || tiles * S > (S == 8 ? 96 : sms))) break;
        const int at_once = pair ? sms / 2 : sms;
        const long long per_sm = (tiles * S + at_once - 1) / at_once;
        const double cost = per_sm * ((vec ? block_vec : block)[i] * ((KB + S - 1) / S) +
                                      (swap ? 3.0 : 1.0) * store[i] / S) +
                            (S > 1 ? 25.0 + (swap ? 2.2 : 1.1) * tn : 0.0);
        if (cost < best_cost) {
          best_cost = cost;
          best = Plan{swap != 0, pair, tn, S};
        }
      }
    }
  return best;
}

template <int TN, bool PAIR = false>
static cudaError_t launch(bool vec, const CUtensorMap &mp, const CUtensorMap &mq, const Params &p,
                          int grid, cudaStream_t stream) {
  using C = Cfg<TN, PAIR>;
  const int cluster = PAIR ? 2 : p.split;
  return vec ? launch_1d(f8_kernel<TN, true, PAIR>, grid, C::THREADS, C::SMEM_BYTES, cluster,
                         stream, mp, mq, p)
             : launch_1d(f8_kernel<TN, false, PAIR>, grid, C::THREADS, C::SMEM_BYTES, cluster,
                         stream, mp, mq, p);
}

template <int TN, bool PAIR = false>
static cudaError_t set_attributes() {
  const int bytes = Cfg<TN, PAIR>::SMEM_BYTES;
  cudaError_t e = cudaFuncSetAttribute(f8_kernel<TN, false, PAIR>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(f8_kernel<TN, true, PAIR>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  return e;
}

static std::once_flag g_once[64];
static cudaError_t g_err[64];

static cudaError_t kernel_setup() {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  std::call_once(g_once[dev], [dev]() {
    cudaError_t err = set_attributes<256, true>();
    if (err == cudaSuccess) err = set_attributes<128>();
    if (err == cudaSuccess) err = set_attributes<64>();
    if (err == cudaSuccess) err = set_attributes<32>();
    if (err == cudaSuccess) err = set_attributes<16>();
    g_err[dev] = err;
  });
  return g_err[dev];
}

// Tensor map of one operand: `extent` rows (columns for Q) by K, k contiguous or not.
static bool side_map(CUtensorMap *map, const void *ptr, int extent, int K, int ld, bool mn_major,
                     int box_extent) {
  return mn_major ? encode_map_2d_narrow(map, ptr, 1, K, extent, ld, BK, std::min(box_extent, 128))
                  : encode_map_2d_narrow(map, ptr, 1, extent, K, ld, box_extent);
}

}  // namespace f8
}  // namespace sgemm

using namespace sgemm;

extern "C" int f8_gemm(int transa, int transb, int M, int N, int K, float alpha, const void *A,
                       int a_format, int lda, const float *a_scale, int a_rows,
                       long long a_scale_mn, long long a_scale_k, const void *B, int b_format,
                       int ldb, const float *b_scale, int b_cols, long long b_scale_mn,
                       long long b_scale_k, float beta, void *D, int d_type, int ldd,
                       cudaStream_t stream) {
  const bool read = M > 0 && N > 0 && K > 0 && alpha != 0.0f;
  const auto bad_ptr = [](const void *q) { return (reinterpret_cast<uintptr_t>(q) & 15u) != 0; };
  if (transa != 0 && transa != 1) return -1;
  if (transb != 0 && transb != 1) return -2;
  if (M < 0) return -3;
  if (N < 0) return -4;
  if (K < 0) return -5;
  if (read && (A == nullptr || bad_ptr(A))) return -7;
  if (a_format != F8_E4M3 && a_format != F8_E5M2) return -8;
  if (lda < std::max(1, transa ? M : K) || lda % 16 != 0) return -9;
  if (read && a_scale == nullptr) return -10;
  if (a_rows != 1 && a_rows != 128) return -11;
  if (a_scale_mn < 0) return -12;
  if (a_scale_k < 0) return -13;
  if (read && (B == nullptr || bad_ptr(B))) return -14;
  if (b_format != F8_E4M3 && b_format != F8_E5M2) return -15;
  if (ldb < std::max(1, transb ? K : N) || ldb % 16 != 0) return -16;
  if (read && b_scale == nullptr) return -17;
  if (b_cols != 1 && b_cols != 128) return -18;
  if (b_scale_mn < 0) return -19;
  if (b_scale_k < 0) return -20;
  if (M > 0 && N > 0 && D == nullptr) return -22;
  if (d_type != F8_D_F32 && d_type != F8_D_BF16 && d_type != F8_D_F16) return -23;
  if (ldd < std::max(1, N)) return -24;
  if (D != nullptr && reinterpret_cast<uintptr_t>(D) % (d_type == F8_D_F32 ? 4 : 2) != 0)
    return -22;
  if (M == 0 || N == 0) return 0;

  int sms = 0;
  cudaError_t e = device_setup(&sms);
  if (e == cudaSuccess) e = f8::kernel_setup();
  if (e != cudaSuccess) return (int)e;

  f8::Params p{};
  p.alpha = alpha;
  p.beta = beta;
  p.D = D;
  p.d_type = d_type;
  if (!read) {
    if (beta == 1.0f) return 0;
    const long long blocks = std::min<long long>(((long long)M * N + 255) / 256, 8LL * sms);
    return (int)launch_1d(f8::f8_scale_kernel, (int)blocks, 256, 0, 1, stream, p, M, N,
                          (long long)ldd);
  }
  p.KB = ceil_div(K, f8::BK);
  const f8::Plan pl =
      f8::make_plan(M, N, p.KB, transa == 1, transb == 0, a_rows == 1, b_cols == 1, sms);
  const f8::Side sa{M, transa == 1, a_scale, a_rows == 128 ? 7 : 0, a_scale_mn, a_scale_k};
  const f8::Side sb{N, transb == 0, b_scale, b_cols == 128 ? 7 : 0, b_scale_mn, b_scale_k};
  p.p = pl.swap ? sb : sa;
  p.q = pl.swap ? sa : sb;
  p.d_p = pl.swap ? 1 : ldd;
  p.d_q = pl.swap ? ldd : 1;
  const int size = d_type == F8_D_F32 ? 4 : 2;
  p.vec = !bad_ptr(D) && (long long)ldd * size % 16 == 0;
  const long long tiles_p = ceil_div(p.p.extent, f8::BP), tiles_q = ceil_div(p.q.extent, pl.tn);
  if (tiles_p * tiles_q > 0x7fffffffLL / f8::MAX_CLUSTER) return (int)cudaErrorInvalidConfiguration;
  p.tiles_p = (int)tiles_p;
  p.tiles_q = (int)tiles_q;
  p.group_p = (int)std::min<long long>(pl.pair ? 8 : 16, tiles_p);
  p.split = pl.split;
  const uint32_t fp = pl.swap ? b_format : a_format, fq = pl.swap ? a_format : b_format;
  // instruction descriptor: D in FP32 (bits 4-5 = 1), formats of P and Q (0 = e4m3, 1 = e5m2;
  // bits 7-9, 10-12), MN-major P and Q (bits 15, 16), N / 8 (bits 17-22), M / 16 (24-28)
  p.idesc = (1u << 4) | (fp << 7) | (fq << 10) | ((uint32_t)p.p.mn_major << 15) |
            ((uint32_t)p.q.mn_major << 16) |
            ((uint32_t)((pl.pair ? pl.tn / 2 : pl.tn) >> 3) << 17) |
            ((uint32_t)((pl.pair ? 2 * f8::BP : f8::BP) >> 4) << 24);

  CUtensorMap mp, mq;
  if (!f8::side_map(&mp, pl.swap ? B : A, p.p.extent, K, pl.swap ? ldb : lda, p.p.mn_major,
                    f8::BP) ||
      !f8::side_map(&mq, pl.swap ? A : B, p.q.extent, K, pl.swap ? lda : ldb, p.q.mn_major,
                    pl.pair ? pl.tn / 2 : pl.tn))
    return (int)cudaErrorInvalidValue;
  const int grid =
      (int)(pl.pair ? 2 * std::min<long long>(ceil_div(tiles_p, 2) * tiles_q, sms / 2)
            : p.split > 1 ? tiles_p * tiles_q * p.split
                          : std::min<long long>(tiles_p * tiles_q, sms));
  const bool vec = p.q.shift == 0;
  switch (pl.tn) {
    case 256: return (int)f8::launch<256, true>(vec, mp, mq, p, grid, stream);
    case 128: return (int)f8::launch<128>(vec, mp, mq, p, grid, stream);
    case 64: return (int)f8::launch<64>(vec, mp, mq, p, grid, stream);
    case 32: return (int)f8::launch<32>(vec, mp, mq, p, grid, stream);
    default: return (int)f8::launch<16>(vec, mp, mq, p, grid, stream);
  }
}

extern "C" int f8_gemm_plan(int transa, int transb, int M, int N, int K, int a_rows, int b_cols,
                            int num_sms, int *exchanged, int *tile_cols, int *split) {
  if (transa != 0 && transa != 1) return -1;
  if (transb != 0 && transb != 1) return -2;
  if (M < 1) return -3;
  if (N < 1) return -4;
  if (K < 1) return -5;
  if (a_rows != 1 && a_rows != 128) return -6;
  if (b_cols != 1 && b_cols != 128) return -7;
  if (num_sms < 0) return -8;
  int sms = num_sms;
  if (sms == 0 && device_setup(&sms) != cudaSuccess) {
    (void)cudaGetLastError();
    sms = 152;  // no device here: the answer for a whole GB300
  }
  const f8::Plan pl = f8::make_plan(M, N, ceil_div(K, f8::BK), transa == 1, transb == 0,
                                    a_rows == 1, b_cols == 1, sms);
  if (exchanged) *exchanged = pl.swap;
  if (tile_cols) *tile_cols = pl.tn;
  if (split) *split = pl.split;
  return 0;
}

extern "C" int f8_gemm_with(const f8_gemm_args *a) {
  if (a == nullptr) return -1;
  return f8_gemm(a->transa, a->transb, a->M, a->N, a->K, a->alpha, a->A, a->a_format, a->lda,
                 a->a_scale, a->a_rows, a->a_scale_mn, a->a_scale_k, a->B, a->b_format, a->ldb,
                 a->b_scale, a->b_cols, a->b_scale_mn, a->b_scale_k, a->beta, a->D, a->d_type,
                 a->ldd, a->stream);
}

extern "C" int f8_gemm_status(int *status) {
  int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, f8::g_f8_status, sizeof(int));
  if (e != cudaSuccess) return (int)e;
  const int zero = 0;
  e = cudaMemcpyToSymbol(f8::g_f8_status, &zero, sizeof(int));
  if (status) *status = v;
  return (int)e;
}

// D = x w^T on 8-bit integers with a scale for each row of x (token) and of w (channel):
//
//   D(i, j) = sx(i) sw(j) sum_k qx(i, k) qw(j, k) + bias(j) + beta D(i, j)
//
// The 8-bit integer rate of sm_103a's tensor cores is a small part of their FP16 rate, and FP16 holds
// every int8 exactly. So the products run as FP16 ones (tcgen05, kind f16): products of two int8 are
// at most 2^14, and a sum of 1024 of them at most 2^24, which FP32 accumulators hold without a
// rounding. After each 1024 of k the epilogue warps take the accumulator from TMEM and add it to
// 32-bit integers in registers. The result is the exact whole number, so that neither tiles nor splits
// show in it.
//
// The weight stays int8 on its way from memory. The kernel sees the product as P = w (128 channels per
// tile, on the instruction's 128-row side, however few tokens there are) times Q = x (TN tokens per
// tile). A warpgroup of converters reads P's bytes from shared memory, where TMA has put them, and
// writes them as FP16 numbers into TMEM, from where the instruction takes P: the numbers never pass
// through shared memory, whose bandwidth (TMA's writes, the converters' and the tensor core's reads) is
// what large tiles are short of. Q is FP16 in shared memory: converted by the same warps where it is
// narrow, and before the kernel (unpack_kernel, into the workspace) where it is wide.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>

#include "../../include/i8_linear.h"
#include "i8_internal.h"
#include "sgemm_internal.h"
#include "sgemm_plan.h"
#include "tc_common.cuh"

namespace sgemm {
namespace i8 {

constexpr int BP = 128;                  // channels per CTA and tile
constexpr int BK = 128;                  // k per block = per pipeline stage
constexpr int CHUNK = 8;                 // blocks of k that an accumulator holds: 1024 products
constexpr int P_BYTES = BP * BK;
constexpr int MAX_CLUSTER = 8;
constexpr int LARGEST_K = 131071;        // 2^14 K < 2^31

// Results on their way out: a warp's buffer of 16 tokens' numbers of its 32 channels. (A pitch of 36: two
// neighbouring rows' 16-byte pieces lie in different banks.)
constexpr int OUT_PITCH = 36;
constexpr int OUT_BYTES = 16 * OUT_PITCH * 4;

// PAIR: two CTAs share a tile of 256 channels and TN tokens (tcgen05 cta_group::2), each with its 128
// channels and half of the tokens.
template <int TN_, bool PAIR_>
struct Cfg {
  static constexpr int TN = TN_;
  static constexpr bool PAIR = PAIR_;
  static constexpr bool CONVERT = TN <= 64;        // Q arrives as int8
  static constexpr int QN = PAIR ? TN / 2 : TN;    // tokens that this CTA holds
  static constexpr int GROUPS = TN >= 64 ? 2 : 1;  // epilogue groups of four warps
  static constexpr int COLS = TN / GROUPS;         // tokens of a group
  static constexpr int EPI_WARPS = 4 * GROUPS;
  // Two converter groups take turns with the blocks of k: 384 x 14336 x 4096 takes a pair 39.5 us, with
  // one group 43.3. (A single CTA with 64 sums per thread has no registers for the second: 24 us for 22.)
  static constexpr int CONV_GROUPS = TN == 128 && !PAIR ? 1 : 2;
  static constexpr int FIRST_EPI = 4 + 4 * CONV_GROUPS;  // warp
  static constexpr int THREADS = 32 * (FIRST_EPI + EPI_WARPS);
  // A pair's registers per thread: control warps, converters, epilogue (where the sums are more than an
  // even share leaves room for).
  static constexpr int CONTROL_REGS = 56, CONV_REGS = 88, EPI_REGS = 120;
  static constexpr int REGS = 128 * CONTROL_REGS + 128 * CONV_GROUPS * CONV_REGS + 32 * EPI_WARPS * EPI_REGS;
  static constexpr int Q_BYTES = QN * BK * (CONVERT ? 1 : 2);
  static constexpr int STAGE_BYTES = P_BYTES + Q_BYTES;
  static constexpr int STAGES = CONVERT ? (TN == 64 ? 4 : 8) : PAIR ? 6 : 4;
  static constexpr int NA = 4;                     // blocks of P in TMEM (and of Q, where converted)
  static constexpr int A_COLS = BK / 2;            // columns of one
  static constexpr int H_BYTES = CONVERT ? QN * BK * 2 : 0;
  static constexpr int NBUF = 2;                   // accumulators
  static constexpr int ACC_COLS = TN < 32 ? 32 : TN;
  static constexpr int ACC_WARPS = EPI_WARPS * (PAIR ? 2 : 1);  // readers of an accumulator
  static constexpr int TMEM_COLS = 512;
  static constexpr int BARS = 3 * STAGES + 2 * NA + 2 * NBUF;
  static constexpr int SMEM_BYTES = 1024 + STAGES * STAGE_BYTES + NA * H_BYTES + EPI_WARPS * OUT_BYTES + 8 * BARS + 16;
  // (a barrier tells only odd uses of a slot from even ones: whoever waits for it must see them all)
  static_assert(STAGES % CONV_GROUPS == 0 && NA % CONV_GROUPS == 0, "each slot belongs to one group");
  static_assert(!PAIR || REGS <= 65536 / THREADS / 8 * 8 * THREADS, "registers that a launch brings");
  static_assert(NBUF * ACC_COLS + NA * A_COLS <= TMEM_COLS, "TMEM columns");
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory per CTA");
  static_assert(BP * TN * 4 <= STAGES * STAGE_BYTES, "a partial tile fits in the ring");
  static_assert(STAGE_BYTES % 1024 == 0 && H_BYTES % 1024 == 0, "swizzled tiles");
};

struct Params {
  int N, M, KB;        // channels, tokens, blocks of k
  int tiles_p, tiles_q, group_p;
  int split;           // CTAs of a cluster, each with its range of k blocks
  uint32_t idesc;
  const float *w_scale, *x_scale;
  Result d;
};

// Device status word: 0 = fine; 1, 2, 3, 4 = a wait of the producer, the MMA issuer, the epilogue
// or the converters gave up.
__device__ int g_i8_status;

__device__ __forceinline__ void async_fence() { asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory"); }

// One channel's finished sums: factor and bias of the channel.
struct Channel {
  int at;
  float scale, bias;
};

// Sums of this lane's channel and COUNT neighbouring tokens, finished and stored. What is not
// unrolled over the sums is unrolled little: the epilogue shares the instruction caches with the
// converters (all inlined and unrolled it took half of their time).
// sx: the scale of token `token` + lane - from in each lane.
constexpr int COUNT = 16;
__device__ __forceinline__ void store_tokens(const Params &p, const Channel &c, float sx, int from, float *buf,
                                             int lane, int token, const int (&sums)[COUNT]) {
  const int rows = min(COUNT, p.M - token);
#pragma unroll
  for (int j = 0; j < COUNT; ++j)
    buf[j * OUT_PITCH + lane] =
        fmaf((float)sums[j], c.scale * __shfl_sync(0xffffffffu, sx, from + j), c.bias);
  __syncwarp();
  const int col0 = c.at - lane;
  if (p.d.vec && p.d.type != tcx::OUT_F32) {
    const int col = (lane & 3) * 8, cols = min(8, p.N - col0 - col);
#pragma unroll 2
    for (int r = lane >> 2; r < rows; r += 8) {
      const float *v = buf + r * OUT_PITCH + col;
      uint16_t *d = static_cast<uint16_t *>(p.d.ptr) + (token + r) * p.d.ld + col0 + col;
      if (cols == 8) {
        const float4 x = *reinterpret_cast<const float4 *>(v), y = *reinterpret_cast<const float4 *>(v + 4);
        *reinterpret_cast<uint4 *>(d) =
            make_uint4(tcx::pack_out(p.d.type, x.x, x.y), tcx::pack_out(p.d.type, x.z, x.w),
                       tcx::pack_out(p.d.type, y.x, y.y), tcx::pack_out(p.d.type, y.z, y.w));
      } else {
#pragma unroll 1
        for (int j = 0; j < cols; ++j) tcx::store_out(d, p.d.type, j, v[j]);
      }
    }
  } else if (p.d.vec) {
    const int col = (lane & 7) * 4, cols = min(4, p.N - col0 - col);
#pragma unroll 2
    for (int r = lane >> 3; r < rows; r += 4) {
      const float *v = buf + r * OUT_PITCH + col;
      float *d = static_cast<float *>(p.d.ptr) + (token + r) * p.d.ld + col0 + col;
      if (cols == 4) {
        *reinterpret_cast<float4 *>(d) = *reinterpret_cast<const float4 *>(v);
      } else {
#pragma unroll 1
        for (int j = 0; j < cols; ++j) d[j] = v[j];
      }
    }
  } else if (c.at < p.N && p.d.type == tcx::OUT_F32 && p.d.beta == 0.0f) {
    float *d = static_cast<float *>(p.d.ptr) + token * p.d.ld + c.at;
#pragma unroll 8
    for (int r = 0; r < rows; ++r) d[r * p.d.ld] = buf[r * OUT_PITCH + lane];
  } else if (c.at < p.N && p.d.beta == 0.0f) {
    uint16_t *d = static_cast<uint16_t *>(p.d.ptr) + token * p.d.ld + c.at;
#pragma unroll 8
    for (int r = 0; r < rows; ++r) d[r * p.d.ld] = (uint16_t)tcx::pack_out(p.d.type, buf[r * OUT_PITCH + lane], 0.0f);
  } else if (c.at < p.N) {
#pragma unroll 2
    for (int r = 0; r < rows; ++r)
      tcx::finish_out(p.d.ptr, p.d.type, (token + r) * p.d.ld + c.at, buf[r * OUT_PITCH + lane], p.d.beta);
  }
  __syncwarp();
}

__device__ __forceinline__ Channel channel_at(const Params &p, int at) {
  const bool in = at < p.N;
  return {at, in ? p.w_scale[at] : 0.0f, in && p.d.bias ? p.d.bias[at] : 0.0f};
}

// What bounds it (GB300, us on the GPU in a stream of calls on weights from memory).
//   8192 x 14336 x 4096: 508 to 515, 1.87 PFLOP/s, 97% of the measured FP16/BF16 rate: the tensor core.
//     (Tiles of 256 channels x 256 tokens took 555; with P converted into shared memory instead of TMEM the
//     shared memory would need 1.5 times the tensor core's time.)
//   2048 x 4096 x 4096: 52; 256 tiles on 76 pairs are 3.4 rounds that take the time of 4, tensor core 71%
//     busy. 512 x 4096 x 4096: 19.5 with 64 tiles, one round of 32 blocks at 0.32 us and 5 us around it.
//   16 x 14336 x 4096: 13.7; 112 tiles for 152 SMs, whose blocks arrive at 5.5 TB/s after the first 2 us.
//   16 x 4096 x 8192: 10.1; 128 CTAs get their 16 blocks in 6.8 us (the first half in 4.7: a call's start,
//     and 128 KB for each CTA at once), then 2 us for the cluster's barrier, exchange and stores.
//   517 x 3001 x 777: 11.0; a launch to convert x, one round of seven blocks, stores of unaligned rows.
// A converter thread takes about 450 cycles for its 128 bytes of a block, and as many again for Q of 64
// tokens; the instructions on a block take 240 cycles with 16 tokens and 512 with a pair's 128.
//
// Warp 0: TMA producer, warp 1: MMA issuer (one elected lane of each), then the converters, one row of P
// per thread of a group; the last warps: epilogue, a group of four warps owns COLS tokens of the tile, warp w of
// it TMEM lanes (channels) 32 (w % 4) .. + 31, one per thread.
template <int TN, bool PAIR>
__global__ void __launch_bounds__(Cfg<TN, PAIR>::THREADS, 1)
    i8_kernel(const __grid_constant__ CUtensorMap map_p, const __grid_constant__ CUtensorMap map_q,
              const Params p) {
  using C = Cfg<TN, PAIR>;
  using namespace tcx;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = saddr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t *sbase = smem_raw + (base - raw);
  const uint32_t halves_at = base + C::STAGES * C::STAGE_BYTES;  // Q in FP16, where it is converted
  const uint32_t out_at = halves_at + C::NA * C::H_BYTES;        // (the epilogue's buffers)
  const uint32_t p_full = out_at + C::EPI_WARPS * OUT_BYTES;
  const uint32_t q_full = p_full + 8 * C::STAGES, empty = q_full + 8 * C::STAGES;
  const uint32_t a_full = empty + 8 * C::STAGES, a_empty = a_full + 8 * C::NA;
  const uint32_t acc_full = a_empty + 8 * C::NA, acc_empty = acc_full + 8 * C::NBUF;
  const uint32_t tmem_slot = acc_empty + 8 * C::NBUF;
  volatile uint32_t *tmem_slot_ptr =
      reinterpret_cast<volatile uint32_t *>(smem_raw + (tmem_slot - raw));

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  // a cluster is S CTAs with a range of k blocks each, or a pair on one tile of 256 channels
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
      mbar_init(p_full + 8 * s, 1);
      mbar_init(q_full + 8 * s, 1);
      mbar_init(empty + 8 * s, C::CONVERT ? 4 : 1);
    }
    for (int a = 0; a < C::NA; ++a) {
      mbar_init(a_full + 8 * a, PAIR ? 8 : 4);
      mbar_init(a_empty + 8 * a, 1);
    }
    for (int b = 0; b < C::NBUF; ++b) {
      mbar_init(acc_full + 8 * b, 1);
      mbar_init(acc_empty + 8 * b, C::ACC_WARPS);
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
  const uint32_t a_tmem = tmem + C::NBUF * C::ACC_COLS;
  const auto tile_at = [&](int t, int &tp, int &tq) {
    tile_coords(t, units, p.tiles_q, p.group_p, tp, tq);
    if (PAIR) tp = 2 * tp + cta;
  };
  // The first blocks of the weight begin their way to L2 while the kernel before this one still runs. (To L2
  // only, where what that kernel may yet write to them is seen.) Every CTA of the grid is resident, so the
  // next launch may take what room is left.
  if (warp == 0 && elect_one()) {
    int tp, tq;
    tile_at(first, tp, tq);
    for (int kb = kb0; kb < min(kb1, kb0 + C::STAGES); ++kb) tma_prefetch_2d(&map_p, kb * BK, tp * BP);
  }
  __syncwarp();
  griddep_launch_dependents();
  griddep_wait();  // (launched with programmatic dependent launch: see launch_1d)

  if (warp < 4) {
    if constexpr (PAIR) reg_dealloc<C::CONTROL_REGS>();
    if (warp == 0) {
      // ---- TMA producer: the k blocks of this CTA's tiles, in order, through the ring of stages
      Ring<C::STAGES> st;
      int issued = 0;  // (up to STAGES)
      bool ok = true;
      for (int t = first; t < tiles && ok; t += step) {
        int tp, tq;
        tile_at(t, tp, tq);
        for (int kb = kb0; kb < kb1; ++kb) {
          ok = __all_sync(0xffffffffu, wait_short(empty + 8 * st.slot, st.parity ^ 1u));
          if (!ok) {
            if (lane == 0) atomicCAS(&g_i8_status, 0, 1);
            break;
          }
          if (elect_one()) {
            const uint32_t dst = base + st.slot * C::STAGE_BYTES;
            const uint32_t pf = p_full + 8 * st.slot, qf = q_full + 8 * st.slot;
            const int k = kb * BK, q0 = tq * TN + cta * (PAIR ? C::QN : 0);
            mbar_expect_tx(pf, P_BYTES);
            tma_load_2d(dst, &map_p, k, tp * BP, pf);
            if constexpr (C::CONVERT) {
              mbar_expect_tx(qf, C::Q_BYTES);
              tma_load_2d(dst + P_BYTES, &map_q, k, q0, qf);
            } else if constexpr (PAIR) {  // both CTAs' copies complete the leader's barrier
              const uint32_t lead = in_cta(qf, 0);
              if (cta == 0) mbar_expect_tx(qf, 2 * C::Q_BYTES);
              tma_load_2d_pair(dst + P_BYTES, &map_q, k, q0, lead);
              tma_load_2d_pair(dst + P_BYTES + C::QN * 128, &map_q, k + 64, q0, lead);
            } else {
              mbar_expect_tx(qf, C::Q_BYTES);
              tma_load_2d(dst + P_BYTES, &map_q, k, q0, qf);
              tma_load_2d(dst + P_BYTES + C::QN * 128, &map_q, k + 64, q0, qf);
            }
          }
          __syncwarp();
          issued = min(issued + 1, C::STAGES);
          st.next();
        }
      }
      // the last loads issued must have landed before this warp leaves (of a pair's Q: the leader
      // waits for both, and the CTAs leave together)
      for (; issued > 0; --issued) {
        st.parity ^= st.slot == 0 ? 1u : 0u;
        st.slot = st.slot == 0 ? C::STAGES - 1 : st.slot - 1;
        wait_short(p_full + 8 * st.slot, st.parity);
        if (!PAIR || cta == 0) wait_short(q_full + 8 * st.slot, st.parity);
      }
    } else if (warp == 1 && (!PAIR || cta == 0)) {
      // ---- MMA issuer
      const uint64_t qd0 = sw128_desc(C::CONVERT ? halves_at : base + P_BYTES, 16);
      Ring<C::STAGES> st;
      Ring<C::NA> ar;
      Ring<C::NBUF> buf;
      bool ok = true;
      for (int t = first; t < tiles && ok; t += step) {
        for (int kb = kb0; kb < kb1; ++kb) {
          const int in_chunk = (kb - kb0) % CHUNK;
          const bool begin = in_chunk == 0, end = in_chunk == CHUNK - 1 || kb == kb1 - 1;
          ok = __all_sync(0xffffffffu, wait_short(a_full + 8 * ar.slot, ar.parity) &&
                                           (C::CONVERT || wait_short(q_full + 8 * st.slot, st.parity)));
          fence_after();
          const uint32_t a = a_tmem + ar.slot * C::A_COLS;
          const uint64_t qd =
              qd0 + (C::CONVERT ? ar.slot * (uint32_t)(C::H_BYTES >> 4) : st.slot * (uint32_t)(C::STAGE_BYTES >> 4));
          if (ok && begin) {
            ok = __all_sync(0xffffffffu, wait_short(acc_empty + 8 * buf.slot, buf.parity ^ 1u));
            fence_after();
          }
          if (ok && elect_one()) {
            const uint32_t d = tmem + buf.slot * C::ACC_COLS;
#pragma unroll
            for (uint32_t kk = 0; kk < BK / 16; ++kk) {
              // 64 of k per box of 128-byte rows
              const uint64_t q = qd + ((kk / 4 * C::QN * 128 + kk % 4 * 32) >> 4);
              const uint32_t more = !begin || kk != 0;
              if constexpr (PAIR)
                mma_f16_tmem_pair(d, a + kk * 8, q, p.idesc, more);
              else
                mma_f16_tmem(d, a + kk * 8, q, p.idesc, more);
            }
            // (the accumulator's last: who has seen the last accumulator knows that no arrival is to come)
            if constexpr (PAIR) {
              mma_commit_pair(a_empty + 8 * ar.slot);
              mma_commit_pair(empty + 8 * st.slot);
              if (end) mma_commit_pair(acc_full + 8 * buf.slot);
            } else {
              mma_commit(a_empty + 8 * ar.slot);
              if constexpr (!C::CONVERT) mma_commit(empty + 8 * st.slot);
              if (end) mma_commit(acc_full + 8 * buf.slot);
            }
          }
          __syncwarp();
          if (!ok) {
            if (lane == 0) atomicCAS(&g_i8_status, 0, 2);
            break;
          }
          st.next();
          ar.next();
          if (end) buf.next();
        }
      }
    }
  } else if (warp < C::FIRST_EPI) {
    // ---- converters
    if constexpr (PAIR) reg_dealloc<C::CONV_REGS>();
    const int row = threadIdx.x % 128;  // of P
    int turns = (warp - 4) >> 2;        // blocks until this group's next one
    const uint32_t a_lane = a_tmem + ((uint32_t)((warp & 3) * 32) << 16);
    Ring<C::STAGES> st;
    Ring<C::NA> ar;
    bool ok = true;
    for (int t = first; t < tiles && ok; t += step) {
      for (int kb = kb0; kb < kb1; ++kb) {
        if (C::CONV_GROUPS > 1 && turns-- != 0) {
          st.next();
          ar.next();
          continue;
        }
        turns = C::CONV_GROUPS - 1;
        ok = __all_sync(0xffffffffu, wait_short(p_full + 8 * st.slot, st.parity) &&
                                         (!C::CONVERT || wait_short(q_full + 8 * st.slot, st.parity)) &&
                                         wait_short(a_empty + 8 * ar.slot, ar.parity ^ 1u));
        if (!ok) {
          if (lane == 0) atomicCAS(&g_i8_status, 0, 4);
          break;
        }
        fence_after();
        const uint8_t *stage = sbase + st.slot * C::STAGE_BYTES;
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {  // 64 of k: 32 columns
          uint32_t v[32];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint4 u =
                *reinterpret_cast<const uint4 *>(stage + row * 128 + (((4 * h + c) ^ (row & 7)) << 4));
            tcx::halves(u.x, v[8 * c], v[8 * c + 1]);
            tcx::halves(u.y, v[8 * c + 2], v[8 * c + 3]);
            tcx::halves(u.z, v[8 * c + 4], v[8 * c + 5]);
            tcx::halves(u.w, v[8 * c + 6], v[8 * c + 7]);
          }
          tmem_st(a_lane + ar.slot * C::A_COLS + h * 32, v);
        }
        if constexpr (C::CONVERT) {
          // Q: 16 of k of a token at a time, into two boxes of 64 of k with 128-byte rows
          uint8_t *to = sbase + C::STAGES * C::STAGE_BYTES + ar.slot * C::H_BYTES;
#pragma unroll
          for (int i = row; i < TN * 8; i += 128) {
            const int r = i >> 3, j = i & 7;
            const uint4 u = *reinterpret_cast<const uint4 *>(stage + P_BYTES + r * 128 + ((j ^ (r & 7)) << 4));
            uint4 lo, hi;
            tcx::halves(u.x, lo.x, lo.y);
            tcx::halves(u.y, lo.z, lo.w);
            tcx::halves(u.z, hi.x, hi.y);
            tcx::halves(u.w, hi.z, hi.w);
            uint8_t *box = to + (j >> 2) * (TN * 128) + r * 128;
            *reinterpret_cast<uint4 *>(box + (((2 * j & 7) ^ (r & 7)) << 4)) = lo;
            *reinterpret_cast<uint4 *>(box + (((2 * j + 1 & 7) ^ (r & 7)) << 4)) = hi;
          }
          async_fence();  // (the tensor core reads them)
        }
        tmem_wait_st();
        fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (PAIR)
            arrive_in(in_cta(a_full + 8 * ar.slot, 0));
          else
            mbar_arrive(a_full + 8 * ar.slot);
          if constexpr (C::CONVERT) mbar_arrive(empty + 8 * st.slot);
        }
        st.next();
        ar.next();
      }
    }
  } else {
    // ---- epilogue
    if constexpr (PAIR) reg_alloc<C::EPI_REGS>();
    const int grp = (warp - C::FIRST_EPI) >> 2, quad = warp & 3;
    const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)(grp * C::COLS);
    float *out = reinterpret_cast<float *>(smem_raw + (out_at - raw) + (warp - C::FIRST_EPI) * OUT_BYTES);
    Ring<C::NBUF> buf;
    bool ok = true;
    for (int t = first; t < tiles && ok; t += step) {
      int tp, tq;
      tile_at(t, tp, tq);
      // Token of column c, and what the results are multiplied with: read now, for the end.
      const auto token_of = [&](int c) { return tq * TN + grp * C::COLS + c; };
      const Channel ch = channel_at(p, tp * BP + quad * 32 + lane);
      float sx[(C::COLS + 31) / 32];
#pragma unroll
      for (int c = 0; c < C::COLS; c += 32) {
        const int token = token_of(c) + lane;
        sx[c / 32] = token < p.M ? p.x_scale[token] : 0.0f;
      }
      int acc[C::COLS];
#pragma unroll
      for (int j = 0; j < C::COLS; ++j) acc[j] = 0;
      for (int kb = kb0; kb < kb1; kb += CHUNK) {
        ok = __all_sync(0xffffffffu, wait_short(acc_full + 8 * buf.slot, buf.parity));
        if (!ok) {
          if (lane == 0) atomicCAS(&g_i8_status, 0, 3);
          break;
        }
        fence_after();
        constexpr int CH = C::COLS < 32 ? 16 : 32;
        const uint32_t src = lane_base + buf.slot * C::ACC_COLS;
#pragma unroll
        for (int c = 0; c < C::COLS; c += CH) {
          uint32_t v[CH];
          tmem_ld(src + (uint32_t)c, v);
          tmem_wait_ld(v);
          if (c + CH >= C::COLS) {  // everything is in registers
            fence_before();
            __syncwarp();
            if (lane == 0) {
              if constexpr (PAIR)
                arrive_in(in_cta(acc_empty + 8 * buf.slot, 0));
              else
                mbar_arrive(acc_empty + 8 * buf.slot);
            }
          }
#pragma unroll
          for (int j = 0; j < CH; ++j) acc[c + j] += __float2int_rn(__uint_as_float(v[j]));
        }
        buf.next();
      }
      if (!ok) break;
      if (S == 1) {
#pragma unroll
        for (int c = 0; c < C::COLS; c += 16) {
          int sums[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) sums[j] = acc[c + j];
          if (token_of(c) < p.M) store_tokens(p, ch, sx[c / 32], c % 32, out, lane, token_of(c), sums);
        }
      } else {
        // partial tile -> the ring, whose every reader has finished (the last accumulator is
        // complete): [token][channel]
        int *part = reinterpret_cast<int *>(sbase);
#pragma unroll
        for (int j = 0; j < C::COLS; ++j) part[(grp * C::COLS + j) * BP + quad * 32 + lane] = acc[j];
      }
    }
  }
  __syncwarp();
  if (S > 1) {
    // CTA `rank` finishes tokens [rank * TN / S, (rank + 1) * TN / S), a warp one of them at a time, a lane
    // four neighbouring channels of it. What the results are multiplied with is read before the wait.
    int tp, tq;
    tile_at(first, tp, tq);
    const int c0 = TN * rank / S, c1 = min(TN * (rank + 1) / S, p.M - tq * TN);
    const int n0 = tp * BP + lane * 4;
    float ws[4], bias[4], sx = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const Channel ch = channel_at(p, n0 + i);
      ws[i] = ch.scale;
      bias[i] = ch.bias;
    }
    if (c0 + warp < c1) sx = p.x_scale[tq * TN + c0 + warp];
    cluster_sync_all();
    for (int c = c0 + warp; c < c1; c += C::THREADS / 32) {
      float4 v[MAX_CLUSTER];
#pragma unroll
      for (int q = 0; q < MAX_CLUSTER; ++q)  // all loads in flight before the adds
        if (q < S) v[q] = ld_cluster4(base + (uint32_t)(c * BP + lane * 4) * 4, (uint32_t)q);
      int sums[4] = {};
#pragma unroll
      for (int q = 0; q < MAX_CLUSTER; ++q)
        if (q < S) {
          sums[0] += __float_as_int(v[q].x);
          sums[1] += __float_as_int(v[q].y);
          sums[2] += __float_as_int(v[q].z);
          sums[3] += __float_as_int(v[q].w);
        }
      // (a load that nothing waits for could still be under way when the other CTA leaves)
      asm volatile("" ::"r"(sums[0]), "r"(sums[1]), "r"(sums[2]), "r"(sums[3]));
      float y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] = fmaf((float)sums[i], ws[i] * sx, bias[i]);
      const int token = tq * TN + c, next = c + C::THREADS / 32;
      if (next < c1) sx = p.x_scale[tq * TN + next];
      const long long at = token * p.d.ld + n0;
      if (p.d.vec && n0 + 4 <= p.N) {
        if (p.d.type == OUT_F32)
          *reinterpret_cast<float4 *>(static_cast<float *>(p.d.ptr) + at) = make_float4(y[0], y[1], y[2], y[3]);
        else
          *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.d.ptr) + at) =
              make_uint2(pack_out(p.d.type, y[0], y[1]), pack_out(p.d.type, y[2], y[3]));
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (n0 + i < p.N) finish_out(p.d.ptr, p.d.type, at + i, y[i], p.d.beta);
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

// D = bias + beta * D (K == 0).
__global__ void i8_bias_kernel(int M, int N, const Result d) {
  griddep_wait();
  const long long total = (long long)M * N;
  for (long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x; i < total;
       i += (long long)gridDim.x * blockDim.x) {
    const int n = (int)(i % N);
    tcx::finish_out(d.ptr, d.type, i / N * d.ld + n, d.bias ? d.bias[n] : 0.0f, d.beta);
  }
}

// ------------------------------------------------------------------------------------
// Host side

struct Plan {
  int tn;              // tokens per tile; 0: few_kernel
  bool pair;           // two CTAs per tile
  int split;           // CTAs per tile, each with its part of k
};

// Estimated time of a plan in microseconds, fitted to times measured on GB300 with every plan forced on 128
// shapes (9 to 8192 rows, N and K of 512 to 14336): a call, each block of k, each round of tiles and a
// cluster's exchange. The estimate's choice is within 0.5% of the best plan on average, 14% at most.
struct Cost {
  int tn;
  bool pair;
  double call, block, round, exchange;
};
static const Cost kCosts[] = {{128, true, 5.30, 0.320, 1.87, 0.0}, {128, false, 4.89, 0.412, 1.12, 2.21},
                              {64, false, 2.58, 0.438, 0.69, 1.73}, {32, false, 2.86, 0.325, 0.25, 1.17},
                              {16, false, 2.28, 0.294, 0.22, 1.17}};

static Plan make_plan(int M, int N, int K, int sms) {
  if (M <= kFewRows) return {0, false, 1};
  const int KB = (int)ceil_div(K, BK);
  Plan best{128, false, 1};
  double best_cost = 1e300;
  for (const Cost &c : kCosts) {
    if (c.pair && sms < 2) continue;
    const long long tiles = ceil_div(N, c.pair ? 2 * BP : BP) * ceil_div(M, c.tn);
    const int at_once = c.pair ? sms / 2 : sms;
    for (int S = 1; S <= (c.pair ? 1 : MAX_CLUSTER); S *= 2) {
      // (clusters of 8 sit in one GPC each: more than about 12 of them do not run at once)
      if (S > 1 && (S > KB || tiles * S > (S == 8 ? std::min(96, sms) : sms))) break;
      const double cost = c.call + (double)ceil_div(tiles * S, at_once) * (c.block * ((KB + S - 1) / S) + c.round) +
                          (S > 1 ? c.exchange : 0.0);
      if (cost < best_cost) {
        best_cost = cost;
        best = {c.tn, c.pair, S};
      }
    }
  }
  return best;
}

template <int TN, bool PAIR = false>
static cudaError_t launch(const CUtensorMap &mp, const CUtensorMap &mq, const Params &p, int grid,
                          cudaStream_t stream) {
  using C = Cfg<TN, PAIR>;
  return launch_1d(i8_kernel<TN, PAIR>, grid, C::THREADS, C::SMEM_BYTES, PAIR ? 2 : p.split, stream, mp, mq, p);
}

template <int TN, bool PAIR = false>
static cudaError_t set_attributes() {
  using C = Cfg<TN, PAIR>;
  cudaError_t e = cudaFuncSetAttribute(i8_kernel<TN, PAIR>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES);
  if (e == cudaSuccess && PAIR) {
    // the registers that the warpgroups ask for must be there: what a launch brings is what the
    // compiler gave the kernel
    cudaFuncAttributes a;
    e = cudaFuncGetAttributes(&a, i8_kernel<TN, PAIR>);
    if (e == cudaSuccess && a.numRegs / 8 * 8 * C::THREADS < C::REGS)
      e = cudaErrorLaunchOutOfResources;
  }
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
    cudaError_t err = set_attributes<128, true>();
    if (err == cudaSuccess) err = set_attributes<128>();
    if (err == cudaSuccess) err = set_attributes<64>();
    if (err == cudaSuccess) err = set_attributes<32>();
    if (err == cudaSuccess) err = set_attributes<16>();
    g_err[dev] = err;
  });
  return g_err[dev];
}

static cudaError_t run(const Plan &pl, int M, int N, int K, const Operand &x, const Operand &w, const Result &d,
                       int sms, cudaStream_t stream) {
  Params p{};
  p.N = N;
  p.M = M;
  p.KB = (int)ceil_div(K, BK);
  p.w_scale = w.scale;
  p.x_scale = x.scale;
  p.d = d;
  const bool pair = pl.pair;
  const long long tiles_p = ceil_div(N, BP), tiles_q = ceil_div(M, pl.tn);
  if (tiles_p * tiles_q > 0x7fffffffLL / MAX_CLUSTER) return cudaErrorInvalidConfiguration;
  p.tiles_p = (int)tiles_p;
  p.tiles_q = (int)tiles_q;
  p.group_p = (int)std::min<long long>(pair ? 8 : 16, tiles_p);
  p.split = pl.split;
  // instruction descriptor: D in FP32 (bits 4-5 = 1), FP16 operands, k contiguous, N / 8 (bits 17-22),
  // M / 16 (24-28)
  p.idesc = (1u << 4) | ((uint32_t)(pl.tn >> 3) << 17) |
            ((uint32_t)((pair ? 2 * BP : BP) >> 4) << 24);
  CUtensorMap mp, mq;
  if (!encode_map_2d_narrow(&mp, w.q, 1, N, K, w.ld, BP)) return cudaErrorInvalidValue;
  char *ws = nullptr;
  cudaError_t e = cudaSuccess;
  if (pl.tn >= 128) {
    const long long ld = ceil_div(K, 16) * 16;
    e = cudaMallocFromPoolAsync(reinterpret_cast<void **>(&ws), (size_t)M * ld * 2, workspace_pool(), stream);
    if (e != cudaSuccess) return e;
    e = encode_map_2d_narrow(&mq, ws, 2, M, K, ld, pair ? pl.tn / 2 : pl.tn)
            ? launch_unpack(M, K, x, ws, ld, sms, stream)
            : cudaErrorInvalidValue;
  } else if (!encode_map_2d_narrow(&mq, x.q, 1, M, K, x.ld, pl.tn)) {
    return cudaErrorInvalidValue;
  }
  const int grid = (int)(pair ? 2 * std::min<long long>(ceil_div(tiles_p, 2) * tiles_q, sms / 2)
                         : p.split > 1 ? tiles_p * tiles_q * p.split
                                       : std::min<long long>(tiles_p * tiles_q, sms));
  if (e == cudaSuccess)
    switch (pl.tn) {
      case 128: e = pair ? launch<128, true>(mp, mq, p, grid, stream) : launch<128>(mp, mq, p, grid, stream); break;
      case 64: e = launch<64>(mp, mq, p, grid, stream); break;
      case 32: e = launch<32>(mp, mq, p, grid, stream); break;
      default: e = launch<16>(mp, mq, p, grid, stream);
    }
  if (ws != nullptr) {
    const cudaError_t ef = cudaFreeAsync(ws, stream);
    if (e == cudaSuccess) e = ef;
  }
  return e;
}

}  // namespace i8
}  // namespace sgemm

using namespace sgemm;

extern "C" int i8_linear(int M, int N, int K, const void *x, int ldx, const float *x_scale, const void *w,
                         int ldw, const float *w_scale, const float *bias, float beta, void *D, int d_type,
                         int ldd, cudaStream_t stream) {
  const bool read = M > 0 && N > 0 && K > 0;
  const auto bad_ptr = [](const void *q) { return (reinterpret_cast<uintptr_t>(q) & 15u) != 0; };
  const auto misplaced = [](const float *q) { return reinterpret_cast<uintptr_t>(q) % 4 != 0; };
  if (M < 0) return -1;
  if (N < 0) return -2;
  if (K < 0 || K > i8::LARGEST_K) return -3;
  if (read && (x == nullptr || bad_ptr(x))) return -4;
  if (ldx < std::max(1, K) || ldx % 16 != 0) return -5;
  if (read && (x_scale == nullptr || misplaced(x_scale))) return -6;
  if (read && (w == nullptr || bad_ptr(w))) return -7;
  if (ldw < std::max(1, K) || ldw % 16 != 0) return -8;
  if (read && (w_scale == nullptr || misplaced(w_scale))) return -9;
  if (misplaced(bias)) return -10;
  if (M > 0 && N > 0 && D == nullptr) return -12;
  if (d_type != I8_F32 && d_type != I8_BF16 && d_type != I8_F16) return -13;
  if (reinterpret_cast<uintptr_t>(D) % (d_type == I8_F32 ? 4 : 2) != 0) return -12;
  if (ldd < std::max(1, N)) return -14;
  if (M == 0 || N == 0) return 0;

  int sms = 0;
  cudaError_t e = device_setup(&sms);
  if (e == cudaSuccess) e = i8::kernel_setup();
  if (e != cudaSuccess) return (int)e;
  const bool vec = beta == 0.0f && !bad_ptr(D) && (M == 1 || (long long)ldd * (d_type == I8_F32 ? 4 : 2) % 16 == 0);
  const i8::Result d{D, d_type, ldd, bias, beta, vec};
  if (K == 0) {
    const long long blocks = std::min<long long>(ceil_div((long long)M * N, 256), 8LL * sms);
    return (int)launch_1d(i8::i8_bias_kernel, (int)blocks, 256, 0, 1, stream, M, N, d);
  }
  const i8::Operand ox{static_cast<const int8_t *>(x), ldx, x_scale}, ow{static_cast<const int8_t *>(w), ldw, w_scale};
  const i8::Plan pl = i8::make_plan(M, N, K, sms);
  if (pl.tn == 0) return (int)i8::launch_few(M, N, K, ox, ow, d, sms, stream);
  return (int)i8::run(pl, M, N, K, ox, ow, d, sms, stream);
}

extern "C" int i8_linear_with(const i8_linear_args *a) {
  if (a == nullptr) return -1;
  return i8_linear(a->M, a->N, a->K, a->x, a->ldx, a->x_scale, a->w, a->ldw, a->w_scale, a->bias, a->beta, a->D,
                   a->d_type, a->ldd, a->stream);
}

extern "C" int i8_linear_plan(int M, int N, int K, int num_sms, int *tile_tokens, int *tile_channels, int *split) {
  if (M < 1) return -1;
  if (N < 1) return -2;
  if (K < 1 || K > i8::LARGEST_K) return -3;
  if (num_sms < 0) return -4;
  int sms = num_sms;
  if (sms == 0 && device_setup(&sms) != cudaSuccess) {
    (void)cudaGetLastError();
    sms = 152;  // no device here: the answer for a whole GB300
  }
  const i8::Plan pl = i8::make_plan(M, N, K, sms);
  if (tile_tokens) *tile_tokens = pl.tn;
  if (tile_channels) *tile_channels = pl.tn == 0 ? 0 : pl.pair ? 2 * i8::BP : i8::BP;
  if (split) *split = pl.split;
  return 0;
}

extern "C" int i8_linear_status(int *status) {
  int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, i8::g_i8_status, sizeof(int));
  if (e != cudaSuccess) return (int)e;
  const int zero = 0;
  e = cudaMemcpyToSymbol(i8::g_i8_status, &zero, sizeof(int));
  if (status) *status = v;
  return (int)e;
}

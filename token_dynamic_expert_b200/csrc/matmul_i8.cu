// matmul_i8.cu -- matrix product in 8-bit integers with a scale for each token
// and each output channel, dense or grouped by expert, on Blackwell tensor
// cores (tcgen05 kind::i8, int32 accumulators in TMEM, operands by TMA).
//
//   out[s][n] = (slot_scale[s] x_scale[r] w_scale[e][n]) sum_k xq[r][k] wq[e][n][k]
//   r = row_of[s] (or s); e = the group of slot s by offsets (or 0)
//
// The integer sum is exact (|sum| <= 2^14 K < 2^31); it is rounded to fp32
// once, then scaled, then rounded to the output type.
//
// Weight rows sit on the MMA's M side, slots on N (16..256): experts get tens
// of slots while their matrices have hundreds of rows, and decode has a handful
// of slots against whole matrices.  A work item is (slot tile, block of weight
// rows); items of one expert run row block by row block with its tiles side by
// side, so that tiles after the first find the weights in L2.  The items of each
// expert follow from the offsets alone: every CTA scans them into shared memory
// as it starts, so no launch prepares a tile list.
//
// PAIR: a cluster of two CTAs works on one item (tcgen05 cta_group::2, 256
// weight rows): each holds 128 of the rows and half of the slots, so a slot row
// that a CTA loads feeds twice the MMA work.  Both CTAs' loads of a stage
// complete on the leader's barrier, its MMA thread issues for both and commits
// to both.  No TMA multicast.
//
//   warp 0       TMA producer: 128 x 128-byte boxes of weights, and of slot rows
//   warp 1       TMEM and the MMAs (one thread): four of K = 32 a stage
//   warps 2-9    epilogue: tcgen05.ld, scales, stores
//   warps 10-17  with row_of: four slot rows an instruction (tile::gather4).  A
//                warp issues these one thread at a time, about 75 cycles each, so
//                several warps share them (65536 gathered rows, 256 x 1024 x 2048:
//                2, 4, 8 warps 258, 205, 199 us, call after call)
// Two TMEM accumulators alternate between items, so an epilogue overlaps the
// next main loop.  All waits are bounded.
// A gather warp without rows in an item passes it over, and begins an item only
// once the weights' warp has: the ring's barriers tell one turn from the next, not
// from the one after.
#include <math.h>

#include <atomic>

#include "ace_common.cuh"
#include "ace_internal.h"
#include "compact.cuh"
#include "launch.cuh"

namespace ace {
namespace {

constexpr int kM = 128;            // weight rows a CTA holds
constexpr int kStepK = 128;        // bytes of K per stage: one swizzle row
constexpr int kWBytes = kM * kStepK;
constexpr int kMaxN = 256;         // slots per tile
constexpr int kStagesMax = 12;
constexpr int kStageRoom = 200 * 1024;
constexpr int kEpiWarps = 8;
constexpr int kGatherWarp = 2 + kEpiWarps;  // the first of them
constexpr int kGatherWarps = 8;
// the gather warps exist with row_of only
__host__ __device__ constexpr int threads_i8(bool gather) {
  return 32 * (kGatherWarp + (gather ? kGatherWarps : 0));
}
constexpr uint32_t kLeaderMask = 0xFEFFFFFFu;  // a barrier's address in the leader CTA
constexpr uint32_t kTmemI8 = 512;

struct MatArgs {
  const float* x_scale;
  const float* w_scale;
  const float* slot_scale;  // or NULL
  const int32_t* row_of;    // or NULL
  const int32_t* offsets;   // or NULL (dense)
  void* out;
  int64_t ldo;
  uint32_t* status;
  int S, E, N, K, n_rows, tile, box;  // tile, box: slots per tile, rows per TMA box
  bool pairs;                         // outputs can be stored two channels at a time
};

struct SmemI8 {
  int first[kMaxE + 1];  // first slot of each expert, then the slots in use
  int cum[kMaxE + 1];    // items of the experts before each
  alignas(16) float scale[kEpiWarps][kMaxN / 2];  // each epilogue warp's slots
  uint64_t full[kStagesMax], empty[kStagesMax], tfull[2], tempty[2], drain;
  int s_warp[32];
  uint32_t tmem;
  int abort_flag;
  int item;  // the last item the weights' warp has begun
};

__host__ __device__ constexpr uint32_t idesc_i8(int M, int N) {
  return (2u << 4)                       // D format int32
         | (1u << 7) | (1u << 10)        // A and B signed 8-bit
         | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

template <bool PAIR>
__device__ __forceinline__ void mma_i8(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc,
                                       uint32_t idesc, uint32_t accumulate) {
  if (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Arrive on `bar` (of both CTAs of a pair) once every MMA issued so far by this
// thread has completed.
template <bool PAIR>
__device__ __forceinline__ void commit_i8(uint64_t* bar) {
  if (PAIR)
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
        " [%0], %1;" ::"r"(smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
  else
    mma_commit(bar);
}

// Box at (x, y) of the matrix, to shared memory; of a pair, completing on the
// leader's barrier.
template <bool PAIR>
__device__ __forceinline__ void load_box(void* dst, const CUtensorMap* m, int x, int y,
                                         uint64_t* bar, uint64_t policy) {
  if (PAIR)
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar) & kLeaderMask), "r"(x), "r"(y),
        "l"(policy)
        : "memory");
  else
    tma_load_2d(dst, m, x, y, bar, policy);
}

// Four rows of the matrix at inner coordinate x, 128 bytes each, to four
// consecutive 128-byte rows of shared memory.
template <bool PAIR>
__device__ __forceinline__ void load_rows4(void* dst, const CUtensorMap* m, int x,
                                           const int (&y)[4], uint64_t* bar, uint64_t policy) {
  if (PAIR)
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile::gather4"
        ".mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4, %5, %6, %7}], [%2], %8;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar) & kLeaderMask), "r"(x), "r"(y[0]),
        "r"(y[1]), "r"(y[2]), "r"(y[3]), "l"(policy)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4"
        ".mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4, %5, %6, %7}], [%2], %8;" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(x), "r"(y[0]), "r"(y[1]),
        "r"(y[2]), "r"(y[3]), "l"(policy)
        : "memory");
}

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}

// 32 lanes x 32 bit, 32 consecutive columns per thread.
__device__ __forceinline__ void tmem_ld32i(uint32_t taddr, int (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, "
      "%20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

// Outputs of 32 slots (n of them in use) of one channel a lane: v holds the
// integer sums, scale the slots' factors, o the first slot's element of this
// lane's channel.
//   pairs (bf16, even N and ldo): neighbouring lanes exchange halves, so that
//   the even lane stores two channels of the even slot and the odd lane two of
//   the odd slot, in 4 bytes: half the stores
//   else one element a store
template <typename TO, bool FULL>
__device__ __forceinline__ void store_slots(const int (&v)[32], const float* scale, float wsc,
                                            TO* o, int64_t ldo, int n, bool in, bool pairs) {
  if (sizeof(TO) == 2 && pairs) {
    const bool odd = threadIdx.x & 1;
    uint32_t* p = reinterpret_cast<uint32_t*>(o + (odd ? ldo - 1 : 0));
#pragma unroll
    for (int c = 0; c < 32; c += 4) {
      const float4 s = *reinterpret_cast<const float4*>(scale + c);
      const float f[4] = {(float)v[c] * (s.x * wsc), (float)v[c + 1] * (s.y * wsc),
                          (float)v[c + 2] * (s.z * wsc), (float)v[c + 3] * (s.w * wsc)};
#pragma unroll
      for (int h = 0; h < 4; h += 2) {
        uint32_t mine;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(mine) : "f"(f[h + 1]), "f"(f[h]));
        const uint32_t other = __shfl_xor_sync(0xffffffffu, mine, 1);
        const uint32_t two = odd ? __byte_perm(other, mine, 0x7632) : __byte_perm(mine, other, 0x5410);
        if (in && (FULL || c + h + (odd ? 1 : 0) < n)) *p = two;
        p += ldo;  // two slots of ldo elements, in units of two elements
      }
    }
  } else if (in) {
#pragma unroll
    for (int c = 0; c < 32; ++c) {
      if (FULL || c < n) *o = from_f<TO>((float)v[c] * (scale[c] * wsc));
      o += ldo;
    }
  }
}

// Slots per tile of an expert of cnt slots: near-equal, multiples of the MMA's
// step of N (16; 32 for a pair).
template <bool PAIR>
__device__ __forceinline__ int tile_rows(int cnt, int ntile) {
  constexpr int q = PAIR ? 32 : 16;
  return ((cnt + ntile - 1) / ntile + q - 1) / q * q;
}

struct Item {
  int e, row0, n, blk;  // expert, first slot, slots, block of weight rows
  // slots each CTA of a pair holds (n for a CTA on its own, up to a step of N)
  template <bool PAIR>
  __device__ __forceinline__ int half() const {
    return PAIR ? (n + 31) / 32 * 16 : (n + 15) / 16 * 16;
  }
  // groups of four slots that CTA `rank` gathers
  template <bool PAIR>
  __device__ __forceinline__ int groups(int rank) const {
    const int h = half<PAIR>(), left = n - rank * h;
    return (max(0, min(left, h)) + 3) / 4;
  }
};

template <bool PAIR>
__device__ __forceinline__ Item item_at(const SmemI8& sm, const MatArgs& A, int nblk, int w) {
  int lo = 0, hi = A.E - 1;  // the expert whose items hold w
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (sm.cum[mid] <= w)
      lo = mid;
    else
      hi = mid - 1;
  }
  const int l = w - sm.cum[lo], ntile = max(1, (sm.cum[lo + 1] - sm.cum[lo]) / nblk);
  const int cnt = sm.first[lo + 1] - sm.first[lo];
  const int each = tile_rows<PAIR>(cnt, ntile), q = l % ntile;
  return {lo, sm.first[lo] + q * each, max(0, min(each, cnt - q * each)), l / ntile};
}

// Bounded wait until the weights' warp has begun item w.
__device__ __forceinline__ bool wait_item(const SmemI8& sm, int w, uint32_t* status,
                                          volatile int* abort_flag) {
  const volatile int* item = &sm.item;
  if (*item < w) {
    const uint64_t t0 = global_ns();
    while (*item < w) {
      if (*abort_flag) return false;
      if (global_ns() - t0 > kWaitLimitNs) {
        *abort_flag = 1;
        raise_flag(status, ACE_FLAG_TIMEOUT);
        return false;
      }
    }
  }
  __threadfence_block();
  return true;
}

// GATHER: the slots' rows come through row_of.
template <typename TO, bool PAIR, bool GATHER>
__global__ void __launch_bounds__(threads_i8(GATHER), 1)
    k_matmul_i8(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                const MatArgs A) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ SmemI8 sm;
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int warp = (int)warp_id(), lane = (int)lane_id(), tid = threadIdx.x;
  volatile int* abort_flag = &sm.abort_flag;
  constexpr int kRows = PAIR ? 2 * kM : kM;  // weight rows per item
  uint32_t rank = 0;
  if (PAIR) asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  const bool leader = rank == 0;
  const int w0 = PAIR ? (int)(blockIdx.x >> 1) : (int)blockIdx.x;  // first item, then every nw-th
  const int nw = PAIR ? (int)(gridDim.x >> 1) : (int)gridDim.x;
  const int nblk = (A.N + kRows - 1) / kRows, ksteps = (A.K + kStepK - 1) / kStepK;
  const int stage_bytes = kWBytes + A.tile / (PAIR ? 2 : 1) * kStepK;
  const int NS = min(kStagesMax, kStageRoom / stage_bytes);

  if (tid == 0) {
    for (int s = 0; s < kStagesMax; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&sm.tfull[a], 1);
      mbar_init(&sm.tempty[a], (PAIR ? 2 : 1) * kEpiWarps);
    }
    mbar_init(&sm.drain, 1);
    sm.abort_flag = 0;
    sm.item = -1;
    fence_barrier_init();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX);
  }
  if (warp == 1) {
    if (PAIR) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                       smem_u32(&sm.tmem)),
                   "r"(kTmemI8)
                   : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      tmem_alloc(&sm.tmem, kTmemI8);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  if (PAIR)
    cluster_barrier();  // both CTAs' barriers exist before either signals the other
  else
    __syncthreads();
  tc_fence_after();
  begin_overlapped();
  // the experts' slots and items, two experts a thread
  int total;
  {
    int first[2], items[2] = {0, 0};
    const int last = A.offsets ? A.offsets[A.E] : A.S;
    bool bad = last < 0 || last > A.S || (A.offsets && A.offsets[0] != 0);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int e = 2 * tid + j;
      if (e >= A.E) continue;
      first[j] = A.offsets ? A.offsets[e] : 0;
      const int end = A.offsets ? A.offsets[e + 1] : A.S;
      bad |= first[j] < 0 || end < first[j] || end > last;
      items[j] = (end - first[j] + A.tile - 1) / A.tile * nblk;
    }
    bad = __syncthreads_or(bad) != 0;
    if (bad) items[0] = items[1] = 0;  // offsets that do not rise from 0 to at most S: nothing runs
    const int before = block_excl_scan(items[0] + items[1], sm.s_warp, &total);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int e = 2 * tid + j;
      if (e >= A.E) continue;
      sm.first[e] = first[j];
      sm.cum[e] = before + (j ? items[0] : 0);
    }
    if (tid == 0) {
      sm.cum[A.E] = total;
      // The call's status word.  Only a wait that ran out raises another flag,
      // seconds after this CTA, the grid's first, has written.
      if (blockIdx.x == 0) *A.status = bad ? ACE_FLAG_BAD_INDEX : 0u;
      sm.first[A.E] = last;
    }
  }
  __syncthreads();
  const uint32_t tmem = sm.tmem;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    const uint64_t pol_w = policy_evict_first(), pol_x = policy_evict_last();
    int stage = 0;
    uint32_t phase = 0;
    for (int w = w0; w < total && !*abort_flag; w += nw) {
      if (GATHER && lane == 0) {
        __threadfence_block();
        *static_cast<volatile int*>(&sm.item) = w;
      }
      const Item it = item_at<PAIR>(sm, A, nblk, w);
      const int half = it.half<PAIR>(), row = it.row0 + (int)rank * half;
      const int nbox = (half + A.box - 1) / A.box;
      // the bytes that complete on this CTA's barrier: of a pair, both CTAs' on
      // the leader's
      uint32_t bytes = (PAIR ? 2u : 1u) * kWBytes;
      if (!GATHER)
        bytes += (PAIR ? 2u : 1u) * (uint32_t)(nbox * A.box * kStepK);
      else
        bytes += (uint32_t)(it.groups<PAIR>(0) + (PAIR ? it.groups<PAIR>(1) : 0)) * 4 * kStepK;
      for (int kb = 0; kb < ksteps; ++kb) {
        if (!mbar_wait(&sm.empty[stage], phase ^ 1u, A.status, abort_flag)) break;
        __syncwarp();
        uint8_t* sw = smem + stage * stage_bytes;
        if (lane == 0) {
          if (leader) mbar_expect_tx(&sm.full[stage], bytes);
          load_box<PAIR>(sw, &tmW, kb * kStepK, it.e * A.N + it.blk * kRows + (int)rank * kM,
                         &sm.full[stage], pol_w);
        }
        __syncwarp();
        if (!GATHER && lane < nbox)
          load_box<PAIR>(sw + kWBytes + lane * A.box * kStepK, &tmX, kb * kStepK,
                         row + lane * A.box, &sm.full[stage], pol_x);
        if (++stage == NS) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
  } else if (warp >= kGatherWarp) {
    // ------------------------------------------------- slot rows through row_of
    if constexpr (GATHER) {
      const uint64_t pol_x = policy_evict_last();
      constexpr int kPer = kMaxN / 4 / kGatherWarps / (PAIR ? 2 : 1);  // groups a warp
      const int g = (warp - kGatherWarp) * kPer + lane;
      int stage = 0;
      uint32_t phase = 0;
      for (int w = w0; w < total && !*abort_flag; w += nw) {
        const Item it = item_at<PAIR>(sm, A, nblk, w);
        const int ng = it.groups<PAIR>((int)rank);
        const bool mine = lane < kPer && g < ng;
        if (g - lane >= ng) {  // the same for the warp
          const int next = stage + ksteps;
          phase ^= (uint32_t)(next / NS) & 1u;
          stage = next % NS;
          continue;
        }
        if (!wait_item(sm, w, A.status, abort_flag)) break;
        int rows[4] = {0, 0, 0, 0};
        if (mine)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int c = (int)rank * it.half<PAIR>() + 4 * g + j;
            const int r = c < it.n ? A.row_of[it.row0 + c] : 0;
            rows[j] = r >= 0 && r < A.n_rows ? r : 0;  // the scale makes such a slot 0
          }
        for (int kb = 0; kb < ksteps; ++kb) {
          if (!mbar_wait(&sm.empty[stage], phase ^ 1u, A.status, abort_flag)) break;
          __syncwarp();
          if (mine)
            load_rows4<PAIR>(smem + stage * stage_bytes + kWBytes + g * 4 * kStepK, &tmX,
                             kb * kStepK, rows, &sm.full[stage], pol_x);
          if (++stage == NS) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    if (leader && lane == 0) {
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int w = w0; w < total && ok; w += nw) {
        const Item it = item_at<PAIR>(sm, A, nblk, w);
        const uint32_t idesc = idesc_i8(kRows, it.half<PAIR>() * (PAIR ? 2 : 1));
        if (!mbar_wait(&sm.tempty[acc], acc_phase ^ 1u, A.status, abort_flag)) break;
        tc_fence_after();
        const uint32_t d0 = tmem + (uint32_t)acc * 256u;
        for (int kb = 0; kb < ksteps; ++kb) {
          if (!mbar_wait(&sm.full[stage], phase, A.status, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a0 = smem_u32(smem + stage * stage_bytes), b0 = a0 + kWBytes;
#pragma unroll
          for (int kk = 0; kk < kStepK / 32; ++kk)
            mma_i8<PAIR>(d0, sw128_kmajor_desc(a0 + kk * 32), sw128_kmajor_desc(b0 + kk * 32), idesc,
                   (kb | kk) != 0);
          commit_i8<PAIR>(&sm.empty[stage]);
          if (++stage == NS) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        commit_i8<PAIR>(&sm.tfull[acc]);
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
      // every MMA issued has completed before TMEM is freed
      if (PAIR)
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                smem_u32(&sm.drain))
            : "memory");
      else
        mma_commit(&sm.drain);
      mbar_drain(&sm.drain, 0);
    }
  } else if (warp < kGatherWarp) {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3, part = (warp - 2) >> 2;  // TMEM lane quarter; every other 32 slots
    int acc = 0;
    uint32_t acc_phase = 0;
    TO* out = static_cast<TO*>(A.out);
    float* scale = sm.scale[warp - 2];
    for (int w = w0; w < total; w += nw) {
      const Item it = item_at<PAIR>(sm, A, nblk, w);
      // the factors of the slots this warp will store, ahead of the wait
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kMaxN / 64; ++i) {
        const int c = part * 32 + i * 64 + lane, s = it.row0 + c;
        float f = 0.f;
        if (c < it.n) {
          const int r = GATHER ? A.row_of[s] : s;
          if (r >= 0 && r < A.n_rows) f = A.x_scale[r] * (A.slot_scale ? A.slot_scale[s] : 1.f);
        }
        scale[i * 32 + lane] = f;
      }
      __syncwarp();
      const int col = it.blk * kRows + (int)rank * kM + q * 32 + lane;
      const float wsc = col < A.N ? A.w_scale[(size_t)it.e * A.N + col] : 0.f;
      if (!mbar_wait(&sm.tfull[acc], acc_phase, A.status, abort_flag)) break;
      tc_fence_after();
      const uint32_t tbase = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)acc * 256u;
      for (int c0 = part * 32; c0 < it.n; c0 += 64) {
        int v[32];
        tmem_ld32i(tbase + (uint32_t)c0, v);
        tmem_ld_wait();
        TO* o = out + (size_t)(it.row0 + c0) * A.ldo + col;
        if (c0 + 32 <= it.n)
          store_slots<TO, true>(v, scale + c0 / 64 * 32, wsc, o, A.ldo, 32, col < A.N, A.pairs);
        else
          store_slots<TO, false>(v, scale + c0 / 64 * 32, wsc, o, A.ldo, it.n - c0, col < A.N, A.pairs);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (PAIR)
          // orders TMEM reads alone; a release at cluster scope would wait for the
          // warp's output stores, a microsecond an item
          asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(
                           smem_u32(&sm.tempty[acc]) & kLeaderMask)
                       : "memory");
        else
          mbar_arrive(&sm.tempty[acc]);
      }
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
  }
  __syncthreads();
  if (*abort_flag) {
    // a wait ran out somewhere: copies this CTA started may still be landing,
    // so give them time before shared memory is given up
    if (tid == 0) {
      const uint64_t t0 = global_ns();
      while (global_ns() - t0 < 100000ull) {
      }
    }
    __syncthreads();
  }
  tc_fence_before();
  if (PAIR)
    cluster_barrier();  // both CTAs are done with TMEM and with each other's barriers
  else
    __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    if (PAIR)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                   "r"(kTmemI8)
                   : "memory");
    else
      tmem_dealloc(tmem, kTmemI8);
  }
}

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static std::atomic<EncodeTiled> fn{nullptr};
  EncodeTiled f = fn.load(std::memory_order_acquire);
  if (!f) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      f = reinterpret_cast<EncodeTiled>(p);
    fn.store(f, std::memory_order_release);
  }
  return f;
}

// int8 matrix of rows x cols, ld bytes a row: boxes of box_rows x 128 bytes,
// 128-byte swizzle, zeros outside.
bool map_i8(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols, uint64_t ld,
            uint32_t box_rows) {
  EncodeTiled fn = encode_tiled();
  if (!fn) return false;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {ld};
  cuuint32_t box[2] = {(cuuint32_t)kStepK, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename TO, bool PAIR, bool GATHER>
cudaError_t launch_form(const CUtensorMap& w, const CUtensorMap& x, const MatArgs& A, int grid,
                       cudaStream_t s) {
  const size_t smem = 1024 + kStageRoom;
  const cudaError_t e = cudaFuncSetAttribute(
      k_matmul_i8<TO, PAIR, GATHER>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  return launch_overlapped(k_matmul_i8<TO, PAIR, GATHER>, grid, threads_i8(GATHER), PAIR ? 2 : 1,
                           smem, s, w, x, A);
}

template <typename TO>
cudaError_t launch_mat(const CUtensorMap& w, const CUtensorMap& x, const MatArgs& A, bool pair,
                       int grid, cudaStream_t s) {
  if (A.row_of)
    return pair ? launch_form<TO, true, true>(w, x, A, grid, s)
                : launch_form<TO, false, true>(w, x, A, grid, s);
  return pair ? launch_form<TO, true, false>(w, x, A, grid, s)
              : launch_form<TO, false, false>(w, x, A, grid, s);
}

bool is_aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace
}  // namespace ace

using namespace ace;

extern "C" {

ace_status ace_matmul_i8(const ace_i8_product* p, int S, void* out, int64_t ldo,
                         ace_dtype out_dtype, void* ws, size_t ws_bytes, void* stream) {
  if (!p || S < 0 || p->N < 1 || p->K < 1 || p->E < 1 || p->n_rows < 0) return ACE_ERR_INVALID_ARG;
  if (out_dtype != ACE_BF16 && out_dtype != ACE_F32) return ACE_ERR_INVALID_ARG;
  if (p->E > kMaxE || p->K % 16 != 0 || p->K > 65536) return ACE_ERR_UNSUPPORTED;
  if ((int64_t)p->E * p->N > kMaxCount || S > kMaxCount || p->n_rows > kMaxCount)
    return ACE_ERR_UNSUPPORTED;
  if (p->E > 1 && !p->offsets) return ACE_ERR_INVALID_ARG;
  if (!p->row_of && p->n_rows < S) return ACE_ERR_INVALID_ARG;
  if (!ws || !is_aligned(ws, 256) || ws_bytes < 256) return ACE_ERR_WORKSPACE;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (S == 0 || p->n_rows == 0) {
    if (S > 0) return ACE_ERR_INVALID_ARG;
    return cuda_status(launch_clear_words(ws, 1, s));
  }
  const size_t es = out_dtype == ACE_BF16 ? 2 : 4;
  if (!p->xq || !p->x_scale || !p->wq || !p->w_scale || !out || !is_aligned(p->xq, 16) ||
      !is_aligned(p->wq, 16) || !is_aligned(p->x_scale, 4) || !is_aligned(p->w_scale, 4) ||
      !is_aligned(p->slot_scale, 4) || !is_aligned(p->row_of, 4) || !is_aligned(p->offsets, 4) ||
      !is_aligned(out, es))
    return ACE_ERR_INVALID_ARG;
  if (p->ldx < p->K || p->ldx % 16 != 0 || ldo < p->N) return ACE_ERR_INVALID_ARG;
  const int64_t EN = (int64_t)p->E * p->N;
  // the output and the status word are written, the rest is read
  const ByteSpan o(out, ldo, S, p->N, es), status(ws, 1, 256, 1, 1);
  const ByteSpan in[7] = {ByteSpan(p->xq, p->ldx, p->n_rows, p->K, 1),
                          ByteSpan(p->wq, p->K, EN, p->K, 1),
                          ByteSpan(p->x_scale, 1, p->n_rows, 1, 4),
                          ByteSpan(p->w_scale, 1, EN, 1, 4),
                          ByteSpan(p->slot_scale, 1, S, 1, 4),
                          ByteSpan(p->row_of, 1, S, 1, 4),
                          ByteSpan(p->offsets, 1, p->E + 1, 1, 4)};
  for (const ByteSpan& i : in)
    if (o.meets(i) || status.meets(i)) return ACE_ERR_INVALID_ARG;
  if (o.meets(status)) return ACE_ERR_INVALID_ARG;
  MatArgs A;
  A.x_scale = p->x_scale;
  A.w_scale = p->w_scale;
  A.slot_scale = p->slot_scale;
  A.row_of = p->row_of;
  A.offsets = p->offsets;
  A.out = out;
  A.ldo = ldo;
  A.status = static_cast<uint32_t*>(ws);
  A.S = S;
  A.E = p->E;
  A.N = p->N;
  A.K = p->K;
  A.n_rows = p->n_rows;
  A.pairs = out_dtype == ACE_BF16 && p->N % 2 == 0 && ldo % 2 == 0 && is_aligned(out, 4);
  const int sms = device_sm_count();
  // Slots per tile, and whether pairs of CTAs work on it.
  //   grouped: the largest tile that still gives every SM an item if experts were
  //   full; tiles follow the experts' sizes below it.  Pairs from 64 slots on.
  //   dense: the least rounds x rows loaded per item (16 for what an item costs
  //   besides), as loads bound the kernel: 1500 and 512 slots of 2048 x 2048 take
  //   12.4 and 10.5 us, with the grouped rule 16.7 and 14.4.
  bool pair = false;
  if (p->offsets) {
    A.tile = kMaxN;
    while (A.tile > 16 && (int64_t)cdiv(S, A.tile) * cdiv(p->N, kM) < sms) A.tile /= 2;
    pair = A.tile >= 64 && p->N > kM;
  } else {
    int64_t best = INT64_MAX;
    for (int t = 16; t <= kMaxN; t *= 2)
      for (int two = 0; two <= (t >= 64 && p->N > kM ? 1 : 0); ++two) {
        const int units = two ? sms / 2 : sms;
        const int64_t items = (int64_t)cdiv(S, t) * cdiv(p->N, two ? 2 * kM : kM);
        const int64_t cost = (items + units - 1) / units * (kM + (two ? t / 2 : t) + 16);
        if (cost < best) {
          best = cost;
          A.tile = t;
          pair = two != 0;
        }
      }
  }
  A.box = pair ? 32 : A.tile < 64 ? A.tile : 64;
  // even slots give cdiv(S, tile) + E tiles at most
  const int64_t items = ((int64_t)cdiv(S, A.tile) + (p->offsets ? p->E : 0)) *
                        cdiv(p->N, pair ? 2 * kM : kM);
  if (items > 0x3fffffff) return ACE_ERR_UNSUPPORTED;
  CUtensorMap tw, tx;
  if (!map_i8(&tw, p->wq, (uint64_t)p->E * p->N, p->K, p->K, kM) ||
      !map_i8(&tx, p->xq, p->n_rows, p->K, p->ldx, p->row_of ? 1 : A.box))
    return cuda_status(cudaErrorInvalidValue);
  const int ctas = pair ? 2 * (int)(items < sms / 2 ? items : sms / 2)
                        : (int)(items < sms ? items : sms);
  return cuda_status(out_dtype == ACE_BF16 ? launch_mat<__nv_bfloat16>(tw, tx, A, pair, ctas, s)
                                           : launch_mat<float>(tw, tx, A, pair, ctas, s));
}

}  // extern "C"

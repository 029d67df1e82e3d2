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
// Weight rows sit on the MMA's M side (128), slots on N (16..256): experts get
// tens of slots while their matrices have hundreds of rows, and decode has a
// handful of slots against whole matrices.  A work item is (slot tile, block of
// 128 weight rows); items of one expert run row block by row block with its
// tiles side by side, so that tiles after the first find the weights in L2.
// The items of each expert follow from the offsets alone: every CTA scans them
// into shared memory as it starts, so no launch prepares a tile list.
//
//   warp 0    TMA producer: 128 x 128-byte boxes of weights; slot rows as
//             boxes, or four rows an instruction (tile::gather4) through row_of
//   warp 1    TMEM and the MMAs (one thread): four of K = 32 a stage
//   warps 2-9 epilogue: tcgen05.ld, scales, stores
// Two TMEM accumulators alternate between items, so an epilogue overlaps the
// next main loop.  All waits are bounded.
#include <math.h>

#include <atomic>

#include "ace_common.cuh"
#include "ace_internal.h"
#include "compact.cuh"

namespace ace {
namespace {

constexpr int kM = 128;            // weight rows per item
constexpr int kStepK = 128;        // bytes of K per stage: one swizzle row
constexpr int kWBytes = kM * kStepK;
constexpr int kMaxN = 256;         // slots per tile
constexpr int kStagesMax = 12;
constexpr int kStageRoom = 200 * 1024;
constexpr int kEpiWarps = 8;
constexpr int kThreadsI8 = 64 + 32 * kEpiWarps;
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
  int S, E, N, K, n_rows, tile, box;
};

struct SmemI8 {
  int first[kMaxE + 1];  // first slot of each expert, then the slots in use
  int cum[kMaxE + 1];    // items of the experts before each
  float scale[2][kMaxN];
  uint64_t full[kStagesMax], empty[kStagesMax], tfull[2], tempty[2], drain;
  int s_warp[32];
  uint32_t tmem;
  int abort_flag;
};

__host__ __device__ constexpr uint32_t idesc_i8(int M, int N) {
  return (2u << 4)                       // D format int32
         | (1u << 7) | (1u << 10)        // A and B signed 8-bit
         | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void mma_i8(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Four rows (y0..y3) of the matrix at inner coordinate x, 128 bytes each, to
// four consecutive 128-byte rows of shared memory.
__device__ __forceinline__ void tma_gather4(void* smem_dst, const CUtensorMap* m, int x, int y0,
                                            int y1, int y2, int y3, uint64_t* bar,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%3, %4, %5, %6, %7}], [%2], %8;" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(x), "r"(y0), "r"(y1), "r"(y2),
      "r"(y3), "l"(policy)
      : "memory");
}

__device__ __forceinline__ void tmem_ld16i(uint32_t taddr, int (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// Slots per tile of an expert of cnt slots: near-equal, multiples of 16.
__device__ __forceinline__ int tile_rows(int cnt, int ntile) {
  return ((cnt + ntile - 1) / ntile + 15) & ~15;
}

struct Item {
  int e, row0, n, blk;
};

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
  const int each = tile_rows(cnt, ntile), q = l % ntile;
  return {lo, sm.first[lo] + q * each, max(0, min(each, cnt - q * each)), l / ntile};
}

template <typename TO>
__global__ void __launch_bounds__(kThreadsI8, 1)
    k_matmul_i8(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                const MatArgs A) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ SmemI8 sm;
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int warp = (int)warp_id(), lane = (int)lane_id(), tid = threadIdx.x;
  volatile int* abort_flag = &sm.abort_flag;
  const int nblk = (A.N + kM - 1) / kM, ksteps = (A.K + kStepK - 1) / kStepK;
  const int stage_bytes = kWBytes + A.tile * kStepK;
  const int NS = min(kStagesMax, kStageRoom / stage_bytes);

  if (tid == 0) {
    for (int s = 0; s < kStagesMax; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&sm.tfull[a], 1);
      mbar_init(&sm.tempty[a], 32 * kEpiWarps);
    }
    mbar_init(&sm.drain, 1);
    sm.abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX);
  }
  if (warp == 1) {
    tmem_alloc(&sm.tmem, kTmemI8);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
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
    uint32_t phase = 0, issued = 0, issued_par = 0;
    for (int w = blockIdx.x; w < total && !*abort_flag; w += gridDim.x) {
      const Item it = item_at(sm, A, nblk, w);
      int rows[2][4];  // gather: rows of slots 4 (lane + 32 h) ..
      const int ng = (it.n + 3) / 4, nbox = (it.n + A.box - 1) / A.box;
      if (A.row_of) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int c = 4 * (lane + 32 * h) + j;
            const int r = c < it.n ? A.row_of[it.row0 + c] : 0;
            rows[h][j] = r >= 0 && r < A.n_rows ? r : 0;  // the scale makes such a slot 0
          }
      }
      const uint32_t bytes =
          kWBytes + (A.row_of ? ng * 4 * kStepK : nbox * A.box * kStepK);
      for (int kb = 0; kb < ksteps; ++kb) {
        if (!mbar_wait(&sm.empty[stage], phase ^ 1u, A.status, abort_flag)) break;
        __syncwarp();
        uint8_t* sw = smem + stage * stage_bytes;
        uint8_t* sx = sw + kWBytes;
        if (lane == 0) {
          mbar_expect_tx(&sm.full[stage], bytes);
          tma_load_2d(sw, &tmW, kb * kStepK, it.e * A.N + it.blk * kM, &sm.full[stage], pol_w);
        }
        __syncwarp();
        if (A.row_of) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (lane + 32 * h < ng)
              tma_gather4(sx + (lane + 32 * h) * 4 * kStepK, &tmX, kb * kStepK, rows[h][0],
                          rows[h][1], rows[h][2], rows[h][3], &sm.full[stage], pol_x);
        } else if (lane < nbox) {
          tma_load_2d(sx + lane * A.box * kStepK, &tmX, kb * kStepK, it.row0 + lane * A.box,
                      &sm.full[stage], pol_x);
        }
        issued |= 1u << stage;
        issued_par = (issued_par & ~(1u << stage)) | (phase << stage);
        if (++stage == NS) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    __syncwarp();
    if (*abort_flag)  // let every copy this warp started land
      for (int s = 0; s < NS; ++s)
        if ((issued >> s) & 1u) mbar_drain(&sm.full[s], (issued_par >> s) & 1u);
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    if (lane == 0) {
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int w = blockIdx.x; w < total && ok; w += gridDim.x) {
        const Item it = item_at(sm, A, nblk, w);
        const uint32_t idesc = idesc_i8(kM, (max(it.n, 1) + 15) & ~15);
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
            mma_i8(d0, sw128_kmajor_desc(a0 + kk * 32), sw128_kmajor_desc(b0 + kk * 32), idesc,
                   (kb | kk) != 0);
          mma_commit(&sm.empty[stage]);
          if (++stage == NS) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        mma_commit(&sm.tfull[acc]);
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
      mma_commit(&sm.drain);  // every MMA issued has completed before TMEM is freed
      mbar_drain(&sm.drain, 0);
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3, half = (warp - 2) >> 2;  // TMEM lane quarter; 16-slot groups taken
    const int et = tid - 64;
    int acc = 0;
    uint32_t acc_phase = 0;
    TO* out = static_cast<TO*>(A.out);
    for (int w = blockIdx.x; w < total; w += gridDim.x) {
      const Item it = item_at(sm, A, nblk, w);
      // the tile's token scales, one thread a slot (the buffer's last readers
      // passed the previous item's barrier)
      float sc = 0.f;
      if (et < it.n) {
        const int s = it.row0 + et;
        const int r = A.row_of ? A.row_of[s] : s;
        if (r >= 0 && r < A.n_rows) sc = A.x_scale[r] * (A.slot_scale ? A.slot_scale[s] : 1.f);
      }
      sm.scale[acc][et] = sc;
      const int col = it.blk * kM + q * 32 + lane;
      const float wsc = col < A.N ? A.w_scale[(size_t)it.e * A.N + col] : 0.f;
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if (!mbar_wait(&sm.tfull[acc], acc_phase, A.status, abort_flag)) break;
      tc_fence_after();
      const uint32_t tbase = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)acc * 256u;
      for (int c0 = half * 16; c0 < it.n; c0 += 32) {
        int v[16];
        tmem_ld16i(tbase + (uint32_t)c0, v);
        tmem_ld_wait();
        if (col < A.N) {
          TO* o = out + (size_t)(it.row0 + c0) * A.ldo + col;
#pragma unroll
          for (int c = 0; c < 16; ++c)
            if (c0 + c < it.n)
              o[(size_t)c * A.ldo] = from_f<TO>((float)v[c] * (sm.scale[acc][c0 + c] * wsc));
        }
      }
      tc_fence_before();
      mbar_arrive(&sm.tempty[acc]);
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
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

template <typename TO>
cudaError_t launch_mat(const CUtensorMap& w, const CUtensorMap& x, const MatArgs& A, int grid,
                       cudaStream_t s) {
  const int smem = 1024 + kStageRoom;
  cudaError_t e = cudaFuncSetAttribute(k_matmul_i8<TO>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       smem);
  if (e != cudaSuccess) return e;
  k_matmul_i8<TO><<<grid, kThreadsI8, smem, s>>>(w, x, A);
  return cudaGetLastError();
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
  if ((int64_t)p->E * p->N > 0x7fffff00) return ACE_ERR_UNSUPPORTED;
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
  const ByteSpan o(out, ldo, S, p->N, es);
  if (o.meets(ByteSpan(p->xq, p->ldx, p->n_rows, p->K, 1)) ||
      o.meets(ByteSpan(p->wq, p->K, EN, p->K, 1)) ||
      o.meets(ByteSpan(p->x_scale, 1, p->n_rows, 1, 4)) ||
      o.meets(ByteSpan(p->w_scale, 1, EN, 1, 4)) ||
      o.meets(ByteSpan(p->slot_scale, 1, S, 1, 4)) || o.meets(ByteSpan(p->row_of, 1, S, 1, 4)) ||
      o.meets(ByteSpan(p->offsets, 1, p->E + 1, 1, 4)) || o.meets(ByteSpan(ws, 1, 256, 1, 1)))
    return ACE_ERR_INVALID_ARG;
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
  const int sms = device_sm_count(), nblk = cdiv(p->N, kM);
  // the largest tile that still gives every SM an item
  A.tile = kMaxN;
  while (A.tile > 16 && (int64_t)cdiv(S, A.tile) * nblk < sms) A.tile /= 2;
  A.box = A.tile < 64 ? A.tile : 64;
  // items of even slots: cdiv(S, tile) + E tiles at most
  const int64_t items = ((int64_t)cdiv(S, A.tile) + (p->offsets ? p->E : 0)) * nblk;
  if (items > 0x3fffffff) return ACE_ERR_UNSUPPORTED;
  CUtensorMap tw, tx;
  if (!map_i8(&tw, p->wq, (uint64_t)p->E * p->N, p->K, p->K, kM) ||
      !map_i8(&tx, p->xq, p->n_rows, p->K, p->ldx, p->row_of ? 1 : A.box))
    return cuda_status(cudaErrorInvalidValue);
  const int grid = items < sms ? (int)items : sms;
  return cuda_status(out_dtype == ACE_BF16 ? launch_mat<__nv_bfloat16>(tw, tx, A, grid, s)
                                           : launch_mat<float>(tw, tx, A, grid, s));
}

}  // extern "C"

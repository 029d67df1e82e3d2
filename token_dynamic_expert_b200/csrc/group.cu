// group.cu -- kept slots grouped by expert: the counting sort between the
// gate and the experts' products.
//
//   slots s = t k + i with keep (and a valid expert) go to positions in the
//   order (expert, token, rank); offsets[e] = first position of expert e,
//   offsets[E] = their number.
//
// One launch: a cluster of 1, 8 or 16 CTAs; every warp has a run of consecutive
// chunks of 32 tokens.  Warps count their runs per expert in their own rows of
// shared memory; a prefix over warps, over the cluster's CTAs (distributed shared
// memory) and over experts gives each (warp, expert) its first position.  Then, a
// chunk at a time, every slot sets its token's bit in the warp's word of its
// expert, and the bits below its own are the slots ahead of it.  A token that
// names an expert twice (no gate does) would lose a slot that way; such a chunk
// is ranked by match.any instead, which for every chunk would cost more than all
// the rest (28 us against 17.8 on 8 SMs at 8192 tokens).  Atomics only add and set
// bits in shared memory, so the order never varies; no global scratch, so nothing
// needs clearing.  Bound by latency, and by the scattered 4-byte stores.
#include <cooperative_groups.h>

#include <atomic>

#include "ace_common.cuh"
#include "ace_internal.h"
#include "compact.cuh"
#include "launch.cuh"

namespace cg = cooperative_groups;

namespace ace {
namespace {

constexpr int kGroupThreads = 1024;
constexpr int kGroupWarps = kGroupThreads / 32;
constexpr int kOneCta = 256;      // tokens up to which one CTA serves
constexpr int kEightCtas = 2048;  // and a cluster of 8; beyond it one of 16
constexpr int kTokens = 32;       // tokens per chunk, a bit each

struct GroupArgs {
  const int32_t* idx;
  const uint8_t* keep;  // or NULL (all kept)
  const float* gate;    // or NULL
  int32_t* offsets;
  int32_t* slot_of;
  int32_t* slot_token;  // or NULL
  float* slot_gate;     // or NULL
  int S, T, k, E;
};

__global__ void __launch_bounds__(kGroupThreads) k_group(const GroupArgs A) {
  extern __shared__ uint32_t s_dyn[];  // per warp: counts, then positions [E]; bits [E]
  __shared__ int s_total[kMaxE];       // this CTA's slots per expert, read by the cluster
  __shared__ int s_warp[32];
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nc = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int E = A.E, k = A.k;
  int* count = reinterpret_cast<int*>(s_dyn) + warp * E;
  uint32_t* bits = s_dyn + (kGroupWarps + warp) * E;
  // chunks of this CTA, and of this warp
  const int chunks = (A.T + kTokens - 1) / kTokens, per_cta = (chunks + nc - 1) / nc;
  const int per_warp = (per_cta + kGroupWarps - 1) / kGroupWarps;
  const int end = min(chunks, (rank + 1) * per_cta);
  const int c0 = min(end, rank * per_cta + warp * per_warp), c1 = min(end, c0 + per_warp);
  const uint32_t by_k = (1u << 16) / k + 1;  // x / k = x by_k >> 16 for x < 512, k <= 16

  for (int i = lane; i < E; i += 32) {
    count[i] = 0;
    bits[i] = 0u;
  }
  __syncwarp();
  begin_overlapped();
  // The chunk's slots x = 32 j + lane: experts of kept slots, else -1.  Every load
  // is in flight before the first is used.
  int e[kMaxK];
  auto load = [&](int c) {
    const int64_t s0 = (int64_t)c * kTokens * k;
    const int n = (int)min((int64_t)kTokens * k, A.S - s0);
    uint8_t kept[kMaxK];
#pragma unroll
    for (int j = 0; j < kMaxK; ++j) {
      const int x = j * 32 + lane;
      e[j] = x < n ? A.idx[s0 + x] : -1;
      kept[j] = x < n && A.keep ? A.keep[s0 + x] : 1;
    }
#pragma unroll
    for (int j = 0; j < kMaxK; ++j)
      if (e[j] >= E || !kept[j]) e[j] = -1;
    return n;
  };
  int n = 0;  // slots of the chunk in registers
  for (int c = c0; c < c1; ++c) {
    n = load(c);
#pragma unroll
    for (int j = 0; j < kMaxK; ++j)
      if (e[j] >= 0) atomicAdd(&count[e[j]], 1);
  }
  __syncthreads();
  // first positions of the warps within the CTA
  for (int i = tid; i < E; i += kGroupThreads) {
    int acc = 0;
#pragma unroll 8
    for (int w = 0; w < kGroupWarps; ++w) {
      int* q = reinterpret_cast<int*>(s_dyn) + w * E + i;
      const int m = *q;
      *q = acc;
      acc += m;
    }
    s_total[i] = acc;
  }
  cluster.sync();
  int all = 0, before = 0;
  if (tid < E)
    for (int r = 0; r < nc; ++r) {
      const int m = cluster.map_shared_rank(s_total, r)[tid];
      all += m;
      before += r < rank ? m : 0;
    }
  cluster.sync();  // every CTA's totals are read before they become positions
  int total;
  const int off = block_excl_scan(all, s_warp, &total);
  if (tid < E) {
    s_total[tid] = off + before;  // from here on: the CTA's first position of the expert
    if (rank == 0) A.offsets[tid] = off;
  }
  if (rank == 0 && tid == 0) A.offsets[E] = total;
  __syncthreads();

  for (int c = c0; c < c1; ++c) {
    if (c1 - c0 > 1) n = load(c);  // a warp's only chunk is still in registers
    const int64_t s0 = (int64_t)c * kTokens * k;
    float g[kMaxK];
    bool twice = false;
#pragma unroll
    for (int j = 0; j < kMaxK; ++j) {
      const int x = j * 32 + lane;
      g[j] = A.slot_gate && e[j] >= 0 ? A.gate[s0 + x] : 0.f;
      const uint32_t bit = 1u << (x * by_k >> 16 & 31);
      if (e[j] >= 0) twice |= (atomicOr(&bits[e[j]], bit) & bit) != 0u;
    }
    twice = __any_sync(0xffffffffu, twice);
    __syncwarp();  // every bit is set before any is read
#pragma unroll
    for (int j = 0; j < kMaxK; ++j) {
      if (j * 32 >= n) break;  // the same for the warp
      const int x = j * 32 + lane, t = x * by_k >> 16 & 31;
      int ahead = 0;
      if (twice) {
        const uint32_t same = __match_any_sync(0xffffffffu, e[j]);
        if (e[j] >= 0) ahead = count[e[j]];
        __syncwarp();
        if (e[j] >= 0) count[e[j]] = ahead + __popc(same);  // equal from all of an expert's lanes
        __syncwarp();
        ahead += __popc(same & ((1u << lane) - 1u));
      } else if (e[j] >= 0) {
        ahead = count[e[j]] + __popc(bits[e[j]] & ((1u << t) - 1u));
      }
      if (x < n) {
        const int pos = e[j] >= 0 ? s_total[e[j]] + ahead : -1;
        A.slot_of[s0 + x] = pos;
        if (e[j] >= 0) {
          if (A.slot_token) A.slot_token[pos] = c * kTokens + t;
          if (A.slot_gate) A.slot_gate[pos] = g[j];
        }
      }
    }
    if (c + 1 < c1) {
      __syncwarp();
      for (int i = lane; i < E; i += 32) {
        if (!twice) count[i] += __popc(bits[i]);
        bits[i] = 0u;
      }
      __syncwarp();
    }
  }
}

bool is_aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Whether the current device can place a cluster of 16 of these CTAs, an SM each, in
// one of its GPCs: 8 is what every device offers, and a partition of one may have no
// more.  Asked once a device (the answer takes as long as a launch).
bool sixteen_fit() {
  static std::atomic<int> known[64] = {};  // 0: not asked, 1: no, 2: yes
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
  int k = known[dev].load(std::memory_order_relaxed);
  if (k == 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(16);
    cfg.blockDim = dim3(kGroupThreads);
    cfg.dynamicSmemBytes = (size_t)2 * kGroupWarps * kMaxE * sizeof(uint32_t);
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 16;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    int n = 0;
    k = cudaFuncSetAttribute(k_group, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) ==
                    cudaSuccess &&
                cudaOccupancyMaxActiveClusters(&n, k_group, &cfg) == cudaSuccess && n > 0
            ? 2
            : 1;
    if (k == 1) cudaGetLastError();  // a refusal is an answer
    known[dev].store(k, std::memory_order_relaxed);
  }
  return k == 2;
}

cudaError_t launch_group(const GroupArgs& A, cudaStream_t s) {
  const size_t smem = (size_t)2 * kGroupWarps * A.E * sizeof(uint32_t);
  cudaError_t e = cudaFuncSetAttribute(k_group, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       2 * kGroupWarps * kMaxE * (int)sizeof(uint32_t));
  if (e != cudaSuccess) return e;
  // One CTA for the chunks of a decode step; beyond it clusters, whose SMs share
  // the scattered stores (8192 tokens of 8: 16.8 us on 8 SMs, 11.3 on 16; 512
  // tokens: 7.7 us on 8).
  const int nc = A.T <= kOneCta ? 1 : A.T <= kEightCtas || !sixteen_fit() ? 8 : 16;
  if (nc == 16) {
    e = cudaFuncSetAttribute(k_group, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  return launch_overlapped(k_group, nc, kGroupThreads, nc, smem, s, A);
}

}  // namespace
}  // namespace ace

using namespace ace;

extern "C" {

ace_status ace_moe_group(const int32_t* idx, const uint8_t* keep, const float* gate, int T, int k,
                         int E, int32_t* offsets, int32_t* slot_of, int32_t* slot_token,
                         float* slot_gate, void* stream) {
  if (T < 0 || k < 1 || k > kMaxK || E < 1 || !offsets) return ACE_ERR_INVALID_ARG;
  if (E > kMaxE || (int64_t)T * k > kMaxCount) return ACE_ERR_UNSUPPORTED;
  if (T > 0 && (!idx || !slot_of || (slot_gate && !gate))) return ACE_ERR_INVALID_ARG;
  if (!is_aligned(idx, 4) || !is_aligned(gate, 4) || !is_aligned(offsets, 4) ||
      !is_aligned(slot_of, 4) || !is_aligned(slot_token, 4) || !is_aligned(slot_gate, 4))
    return ACE_ERR_INVALID_ARG;
  const int64_t S = (int64_t)T * k;
  const ByteSpan in[3] = {ByteSpan(idx, 1, S, 1, 4), ByteSpan(keep, 1, S, 1, 1),
                          ByteSpan(gate, 1, S, 1, 4)};
  const ByteSpan out[4] = {ByteSpan(offsets, 1, E + 1, 1, 4), ByteSpan(slot_of, 1, S, 1, 4),
                           ByteSpan(slot_token, 1, S, 1, 4), ByteSpan(slot_gate, 1, S, 1, 4)};
  for (int o = 0; o < 4; ++o) {
    for (const ByteSpan& i : in)
      if (out[o].meets(i)) return ACE_ERR_INVALID_ARG;
    for (int p = 0; p < o; ++p)
      if (out[o].meets(out[p])) return ACE_ERR_INVALID_ARG;
  }
  const GroupArgs A = {idx, keep, gate, offsets, slot_of, slot_token, slot_gate, T * k, T, k, E};
  return cuda_status(launch_group(A, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

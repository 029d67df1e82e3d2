// group.cu -- kept slots grouped by expert: the counting sort between the
// gate and the experts' products.
//
//   slots s = t k + i with keep (and a valid expert) go to positions in the
//   order (expert, token, rank); offsets[e] = first position of expert e,
//   offsets[E] = their number.
//
// One launch: a cluster of 1 or 8 CTAs, every warp with one run of
// consecutive slots.  A warp counts its run per expert in its own row of
// shared memory (lanes of equal expert find each other by match.any, the first
// of them adds their number), a prefix over warps, then over the cluster's CTAs
// through distributed shared memory, then over experts gives each (warp,
// expert) its first position, and a second pass hands positions out in slot
// order.  No atomics, so the order never varies; no global scratch, so nothing
// needs clearing.  Latency bound: two dependent passes over at most 2^13 slots
// a warp at 10^6 tokens, and three cluster barriers.
#include <cooperative_groups.h>

#include "ace_common.cuh"
#include "ace_internal.h"
#include "compact.cuh"

namespace cg = cooperative_groups;

namespace ace {
namespace {

constexpr int kGroupThreads = 1024;
constexpr int kGroupWarps = kGroupThreads / 32;
constexpr int kGroupCluster = 8;  // portable cluster size
constexpr int kUnroll = 4;        // loads of a lane in flight

struct GroupArgs {
  const int32_t* idx;
  const uint8_t* keep;  // or NULL (all kept)
  const float* gate;    // or NULL
  int32_t* offsets;
  int32_t* slot_of;
  int32_t* slot_token;  // or NULL
  float* slot_gate;     // or NULL
  int S, k, E;
};

__global__ void __launch_bounds__(kGroupThreads) k_group(const GroupArgs A) {
  extern __shared__ int s_hist[];  // [warps][E]
  __shared__ int s_total[kMaxE];   // this CTA's slots per expert, read by the cluster
  __shared__ int s_base[kMaxE];
  __shared__ int s_warp[32];
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nc = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int E = A.E;
  int* hist = s_hist + warp * E;
  for (int e = lane; e < E; e += 32) hist[e] = 0;
  __syncwarp();
  const int nw = nc * kGroupWarps, gw = rank * kGroupWarps + warp;
  const int64_t run = (((int64_t)A.S + nw - 1) / nw + 31) / 32 * 32;
  const int64_t s0 = gw * run, s1 = s0 + run < A.S ? s0 + run : A.S;
  auto expert = [&](int64_t s) {
    int e = -1;
    if (s < s1 && (A.keep == nullptr || A.keep[s] != 0)) {
      e = A.idx[s];
      if (e < 0 || e >= E) e = -1;
    }
    return e;
  };
  for (int64_t b = s0; b < s1; b += 32 * kUnroll) {
    int e[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) e[u] = expert(b + u * 32 + lane);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const uint32_t same = __match_any_sync(0xffffffffu, e[u]);
      if (e[u] >= 0 && lane == __ffs((int)same) - 1) hist[e[u]] += __popc(same);
      __syncwarp();
    }
  }
  __syncthreads();
  // warps' first positions within the CTA
  for (int e = tid; e < E; e += kGroupThreads) {
    int acc = 0;
#pragma unroll 8
    for (int w = 0; w < kGroupWarps; ++w) {
      const int c = s_hist[w * E + e];
      s_hist[w * E + e] = acc;
      acc += c;
    }
    s_total[e] = acc;
  }
  cluster.sync();
  int all = 0, before = 0;
  if (tid < E)
    for (int r = 0; r < nc; ++r) {
      const int c = cluster.map_shared_rank(s_total, r)[tid];
      all += c;
      before += r < rank ? c : 0;
    }
  cluster.sync();  // every CTA's totals are read before any CTA leaves
  int total;
  const int off = block_excl_scan(all, s_warp, &total);
  if (tid < E) {
    s_base[tid] = off + before;
    if (rank == 0) A.offsets[tid] = off;
  }
  if (rank == 0 && tid == 0) A.offsets[E] = total;
  __syncthreads();
  for (int64_t b = s0; b < s1; b += 32 * kUnroll) {
    int e[kUnroll];
    float g[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t s = b + u * 32 + lane;
      e[u] = expert(s);
      g[u] = A.slot_gate && e[u] >= 0 ? A.gate[s] : 0.f;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t s = b + u * 32 + lane;
      const uint32_t same = __match_any_sync(0xffffffffu, e[u]);
      int pos = -1;
      if (e[u] >= 0) pos = s_base[e[u]] + hist[e[u]] + __popc(same & ((1u << lane) - 1u));
      __syncwarp();
      if (e[u] >= 0 && lane == __ffs((int)same) - 1) hist[e[u]] += __popc(same);
      __syncwarp();
      if (s < s1) A.slot_of[s] = pos;
      if (pos >= 0) {
        if (A.slot_token) A.slot_token[pos] = (int)(s / A.k);
        if (A.slot_gate) A.slot_gate[pos] = g[u];
      }
    }
  }
}

bool is_aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

cudaError_t launch_group(const GroupArgs& A, cudaStream_t s) {
  const size_t smem = (size_t)kGroupWarps * A.E * sizeof(int);
  cudaError_t e = cudaFuncSetAttribute(k_group, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       kGroupWarps * kMaxE * (int)sizeof(int));
  if (e != cudaSuccess) return e;
  // one CTA while its warps have at most two steps each, then the cluster
  const int nc = A.S <= kGroupWarps * 32 * 2 ? 1 : kGroupCluster;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)nc);
  cfg.blockDim = dim3(kGroupThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)nc;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_group, A);
}

}  // namespace
}  // namespace ace

using namespace ace;

extern "C" {

ace_status ace_moe_group(const int32_t* idx, const uint8_t* keep, const float* gate, int T, int k,
                         int E, int32_t* offsets, int32_t* slot_of, int32_t* slot_token,
                         float* slot_gate, void* stream) {
  if (T < 0 || k < 1 || k > kMaxK || E < 1 || !offsets) return ACE_ERR_INVALID_ARG;
  if (E > kMaxE || (int64_t)T * k > 0x7fffffff) return ACE_ERR_UNSUPPORTED;
  if (T > 0 && (!idx || !slot_of || (slot_gate && !gate))) return ACE_ERR_INVALID_ARG;
  if (!is_aligned(idx, 4) || !is_aligned(gate, 4) || !is_aligned(offsets, 4) ||
      !is_aligned(slot_of, 4) || !is_aligned(slot_token, 4) || !is_aligned(slot_gate, 4))
    return ACE_ERR_INVALID_ARG;
  const GroupArgs A = {idx, keep, gate, offsets, slot_of, slot_token, slot_gate, T * k, k, E};
  return cuda_status(launch_group(A, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

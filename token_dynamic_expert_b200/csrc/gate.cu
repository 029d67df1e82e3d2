// gate.cu -- the gate of a routed layer from its logits: softmax or sigmoid
// scores, a balance bias that takes part in the choice alone, a limit to the
// best groups of experts, top-k, weights.
//
//   s_e = softmax(l)_e or 1 / (1 + e^-l_e)
//   c_e = s_e + b_e; without a bias the choice goes by l_e (the same order)
//   group value = largest c of the group, or the sum of its two largest
//   allowed: the topk_groups groups of the largest values (ties: lower index)
//   chosen: the k largest c of the allowed groups (ties: lower index), in order
//   w_i = scale s_i [ / sum of the chosen s ]
//   keep_i = i is the token's largest weight, or !(w_i A_e < tau)
//
// One warp per token.  A group lies on 32 / (groups rounded up to a power of
// two) neighbouring lanes, so its value needs only shuffles inside them; a lane
// sorts its experts once (packed as key << 32 | ~expert, largest first) and the
// k rounds look at the lanes' heads.  Bound by latency: a chain of shuffles and
// warp reductions per token, 8.9 MB of logits and results at 8192 x 256.
//
// The choice is the one of exact arithmetic on the given logits: without a bias
// it compares logits; with one, or where two groups' sums decide, scores whose
// fp32 difference is within the error bound below are compared again in fp64
// (a token in some hundreds).
#include <math.h>

#include "ace_common.cuh"
#include "ace_internal.h"

namespace ace {
namespace {

constexpr int kGateWarps = 4;

struct GateArgs {
  const void* logits;
  int64_t ld;
  const float* bias;    // [E] or NULL
  const float* factor;  // [E] ACE factors or NULL (1)
  int32_t* idx;
  float* weight;
  uint8_t* keep;  // or NULL
  int T, E, k, sigmoid, G, topk_groups, top2, renorm, vec;
  float scale, tau;
};

// Where a lane's experts are: e0 + j * step for j < n, below end.
struct LaneMap {
  int e0, step, n, end, group;
};

__device__ __forceinline__ LaneMap lane_map(const GateArgs& A, int lane, int lg) {
  if (A.G == 1) return {lane, 32, (A.E + 31) / 32, A.E, 0};
  const int per = A.E / A.G, g = lane / lg, n = (per + lg - 1) / lg;
  if (g >= A.G) return {0, 1, 0, 0, g};
  const int e0 = g * per + (lane % lg) * n;
  return {e0, 1, n, min(e0 + n, (g + 1) * per), g};
}

template <typename TL>
__device__ __forceinline__ float logit_at(const TL* row, int e) {
  return to_f(row[e]);
}

// fkey with -0 equal to +0 and every NaN above +infinity.  On the bits: the
// sign and payload of a computed NaN are not to be relied on.
__device__ __forceinline__ uint32_t gate_key(float v) {
  const uint32_t b = __float_as_uint(v), a = b & 0x7fffffffu;
  return a > 0x7f800000u ? 0xffffffffu : a == 0u ? 0x80000000u : fkey(v);
}

// Largest two of the values held by the lg neighbouring lanes of a group.
template <typename F>
__device__ __forceinline__ void group_top2(F& a, F& b, int lg) {
  for (int o = 1; o < lg; o <<= 1) {
    const F oa = __shfl_xor_sync(0xffffffffu, a, o), ob = __shfl_xor_sync(0xffffffffu, b, o);
    const F second = oa > a ? a : oa;
    a = oa > a ? oa : a;
    b = b > ob ? b : ob;
    b = second > b ? second : b;
  }
}

// The choice in fp64 (see the head of the file); lane i < k receives rank i.
template <typename TL>
__device__ __noinline__ int choose64(const GateArgs& A, const TL* row, int lane, int lg) {
  const LaneMap L = lane_map(A, lane, lg);
  double m = -INFINITY, z = 0.0;
  if (!A.sigmoid) {
    float mf = -INFINITY;
    for (int j = 0, e = L.e0; j < L.n && e < L.end; ++j, e += L.step)
      mf = fmaxf(mf, logit_at(row, e));
    for (int o = 16; o > 0; o >>= 1) mf = fmaxf(mf, __shfl_xor_sync(0xffffffffu, mf, o));
    m = isinf(mf) && mf < 0.f ? 0.0 : (double)mf;
    for (int j = 0, e = L.e0; j < L.n && e < L.end; ++j, e += L.step)
      z += exp((double)logit_at(row, e) - m);
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
  }
  auto score = [&](int e) {
    const double x = (double)logit_at(row, e);
    if (A.sigmoid) return 1.0 / (1.0 + exp(-x));
    return z > 0.0 ? exp(x - m) / z : 0.0;
  };
  bool allowed = true;
  if (A.G > 1) {
    double a = -INFINITY, b = -INFINITY;
    for (int j = 0, e = L.e0; j < L.n && e < L.end; ++j, e += L.step) {
      const double c = A.bias ? score(e) + (double)A.bias[e]
                              : (A.top2 ? score(e) : (double)logit_at(row, e));
      if (c > a) {
        b = a;
        a = c;
      } else if (c > b) {
        b = c;
      }
    }
    group_top2(a, b, lg);
    const double gv = A.top2 && A.E / A.G > 1 ? a + b : a;
    int rank = 0;
    for (int h = 0; h < A.G; ++h) {
      const double o = __shfl_sync(0xffffffffu, gv, h * lg);
      rank += o > gv || (o == gv && h < L.group);
    }
    allowed = L.group < A.G && rank < A.topk_groups;
  }
  uint32_t taken = 0u;
  int mine = 0;
  for (int i = 0; i < A.k; ++i) {
    double best = -INFINITY;
    int be = 0x7fffffff;
    if (allowed)
      for (int j = 0, e = L.e0; j < L.n && e < L.end; ++j, e += L.step) {
        if ((taken >> j) & 1u) continue;
        const double c = A.bias ? score(e) + (double)A.bias[e] : (double)logit_at(row, e);
        if (be == 0x7fffffff || c > best) {
          best = c;
          be = e;
        }
      }
    for (int o = 16; o > 0; o >>= 1) {
      const double ob = __shfl_xor_sync(0xffffffffu, best, o);
      const int oe = __shfl_xor_sync(0xffffffffu, be, o);
      if (oe != 0x7fffffff && (be == 0x7fffffff || ob > best || (ob == best && oe < be))) {
        best = ob;
        be = oe;
      }
    }
    for (int j = 0, e = L.e0; j < L.n && e < L.end; ++j, e += L.step)
      if (e == be) taken |= 1u << j;
    if (lane == i) mine = be;
  }
  return mine;
}

template <typename TL, int NV>
__global__ void __launch_bounds__(kGateWarps * 32) k_gate_topk(const GateArgs A) {
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (t >= A.T) return;
  const TL* row = static_cast<const TL*>(A.logits) + (size_t)t * A.ld;
  int gp = 1;
  while (gp < A.G) gp <<= 1;
  const int lg = 32 / gp;
  const LaneMap L = lane_map(A, lane, lg);
  const bool biased = A.bias != nullptr;

  float x[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) x[j] = -INFINITY;
  constexpr int VL = NV < 4 ? 1 : 4;
  if (VL > 1 && A.vec && L.n == NV) {  // a lane's neighbouring experts, 4 a load
#pragma unroll
    for (int j = 0; j < NV; j += VL) {
      struct alignas(sizeof(TL) * VL) Q {
        TL e[VL];
      };
      const Q v = *reinterpret_cast<const Q*>(row + L.e0 + j);
#pragma unroll
      for (int c = 0; c < VL; ++c) x[j + c] = to_f(v.e[c]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int e = L.e0 + j * L.step;
      if (j < L.n && e < L.end) x[j] = to_f(row[e]);
    }
  }
  float bv[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int e = L.e0 + j * L.step;
    bv[j] = biased && j < L.n && e < L.end ? A.bias[e] : 0.f;
  }

  // softmax: maximum and sum over all experts
  float m = 0.f, z = 1.f;
  if (!A.sigmoid) {
    m = -INFINITY;
#pragma unroll
    for (int j = 0; j < NV; ++j) m = fmaxf(m, x[j]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (m == -INFINITY) m = 0.f;  // nothing left: every score is 0
    z = 0.f;
    if (biased || A.top2 || !A.renorm) {
#pragma unroll
      for (int j = 0; j < NV; ++j) z += x[j] == -INFINITY ? 0.f : expf(x[j] - m);
      z = warp_sum(z);
    }
  }
  const float inv_z = z > 0.f ? 1.f / z : 0.f;
  auto score = [&](float v) {
    return A.sigmoid ? 1.f / (1.f + expf(-v)) : (v == -INFINITY ? 0.f : expf(v - m) * inv_z);
  };

  // keys, sorted largest first within the lane
  uint64_t c[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int e = L.e0 + j * L.step;
    const float key = biased ? score(x[j]) + bv[j] : x[j];
    c[j] = j < L.n && e < L.end ? ((uint64_t)gate_key(key) << 32) | (uint64_t)(~(uint32_t)e) : 0ull;
  }
#pragma unroll
  for (int p = 1; p < NV; p <<= 1)
#pragma unroll
    for (int kk = p; kk >= 1; kk >>= 1)
#pragma unroll
      for (int j = kk % p; j + kk < NV; j += 2 * kk)
#pragma unroll
        for (int i = 0; i < kk; ++i) {
          const int a = i + j, b = i + j + kk;
          if (b < NV && a / (2 * p) == b / (2 * p)) {
            const uint64_t va = c[a], vb = c[b];
            const bool sw = vb > va;
            c[a] = sw ? vb : va;
            c[b] = sw ? va : vb;
          }
        }

  // Half the difference two exact scores may have where fp32 sees them equal:
  // sigmoid: expf 2 ulp, the sum, the quotient: 4 x 2^-24 of s <= 1; softmax:
  // the exponent's rounding (at most 0.37 x 2^-24 of the largest score), expf,
  // and a sum of E <= 512 terms: 44 x 2^-24 of the largest score 1 / z; both:
  // the addition of the bias, 2^-24 of c.  Doubled for two scores, and again
  // for room.
  const float err = A.sigmoid ? 9.6e-7f : 1.1e-5f * inv_z;
  bool near = false;

  if (A.G > 1) {
    float a = -INFINITY, b = -INFINITY;
    if (c[0] != 0ull) a = fkey_inv((uint32_t)(c[0] >> 32));
    if (NV > 1 && c[NV > 1 ? 1 : 0] != 0ull) b = fkey_inv((uint32_t)(c[NV > 1 ? 1 : 0] >> 32));
    float gv;
    if (A.top2 && A.E / A.G > 1) {
      if (!biased) {  // the keys are logits
        a = c[0] != 0ull ? score(a) : a;
        b = (NV > 1 && c[NV > 1 ? 1 : 0] != 0ull) ? score(b) : -INFINITY;
      }
      group_top2(a, b, lg);
      gv = a + b;
    } else {
      group_top2(a, b, lg);
      gv = a;
      b = 0.f;
    }
    const float mag = fabsf(a) + fabsf(b);
    const uint32_t gk = L.group < A.G ? gate_key(gv) : 0u;
    int rank = 0;
    for (int h = 0; h < A.G; ++h) {
      const uint32_t o = __shfl_sync(0xffffffffu, gk, h * lg);
      rank += o > gk || (o == gk && h < L.group);
    }
    const bool allowed = L.group < A.G && rank < A.topk_groups;
    if (biased || A.top2) {
      // the last group inside against the first outside
      const uint32_t last = __reduce_min_sync(0xffffffffu, allowed ? gk : 0xffffffffu);
      const uint32_t next = __reduce_max_sync(0xffffffffu, !allowed && L.group < A.G ? gk : 0u);
      const float top = __uint_as_float(
          __reduce_max_sync(0xffffffffu, L.group < A.G ? __float_as_uint(mag) : 0u));
      near = next != 0u && fkey_inv(last) - fkey_inv(next) <= 2.f * (err + 4.8e-7f * top);
    }
    if (!allowed) {
#pragma unroll
      for (int j = 0; j < NV; ++j) c[j] = 0ull;
    }
  }

  // k rounds; with a bias one more, for the border between k and k + 1
  int my_e = 0;
  uint32_t my_k = 0u;
  const int rounds = A.k + (biased ? 1 : 0);
  for (int i = 0; i < rounds; ++i) {
    const uint32_t hk = (uint32_t)(c[0] >> 32);
    const uint32_t mk = __reduce_max_sync(0xffffffffu, hk);
    const uint32_t ne = __reduce_max_sync(0xffffffffu, hk == mk ? (uint32_t)c[0] : 0u);
    const bool pop = mk != 0u && hk == mk && (uint32_t)c[0] == ne;
#pragma unroll
    for (int j = 0; j + 1 < NV; ++j) c[j] = pop ? c[j + 1] : c[j];
    if (pop) c[NV - 1] = 0ull;
    if (lane == i) {
      my_e = mk != 0u ? (int)~ne : -1;
      my_k = mk;
    }
  }
  float my_x = -INFINITY;
  if (biased) {
    float my_b = 0.f;
    if (lane <= A.k && my_e >= 0) {
      my_x = logit_at(row, my_e);
      my_b = A.bias[my_e];
    }
    const float v = fkey_inv(my_k);
    const uint32_t nk = __shfl_down_sync(0xffffffffu, my_k, 1);
    const float nx = __shfl_down_sync(0xffffffffu, my_x, 1);
    const float nb = __shfl_down_sync(0xffffffffu, my_b, 1);
    const float nvv = fkey_inv(nk);
    const bool same = nx == my_x && nb == my_b;  // a true tie: the index decides
    if (lane < A.k && nk != 0u && !same)
      near |= v - nvv <= 2.f * (err + 1.2e-7f * fmaxf(fabsf(v), fabsf(nvv)));
  }
  if (__any_sync(0xffffffffu, near)) my_e = choose64(A, row, lane, lg);

  // weights
  const bool on = lane < A.k;
  if (on) my_x = logit_at(row, my_e);
  float w = 0.f;
  if (A.renorm) {
    // relative to the largest chosen logit, so that no sum underflows
    float top = on ? my_x : -INFINITY;
    const bool nan = __any_sync(0xffffffffu, on && my_x != my_x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (top != -INFINITY && on) {
      if (!A.sigmoid) {
        w = expf(my_x - top);
      } else {  // s = e^x / (1 + e^x); below 0 in units of e^min(top, 0)
        w = my_x > 0.f ? 1.f / (1.f + expf(-my_x))
                       : expf(my_x - fminf(top, 0.f)) / (1.f + expf(my_x));
      }
    }
    const float sum = warp_sum(w);
    w = nan ? __uint_as_float(0x7fffffffu) : (sum > 0.f ? w / sum : (sum != sum ? sum : 0.f));
  } else if (on) {
    w = score(my_x);
  }
  w *= A.scale;
  if (on) {
    const size_t o = (size_t)t * A.k + lane;
    A.idx[o] = my_e;
    A.weight[o] = w;
  }
  if (A.keep != nullptr) {
    // the token's largest weight (ties: the earlier slot) is always kept
    const uint32_t wk = on ? gate_key(w) : 0u;
    const uint32_t lead = __reduce_max_sync(0xffffffffu, wk);
    const int first = __ffs((int)__ballot_sync(0xffffffffu, on && wk == lead)) - 1;
    if (on)
      A.keep[(size_t)t * A.k + lane] =
          lane == first || !(w * (A.factor ? A.factor[my_e] : 1.f) < A.tau);
  }
}

bool is_aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

template <typename TL>
cudaError_t launch_gate(const GateArgs& A, cudaStream_t s) {
  int gp = 1;
  while (gp < A.G) gp <<= 1;
  const int n = A.G == 1 ? cdiv(A.E, 32) : cdiv(A.E / A.G, 32 / gp);
  const int warps = A.T < kGateWarps ? A.T : kGateWarps;
  const dim3 grid((unsigned)cdiv(A.T, warps)), block((unsigned)(32 * warps));
  if (n <= 1)
    k_gate_topk<TL, 1><<<grid, block, 0, s>>>(A);
  else if (n <= 2)
    k_gate_topk<TL, 2><<<grid, block, 0, s>>>(A);
  else if (n <= 4)
    k_gate_topk<TL, 4><<<grid, block, 0, s>>>(A);
  else if (n <= 8)
    k_gate_topk<TL, 8><<<grid, block, 0, s>>>(A);
  else if (n <= 16)
    k_gate_topk<TL, 16><<<grid, block, 0, s>>>(A);
  else
    k_gate_topk<TL, 32><<<grid, block, 0, s>>>(A);
  return cudaGetLastError();
}

}  // namespace
}  // namespace ace

using namespace ace;

extern "C" {

ace_status ace_gate_topk(const void* logits, int64_t ld, ace_dtype dtype, int T, int E, int k,
                         const float* bias, const ace_gate_opts* opts, int32_t* idx,
                         float* weight, const float* factor, uint8_t* keep, void* stream) {
  if (!opts || (dtype != ACE_BF16 && dtype != ACE_F32)) return ACE_ERR_INVALID_ARG;
  if (T < 0 || E < 1 || k < 1 || k > E || k > kMaxK) return ACE_ERR_INVALID_ARG;
  if (E > kMaxE) return ACE_ERR_UNSUPPORTED;
  if (opts->score != ACE_SCORE_SOFTMAX && opts->score != ACE_SCORE_SIGMOID)
    return ACE_ERR_INVALID_ARG;
  if (opts->group_score != ACE_GROUP_MAX && opts->group_score != ACE_GROUP_TOP2)
    return ACE_ERR_INVALID_ARG;
  const int G = opts->n_groups, tg = opts->topk_groups;
  if (G < 1 || tg < 1 || tg > G || E % G != 0) return ACE_ERR_INVALID_ARG;
  if (G > 32) return ACE_ERR_UNSUPPORTED;
  if ((int64_t)tg * (E / G) < k) return ACE_ERR_INVALID_ARG;
  if (!(opts->scale > 0.f) || !(opts->scale <= 3.4e38f)) return ACE_ERR_INVALID_ARG;
  if (T == 0) return ACE_OK;
  const size_t es = dtype == ACE_BF16 ? 2 : 4;
  if (!logits || !idx || !weight || !is_aligned(logits, es) || !is_aligned(idx, 4) ||
      !is_aligned(weight, 4) || !is_aligned(bias, 4) || !is_aligned(factor, 4) || ld < E)
    return ACE_ERR_INVALID_ARG;
  GateArgs A;
  A.logits = logits;
  A.ld = ld;
  A.bias = bias;
  A.factor = factor;
  A.idx = idx;
  A.weight = weight;
  A.keep = keep;
  A.T = T;
  A.E = E;
  A.k = k;
  A.sigmoid = opts->score == ACE_SCORE_SIGMOID;
  A.G = tg == G ? 1 : G;  // every group allowed: no limit
  A.topk_groups = tg;
  A.top2 = A.G > 1 && opts->group_score == ACE_GROUP_TOP2;
  A.renorm = opts->renorm_topk != 0;
  // a lane's experts are neighbours and start at a multiple of 4 of them
  int gp = 1;
  while (gp < A.G) gp <<= 1;
  const int per = E / A.G, lg = 32 / gp;
  A.vec = A.G > 1 && per % lg == 0 && (per / lg) % 4 == 0 && ld % 4 == 0 &&
          is_aligned(logits, 4 * es);
  A.scale = opts->scale;
  A.tau = opts->tau;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return cuda_status(dtype == ACE_BF16 ? launch_gate<__nv_bfloat16>(A, s) : launch_gate<float>(A, s));
}

}  // extern "C"

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
// One warp per token.  A lane holds neighbouring experts, and a group lies on
// 32 / (groups rounded up to a power of two) neighbouring lanes, so its value
// needs only shuffles inside them, and of two equal keys the lower lane's is the
// lower expert.  A lane sorts its experts once (packed as key << 32 | ~expert,
// largest first) and leaves the list in shared memory; each of the k rounds takes
// the largest of the lanes' heads by redux.max and moves one lane on.  Bound by
// instruction issue (about 1050 a token) and the latency of the rounds; the data
// are 8.9 MB at 8192 tokens of 256 experts: 14.9 us with a bias and 8 groups, 10.7
// without; one token 2.5 us.  Lists kept in registers and shifted, with 64-bit
// scores throughout the ties, took 43 us.
//
// The choice is the one of exact arithmetic on the given logits: without a bias
// it compares logits; with one, or where two groups' sums decide, scores whose
// fp32 difference is within the error bound below are compared again in fp64
// (a token in some hundreds).  The scores that only decide are therefore formed
// with the hardware's base-2 exponential; weights are formed with expf.
#include <math.h>

#include "ace_common.cuh"
#include "ace_internal.h"
#include "launch.cuh"

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
  int T, E, k, sigmoid, G, lanes, topk_groups, top2, renorm, vec;
  float scale, tau;
};

// A lane's experts: e0 .. e0 + n - 1, of group `group`.
struct LaneMap {
  int e0, n, group;
};

__device__ __forceinline__ LaneMap lane_map(const GateArgs& A, int lane, int lg) {
  const int per = A.E / A.G, g = lane / lg, n = (per + lg - 1) / lg;
  const int at = (lane % lg) * n;
  return {g * per + at, g < A.G ? max(0, min(n, per - at)) : 0, g};
}

template <typename TL>
__device__ __forceinline__ float logit_at(const TL* row, int e) {
  return to_f(row[e]);
}

__device__ __forceinline__ float exp2_approx(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float rcp_approx(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// fkey with -0 equal to +0 and every NaN above +infinity, whatever its sign.
__device__ __forceinline__ uint32_t gate_key(float v) {
  const uint32_t b = __float_as_uint(__fadd_rn(v, 0.f));
  return v == v ? b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u) : 0xffffffffu;
}

// Largest two of the keys held by the lg neighbouring lanes of a group (a >= b in
// each lane).  Keys are integers, so every lane of the group ends with the same two,
// whatever the values were; floats compared by > would leave a NaN with its own lane.
template <typename U>
__device__ __forceinline__ void group_top2(U& a, U& b, int lg) {
  for (int o = 1; o < lg; o <<= 1) {
    const U oa = __shfl_xor_sync(0xffffffffu, a, o), ob = __shfl_xor_sync(0xffffffffu, b, o);
    b = max(max(b, ob), min(a, oa));
    a = max(a, oa);
  }
}

// gate_key for doubles, and the double of a key.
__device__ __forceinline__ unsigned long long dkey(double v) {
  const unsigned long long b = (unsigned long long)__double_as_longlong(v + 0.0);
  return v != v ? ~0ull : (b >> 63) ? ~b : b | 0x8000000000000000ull;
}
__device__ __forceinline__ double dkey_inv(unsigned long long k) {
  return __longlong_as_double(
      (long long)((k >> 63) ? k & 0x7fffffffffffffffull : ~k));
}

// A softmax score from t = e^(x - m) and the sum z.  NaN stays with the experts that
// cause it (a NaN logit, +infinity less the maximum); it makes z NaN, and the
// token's other scores count as 0.
__device__ __forceinline__ double share64(double t, double z) {
  return t != t ? t : z > 0.0 ? t / z : 0.0;
}

// Largest 64-bit value over the warp, by its halves.
__device__ __forceinline__ unsigned long long max64(unsigned long long v) {
  const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(v >> 32));
  const uint32_t lo =
      __reduce_max_sync(0xffffffffu, (uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
  return ((unsigned long long)hi << 32) | lo;
}

// The choice in fp64 (see the head of the file); lane i < k receives rank i.
template <typename TL, int NV>
__device__ __noinline__ int choose64(const GateArgs& A, const TL* row, int lane, int lg) {
  const LaneMap L = lane_map(A, lane, lg);
  double c[NV], m = 0.0, z = 1.0;
#pragma unroll
  for (int j = 0; j < NV; ++j) c[j] = j < L.n ? (double)logit_at(row, L.e0 + j) : -INFINITY;
  const bool scored = A.bias != nullptr || A.top2;  // else experts compare by logit alone
  if (scored) {
    if (!A.sigmoid) {
      float mf = -INFINITY;
#pragma unroll
      for (int j = 0; j < NV; ++j) mf = fmaxf(mf, (float)c[j]);
      for (int o = 16; o > 0; o >>= 1) mf = fmaxf(mf, __shfl_xor_sync(0xffffffffu, mf, o));
      m = mf == -INFINITY ? 0.0 : (double)mf;
      z = 0.0;
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      c[j] = exp(A.sigmoid ? -c[j] : c[j] - m);
      if (A.sigmoid)
        c[j] = 1.0 / (1.0 + c[j]);
      else if (j < L.n)
        z += c[j];
    }
    if (!A.sigmoid)
      for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (!A.sigmoid) c[j] = share64(c[j], z);
      if (A.bias && j < L.n) c[j] += (double)A.bias[L.e0 + j];
    }
  }
  bool allowed = true;
  if (A.G > 1) {
    unsigned long long a = 0ull, b = 0ull;  // below every key
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const unsigned long long v = j < L.n ? dkey(c[j]) : 0ull;
      b = max(b, min(a, v));
      a = max(a, v);
    }
    group_top2(a, b, lg);
    const unsigned long long gv = A.top2 ? dkey(dkey_inv(a) + dkey_inv(b)) : a;
    int rank = 0;
    for (int h = 0; h < A.G; ++h) {
      const unsigned long long o = __shfl_sync(0xffffffffu, gv, h * lg);
      rank += o > gv || (o == gv && h < L.group);
    }
    allowed = L.group < A.G && rank < A.topk_groups;
  }
  uint32_t left = allowed ? (L.n >= 32 ? 0xffffffffu : (1u << L.n) - 1u) : 0u;
  int mine = 0;
  for (int i = 0; i < A.k; ++i) {
    unsigned long long best = 0ull;
    int bj = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      // without a bias experts compare by logit
      const unsigned long long v =
          (left >> j) & 1u ? dkey(A.bias ? c[j] : (double)logit_at(row, L.e0 + j)) : 0ull;
      if (v > best) {
        best = v;
        bj = j;
      }
    }
    const unsigned long long top = max64(best);  // every lane takes part
    const uint32_t win = __ballot_sync(0xffffffffu, best != 0ull && best == top);
    const int from = win ? __ffs((int)win) - 1 : 0;
    const int e = __shfl_sync(0xffffffffu, L.e0 + bj, from);
    if (lane == from) left &= ~(1u << bj);
    if (lane == i) mine = e;
  }
  return mine;
}

// Puts the first k + 1 experts (lane i has that of rank i, or -1) in the order of
// their fp64 choice values; lane i < k receives rank i.
template <typename TL, int NV>
__device__ __noinline__ int order64(const GateArgs& A, const TL* row, const LaneMap L, int lane,
                                    int e) {
  double m = 0.0, z = 1.0;
  if (!A.sigmoid) {
    float x[NV], mf = -INFINITY;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      x[j] = j < L.n ? logit_at(row, L.e0 + j) : -INFINITY;
      mf = fmaxf(mf, x[j]);
    }
    for (int o = 16; o > 0; o >>= 1) mf = fmaxf(mf, __shfl_xor_sync(0xffffffffu, mf, o));
    m = mf == -INFINITY ? 0.0 : (double)mf;
    z = 0.0;
#pragma unroll
    for (int j = 0; j < NV; ++j) z += exp((double)x[j] - m);
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
  }
  const bool on = lane <= A.k && e >= 0;
  unsigned long long c = 0ull;
  if (on) {
    const double x = (double)logit_at(row, e);
    c = dkey((A.sigmoid ? 1.0 / (1.0 + exp(-x)) : share64(exp(x - m), z)) + (double)A.bias[e]);
  }
  int rank = 0;  // a place of its own for every expert: keys order NaN too
  for (int j = 0; j <= A.k; ++j) {
    const unsigned long long o = __shfl_sync(0xffffffffu, c, j);
    const int oe = __shfl_sync(0xffffffffu, e, j);
    rank += oe >= 0 && (o > c || (o == c && oe < e));
  }
  int mine = 0;
  for (int j = 0; j <= A.k; ++j) {
    const int r = __shfl_sync(0xffffffffu, on ? rank : -1, j);
    const int oe = __shfl_sync(0xffffffffu, e, j);
    if (r == lane) mine = oe;
  }
  return mine;
}

// SIG: sigmoid scores, else softmax; BIAS: a balance bias is given.
template <typename TL, int NV, bool SIG, bool BIAS>
__global__ void __launch_bounds__(kGateWarps * 32) k_gate_topk(const GateArgs A) {
  __shared__ unsigned long long s_list[kGateWarps][NV][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x * (blockDim.x >> 5) + warp;
  begin_overlapped();
  if (t >= A.T) return;
  const TL* row = static_cast<const TL*>(A.logits) + (size_t)t * A.ld;
  const int lg = A.lanes;  // lanes of a group
  const LaneMap L = lane_map(A, lane, lg);

  float x[NV], bv[NV];
  constexpr int VL = NV < 4 ? 1 : 4;
  if (VL > 1 && A.vec) {  // every lane has NV experts or none: 4 a load
    struct alignas(sizeof(TL) * VL) QL {
      TL e[VL];
    };
#pragma unroll
    for (int j = 0; j < NV; j += VL) {
      if (L.n != 0) {
        const QL v = *reinterpret_cast<const QL*>(row + L.e0 + j);
#pragma unroll
        for (int c = 0; c < VL; ++c) x[j + c] = to_f(v.e[c]);
      } else {
#pragma unroll
        for (int c = 0; c < VL; ++c) x[j + c] = -INFINITY;
      }
#pragma unroll
      for (int c = 0; c < VL; ++c) bv[j + c] = 0.f;
      if (BIAS && L.n != 0) {
        const float4 b4 = *reinterpret_cast<const float4*>(A.bias + L.e0 + j);
        bv[j] = b4.x;
        bv[j + 1 < NV ? j + 1 : j] = b4.y;
        bv[j + 2 < NV ? j + 2 : j] = b4.z;
        bv[j + 3 < NV ? j + 3 : j] = b4.w;
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      x[j] = j < L.n ? to_f(row[L.e0 + j]) : -INFINITY;
      bv[j] = BIAS && j < L.n ? A.bias[L.e0 + j] : 0.f;
    }
  }

  // softmax: maximum, and the sum where scores are asked for
  constexpr float kLog2e = 1.442695041f;
  float m = 0.f, z = 1.f;
  if (!SIG) {
    m = -INFINITY;
#pragma unroll
    for (int j = 0; j < NV; ++j) m = fmaxf(m, x[j]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (m == -INFINITY) m = 0.f;  // nothing left: every score is 0
    z = 0.f;
    if (!A.renorm) {  // weights are scores
#pragma unroll
      for (int j = 0; j < NV; ++j) z += expf(x[j] - m);
      z = warp_sum(z);
    } else if (BIAS || A.top2) {
#pragma unroll
      for (int j = 0; j < NV; ++j) z += exp2_approx((x[j] - m) * kLog2e);
      z = warp_sum(z);
    }
  }
  const float inv_z = z > 0.f ? 1.f / z : 0.f;
  // a score to decide by, and one to weigh by
  auto about = [&](float v) {
    return SIG ? rcp_approx(1.f + exp2_approx(-kLog2e * v))
                     : exp2_approx((v - m) * kLog2e) * inv_z;
  };
  auto score = [&](float v) {
    return SIG ? 1.f / (1.f + expf(-v)) : expf(v - m) * inv_z;
  };

  // keys, sorted largest first within the lane
  uint64_t c[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const float key = BIAS ? about(x[j]) + bv[j] : x[j];
    c[j] = j < L.n ? ((uint64_t)gate_key(key) << 32) | (uint64_t)(~(uint32_t)(L.e0 + j)) : 0ull;
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

  // A NaN logit, or +infinity under softmax, leaves the token's weights undefined.
  // A lane's first key shows whether to look (a NaN may come from the bias alone).
  bool undefined = false;
  if (__any_sync(0xffffffffu, (uint32_t)(c[0] >> 32) >= (SIG || BIAS ? 0xffffffffu : 0xff800000u))) {
    for (int j = 0; j < L.n; ++j) {
      const float v = logit_at(row, L.e0 + j);
      undefined |= v != v || (!SIG && v == INFINITY);
    }
    undefined = __any_sync(0xffffffffu, undefined);
  }

  // Bound on the fp32 error of a score that decides, u = 2^-24:
  //   sigmoid: e^-x has the relative error of its argument's rounding and of
  //   log2 e, 1.22 |x| u, and of ex2.approx, 4 u; s moves by s (1 - s) of that, at
  //   most (0.28 + 1) u; 1 + e 1 u, rcp.approx 2 u: 4.3 u
  //   softmax, in units of the largest score 1 / z: the exponent d = m - x 2.22 d u
  //   and ex2.approx 4 u, of e^-d: 4.9 u; z the same, weighted (d is 6.3 on average
  //   at most), and its 36 additions: 54 u; 1 / z and the product 2 u: 61 u
  // A choice value adds the rounding of the bias, u |c|, a group's sum that of two
  // values and its own.  Two values that differ by less than twice the bound, with a
  // quarter to spare, are compared in fp64.
  const float err = SIG ? 3.8e-7f : 4.6e-6f * inv_z;
  bool near = false;

  if (A.G > 1) {
    uint32_t a = (uint32_t)(c[0] >> 32), b = NV > 1 ? (uint32_t)(c[NV > 1 ? 1 : 0] >> 32) : 0u;
    if (!BIAS && A.top2) {  // the keys are logits
      a = a != 0u ? gate_key(about(fkey_inv(a))) : 0u;
      b = b != 0u ? gate_key(about(fkey_inv(b))) : 0u;
    }
    group_top2(a, b, lg);
    uint32_t gk = a;  // a group's lanes agree on it; 0 beyond the last group
    float mag = fabsf(fkey_inv(a));
    if (A.top2) {  // then a group has two experts at least
      mag += fabsf(fkey_inv(b));
      gk = a != 0u ? gate_key(fkey_inv(a) + fkey_inv(b)) : 0u;
    }
    mag = mag == mag ? mag : 0.f;  // a NaN group is above all others, whatever they are
    int rank = 0;
    for (int h = 0; h < A.G; ++h) {
      const uint32_t o = __shfl_sync(0xffffffffu, gk, h * lg);
      rank += o > gk || (o == gk && h < L.group);
    }
    const bool allowed = L.group < A.G && rank < A.topk_groups;
    if (BIAS || A.top2) {
      // the last group inside against the first outside
      const uint32_t last = __reduce_min_sync(0xffffffffu, allowed ? gk : 0xffffffffu);
      const uint32_t next = __reduce_max_sync(0xffffffffu, !allowed && L.group < A.G ? gk : 0u);
      const float top = __uint_as_float(
          __reduce_max_sync(0xffffffffu, L.group < A.G ? __float_as_uint(mag) : 0u));
      // (a difference of two infinities, fp32 sums that overflowed, counts as near)
      near = next != 0u &&
             !(fkey_inv(last) - fkey_inv(next) > 2.f * (2.f * err + 1.5e-7f * top));
    }
    if (!allowed) c[0] = 0ull;
  }

  // k rounds; with a bias two more, for the border behind k
#pragma unroll
  for (int j = 1; j < NV; ++j) s_list[warp][j][lane] = c[j];
  uint64_t head = c[0];
  int at = head != 0ull ? 0 : NV, my_e = 0;
  uint32_t my_k = 0u;
  const int rounds = A.k + (BIAS ? 2 : 0);
  for (int i = 0; i < rounds; ++i) {
    const uint32_t hk = (uint32_t)(head >> 32);
    const uint32_t mk = __reduce_max_sync(0xffffffffu, hk);
    // equal keys: the lower lane has the lower experts
    const int from = __ffs((int)__ballot_sync(0xffffffffu, hk == mk)) - 1;
    const uint32_t ne = __shfl_sync(0xffffffffu, (uint32_t)head, from);
    if (lane == from) {  // its next expert (only this lane's own column is read)
      ++at;
      head = at < NV ? s_list[warp][at < NV ? at : 0][lane] : 0ull;
    }
    if (lane == i) {
      my_e = mk != 0u ? (int)~ne : -1;
      my_k = mk;
    }
  }
  float my_x = -INFINITY;
  bool close = false;  // experts in question, none beyond the first k + 1
  if (BIAS) {
    float my_b = 0.f;
    if (lane < rounds && my_e >= 0) {
      my_x = logit_at(row, my_e);
      my_b = A.bias[my_e];
    }
    const float v = fkey_inv(my_k);
    const uint32_t nk = __shfl_down_sync(0xffffffffu, my_k, 1);
    const float nx = __shfl_down_sync(0xffffffffu, my_x, 1);
    const float nb = __shfl_down_sync(0xffffffffu, my_b, 1);
    const float nvv = fkey_inv(nk);
    const bool next = lane <= A.k && nk != 0u;
    const bool same = next && nx == my_x && nb == my_b;  // a true tie: the index decides
    const bool touch = next && !same &&
                       v - nvv <= 2.f * (err + 7.5e-8f * fmaxf(fabsf(v), fabsf(nvv)));
    // ranks i and i + 1 that touch; the first k + 1 experts settle it among themselves
    // unless equal or touching ones lead on behind them
    close = (__ballot_sync(0xffffffffu, touch) & ((1u << A.k) - 1u)) != 0u;
    near |= ((__ballot_sync(0xffffffffu, touch || same) >> (A.k - 1)) & 3u) == 3u;
  }
  const bool all64 = __any_sync(0xffffffffu, near);
  if (all64)
    my_e = choose64<TL, NV>(A, row, lane, lg);
  else if (close)
    my_e = order64<TL, NV>(A, row, L, lane, my_e);

  // weights
  const bool on = lane < A.k;
  my_e = max(my_e, 0);  // lanes behind the experts that were found
  if (on) my_x = logit_at(row, my_e);
  float w = 0.f;
  if (A.renorm) {
    // relative to the largest chosen logit, so that no sum underflows
    float top = on ? my_x : -INFINITY;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (top != -INFINITY && on) {
      if (!SIG) {
        w = expf(my_x - top);
      } else {  // s = e^x / (1 + e^x); below 0 in units of e^min(top, 0)
        w = my_x > 0.f ? 1.f / (1.f + expf(-my_x))
                       : expf(my_x - fminf(top, 0.f)) / (1.f + expf(my_x));
      }
    }
    float sum = w;  // the k <= 16 chosen lie on the first 16 lanes
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    w = sum > 0.f ? w / sum : 0.f;
  } else if (on) {
    w = score(my_x);
  }
  w = undefined ? __uint_as_float(0x7fffffffu) : w * A.scale;
  if (on) {
    const size_t o = (size_t)t * A.k + lane;
    A.idx[o] = my_e;
    A.weight[o] = w;
  }
  if (A.keep != nullptr) {
    // the token's largest weight (ties: the earlier slot) is always kept
    const uint32_t wk = on ? gate_key(w) : 0u;
    const uint32_t lead = __reduce_max_sync(0xffffffffu, wk);
    const int lead_lane = __ffs((int)__ballot_sync(0xffffffffu, on && wk == lead)) - 1;
    if (on)
      A.keep[(size_t)t * A.k + lane] =
          lane == lead_lane || !(w * (A.factor ? A.factor[my_e] : 1.f) < A.tau);
  }
}

bool is_aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

template <typename TL, int NV>
cudaError_t launch_nv(const GateArgs& A, cudaStream_t s) {
  const int warps = A.T < kGateWarps ? A.T : kGateWarps;
  const unsigned grid = (unsigned)cdiv(A.T, warps), block = 32u * warps;
  if (A.sigmoid)
    return A.bias ? launch_overlapped(k_gate_topk<TL, NV, true, true>, grid, block, 1, 0, s, A)
                  : launch_overlapped(k_gate_topk<TL, NV, true, false>, grid, block, 1, 0, s, A);
  return A.bias ? launch_overlapped(k_gate_topk<TL, NV, false, true>, grid, block, 1, 0, s, A)
                : launch_overlapped(k_gate_topk<TL, NV, false, false>, grid, block, 1, 0, s, A);
}

template <typename TL>
cudaError_t launch_gate(const GateArgs& A, cudaStream_t s) {
  const int n = cdiv(A.E / A.G, A.lanes);
  if (n <= 1) return launch_nv<TL, 1>(A, s);
  if (n <= 2) return launch_nv<TL, 2>(A, s);
  if (n <= 4) return launch_nv<TL, 4>(A, s);
  if (n <= 8) return launch_nv<TL, 8>(A, s);
  if (n <= 16) return launch_nv<TL, 16>(A, s);
  return launch_nv<TL, 32>(A, s);
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
  if (E > kMaxE || T > kMaxCount) return ACE_ERR_UNSUPPORTED;
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
  const ByteSpan in[3] = {ByteSpan(logits, ld, T, E, es), ByteSpan(bias, 1, E, 1, 4),
                          ByteSpan(factor, 1, E, 1, 4)};
  const ByteSpan out[3] = {ByteSpan(idx, k, T, k, 4), ByteSpan(weight, k, T, k, 4),
                           ByteSpan(keep, k, T, k, 1)};
  for (int o = 0; o < 3; ++o) {
    for (const ByteSpan& i : in)
      if (out[o].meets(i)) return ACE_ERR_INVALID_ARG;
    for (int p = 0; p < o; ++p)
      if (out[o].meets(out[p])) return ACE_ERR_INVALID_ARG;
  }
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
  A.top2 = A.G > 1 && E > A.G && opts->group_score == ACE_GROUP_TOP2;  // of one expert: its own
  A.renorm = opts->renorm_topk != 0;
  int gp = 1;
  while (gp < A.G) gp <<= 1;
  A.lanes = 32 / gp;
  // 4 logits a load where every lane in use holds the same number of experts, the
  // template's NV (a power of two), and every address allows it
  const int per = E / A.G, n = cdiv(per, A.lanes);
  A.vec = per % n == 0 && n >= 4 && (n & (n - 1)) == 0 && ld % 4 == 0 &&
          is_aligned(logits, 4 * es) && (!bias || is_aligned(bias, 16));
  A.scale = opts->scale;
  A.tau = opts->tau;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return cuda_status(dtype == ACE_BF16 ? launch_gate<__nv_bfloat16>(A, s) : launch_gate<float>(A, s));
}

}  // extern "C"

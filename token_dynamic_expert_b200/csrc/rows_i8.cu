// rows_i8.cu -- the two row operators around the 8-bit experts: the residual
// addition + RMSNorm in front of the layer and the SwiGLU between the two
// products, each with an int8 output and one scale per row.
//
//   norm    s = round(x + residual);  r = 1 / sqrt(mean s^2 + eps);
//           y = s r gamma;  int8 of p = s gamma (r cancels), unit r
//   swiglu  h = g / (1 + e^-g) * u;  int8 of p = h, unit 1
//   int8    M = max_j |p_j|;  q_i = round-half-even(127 p_i / M);
//           scale = M unit / 127, so q_i scale stands for p_i unit
//
// One pass over the data: a row's elements stay in registers between the
// statistics and the outputs.  Both kernels are bound by HBM for many rows and
// by latency (launch, one load, two barriers) for few.
//
// Rounding of q.  127 p / M is formed in fp32 with a relative error of at most
// kRel (counted below), which misplaces about one element in 10^4 next to a
// half.  Elements whose interval q (1 -+ kRel) straddles a half are settled in
// fp64 from the stored inputs, with M in fp64 too, so q is the correctly
// rounded quotient; about one row in eight (d = 2048) has such an element.
#include <math.h>

#include "ace_common.cuh"
#include "ace_internal.h"

namespace ace {
namespace {

constexpr int kMaxRow = 16384;        // elements per row
constexpr float kTinyMax = 7.9e-31f;  // 2^-100: below it 127 / M may overflow, fp64 decides

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  T e[V];
};

// Bits of |p|: as unsigned integers they order like the values, NaN above
// infinity, so one integer maximum finds the largest and keeps a NaN.
__device__ __forceinline__ uint32_t abs_bits(float p) { return __float_as_uint(p) & 0x7fffffffu; }

__device__ __forceinline__ double silu64(double g) { return g / (1.0 + exp(-g)); }

struct RowArgs {
  const void* a;    // x, or gate|up rows
  const void* b;    // residual or NULL
  void* sum;        // norm: s rows or NULL
  void* y;          // unquantised rows or NULL
  int8_t* q;        // int8 rows or NULL
  float* q_scale;   // [rows] (with q)
  const float* gamma;
  const int32_t* n_valid;  // swiglu: rows in use, or NULL (all)
  int64_t lda, ldb, lds, ldy, ldq;
  int rows, d;
  float eps;
};

// Relative error of v = p * (127 / M) in units of 2^-24.
//   norm:   p 1 rounding, M 1, 127 / M 1, the product 1; + 2 for forming the interval   -> 8
//   swiglu: h: expf 2 ulp (4 half steps), 1 + e, the division, the product (3) = 7;
//           M 7; quotient 1, product 1; interval 2                                    -> 20
template <bool SWIGLU>
__device__ __forceinline__ constexpr float rel_bound() {
  return (SWIGLU ? 20.f : 8.f) * 5.9604645e-8f;
}

template <typename T, int V, int ITEMS, bool SWIGLU>
__global__ void __launch_bounds__(1024) k_rows_i8(const RowArgs A) {
  __shared__ float s_ss[32];
  __shared__ uint32_t s_mx[32];
  __shared__ unsigned long long s_top;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
  const int64_t row = blockIdx.x;
  if (SWIGLU && A.n_valid != nullptr && row >= *A.n_valid) return;  // uniform over the CTA
  const T* a = static_cast<const T*>(A.a) + row * A.lda;
  const T* b = A.b ? static_cast<const T*>(A.b) + row * A.ldb : nullptr;
  const int d = A.d, nv = d / V;
  if (tid == 0) s_top = 0ull;

  float v[ITEMS][V];  // norm: s; swiglu: h
  float p[ITEMS][V];  // norm: s gamma; swiglu: unused (h)
  float ss = 0.f;
  uint32_t mx = 0u;
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int at = i * blockDim.x + tid;
    if (at >= nv) {
#pragma unroll
      for (int c = 0; c < V; ++c) v[i][c] = p[i][c] = 0.f;
      continue;
    }
    const Vec<T, V> va = reinterpret_cast<const Vec<T, V>*>(a)[at];
    if constexpr (SWIGLU) {
      const Vec<T, V> vu = reinterpret_cast<const Vec<T, V>*>(a + d)[at];
#pragma unroll
      for (int c = 0; c < V; ++c) {
        const float g = to_f(va.e[c]);
        v[i][c] = __fdiv_rn(g, 1.f + expf(-g)) * to_f(vu.e[c]);
        mx = max(mx, abs_bits(v[i][c]));
      }
    } else {
      if (b != nullptr) {
        const Vec<T, V> vb = reinterpret_cast<const Vec<T, V>*>(b)[at];
        Vec<T, V> vs;
#pragma unroll
        for (int c = 0; c < V; ++c) {
          vs.e[c] = from_f<T>(to_f(va.e[c]) + to_f(vb.e[c]));
          v[i][c] = to_f(vs.e[c]);
        }
        if (A.sum) reinterpret_cast<Vec<T, V>*>(static_cast<T*>(A.sum) + row * A.lds)[at] = vs;
      } else {
#pragma unroll
        for (int c = 0; c < V; ++c) v[i][c] = to_f(va.e[c]);
        if (A.sum) reinterpret_cast<Vec<T, V>*>(static_cast<T*>(A.sum) + row * A.lds)[at] = va;
      }
      const Vec<float, V> g = reinterpret_cast<const Vec<float, V>*>(A.gamma)[at];
#pragma unroll
      for (int c = 0; c < V; ++c) {
        ss = fmaf(v[i][c], v[i][c], ss);
        p[i][c] = v[i][c] * g.e[c];
        mx = max(mx, abs_bits(p[i][c]));
      }
    }
  }
  mx = __reduce_max_sync(0xffffffffu, mx);
  if (!SWIGLU) ss = warp_sum(ss);
  if (lane == 0) {
    s_mx[warp] = mx;
    if (!SWIGLU) s_ss[warp] = ss;
  }
  __syncthreads();
  mx = __reduce_max_sync(0xffffffffu, lane < nw ? s_mx[lane] : 0u);
  float r = 1.f;
  if (!SWIGLU) {
    ss = warp_sum(lane < nw ? s_ss[lane] : 0.f);
    r = 1.0f / sqrtf(ss / (float)d + A.eps);
  }
  const float M = __uint_as_float(mx);

  if (A.y != nullptr) {
    Vec<T, V>* y = reinterpret_cast<Vec<T, V>*>(static_cast<T*>(A.y) + row * A.ldy);
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int at = i * blockDim.x + tid;
      if (at >= nv) continue;
      Vec<T, V> o;
      if constexpr (SWIGLU) {
#pragma unroll
        for (int c = 0; c < V; ++c) o.e[c] = from_f<T>(v[i][c]);
      } else {
        const Vec<float, V> g = reinterpret_cast<const Vec<float, V>*>(A.gamma)[at];
#pragma unroll
        for (int c = 0; c < V; ++c) o.e[c] = from_f<T>(xhat(v[i][c], r, g.e[c]));
      }
      y[at] = o;
    }
  }
  if (A.q == nullptr) return;

  Vec<int8_t, V>* q = reinterpret_cast<Vec<int8_t, V>*>(A.q + row * A.ldq);
  const bool finite = isfinite(M) && (SWIGLU || isfinite(ss));
  if (!finite || M < 1.17549435e-38f) {  // uniform: no element to scale by
    Vec<int8_t, V> z;
#pragma unroll
    for (int c = 0; c < V; ++c) z.e[c] = 0;
    for (int at = tid; at < nv; at += blockDim.x) q[at] = z;
    if (tid == 0) A.q_scale[row] = finite ? 0.f : __uint_as_float(0x7fc00000u);
    return;
  }
  constexpr float kRel = rel_bound<SWIGLU>();
  const bool tiny = M < kTinyMax;
  const float inv = tiny ? 0.f : __fdiv_rn(127.f, M);
  bool near = tiny;
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int at = i * blockDim.x + tid;
    if (at >= nv) continue;
    Vec<int8_t, V> o;
#pragma unroll
    for (int c = 0; c < V; ++c) {
      const float t = (SWIGLU ? v[i][c] : p[i][c]) * inv;
      const int lo = __float2int_rn(t * (1.f - kRel)), hi = __float2int_rn(t * (1.f + kRel));
      near |= lo != hi;
      o.e[c] = (int8_t)lo;
    }
    q[at] = o;
  }
  if (tid == 0) A.q_scale[row] = M * r / 127.f;
  if (!__syncthreads_or(near)) return;

  // fp64: first M, from the elements that fp32 cannot tell from the largest
  const float cand = M * (1.f - 4.f * kRel);
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int at = i * blockDim.x + tid;
    if (at >= nv) continue;
#pragma unroll
    for (int c = 0; c < V; ++c) {
      if (!(fabsf(SWIGLU ? v[i][c] : p[i][c]) >= cand)) continue;
      double w;
      if constexpr (SWIGLU)
        w = silu64((double)to_f(a[at * V + c])) * (double)to_f(a[d + at * V + c]);
      else
        w = (double)v[i][c] * (double)A.gamma[at * V + c];
      atomicMax(&s_top, (unsigned long long)__double_as_longlong(fabs(w)));
    }
  }
  __syncthreads();
  const double top = __longlong_as_double((long long)s_top);
  if (!near) return;
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int at = i * blockDim.x + tid;
    if (at >= nv) continue;
#pragma unroll
    for (int c = 0; c < V; ++c) {
      const float t = (SWIGLU ? v[i][c] : p[i][c]) * inv;
      if (!tiny && __float2int_rn(t * (1.f - kRel)) == __float2int_rn(t * (1.f + kRel))) continue;
      double w;
      if constexpr (SWIGLU)
        w = silu64((double)to_f(a[at * V + c])) * (double)to_f(a[d + at * V + c]);
      else
        w = (double)v[i][c] * (double)A.gamma[at * V + c];
      A.q[row * A.ldq + at * V + c] = (int8_t)__double2int_rn(w * 127.0 / top);
    }
  }
}

template <typename T, int V, bool SWIGLU>
cudaError_t launch_v(const RowArgs& A, cudaStream_t s) {
  const int nv = cdiv(A.d, V);
  // about 256 threads a row; rows beyond that size take more threads, then
  // more vectors a thread
  int items = 1;
  while (cdiv(nv, items) > 1024) items *= 2;
  const int threads = cdiv(cdiv(nv, items), 32) * 32;
  const dim3 grid((unsigned)A.rows);
  if (items == 1)
    k_rows_i8<T, V, 1, SWIGLU><<<grid, threads, 0, s>>>(A);
  else if (items == 2)
    k_rows_i8<T, V, 2, SWIGLU><<<grid, threads, 0, s>>>(A);
  else if constexpr (V <= 4) {
    if (items == 4) {
      k_rows_i8<T, V, 4, SWIGLU><<<grid, threads, 0, s>>>(A);
    } else if constexpr (V <= 2) {
      if (items == 8)
        k_rows_i8<T, V, 8, SWIGLU><<<grid, threads, 0, s>>>(A);
      else if constexpr (V == 1)
        k_rows_i8<T, V, 16, SWIGLU><<<grid, threads, 0, s>>>(A);
    }
  }
  return cudaGetLastError();
}

// Whether every row can be moved in vectors of v elements.
bool rows_allow(const RowArgs& A, size_t es, int v) {
  auto ok = [&](const void* p, int64_t ld, size_t e) {
    return p == nullptr || ((reinterpret_cast<uintptr_t>(p) % (e * v)) == 0 && ld % v == 0);
  };
  return A.d % v == 0 && ok(A.a, A.lda, es) && ok(A.b, A.ldb, es) && ok(A.sum, A.lds, es) &&
         ok(A.y, A.ldy, es) && ok(A.q, A.ldq, 1) &&
         reinterpret_cast<uintptr_t>(A.gamma) % (v >= 4 ? 16 : 4 * v) == 0;
}

template <bool SWIGLU>
cudaError_t launch_rows(const RowArgs& A, ace_dtype dt, cudaStream_t s) {
  // vectors of 16 bytes, else of two bf16 elements, else single elements
  if (dt == ACE_BF16) {
    if (rows_allow(A, 2, 8)) return launch_v<__nv_bfloat16, 8, SWIGLU>(A, s);
    if (rows_allow(A, 2, 2)) return launch_v<__nv_bfloat16, 2, SWIGLU>(A, s);
    return launch_v<__nv_bfloat16, 1, SWIGLU>(A, s);
  }
  if (rows_allow(A, 4, 4)) return launch_v<float, 4, SWIGLU>(A, s);
  return launch_v<float, 1, SWIGLU>(A, s);
}

bool is_aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace
}  // namespace ace

using namespace ace;

extern "C" {

ace_status ace_add_rmsnorm(const void* x, int64_t ldx, const void* residual, int64_t ldr, int T,
                           int d, ace_dtype dtype, const float* gamma, float eps, void* sum,
                           int64_t lds, void* y, int64_t ldy, int8_t* q, int64_t ldq,
                           float* q_scale, void* stream) {
  if (dtype != ACE_BF16 && dtype != ACE_F32) return ACE_ERR_INVALID_ARG;
  if (T < 0 || d < 1 || !(eps >= 0.f)) return ACE_ERR_INVALID_ARG;
  if (d > kMaxRow) return ACE_ERR_UNSUPPORTED;
  if (T == 0) return ACE_OK;
  if ((!sum && !y && !q) || (q && !q_scale)) return ACE_ERR_INVALID_ARG;
  const size_t es = dtype == ACE_BF16 ? 2 : 4;
  if (!x || !gamma || !is_aligned(x, es) || !is_aligned(residual, es) || !is_aligned(sum, es) ||
      !is_aligned(y, es) || !is_aligned(gamma, 4) || !is_aligned(q_scale, 4))
    return ACE_ERR_INVALID_ARG;
  if (ldx < d || (residual && ldr < d) || (sum && lds < d) || (y && ldy < d) || (q && ldq < d))
    return ACE_ERR_INVALID_ARG;
  // an output may be an input (same pointer, same stride); nothing else overlaps
  const ByteSpan in[2] = {ByteSpan(x, ldx, T, d, es), ByteSpan(residual, ldr, T, d, es)};
  const int64_t in_ld[2] = {ldx, ldr};
  const ByteSpan out[4] = {ByteSpan(sum, lds, T, d, es), ByteSpan(y, ldy, T, d, es), ByteSpan(q, ldq, T, d, 1),
                       ByteSpan(q ? q_scale : nullptr, 1, T, 1, 4)};
  const int64_t out_ld[4] = {lds, ldy, -1, -1};
  for (int o = 0; o < 4; ++o) {
    for (int i = 0; i < 2; ++i)
      if (out[o].meets(in[i]) && !(o < 2 && out[o].lo == in[i].lo && out_ld[o] == in_ld[i]))
        return ACE_ERR_INVALID_ARG;
    for (int p = 0; p < o; ++p)
      if (out[o].meets(out[p])) return ACE_ERR_INVALID_ARG;
    if (out[o].meets(ByteSpan(gamma, d, 1, d, 4))) return ACE_ERR_INVALID_ARG;
  }
  RowArgs A = {x, residual, sum, y, q, q_scale, gamma, nullptr, ldx, ldr, lds, ldy, ldq, T, d, eps};
  return cuda_status(launch_rows<false>(A, dtype, static_cast<cudaStream_t>(stream)));
}

ace_status ace_swiglu(const void* gu, int64_t ldgu, int S, int m, ace_dtype dtype,
                      const int32_t* n_valid, void* y, int64_t ldy, int8_t* q, int64_t ldq,
                      float* q_scale, void* stream) {
  if (dtype != ACE_BF16 && dtype != ACE_F32) return ACE_ERR_INVALID_ARG;
  if (S < 0 || m < 1) return ACE_ERR_INVALID_ARG;
  if (m > kMaxRow) return ACE_ERR_UNSUPPORTED;
  if (S == 0) return ACE_OK;
  if ((!y && !q) || (q && !q_scale)) return ACE_ERR_INVALID_ARG;
  const size_t es = dtype == ACE_BF16 ? 2 : 4;
  if (!gu || !is_aligned(gu, es) || !is_aligned(y, es) || !is_aligned(q_scale, 4) ||
      !is_aligned(n_valid, 4))
    return ACE_ERR_INVALID_ARG;
  if (ldgu < 2 * (int64_t)m || (y && ldy < m) || (q && ldq < m)) return ACE_ERR_INVALID_ARG;
  const ByteSpan in(gu, ldgu, S, 2 * (int64_t)m, es), cnt(n_valid, 1, n_valid ? 1 : 0, 1, 4);
  const ByteSpan out[3] = {ByteSpan(y, ldy, S, m, es), ByteSpan(q, ldq, S, m, 1),
                       ByteSpan(q ? q_scale : nullptr, 1, S, 1, 4)};
  for (int o = 0; o < 3; ++o) {
    if (out[o].meets(in) || out[o].meets(cnt)) return ACE_ERR_INVALID_ARG;
    for (int p = 0; p < o; ++p)
      if (out[o].meets(out[p])) return ACE_ERR_INVALID_ARG;
  }
  RowArgs A = {gu, nullptr, nullptr, y, q, q_scale, nullptr, n_valid, ldgu, 0, 0, ldy, ldq, S, m, 0.f};
  return cuda_status(launch_rows<true>(A, dtype, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

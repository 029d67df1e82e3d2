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
// statistics and the outputs.  Few rows are bound by latency (launch, one load, two
// barriers: 2.0 us for one row of 2048); many by HBM and, just before it, by
// instruction issue (norm of 8191 rows of 2048 with residual, y and int8 28.7 us, 5.3
// TB/s; SwiGLU of 65536 rows of 512 36 us, 4.7 TB/s).
//
// Rounding of q.  127 p / M is formed in fp32 with a relative error of at most
// kRel (counted below), which misplaces about one element in 50000 next to a
// half.  Elements whose interval q (1 -+ kRel) straddles a half are settled in
// fp64 from the stored inputs, with M in fp64 too, so q is the correctly
// rounded quotient; about one norm row of 2048 in thirty has such an element.
#include <math.h>
#include <string.h>

#include "ace_common.cuh"
#include "ace_internal.h"
#include "launch.cuh"

namespace ace {
namespace {

constexpr int kRowWarps = 4;          // rows of a CTA, where a warp holds one
constexpr int kMaxRow = 16384;        // elements per row
constexpr float kMinMax = 1.17549435e-38f;  // 2^-126: below it q = 0
constexpr float kTinyMax = 7.9e-31f;  // 2^-100: below it 127 / M may overflow
constexpr float kHugeMax = 8.5e37f;   // 2^126: above it the fast quotient is 0

// A sum of squares that fp32 does not hold.  Above kHugeSum it has overflowed.  Below
// kTinySum the squares of elements under 2^-63 have lost bits: 16384 roundings of
// 2^-150 at most, 2^-36 of kTinySum, and nothing to an eps from kSmallEps on.
constexpr float kHugeSum = 3.4e38f;
constexpr float kTinySum = 7.9e-31f;   // 2^-100
constexpr float kSmallEps = 8.1e-28f;  // 2^-90

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  T e[V];
};

// Two fp32 values in a register pair.  Blackwell's f32x2 instructions work on
// both at once, which halves the arithmetic of SwiGLU's exponential (41 against 45
// us at 65536 rows of 512 when it came); the norm's few operations lost more to
// pairing registers than they gained.
typedef unsigned long long F2;
__device__ __forceinline__ F2 two(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ F2 two(float a) { return two(a, a); }
__device__ __forceinline__ float first(F2 a) {
  return __uint_as_float((uint32_t)a);
}
__device__ __forceinline__ float second(F2 a) {
  return __uint_as_float((uint32_t)(a >> 32));
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Elements of a vector as fp32, and back with one rounding: bf16 by one shift
// or mask an element and one conversion a pair.
template <typename T, int V>
__device__ __forceinline__ void unpack(const Vec<T, V>& a, float (&f)[V]) {
  if constexpr (sizeof(T) == 2 && V % 2 == 0) {
    uint32_t w[V / 2];
    memcpy(w, &a, sizeof(w));
#pragma unroll
    for (int c = 0; c < V / 2; ++c) {
      f[2 * c] = __uint_as_float(w[c] << 16);
      f[2 * c + 1] = __uint_as_float(w[c] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int c = 0; c < V; ++c) f[c] = to_f(a.e[c]);
  }
}

template <typename T, int V>
__device__ __forceinline__ Vec<T, V> pack(const float (&f)[V]) {
  Vec<T, V> a;
  if constexpr (sizeof(T) == 2 && V % 2 == 0) {
    uint32_t w[V / 2];
#pragma unroll
    for (int c = 0; c < V / 2; ++c)
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[c]) : "f"(f[2 * c + 1]), "f"(f[2 * c]));
    memcpy(&a, w, sizeof(w));
  } else {
#pragma unroll
    for (int c = 0; c < V; ++c) a.e[c] = from_f<T>(f[c]);
  }
  return a;
}

// The low bytes of V words.
template <int V>
__device__ __forceinline__ Vec<int8_t, V> low_bytes(const uint32_t (&w)[V]) {
  Vec<int8_t, V> o;
  if constexpr (V % 4 == 0) {
    uint32_t b[V / 4];
#pragma unroll
    for (int c = 0; c < V / 4; ++c)
      b[c] = __byte_perm(__byte_perm(w[4 * c], w[4 * c + 1], 0x0040),
                         __byte_perm(w[4 * c + 2], w[4 * c + 3], 0x0040), 0x5410);
    memcpy(&o, b, sizeof(b));
  } else {
#pragma unroll
    for (int c = 0; c < V; ++c) o.e[c] = (int8_t)(w[c] & 0xffu);
  }
  return o;
}

// silu(g) u of a pair.  e^-g = 2^y with y = -g log2 e: the product's rounding
// and the constant's are formed exactly enough (r) and put back as a factor
// 1 + r ln 2, since 2^(y + r) = 2^y (1 + r ln 2 + ...) and |r| < 2^-16 where e^-g is
// neither 0 nor infinite.
// Relative error in half steps: ex2.approx 4, the factor 1 and its product 1,
// 1 + e 1, rcp.approx 2, the two products 2: 11.  Above g = 128 e^-g is far
// below half a step of 1.  Below g = -126 ln 2 the reciprocal underflows: rows with
// a g under kSiluLow are formed again in fp64 (low_row).
constexpr float kSiluLow = -87.f;
__device__ __forceinline__ F2 silu_mul(F2 g, F2 u) {
  const F2 n = two(fmaxf(-first(g), -128.f), fmaxf(-second(g), -128.f));
  const F2 y = mul2(n, two(-1.442695041f));  // -y
  F2 r = fma2(n, two(1.442695041f), y);
  r = fma2(n, two(1.925963033e-8f), r);  // log2 e = 1.44269502162933... + 1.92596e-8
  float e0, e1, s0, s1;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e0) : "f"(-first(y)));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e1) : "f"(-second(y)));
  const F2 d = fma2(two(e0, e1), fma2(r, two(0.693147181f), two(1.f)), two(1.f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s0) : "f"(first(d)));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s1) : "f"(second(d)));
  return mul2(mul2(g, two(s0, s1)), u);
}

// a / b within 2 ulp, for b below 2^126.
__device__ __forceinline__ float quotient(float a, float b) {
  float r;
  asm("div.approx.ftz.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// max(m, |a|, |b|) that keeps a NaN of any (m is not negative).
__device__ __forceinline__ float max_abs(float m, float a, float b) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(a), "f"(b));
  return r;
}
template <int V>
__device__ __forceinline__ float max_abs(float m, const float (&p)[V]) {
#pragma unroll
  for (int c = 0; c < V; c += 2) m = max_abs(m, p[c], c + 1 < V ? p[c + 1] : 0.f);
  return m;
}

// The same in fp64 (-infinity counts as its limit, 0); and the nearest integer of
// 127 w / top.  Calls, not inlined: rare, and large in registers.
__device__ __noinline__ double silu_mul64(float g, float u) {
  return (g == -INFINITY ? -0.0 : (double)g / (1.0 + exp(-(double)g))) * (double)u;
}
__device__ __noinline__ int quotient64(double w, double top) {
  return __double2int_rn(w * 127.0 / top);
}

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
  bool overlap;  // launched with programmatic stream serialisation
};

// Relative error of p (127 / M) in units of 2^-24, and so half the width of the
// interval that has to hold no half.
//   norm:   p 1 rounding, M 1, 127 / M 1, its widening by the interval 1        -> 6
//   swiglu: h 11 (silu_mul; 1 + e is formed with the factor's product, 1 less);
//           M 11; 127 / M 2 ulp (4), widening 1                                 -> 28
template <bool SWIGLU>
__device__ __forceinline__ constexpr float rel_bound() {
  return (SWIGLU ? 28.f : 6.f) * 5.9604645e-8f;
}

// 1.5 x 2^23: fmaf(p, inv, kMagic) rounds p inv to the nearest integer (ties to
// even) in one step, and its low byte is that integer in two's complement.
constexpr float kMagic = 12582912.f;

// An element's p in fp64, from the stored inputs.
template <typename T>
__device__ __forceinline__ double exact_p(const T* a, const float* gamma, float s, int d, int i,
                                          bool swiglu) {
  return swiglu ? silu_mul64(to_f(a[i]), to_f(a[d + i])) : (double)s * (double)gamma[i];
}

// gamma's V elements of vector `at` (16-byte loads from 4 elements on).
template <int V>
__device__ __forceinline__ void load_gamma(const float* gamma, int at, float (&g)[V]) {
  constexpr int W = V < 4 ? V : 4;
#pragma unroll
  for (int h = 0; h < V / W; ++h) {
    const Vec<float, W> q = reinterpret_cast<const Vec<float, W>*>(gamma)[at * (V / W) + h];
#pragma unroll
    for (int c = 0; c < W; ++c) g[h * W + c] = q.e[c];
  }
}

// y and q_scale of a row (norm) whose sum of squares fp32 does not hold: sum and r in
// fp64, which holds the squares of fp32 values of any size.  q_scale comes with M in it.
// s is read again (each thread its own elements, so y may be in place): a call at the
// kernel's end with nothing but its arguments alive leaves the kernel its registers.
// Forms that kept s or M for it took 8 more, a block less on an SM (4000 rows of 4096:
// 26.5 us without any of this, 28.6 with those, 26.8 with this).
template <typename T, int V, bool ONE>
__device__ __noinline__ void far_row(const RowArgs& A) {
  __shared__ double s_sum[32];
  const int lane = threadIdx.x & 31, tid = ONE ? lane : threadIdx.x;
  const int64_t row =
      ONE ? (int64_t)blockIdx.x * kRowWarps + (threadIdx.x >> 5) : (int64_t)blockIdx.x;
  const int step = ONE ? 32 : blockDim.x;
  const T* x = static_cast<const T*>(A.sum ? A.sum : A.a) + row * (A.sum ? A.lds : A.lda);
  const T* b = A.sum || !A.b ? nullptr : static_cast<const T*>(A.b) + row * A.ldb;
  auto s_at = [&](int j) { return b ? to_f(from_f<T>(to_f(x[j]) + to_f(b[j]))) : to_f(x[j]); };
  double sum = 0.0;
#pragma unroll 1
  for (int at = tid * V; at < A.d; at += step * V)
#pragma unroll 1
    for (int j = at; j < at + V; ++j) sum += (double)s_at(j) * (double)s_at(j);
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (!ONE) {
    if (lane == 0) s_sum[threadIdx.x >> 5] = sum;
    __syncthreads();
    sum = 0.0;
#pragma unroll 1
    for (int w = 0; w < step / 32; ++w) sum += s_sum[w];
  }
  const double r = 1.0 / sqrt(sum / A.d + (double)A.eps);
  if (A.y != nullptr)
#pragma unroll 1
    for (int at = tid * V; at < A.d; at += step * V)
#pragma unroll 1
      for (int j = at; j < at + V; ++j)
        static_cast<T*>(A.y)[row * A.ldy + j] =
            from_f<T>(__fmul_rn((float)((double)s_at(j) * r), A.gamma[j]));
  if (A.q != nullptr && tid == 0) {
    const float M = A.q_scale[row];  // 0 and NaN stay
    if (M > 0.f) A.q_scale[row] = (float)((double)M * r / 127.0);
  }
}

// A row (swiglu) with a gate so far below zero that fp32 loses SiLU(g): all of its
// outputs once more in fp64, each thread its own elements.  The other rows pay for
// the smallest gate of a thread (65536 rows of 512: 35.2 -> 35.9 us; a thread that
// formed such elements again on the way took 43.6).
template <typename T, int V, bool ONE>
__device__ __noinline__ void low_row(const RowArgs& A) {
  __shared__ double s_max[32];
  const int lane = threadIdx.x & 31, tid = ONE ? lane : threadIdx.x;
  const int step = ONE ? 32 : blockDim.x;
  const int64_t row =
      ONE ? (int64_t)blockIdx.x * kRowWarps + (threadIdx.x >> 5) : (int64_t)blockIdx.x;
  const T* g = static_cast<const T*>(A.a) + row * A.lda;
  auto larger = [](double a, double b) { return b <= a || a != a ? a : b; };  // NaN stays
  double top = 0.0;
#pragma unroll 1
  for (int at = tid * V; at < A.d; at += step * V)
#pragma unroll 1
    for (int j = at; j < at + V; ++j) {
      const double h = silu_mul64(to_f(g[j]), to_f(g[A.d + j]));
      if (A.y != nullptr) static_cast<T*>(A.y)[row * A.ldy + j] = from_f<T>((float)h);
      top = larger(top, fabs(h));
    }
  for (int o = 16; o > 0; o >>= 1) top = larger(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (!ONE) {
    if (lane == 0) s_max[threadIdx.x >> 5] = top;
    __syncthreads();
#pragma unroll 1
    for (int w = 0; w < step / 32; ++w) top = larger(top, s_max[w]);
  }
  if (A.q == nullptr) return;
  const float M = (float)top;
  const bool usable = isfinite(M) && M >= kMinMax;
#pragma unroll 1
  for (int at = tid * V; at < A.d; at += step * V)
#pragma unroll 1
    for (int j = at; j < at + V; ++j)
      A.q[row * A.ldq + j] =
          usable ? (int8_t)quotient64(silu_mul64(to_f(g[j]), to_f(g[A.d + j])), top) : (int8_t)0;
  if (tid == 0)
    A.q_scale[row] = usable        ? (float)(top / 127.0)
                     : isfinite(M) ? 0.f
                                   : __uint_as_float(0x7fc00000u);
}

// ONE: a warp a row and kRowWarps rows a CTA, no barrier; else a CTA a row.
// far_args: A once more, for far_row and low_row, which take its address (with A's own
// address taken the norm of 21845 rows of 768 took 36.7 us instead of 30.5).
template <typename T, int V, int ITEMS, bool SWIGLU, bool ONE>
__global__ void __launch_bounds__(ONE ? 32 * kRowWarps : 1024, 1)
    k_rows_i8(const RowArgs A, const __grid_constant__ RowArgs far_args) {
  constexpr float kRel = rel_bound<SWIGLU>();
  __shared__ float s_ss[32];
  __shared__ uint32_t s_mx[32];
  __shared__ unsigned long long s_tops[ONE ? kRowWarps : 1];  // fp64 maxima, as bits
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tid = ONE ? lane : threadIdx.x;
  const int nt = ONE ? 32 : blockDim.x, nw = nt >> 5;
  const int64_t row = ONE ? (int64_t)blockIdx.x * kRowWarps + warp : blockIdx.x;
  unsigned long long& s_top = s_tops[ONE ? warp : 0];
  if (ONE && row >= A.rows) return;
  if (A.overlap) begin_overlapped();
  if (SWIGLU && A.n_valid != nullptr && row >= *A.n_valid) return;  // uniform over the row
  const T* a = static_cast<const T*>(A.a) + row * A.lda;
  const int d = A.d, nv = d / V;
  const T* b = SWIGLU ? a + d : A.b ? static_cast<const T*>(A.b) + row * A.ldb : nullptr;
  if (tid == 0) s_top = 0ull;

  // every load of the row is in flight before the first is used
  Vec<T, V> va[ITEMS], vb[ITEMS] = {};
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int at = i * nt + tid;
    if (at < nv) {
      va[i] = reinterpret_cast<const Vec<T, V>*>(a)[at];
      if (SWIGLU || b != nullptr) vb[i] = reinterpret_cast<const Vec<T, V>*>(b)[at];
    }
  }
  float v[ITEMS][V];  // norm: s; swiglu: h
  float ss = 0.f, mx = 0.f, low = 0.f;
#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int at = i * nt + tid;
    if (at >= nv) continue;
    float w[V];
    unpack(va[i], v[i]);
    unpack(vb[i], w);
    if constexpr (SWIGLU) {
#pragma unroll
      for (int c = 0; c < V; c += 2) {
        const bool pair = c + 1 < V;
        low = fminf(low, fminf(v[i][c], pair ? v[i][c + 1] : 0.f));
        const F2 h = silu_mul(two(v[i][c], pair ? v[i][c + 1] : 0.f), two(w[c], pair ? w[c + 1] : 0.f));
        v[i][c] = first(h);
        if (pair) v[i][c + 1] = second(h);
      }
      mx = max_abs(mx, v[i]);
    } else {
      if (b != nullptr) {
#pragma unroll
        for (int c = 0; c < V; ++c) v[i][c] += w[c];
        va[i] = pack<T, V>(v[i]);
        unpack(va[i], v[i]);
      }
      if (A.sum) reinterpret_cast<Vec<T, V>*>(static_cast<T*>(A.sum) + row * A.lds)[at] = va[i];
      float g[V], p[V];
      load_gamma<V>(A.gamma, at, g);
#pragma unroll
      for (int c = 0; c < V; ++c) {
        ss = fmaf(v[i][c], v[i][c], ss);
        p[c] = v[i][c] * g[c];
      }
      mx = max_abs(mx, p);
    }
  }
  // the bits of non-negative floats order like the values, NaN above infinity
  uint32_t mb = __reduce_max_sync(0xffffffffu, __float_as_uint(mx) & 0x7fffffffu);
  if (!SWIGLU) ss = warp_sum(ss);
  if (!ONE) {
    if (lane == 0) {
      s_mx[warp] = mb;
      if (!SWIGLU) s_ss[warp] = ss;
    }
    __syncthreads();
    mb = __reduce_max_sync(0xffffffffu, lane < nw ? s_mx[lane] : 0u);
    if (!SWIGLU) ss = warp_sum(lane < nw ? s_ss[lane] : 0.f);
  }
  const float r = SWIGLU ? 1.f : 1.0f / sqrtf(ss / (float)d + A.eps);
  const float M = __uint_as_float(mb);
  const bool finite = isfinite(M);  // an element that is not makes M so
  const bool far_ss = !SWIGLU && (ss > kHugeSum || (ss < kTinySum && A.eps < kSmallEps));
  const bool usable = finite && M >= kMinMax;  // else no element to scale by: q = 0
  const bool far = M < kTinyMax || M > kHugeMax;  // 127 / M in fp32 is no use: fp64 decides all
  // (the exact division costs SwiGLU 1 us of 36 at 65536 rows of 512)
  const float inv = !usable || far ? 0.f : SWIGLU ? quotient(127.f, M) : __fdiv_rn(127.f, M);
  const float inv_lo = inv * (1.f - kRel), inv_hi = inv * (1.f + kRel);
  // bit 31: a low gate (the differences of sums with kMagic leave it 0)
  uint32_t differ = (usable && far ? 1u : 0u) | (SWIGLU && low < kSiluLow ? 0x80000000u : 0u);

#pragma unroll
  for (int i = 0; i < ITEMS; ++i) {
    const int at = i * nt + tid;
    if (at >= nv) continue;
    float g[V];
    if (!SWIGLU) load_gamma<V>(A.gamma, at, g);
    if (A.y != nullptr && !far_ss) {
      float o[V];
#pragma unroll
      for (int c = 0; c < V; ++c) o[c] = SWIGLU ? v[i][c] : xhat(v[i][c], r, g[c]);
      reinterpret_cast<Vec<T, V>*>(static_cast<T*>(A.y) + row * A.ldy)[at] = pack<T, V>(o);
    }
    if (A.q != nullptr) {
      uint32_t o[V];
#pragma unroll
      for (int c = 0; c < V; ++c) o[c] = 0u;
      if (usable)  // the same for the whole row
#pragma unroll
        for (int c = 0; c < V; ++c) {
          const float p = SWIGLU ? v[i][c] : v[i][c] * g[c];
          o[c] = __float_as_uint(fmaf(p, inv_lo, kMagic));
          differ |= o[c] ^ __float_as_uint(fmaf(p, inv_hi, kMagic));
        }
      reinterpret_cast<Vec<int8_t, V>*>(A.q + row * A.ldq)[at] = low_bytes<V>(o);
    }
  }
  if (A.q != nullptr && tid == 0)
    A.q_scale[row] = usable ? (far_ss ? M : M * (r * (1.f / 127.f))) : finite ? 0.f : __uint_as_float(0x7fc00000u);
  if ((SWIGLU || A.q != nullptr) &&
      (ONE ? __any_sync(0xffffffffu, differ != 0u) : __syncthreads_or((int)differ) != 0)) {
    if (SWIGLU) {
      const int is_low = (int)(differ >> 31);
      if (ONE ? __any_sync(0xffffffffu, is_low) : __syncthreads_or(is_low) != 0) {
        low_row<T, V, ONE>(far_args);
        return;
      }
      if (A.q == nullptr) return;
    }
    // fp64: first M, from the elements that fp32 cannot tell from the largest
    if (ONE) __syncwarp();  // s_top is 0 for every lane
    const float cand = M * (1.f - 4.f * kRel);
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
      const int at = i * nt + tid;
      if (at >= nv) continue;
#pragma unroll
      for (int c = 0; c < V; ++c) {
        const float p = SWIGLU ? v[i][c] : v[i][c] * A.gamma[at * V + c];
        if (fabsf(p) >= cand)
          atomicMax(&s_top, (unsigned long long)__double_as_longlong(
                                fabs(exact_p(a, A.gamma, v[i][c], d, at * V + c, SWIGLU))));
      }
    }
    if (ONE)
      __syncwarp();
    else
      __syncthreads();
    const double top = __longlong_as_double((long long)s_top);
    if (differ != 0u) {
#pragma unroll
      for (int i = 0; i < ITEMS; ++i) {
        const int at = i * nt + tid;
        if (at >= nv) continue;
#pragma unroll
        for (int c = 0; c < V; ++c) {
          const float p = SWIGLU ? v[i][c] : v[i][c] * A.gamma[at * V + c];
          if (far || fmaf(p, inv_lo, kMagic) != fmaf(p, inv_hi, kMagic))
            A.q[row * A.ldq + at * V + c] =
                (int8_t)quotient64(exact_p(a, A.gamma, v[i][c], d, at * V + c, SWIGLU), top);
        }
      }
    }
  }
  if (far_ss) far_row<T, V, ONE>(far_args);  // the same for the whole row
}

template <typename T, int V, int ITEMS, bool SWIGLU>
cudaError_t launch_cta(const RowArgs& A, cudaStream_t s) {
  const int threads = cdiv(cdiv(cdiv(A.d, V), ITEMS), 32) * 32;
  auto kernel = k_rows_i8<T, V, ITEMS, SWIGLU, false>;
  // Few rows may start while the kernel before ends (3.0 -> 2.7 us for 61 rows of
  // SwiGLU).  With many, a wait in each of the small CTAs costs more than the
  // launch (65536 rows: 51 -> 81 us).
  if (A.overlap) return launch_overlapped(kernel, (unsigned)A.rows, threads, 1, 0, s, A, A);
  kernel<<<(unsigned)A.rows, threads, 0, s>>>(A, A);
  return cudaGetLastError();
}

template <typename T, int V, int ITEMS, bool SWIGLU>
cudaError_t launch_warp(const RowArgs& A, cudaStream_t s) {
  k_rows_i8<T, V, ITEMS, SWIGLU, true>
      <<<(unsigned)cdiv(A.rows, kRowWarps), 32 * kRowWarps, 0, s>>>(A, A);
  return cudaGetLastError();
}

// Vectors per thread, and whether a warp or a CTA holds a row.
//   few rows: one vector, the shortest chain (2.3 us against 2.6 with two, one row
//   of 2048)
//   many rows of up to 128 16-byte vectors: a warp, since the work per row besides
//   its elements would be most of a CTA's (65536 rows of 512, SwiGLU, bf16: 41 ->
//   35 us; 32768 of 1024: 41 -> 36; norm of 21845 rows of 768: 34 -> 30)
//   longer ones: two 16-byte vectors a thread, enough loads in flight and little
//   besides the elements (8191 rows of 2048, norm, bf16: 1, 2, 4, 8 vectors 35, 28,
//   31, 39 us; 16384 rows of 2048, SwiGLU: 1, 2 vectors 43, 33 us)
//   narrower vectors: eight (4000 rows of 2050: 8 and 16 of them 25 and 34 us)
// More where a row needs more than 1024 threads.
template <typename T, int V, bool SWIGLU>
cudaError_t launch_v(const RowArgs& A, cudaStream_t s) {
  const int nv = cdiv(A.d, V);
  if constexpr (V >= 4) {
    if (!A.overlap && nv <= 32) return launch_warp<T, V, 1, SWIGLU>(A, s);
    if (!A.overlap && nv <= 64) return launch_warp<T, V, 2, SWIGLU>(A, s);
    if (!A.overlap && nv <= 128) return launch_warp<T, V, 4, SWIGLU>(A, s);
    const int items = A.overlap ? 1 : 2;
    if (items == 1 && nv <= 1024) return launch_cta<T, V, 1, SWIGLU>(A, s);
    if (nv <= 2048) return launch_cta<T, V, 2, SWIGLU>(A, s);
    if constexpr (V == 4) return launch_cta<T, V, 4, SWIGLU>(A, s);
  } else {
    if (A.overlap && nv <= 1024) return launch_cta<T, V, 1, SWIGLU>(A, s);
    if (nv <= 8192) return launch_cta<T, V, 8, SWIGLU>(A, s);
    if constexpr (V == 1) return launch_cta<T, V, 16, SWIGLU>(A, s);
  }
  return cudaErrorInvalidValue;  // not reached: d <= kMaxRow
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
cudaError_t launch_rows(RowArgs A, ace_dtype dt, cudaStream_t s) {
  A.overlap = A.rows < 2 * device_sm_count();  // few rows
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
  if (d > kMaxRow || T > kMaxCount) return ACE_ERR_UNSUPPORTED;
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
  RowArgs A = {x, residual, sum, y, q, q_scale, gamma, nullptr, ldx, ldr, lds, ldy, ldq, T, d, eps, false};
  return cuda_status(launch_rows<false>(A, dtype, static_cast<cudaStream_t>(stream)));
}

ace_status ace_swiglu(const void* gu, int64_t ldgu, int S, int m, ace_dtype dtype,
                      const int32_t* n_valid, void* y, int64_t ldy, int8_t* q, int64_t ldq,
                      float* q_scale, void* stream) {
  if (dtype != ACE_BF16 && dtype != ACE_F32) return ACE_ERR_INVALID_ARG;
  if (S < 0 || m < 1) return ACE_ERR_INVALID_ARG;
  if (m > kMaxRow || S > kMaxCount) return ACE_ERR_UNSUPPORTED;
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
  RowArgs A = {gu, nullptr, nullptr, y, q, q_scale, nullptr, n_valid, ldgu, 0, 0, ldy, ldq, S, m, 0.f, false};
  return cuda_status(launch_rows<true>(A, dtype, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"

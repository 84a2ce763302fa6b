// Window attention a row (or a key) at a time, by one warp: the definition, from visible keys
// only. The mathematics stands in irs_window.cu.
#pragma once

#include "irs_internal.h"
#include "irs_ptx.cuh"

namespace irs {

namespace {

// Bits [from, to) of a 64-bit word, both clamped to [0, 64].
__device__ __forceinline__ uint64_t bit_range(int from, int to) {
  from = max(from, 0);
  to = min(to, 64);
  if (from >= to) return 0ull;
  return (~0ull >> (64 - (to - from))) << from;
}

__device__ __forceinline__ uint32_t bit_range32(int from, int to) {
  from = max(from, 0);
  to = min(to, 32);
  if (from >= to) return 0u;
  return (~0u >> (32 - (to - from))) << from;
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Lane l of a row holds the element pairs 2l, 2l + 1 of every 64 elements.
template <int N>
__device__ __forceinline__ void load_row(float2 (&r)[N], const __nv_bfloat16* p, int lane) {
#pragma unroll
  for (int i = 0; i < N; ++i) r[i] = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(p + 64 * i + 2 * lane));
}
template <int N>
__device__ __forceinline__ void store_row(const float2 (&r)[N], float f, __nv_bfloat16* p, int lane) {
#pragma unroll
  for (int i = 0; i < N; ++i)
    *reinterpret_cast<__nv_bfloat162*>(p + 64 * i + 2 * lane) = __floats2bfloat162_rn(r[i].x * f, r[i].y * f);
}
template <int N>
__device__ __forceinline__ float dot_row(const float2 (&x)[N], const float2 (&y)[N]) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) s = fmaf(x[i].x, y[i].x, fmaf(x[i].y, y[i].y, s));
  return warp_sum(s);
}
template <int N>
__device__ __forceinline__ void axpy_row(float2 (&acc)[N], float f, const float2 (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    acc[i].x = fmaf(f, x[i].x, acc[i].x);
    acc[i].y = fmaf(f, x[i].y, acc[i].y);
  }
}

__device__ __forceinline__ void check_documents(const WinArgs& a) {
  if (blockIdx.x != 0) return;
  bool bad = threadIdx.x == 0 && (a.cu[0] != 0 || a.cu[a.ndocs] != a.T);
  for (int i = threadIdx.x; i < a.ndocs; i += blockDim.x) bad |= a.cu[i + 1] <= a.cu[i];
  if (bad) record_error(a.err, IRS_DEVERR_CU_SEQLENS);
}

template <int NQ, int NV>
__device__ __noinline__ void fwd_row(const WinArgs& a, int t, int h, int lane) {
  const int g = h / a.G;
  const WinDoc doc = window_doc(a.cu, a.ndocs, a.T, t);
  const int lo = max(doc.start, t - a.window + 1);
  const int early = min(doc.start + a.sinks, lo);
  float2 q[NQ], o[NV];
  load_row<NQ>(q, a.q + (int64_t)t * a.q_st + (int64_t)h * a.q_sh, lane);
#pragma unroll
  for (int i = 0; i < NV; ++i) o[i] = make_float2(0.f, 0.f);
  float m = -INFINITY, l = 0.f;
  // once a weight is NaN, so are the sum and every column: the remaining keys change nothing
  for (int s = doc.start < early ? doc.start : lo; s <= t && l == l; s = s + 1 == early ? lo : s + 1) {
    float2 x[NQ], y[NV];
    load_row<NQ>(x, a.k + (int64_t)s * a.k_st + (int64_t)g * a.k_sh, lane);
    load_row<NV>(y, a.v + (int64_t)s * a.v_st + (int64_t)g * a.v_sh, lane);
    const float sc = dot_row<NQ>(q, x) * a.scale_log2, was = m;
    m = fmaxf(m, sc);
    const float off = m == -INFINITY ? 0.f : m;   // scores of -inf so far: weights of 0
    const float c = ex2_approx(was - off), p = ex2_approx(sc - off);
    l = fmaf(l, c, p);
#pragma unroll
    for (int i = 0; i < NV; ++i) { o[i].x *= c; o[i].y *= c; }
    axpy_row<NV>(o, p, y);
  }
  if (l == 0.f) l = NAN;   // no score above -inf: 0 / 0
  store_row<NV>(o, 1.f / l, a.out + ((int64_t)t * a.Hq + h) * (64 * NV), lane);
  if (a.lse != nullptr && lane == 0) a.lse[(int64_t)t * a.Hq + h] = fmaf(m, kLn2, logf(l));
}

template <int NQ, int NV>
__device__ __noinline__ void dq_row(const WinArgs& a, int t, int h, int lane) {
  const int g = h / a.G;
  const WinDoc doc = window_doc(a.cu, a.ndocs, a.T, t);
  const int lo = max(doc.start, t - a.window + 1);
  const int early = min(doc.start + a.sinks, lo);
  const int64_t row = (int64_t)t * a.Hq + h;
  float2 q[NQ], d[NV], acc[NQ];
  load_row<NQ>(q, a.q + (int64_t)t * a.q_st + (int64_t)h * a.q_sh, lane);
  load_row<NV>(d, a.dout + row * (64 * NV), lane);
#pragma unroll
  for (int i = 0; i < NQ; ++i) acc[i] = make_float2(0.f, 0.f);
  const float l2 = a.lse_in[row] * kLog2e, D = a.delta[row];
  float ds = 0.f;   // once it is NaN, so is every column: the remaining keys change nothing
  for (int s = doc.start < early ? doc.start : lo; s <= t && ds == ds; s = s + 1 == early ? lo : s + 1) {
    float2 x[NQ], y[NV];
    load_row<NQ>(x, a.k + (int64_t)s * a.k_st + (int64_t)g * a.k_sh, lane);
    load_row<NV>(y, a.v + (int64_t)s * a.v_st + (int64_t)g * a.v_sh, lane);
    ds = ex2_approx(fmaf(dot_row<NQ>(q, x), a.scale_log2, -l2)) * (dot_row<NV>(d, y) - D);
    axpy_row<NQ>(acc, ds, x);
  }
  store_row<NQ>(acc, a.scale, a.dq + row * (64 * NQ), lane);
}

// The first query past those that see key s.
__device__ __forceinline__ int key_end(const WinArgs& a, int s) {
  const WinDoc doc = window_doc(a.cu, a.ndocs, a.T, s);
  const int64_t last = (int64_t)s + a.window;
  return s - doc.start < a.sinks || last > doc.end ? doc.end : (int)last;
}

// Sums [dk | dv] of a key over the queries `first`, `first` + `step`, ... of those that see it.
// Once every column is NaN (as with the first weight that is) the rest changes nothing; warps that
// share a key say so in *nan.
template <int NQ, int NV>
__device__ __forceinline__ void dkv_sums(const WinArgs& a, int s, int g, int lane, int first, int step, volatile int* nan,
                                         float2 (&dk)[NQ], float2 (&dv)[NV]) {
  const int end = key_end(a, s);
  float2 k[NQ], v[NV];
  load_row<NQ>(k, a.k + (int64_t)s * a.k_st + (int64_t)g * a.k_sh, lane);
  load_row<NV>(v, a.v + (int64_t)s * a.v_st + (int64_t)g * a.v_sh, lane);
#pragma unroll
  for (int i = 0; i < NQ; ++i) dk[i] = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < NV; ++i) dv[i] = make_float2(0.f, 0.f);
  bool dk_nan = false;
  for (int t = s + first; t < end; t += step) {
    float p = 0.f;
    for (int h = g * a.G; h < (g + 1) * a.G && p == p; ++h) {
      const int64_t row = (int64_t)t * a.Hq + h;
      float2 q[NQ], d[NV];
      load_row<NQ>(q, a.q + (int64_t)t * a.q_st + (int64_t)h * a.q_sh, lane);
      load_row<NV>(d, a.dout + row * (64 * NV), lane);
      p = ex2_approx(fmaf(dot_row<NQ>(q, k), a.scale_log2, -a.lse_in[row] * kLog2e));
      const float ds = p * (dot_row<NV>(d, v) - a.delta[row]);
      axpy_row<NQ>(dk, ds, q);
      axpy_row<NV>(dv, p, d);
      dk_nan |= ds != ds;
    }
    bool over = p != p;
    if (dk_nan && !over) {
      over = true;
#pragma unroll
      for (int i = 0; i < NV; ++i) over &= dv[i].x != dv[i].x && dv[i].y != dv[i].y;
      over = __all_sync(0xffffffffu, over);
    }
    if (over) {
      if (nan != nullptr) *nan = 1;
      return;
    }
    if (nan != nullptr && *nan) return;
  }
}

template <int NQ, int NV>
__device__ __noinline__ void dkv_row(const WinArgs& a, int s, int g, int lane) {
  float2 dk[NQ], dv[NV];
  dkv_sums<NQ, NV>(a, s, g, lane, 0, 1, nullptr, dk, dv);
  const int64_t row = (int64_t)s * a.Hkv + g;
  store_row<NQ>(dk, a.scale, a.dk + row * (64 * NQ), lane);
  store_row<NV>(dv, 1.f, a.dv + row * (64 * NV), lane);
}

}  // namespace

}  // namespace irs

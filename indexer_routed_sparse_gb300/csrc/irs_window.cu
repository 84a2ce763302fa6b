// Attention of packed documents over a sliding window and the documents' first tokens, one
// warp per row.
//
// Mathematics. Query t of document [s_d, e_d) sees the keys
//   s_d <= s < min(s_d + sinks, lo)   and   lo <= s <= t,   lo = max(s_d, t - window + 1)
// Forward: one pass with the running maximum m and sum l of the softmax, in FP32:
//   x_s = scale * q.k_s,  out = sum e^{x_s - m} v_s / l,  lse = m + ln l
// Backward, from the saved out and lse, with D = dout.out:
//   p_s = e^{x_s - lse},  ds_s = scale * p_s (dout.v_s - D)
//   dq = sum_s ds_s k_s;   dk_s = sum_{t,h} ds_s q,   dv_s = sum_{t,h} p_s dout
// A key's gradient is summed by one warp over the queries that see it, in order, so it is the
// same in every run. Only visible keys are read: what a masked row holds does not matter.
#include "irs_internal.h"
#include "irs_ptx.cuh"

namespace irs {

namespace {

constexpr int kWinThreads = 256;
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
__device__ void fwd_row(const WinArgs& a, int t, int h, int lane) {
  const int g = h / a.G;
  const WinDoc doc = window_doc(a.cu, a.ndocs, a.T, t);
  const int lo = max(doc.start, t - a.window + 1);
  const int early = min(doc.start + a.sinks, lo);
  float2 q[NQ], o[NV];
  load_row<NQ>(q, a.q + (int64_t)t * a.q_st + (int64_t)h * a.q_sh, lane);
#pragma unroll
  for (int i = 0; i < NV; ++i) o[i] = make_float2(0.f, 0.f);
  float m = -INFINITY, l = 0.f;
  for (int s = doc.start < early ? doc.start : lo; s <= t; s = s + 1 == early ? lo : s + 1) {
    float2 x[NQ], y[NV];
    load_row<NQ>(x, a.k + (int64_t)s * a.k_st + (int64_t)g * a.k_sh, lane);
    load_row<NV>(y, a.v + (int64_t)s * a.v_st + (int64_t)g * a.v_sh, lane);
    const float sc = dot_row<NQ>(q, x) * a.scale_log2;
    const float mn = fmaxf(m, sc);
    const float c = ex2_approx(m - mn), p = ex2_approx(sc - mn);
    m = mn;
    l = fmaf(l, c, p);
#pragma unroll
    for (int i = 0; i < NV; ++i) { o[i].x *= c; o[i].y *= c; }
    axpy_row<NV>(o, p, y);
  }
  store_row<NV>(o, 1.f / l, a.out + ((int64_t)t * a.Hq + h) * (64 * NV), lane);
  if (a.lse != nullptr && lane == 0) a.lse[(int64_t)t * a.Hq + h] = fmaf(m, kLn2, logf(l));
}

template <int NQ, int NV>
__device__ void dq_row(const WinArgs& a, int t, int h, int lane) {
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
  for (int s = doc.start < early ? doc.start : lo; s <= t; s = s + 1 == early ? lo : s + 1) {
    float2 x[NQ], y[NV];
    load_row<NQ>(x, a.k + (int64_t)s * a.k_st + (int64_t)g * a.k_sh, lane);
    load_row<NV>(y, a.v + (int64_t)s * a.v_st + (int64_t)g * a.v_sh, lane);
    const float p = ex2_approx(fmaf(dot_row<NQ>(q, x), a.scale_log2, -l2));
    axpy_row<NQ>(acc, p * (dot_row<NV>(d, y) - D), x);
  }
  store_row<NQ>(acc, a.scale, a.dq + row * (64 * NQ), lane);
}

template <int NQ, int NV>
__device__ void dkv_row(const WinArgs& a, int s, int g, int lane) {
  const WinDoc doc = window_doc(a.cu, a.ndocs, a.T, s);
  const int64_t last = (int64_t)s + a.window;   // first query past the window
  const int end = s - doc.start < a.sinks || last > doc.end ? doc.end : (int)last;
  float2 k[NQ], v[NV], dk[NQ], dv[NV];
  load_row<NQ>(k, a.k + (int64_t)s * a.k_st + (int64_t)g * a.k_sh, lane);
  load_row<NV>(v, a.v + (int64_t)s * a.v_st + (int64_t)g * a.v_sh, lane);
#pragma unroll
  for (int i = 0; i < NQ; ++i) dk[i] = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < NV; ++i) dv[i] = make_float2(0.f, 0.f);
  for (int t = s; t < end; ++t) {
    for (int h = g * a.G; h < (g + 1) * a.G; ++h) {
      const int64_t row = (int64_t)t * a.Hq + h;
      float2 q[NQ], d[NV];
      load_row<NQ>(q, a.q + (int64_t)t * a.q_st + (int64_t)h * a.q_sh, lane);
      load_row<NV>(d, a.dout + row * (64 * NV), lane);
      const float p = ex2_approx(fmaf(dot_row<NQ>(q, k), a.scale_log2, -a.lse_in[row] * kLog2e));
      const float ds = p * (dot_row<NV>(d, v) - a.delta[row]);
      axpy_row<NQ>(dk, ds, q);
      axpy_row<NV>(dv, p, d);
    }
  }
  const int64_t row = (int64_t)s * a.Hkv + g;
  store_row<NQ>(dk, a.scale, a.dk + row * (64 * NQ), lane);
  store_row<NV>(dv, 1.f, a.dv + row * (64 * NV), lane);
}

// MODE 0: forward rows, 1: dq rows, 2: dk/dv rows, 3: D = dout.out rows.
template <int NQ, int NV, int MODE>
__global__ void __launch_bounds__(kWinThreads) window_rows_kernel(WinArgs a) {
  if (MODE == 0 || MODE == 3) check_documents(a);
  const int lane = threadIdx.x & 31;
  const int H = MODE == 2 ? a.Hkv : a.Hq;
  const int64_t row = (int64_t)blockIdx.x * (kWinThreads / 32) + (threadIdx.x >> 5);
  if (row >= (int64_t)a.T * H) return;
  const int t = (int)(row / H), h = (int)(row % H);
  if constexpr (MODE == 0) fwd_row<NQ, NV>(a, t, h, lane);
  if constexpr (MODE == 1) dq_row<NQ, NV>(a, t, h, lane);
  if constexpr (MODE == 2) dkv_row<NQ, NV>(a, t, h, lane);
  if constexpr (MODE == 3) {
    float2 x[NV], y[NV];
    load_row<NV>(x, a.dout + row * (64 * NV), lane);
    load_row<NV>(y, a.out + row * (64 * NV), lane);
    const float D = dot_row<NV>(x, y);
    if (lane == 0) a.delta[row] = D;
  }
}

template <int NQ, int NV>
cudaError_t launch_rows(const WinArgs& a, int mode, cudaStream_t stream) {
  const int64_t rows = (int64_t)a.T * (mode == 2 ? a.Hkv : a.Hq);
  const unsigned grid = (unsigned)((rows + kWinThreads / 32 - 1) / (kWinThreads / 32));
  switch (mode) {
    case 0: window_rows_kernel<NQ, NV, 0><<<grid, kWinThreads, 0, stream>>>(a); break;
    case 1: window_rows_kernel<NQ, NV, 1><<<grid, kWinThreads, 0, stream>>>(a); break;
    case 2: window_rows_kernel<NQ, NV, 2><<<grid, kWinThreads, 0, stream>>>(a); break;
    default: window_rows_kernel<NQ, NV, 3><<<grid, kWinThreads, 0, stream>>>(a); break;
  }
  return cudaGetLastError();
}

cudaError_t launch_rows_any(const WinArgs& a, int mode, cudaStream_t stream) {
  switch (a.Dqk / 64 * 4 + a.Dv / 64) {
    case 5: return launch_rows<1, 1>(a, mode, stream);
    case 6: return launch_rows<1, 2>(a, mode, stream);
    case 9: return launch_rows<2, 1>(a, mode, stream);
    case 10: return launch_rows<2, 2>(a, mode, stream);
    case 13: return launch_rows<3, 1>(a, mode, stream);
    default: return launch_rows<3, 2>(a, mode, stream);
  }
}

}  // namespace

size_t window_bwd_workspace_bytes(int T, int Hq, int, int, int, int, int, int) {
  return (((size_t)T * Hq * 4 + 255) & ~size_t(255)) + 256;
}

cudaError_t launch_window_fwd(const WinArgs& a, cudaStream_t stream) { return launch_rows_any(a, 0, stream); }

cudaError_t launch_window_bwd(const WinArgs& a, cudaStream_t stream) {
  for (int mode : {3, 1, 2}) {
    const cudaError_t e = launch_rows_any(a, mode, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace irs

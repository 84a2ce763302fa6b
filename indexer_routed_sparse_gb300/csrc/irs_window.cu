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
#include "irs_window_rows.cuh"

namespace irs {

namespace {

constexpr int kWinThreads = 256;

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

cudaError_t launch_window_fwd_rows(const WinArgs& a, cudaStream_t stream) { return launch_rows_any(a, 0, stream); }

cudaError_t launch_window_bwd_rows(const WinArgs& a, cudaStream_t stream) {
  for (int mode : {3, 1, 2}) {
    const cudaError_t e = launch_rows_any(a, mode, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace irs
